// Tree attention and accumulated key weights over a cache on the CUDA cores:
// the fp32 path.
//
// Tree attention.  A block owns 8 query rows (row = (drafted token t, head g of
// the group), one per warp) of one (sequence, KV head) and walks every
// num_splits-th 32-key tile of the cached slots and then of the drafted keys:
// K and V tiles in shared memory, lane = key for the scores, lane = column
// group for P V, the running softmax state (m, l, a) in registers ("Softmax
// does not need the matrix", "Carry the Normalizer").  The splits' partials are
// merged by merge.cu.  Splitting strides over tiles, so that splits of ragged
// sequences stay level without the host knowing a length.  K and V are read again for
// every 8 rows: 8 sequences of 8191 slots, one token of 32 heads on 8, d = 128 take 316
// us (bytes once: 83), 4 of 4000 slots with 61 tokens 1.92 ms (8.4 TFLOP/s).
//
// Key weights.  A block owns 32 slots of one (sequence, KV head): lane = slot,
// the warps share out the counted (row, head) pairs, and their sums are added
// in warp order.
#include <algorithm>

#include "cache.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int KT = 32;    // keys per tile
constexpr int ROWS = 8;   // query rows (warps) per block

ATTN_DEVINL float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

ATTN_DEVINL float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
ATTN_DEVINL float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D>
__global__ void __launch_bounds__(32 * ROWS) tree_f32_kernel(TreeParams p) {
  constexpr int S = D + 4;  // padded row: 16-byte reads of 8 consecutive rows hit distinct banks
  constexpr int E = D / 32;
  __shared__ float ks[KT * S], vs[KT * S], qs[ROWS * D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const int b = blockIdx.z, split = blockIdx.y % p.num_splits, hk = blockIdx.y / p.num_splits;
  const int r = blockIdx.x * ROWS + warp;  // row (t, g) of the group
  const int t = r / G, h = hk * G + r % G;
  int len, nr;
  if (!cache_len(p.c, b, kMaxSlots, p.status, len) || !row_count(p.row_lens, b, p.Nq, p.status, nr)) len = nr = 0;
  const bool valid = t < p.Nq;
  const bool row_ok = t < nr;
  const int n_new = p.k_new ? nr : 0;
  const float* q = static_cast<const float*>(p.q) + (((long long)b * p.Nq + (valid ? t : 0)) * p.Hq + h) * D;
  for (int c = lane; c < D / 4; c += 32)
    *reinterpret_cast<float4*>(&qs[warp * D + 4 * c]) = load4(q + 4 * c);
  const unsigned long long* mrow =
      p.mask && valid ? p.mask + (long long)b * p.mask_bstride + (long long)t * p.mask_words : nullptr;

  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const int tiles_c = (len + KT - 1) / KT, tiles = tiles_c + (n_new + KT - 1) / KT;
  for (int tile = split; tile < tiles; tile += p.num_splits) {
    const bool cached = tile < tiles_c;
    const int base = (cached ? tile : tile - tiles_c) * KT;
    const int n = min(KT, (cached ? len : n_new) - base);
    __syncthreads();
    for (int i = threadIdx.x; i < KT * (D / 4); i += 32 * ROWS) {
      const int key = i / (D / 4), c = 4 * (i % (D / 4));
      float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
      if (key < n) {
        const long long row = cached ? cache_row(p.c, b, base + key, p.status) : (long long)b * p.Nq + base + key;
        if (row >= 0) {
          const long long at = (row * p.Hkv + hk) * D + c;
          kk = load4(static_cast<const float*>(cached ? p.c.k : p.k_new) + at);
          vv = load4(static_cast<const float*>(cached ? p.c.v : p.v_new) + at);
        }
      }
      *reinterpret_cast<float4*>(&ks[key * S + c]) = kk;
      *reinterpret_cast<float4*>(&vs[key * S + c]) = vv;
    }
    __syncthreads();
    if (!row_ok) continue;
    float s = 0.f;
#pragma unroll 8
    for (int c = 0; c < D; c += 4) {
      const float4 a = *reinterpret_cast<const float4*>(&qs[warp * D + c]);
      const float4 k = *reinterpret_cast<const float4*>(&ks[lane * S + c]);
      s = fmaf(a.x, k.x, fmaf(a.y, k.y, fmaf(a.z, k.z, fmaf(a.w, k.w, s))));
    }
    bool see = lane < n;
    if (see && !cached) {
      const int j = base + lane;
      see = mrow ? (mrow[j >> 6] >> (j & 63)) & 1 : j <= t;
    }
    s = see ? s * p.scale : -INFINITY;
    // (a score of NaN leaves m as it is and l at NaN, which the row keeps)
    const float m_new = fmaxf(m, warp_max(s));
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = expf(m - ref), w = see ? expf(s - ref) : 0.f;
    l = l * alpha + warp_sum(w);
    m = m_new;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= alpha;
    // only seen keys enter the sum: a hidden key's V may hold anything
    for (unsigned live = __ballot_sync(0xffffffffu, see); live; live &= live - 1) {
      const int j = __ffs(live) - 1;
      const float wj = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(wj, vs[j * S + lane * E + e], acc[e]);
    }
  }
  if (!valid) return;
  const bool none = l == 0.f;  // sees no key
  const float inv = none ? 0.f : 1.f / l;
  const long long at = (long long)b * p.Nq + t;
  float* o = p.o_part + ((long long)split * p.B * p.Nq + at) * p.Hq * D + (long long)h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = none ? 0.f : acc[e] * inv;
  if (lane == 0)
    p.lse_part[(((long long)split * p.B + b) * p.Hq + h) * p.Nq + t] = none ? -INFINITY : m + logf(l);
}

// Weights.  A block has 32 slots, a lane each; its warps take AT (row, head)s at a
// time.  Four in 16 warps, so that a key read from shared memory serves four dot
// products and four rows' loads are on their way at once: a prompt of 606 tokens of 3
// heads on one KV head takes 195 us, with one at a time in 8 warps 655 (19 blocks then
// walk all counted rows each, and 129 SMs have none).  One in 8 warps
// where these have two rows each at most, as in a decode step, whose time is the
// latency of a row (4 sequences of 800 .. 1000 slots, 16 heads on 8: 10 to 12 us, the
// other way 29).
constexpr int weights_warps(int at) { return at == 1 ? 8 : 16; }

template <int D, int AT>
__global__ void __launch_bounds__(32 * weights_warps(AT)) weights_f32_kernel(WeightsParams p) {
  constexpr int S = D + 4, kWarps = weights_warps(AT);
  __shared__ float ks[KT * S], part[kWarps][KT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, hk = blockIdx.y, b = blockIdx.z, base = blockIdx.x * KT;
  int len, nr;
  if (!cache_len(p.c, b, p.cap, p.status, len) || !row_count(p.row_lens, b, p.max_rows, p.status, nr)) return;
  const int n = min(KT, len - base);  // slots of this tile in use (may be negative)
  for (int i = threadIdx.x; i < KT * (D / 4); i += 32 * kWarps) {
    const int key = i / (D / 4), c = 4 * (i % (D / 4));
    float4 kk = make_float4(0.f, 0.f, 0.f, 0.f);
    if (key < n) {
      const long long row = cache_row(p.c, b, base + key, p.status);
      if (row >= 0) kk = load4(static_cast<const float*>(p.c.k) + (row * p.Hkv + hk) * D + c);
    }
    *reinterpret_cast<float4*>(&ks[key * S + c]) = kk;
  }
  __syncthreads();
  float acc = 0.f;
  if (n > 0) {
    const long long first = (long long)max(0, base - (len - nr)) * G;  // earlier rows see no slot of this tile
    for (long long i0 = first + warp * AT; i0 < (long long)nr * G; i0 += kWarps * AT) {
      const float* q[AT];
      float z[AT], s[AT];
      int last[AT];  // the last slot that the row sees
#pragma unroll
      for (int x = 0; x < AT; ++x) {
        const int row = (int)((i0 + x) / G), h = hk * G + (int)((i0 + x) % G);
        int t = row;
        bool on = row < nr;
        if (on && p.rows) t = p.rows[(long long)b * p.max_rows + row];
        if (on && (t < 0 || t >= p.Nq)) {
          if (lane == 0) atomicExch(p.status, ATTN_ERR_INVALID);
          on = false;
        }
        q[x] = static_cast<const float*>(p.q) + (on ? (((long long)b * p.Nq + t) * p.Hq + h) * D : 0);
        z[x] = on ? p.lse[((long long)b * p.Hq + h) * p.Nq + t] : -INFINITY;
        last[x] = len - nr + row;
        s[x] = 0.f;
      }
#pragma unroll(AT > 1 ? 4 : 16)
      for (int c = 0; c < D; c += 4) {
        const float4 k = *reinterpret_cast<const float4*>(&ks[lane * S + c]);
#pragma unroll
        for (int x = 0; x < AT; ++x) {
          const float4 a = load4(q[x] + c);
          s[x] = fmaf(a.x, k.x, fmaf(a.y, k.y, fmaf(a.z, k.z, fmaf(a.w, k.w, s[x]))));
        }
      }
      // a row without a visible key (LSE = -inf) weighs nothing
#pragma unroll
      for (int x = 0; x < AT; ++x)
        if (lane < n && base + lane <= last[x] && z[x] != -INFINITY) acc += expf(s[x] * p.scale - z[x]);
    }
  }
  part[warp][lane] = acc;
  __syncthreads();
  const int j = base + lane;
  if (warp == 0 && j < p.cap) {
    const long long at = ((long long)b * p.Hkv + hk) * p.cap + j;
    float w = p.weights ? p.weights[at] : 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += part[i][lane];
    if (lane < n) w += sum;
    p.out[at] = w;
  }
}

}  // namespace

// Splits of the keys such that about two blocks land on each SM.
int tree_f32_splits(int B, int Hq, int Hkv, int Nq, long long capacity) {
  const long long blocks = (long long)B * Hkv * (((long long)Nq * (Hq / Hkv) + ROWS - 1) / ROWS);
  const long long tiles = (capacity + Nq + KT - 1) / KT;
  const long long want = std::min((4ll * sm_count() + blocks - 1) / blocks, 65535ll / Hkv);
  return (int)std::max(1ll, std::min(std::min(want, tiles), 64ll));
}

int launch_tree_f32(const TreeParams& p, cudaStream_t st) {
  const int G = p.Hq / p.Hkv;
  const dim3 grid((unsigned)(((long long)p.Nq * G + ROWS - 1) / ROWS), (unsigned)(p.Hkv * p.num_splits), (unsigned)p.B);
  (p.D == 64 ? tree_f32_kernel<64> : tree_f32_kernel<128>)<<<grid, 32 * ROWS, 0, st>>>(p);
  count_launch();
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  return launch_merge(p.o_part, p.lse_part, p.num_splits, p.o, p.lse, p.B, p.Hq, p.Nq, p.D, 1, st);
}

int launch_weights_f32(const WeightsParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.cap + KT - 1) / KT), (unsigned)p.Hkv, (unsigned)p.B);
  const bool few = (long long)p.max_rows * (p.Hq / p.Hkv) <= 2 * weights_warps(1);
  const auto kernel = p.D == 64 ? (few ? weights_f32_kernel<64, 1> : weights_f32_kernel<64, 4>)
                                : (few ? weights_f32_kernel<128, 1> : weights_f32_kernel<128, 4>);
  kernel<<<grid, 32 * weights_warps(few ? 1 : 4), 0, st>>>(p);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
