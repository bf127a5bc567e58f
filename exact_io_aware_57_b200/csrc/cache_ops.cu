// Rows into a cache (append) and a cache cut down to a budget (evict).  Both
// move whole rows and are bound by memory; neither rounds anything.
//
// Evict.  For one (sequence, KV head) with len slots: when len > keep, the last
// `recent` slots stay and keep - recent of the others, those of the largest
// weight (equal weights: the lowest slot first; NaN counts as -inf); else all
// stay.  Two kernels: one chooses slots, the other gathers their rows.
//   choose  a radix selection over order-preserving 32-bit keys of the weights
//           finds the last weight that stays, then one ordered pass writes the
//           chosen slots ascending; a cluster of up to eight CTAs per (sequence,
//           head) holds the keys in shared memory and adds its counts through
//           distributed shared memory, so the weights are read once (one CTA that
//           read them five times took 97 us for 8 heads of 32768 slots, the
//           cluster takes about 14 us)
//   gather  each block moves a run of destination slots, all heads of a slot
//           together: the writes are contiguous, the reads are one head's row
#include <cooperative_groups.h>

#include <algorithm>

#include "cache.cuh"
#include "kernels.h"

namespace attn {
namespace {

namespace cg = cooperative_groups;

constexpr int kCopyThreads = 256;

// ------------------------------------------------------------------- append
// `lanes` threads (a power of two, a warp at most) share a row, so that one of them
// has up to four chunks of K and of V on their way at once.  The sequence's first block
// looks through its row list before it states the new length: with a row that does not
// exist the sequence keeps its length, and what the others write lies behind its end.
__global__ void __launch_bounds__(kCopyThreads) append_kernel(AppendParams p, int lanes) {
  const int b = blockIdx.y;
  int len, n;
  bool ok = cache_len(p.c, b, kMaxSlots, p.status, len) && row_count(p.row_lens, b, p.max_rows, p.status, n);
  if (ok && len + (long long)n > cache_capacity(p.c)) {
    atomicExch(p.status, ATTN_ERR_INVALID);
    ok = false;
  }
  if (blockIdx.x == 0) {
    bool bad = !ok;
    if (ok && p.rows) {
#pragma unroll 4
      for (int i = threadIdx.x; i < n; i += kCopyThreads)
        bad |= (unsigned)__ldg(p.rows + (long long)b * p.max_rows + i) >= (unsigned)p.n_new;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) p.new_lens[b] = bad ? p.c.lens[b] : len + n;
  }
  const int per = kCopyThreads / lanes, first = threadIdx.x % lanes, chunks = p.row_bytes / 16;
  const long long row = (long long)blockIdx.x * per + threadIdx.x / lanes;
  if (!ok || row >= n) return;
  const int t = p.rows ? __ldg(p.rows + (long long)b * p.max_rows + row) : (int)row;
  if (t < 0 || t >= p.n_new) {
    atomicExch(p.status, ATTN_ERR_INVALID);
    return;
  }
  const long long to = cache_row(p.c, b, len + (int)row, p.status);
  if (to < 0) return;
  const uint4* k = static_cast<const uint4*>(p.k_new) + ((long long)b * p.n_new + t) * chunks;
  const uint4* v = static_cast<const uint4*>(p.v_new) + ((long long)b * p.n_new + t) * chunks;
  uint4* k_to = static_cast<uint4*>(p.c.k) + to * chunks;
  uint4* v_to = static_cast<uint4*>(p.c.v) + to * chunks;
  int c = first;
  for (; c + 3 * lanes < chunks; c += 4 * lanes) {
    uint4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __ldg(k + c + i * lanes);
      y[i] = __ldg(v + c + i * lanes);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k_to[c + i * lanes] = x[i];
      v_to[c + i * lanes] = y[i];
    }
  }
  for (; c < chunks; c += lanes) {
    const uint4 x = __ldg(k + c), y = __ldg(v + c);
    k_to[c] = x;
    v_to[c] = y;
  }
}

// -------------------------------------------------------------------- evict
// Larger weights give larger keys; -0 equals +0, and NaN equals -inf.
ATTN_DEVINL uint32_t order_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Sequence b's slots before and after; false when its length is not acceptable.
ATTN_DEVINL bool evict_lens(const EvictParams& p, int b, int& len, int& n) {
  if (!cache_len(p.src, b, p.cap, p.status, len)) return false;
  n = min(len, p.keep);
  if (n > cache_capacity(p.dst)) {
    atomicExch(p.status, ATTN_ERR_INVALID);
    return false;
  }
  return true;
}

// A cluster of CTAs chooses the slots of one (sequence, KV head), each its own
// contiguous share of them; `kept` and the weights are written by all.
constexpr int kChoose = 512, kChooseWarps = kChoose / 32;
constexpr int kChooseCached = 12288;  // weights of a share kept in shared memory as keys

struct ChooseSmem {
  uint32_t key[kChooseCached];
  int hist[kChooseWarps][256];  // a warp's own: most weights share their first digits
  int sum[2][256];              // the CTA's counts, by turns: read by the whole cluster
  int total[256];               // the cluster's, largest digit first
  int share[2];                 // the CTA's larger keys and ties
  int warp_gt[kChooseWarps], warp_eq[kChooseWarps];
  int before_gt, before_eq, digit, left;
};

__global__ void __launch_bounds__(kChoose) choose_kernel(EvictParams p) {
  extern __shared__ uint8_t smem_raw[];
  ChooseSmem& s = *reinterpret_cast<ChooseSmem*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = cluster.num_blocks(), rank = cluster.block_rank();
  const int u = blockIdx.x / nc, hk = u % p.Hkv, b = u / p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int len, n;
  const bool ok = evict_lens(p, b, len, n);  // the same in the whole cluster
  if (hk == 0 && rank == 0 && tid == 0) p.new_lens[b] = ok ? n : p.src.lens[b];
  int* kept = p.kept + (long long)u * p.keep;
  if (!ok) {
    for (int i = rank * kChoose + tid; i < p.keep; i += nc * kChoose) kept[i] = -1;
    return;
  }
  const float* w = p.weights + (long long)u * p.cap;
  float* w_out = p.weights_out + (long long)u * p.cap;
  const int old = len > p.keep ? len - p.recent : 0;  // slots that compete
  const int H = len > p.keep ? p.keep - p.recent : 0;  // of which this many stay
  if (H > 0) {
    const int size = (old + nc - 1) / nc, j0 = min(old, rank * size), j1 = min(old, j0 + size);
    const bool cached = size <= kChooseCached;
    if (cached)
      for (int j = j0 + tid; j < j1; j += kChoose) s.key[j - j0] = order_key(__ldg(w + j));
    auto key_of = [&](int j) { return cached ? s.key[j - j0] : order_key(__ldg(w + j)); };
    // the H-th largest key, eight bits at a time from the top
    uint32_t prefix = 0;
    int need = H, turn = 0;
    for (int shift = 24; shift >= 0; shift -= 8, turn ^= 1) {
      for (int i = tid; i < kChooseWarps * 256; i += kChoose) (&s.hist[0][0])[i] = 0;
      __syncthreads();
      for (int j = j0 + tid; j < j1; j += kChoose) {
        const uint32_t key = key_of(j);
        if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&s.hist[warp][(key >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid < 256) {
        int x = 0;
#pragma unroll
        for (int i = 0; i < kChooseWarps; ++i) x += s.hist[i][tid];
        s.sum[turn][tid] = x;
      }
      cluster.sync();
      if (tid < 256) {
        int x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = k < nc ? cluster.map_shared_rank(s.sum[turn], k)[tid] : 0;
        s.total[255 - tid] = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
      }
      __syncthreads();
      // sums from the largest digit down, eight per lane of one warp: the digit at
      // which the count reaches `need`
      if (warp == 0) {
        int c[8], mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = s.total[8 * lane + i];
          mine += c[i];
        }
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        int at = upto - mine;  // keys with a larger digit than this lane's first
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (at < need && need <= at + c[i]) {
            s.digit = 255 - (8 * lane + i);
            s.left = need - at;
          }
          at += c[i];
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | s.digit;
      need = s.left;
    }
    // ascending slots with a larger key, and the first `need` with that key: each
    // warp counts a contiguous part of the share, then writes it
    const int part = (j1 - j0 + kChooseWarps - 1) / kChooseWarps;
    const int a = min(j1, j0 + warp * part), e = min(j1, a + part);
    int gt = 0, eq = 0;
    for (int j = a + lane; j < e; j += 32) {
      const uint32_t key = key_of(j);
      gt += key > prefix;
      eq += key == prefix;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      gt += __shfl_xor_sync(0xffffffffu, gt, o);
      eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    if (lane == 0) {
      s.warp_gt[warp] = gt;
      s.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
      int x = 0, y = 0;
      for (int i = 0; i < kChooseWarps; ++i) {
        const int g = s.warp_gt[i], t = s.warp_eq[i];
        s.warp_gt[i] = x;
        s.warp_eq[i] = y;
        x += g;
        y += t;
      }
      s.share[0] = x;
      s.share[1] = y;
    }
    cluster.sync();
    if (tid == 0) {
      int x = 0, y = 0;
      for (int k = 0; k < rank; ++k) {
        const int* other = cluster.map_shared_rank(s.share, k);
        x += other[0];
        y += other[1];
      }
      s.before_gt = x;
      s.before_eq = y;
    }
    __syncthreads();
    int before_gt = s.before_gt + s.warp_gt[warp], before_eq = s.before_eq + s.warp_eq[warp];
    const unsigned below = (1u << lane) - 1;
    for (int j = a; j < e; j += 32) {
      const uint32_t key = j + lane < e ? key_of(j + lane) : 0;
      const bool larger = j + lane < e && key > prefix, tie = j + lane < e && key == prefix;
      const unsigned mg = __ballot_sync(0xffffffffu, larger), me = __ballot_sync(0xffffffffu, tie);
      const int ties = before_eq + __popc(me & below);
      if (larger || (tie && ties < need)) {
        const int pos = before_gt + __popc(mg & below) + min(ties, need);
        kept[pos] = j + lane;
        w_out[pos] = w[j + lane];
      }
      before_gt += __popc(mg);
      before_eq += __popc(me);
    }
  }
  // the slots that stay whatever they weigh, then nothing
  for (int i = H + rank * kChoose + tid; i < p.cap || i < p.keep; i += nc * kChoose) {
    const int j = i < n ? i - H + old : -1;
    if (i < p.keep) kept[i] = j;
    if (i < p.cap) w_out[i] = j >= 0 ? w[j] : 0.f;
  }
  cluster.sync();  // its shared memory is read by the others
}

constexpr int kGatherRows = 64;  // (slot, head) rows per block

__global__ void __launch_bounds__(kCopyThreads) gather_kernel(EvictParams p) {
  __shared__ long long from[kGatherRows], to[kGatherRows];
  const int b = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the slots are chosen
  int len, n;
  if (!evict_lens(p, b, len, n)) return;
  const long long r0 = (long long)blockIdx.x * kGatherRows;  // row = slot * Hkv + head
  const int rows = (int)min((long long)kGatherRows, (long long)n * p.Hkv - r0);
  if (rows <= 0) return;
  if (threadIdx.x < rows) {
    const int slot = (int)((r0 + threadIdx.x) / p.Hkv), hk = (int)((r0 + threadIdx.x) % p.Hkv);
    const int j = p.kept[((long long)b * p.Hkv + hk) * p.keep + slot];
    const long long s = cache_row(p.src, b, j, p.status), d = cache_row(p.dst, b, slot, p.status);
    from[threadIdx.x] = s < 0 ? -1 : s * p.Hkv + hk;
    to[threadIdx.x] = d < 0 ? -1 : d * p.Hkv + hk;
  }
  __syncthreads();
  const int chunks = p.head_bytes / 16;
  for (int i = threadIdx.x; i < rows * chunks; i += kCopyThreads) {
    const int r = i / chunks, c = i % chunks;
    if (from[r] < 0 || to[r] < 0) continue;
    const long long s = from[r] * chunks + c, d = to[r] * chunks + c;
    const uint4 kk = __ldg(static_cast<const uint4*>(p.src.k) + s);
    const uint4 vv = __ldg(static_cast<const uint4*>(p.src.v) + s);
    static_cast<uint4*>(p.dst.k)[d] = kk;
    static_cast<uint4*>(p.dst.v)[d] = vv;
  }
}

}  // namespace

int launch_append(const AppendParams& p, cudaStream_t st) {
  int lanes = 32;
  while (lanes > 1 && lanes / 2 >= p.row_bytes / 16) lanes /= 2;
  const int per = kCopyThreads / lanes;
  append_kernel<<<dim3((unsigned)((p.max_rows + per - 1) / per), (unsigned)p.B), kCopyThreads, 0, st>>>(p, lanes);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int launch_evict(const EvictParams& p, cudaStream_t st) {
  // CTAs per (sequence, head): shares of about 2048 weights, eight at most, and no
  // more than run at one time (three per SM)
  const long long units = (long long)p.B * p.Hkv;
  int nc = 1;
  while (nc < 8 && (long long)nc * 2048 < p.cap && 2 * nc * units <= 3ll * sm_count()) nc *= 2;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * nc));
  cfg.blockDim = dim3(kChoose);
  cfg.dynamicSmemBytes = sizeof(ChooseSmem);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ChooseSmem)) !=
      cudaSuccess)
    return ATTN_ERR_CUDA;
  if (cudaLaunchKernelEx(&cfg, choose_kernel, p) != cudaSuccess) return ATTN_ERR_CUDA;
  const long long rows = (long long)std::min(p.keep, p.cap) * p.Hkv;  // (len <= cap)
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((rows + kGatherRows - 1) / kGatherRows), (unsigned)p.B);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.attrs = attr + 1;
  if (cudaLaunchKernelEx(&cfg, gather_kernel, p) != cudaSuccess) return ATTN_ERR_CUDA;
  count_launch(2);
  return ATTN_OK;
}

}  // namespace attn
