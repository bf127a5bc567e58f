// Rows into a cache (append) and a cache cut down to a budget (evict).  Both
// move whole rows and are bound by memory; neither rounds anything.
//
// Evict.  For one (sequence, KV head) with len slots: when len > keep, the last
// `recent` slots stay and keep - recent of the others, those of the largest
// weight (equal weights: the lowest slot first; NaN counts as -inf); else all
// stay.  Two kernels: one chooses slots, the other gathers their rows.
//   choose  a radix selection over order-preserving 32-bit keys of the weights
//           finds the last weight that stays, then one ordered pass writes the
//           chosen slots ascending
//   gather  each block moves a run of destination slots, all heads of a slot
//           together: the writes are contiguous, the reads are one head's row
#include <algorithm>

#include "cache.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kCopyThreads = 256;

// ------------------------------------------------------------------- append
__global__ void __launch_bounds__(kCopyThreads) append_kernel(AppendParams p) {
  const int b = blockIdx.y;
  int len, n;
  bool ok = cache_len(p.c, b, 1ll << 31, p.status, len) && row_count(p.row_lens, b, p.max_rows, p.status, n);
  if (ok && len + (long long)n > cache_capacity(p.c)) {
    atomicExch(p.status, ATTN_ERR_INVALID);
    ok = false;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.new_lens[b] = ok ? len + n : p.c.lens[b];
  if (!ok) return;
  const int chunks = p.row_bytes / 16;
  const long long total = (long long)n * chunks;
  for (long long i = (long long)blockIdx.x * kCopyThreads + threadIdx.x; i < total;
       i += (long long)gridDim.x * kCopyThreads) {
    const int row = (int)(i / chunks), c = (int)(i % chunks);
    const int t = p.rows ? __ldg(p.rows + (long long)b * p.max_rows + row) : row;
    if (t < 0 || t >= p.n_new) {
      atomicExch(p.status, ATTN_ERR_INVALID);
      continue;
    }
    const long long to = cache_row(p.c, b, len + row, p.status);
    if (to < 0) continue;
    const long long src = ((long long)b * p.n_new + t) * chunks + c, dst = to * chunks + c;
    const uint4 kk = __ldg(static_cast<const uint4*>(p.k_new) + src);
    const uint4 vv = __ldg(static_cast<const uint4*>(p.v_new) + src);
    static_cast<uint4*>(p.c.k)[dst] = kk;
    static_cast<uint4*>(p.c.v)[dst] = vv;
  }
}

// -------------------------------------------------------------------- evict
// Larger weights give larger keys; -0 equals +0, and NaN equals -inf.
ATTN_DEVINL uint32_t order_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

constexpr int kChoose = 1024;

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

__global__ void __launch_bounds__(kChoose) choose_kernel(EvictParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sum[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int hk = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  int len, n;
  const bool ok = evict_lens(p, b, len, n);
  if (hk == 0 && tid == 0) p.new_lens[b] = ok ? n : p.src.lens[b];
  const long long u = (long long)b * p.Hkv + hk;
  int* kept = p.kept + u * p.keep;
  if (!ok) {
    for (int i = tid; i < p.keep; i += kChoose) kept[i] = -1;
    return;
  }
  const float* w = p.weights + u * p.cap;
  float* w_out = p.weights_out + u * p.cap;
  const int old = len > p.keep ? len - p.recent : 0;  // slots that compete
  const int H = len > p.keep ? p.keep - p.recent : 0;  // of which this many stay
  // the H-th largest key, eight bits at a time from the top
  uint32_t prefix = 0;
  int need = H;
  for (int shift = 24; H > 0 && shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kChoose) hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < old; j += kChoose) {
      const uint32_t key = order_key(w[j]);
      if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int left = need, d = 255;
      while (d > 0 && left > hist[d]) left -= hist[d--];
      s_prefix = (prefix << 8) | d;
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // ascending slots with a larger key, and the first `need` with that key
  int at = 0, ties = 0;  // slots written, ties met so far
  for (int j0 = 0; H > 0 && j0 < old; j0 += kChoose) {
    const int j = j0 + tid;
    const uint32_t key = j < old ? order_key(w[j]) : 0;
    const bool gt = j < old && key > prefix, eq = j < old && key == prefix;
    // running counts of both kinds: larger keys in the low half, ties in the high half
    const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    const int lane = tid & 31, warp = tid >> 5;
    const unsigned below = (1u << lane) - 1;
    if (lane == 0) warp_sum[warp] = __popc(mg) | (__popc(me) << 16);
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < kChoose / 32; ++i) {
      if (i < warp) before += warp_sum[i];
      all += warp_sum[i];
    }
    const int g = (before & 0xffff) + __popc(mg & below), e = ties + (before >> 16) + __popc(me & below);
    if (gt || (eq && e < need)) {
      const int pos = at + g + min(e, need) - min(ties, need);
      kept[pos] = j;
      w_out[pos] = w[j];
    }
    const int ties_after = ties + (all >> 16);
    at += (all & 0xffff) + min(ties_after, need) - min(ties, need);
    ties = ties_after;
    __syncthreads();
  }
  // the slots that stay whatever they weigh, then nothing
  for (int i = H + tid; i < p.cap || i < p.keep; i += kChoose) {
    const int j = i < n ? i - H + old : -1;
    if (i < p.keep) kept[i] = j;
    if (i < p.cap) w_out[i] = j >= 0 ? w[j] : 0.f;
  }
}

constexpr int kGatherRows = 64;  // (slot, head) rows per block

__global__ void __launch_bounds__(kCopyThreads) gather_kernel(EvictParams p) {
  __shared__ long long from[kGatherRows], to[kGatherRows];
  const int b = blockIdx.y;
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
  const long long chunks = (long long)p.max_rows * (p.row_bytes / 16);
  const dim3 grid((unsigned)std::max(1ll, std::min((chunks + kCopyThreads - 1) / kCopyThreads, 1ll << 20)), (unsigned)p.B);
  append_kernel<<<grid, kCopyThreads, 0, st>>>(p);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int launch_evict(const EvictParams& p, cudaStream_t st) {
  choose_kernel<<<dim3((unsigned)p.Hkv, (unsigned)p.B), kChoose, 0, st>>>(p);
  const long long rows = (long long)p.keep * p.Hkv;
  gather_kernel<<<dim3((unsigned)((rows + kGatherRows - 1) / kGatherRows), (unsigned)p.B), kCopyThreads, 0, st>>>(p);
  count_launch(2);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
