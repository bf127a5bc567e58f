// C-ABI entry points of the key/value cache (declared in include/attn.h):
// argument validation, workspace carving and dispatch by dtype.
#include <algorithm>
#include <climits>

#include "cache.cuh"
#include "kernels.h"

using namespace attn;

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Most drafted rows per sequence of one tree-attention call.
constexpr int kMaxTreeRows = 4096;

int check_sizes(int batch, int h_q, int h_kv, int d, int dtype) {
  if (batch <= 0 || h_q <= 0 || h_kv <= 0 || h_q % h_kv != 0) return ATTN_ERR_INVALID;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (dtype != ATTN_BF16 && dtype != ATTN_F32) return ATTN_ERR_UNSUPPORTED;
  if (h_q > 65535 || batch > 65535) return ATTN_ERR_UNSUPPORTED;
  if ((long long)batch * h_kv > INT_MAX) return ATTN_ERR_UNSUPPORTED;  // (a block per sequence and KV head)
  return ATTN_OK;
}

// Validates a cache and fills the kernels' view of it.
int check_cache(const attn_kv_cache* c, int batch, bool need_v, bool need_lens, CacheView& v) {
  if (!c || !c->k || (need_v && !c->v) || (need_lens && !c->lens)) return ATTN_ERR_INVALID;
  if (!aligned16(c->k) || !aligned16(c->v)) return ATTN_ERR_INVALID;
  if (!aligned(c->block_table, 4) || !aligned(c->lens, 4)) return ATTN_ERR_INVALID;
  if (c->num_pages <= 0 || c->page_size <= 0) return ATTN_ERR_INVALID;
  if (c->block_table) {
    if (c->max_pages <= 0 || c->page_size % 8 != 0) return ATTN_ERR_INVALID;
  } else if (c->num_pages < batch) {
    return ATTN_ERR_INVALID;
  }
  if (c->page_size > kMaxSeqLen) return ATTN_ERR_UNSUPPORTED;
  v.k = c->k;
  v.v = c->v;
  v.table = c->block_table;
  v.lens = c->lens;
  v.num_pages = c->num_pages;
  v.page_size = c->page_size;
  v.max_pages = c->block_table ? c->max_pages : 1;
  return ATTN_OK;
}

// Slots a sequence of the cache can hold, bounded by the longest sequence taken.
long long capacity_of(const CacheView& v) {
  return std::min((long long)v.max_pages * v.page_size, (long long)kMaxSeqLen);
}

// Elements of the split partials of the fp32 path.
size_t partial_bytes(int splits, int batch, int h_q, int n_q, int d) {
  const size_t rows = (size_t)splits * batch * n_q * h_q;
  return align256(rows * d * sizeof(float)) + align256(rows * sizeof(float));
}

}  // namespace

extern "C" {

int attn_cache_append(const void* k_new, const void* v_new, const attn_kv_cache* cache, const int* rows, int max_rows,
                      const int* row_lens, int* new_lens, int batch, int n_new, int h_kv, int d, int dtype,
                      void* stream) {
  int rc = check_sizes(batch, h_kv, h_kv, d, dtype);
  if (rc) return rc;
  AppendParams p{};
  if ((rc = check_cache(cache, batch, true, true, p.c))) return rc;
  if (!k_new || !v_new || !new_lens || new_lens == cache->lens || n_new <= 0 || max_rows <= 0) return ATTN_ERR_INVALID;
  if (!rows && max_rows > n_new) return ATTN_ERR_INVALID;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned(rows, 4) || !aligned(row_lens, 4) || !aligned(new_lens, 4))
    return ATTN_ERR_INVALID;
  if (n_new > kMaxSeqLen || max_rows > kMaxSeqLen) return ATTN_ERR_UNSUPPORTED;
  if (!supported_device()) return ATTN_ERR_UNSUPPORTED;
  p.k_new = k_new;
  p.v_new = v_new;
  p.rows = rows;
  p.row_lens = row_lens;
  p.max_rows = max_rows;
  p.n_new = n_new;
  p.B = batch;
  p.row_bytes = h_kv * d * (dtype == ATTN_BF16 ? 2 : 4);
  p.new_lens = new_lens;
  if (!(p.status = device_status_ptr())) return ATTN_ERR_CUDA;
  return launch_append(p, static_cast<cudaStream_t>(stream));
}

size_t attn_fwd_tree_workspace_size(int batch, int h_q, int h_kv, int n_q, int d, int dtype) {
  if (check_sizes(batch, h_q, h_kv, d, dtype) || n_q <= 0) return 0;
  if (dtype == ATTN_BF16) return tree_sm100_workspace(h_q, h_kv, n_q, d);
  const int splits = tree_f32_splits(batch, h_q, h_kv, n_q, kMaxSeqLen);
  return partial_bytes(splits, batch, h_q, n_q, d);
}

int attn_fwd_tree(const void* q, const void* k_new, const void* v_new, const attn_kv_cache* cache,
                  const long long* tree_mask, long long mask_batch_stride, const int* row_lens, void* o, float* lse,
                  int batch, int h_q, int h_kv, int n_q, int d, float scale, void* workspace, size_t workspace_bytes,
                  int dtype, void* stream) {
  int rc = check_sizes(batch, h_q, h_kv, d, dtype);
  if (rc) return rc;
  TreeParams p{};
  if ((rc = check_cache(cache, batch, true, true, p.c))) return rc;
  if (!q || !o || !lse || n_q <= 0 || !k_new != !v_new) return ATTN_ERR_INVALID;
  if (n_q > kMaxTreeRows) return ATTN_ERR_UNSUPPORTED;
  p.mask_words = (n_q + 63) / 64;
  if (tree_mask && (!k_new || (mask_batch_stride != 0 && mask_batch_stride < (long long)n_q * p.mask_words)))
    return ATTN_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(o)) return ATTN_ERR_INVALID;
  if (!aligned(tree_mask, 8) || !aligned(row_lens, 4) || !aligned(lse, 4)) return ATTN_ERR_INVALID;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return ATTN_ERR_WORKSPACE;
  if (!supported_device()) return ATTN_ERR_UNSUPPORTED;
  p.q = q;
  p.k_new = k_new;
  p.v_new = v_new;
  p.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  p.mask_bstride = mask_batch_stride;
  p.row_lens = row_lens;
  p.o = o;
  p.lse = lse;
  p.B = batch;
  p.Hq = h_q;
  p.Hkv = h_kv;
  p.Nq = n_q;
  p.D = d;
  p.scale = scale;
  if (!(p.status = device_status_ptr())) return ATTN_ERR_CUDA;
  if (dtype == ATTN_BF16) {
    if (workspace_bytes < tree_sm100_workspace(h_q, h_kv, n_q, d)) return ATTN_ERR_WORKSPACE;
    return launch_tree_sm100(p, workspace, static_cast<cudaStream_t>(stream));
  }
  p.num_splits = tree_f32_splits(batch, h_q, h_kv, n_q, capacity_of(p.c));
  if (workspace_bytes < partial_bytes(p.num_splits, batch, h_q, n_q, d)) return ATTN_ERR_WORKSPACE;
  p.o_part = static_cast<float*>(workspace);
  p.lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                        align256((size_t)p.num_splits * batch * n_q * h_q * d * sizeof(float)));
  return launch_tree_f32(p, static_cast<cudaStream_t>(stream));
}

size_t attn_cache_weights_workspace_size(int batch, int h_q, int h_kv, int d, int dtype) {
  if (check_sizes(batch, h_q, h_kv, d, dtype)) return 0;
  return dtype == ATTN_BF16 ? weights_sm100_workspace() : 256;
}

int attn_cache_weights(const void* q, const float* lse, const attn_kv_cache* cache, const int* rows, int max_rows,
                       const int* row_lens, const float* weights, float* out, int cap, int batch, int h_q, int h_kv,
                       int n_q, int d, float scale, void* workspace, size_t workspace_bytes, int dtype, void* stream) {
  int rc = check_sizes(batch, h_q, h_kv, d, dtype);
  if (rc) return rc;
  WeightsParams p{};
  if ((rc = check_cache(cache, batch, false, true, p.c))) return rc;
  if (!q || !lse || !out || n_q <= 0 || max_rows <= 0 || cap <= 0) return ATTN_ERR_INVALID;
  if (!rows && max_rows > n_q) return ATTN_ERR_INVALID;
  if (!aligned16(q) || !aligned(lse, 4) || !aligned(rows, 4) || !aligned(row_lens, 4) || !aligned(weights, 4) ||
      !aligned(out, 4))
    return ATTN_ERR_INVALID;
  if (n_q > kMaxSeqLen || max_rows > kMaxSeqLen || cap > kMaxSeqLen) return ATTN_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < attn_cache_weights_workspace_size(batch, h_q, h_kv, d, dtype))
    return ATTN_ERR_WORKSPACE;
  if (!supported_device()) return ATTN_ERR_UNSUPPORTED;
  p.q = q;
  p.lse = lse;
  p.rows = rows;
  p.row_lens = row_lens;
  p.max_rows = max_rows;
  p.weights = weights;
  p.out = out;
  p.cap = cap;
  p.B = batch;
  p.Hq = h_q;
  p.Hkv = h_kv;
  p.Nq = n_q;
  p.D = d;
  p.scale = scale;
  if (!(p.status = device_status_ptr())) return ATTN_ERR_CUDA;
  if (dtype == ATTN_BF16) return launch_weights_sm100(p, workspace, static_cast<cudaStream_t>(stream));
  return launch_weights_f32(p, static_cast<cudaStream_t>(stream));
}

int attn_cache_evict(const attn_kv_cache* cache, const float* weights, int cap, int keep, int recent,
                     const attn_kv_cache* dst, float* weights_out, int* kept, int* new_lens, int batch, int h_kv,
                     int d, int dtype, void* stream) {
  int rc = check_sizes(batch, h_kv, h_kv, d, dtype);
  if (rc) return rc;
  EvictParams p{};
  if ((rc = check_cache(cache, batch, true, true, p.src))) return rc;
  if ((rc = check_cache(dst, batch, true, false, p.dst))) return rc;
  if (!weights || !weights_out || weights == weights_out || !kept || !new_lens || new_lens == cache->lens)
    return ATTN_ERR_INVALID;
  if (!aligned(weights, 4) || !aligned(weights_out, 4) || !aligned(kept, 4) || !aligned(new_lens, 4)) return ATTN_ERR_INVALID;
  if (cap <= 0 || keep <= 0 || recent < 0 || recent > keep) return ATTN_ERR_INVALID;
  // Rows move in no order: the source has to stay as it is.  Within one pool that takes
  // other pages of the same size, named by another table.
  if (cache->k == dst->v || cache->v == dst->k) return ATTN_ERR_INVALID;
  if ((cache->k == dst->k || cache->v == dst->v) &&
      (cache->block_table == dst->block_table || cache->page_size != dst->page_size))
    return ATTN_ERR_INVALID;
  if (cap > kMaxSeqLen || keep > kMaxSeqLen) return ATTN_ERR_UNSUPPORTED;
  if (!supported_device()) return ATTN_ERR_UNSUPPORTED;
  p.weights = weights;
  p.weights_out = weights_out;
  p.cap = cap;
  p.keep = keep;
  p.recent = recent;
  p.kept = kept;
  p.new_lens = new_lens;
  p.B = batch;
  p.Hkv = h_kv;
  p.head_bytes = d * (dtype == ATTN_BF16 ? 2 : 4);
  if (!(p.status = device_status_ptr())) return ATTN_ERR_CUDA;
  return launch_evict(p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
