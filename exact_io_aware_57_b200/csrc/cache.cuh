// Key/value cache shared by the cache kernels: where a slot lies and which
// lengths and page numbers are accepted.
#pragma once

#include "common.cuh"

namespace attn {

// A cache of `batch` sequences: slot s of sequence b is row s % page_size of
// page table[b * max_pages + s / page_size], or row s of page b without a table.
struct CacheView {
  void *k, *v;
  const int* table;  // device [batch, max_pages] or null
  const int* lens;   // device [batch]
  int num_pages, page_size, max_pages;  // max_pages 1 without a table
};

// Slots per TMA box: a box never straddles a page (the largest power of two that
// divides it; a table's pages are multiples of 8).
inline int cache_box_rows(const CacheView& c) {
  int box = 128;
  if (c.table)
    while (c.page_size % box) box >>= 1;
  return box;
}

ATTN_DEVINL long long cache_capacity(const CacheView& c) { return (long long)c.max_pages * c.page_size; }

// Slots of sequence b in use; false (and ATTN_ERR_INVALID in the status word)
// for a length that is negative or beyond `most` slots.
ATTN_DEVINL bool cache_len(const CacheView& c, int b, long long most, int* status, int& len) {
  len = c.lens[b];
  if (len < 0 || len > min(most, cache_capacity(c))) {
    atomicExch(status, ATTN_ERR_INVALID);
    return false;
  }
  return true;
}

// Rows of sequence b that count: row_lens[b], or all; false (and
// ATTN_ERR_INVALID) outside [0, most].
ATTN_DEVINL bool row_count(const int* row_lens, int b, int most, int* status, int& n) {
  n = row_lens ? row_lens[b] : most;
  if (n < 0 || n > most) {
    atomicExch(status, ATTN_ERR_INVALID);
    return false;
  }
  return true;
}

// Row of the page pools (a row holds h_kv * d elements) of slot s; -1 (and
// ATTN_ERR_INVALID) when the table names a page outside the pool.
ATTN_DEVINL long long cache_row(const CacheView& c, int b, int s, int* status) {
  if (!c.table) return (long long)b * c.page_size + s;
  const int page = __ldg(c.table + (long long)b * c.max_pages + s / c.page_size);
  if (page < 0 || page >= c.num_pages) {
    atomicExch(status, ATTN_ERR_INVALID);
    return -1;
  }
  return (long long)page * c.page_size + s % c.page_size;
}

// ---- equal runs.  The work of a launch is a line of `total` steps, sequence b
// owning cost(b) of them; CTA c takes the steps [run0, run1), its share when at
// most `total` CTAs take part, and its run begins `off` steps into sequence b.
struct Run {
  long long total, run0, run1, off;
  int ctas, b;
};

template <int THREADS>
struct RunSmem {
  long long sum[THREADS / 32];
  long long off;
  int b;
};

// All THREADS threads of the block take part; the block is synchronised on return.
template <int THREADS, class Cost>
ATTN_DEVINL Run find_run(RunSmem<THREADS>& s, int B, Cost cost) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long mine = 0;
  for (int b = threadIdx.x; b < B; b += THREADS) mine += cost(b);
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s.sum[warp] = mine;
  __syncthreads();
  Run r;
  r.total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) r.total += s.sum[i];
  r.ctas = (int)min((long long)gridDim.x, r.total);
  r.run0 = r.ctas ? min((int)blockIdx.x, r.ctas) * r.total / r.ctas : 0;
  r.run1 = r.ctas ? min((int)blockIdx.x + 1, r.ctas) * r.total / r.ctas : 0;
  r.b = 0;
  r.off = 0;
  if (r.run1 == r.run0) return r;  // uniform
  long long before = 0;
  for (int b0 = 0; b0 < B && before <= r.run0; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    const long long w = b < B ? cost(b) : 0;
    long long x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s.sum[warp] = x;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) x += s.sum[i];
      all += s.sum[i];
    }
    const long long lo = before + x - w;
    if (lo <= r.run0 && r.run0 < lo + w) {
      s.b = b;
      s.off = r.run0 - lo;
    }
    before += all;
  }
  __syncthreads();
  r.b = s.b;
  r.off = s.off;
  return r;
}

// CTAs behind the one whose run ends at run1 that a unit reaches into when it
// still has `rest` steps there.
ATTN_DEVINL int run_parts(const Run& r, long long rest) {
  int c = blockIdx.x + 1;
  while ((c + 1ll) * r.total / r.ctas < r.run1 + rest) ++c;
  return c - (int)blockIdx.x;
}

// Where a lane's box of a 128-key tile of cached slots lies: boxes of box_rows
// slots that never straddle a page, lane = (piece of the tile, 64-element block).
// Looked up a tile ahead of its load, so that no load waits for the page table.
struct TileBox {
  int page, row, live;  // live: boxes of the tile that begin below the length
};

template <int D>
ATTN_DEVINL TileBox find_box(const CacheView& c, int b, int base, int len, int box_rows) {
  const int lane = threadIdx.x & 31;
  TileBox t;
  t.live = min(128 / box_rows, (len - base + box_rows - 1) / box_rows);
  const int piece = lane / (D / 64), slot = base + piece * box_rows;
  t.page = b;
  t.row = slot;
  if (c.table && piece < t.live) {
    t.page = __ldg(c.table + (long long)b * c.max_pages + slot / c.page_size);
    t.row = slot % c.page_size;
  }
  return t;
}

// Load that tile of KV head hk into dst (64-element blocks of 128 rows each), all
// lanes of a warp taking part.  Rows behind its last live box are not written.
template <int D>
ATTN_DEVINL void load_cache_tile(uint8_t* dst, uint64_t* bar, const CUtensorMap* map, const CacheView& c,
                                 const TileBox& t, int hk, int box_rows, int* status) {
  constexpr int KB = D / 64;
  const int lane = threadIdx.x & 31;
  if (lane == 0) mbar_expect_tx(bar, t.live * box_rows * KB * 128);
  __syncwarp();
  const int piece = lane / KB, kb = lane % KB;
  if (piece < t.live) {
    int page = t.page;
    if (page < 0 || page >= c.num_pages) {
      atomicExch(status, ATTN_ERR_INVALID);
      page = c.num_pages;  // outside the tensor: zeros are loaded
    }
    tma_load_4d(dst + kb * 128 * 128 + piece * box_rows * 128, map, bar, kb * 64, hk, t.row, page);
  }
  __syncwarp();
}

}  // namespace attn
