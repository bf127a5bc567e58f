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

constexpr int kMaxSlots = 1 << 28;  // per sequence

ATTN_DEVINL long long cache_capacity(const CacheView& c) {
  return min((long long)kMaxSlots, (long long)c.max_pages * c.page_size);
}

// Slots of sequence b in use; false (and ATTN_ERR_INVALID in the status word)
// for a length that is negative or beyond `most` slots.
ATTN_DEVINL bool cache_len(const CacheView& c, int b, int most, int* status, int& len) {
  len = c.lens[b];
  if (len < 0 || len > min((long long)most, cache_capacity(c))) {
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
// owning cost(b) of them.  It is cut into equal runs, one per worker; a block has
// LANES workers, blockIdx + lane * gridDim, so that with few steps every block
// has its first worker busy.  No more workers take part than have steps: worker w
// then takes the steps [run0, run1), beginning `off` steps into sequence b.
struct Run {
  long long run0, run1, off;
  int b;
};

template <int LANES>
struct Runs {
  long long total;
  int workers;
  Run lane[LANES];
};

template <int THREADS, int LANES>
struct RunSmem {
  long long sum[THREADS / 32];
  Runs<LANES> runs;  // the result
};

ATTN_DEVINL long long run_begin(long long total, int workers, int w) {
  // 32-bit products and quotients where they do
  if (total < (1 << 20) && workers < (1 << 11)) return (unsigned)w * (unsigned)total / (unsigned)workers;
  return w * total / workers;
}

// Leaves the block's runs in s.runs, of `least` steps at least if there are that many.  All THREADS threads of the block take part;
// the block is synchronised on return.
template <int THREADS, int LANES, class Cost>
ATTN_DEVINL void find_runs(RunSmem<THREADS, LANES>& s, int B, int least, Cost cost) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // inclusive sum over the block's threads; all: their total
  auto scan = [&](long long x, long long& all) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s.sum[warp] = x;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) x += s.sum[i];
      all += s.sum[i];
    }
    return x;
  };
  long long w = (int)threadIdx.x < B ? cost(threadIdx.x) : 0, all;
  long long x = scan(w, all);
  long long total = all;
  for (int b0 = THREADS; b0 < B; b0 += THREADS) {
    __syncthreads();
    const int b = b0 + threadIdx.x;
    scan(b < B ? cost(b) : 0, all);
    total += all;
  }
  const int workers = (int)min((long long)gridDim.x * LANES, max(total / least, min(total, 1ll)));
  long long run0[LANES];
#pragma unroll
  for (int l = 0; l < LANES; ++l) {
    const int me = blockIdx.x + l * gridDim.x;
    run0[l] = me < workers ? run_begin(total, workers, me) : -1;
    if (threadIdx.x == 0) s.runs.lane[l] = Run{0, 0, 0, 0};
  }
  __syncthreads();
  auto look = [&](int b, long long lo) {
#pragma unroll
    for (int l = 0; l < LANES; ++l)
      if (lo <= run0[l] && run0[l] < lo + w)
        s.runs.lane[l] = Run{run0[l], run_begin(total, workers, blockIdx.x + l * gridDim.x + 1), run0[l] - lo, b};
  };
  if (B <= THREADS) {
    look(threadIdx.x, x - w);
  } else {
    long long before = 0;
    for (int b0 = 0; b0 < B; b0 += THREADS) {
      __syncthreads();
      const int b = b0 + threadIdx.x;
      w = b < B ? cost(b) : 0;
      x = scan(w, all);
      look(b, before + x - w);
      before += all;
    }
  }
  if (threadIdx.x == 0) {
    s.runs.total = total;
    s.runs.workers = workers;
  }
  __syncthreads();
}

// Workers behind worker w, whose run ends at run1, into which the `rest` steps behind
// it reach.
ATTN_DEVINL int run_parts(long long total, int workers, int w, long long run1, long long rest) {
  int c = w + 1;
  while (run_begin(total, workers, c + 1) < run1 + rest) ++c;
  return c - w;
}

// ---- tiles of 128 slots in shared memory.  Groups of 8 slots, and in a group the
// 64-element blocks of the rows one after the other, 8 lines of 128 bytes each
// (the 128-byte swizzle's unit), so that one TMA box of any multiple of 8 slots
// brings whole rows:
//   slot s, block kb: (s / 8) * group + kb * 1024 + s % 8 * 128,  group = d * 16.
template <int D>
constexpr int kGroupBytes = D * 16;

// A tensor map of rows [.., h_kv, d] as {64, row, block of a row, group, page}:
// coordinates (0, row, hk * d / 64, group, page).  Grouped, a row is one of 8 and
// boxes are any number of slots; else a row is any and groups are not used (rows that
// are no multiple of 8, where a group would pass the last one: boxes of 8; d = 64,
// where groups lie end to end: boxes of any multiple of 8).
struct TileForm {
  int shift;  // log2 of the slots per box
  int grouped;
  int dp, ds;  // 128 slots on: pages, and slots in a page
};

// The place of a lane's box (a lane per box) in a sequence, moved on tile by tile:
// the loading warp's own instructions bound how fast tiles come, and a division by
// the page size would be a third of them.
struct TileCursor {
  int page, slot;
  ATTN_DEVINL void begin(const CacheView& c, const TileForm& f, int base) {
    slot = base + ((threadIdx.x & 31) << f.shift);
    page = c.table ? slot / c.page_size : 0;
    slot -= page * c.page_size;
  }
  ATTN_DEVINL void next(const CacheView& c, const TileForm& f) {
    page += f.dp;
    slot += f.ds;
    if (c.table && slot >= c.page_size) {
      slot -= c.page_size;
      ++page;
    }
  }
};

// A lane's box of a tile.  Looked up a tile ahead of its load, so that no load
// waits for the page table.
struct TileBox {
  int row, group, page, live;  // live: boxes of the tile that begin below the length
};

// left: slots from the tile's first one to the length.
ATTN_DEVINL TileBox find_box(const CacheView& c, const TileForm& f, const TileCursor& at, int b, int left) {
  TileBox t;
  t.live = min(128 >> f.shift, (left + (1 << f.shift) - 1) >> f.shift);
  t.page = b;
  if (c.table)
    t.page = ldg_if(c.table + (long long)b * c.max_pages + at.page, (int)(threadIdx.x & 31) < t.live, 0);
  t.row = f.grouped ? 0 : at.slot;
  t.group = f.grouped ? at.slot >> 3 : 0;
  return t;
}

// Load the tile of KV head hk into dst, all lanes of a warp taking part.  Slots
// behind the last live box are not written.
template <int D>
ATTN_DEVINL void load_tile(uint8_t* dst, uint64_t* bar, const CUtensorMap* map, const TileForm& f, const TileBox& t,
                           int hk, int pages, int* status) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) mbar_expect_tx(bar, (t.live << f.shift) * D * 2);
  __syncwarp();
  if (lane < t.live) {
    int page = t.page;
    if (page < 0 || page >= pages) {
      atomicExch(status, ATTN_ERR_INVALID);
      page = pages;  // outside the tensor: zeros are loaded
    }
    tma_load_5d(dst + (lane << f.shift) * (D * 2), map, bar, 0, t.row, hk * (D / 64), t.group, page);
  }
  __syncwarp();
}

// Zero slot r of a tile.
template <int D>
ATTN_DEVINL void zero_slot(uint8_t* tile, int r) {
#pragma unroll
  for (int kb = 0; kb < D / 64; ++kb)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint4*>(tile + (r >> 3) * kGroupBytes<D> + kb * 1024 + (r & 7) * 128 + i * 16) =
          make_uint4(0, 0, 0, 0);
}

// Descriptors of a tile for the tensor cores: as rows of K (16 elements of a row
// per instruction), and as rows of V (16 slots per instruction; with d = 64 every
// further block of columns is the first again).
template <int D>
ATTN_DEVINL uint64_t k_tile_desc(const uint8_t* tile) {
  return sdesc_sw128(smem_u32(tile), 16, kGroupBytes<D>);
}
ATTN_DEVINL uint64_t k_tile_step(uint64_t desc, int kk) { return sdesc_at(desc, (kk >> 2) * 1024 + (kk & 3) * 32); }
template <int D>
ATTN_DEVINL uint64_t v_tile_desc(const uint8_t* tile) {
  return sdesc_sw128(smem_u32(tile), D > 64 ? 1024 : 0, kGroupBytes<D>);
}
template <int D>
ATTN_DEVINL uint64_t v_tile_step(uint64_t desc, int kk) {
  return sdesc_at(desc, kk * 2 * kGroupBytes<D>);
}

}  // namespace attn
