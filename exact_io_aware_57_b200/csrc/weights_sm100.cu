// Attention weight received by each cached slot, on sm_100a tensor cores (bf16):
//   out[b, hk, j] = weights[b, hk, j] + sum_(i, g) exp(scale q_(i, g) . k_j - LSE_(i, g))
// over the counted rows i that see j and the heads g of the group.
//
// The scores are formed transposed, S^T = K Q^T: the 128 keys of a tile are the
// TMEM lanes and the query rows the columns, so that a thread owns one key, its
// sum stays in a register, and nothing is reduced across threads.  With the LSE
// at hand there is no running maximum: each score costs one FMA, one
// exponential and one addition.  A decode step has few rows and is bound by
// reading K (32 sequences of 1000 .. 8191 slots, 8 KV heads: 73 us for 330 MB).  A
// prompt's largest share is the exponentials (16 a cycle and SM against 32 scores of
// 128-wide dot products on the tensor cores), but they do not bound it by themselves:
// 8192 tokens of 32 heads take 326 us, 239 if their unit never stood still, and 285
// with no exponential at all (of the state that took 341; 313 with one MMA of eight,
// 266 with neither): what is left is a step's hand-overs between the tensor cores and
// the warpgroup that owns its one score buffer.  Measured at 341 and not kept: a quarter of the exponentials as polynomials
// (355 us: four warps per scheduler do not hide their chains), two issuing threads
// (357: 80 registers a thread, spills), each Q tile kept for two key tiles (341).
//
// Work.  A unit is one (sequence, KV head, 128-key tile); its steps are the row
// tiles (up to 128 rows: tt counted rows x gb heads) from the first that sees
// the tile.  All steps, in unit order, are cut into equal runs, one CTA per SM; a
// unit that a cut divides leaves partial sums, added in CTA order by
// weights_finish_kernel.
//
//   warps 0..15  sums: warpgroup g takes the steps g, g + 4, ... of the run, thread
//                r key r (with two warpgroups the exponentials' unit stood idle
//                half the time behind TMEM reads and barriers: that prompt took
//                485 us instead of 457, before the producers below were split)
//   warp 16      TMEM owner + single-thread tcgen05.mma issuer
//   warp 17      TMA producer of K tiles, through the page table
//   warp 18      producer of Q tiles: TMA, or copies by the row list
//   warp 19      producer of the rows' -LSE and visible ends
//
// TMEM: four score buffers of 128 columns, step s in buffer s & 3.
#include <algorithm>
#include <cstring>

#include "cache.cuh"
#include "kernels.h"

namespace attn {

namespace {

constexpr int KT = 128;  // keys per tile (TMEM lanes)
constexpr int BR = 128;  // rows per tile (columns) at most
constexpr int kSums = 4;  // warpgroups of sums, one per score buffer
constexpr int kWarpMma = 16, kWarpLoad = 17, kWarpQ = 18, kWarpZ = 19;
constexpr int kThreads = 640;
constexpr uint32_t kTmemCols = 512;
constexpr int NZ = 8;  // row-term ring

template <int D>
struct WeightsSmem {
  static constexpr int kTileBytes = 128 * D * 2;
  // K tiles [0, nk) and Q tiles [nk, NT) share the space: a launch of one row
  // tile per head streams K past it, one of many streams Q past a K tile
  static constexpr int NT = D == 128 ? 6 : 12;
  static constexpr int kKeysFew = NT / 3, kKeysMany = 2 * NT / 3;  // nk of the two
  alignas(1024) uint8_t tile[NT][kTileBytes];
  alignas(16) float z[NZ][BR];  // -LSE log2(e); -inf for a row that counts for nothing
  alignas(16) int last[NZ][BR];  // last slot the row sees; -1 for a row that counts for nothing
  int hides[NZ];  // a row that counts has LSE = -inf
  float part[kSums][KT];  // a unit's sums by the warpgroups that do not finish it
  uint64_t t_full[NT], t_empty[NT];
  uint64_t z_full[NZ], z_empty[NZ], s_full[4], s_empty[4];
  uint64_t part_full, part_empty, drain;
  RunSmem<kThreads, 1> run;
  uint32_t tmem_base;
  int abort_flag;
};

// Row tiles: tt counted rows x gb heads, gblk blocks of heads.
using Rows = RowTiles;

Rows row_tiles(int Hq, int Hkv, int max_rows) {
  Rows r{};
  r.G = Hq / Hkv;
  r.gb = std::min(r.G, BR);
  r.tt = std::min(BR / r.gb, max_rows);
  r.gblk = (r.G + r.gb - 1) / r.gb;
  r.tiles = (max_rows + r.tt - 1) / r.tt * r.gblk;
  return r;
}

// Sum of floor((y + KT x) / tt) over x < n: the row tiles wholly before each of n key
// tiles.  With the whole parts of slope and offset taken out, 0 <= a, b < m, the terms
// t(x) = floor((a x + b) / m) rise to t = t(n - 1), and summed the other way round,
//   sum_x t(x) = sum_(1 <= j <= t) #{x < n : a x + b >= j m}
//              = t n - sum_(0 <= j < t) floor((m j + m - b + a - 1) / a),
// the same sum with slope and divisor exchanged (the law of reciprocity of such sums:
// Graham, Knuth, Patashnik, Concrete Mathematics, 3.5): as many turns as Euclid's
// algorithm takes for KT and tt.  Only the sum passes 32 bits (n < 2^22, y < 2^29).
ATTN_DEVINL long long tiles_before(unsigned n, unsigned y, unsigned tt) {
  long long sum = 0;
  unsigned a = KT, b = y, m = tt;
  for (int sign = 1; n > 0; sign = -sign) {
    const unsigned qa = a / m, qb = b / m;
    a -= qa * m;
    b -= qb * m;
    const unsigned t = (a * (n - 1) + b) / m;
    sum += sign * ((long long)n * (n - 1) / 2 * qa + (long long)n * qb + (long long)n * t);
    b = m - b + a - 1;
    n = t;  // 0 where a is
    const unsigned x = a;
    a = m;
    m = x;
  }
  return sum;
}

// One sequence's share: per KV head, key tile kt has its row tiles from
// first_tile(kt) on, times the blocks of heads.
struct Seq {
  int len, cnt, nk, tiles;  // slots, counted rows, key tiles, row tiles (of one block of heads)
  long long per_head;
};

ATTN_DEVINL int first_tile(const Rows& rw, const Seq& s, int kt) {
  const int i = kt * KT - (s.len - s.cnt);  // the first row that sees the tile
  return i > 0 ? i / rw.tt : 0;
}

// Steps that a unit of several row tiles counts for beyond its own when the work is
// cut into runs (its K tile and the joining of its sums): with 0, the CTAs with the
// short units at a head's end took longest, and an 8192-token prompt 341 us instead of
// 326 (2: 334, 6: 329).
constexpr int kUnitCost = 4;
ATTN_DEVINL int unit_cost(const Rows& rw) { return rw.tiles > 1 ? kUnitCost : 0; }

// Steps of the key tiles below kt of a head.
ATTN_DEVINL long long steps_below(const Rows& rw, const Seq& s, int kt) {
  const int shift = s.len - s.cnt;
  const int k0 = shift >= 0 ? shift / KT + 1 : 0;  // the first tile that early rows do not see
  long long cut = 0;
  if (kt > k0) cut = tiles_before(kt - k0, k0 * KT - shift, rw.tt);
  return ((long long)kt * s.tiles - cut) * rw.gblk + (long long)kt * unit_cost(rw);
}

ATTN_DEVINL Seq load_seq(const WeightsParams& p, const Rows& rw, int b) {
  Seq s;
  if (!cache_len(p.c, b, p.cap, p.status, s.len) || !row_count(p.row_lens, b, p.max_rows, p.status, s.cnt))
    s.len = s.cnt = 0;
  s.nk = s.cnt > 0 ? (s.len + KT - 1) / KT : 0;
  s.tiles = (s.cnt + rw.tt - 1) / rw.tt;
  s.per_head = s.nk > 0 ? steps_below(rw, s, s.nk) : 0;
  return s;
}

// A place in a ring whose length is known at run time only, kept by counting: a
// division a step costs the issuing thread as much as its MMAs' issue.
struct Place {
  int slot = 0;
  uint32_t lap = 0;
  ATTN_DEVINL void next(int n) {
    if (++slot == n) {
      slot = 0;
      lap ^= 1;
    }
  }
};

struct Unit {
  int b, hk, kt;
  int first;      // first row tile (of a block of heads)
  int jb, je, n;  // steps [jb, je) of n: row tile first + j / gblk, block of heads j % gblk
  bool same_q;    // launches of one row tile: it is the previous unit's; else each step has its own
};

struct Walk {
  int b, hk, kt, j, left;
  bool any;
  Seq s;

  ATTN_DEVINL void begin(const WeightsParams& p, const Rows& rw, const Run& run) {
    left = (int)(run.run1 - run.run0);
    any = false;
    if (left <= 0) return;
    b = run.b;
    s = load_seq(p, rw, b);
    hk = (int)(run.off / s.per_head);
    const long long off = run.off % s.per_head;
    int lo = 0, hi = s.nk - 1;  // the last tile with steps_below <= off
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (steps_below(rw, s, mid) <= off)
        lo = mid;
      else
        hi = mid - 1;
    }
    kt = lo;
    j = (int)(off - steps_below(rw, s, kt));
    // (a run that begins behind a unit's steps begins with the next unit)
    const int n = (s.tiles - first_tile(rw, s, kt)) * rw.gblk;
    if (j >= n) {
      left -= n + unit_cost(rw) - j;
      j = 0;
      ++kt;
    }
  }
  ATTN_DEVINL bool next(const WeightsParams& p, const Rows& rw, Unit& u) {
    if (left <= 0) return false;
    bool fresh = !any;
    any = true;
    if (kt == s.nk) {
      kt = 0;
      fresh = true;
      if (++hk == p.Hkv) {
        hk = 0;
        do s = load_seq(p, rw, ++b);
        while (s.per_head == 0);
      }
    }
    u.b = b;
    u.hk = hk;
    u.kt = kt;
    u.first = first_tile(rw, s, kt);
    u.n = (s.tiles - u.first) * rw.gblk;
    u.jb = j;
    u.je = min(u.n, j + left);
    u.same_q = !fresh && rw.tiles == 1;
    left -= u.je - u.jb + unit_cost(rw);
    j = 0;
    ++kt;
    return true;
  }
};

// Sum of exponentials of N columns of a key, x = s * sc2 + z in pairs (sc2 twice
// in sc).  EDGE: a column whose row does not see the key, or does not count, adds
// nothing whatever its score.
template <bool EDGE, int N>
ATTN_DEVINL void add_columns(const uint32_t (&sr)[N], const float* z, const int* last, int key, uint64_t sc,
                             uint64_t& a0, uint64_t& a1) {
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    const ulonglong2 zz = *reinterpret_cast<const ulonglong2*>(z + e);
    const uint64_t s01 = pack_f32x2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
    const uint64_t s23 = pack_f32x2(__uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3]));
    float x0, x1, x2, x3;
    unpack_f32x2(fma_f32x2(s01, sc, zz.x), x0, x1);
    unpack_f32x2(fma_f32x2(s23, sc, zz.y), x2, x3);
    if constexpr (EDGE) {
      const int4 ll = *reinterpret_cast<const int4*>(last + e);
      if (key > ll.x) x0 = -INFINITY;
      if (key > ll.y) x1 = -INFINITY;
      if (key > ll.z) x2 = -INFINITY;
      if (key > ll.w) x3 = -INFINITY;
    }
    a0 = add_f32x2(a0, pack_f32x2(ex2(x0), ex2(x1)));
    a1 = add_f32x2(a1, pack_f32x2(ex2(x2), ex2(x3)));
  }
}

// The same of a whole row tile in TMEM; a full one's next 16 columns are on
// their way while 16 are summed.
template <bool EDGE>
ATTN_DEVINL float add_tile(uint32_t col, int width, const float* z, const int* last, int key, uint64_t sc) {
  uint64_t a0 = 0, a1 = 0;  // a tile's own sums: short chains round less
  uint32_t sr[2][16];
  tmem_ld16(col, sr[0]);
  if (width == BR) {
#pragma unroll
    for (int c = 0; c < BR / 16; ++c) {
      tmem_wait_ld();
      reg_fence(sr[c & 1]);
      if (c + 1 < BR / 16) tmem_ld16(col + 16 * (c + 1), sr[(c + 1) & 1]);
      add_columns<EDGE>(sr[c & 1], z + 16 * c, last + 16 * c, key, sc, a0, a1);
    }
  } else {
    for (int c = 0; c < width; c += 16) {
      tmem_wait_ld();
      reg_fence(sr[0]);
      add_columns<EDGE>(sr[0], z + c, last + c, key, sc, a0, a1);
      if (c + 16 < width) tmem_ld16(col + c + 16, sr[0]);
    }
  }
  float x, y;
  unpack_f32x2(add_f32x2(a0, a1), x, y);
  return x + y;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                   const WeightsParams p, const TileForm form) {
  using Smem = WeightsSmem<D>;
  constexpr int NT = Smem::NT;
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Rows& rw = p.rw;
  const int width = min(BR, (rw.gb * rw.tt + 15) / 16 * 16);  // columns of a row tile
  const int nk = rw.tiles == 1 ? Smem::kKeysMany : Smem::kKeysFew, nq = NT - nk;
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < NT; ++i) {
      mbar_init(&s.t_full[i], 1);
      mbar_init(&s.t_empty[i], 1);
    }
    for (int i = 0; i < NZ; ++i) {
      mbar_init(&s.z_full[i], 1);
      mbar_init(&s.z_empty[i], rw.tiles == 1 ? 4 * kSums : 4);  // warps that use a slot (see same_q)
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_empty[i], 4);
    }
    mbar_init(&s.part_full, 4 * (kSums - 1));
    mbar_init(&s.part_empty, 4);
    mbar_init(&s.drain, 1);
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(&s.tmem_base, kTmemCols);
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tm_k);
    if (!p.rows) tma_prefetch_desc(&tm_q);  // (listed rows have no map)
  }
  // columns that no load writes: zeros, so that their scores are finite
  for (int i = threadIdx.x; i < nq * (width - rw.gb * rw.tt) * (D / 8); i += kThreads) {
    const int c = i % (D / 8), r = rw.gb * rw.tt + i / (D / 8) % (width - rw.gb * rw.tt);
    const int t = nk + i / (D / 8) / (width - rw.gb * rw.tt);
    *reinterpret_cast<uint4*>(s.tile[t] + (c >> 3) * (BR * 128) + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  find_runs<kThreads, 1>(s.run, p.B, 1, [&](int b) { return load_seq(p, rw, b).per_head * p.Hkv; });
  const Run& run = s.run.runs.lane[0];
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const Abort ab{&s.abort_flag, p.status, p.wait_limit};
  Walk w;
  w.begin(p, rw, run);
  Unit u{};

  if (warp == kWarpLoad) {
    // ===================================================== K producer
    TileCursor at{0, 0};
    int b = -1, hk = -1;  // where the cursor is
    auto find = [&](const Unit& u) {
      if (u.hk == hk && u.b == b) {
        at.next(p.c, form);
      } else {
        at.begin(p.c, form, u.kt * KT);
        hk = u.hk;
        b = u.b;
      }
      return find_box(p.c, form, at, u.b, w.s.len - u.kt * KT);
    };
    bool ok = true, more = w.next(p, rw, u);
    TileBox box{};
    if (more) box = find(u);
    for (Place k; more; k.next(nk)) {
      const TileBox cur = box;
      const int cur_hk = u.hk;
      if ((more = w.next(p, rw, u))) box = find(u);
      ok = __all_sync(0xffffffffu, mbar_wait(&s.t_empty[k.slot], k.lap ^ 1, ab));
      if (!ok) break;
      load_tile<D>(s.tile[k.slot], &s.t_full[k.slot], &tm_k, form, cur, cur_hk, p.c.num_pages, p.status);
    }
    if (s.abort_flag) {
      // leave no copy in flight into shared memory that is about to be released
      for (int st = 0; st < nk; ++st) {
        mbar_wait_drain(&s.t_full[st], 0, p.wait_limit / 64);
        mbar_wait_drain(&s.t_full[st], 1, p.wait_limit / 64);
      }
    }
  } else if (warp == kWarpQ) {
    // ===================================================== Q producer
    // Rows in their own order come by TMA; listed rows by 16-byte copies, a row's
    // address per lane, into the same 128-byte swizzle (chunk c of row r at chunk
    // c ^ (r & 7)).
    constexpr int CH = D / 8;  // 16-byte chunks per row
    Place q;
    bool ok = true;
    while (ok && w.next(p, rw, u)) {
      if (u.same_q) continue;
      for (int j = u.jb; j < u.je; ++j, q.next(nq)) {
        const int st = nk + q.slot, i0 = (u.first + j / rw.gblk) * rw.tt, g0 = j % rw.gblk * rw.gb;
        ok = __all_sync(0xffffffffu, mbar_wait(&s.t_empty[st], q.lap ^ 1, ab));
        if (!ok) break;
        if (!p.rows) {
          if (lane == 0) {
            mbar_expect_tx(&s.t_full[st], rw.gb * rw.tt * (D / 64) * 128);
#pragma unroll
            for (int kb = 0; kb < D / 64; ++kb)
              tma_load_4d(s.tile[st] + kb * BR * 128, &tm_q, &s.t_full[st], kb * 64, u.hk * rw.G + g0, i0, u.b);
          }
          __syncwarp();
          continue;
        }
        const char* base = static_cast<const char*>(p.q);
        const uint32_t qs = smem_u32(s.tile[st]);
#pragma unroll 1
        for (int x = 0; x < width; x += 32) {
          const int row = i0 + (x + lane) / rw.gb, g = g0 + (x + lane) % rw.gb;
          long long src = -1;
          if (x + lane < rw.gb * rw.tt && row < w.s.cnt && g < rw.G) {
            const int t = __ldg(p.rows + (long long)u.b * p.max_rows + row);
            if (t >= 0 && t < p.Nq) src = (((long long)u.b * p.Nq + t) * p.Hq + u.hk * rw.G + g) * D;
          }
#pragma unroll 1
          for (int y = 0; y < CH; ++y) {
            const int rr = y * (32 / CH) + lane / CH, c = lane % CH;  // row of the 32, chunk of the row
            const long long at = __shfl_sync(0xffffffffu, src, rr);
            const int r = x + rr;
            const uint32_t dst = qs + (c >> 3) * (BR * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            // a row that counts for nothing is zeros
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                         "l"(base + (at < 0 ? 0 : at * 2 + c * 16)), "r"(at < 0 ? 0 : 16)
                         : "memory");
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.t_full[st]);
      }
    }
    if (s.abort_flag && !p.rows) {
      for (int st = nk; st < NT; ++st) {
        mbar_wait_drain(&s.t_full[st], 0, p.wait_limit / 64);
        mbar_wait_drain(&s.t_full[st], 1, p.wait_limit / 64);
      }
    }
  } else if (warp == kWarpZ) {
    // ===================================================== rows' terms
    // -LSE and the last visible slot of each row, four rows a lane.
    int tq[4], gq[4];  // a row's place in a row tile
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = x * 32 + lane;
      tq[x] = r < rw.gb * rw.tt ? r / rw.gb : 1 << 29;  // (no row)
      gq[x] = r % rw.gb;
    }
    struct Terms {
      float lse[4];
      int last[4];
    };
    int i = 0, j = 0;  // row tiles stored; step of the unit
    bool ok = true;
    u.je = 0;
    long long base[4];  // lse of the lane's heads in this unit
    int row[4], len = 0, cnt = 0, gi = 0;  // the lane's rows in this step; block of heads
    auto place = [&]() {  // rows and heads of the unit's first step here
      const int i0 = (u.first + j / rw.gblk) * rw.tt;
      gi = j % rw.gblk;
      len = w.s.len;
      cnt = w.s.cnt;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        row[v] = i0 + tq[v];
        base[v] = ((long long)u.b * p.Hq + u.hk * rw.G + gi * rw.gb + gq[v]) * p.Nq;
      }
    };
    auto advance = [&]() -> bool {  // to the next step that has a row tile of its own
      if (++j < u.je) {
        const bool next_rows = ++gi == rw.gblk;
        if (next_rows) gi = 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          row[v] += next_rows ? rw.tt : 0;
          base[v] += rw.gblk > 1 ? (long long)(next_rows ? 1 - rw.gblk : 1) * rw.gb * p.Nq : 0;
        }
        return true;
      }
      do {
        if (!w.next(p, rw, u)) return false;
        // the slots' weights into L2, before their sums are ready
        const int key = u.kt * KT + lane * 32;
        if (p.weights && lane < 5 && key < w.s.len)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.weights + ((long long)u.b * p.Hkv + u.hk) * p.cap + key));
      } while (u.same_q);
      j = u.jb;
      place();
      return true;
    };
    auto load = [&](Terms& t) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        bool on = row[v] < cnt && gi * rw.gb + gq[v] < rw.G;
        int k = row[v];
        if (p.rows) {
          k = ldg_if(p.rows + (long long)u.b * p.max_rows + row[v], on, 0);
          if (k < 0 || k >= p.Nq) {
            atomicExch(p.status, ATTN_ERR_INVALID);
            on = false;
          }
        }
        t.lse[v] = ldg_if(p.lse + base[v] + k, on, 0.f);
        t.last[v] = on ? len - cnt + row[v] : -1;
      }
    };
    auto store = [&](const Terms& t) {
      const int zt = i % NZ;
      ok = __all_sync(0xffffffffu, mbar_wait(&s.z_empty[zt], ((i / NZ) & 1) ^ 1, ab));
      if (!ok) return;
      bool hides = false;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const bool none = t.lse[v] == -INFINITY;
        hides |= none && t.last[v] >= 0;
        s.z[zt][v * 32 + lane] = none || t.last[v] < 0 ? -INFINITY : -t.lse[v] * kLog2e;
        s.last[zt][v * 32 + lane] = none ? -1 : t.last[v];
      }
      hides = __any_sync(0xffffffffu, hides);
      if (lane == 0) s.hides[zt] = hides;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.z_full[zt]);
      ++i;
    };
    // two sets in turn: nothing waits for a load but its own store
    Terms t0, t1;
    bool more = advance();
    if (more) load(t0);
    while (ok && more) {
      if ((more = advance())) load(t1);
      store(t0);
      if (!ok || !more) break;
      if ((more = advance())) load(t0);
      store(t1);
    }
  } else if (warp == kWarpMma) {
    // ===================================================== MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(KT, width, 0, 0);
      int step = 0;
      Place k, q;  // the K tile in use; the next Q tile
      int q_slot = -1;
      bool ok = true;
      for (; ok && w.next(p, rw, u); k.next(nk)) {
        if (!(ok = mbar_wait(&s.t_full[k.slot], k.lap, ab))) break;
        const uint64_t kd = k_tile_desc<D>(s.tile[k.slot]);
        for (int j = u.jb; j < u.je; ++j, ++step) {
          if (!u.same_q) {
            if (q_slot >= 0) mma_commit(&s.t_empty[q_slot]);  // the previous row tile has been used
            q_slot = nk + q.slot;
            if (!(ok = mbar_wait(&s.t_full[q_slot], q.lap, ab))) break;
            q.next(nq);
          }
          const int buf = step & 3;
          if (!(ok = mbar_wait(&s.s_empty[buf], ((step >> 2) & 1) ^ 1, ab))) break;
          tc_fence_after();
          const uint64_t qd = sdesc_sw128(smem_u32(s.tile[q_slot]), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + buf * BR, k_tile_step(kd, kk), sdesc_at(qd, (kk >> 2) * (BR * 128) + (kk & 3) * 32), idesc,
                   kk > 0);
          mma_commit(&s.s_full[buf]);
        }
        if (ok) mma_commit(&s.t_empty[k.slot]);
      }
      // TMEM must be quiescent before it is released
      mma_commit(&s.drain);
      mbar_wait_drain(&s.drain, 0, p.wait_limit);
    }
  } else {
    // ===================================================== sums
    const int wg = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t col = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + wg * BR;
    const uint64_t sc = pack_f32x2(p.scale * kLog2e, p.scale * kLog2e);
    const bool one = rw.tiles == 1;  // rows' terms shared by all steps of a head, else one step's
    int step = 0, iz = -1, shared = 0;
    bool ok = true;
    while (ok && w.next(p, rw, u)) {
      const int key = u.kt * KT + r, n = u.je - u.jb, s0 = step;
      const bool whole = n == u.n;
      // who adds up: the warpgroup of the first step here
      const bool owner = (s0 & 3) == wg;
      const long long at = ((long long)u.b * p.Hkv + u.hk) * p.cap + key;
      float before = 0.f;
      if (owner && whole && key < w.s.len && p.weights) before = p.weights[at];
      float sum = 0.f;
      if (one && !u.same_q) {
        if (iz >= 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.z_empty[iz % NZ]);
        }
        ++iz;
        ok = __all_sync(0xffffffffu, mbar_wait(&s.z_full[iz % NZ], (iz / NZ) & 1, ab));
        if (!ok) break;
      }
      // this warpgroup's steps
      step = s0 + ((wg - s0) & 3);
      for (; step < s0 + n; step += kSums) {
        const int zt = one ? iz % NZ : step % NZ, j = u.jb + step - s0;
        if (!one) {
          ok = __all_sync(0xffffffffu, mbar_wait(&s.z_full[zt], (step / NZ) & 1, ab));
          if (!ok) break;
        }
        const int hides = s.hides[zt];
        ok = __all_sync(0xffffffffu, mbar_wait(&s.s_full[wg], (step >> 2) & 1, ab));
        if (!ok) break;
        tc_fence_after();
        const float* z = s.z[zt];
        const int* last = s.last[zt];
        // rows from i0 on: the tile's last key is hidden from the first of them, or
        // some of them count for nothing (q may hold anything there)
        const int i0 = (u.first + j / rw.gblk) * rw.tt;
        const bool edge = u.kt * KT + KT - 1 > w.s.len - w.s.cnt + i0 || i0 + rw.tt > w.s.cnt ||
                          rw.gblk > 1 || hides;
        sum += edge ? add_tile<true>(col, width, z, last, key, sc) : add_tile<false>(col, width, z, last, key, sc);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.s_empty[wg]);
          if (!one) mbar_arrive(&s.z_empty[zt]);
        }
      }
      if (!ok) break;
      step = s0 + n;
      if (n > 1) {  // several warpgroups took steps
        // The previous unit's sums have been read.  All of them wait for that, the
        // owner too: it may have been among those that handed theirs over, and the
        // others of that unit may still be at it, whose phase it must not skip.
        ok = __all_sync(0xffffffffu, mbar_wait(&s.part_empty, (shared & 1) ^ 1, ab));
        if (!ok) break;
        if (owner) {
          ok = __all_sync(0xffffffffu, mbar_wait(&s.part_full, shared & 1, ab));
          if (!ok) break;
          for (int x = 1; x < min(n, kSums); ++x) sum += s.part[(wg + x) & 3][r];
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.part_empty);
        } else {
          s.part[wg][r] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.part_full);
        }
        ++shared;
      }
      if (owner) {
        if (!whole)
          p.part[((long long)blockIdx.x * 2 + (u.jb > 0 ? 0 : 1)) * KT + r] = sum;
        else if (key < w.s.len)
          p.out[at] = before + sum;
      }
    }
  }

  // ---- teardown; the finishing kernel may be launched (it waits for this grid's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // The unit that this run ends in the middle of, having held its beginning (u is
  // the run's last unit): its later parts are the next CTAs' first ones.
  if (threadIdx.x == 0) {
    WeightsCut cut{0, 0, 0, 0};
    if (!s.abort_flag && run.run1 > run.run0 && u.jb == 0 && u.je < u.n)
      cut = WeightsCut{u.b, u.hk, u.kt, run_parts(s.run.runs.total, s.run.runs.workers, blockIdx.x, run.run1, u.n - u.je)};
    p.cuts[blockIdx.x] = cut;
  }
}

// Blocks (c < ctas, 0) add the parts of the unit whose first part CTA c holds, in
// CTA order.  When out is another buffer than weights, block (u, y) copies every
// gridDim.y-th run, from the y-th on, of the slots of (sequence, KV head) u that no unit
// covers (behind the sequence's end); it need not wait for that.
constexpr int kFinish = 256, kCopyRun = 8 * kFinish;

__global__ void __launch_bounds__(kFinish) weights_finish_kernel(const WeightsParams p, const int ctas) {
  const int r = threadIdx.x;
  if (p.weights != p.out && blockIdx.x < (unsigned)(p.B * p.Hkv)) {
    int len, cnt;
    const int b = blockIdx.x / p.Hkv;
    // a sequence that is not acceptable is left as it is
    if (cache_len(p.c, b, p.cap, p.status, len) && row_count(p.row_lens, b, p.max_rows, p.status, cnt)) {
      const int from = cnt > 0 ? len : 0;
      const float* src = p.weights ? p.weights + (long long)blockIdx.x * p.cap : nullptr;
      float* dst = p.out + (long long)blockIdx.x * p.cap;
      for (int j0 = blockIdx.y * kCopyRun + r; j0 < p.cap; j0 += gridDim.y * kCopyRun) {
        float x[kCopyRun / kFinish];
#pragma unroll
        for (int i = 0; i < kCopyRun / kFinish; ++i) {
          const int j = j0 + i * kFinish;
          x[i] = src && j >= from && j < p.cap ? src[j] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kCopyRun / kFinish; ++i) {
          const int j = j0 + i * kFinish;
          if (j >= from && j < p.cap) dst[j] = x[i];
        }
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x < ctas && blockIdx.y == 0 && r < KT) {
    const WeightsCut cut = p.cuts[blockIdx.x];
    const int key = cut.kt * KT + r;
    if (cut.more > 0 && key < p.c.lens[cut.b]) {
      float sum = p.part[((long long)blockIdx.x * 2 + 1) * KT + r];
      for (int i = 1; i <= cut.more; ++i) sum += p.part[(long long)(blockIdx.x + i) * 2 * KT + r];
      const long long at = ((long long)cut.b * p.Hkv + cut.hk) * p.cap + key;
      p.out[at] = (p.weights ? p.weights[at] : 0.f) + sum;
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

template <int D>
int launch_t(const WeightsParams& p, cudaStream_t st) {
  CUtensorMap mk;
  TileForm form;
  int rc;
  if ((rc = cache_tile_map(&mk, &form, p.c, p.c.k, p.Hkv, D))) return rc;
  const Rows& rw = p.rw;
  CUtensorMap mq;
  const uint64_t rq = (uint64_t)p.Hq * D * 2;
  const uint64_t qd[4] = {D, (uint64_t)p.Hq, (uint64_t)p.Nq, (uint64_t)p.B}, qs[3] = {D * 2, rq, rq * p.Nq};
  const uint32_t qb[4] = {64, (uint32_t)rw.gb, (uint32_t)rw.tt, 1};
  std::memset(&mq, 0, sizeof(mq));
  if (!p.rows && (rc = encode_tmap_bf16(&mq, p.q, 4, qd, qs, qb))) return rc;
  const size_t smem = sizeof(WeightsSmem<D>) + 1024;
  static_assert(sizeof(WeightsSmem<D>) + 1024 <= 232448, "shared memory");
  if (cudaFuncSetAttribute(weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATTN_ERR_CUDA;
  const int ctas = sm_count();
  weights_kernel<D><<<ctas, kThreads, smem, st>>>(mk, mq, p, form);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (rw.tiles == 1 && p.weights == p.out) {  // no unit is cut, no slot left to copy
    count_launch();
    return ATTN_OK;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = p.weights == p.out ? dim3((unsigned)ctas)
                                   : dim3((unsigned)std::max((long long)ctas, (long long)p.B * p.Hkv),
                                          (unsigned)std::min((p.cap + kCopyRun - 1) / kCopyRun, 65535));
  cfg.blockDim = dim3(kFinish);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, weights_finish_kernel, p, ctas) != cudaSuccess) return ATTN_ERR_CUDA;
  count_launch(2);
  return ATTN_OK;
}

}  // namespace

size_t weights_sm100_workspace() {
  return align256((size_t)sm_count() * 2 * KT * 4) + align256((size_t)sm_count() * sizeof(WeightsCut));
}

int launch_weights_sm100(WeightsParams p, void* workspace, cudaStream_t st) {
  p.part = static_cast<float*>(workspace);
  p.cuts = reinterpret_cast<WeightsCut*>(static_cast<char*>(workspace) + align256((size_t)sm_count() * 2 * KT * 4));
  p.wait_limit = kWaitLimitCycles;
  p.rw = row_tiles(p.Hq, p.Hkv, p.max_rows);
  return p.D == 64 ? launch_t<64>(p, st) : launch_t<128>(p, st);
}

}  // namespace attn
