// Tree attention over a key/value cache on sm_100a tensor cores (bf16).
//
// A few new tokens per sequence (one, a chunk, a drafted tree) attend to a long
// cache: every K/V row is read once for the few query rows of its sequence and
// KV head, so the kernel is bound by HBM and is built to stream.
//
// Rows.  The query rows of one (sequence, KV head) are all (token t, head g of
// the group), packed as tiles of up to 128 rows: `tt` tokens x `gb` heads, row
// r = (t0 + r / gb, g0 + r % gb), so that the group shares each K/V tile
// ("Understanding FlashAttention Pt 1", contents 4.1).
//
// Work.  A unit is one (sequence, KV head, one or two row tiles); its tiles are
// the 128-key tiles of its cached slots followed by those of its new keys.  The
// units' tiles are laid end to end and cut into equal runs, one per CTA (one CTA
// per SM), whatever the lengths are: they are read on the device.  A unit that a
// cut divides leaves one partial (O, m, l) per CTA in the workspace, and
// tree_merge_kernel combines them in CTA order, so results do not vary from run
// to run.
//
//   warps 0..3  softmax of stream 0: thread r owns row r (TMEM lane r)
//   warps 4..7  softmax of stream 1
//   warp 8      TMEM owner + single-thread tcgen05.mma issuer
//   warp 9      TMA producer: a lane per box, looked up in the page table
//
// Streams.  With one row tile the two streams take alternate key tiles, each
// with a running state (m, l) and an accumulator O of its own, merged in the
// epilogue ("Softmax does not need the matrix", "Carry the Normalizer").  With
// two row tiles (more than 128 rows) stream t is row tile t and both read every
// key tile, so K and V cross HBM once for up to 256 rows.  Either way item m
// belongs to stream m & 1 and the issue order is
//   S(0); S(1), O += P(0) V; S(2), O += P(1) V; ...
// S(m) overwrites the buffer of P(m - 2), whose product was issued before it,
// and once S(m) is complete so is that product: the stream's O may be rescaled
// before P(m) is handed over.
//
// TMEM (512 columns): [128 s, +128) scores of stream s, P (bf16 pairs) over its
// first 64; [256 + D s, +D) O of stream s.
//
// The last key tile of a sequence ends inside a page or box.  Its hidden scores
// are set to -inf whatever they hold, and its hidden V rows are zeroed in shared
// memory before the product, so rows behind the sequence's end may hold anything.
#include <algorithm>
#include <cstring>

#include "cache.cuh"
#include "kernels.h"

namespace attn {

namespace {

constexpr int KT = 128;  // keys per tile
constexpr int BM = 128;  // rows per tile
constexpr int kWarpMma = 8, kWarpLoad = 9;
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.f;  // log2 units: P stays <= 256

template <int D>
struct TreeSmem {
  static constexpr int kTileBytes = 128 * D * 2;
  // K and V tiles share one ring; two Q tiles (the next unit's while one is used)
  static constexpr int NST = std::min(12, (223 * 1024 - 2 * kTileBytes) / kTileBytes);
  alignas(1024) uint8_t q[2][kTileBytes];
  alignas(1024) uint8_t kv[NST][kTileBytes];
  float2 ml[2][BM];  // (m, l) of the two streams
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[NST], kv_empty[NST];
  uint64_t s_full[2], p_full[2];
  uint64_t o_done, o_free, ml_full, drain;
  RunSmem<kThreads> run;
  uint32_t tmem_base;
  int abort_flag;
};

// Row tiles of a launch: tt tokens x gb heads each, gblk blocks of heads.
struct Rows {
  int G, gb, tt, gblk, tiles;  // tiles = token blocks * gblk
};

__host__ __device__ inline Rows row_tiles(int Hq, int Hkv, int Nq) {
  Rows r;
  r.G = Hq / Hkv;
  r.gb = r.G < BM ? r.G : BM;
  const int fit = BM / r.gb;
  r.tt = fit < Nq ? fit : Nq;
  r.gblk = (r.G + r.gb - 1) / r.gb;
  r.tiles = (Nq + r.tt - 1) / r.tt * r.gblk;
  return r;
}

// One sequence's share of the work: per KV head `active` units of n tiles, then
// the units whose rows are all padding (one empty step each).
struct Seq {
  int len, nr, nc, n, row_tiles, active;
  long long per_head;
};

ATTN_DEVINL Seq load_seq(const TreeParams& p, const Rows& rw, int b) {
  Seq s;
  if (!cache_len(p.c, b, 1ll << 31, p.status, s.len) || !row_count(p.row_lens, b, p.Nq, p.status, s.nr))
    s.len = s.nr = 0;
  s.nc = (s.len + KT - 1) / KT;
  s.n = s.nc + (p.k_new ? (s.nr + KT - 1) / KT : 0);
  s.row_tiles = s.n > 0 ? (s.nr + rw.tt - 1) / rw.tt * rw.gblk : 0;
  s.active = (s.row_tiles + 1) / 2;
  s.per_head = (long long)s.active * s.n + ((rw.tiles + 1) / 2 - s.active);
  return s;
}

// A CTA's run of tiles, unit by unit.
struct Unit {
  int b, hk, pair;      // row tiles 2 pair, 2 pair + 1
  int tb, te, n;        // tiles [tb, te) of n
  bool two, empty;      // two row tiles; no row of it sees anything
};

struct Walk {
  int b, hk;
  long long off, left;  // position inside (b, hk); tiles left in the run
  Seq s;

  ATTN_DEVINL void begin(const TreeParams& p, const Rows& rw, int b0, long long off0, long long run) {
    b = b0;
    left = run;
    if (left <= 0) return;
    s = load_seq(p, rw, b);
    hk = (int)(off0 / s.per_head);
    off = off0 % s.per_head;
  }
  ATTN_DEVINL bool next(const TreeParams& p, const Rows& rw, Unit& u) {
    if (left <= 0) return false;
    if (off == s.per_head) {
      off = 0;
      if (++hk == p.Hkv) {
        hk = 0;
        s = load_seq(p, rw, ++b);
      }
    }
    u.b = b;
    u.hk = hk;
    const long long busy = (long long)s.active * s.n;
    if (off < busy) {
      u.pair = (int)(off / s.n);
      u.tb = (int)(off % s.n);
      u.n = s.n;
      u.te = (int)min((long long)s.n, u.tb + left);
      u.two = 2 * u.pair + 1 < s.row_tiles;
      u.empty = false;
    } else {
      u.pair = s.active + (int)(off - busy);
      u.tb = 0;
      u.te = u.n = 1;
      u.two = false;
      u.empty = true;
    }
    off += u.te - u.tb;
    left -= u.te - u.tb;
    return true;
  }
};

// Position of K / V tile i of a unit of `n` tiles in the order of its loads
// (K_i before S(i), V_i before the product with P(i)).
ATTN_DEVINL int seq_k(bool two, int i) { return two ? 2 * i : (i == 0 ? 0 : 2 * i - 1); }
ATTN_DEVINL int seq_v(bool two, int i, int n) { return two ? 2 * i + 1 : (i == n - 1 ? 2 * n - 1 : 2 * i + 2); }

template <int N>
ATTN_DEVINL void reg_fence(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

ATTN_DEVINL void store_bf16_32(__nv_bfloat16* dst, const float (&x)[32]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    reinterpret_cast<uint4*>(dst)[e] =
        make_uint4(pack_bf16(x[8 * e], x[8 * e + 1]), pack_bf16(x[8 * e + 2], x[8 * e + 3]),
                   pack_bf16(x[8 * e + 4], x[8 * e + 5]), pack_bf16(x[8 * e + 6], x[8 * e + 7]));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kn,
                const __grid_constant__ CUtensorMap tm_vn, const TreeParams p, const int box_rows,
                const int new_box_rows) {
  using Smem = TreeSmem<D>;
  constexpr int NST = Smem::NST;
  constexpr int KB = D / 64;  // 128-byte blocks per row
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Rows rw = row_tiles(p.Hq, p.Hkv, p.Nq);

  // ---- setup
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.q_full[i], 1);
      mbar_init(&s.q_empty[i], 1);
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 4);
    }
    for (int i = 0; i < NST; ++i) {
      mbar_init(&s.kv_full[i], 1);
      mbar_init(&s.kv_empty[i], 1);
    }
    mbar_init(&s.o_done, 1);
    mbar_init(&s.o_free, 8);
    mbar_init(&s.ml_full, 8);
    mbar_init(&s.drain, 1);
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(&s.tmem_base, kTmemCols);
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }

  tc_fence_before();
  const Run run = find_run<kThreads>(s.run, p.B, [&](int b) { return load_seq(p, rw, b).per_head * p.Hkv; });
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const Abort ab{&s.abort_flag, p.status, p.wait_limit};
  Walk w;
  w.begin(p, rw, run.b, run.off, run.run1 - run.run0);
  Unit u{};

  if (warp == kWarpLoad) {
    // ===================================================== TMA producer
    uint32_t seq = 0;  // K/V tiles loaded
    int nq = 0;         // Q tiles loaded
    bool ok = true;
    auto find = [&](const Unit& u, const Seq& q, int tile) {
      return tile < q.nc ? find_box<D>(p.c, u.b, tile * KT, q.len, box_rows) : TileBox{};
    };
    auto load_tile = [&](const CUtensorMap* ctx, const CUtensorMap* fresh, const Unit& u, int nc, int tile,
                         const TileBox& box, uint32_t at) -> bool {
      const int st = (int)(at % NST);
      if (!__all_sync(0xffffffffu, mbar_wait(&s.kv_empty[st], ((at / NST) & 1) ^ 1, ab))) return false;
      if (tile < nc) {
        load_cache_tile<D>(s.kv[st], &s.kv_full[st], ctx, p.c, box, u.hk, box_rows, p.status);
      } else {
        if (lane == 0) {
          mbar_expect_tx(&s.kv_full[st], new_box_rows * KB * 128);
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
            tma_load_4d(s.kv[st] + kb * KT * 128, fresh, &s.kv_full[st], kb * 64, u.hk, (tile - nc) * KT, u.b);
        }
        __syncwarp();
      }
      return true;
    };
    auto advance = [&](Unit& u) {  // to the next unit with something to load
      while (w.next(p, rw, u))
        if (!u.empty) return true;
      return false;
    };
    bool more = advance(u);
    TileBox box{};
    if (more) box = find(u, w.s, u.tb);
    while (more) {
      const Unit v = u;
      const Seq sq = w.s;
      const int n = v.te - v.tb;
      for (int t = 0; ok && t <= (v.two ? 1 : 0); ++t, ++nq) {
        const int slot = nq & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&s.q_empty[slot], ((nq >> 1) & 1) ^ 1, ab));
        if (ok && lane == 0) {
          const int rt = 2 * v.pair + t;
          mbar_expect_tx(&s.q_full[slot], rw.gb * rw.tt * KB * 128);
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
            tma_load_4d(s.q[slot] + kb * BM * 128, &tm_q, &s.q_full[slot], kb * 64,
                        v.hk * rw.G + rt % rw.gblk * rw.gb, rt / rw.gblk * rw.tt, v.b);
        }
        __syncwarp();
      }
      more = advance(u);
      // the order the products consume them in; the next tile's box is looked up
      // before this one's loads wait for their buffers
      TileBox prev{};
      for (int i = 0; ok && i <= n; ++i) {
        const TileBox cur = box;
        if (i + 1 < n)
          box = find(v, sq, v.tb + i + 1);
        else if (i + 1 == n && more)
          box = find(u, w.s, u.tb);
        if (v.two) {
          if (i == n) break;
          if (!(ok = load_tile(&tm_k, &tm_kn, v, sq.nc, v.tb + i, cur, seq + seq_k(true, i)))) break;
          ok = load_tile(&tm_v, &tm_vn, v, sq.nc, v.tb + i, cur, seq + seq_v(true, i, n));
        } else {
          if (i < n && !(ok = load_tile(&tm_k, &tm_kn, v, sq.nc, v.tb + i, cur, seq + seq_k(false, i)))) break;
          if (i > 0) ok = load_tile(&tm_v, &tm_vn, v, sq.nc, v.tb + i - 1, prev, seq + seq_v(false, i - 1, n));
          prev = cur;
        }
      }
      if (!ok) break;
      seq += 2 * n;
    }
    if (s.abort_flag) {
      // leave no copy in flight into shared memory that is about to be released:
      // every barrier with a load outstanding completes its current phase
      for (int i = 0; i < NST; ++i) {
        mbar_wait_drain(&s.kv_full[i], 0, p.wait_limit / 64);
        mbar_wait_drain(&s.kv_full[i], 1, p.wait_limit / 64);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_wait_drain(&s.q_full[i], 0, p.wait_limit / 64);
        mbar_wait_drain(&s.q_full[i], 1, p.wait_limit / 64);
      }
    }
  } else if (warp == kWarpMma) {
    // ===================================================== MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16(BM, KT, 0, 0);  // Q: K-major, K tile: K-major
      constexpr uint32_t idesc_pv = idesc_bf16(BM, D, 0, 1);  // P: TMEM, V tile: MN-major
      uint32_t seq = 0;
      int nq = 0, units = 0;
      uint32_t done[2] = {0, 0};  // items of each stream whose P has been taken
      bool ok = true;
      while (ok && w.next(p, rw, u)) {
        if (u.empty) continue;
        const int n = u.te - u.tb, items = u.two ? 2 * n : n;
        for (int t = 0; ok && t <= (u.two ? 1 : 0); ++t)
          ok = mbar_wait(&s.q_full[(nq + t) & 1], ((nq + t) >> 1) & 1, ab);
        for (int m = 0; ok && m <= items; ++m) {
          if (m < items) {
            const int i = u.two ? m >> 1 : m;
            const uint32_t at = seq + seq_k(u.two, i);
            const int st = (int)(at % NST);
            if (!(ok = mbar_wait(&s.kv_full[st], (at / NST) & 1, ab))) break;
            tc_fence_after();
            const uint32_t qa = smem_u32(s.q[(nq + (u.two ? m & 1 : 0)) & 1]), ka = smem_u32(s.kv[st]);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tmem + (m & 1) * 128, sdesc_sw128(qa + (kk >> 2) * (BM * 128) + (kk & 3) * 32, 16, 1024),
                     sdesc_sw128(ka + (kk >> 2) * (KT * 128) + (kk & 3) * 32, 16, 1024), idesc_s, kk > 0);
            mma_commit(&s.s_full[m & 1]);
            if (!u.two || (m & 1)) mma_commit(&s.kv_empty[st]);
            // the last S of a Q tile frees it
            if (u.two ? m >= items - 2 : m == items - 1) mma_commit(&s.q_empty[(nq + (u.two ? m & 1 : 0)) & 1]);
          }
          if (m > 0) {
            const int j = m - 1, i = u.two ? j >> 1 : j, str = j & 1;
            const uint32_t at = seq + seq_v(u.two, i, n);
            const int st = (int)(at % NST);
            const bool first = j < 2;
            // the previous unit's O has been read
            if (j == 0 && units > 0 && !(ok = mbar_wait(&s.o_free, (units - 1) & 1, ab))) break;
            if (!(ok = mbar_wait(&s.kv_full[st], (at / NST) & 1, ab))) break;
            if (!(ok = mbar_wait(&s.p_full[str], done[str] & 1, ab))) break;
            ++done[str];
            tc_fence_after();
            const uint32_t va = smem_u32(s.kv[st]);
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk)
              mma_ts(tmem + 256 + str * D, tmem + str * 128 + kk * 8, sdesc_sw128(va + kk * 2048, KT * 128, 1024),
                     idesc_pv, !first || kk > 0);
            if (!u.two || (j & 1)) mma_commit(&s.kv_empty[st]);
            if (j == items - 1) mma_commit(&s.o_done);
          }
        }
        seq += 2 * n;
        nq += u.two ? 2 : 1;
        ++units;
      }
      // TMEM must be quiescent before it is released
      mma_commit(&s.drain);
      mbar_wait_drain(&s.drain, 0, p.wait_limit);
    }
  } else {
    // ===================================================== softmax warpgroups
    const int str = warp >> 2;     // stream
    const int quarter = warp & 3;  // TMEM lanes [32 quarter, +32)
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t col_s = tmem + lane_off + str * 128;
    const uint32_t col_o = tmem + lane_off + 256;
    const float sc2 = p.scale * kLog2e;
    const int rows_in_tile = rw.gb * rw.tt;
    uint32_t seq = 0;
    uint32_t seen = 0;  // items of this stream
    int units = 0, singles = 0;
    bool ok = true;
    while (ok && w.next(p, rw, u)) {
      const int n = u.te - u.tb, items = u.empty ? 0 : (u.two ? 2 * n : n);
      const int len = w.s.len, nr = w.s.nr, nc = w.s.nc;
      const int rt = 2 * u.pair + (u.two ? str : 0);
      const int t = rt / rw.gblk * rw.tt + r / rw.gb, g = rt % rw.gblk * rw.gb + r % rw.gb;
      const bool in_q = r < rows_in_tile && t < p.Nq && g < rw.G;  // a row of q
      const bool live = in_q && t < nr;
      const bool warp_live = __any_sync(0xffffffffu, live);
      const unsigned long long* mrow =
          p.mask && live ? p.mask + u.b * p.mask_bstride + (long long)t * p.mask_words : nullptr;
      float m = -INFINITY, l = 0.f;
      for (int it = str; it < items; it += 2, ++seen) {
        const int i = u.two ? it >> 1 : it, tile = u.tb + i;
        ok = __all_sync(0xffffffffu, mbar_wait(&s.s_full[str], seen & 1, ab));
        if (!ok) break;
        const bool cached = tile < nc;
        const int base = (cached ? tile : tile - nc) * KT;
        const int keys = min(KT, (cached ? len : nr) - base);  // keys of this tile that exist
        if (keys < KT && (!u.two || str == 0)) {
          // V rows that do not exist take part with P = 0: they have to be finite
          const uint32_t at = seq + seq_v(u.two, i, n);
          const int st = (int)(at % NST);
          ok = __all_sync(0xffffffffu, mbar_wait(&s.kv_full[st], (at / NST) & 1, ab));
          if (!ok) break;
          if (r >= keys) {
            const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(s.kv[st] + kb * KT * 128 + r * 128 + c * 16) = z;
          }
          fence_proxy_async_smem();
        }
        if (warp_live) {
          tc_fence_after();
          // which keys of an edge tile the row sees: those below hi, of a drafted
          // tree those of its mask words too
          const bool edge = !cached || keys < KT;
          uint32_t bits[4];
          if (edge) {
            const int hi = cached || mrow ? keys : min(keys, t + 1 - base);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int c = hi - 32 * x;
              bits[x] = c >= 32 ? 0xffffffffu : (c <= 0 ? 0u : (1u << c) - 1u);
            }
            if (!cached && mrow) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int word = base / 64 + x;
                const unsigned long long mw = word < p.mask_words ? __ldg(mrow + word) : 0ull;
                bits[2 * x] &= (uint32_t)mw;
                bits[2 * x + 1] &= (uint32_t)(mw >> 32);
              }
            }
          }
          // half a row of scores in base-2 units, hidden ones at -inf
          uint32_t sr[KT / 2];
          auto load_half = [&](int half) {
            tmem_ld32(col_s + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
            tmem_ld32(col_s + 64 * half + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
            tmem_wait_ld();
            reg_fence(sr);
#pragma unroll
            for (int c = 0; c < KT / 2; ++c) sr[c] = __float_as_uint(__uint_as_float(sr[c]) * sc2);
            if (edge) {
              const uint32_t lo = half ? bits[2] : bits[0], hi = half ? bits[3] : bits[1];
#pragma unroll
              for (int c = 0; c < KT / 2; ++c)
                if (!(((c < 32 ? lo : hi) >> (c & 31)) & 1u)) sr[c] = 0xff800000u;  // -inf
            }
          };
          float mx0 = -INFINITY, mx1 = -INFINITY;
          auto max_half = [&]() {
#pragma unroll
            for (int c = 0; c < KT / 2; c += 2) {
              mx0 = fmaxf(mx0, __uint_as_float(sr[c]));
              mx1 = fmaxf(mx1, __uint_as_float(sr[c + 1]));
            }
          };
          // the second half is read twice, which takes half the registers of one
          // read (128 scores at once spill); P of the first half overwrites only
          // scores that are in registers
          load_half(1);
          max_half();
          load_half(0);
          max_half();
          const float mx = fmaxf(mx0, mx1);
          const bool move = mx > m + kRescaleThreshold;
          const float m_next = move ? mx : m;
          const float alpha = move ? ex2(m - m_next) : 1.f;
          const float neg_m = m_next == -INFINITY ? 0.f : -m_next;
          float rs0 = 0.f, rs1 = 0.f;
          auto store_half = [&](int half) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float p0 = ex2(__uint_as_float(sr[c * 32 + 2 * e]) + neg_m);
                const float p1 = ex2(__uint_as_float(sr[c * 32 + 2 * e + 1]) + neg_m);
                rs0 += p0;
                rs1 += p1;
                pk[e] = pack_bf16(p0, p1);  // the product's operand; the sum l keeps 32 bits
              }
              tmem_st16(col_s + half * 32 + c * 16, pk);
            }
          };
          store_half(0);
          load_half(1);
          store_half(1);
          l = l * alpha + (rs0 + rs1);
          m = m_next;
          if (it >= 2 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t orr[32];
              tmem_ld32(col_o + str * D + c * 32, orr);
              tmem_wait_ld();
              reg_fence(orr);
#pragma unroll
              for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
              tmem_st32(col_o + str * D + c * 32, orr);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[str]);
      }
      if (!ok) break;
      if (!u.empty) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s.o_done, units & 1, ab));
        if (!ok) break;
        tc_fence_after();
      }
      // ---- epilogue.  One row tile: the two streams' states merge, and each
      // warpgroup writes its half of the columns; two: each writes its own rows.
      float a0 = 1.f, a1 = 1.f;
      if (!u.empty && !u.two) {
        s.ml[str][r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.ml_full);
        ok = __all_sync(0xffffffffu, mbar_wait(&s.ml_full, singles & 1, ab));
        if (!ok) break;
        ++singles;
        const float2 x0 = s.ml[0][r], x1 = s.ml[1][r];
        m = fmaxf(x0.x, x1.x);
        a0 = x0.x == -INFINITY ? 0.f : ex2(x0.x - m);
        a1 = x1.x == -INFINITY ? 0.f : ex2(x1.x - m);
        // a score of NaN leaves m at -inf and l at NaN: keep the NaN
        l = (x0.x == -INFINITY ? x0.y : x0.y * a0) + (x1.x == -INFINITY ? x1.y : x1.y * a1);
      }
      if (!live) {
        m = -INFINITY;
        l = 0.f;
      }
      const bool whole = u.tb == 0 && u.te == u.n;
      const bool none = l == 0.f;  // sees no key
      const float inv = none ? 0.f : 1.f / l;
      const int c0 = u.two ? 0 : str * (D / 2), c1 = u.two ? D : c0 + D / 2;
      const long long orow = ((long long)u.b * p.Nq + t) * p.Hq + u.hk * rw.G + g;
      const int slot = (int)blockIdx.x * 2 + (u.tb > 0 ? 0 : 1);
      const long long prow = ((long long)slot * p.part_tiles + (u.two ? str : 0)) * rows_in_tile + r;
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        float x[32];
        if (warp_live && !u.empty) {
          uint32_t v[32];
          if (u.two) {
            tmem_ld32(col_o + str * D + c, v);
            tmem_wait_ld();
            reg_fence(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(v[e]);
          } else {
            tmem_ld32(col_o + c, v);
            tmem_wait_ld();
            reg_fence(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(v[e]) * a0;
            if (n > 1) {  // the second stream had a tile
              tmem_ld32(col_o + D + c, v);
              tmem_wait_ld();
              reg_fence(v);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(v[e]), a1, x[e]);
            }
          }
        }
        if (in_q) {
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = none ? 0.f : x[e] * inv;
            store_bf16_32(static_cast<__nv_bfloat16*>(p.o) + orow * D + c, x);
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(p.o_part + prow * D + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        }
      }
      if (in_q && (u.two || str == 0)) {
        if (whole)
          p.lse[((long long)u.b * p.Hq + u.hk * rw.G + g) * p.Nq + t] = none ? -INFINITY : (m + log2f(l)) * kLn2;
        else
          reinterpret_cast<float2*>(p.lse_part)[prow] = make_float2(m, l);
      }
      // a second row tile that is all padding
      if (!u.two && u.tb == 0 && 2 * u.pair + 1 < rw.tiles && str == 0) {
        const int rt2 = 2 * u.pair + 1;
        const int t2 = rt2 / rw.gblk * rw.tt + r / rw.gb, g2 = rt2 % rw.gblk * rw.gb + r % rw.gb;
        if (r < rows_in_tile && t2 < p.Nq && g2 < rw.G) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) +
                                                (((long long)u.b * p.Nq + t2) * p.Hq + u.hk * rw.G + g2) * D);
          for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0, 0, 0, 0);
          p.lse[((long long)u.b * p.Hq + u.hk * rw.G + g2) * p.Nq + t2] = -INFINITY;
        }
      }
      if (!u.empty) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o_free);
        ++units;
        seq += 2 * n;
      }
    }
  }

  // ---- teardown; the merge may be launched (it waits for this grid's end)
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
    TreeCut cut{0, 0, 0, 0};
    if (run.run1 > run.run0 && u.tb == 0 && u.te < u.n)
      cut = TreeCut{u.b, u.hk, u.pair * 2 + u.two, run_parts(run, u.n - u.te)};
    p.cuts[blockIdx.x] = cut;
  }
}

// Combine the partials of the units that a cut divides.  Block (c, y): the unit
// whose first part CTA c holds (second slot) and whose others are the first
// slots of CTAs c + 1 .. c + more; a warp per row, a lane per D / 32 columns:
//   m = max m_i, l = sum 2^(m_i - m) l_i, O = sum 2^(m_i - m) O_i / l.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams p) {
  constexpr int E = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const TreeCut cut = p.cuts[blockIdx.x];
  if (cut.more == 0) return;
  const Rows rw = row_tiles(p.Hq, p.Hkv, p.Nq);
  const int rows = rw.gb * rw.tt, lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5), tile = row / rows, r = row % rows;
  if (tile > (cut.pair2 & 1)) return;
  const int rt = (cut.pair2 >> 1) * 2 + tile;
  const int t = rt / rw.gblk * rw.tt + r / rw.gb, g = rt % rw.gblk * rw.gb + r % rw.gb;
  if (t >= p.Nq || g >= rw.G) return;
  const float2* ml = reinterpret_cast<const float2*>(p.lse_part);
  auto part_row = [&](int i) {
    return ((long long)((blockIdx.x + i) * 2 + (i == 0)) * p.part_tiles + tile) * rows + r;
  };
  float m = -INFINITY;
  for (int i = lane; i <= cut.more; i += 32) m = fmaxf(m, ml[part_row(i)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i <= cut.more; ++i) {
    const long long at = part_row(i);
    const float2 x = ml[at];
    if (x.y == 0.f) continue;  // sees no key of this part; nothing was stored
    const float w = x.x == -INFINITY ? 1.f : ex2(x.x - m);  // NaN scores: m_i = -inf, l_i = NaN
    l = fmaf(w, x.y, l);
    const float* src = p.o_part + at * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 o2 = *reinterpret_cast<const float2*>(src + e);
      acc[e] = fmaf(w, o2.x, acc[e]);
      acc[e + 1] = fmaf(w, o2.y, acc[e + 1]);
    }
  }
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) +
                     (((long long)cut.b * p.Nq + t) * p.Hq + cut.hk * rw.G + g) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0)
    p.lse[((long long)cut.b * p.Hq + cut.hk * rw.G + g) * p.Nq + t] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

template <int D>
int launch_t(TreeParams p, const Rows& rw, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mkn, mvn;
  const uint64_t B = p.B, Hq = p.Hq, Hkv = p.Hkv, Nq = p.Nq, S = p.c.page_size;
  const uint64_t rq = Hq * D * 2, rk = Hkv * D * 2;
  const uint64_t qd[4] = {D, Hq, Nq, B}, qs[3] = {D * 2, rq, rq * Nq};
  const uint32_t qb[4] = {64, (uint32_t)rw.gb, (uint32_t)rw.tt, 1};
  const uint64_t kd[4] = {D, Hkv, S, (uint64_t)p.c.num_pages}, ks[3] = {D * 2, rk, rk * S};
  const int box = cache_box_rows(p.c);
  const uint32_t kb[4] = {64, 1, (uint32_t)box, 1};
  const int nbox = std::min(KT, (p.Nq + 7) / 8 * 8);
  const uint64_t nd[4] = {D, Hkv, Nq, B}, ns[3] = {D * 2, rk, rk * Nq};
  const uint32_t nb[4] = {64, 1, (uint32_t)nbox, 1};
  int rc;
  if ((rc = encode_tmap_bf16(&mq, p.q, 4, qd, qs, qb))) return rc;
  if ((rc = encode_tmap_bf16(&mk, p.c.k, 4, kd, ks, kb))) return rc;
  if ((rc = encode_tmap_bf16(&mv, p.c.v, 4, kd, ks, kb))) return rc;
  std::memset(&mkn, 0, sizeof(mkn));
  std::memset(&mvn, 0, sizeof(mvn));
  if (p.k_new) {
    if ((rc = encode_tmap_bf16(&mkn, p.k_new, 4, nd, ns, nb))) return rc;
    if ((rc = encode_tmap_bf16(&mvn, p.v_new, 4, nd, ns, nb))) return rc;
  }
  const size_t smem = sizeof(TreeSmem<D>) + 1024;
  static_assert(sizeof(TreeSmem<D>) + 1024 <= 232448, "shared memory");
  if (cudaFuncSetAttribute(tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATTN_ERR_CUDA;
  const unsigned ctas = sm_count();
  tree_kernel<D><<<ctas, kThreads, smem, st>>>(mq, mk, mv, mkn, mvn, p, box, nbox);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  // the merge's launch overlaps the end of the kernel above and waits for it
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, (unsigned)((rw.gb * rw.tt * p.part_tiles + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, (const TreeParams)p) != cudaSuccess) return ATTN_ERR_CUDA;
  count_launch(2);
  return ATTN_OK;
}

}  // namespace

// Two slots per CTA (the unit its run begins in, the unit it ends in) of one or
// two row tiles, and one cut record per CTA.
size_t tree_sm100_workspace(int Hq, int Hkv, int Nq, int D) {
  const Rows rw = row_tiles(Hq, Hkv, Nq);
  const size_t rows = (size_t)sm_count() * 2 * (rw.tiles > 1 ? 2 : 1) * rw.gb * rw.tt;
  return align256(rows * D * 4) + align256(rows * 8) + align256((size_t)sm_count() * sizeof(TreeCut));
}

int launch_tree_sm100(TreeParams p, void* workspace, cudaStream_t st) {
  const Rows rw = row_tiles(p.Hq, p.Hkv, p.Nq);
  p.part_tiles = rw.tiles > 1 ? 2 : 1;
  p.wait_limit = kWaitLimitCycles;
  const size_t rows = (size_t)sm_count() * 2 * p.part_tiles * rw.gb * rw.tt;
  char* ws = static_cast<char*>(workspace);
  p.o_part = reinterpret_cast<float*>(ws);
  p.lse_part = reinterpret_cast<float*>(ws + align256(rows * p.D * 4));
  p.cuts = reinterpret_cast<TreeCut*>(ws + align256(rows * p.D * 4) + align256(rows * 8));
  return p.D == 64 ? launch_t<64>(p, rw, st) : launch_t<128>(p, rw, st);
}

}  // namespace attn
