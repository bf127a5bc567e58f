// Tree attention over a key/value cache on sm_100a tensor cores (bf16) for more than
// 16 query rows per (sequence, KV head), and the combination of partials that both
// kernels leave (tree_few_sm100.cu has up to 16 rows).
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
#include <type_traits>

#include "tree.cuh"

namespace attn {

namespace {

constexpr int KT = kTreeKeys;  // keys per tile
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
  RunSmem<kThreads, 1> run;
  uint32_t tmem_base;
  int abort_flag;
};

// Position of K / V tile i of a unit of `n` tiles in the order of its loads
// (K_i before S(i), V_i before the product with P(i)).
ATTN_DEVINL int seq_k(bool two, int i) { return two ? 2 * i : (i == 0 ? 0 : 2 * i - 1); }
ATTN_DEVINL int seq_v(bool two, int i, int n) { return two ? 2 * i + 1 : (i == n - 1 ? 2 * n - 1 : 2 * i + 2); }

// One key tile of one row: scores from TMEM, the reference maximum m moved when
// the tile's exceeds it by more than 2^8, P over the scores.  EDGE: keys whose
// bit is clear are hidden, whatever their score.
struct SoftmaxStep {
  float m, alpha, sum;  // alpha = 2^(old m - m); sum of the tile's P
};

template <bool EDGE>
ATTN_DEVINL SoftmaxStep softmax_tile(uint32_t col_s, uint64_t sc2, float m, const uint32_t (&bits)[4]) {
  // half a row of scores, x = s * scale * log2(e) in pairs
  uint64_t x[KT / 4];
  auto load_half = [&](int half) {
    uint32_t sr[KT / 2];
    tmem_ld32(col_s + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
    tmem_ld32(col_s + 64 * half + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
    tmem_wait_ld();
    reg_fence(sr);
    const uint32_t lo = half ? bits[2] : bits[0], hi = half ? bits[3] : bits[1];
#pragma unroll
    for (int c = 0; c < KT / 2; c += 2) {
      uint64_t y = fma_f32x2(pack_f32x2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sc2, 0ull);
      if constexpr (EDGE) {
        float y0, y1;
        unpack_f32x2(y, y0, y1);
        const uint32_t b = (c < 32 ? lo : hi) >> (c & 31);
        y = pack_f32x2(b & 1u ? y0 : -INFINITY, b & 2u ? y1 : -INFINITY);
      }
      x[c / 2] = y;
    }
  };
  float mx0 = -INFINITY, mx1 = -INFINITY;
  auto max_half = [&]() {
#pragma unroll
    for (int c = 0; c < KT / 4; c += 2) {
      float a, b, d, e;
      unpack_f32x2(x[c], a, b);
      unpack_f32x2(x[c + 1], d, e);
      mx0 = fmaxf(mx0, fmaxf(a, b));
      mx1 = fmaxf(mx1, fmaxf(d, e));
    }
  };
  // the second half is read twice, which takes half the registers of one read
  // (128 scores at once spill); P of the first half overwrites only scores that
  // are in registers
  load_half(1);
  max_half();
  load_half(0);
  max_half();
  SoftmaxStep r;
  const float mx = fmaxf(mx0, mx1);
  const bool move = mx > m + kRescaleThreshold;
  r.m = move ? mx : m;
  r.alpha = move ? ex2(m - r.m) : 1.f;
  const float neg_m = r.m == -INFINITY ? 0.f : -r.m;
  const uint64_t nm = pack_f32x2(neg_m, neg_m);
  uint64_t sum0 = 0, sum1 = 0;
  auto store_half = [&](int half) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float y0, y1;
        unpack_f32x2(add_f32x2(x[c * 16 + e], nm), y0, y1);
        const float p0 = ex2(y0), p1 = ex2(y1);
        uint64_t& sum = e & 1 ? sum1 : sum0;
        sum = add_f32x2(sum, pack_f32x2(p0, p1));
        pk[e] = pack_bf16(p0, p1);  // the product's operand; the sum l keeps 32 bits
      }
      tmem_st16(col_s + half * 32 + c * 16, pk);
    }
  };
  store_half(0);
  load_half(1);
  store_half(1);
  float y0, y1;
  unpack_f32x2(add_f32x2(sum0, sum1), y0, y1);
  r.sum = y0 + y1;
  return r;
}

// (a call of its own: it is rare, and its registers would be the loop's)
__device__ __noinline__ SoftmaxStep softmax_edge_tile(uint32_t col_s, uint64_t sc2, float m, uint32_t b0, uint32_t b1,
                                                      uint32_t b2, uint32_t b3) {
  const uint32_t bits[4] = {b0, b1, b2, b3};
  return softmax_tile<true>(col_s, sc2, m, bits);
}

// O of a row times alpha (likewise).
template <int D>
__device__ __noinline__ void rescale_row(uint32_t col_o, float alpha) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t v[32];
    tmem_ld32(col_o + c, v);
    tmem_wait_ld();
    reg_fence(v);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
    tmem_st32(col_o + c, v);
  }
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
                const __grid_constant__ CUtensorMap tm_vn, const TreeParams p, const TileForm form,
                const TileForm new_form) {
  using Smem = TreeSmem<D>;
  constexpr int NST = Smem::NST;
  constexpr int KB = D / 64;  // 128-byte blocks per row
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RowTiles& rw = p.rw;

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
  find_runs<kThreads, 1>(s.run, p.B, rw.tiles > 1 ? 2 : 1, [&](int b) { return tree_seq(p, rw, b).per_head * p.Hkv; });
  tc_fence_after();
  const Runs<1>& runs = s.run.runs;
  const Run& run = runs.lane[0];
  const uint32_t tmem = s.tmem_base;
  const Abort ab{&s.abort_flag, p.status, p.wait_limit};
  TreeWalk w;
  w.begin(p, rw, run);
  TreeUnit u{};

  if (warp == kWarpLoad) {
    // ===================================================== TMA producer
    uint32_t seq = 0;  // K/V tiles loaded
    int nq = 0;         // Q tiles loaded
    bool ok = true;
    TreeBoxes boxes;
    auto find = [&](const TreeUnit& u, const TreeSeq& q, int tile) {
      return boxes.find(p, form, new_form, q, u.b, tile, tile == u.tb);
    };
    auto load = [&](const CUtensorMap* ctx, const CUtensorMap* fresh, const TreeUnit& u, int nc, int tile,
                    const TileBox& box, uint32_t at) -> bool {
      const int st = (int)(at % NST);
      if (!__all_sync(0xffffffffu, mbar_wait(&s.kv_empty[st], ((at / NST) & 1) ^ 1, ab))) return false;
      if (tile < nc)
        load_tile<D>(s.kv[st], &s.kv_full[st], ctx, form, box, u.hk, p.c.num_pages, p.status);
      else
        load_tile<D>(s.kv[st], &s.kv_full[st], fresh, new_form, box, u.hk, p.B, p.status);
      return true;
    };
    auto advance = [&](TreeUnit& u) {  // to the next unit with something to load
      while (w.next(p, rw, u))
        if (!u.empty) return true;
      return false;
    };
    bool more = advance(u);
    TileBox box{};
    if (more) box = find(u, w.s, u.tb);
    while (more) {
      const TreeUnit v = u;
      const TreeSeq sq = w.s;
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
      // the order the products consume them in; the next tile's box is looked up
      // between this one's loads
      TileBox prev{};
      for (int i = 0; ok && i <= n; ++i) {
        const TileBox cur = box;
        if (i < n && !(ok = load(&tm_k, &tm_kn, v, sq.nc, v.tb + i, cur, seq + seq_k(v.two, i)))) break;
        if (i + 1 < n) {
          box = find(v, sq, v.tb + i + 1);
        } else if (i + 1 == n) {
          more = advance(u);
          if (more) box = find(u, w.s, u.tb);
        }
        // with two row tiles V follows its K, else the next K
        const int iv = v.two ? i : i - 1;
        if (iv >= 0 && iv < n)
          ok = load(&tm_v, &tm_vn, v, sq.nc, v.tb + iv, v.two ? cur : prev, seq + seq_v(v.two, iv, n));
        prev = cur;
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
      // What the issuing thread does between the MMAs leaves the tensor cores idle,
      // so the streams are unrolled and little is worked out between them.
      uint32_t seq = 0;
      int nq = 0, units = 0;
      uint32_t done0 = 0, done1 = 0;  // items of each stream whose P has been taken
      bool ok = true;
      while (ok && w.next(p, rw, u)) {
        if (u.empty) continue;
        const int n = u.te - u.tb, turns = u.two ? n : (n + 1) / 2;
        const bool two = u.two;
        const uint64_t q0 = sdesc_sw128(smem_u32(s.q[nq & 1]), 16, 1024);
        const uint64_t q1 = two ? sdesc_sw128(smem_u32(s.q[(nq + 1) & 1]), 16, 1024) : q0;
        for (int t = 0; ok && t <= (two ? 1 : 0); ++t)
          ok = mbar_wait(&s.q_full[(nq + t) & 1], ((nq + t) >> 1) & 1, ab);
        // S of stream str over key tile i
        auto scores = [&](auto str_c, int i) {
          constexpr int str = decltype(str_c)::value;
          const uint32_t at = seq + seq_k(two, i);
          const int st = (int)(at % NST);
          if (!(ok = mbar_wait(&s.kv_full[st], (at / NST) & 1, ab))) return;
          tc_fence_after();
          const uint64_t qd = str ? q1 : q0, kd = k_tile_desc<D>(s.kv[st]);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + str * 128, sdesc_at(qd, (kk >> 2) * (BM * 128) + (kk & 3) * 32), k_tile_step(kd, kk), idesc_s,
                   kk > 0);
          mma_commit(&s.s_full[str]);
          if (!two || str == 1) mma_commit(&s.kv_empty[st]);
          if (i == n - 1) mma_commit(&s.q_empty[(nq + (two ? str : 0)) & 1]);  // the last S of a Q tile frees it
        };
        // O of stream str += P V_i; first: its first of the unit
        auto product = [&](auto str_c, int i, bool first) {
          constexpr int str = decltype(str_c)::value;
          if (!ok) return;
          // the previous unit's O has been read
          if (str == 0 && first && units > 0 && !(ok = mbar_wait(&s.o_free, (units - 1) & 1, ab))) return;
          const uint32_t at = seq + seq_v(two, i, n);
          const int st = (int)(at % NST);
          uint32_t& done = str ? done1 : done0;
          // (V first: it is there as a rule, and is looked at while P is not)
          if (!(ok = mbar_wait(&s.kv_full[st], (at / NST) & 1, ab))) return;
          if (!(ok = mbar_wait(&s.p_full[str], done & 1, ab))) return;
          ++done;
          tc_fence_after();
          const uint64_t vd = v_tile_desc<D>(s.kv[st]);
          const uint32_t accum = !first;
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            mma_ts(tmem + 256 + str * D, tmem + str * 128 + kk * 8, v_tile_step<D>(vd, kk), idesc_pv, kk > 0 ? 1u : accum);
          if (!two || str == 1) mma_commit(&s.kv_empty[st]);
        };
        const std::integral_constant<int, 0> s0;
        const std::integral_constant<int, 1> s1;
        for (int k = 0; ok && k < turns; ++k) {
          scores(s0, two ? k : 2 * k);
          if (k > 0) product(s1, two ? k - 1 : 2 * k - 1, k == 1);
          if (ok && (two || 2 * k + 1 < n)) scores(s1, two ? k : 2 * k + 1);
          product(s0, two ? k : 2 * k, k == 0);
        }
        if (two || n % 2 == 0) product(s1, n - 1, turns == 1);
        if (!ok) break;
        mma_commit(&s.o_done);
        seq += 2 * n;
        nq += two ? 2 : 1;
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
    const uint64_t sc2 = pack_f32x2(p.scale * kLog2e, p.scale * kLog2e);
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
        if (warp_live) {
          tc_fence_after();
          // which keys of an edge tile the row sees: those below hi, of a drafted
          // tree those of its mask words too
          const bool edge = !cached || keys < KT;
          uint32_t bits[4] = {0, 0, 0, 0};
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
          const SoftmaxStep st = edge ? softmax_edge_tile(col_s, sc2, m, bits[0], bits[1], bits[2], bits[3])
                                      : softmax_tile<false>(col_s, sc2, m, bits);
          const float alpha = st.alpha;
          l = l * alpha + st.sum;
          m = st.m;
          if (it >= 2 && __any_sync(0xffffffffu, alpha != 1.f)) {
            rescale_row<D>(col_o + str * D, alpha);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        if (keys < KT && (!u.two || str == 0)) {
          // V rows that do not exist take part with P = 0: they have to be finite
          // (of two row tiles the first one's product comes first)
          const uint32_t at = seq + seq_v(u.two, i, n);
          const int st = (int)(at % NST);
          ok = __all_sync(0xffffffffu, mbar_wait(&s.kv_full[st], (at / NST) & 1, ab));
          if (!ok) break;
          if (r >= keys) zero_slot<D>(s.kv[st], r);
          fence_proxy_async_smem();
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
    TreeCut cut{0, 0, 0, 0, 0};
    if (!s.abort_flag && run.run1 > run.run0 && u.tb == 0 && u.te < u.n)
      cut = TreeCut{u.b, u.hk, u.pair, u.two ? 2 : 1, run_parts(runs.total, runs.workers, blockIdx.x, run.run1, u.rest)};
    p.cuts[blockIdx.x] = cut;
  }
}

// Combine the partials of the units that a cut divides.  Block (w, y): the unit
// whose first part worker w holds (second slot) and whose others are the first
// slots of workers w + 1 .. w + more; a warp per row, a lane per D / 32 columns:
//   m = max m_i, l = sum 2^(m_i - m) l_i, O = sum 2^(m_i - m) O_i / l.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams p) {
  constexpr int E = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const TreeCut cut = p.cuts[blockIdx.x];
  if (cut.more == 0) return;
  const RowTiles& rw = p.rw;
  const int rows = rw.gb * rw.tt, lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5), tile = row / rows, r = row % rows;
  if (tile >= cut.tiles) return;
  const int rt = 2 * cut.pair + tile;
  const int t = rt / rw.gblk * rw.tt + r / rw.gb, g = rt % rw.gblk * rw.gb + r % rw.gb;
  if (t >= p.Nq || g >= rw.G) return;
  const float2* ml = reinterpret_cast<const float2*>(p.lse_part);
  auto part_row = [&](int i) {
    return ((long long)((blockIdx.x + i) * 2 + (i == 0)) * p.part_tiles + tile) * rows + r;
  };
  // 32 parts at a time, a lane per part for its (m, l); a part's weight is 0 when
  // none of its keys is seen (nothing was stored then)
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 <= cut.more; i0 += 32) {
    const int n = min(32, cut.more + 1 - i0);
    const float2 x = lane < n ? ml[part_row(i0 + lane)] : make_float2(-INFINITY, 0.f);
    float mx = x.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float m2 = fmaxf(m, mx), a = m == -INFINITY ? 1.f : ex2(m - m2);
    // NaN scores: m_i = -inf and l_i = NaN
    const float w = x.y == 0.f ? 0.f : (x.x == -INFINITY ? 1.f : ex2(x.x - m2));
    float part = w * x.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    l = fmaf(l, a, part);
    m = m2;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= a;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* src = p.o_part + part_row(i0 + i) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float2 o2 = make_float2(0.f, 0.f);
        if (wi != 0.f) o2 = *reinterpret_cast<const float2*>(src + e);
        acc[e] = fmaf(wi, o2.x, acc[e]);
        acc[e + 1] = fmaf(wi, o2.y, acc[e + 1]);
      }
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

template <int D>
int launch_wide(const TreeParams& p, const TreeMaps& m, cudaStream_t st) {
  const size_t smem = sizeof(TreeSmem<D>) + 1024;
  static_assert(sizeof(TreeSmem<D>) + 1024 <= 232448, "shared memory");
  if (cudaFuncSetAttribute(tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATTN_ERR_CUDA;
  tree_kernel<D><<<sm_count(), kThreads, smem, st>>>(m.q, m.k, m.v, m.k_new, m.v_new, p, m.form, m.new_form);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// The merge's launch overlaps the end of the kernel before it, whose end it waits for.
template <int D>
int launch_merge_parts(const TreeParams& p, int workers, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)workers, (unsigned)((p.rw.gb * p.rw.tt * p.part_tiles + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int make_maps(const TreeParams& p, TreeMaps& m) {
  const uint64_t D = p.D, B = p.B, Hq = p.Hq, Nq = p.Nq, rq = Hq * D * 2;
  const uint64_t qd[4] = {D, Hq, Nq, B}, qs[3] = {D * 2, rq, rq * Nq};
  const uint32_t qb[4] = {64, (uint32_t)p.rw.gb, (uint32_t)p.rw.tt, 1};
  int rc;
  if ((rc = encode_tmap_bf16(&m.q, p.q, 4, qd, qs, qb))) return rc;
  if ((rc = cache_tile_map(&m.k, &m.form, p.c, p.c.k, p.Hkv, p.D))) return rc;
  if ((rc = cache_tile_map(&m.v, &m.form, p.c, p.c.v, p.Hkv, p.D))) return rc;
  std::memset(&m.k_new, 0, sizeof(m.k_new));
  std::memset(&m.v_new, 0, sizeof(m.v_new));
  m.new_form = TileForm{};
  if (p.k_new) {
    if ((rc = rows_tile_map(&m.k_new, &m.new_form, p.k_new, p.Hkv, p.D, p.Nq, p.B))) return rc;
    if ((rc = rows_tile_map(&m.v_new, &m.new_form, p.v_new, p.Hkv, p.D, p.Nq, p.B))) return rc;
  }
  return ATTN_OK;
}

RowTiles row_tiles(int Hq, int Hkv, int Nq) {
  RowTiles r{};
  r.G = Hq / Hkv;
  r.gb = std::min(r.G, BM);
  r.gblk = (r.G + r.gb - 1) / r.gb;
  const int fit = BM / r.gb;  // tokens that fit a tile
  int blocks = (Nq + fit - 1) / fit;
  if (blocks > 1 && r.gblk == 1) blocks = (blocks + 1) / 2 * 2;  // pairs: the same passes over K and V
  r.tt = (Nq + blocks - 1) / blocks;
  r.tiles = (Nq + r.tt - 1) / r.tt * r.gblk;
  return r;
}

// Rows up to which the transposed kernel (tree_few_sm100.cu) is taken.  At 4 rows, 64
// sequences: 204 us against 219 here at 300 .. 8191 slots, 78 against 96 at 1024, 50
// against 67 at about 250.  A transposed form of 32 rows took 152 us against 130 here at
// 8 tokens of 4 heads: its P and O columns cost more than the rows that are padding here.
constexpr int kFewRows = 16;
// Tiles that a unit's ends count for in the two kernels.  Here 16 sequences of 2000 ..
// 12345 slots with up to 61 tokens took 169 us with 4, 163 with 6, 157 with 8, 163 with
// 12; 32 tokens 145 with 0 and 136 with 2 to 8.  The other kernel's two workers per
// CTA cover for each other: 4 sequences of 16 heads with two rows took 26 us with 4,
// 27 .. 35 with 6 to 12.
constexpr int kUnitCost = 8, kFewUnitCost = 4;

// Two slots per worker (the unit its run begins in, the unit it ends in): few rows,
// two workers per CTA and one row tile; else one worker and one or two.
struct Layout {
  RowTiles rw;
  int workers, part_tiles;
  size_t rows, o_bytes, ml_bytes, total;
};

Layout layout(int Hq, int Hkv, int Nq, int D) {
  auto align256 = [](size_t x) { return (x + 255) & ~size_t(255); };
  Layout a;
  a.rw = row_tiles(Hq, Hkv, Nq);
  const bool few = a.rw.tiles == 1 && a.rw.gb * a.rw.tt <= kFewRows;
  a.workers = sm_count() * (few ? 2 : 1);
  a.part_tiles = a.rw.tiles > 1 ? 2 : 1;
  a.rows = (size_t)a.workers * 2 * a.part_tiles * a.rw.gb * a.rw.tt;
  a.o_bytes = align256(a.rows * D * 4);
  a.ml_bytes = align256(a.rows * 8);
  a.total = a.o_bytes + a.ml_bytes + align256(a.workers * sizeof(TreeCut));
  return a;
}

int tile_map(CUtensorMap* map, TileForm* form, const void* base, int Hkv, int D, uint64_t rows, uint64_t pages,
             int box_rows) {
  const uint64_t rk = (uint64_t)Hkv * D * 2, KB = D / 64;
  // with one 64-element block per row groups lie end to end, as rows do
  form->grouped = KB > 1 && rows % 8 == 0;
  if (!form->grouped && KB > 1) box_rows = 8;
  form->shift = 0;
  while (1 << form->shift < box_rows) ++form->shift;
  form->dp = 0;
  form->ds = KT;
  const uint64_t dims[5] = {64, form->grouped ? 8 : rows, Hkv * KB, form->grouped ? rows / 8 : 1, pages};
  const uint64_t strides[4] = {rk, 128, form->grouped ? rk * 8 : rk * rows, rk * rows};
  const uint32_t box[5] = {64, form->grouped ? 8u : (uint32_t)box_rows, (uint32_t)KB,
                           form->grouped ? (uint32_t)box_rows / 8 : 1u, 1};
  return encode_tmap_bf16(map, base, 5, dims, strides, box);
}

}  // namespace

// Boxes never straddle a page: the largest power of two that divides it.
int cache_tile_map(CUtensorMap* map, TileForm* form, const CacheView& c, const void* base, int Hkv, int D) {
  int box = KT;
  if (c.table)
    while (c.page_size % box) box >>= 1;
  const int rc = tile_map(map, form, base, Hkv, D, c.page_size, c.num_pages, box);
  if (c.table) {
    form->dp = KT / c.page_size;
    form->ds = KT % c.page_size;
  }
  return rc;
}

// Few rows in all: boxes of a power of two that holds them.
int rows_tile_map(CUtensorMap* map, TileForm* form, const void* base, int Hkv, int D, int n, int batch) {
  int box = KT;
  while (box > 8 && box / 2 >= n) box >>= 1;
  return tile_map(map, form, base, Hkv, D, n, batch, box);
}

size_t tree_sm100_workspace(int Hq, int Hkv, int Nq, int D) { return layout(Hq, Hkv, Nq, D).total; }

int launch_tree_sm100(TreeParams p, void* workspace, cudaStream_t st) {
  const Layout a = layout(p.Hq, p.Hkv, p.Nq, p.D);
  p.rw = a.rw;
  p.part_tiles = a.part_tiles;
  p.unit_cost = a.workers > sm_count() ? kFewUnitCost : kUnitCost;
  p.wait_limit = kWaitLimitCycles;
  char* ws = static_cast<char*>(workspace);
  p.o_part = reinterpret_cast<float*>(ws);
  p.lse_part = reinterpret_cast<float*>(ws + a.o_bytes);
  p.cuts = reinterpret_cast<TreeCut*>(ws + a.o_bytes + a.ml_bytes);
  TreeMaps m;
  int rc = make_maps(p, m);
  if (rc) return rc;
  if (a.workers > sm_count())
    rc = launch_tree_few(p, m, st);
  else
    rc = p.D == 64 ? launch_wide<64>(p, m, st) : launch_wide<128>(p, m, st);
  if (rc) return rc;
  if ((rc = p.D == 64 ? launch_merge_parts<64>(p, a.workers, st) : launch_merge_parts<128>(p, a.workers, st))) return rc;
  count_launch(2);
  return ATTN_OK;
}

}  // namespace attn
