// Tree attention over a key/value cache on sm_100a tensor cores (bf16) for up to
// 16 query rows per (sequence, KV head): decode steps and small trees.
//
// Every K/V row is read once for the few query rows of its sequence and KV head,
// so the kernel is bound by HBM and is built to stream.
//
// Transposed products.  S^T = K Q^T and O^T += V^T P^T: the 128 keys of a tile are
// the M = 128 rows of the first product and the d columns those of the second,
// and the query rows are N = 16.  The exponentials and the tensor
// cores' share of shared memory then go by the rows there are, not by 128.  A
// thread owns a key in the softmax and a column of O in the epilogue.
//
// Softmax.  x = s * scale * log2(e); P = 2^(x - m) with one reference m per row,
// shared by all keys: the x of the row's first key, raised to the largest of a tile
// (and O, l rescaled) when that exceeds it by more than 2^8.  The final O / l and LSE
// do not depend on the reference ("Softmax does not need the matrix", "Carry the
// Normalizer"), and P keeps its relative precision at any size.  Whether a tile
// needs that is known when all four warps have looked at their keys, so they meet
// on a barrier before P is handed over.  Each thread keeps its keys' share of
// every row's sum of P in registers, in fp32, until the unit ends.
//
// Rows.  The query rows of one (sequence, KV head) are all (token t, head g of
// the group): row r = (r / G, r % G), so that the group shares each K/V tile
// ("Understanding FlashAttention Pt 1", contents 4.1).
//
// Work.  A unit is one (sequence, KV head); its tiles are the 128-key tiles of its
// cached slots followed by that of its new keys.  The units' tiles are laid end to
// end and cut into equal runs, one per worker, whatever the lengths are: they are
// read on the device.  A unit that a cut divides leaves one partial (O, m, l) per
// worker in the workspace, combined in worker order, so results do not vary from
// run to run.
//
// Lanes.  Each CTA (one per SM) has two lanes, which are workers with runs of
// their own: each has its scores and O in TMEM, its P in shared memory and a
// softmax warpgroup, and they take turns on the tensor cores:
//   S(0, i); O_1 += P(1, i - 1) V; S(1, i); O_0 += P(0, i) V; S(0, i + 1); ...
// K and V tiles are loaded in that order.  Once S of a lane's next step is
// complete so is its last product, which was issued before it: O may be rescaled
// and P overwritten.  While one lane finishes a unit (its last product, O to
// memory), the other one's tiles keep the memory busy.
//
//   warps 0..3  softmax of lane 0: thread r owns key r of a tile, column r of O
//   warps 4..7  softmax of lane 1
//   warp 8      TMEM owner + single-thread tcgen05.mma issuer
//   warp 9      TMA producer: a thread per box, looked up in the page table
//
// TMEM (64 columns x 128 lanes): [16 l, +16) scores of lane l (TMEM lane = key);
// [32 + 16 l, +16) O of lane l (TMEM lane = column of O; with d = 64 the upper 64
// repeat the lower ones).
//
// The last key tile of a sequence ends inside a page or box.  Its hidden scores
// are set to -inf whatever they hold, and its hidden V rows are zeroed in shared
// memory before the product, so rows behind the sequence's end may hold anything.
#include <algorithm>
#include <cstring>

#include "tree.cuh"

namespace attn {

namespace {

constexpr int KT = kTreeKeys;
constexpr int kWarpMma = 8, kWarpLoad = 9;
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 64;
constexpr int W = 16;  // rows there is room for, the columns of the products
// log2 units: P stays <= 256, and P V in fp32's range for V up to 2^119 over the number of
// keys.  (With 64 the references hardly ever rise, and 64 sequences of 300 .. 8191 slots
// take 206 us instead of 208, but |V| of 2^64 can leave the range.)
constexpr float kRaise = 8.f;
constexpr float kNoKey = 1e30f;  // -m of a row that has seen no key: any score raises it
// -m of a column that is no row, or a row that does not count: its x - m is -inf or NaN
// whatever its scores are (of Q rows in shared memory that no load wrote, or of a
// caller's padding), so that it never raises the references of the others.
constexpr float kNoRow = -INFINITY;

template <int D>
struct FewSmem {
  static constexpr int kTileBytes = KT * D * 2;
  static constexpr int kQBytes = W * D * 2;
  // K and V tiles on their way or in use: 6 at d = 128
  static constexpr int NST = std::min(11, (226 * 1024 - 4 * kQBytes - KT * 128) / kTileBytes);
  alignas(1024) uint8_t q[2][2][kQBytes];  // [lane][the unit's and the next one's]
  alignas(1024) uint8_t p[KT * 128];       // P: a line of 128 bytes per key, half of it for each lane
  alignas(1024) uint8_t kv[NST][kTileBytes];
  alignas(16) float neg_m[2][W];  // -m of each row
  // the warps' maxima or sums of each row, then what to multiply its O by
  alignas(16) float scratch[2][5 * W];
  uint64_t q_full[2][2], q_empty[2][2];
  uint64_t kv_full[NST], kv_empty[NST];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2], meet[2], drain;
  RunSmem<kThreads, 2> run;
  uint32_t raise[2];  // the last step of each lane that had to raise its reference
  uint32_t tmem_base;
  int abort_flag;
};

// A run step by step.
struct Steps {
  TreeWalk w;
  TreeUnit u;
  int tile;
  bool have;  // false: the run is over

  ATTN_DEVINL void begin(const TreeParams& p, const RowTiles& rw, const Run& run) {
    w.begin(p, rw, run);
    u = TreeUnit{};
    tile = -1;
    have = true;
  }
  ATTN_DEVINL void step(const TreeParams& p, const RowTiles& rw) {
    if (++tile < u.te) return;
    have = w.next(p, rw, u);
    tile = u.tb;
  }
  ATTN_DEVINL bool first() const { return tile == u.tb; }
  ATTN_DEVINL bool last() const { return tile == u.te - 1; }
  ATTN_DEVINL bool busy() const { return have && !u.empty; }  // the step has a key tile
};

// Ring positions of the K and V tiles of step i of lane l: the order of the
// products, of which the very first has no V of lane 1 before it.
ATTN_DEVINL uint32_t at_k(int l, int i) { return l ? 4u * i + 1u : (i ? 4u * i - 1u : 0u); }
ATTN_DEVINL uint32_t at_v(int l, int i) { return l ? 4u * i + 4u : 4u * i + 2u; }

// Largest x of the warp.
ATTN_DEVINL float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Sums of 16 columns over the warp's lanes; lane i is left with column i >> 1.
ATTN_DEVINL float warp_sums(const float (&v)[16]) {
  const int lane = threadIdx.x & 31;
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[i + 8] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 8], 16);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 8;
    b[i] = (up ? a[i + 4] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 4], 8);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 4;
    c[i] = (up ? b[i + 2] : b[i]) + __shfl_xor_sync(0xffffffffu, up ? b[i] : b[i + 2], 4);
  }
  const bool up = lane & 2;
  const float d = (up ? c[1] : c[0]) + __shfl_xor_sync(0xffffffffu, up ? c[0] : c[1], 2);
  return d + __shfl_xor_sync(0xffffffffu, d, 1);
}

// Which rows see which of a warp's 32 keys of an edge tile: of cached slots those
// that exist are seen by all; of new keys lane i holds the bits of row i, read
// before the tile's scores are waited for.
struct Sight {
  bool exists, cached;
  uint32_t row;
};

ATTN_DEVINL Sight find_sight(const TreeParams& p, bool cached, bool exists, int key0, int b, int rows) {
  Sight v{exists, cached, 0u};
  const int r = threadIdx.x & 31;
  if (!cached && r < rows) {
    const int t = r / p.rw.gb;  // sees the keys from key0 on of its mask words, or those up to t
    if (p.mask) {
      if (key0 < 64 * p.mask_words)
        v.row = (uint32_t)(__ldg(p.mask + b * p.mask_bstride + (long long)t * p.mask_words + (key0 >> 6)) >> (key0 & 63));
    } else {
      const int n = t + 1 - key0;
      v.row = n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
    }
  }
  return v;
}

// Bit i: row i sees this thread's key.
ATTN_DEVINL uint32_t sight(const Sight& v) {
  uint32_t bits = 0xffffu;
  if (!v.cached) {
    bits = 0;
#pragma unroll
    for (int i = 0; i < W; ++i)
      bits |= ((__shfl_sync(0xffffffffu, v.row, i) >> (threadIdx.x & 31)) & 1u) << i;
  }
  return v.exists ? bits : 0u;
}

// x - m of one key for every row from its scores; hidden ones at -inf.
ATTN_DEVINL void shifted(const uint32_t (&v)[W], uint64_t sc2, const uint64_t (&nm)[W / 2], bool edge, uint32_t see,
                         float (&y)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 2)
    unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2, nm[i / 2]), y[i], y[i + 1]);
  if (edge) {
#pragma unroll
    for (int i = 0; i < W; ++i) y[i] = (see >> i) & 1u ? y[i] : -INFINITY;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kn,
                    const __grid_constant__ CUtensorMap tm_vn, const TreeParams p, const TileForm form,
                    const TileForm new_form) {
  using Smem = FewSmem<D>;
  constexpr int NST = Smem::NST;
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RowTiles& rw = p.rw;
  const int rows = rw.gb * rw.tt;  // query rows of a unit

  // ---- setup
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int l = 0; l < 2; ++l) {
      for (int j = 0; j < 2; ++j) {
        mbar_init(&s.q_full[l][j], 1);
        mbar_init(&s.q_empty[l][j], 1);
      }
      mbar_init(&s.s_full[l], 1);
      mbar_init(&s.p_full[l], 4);
      mbar_init(&s.o_done[l], 1);
      mbar_init(&s.o_free[l], 4);
      mbar_init(&s.meet[l], 4);
      s.raise[l] = 0xffffffffu;
    }
    for (int i = 0; i < NST; ++i) {
      mbar_init(&s.kv_full[i], 1);
      mbar_init(&s.kv_empty[i], 1);
    }
    mbar_init(&s.drain, 1);
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(&s.tmem_base, kTmemCols);
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    if (p.k_new) {
      tma_prefetch_desc(&tm_kn);
      tma_prefetch_desc(&tm_vn);
    }
  }
  tc_fence_before();
  find_runs<kThreads, 2>(s.run, p.B, 1, [&](int b) { return tree_seq(p, rw, b).per_head * p.Hkv; });
  tc_fence_after();
  const Runs<2>& runs = s.run.runs;
  const uint32_t tmem = s.tmem_base;
  const Abort ab{&s.abort_flag, p.status, p.wait_limit};

  if (warp == kWarpLoad) {
    // ===================================================== TMA producer
    Steps it[2];
    TileBox box[2], ahead[2];  // of the step's tile and of the next one, looked up early
    TreeBoxes boxes[2];
    int nq[2] = {0, 0};        // Q tiles loaded
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      it[l].begin(p, rw, runs.lane[l]);
      ahead[l] = TileBox{};
    }
    bool ok = true;
    auto load = [&](int l, int v, uint32_t at) {  // the step's K (v = 0) or V tile to ring position at
      const Steps& x = it[l];
      const TreeUnit& u = x.u;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&s.kv_empty[at % NST], ((at / NST) & 1) ^ 1, ab));
      if (!ok) return;
      uint64_t* bar = &s.kv_full[at % NST];
      uint8_t* dst = s.kv[at % NST];
      if (!x.busy()) {
        if (lane == 0) mbar_arrive(bar);  // nothing to load: the ring goes on
        __syncwarp();
      } else if (x.tile < x.w.s.nc) {
        load_tile<D>(dst, bar, v ? &tm_v : &tm_k, form, box[l], u.hk, p.c.num_pages, p.status);
      } else {
        load_tile<D>(dst, bar, v ? &tm_vn : &tm_kn, new_form, box[l], u.hk, p.B, p.status);
      }
    };
    auto advance = [&](int l) {
      Steps& x = it[l];
      x.step(p, rw);
      if (!x.busy()) return;
      const TreeUnit& u = x.u;
      if (x.first()) {
        ahead[l] = boxes[l].find(p, form, new_form, x.w.s, u.b, x.tile, true);
        const int slot = nq[l] & 1;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&s.q_empty[l][slot], ((nq[l] >> 1) & 1) ^ 1, ab));
        if (ok && lane == 0) {
          mbar_expect_tx(&s.q_full[l][slot], rows * D * 2);
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_4d(s.q[l][slot] + kb * W * 128, &tm_q, &s.q_full[l][slot], kb * 64, u.hk * rw.G, 0, u.b);
        }
        __syncwarp();
        ++nq[l];
      }
      box[l] = ahead[l];
      if (x.tile + 1 < u.te) ahead[l] = boxes[l].find(p, form, new_form, x.w.s, u.b, x.tile + 1, false);
    };
    // until both runs are over; a lane whose own is passes its positions on
    for (int i = 0; ok; ++i) {
      advance(0);
      load(0, 0, at_k(0, i));
      if (i > 0) load(1, 1, at_v(1, i - 1));
      advance(1);
      load(1, 0, at_k(1, i));
      load(0, 1, at_v(0, i));
      if (!it[0].have && !it[1].have) break;
    }
    if (s.abort_flag) {
      // leave no copy in flight into shared memory that is about to be released:
      // every barrier with a load outstanding completes its current phase
      for (int i = 0; i < NST; ++i) {
        mbar_wait_drain(&s.kv_full[i], 0, p.wait_limit / 64);
        mbar_wait_drain(&s.kv_full[i], 1, p.wait_limit / 64);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_wait_drain(&s.q_full[i >> 1][i & 1], 0, p.wait_limit / 64);
        mbar_wait_drain(&s.q_full[i >> 1][i & 1], 1, p.wait_limit / 64);
      }
    }
  } else if (warp == kWarpMma) {
    // ===================================================== MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16(KT, W, 0, 0);    // K tile and Q: K-major
      constexpr uint32_t idesc_pv = idesc_bf16(128, W, 1, 1);  // V tile and P: MN-major
      // what a lane does in its step: nothing, or its unit's first / last tile there
      struct Turn {
        bool works, first, last;
      };
      Steps it[2];
      Turn now[2];
      int nq[2], items[2], units[2];  // Q tile in use; P taken; units whose O has begun
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        it[l].begin(p, rw, runs.lane[l]);
        nq[l] = -1;
        items[l] = units[l] = 0;
      }
      bool ok = true;
      auto wait_full = [&](uint32_t at) { return mbar_wait(&s.kv_full[at % NST], (at / NST) & 1, ab); };
      auto scores = [&](int l, int i) {
        const uint32_t at = at_k(l, i);
        it[l].step(p, rw);
        now[l] = Turn{it[l].busy(), it[l].first(), it[l].last()};
        if (now[l].works && now[l].first) {
          ++nq[l];
          ok = mbar_wait(&s.q_full[l][nq[l] & 1], (nq[l] >> 1) & 1, ab);
        }
        if (!ok || !(ok = wait_full(at))) return;
        if (!now[l].works) {  // a ring position without a tile: passed on
          mbar_arrive(&s.kv_empty[at % NST]);
          return;
        }
        tc_fence_after();
        const uint64_t qd = sdesc_sw128(smem_u32(s.q[l][nq[l] & 1]), 16, 1024);
        const uint64_t kd = k_tile_desc<D>(s.kv[at % NST]);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + l * 16, k_tile_step(kd, kk), sdesc_at(qd, (kk >> 2) * (W * 128) + (kk & 3) * 32), idesc_s, kk > 0);
        mma_commit(&s.s_full[l]);
        mma_commit(&s.kv_empty[at % NST]);
        if (now[l].last) mma_commit(&s.q_empty[l][nq[l] & 1]);
      };
      auto product = [&](int l, int i) {
        const uint32_t at = at_v(l, i);
        if (!ok || !(ok = wait_full(at))) return;
        if (!now[l].works) {
          mbar_arrive(&s.kv_empty[at % NST]);
          return;
        }
        if (now[l].first) {  // the lane's last unit has been read out of O
          if (units[l] > 0) ok = mbar_wait(&s.o_free[l], (units[l] - 1) & 1, ab);
          ++units[l];
        }
        if (!ok || !(ok = mbar_wait(&s.p_full[l], items[l] & 1, ab))) return;
        ++items[l];
        tc_fence_after();
        const uint64_t vd = v_tile_desc<D>(s.kv[at % NST]);
        const uint64_t pd = sdesc_sw128(smem_u32(s.p) + l * 64, KT * 128, 1024);
        const uint32_t accum = !now[l].first;
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          mma_ss(tmem + 32 + l * 16, v_tile_step<D>(vd, kk), sdesc_at(pd, kk * 2048), idesc_pv, kk > 0 ? 1u : accum);
        mma_commit(&s.kv_empty[at % NST]);
        if (now[l].last) mma_commit(&s.o_done[l]);
      };
      for (int i = 0; ok; ++i) {
        scores(0, i);
        if (i > 0) product(1, i - 1);
        if (ok) scores(1, i);
        product(0, i);
        if (!it[0].have && !it[1].have) break;
      }
      // TMEM must be quiescent before it is released
      mma_commit(&s.drain);
      mbar_wait_drain(&s.drain, 0, p.wait_limit);
    }
  } else {
    // ===================================================== softmax warpgroups
    const int l = warp >> 2;       // lane of this warpgroup
    const int quarter = warp & 3;  // TMEM lanes [32 quarter, +32)
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t col_s = tmem + lane_off + l * 16;
    const uint32_t col_o = tmem + lane_off + 32 + l * 16;
    const float sc = p.scale * kLog2e;
    const uint64_t sc2 = pack_f32x2(sc, sc);
    const uint32_t p_line = smem_u32(s.p) + r * 128;
    float* const neg_m = s.neg_m[l];
    float* const parts = s.scratch[l];
    float* const factor = parts + 4 * W;
    const Run& run = runs.lane[l];
    const int worker = blockIdx.x + l * gridDim.x;
    uint32_t meets = 0;
    auto meet = [&]() -> bool {  // the lane's four warps
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.meet[l]);
      return __all_sync(0xffffffffu, mbar_wait(&s.meet[l], meets++ & 1, ab));
    };
    // -m of every row in registers: the tensor cores' reads leave little of the
    // shared memory's bandwidth
    uint64_t nm[W / 2];
    auto fetch_nm = [&]() {
#pragma unroll
      for (int c = 0; c < W / 2; ++c) nm[c] = *reinterpret_cast<const uint64_t*>(neg_m + 2 * c);
    };
    TreeWalk w;
    w.begin(p, rw, run);
    TreeUnit u{};
    uint32_t items = 0;
    int units = 0, step = 0;  // units and tiles behind
    bool ok = true;
    while (ok && w.next(p, rw, u)) {
      const int n = u.te - u.tb, len = w.s.len, nr = w.s.nr, nc = w.s.nc;
      const int counted = nr * rw.gb;  // rows of the unit that count
      const bool mine = !u.empty;
      uint64_t sums[W / 2];  // this thread's keys' share of l, by pairs of rows
#pragma unroll
      for (int c = 0; c < W / 2; ++c) sums[c] = 0;
      for (int i = 0; mine && i < n; ++i, ++items) {
        const int tile = u.tb + i;
        const bool cached = tile < nc;
        const int base = (cached ? tile : tile - nc) * KT;
        const int keys = min(KT, (cached ? len : nr) - base);  // keys of this tile that exist
        const bool edge = !cached || keys < KT;
        Sight sg{true, true, 0u};
        if (edge) sg = find_sight(p, cached, r < keys, base + 32 * quarter, u.b, rows);
        ok = __all_sync(0xffffffffu, mbar_wait(&s.s_full[l], items & 1, ab));
        if (!ok) break;
        tc_fence_after();
        uint32_t v[W];
        tmem_ld16(col_s, v);
        tmem_wait_ld();
        reg_fence(v);
        const uint32_t see = edge ? sight(sg) : 0xffffu;
        bool raise = i == 0 && !cached;
        if (i == 0 && cached) {
          // the first key's score is as good a reference as the largest one, unless
          // that exceeds it by more than 2^8
          if (r == 0) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
              const float x = __uint_as_float(v[e]) * sc;
              neg_m[e] = e >= counted ? kNoRow : x == -INFINITY ? kNoKey : -x;
            }
          }
          if (!(ok = meet())) break;
          fetch_nm();
        }
        float y[W];
        if (!raise) {
          shifted(v, sc2, nm, edge, see, y);
          float top0 = y[0], top1 = y[1];
#pragma unroll
          for (int e = 2; e < W; e += 4) {
            top0 = fmaxf(top0, fmaxf(y[e], y[e + 1]));
            if (e + 2 < W) top1 = fmaxf(top1, fmaxf(y[e + 2], y[e + 3]));
          }
          if (__any_sync(0xffffffffu, fmaxf(top0, top1) > kRaise) && lane == 0) s.raise[l] = items;
          if (!(ok = meet())) break;
          raise = *(volatile uint32_t*)&s.raise[l] == items;
        }
        if (raise) {
          // the rows' references rise to the tile's maxima, O and l with them
          float mine_max = 0.f;
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float m = warp_max((see >> e) & 1u ? __uint_as_float(v[e]) * sc : -INFINITY);
            if (lane == e) mine_max = m;
          }
          if (lane < W) parts[quarter * W + lane] = mine_max;
          if (!(ok = meet())) break;
          if (r < W) {
            const float nm_old = i == 0 ? kNoKey : neg_m[r];
            const float old = nm_old == kNoKey ? -INFINITY : -nm_old;
            float m = old;
#pragma unroll
            for (int x = 0; x < 4; ++x) m = fmaxf(m, parts[x * W + r]);
            factor[r] = r >= counted || old == -INFINITY ? 0.f : ex2(old - m);
            neg_m[r] = r >= counted ? kNoRow : m == -INFINITY ? kNoKey : -m;
          }
          if (!(ok = meet())) break;
          fetch_nm();
          if (i > 0) {
            uint32_t o[W];
            tmem_ld16(col_o, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int e = 0; e < W; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor[e]);
            tmem_st16(col_o, o);
            tmem_wait_st();
#pragma unroll
            for (int c = 0; c < W / 2; ++c)
              sums[c] = fma_f32x2(sums[c], pack_f32x2(factor[2 * c], factor[2 * c + 1]), 0ull);
          }
          shifted(v, sc2, nm, edge, see, y);
        }
        // P into this key's line (16-byte chunk c at c ^ (key & 7), the lane's two
        // from 4 l on) in bf16, the product's operand; the sums keep 32 bits
#pragma unroll
        for (int e = 0; e < W; ++e) y[e] = ex2(y[e]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p_line + (((4 * l + h) ^ (r & 7)) << 4)),
                       "r"(pack_bf16(y[8 * h], y[8 * h + 1])), "r"(pack_bf16(y[8 * h + 2], y[8 * h + 3])),
                       "r"(pack_bf16(y[8 * h + 4], y[8 * h + 5])), "r"(pack_bf16(y[8 * h + 6], y[8 * h + 7]))
                       : "memory");
#pragma unroll
        for (int c = 0; c < W / 2; ++c) sums[c] = add_f32x2(sums[c], pack_f32x2(y[2 * c], y[2 * c + 1]));
        if (keys < KT) {
          // V rows that do not exist take part with P = 0: they have to be finite
          const uint32_t at = at_v(l, step + i);
          ok = __all_sync(0xffffffffu, mbar_wait(&s.kv_full[at % NST], (at / NST) & 1, ab));
          if (!ok) break;
          if (r >= keys) zero_slot<D>(s.kv[at % NST], r);
        }
        fence_proxy_async_smem();  // P and zeroed V rows to the products
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[l]);
      }
      if (!ok) break;
      // ---- epilogue: O / l and LSE of a whole unit (rows that are padding: 0 and
      // -inf), or this worker's partial.  Thread r sums up row r, then writes
      // column r of O for every row.
      const bool whole = n == u.n;
      const long long prow = ((long long)worker * 2 + (u.tb > 0 ? 0 : 1)) * rows;
      if (mine) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s.o_done[l], units & 1, ab));
        if (!ok) break;
        tc_fence_after();
        float v[W];
#pragma unroll
        for (int e = 0; e < W / 2; ++e) unpack_f32x2(sums[e], v[2 * e], v[2 * e + 1]);
        const float x = warp_sums(v);
        if (!(lane & 1)) parts[quarter * W + (lane >> 1)] = x;
        if (!(ok = meet())) break;
      }
      if (r < rows) {
        const int t = r / rw.gb;
        float m = -INFINITY, sum = 0.f;
        if (mine && t < nr) {
          m = neg_m[r] == kNoKey ? -INFINITY : -neg_m[r];
          sum = (parts[r] + parts[W + r]) + (parts[2 * W + r] + parts[3 * W + r]);
        }
        // sum = 0: sees no key (a NaN score leaves m = -inf and sum = NaN)
        if (mine) factor[r] = sum == 0.f ? 0.f : 1.f / sum;
        if (whole)
          p.lse[((long long)u.b * p.Hq + u.hk * rw.G + r % rw.gb) * p.Nq + t] =
              sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        else
          reinterpret_cast<float2*>(p.lse_part)[prow + r] = make_float2(m, sum);
      }
      if (mine && !(ok = meet())) break;
      uint32_t v[W];
      if (mine) {
        tmem_ld16(col_o, v);
        tmem_wait_ld();
        reg_fence(v);
      }
      if (whole) {
        // rows in order: the group's heads side by side, tokens Hq heads apart
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + ((long long)u.b * p.Nq * p.Hq + u.hk * rw.G) * D + r;
        int g = 0;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if (e < rows) {  // uniform
            // 0: padding, or sees no key; O may hold anything then
            const float f = mine ? factor[e] : 0.f;
            if (r < D) *dst = __float2bfloat16_rn(f == 0.f ? 0.f : __uint_as_float(v[e]) * f);
            dst += D;
            if (++g == rw.gb) {
              g = 0;
              dst += (p.Hq - rw.gb) * D;
            }
          }
        }
      } else if (mine) {
        float* dst = p.o_part + prow * D + r;
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (r < D && e < rows) dst[e * D] = __uint_as_float(v[e]);
      }
      if (mine) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o_free[l]);
        ++units;
      }
      step += n;
    }
    // The unit that this run ends in the middle of, having held its beginning: its
    // later parts are the next workers' first ones.
    if (r == 0) {
      TreeCut cut{0, 0, 0, 0, 0};
      if (ok && run.run1 > run.run0 && u.tb == 0 && u.te < u.n)
        cut = TreeCut{u.b, u.hk, u.pair, 1, run_parts(runs.total, runs.workers, worker, run.run1, u.rest)};
      p.cuts[worker] = cut;
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
}

template <int D>
int launch_few_t(const TreeParams& p, const TreeMaps& m, cudaStream_t st) {
  const size_t smem = sizeof(FewSmem<D>) + 1024;
  static_assert(sizeof(FewSmem<D>) + 1024 <= 232448, "shared memory");
  if (cudaFuncSetAttribute(tree_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATTN_ERR_CUDA;
  tree_few_kernel<D><<<sm_count(), kThreads, smem, st>>>(m.q, m.k, m.v, m.k_new, m.v_new, p, m.form, m.new_form);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

int launch_tree_few(const TreeParams& p, const TreeMaps& m, cudaStream_t st) {
  return p.D == 64 ? launch_few_t<64>(p, m, st) : launch_few_t<128>(p, m, st);
}

}  // namespace attn
