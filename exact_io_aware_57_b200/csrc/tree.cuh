// What the two tree-attention kernels share: how a launch's work is laid out and
// walked, and the combination of the partials of a unit that a cut divides.
#pragma once

#include "cache.cuh"
#include "kernels.h"

namespace attn {

constexpr int kTreeKeys = 128;  // keys per tile
// Steps that a unit counts for beyond its tiles when the work is cut into runs: its
// first and last tiles, Q and O cost about as much as this many others (with 0,
// the workers whose runs hold several short units end last: 16 sequences of 2000 ..
// 12345 slots with 32 tokens each took 145 us instead of 136; 2 to 8 measured equal).
constexpr int kUnitCost = 4;

// One sequence's share of the work: per KV head `active` units (pairs of row
// tiles; with one row tile in all, that one) of n tiles and kUnitCost steps, then
// the units whose rows are all padding (one empty step each).
struct TreeSeq {
  int len, nr, nc, n, row_tiles, active;
  long long per_head;
};

ATTN_DEVINL TreeSeq tree_seq(const TreeParams& p, const RowTiles& rw, int b) {
  TreeSeq s;
  if (!cache_len(p.c, b, kMaxSlots, p.status, s.len) || !row_count(p.row_lens, b, p.Nq, p.status, s.nr))
    s.len = s.nr = 0;
  s.nc = (s.len + kTreeKeys - 1) / kTreeKeys;
  s.n = s.nc + (p.k_new ? (s.nr + kTreeKeys - 1) / kTreeKeys : 0);
  s.row_tiles = s.n > 0 ? (s.nr + rw.tt - 1) / rw.tt * rw.gblk : 0;
  s.active = (s.row_tiles + 1) / 2;
  s.per_head = (long long)s.active * (s.n + kUnitCost) + ((rw.tiles + 1) / 2 - s.active);
  return s;
}

// A worker's run of steps, unit by unit: the units of which it has tiles.
struct TreeUnit {
  int b, hk, pair;  // row tiles 2 pair, 2 pair + 1
  int tb, te, n;    // tiles [tb, te) of n
  bool two, empty;  // two row tiles; no row of it sees anything
};

struct TreeWalk {
  int b, hk, pair, step;  // the next step (tiles first, then kUnitCost without one)
  int left;               // steps left in the run
  TreeSeq s;

  ATTN_DEVINL void begin(const TreeParams& p, const RowTiles& rw, const Run& run) {
    left = (int)(run.run1 - run.run0);
    if (left <= 0) return;
    b = run.b;
    s = tree_seq(p, rw, b);
    hk = (int)(run.off / s.per_head);
    const int cost = s.n + kUnitCost;
    const long long off = run.off - hk * s.per_head, busy = (long long)s.active * cost;
    pair = off < busy ? (int)(off / cost) : s.active + (int)(off - busy);
    step = off < busy ? (int)(off - (long long)pair * cost) : 0;
  }
  ATTN_DEVINL bool next(const TreeParams& p, const RowTiles& rw, TreeUnit& u) {
    while (left > 0) {
      if (pair == (rw.tiles + 1) / 2) {
        pair = 0;
        if (++hk == p.Hkv) {
          hk = 0;
          s = tree_seq(p, rw, ++b);
        }
      }
      const bool empty = pair >= s.active;
      const int n = empty ? 1 : s.n, end = min(empty ? 1 : s.n + kUnitCost, step + left);
      const int tb = step, te = min(n, end);
      u.b = b;
      u.hk = hk;
      u.pair = pair++;
      u.empty = empty;
      u.two = !empty && 2 * u.pair + 1 < s.row_tiles;
      left -= end - step;
      step = 0;
      if (tb < te) {
        u.tb = tb;
        u.te = te;
        u.n = n;
        return true;
      }
    }
    return false;
  }
};

// A loading warp's place in a unit: boxes of its tiles, of cached slots and then of
// sequence b's new keys.
struct TreeBoxes {
  TileCursor at;

  ATTN_DEVINL TileBox find(const TreeParams& p, const TileForm& form, const TileForm& new_form, const TreeSeq& s, int b,
                           int tile, bool first) {
    if (tile < s.nc) {
      if (first)
        at.begin(p.c, form, tile * kTreeKeys);
      else
        at.next(p.c, form);
      return find_box(p.c, form, at, b, s.len - tile * kTreeKeys);
    }
    CacheView rows = p.c;
    rows.table = nullptr;
    TileCursor c;
    c.begin(rows, new_form, (tile - s.nc) * kTreeKeys);
    return find_box(rows, new_form, c, b, s.nr - (tile - s.nc) * kTreeKeys);
  }
};

template <int N>
ATTN_DEVINL void reg_fence(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

}  // namespace attn
