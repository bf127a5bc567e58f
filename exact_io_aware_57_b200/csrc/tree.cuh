// What the two tree-attention kernels share: how a launch's work is laid out and
// walked, and the combination of the partials of a unit that a cut divides.
#pragma once

#include "cache.cuh"
#include "kernels.h"

namespace attn {

constexpr int kTreeKeys = 128;  // keys per tile
// The work is cut into runs by steps.  A key tile is one step for each of the unit's
// row tiles: two row tiles' softmax takes twice one's (counted alike, the workers of
// sequences that fill one row tile ended after half the others' time: 16 sequences
// of up to 61 tokens took 184 us instead of 169).  And each row tile counts for
// unit_cost tiles more, as its first and last tiles, Q and O cost: otherwise the
// workers whose runs hold several short units end last.
// One sequence's share of the work: per KV head `active` units (pairs of row
// tiles; of an odd number the last by itself) of n tiles, then the units whose rows
// are all padding (one empty step each).
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
  s.per_head = (long long)s.row_tiles * (s.n + p.unit_cost) + ((rw.tiles + 1) / 2 - s.active);
  return s;
}

// A worker's run of steps, unit by unit: the units of which it has tiles.
struct TreeUnit {
  int b, hk, pair;  // row tiles 2 pair, 2 pair + 1
  int tb, te, n;    // tiles [tb, te) of n
  int rest;         // steps from the run's end to its last tile's first (and that one)
  bool two, empty;  // two row tiles; no row of it sees anything
};

struct TreeWalk {
  int b, hk, pair, step;  // the next step (the tiles' first, then those without one)
  int left;               // steps left in the run
  TreeSeq s;

  ATTN_DEVINL void begin(const TreeParams& p, const RowTiles& rw, const Run& run) {
    left = (int)(run.run1 - run.run0);
    if (left <= 0) return;
    b = run.b;
    s = tree_seq(p, rw, b);
    hk = (int)(run.off / s.per_head);
    const long long cost = 2ll * (s.n + p.unit_cost);
    const long long off = run.off - hk * s.per_head, busy = (long long)s.row_tiles * (s.n + p.unit_cost);
    pair = off < busy ? (int)(off / cost) : s.active + (int)(off - busy);
    step = off < busy ? (int)(off - pair * cost) : 0;
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
      const int shift = !empty && 2 * pair + 1 < s.row_tiles;  // log2 of the steps per tile
      const int n = empty ? 1 : s.n, end = min(empty ? 1 : (s.n + p.unit_cost) << shift, step + left);
      // a tile belongs to the run that has its first step (runs are two steps at least
      // where tiles are: every run inside the tiles has one)
      const int tb = (step + shift) >> shift, te = min(n, (end + shift) >> shift);
      u.b = b;
      u.hk = hk;
      u.pair = pair++;
      u.empty = empty;
      u.two = shift;
      u.rest = ((n - 1) << shift) + 1 - end;
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

}  // namespace attn
