// Work split of the cache attention kernels.  Plain C++ apart from the
// __host__ __device__ marks, so that it also builds (and is tested) without
// the CUDA compiler.
//
// Sequence b has T query tokens on n cached keys and `group` query heads per
// key/value head.  The rows of a key/value head are its T * group (token,
// head) pairs, token major, cut into row tiles of RT rows; an item is one row
// tile of one key/value head of one sequence, and needs the 16-key tiles
// [lo, hi) that some row of it may see, in units of `per` tiles (an item
// without keys has one unit: its zeros are written).  Items are numbered
// sequence major, then head, then row tile.  An item's start and end cost a CTA
// about as much as `extra` units, so an item weighs that much more, in front of
// its units; all items, in that order, go to the CTAs in contiguous ranges of
// that weight (the cut of lw_tcplan.h): every CTA has the same work to within a
// unit whatever the lengths are.
#pragma once

#include "lw_tcplan.h"

namespace lw {

struct KvSpan {
  int lo, hi;   // 16-key tiles
};

// Keys [lo, hi) that token t of T sees among n.
LW_TC_HD void kv_token_keys(int T, int n, int t, int causal, int window, int& lo, int& hi) {
  const long long pos = (long long)n - T + t;
  hi = n;
  if (causal && pos + 1 < n) hi = pos + 1 > 0 ? (int)(pos + 1) : 0;
  lo = window && pos - window + 1 > 0 ? (int)(pos - window + 1) : 0;
  if (lo > hi) lo = hi;
}

// Tiles that tokens t0..t1 of T see: the first one's window to the last one's
// end.
LW_TC_HD KvSpan kv_span(int T, int n, int t0, int t1, int causal, int window) {
  int lo, hi, x, y;
  kv_token_keys(T, n, t0, causal, window, lo, x);
  kv_token_keys(T, n, t1, causal, window, y, hi);
  if (hi <= lo) return KvSpan{0, 0};
  return KvSpan{lo / 16, (hi + 15) / 16};
}

LW_TC_HD int kv_row_tiles(int T, int group, int RT) { return (T * group + RT - 1) / RT; }

LW_TC_HD KvSpan kv_tile_span(int T, int n, int group, int RT, int rt, int causal, int window) {
  const int t0 = rt * RT / group;
  int t1 = (rt * RT + RT - 1) / group;
  if (t1 > T - 1) t1 = T - 1;
  return kv_span(T, n, t0, t1, causal, window);
}

LW_TC_HD int kv_units(KvSpan s, int per) {
  const int k = (s.hi - s.lo + per - 1) / per;
  return k > 0 ? k : 1;
}

// What the items are cut by, but for the sequences.
struct KvShape {
  int group, RT, per, extra, causal, window;
};

// Weight of an item, and of one key/value head of a sequence.
LW_TC_HD int kv_item_weight(const KvShape& c, int T, int n, int rt) {
  return c.extra + kv_units(kv_tile_span(T, n, c.group, c.RT, rt, c.causal, c.window), c.per);
}
LW_TC_HD long long kv_head_weight(const KvShape& c, int T, int n) {
  const int nrt = kv_row_tiles(T, c.group, c.RT);
  long long s = 0;
  for (int rt = 0; rt < nrt; ++rt) s += kv_item_weight(c, T, n, rt);
  return s;
}

// A CTA's walk over its range of the weight, item by item.
struct KvWalk {
  long long x, xe;      // what is left of the range: [x, xe), x in the current item
  long long base;       // where sequence b begins
  int b, h, rt, nrt;    // current item
  int T, n;             // current sequence
  long long first;      // where the item's units begin (its `extra` is before)
  int k0, k1, units;    // this CTA's units of the item: [k0, k1) of `units`, none if k0 >= k1
  KvSpan span;
};

// Where the range of CTA c of G begins.
LW_TC_HD long long kv_first(long long U, int c, int G) {
  if (U < 0x100000000ll / (G + 1)) return (long long)((uint32_t)U * (uint32_t)c / (uint32_t)G);
  return U * c / G;
}

// The CTA in whose range x lies (tc_owner, in 32 bits where they suffice).
LW_TC_HD int kv_owner(long long x, long long U, int G) {
  if (U < 0x100000000ll / (G + 1)) {
    const uint32_t u = (uint32_t)U, g = (uint32_t)G;
    return (int)((((uint32_t)x + 1u) * g + u - 1u) / u) - 1;
  }
  return tc_owner(x, U, G);
}

// The current item's span and this CTA's units of it; its weight begins at
// w.first - extra.
LW_TC_HD void kv_item(const KvShape& c, KvWalk& w, long long begin) {
  w.span = kv_tile_span(w.T, w.n, c.group, c.RT, w.rt, c.causal, c.window);
  w.units = kv_units(w.span, c.per);
  w.first = begin + c.extra;
  const long long lo = w.x - w.first, hi = w.xe - w.first;
  w.k0 = lo > 0 ? (int)lo : 0;
  w.k1 = hi < w.units ? (int)hi : w.units;
}

// The item at w.x; w.b, w.base, w.T and w.n are its sequence's.
LW_TC_HD void kv_seek(const KvShape& c, KvWalk& w) {
  const long long per_head = kv_head_weight(c, w.T, w.n);
  long long begin = w.base;
  w.h = 0;
  if (w.x - begin >= per_head) {
    w.h = (int)((w.x - begin) / per_head);
    begin += per_head * w.h;
  }
  w.nrt = kv_row_tiles(w.T, c.group, c.RT);
  for (w.rt = 0;; ++w.rt) {
    kv_item(c, w, begin);
    if (w.x < w.first + w.units) break;
    begin = w.first + w.units;
  }
}

// Past the current item; false when the sequence has no further item (the
// caller then sets w.b, w.T and w.n to the next sequence with rows, w.base =
// w.x, w.h = w.rt = 0) -- or the range none, w.x >= w.xe.  Before the new
// item's values are used: kv_enter.
LW_TC_HD bool kv_next(KvWalk& w, int heads) {
  w.x = w.first + w.units;
  if (++w.rt < w.nrt) return true;
  w.rt = 0;
  return ++w.h < heads;
}
LW_TC_HD void kv_enter(const KvShape& c, KvWalk& w) {
  w.nrt = kv_row_tiles(w.T, c.group, c.RT);
  kv_item(c, w, w.x);
}

}  // namespace lw
