// Work split of the cache attention kernels.  Plain C++ apart from the
// __host__ __device__ marks, so that it also builds (and is tested) without
// the CUDA compiler.
//
// Sequence b has T query tokens on n cached keys and `group` query heads per
// key/value head.  The rows of a key/value head are its T * group (token,
// head) pairs, token major, cut into row tiles of RT rows; an item is one row
// tile of one key/value head of one sequence, and needs the 16-key tiles
// [lo, hi) that some row of it may see, in units of `per` tiles (an item
// without keys counts one unit: its zeros are written).  Items are numbered
// sequence major, then head, then row tile; all their units, in that order,
// go to the CTAs in contiguous ranges (the cut of lw_tcplan.h), so every CTA
// has the same work to within a unit whatever the lengths are.
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

// Units of one key/value head of a sequence.
LW_TC_HD long long kv_head_units(int T, int n, int group, int RT, int per, int causal, int window) {
  const int nrt = kv_row_tiles(T, group, RT);
  long long s = 0;
  for (int rt = 0; rt < nrt; ++rt) s += kv_units(kv_tile_span(T, n, group, RT, rt, causal, window), per);
  return s;
}

// A CTA's walk over its range of units, item by item.
struct KvWalk {
  long long x, xe;      // this CTA's units [x, xe)
  long long base;       // first unit of sequence b
  int b, h, rt, nrt;    // current item
  int T, n;             // current sequence
  int k0, k1, units;    // this CTA's units of the item: [k0, k1) of `units`
  KvSpan span;
};

// First unit of CTA c of G.
LW_TC_HD long long kv_first(long long U, int c, int G) { return U * c / G; }

// The item at unit w.x; w.b, w.base, w.T and w.n are its sequence's.
LW_TC_HD void kv_seek(KvWalk& w, int group, int RT, int per, int causal, int window) {
  const long long per_head = kv_head_units(w.T, w.n, group, RT, per, causal, window);
  long long r = w.x - w.base;
  w.h = (int)(r / per_head);
  r -= per_head * w.h;
  w.nrt = kv_row_tiles(w.T, group, RT);
  for (w.rt = 0;; ++w.rt) {
    w.span = kv_tile_span(w.T, w.n, group, RT, w.rt, causal, window);
    w.units = kv_units(w.span, per);
    if (r < w.units) break;
    r -= w.units;
  }
  w.k0 = (int)r;
  w.k1 = w.xe - w.x < w.units - w.k0 ? w.k0 + (int)(w.xe - w.x) : w.units;
}

// Past the current item; false when the sequence has no further item (the
// caller then sets w.b, w.T, w.n and w.base = w.x and calls kv_start).
LW_TC_HD void kv_start(KvWalk& w, int group, int RT, int per, int causal, int window) {
  w.nrt = kv_row_tiles(w.T, group, RT);
  w.span = kv_tile_span(w.T, w.n, group, RT, w.rt, causal, window);
  w.units = kv_units(w.span, per);
  w.k0 = 0;
  w.k1 = w.xe - w.x < w.units ? (int)(w.xe - w.x) : w.units;
}
LW_TC_HD bool kv_next(KvWalk& w, int heads) {
  w.x += w.k1 - w.k0;
  if (++w.rt < w.nrt) return true;
  w.rt = 0;
  if (++w.h < heads) return true;
  w.h = 0;
  return false;
}

}  // namespace lw
