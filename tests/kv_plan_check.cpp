// CPU check of the cache attention's work split (lw_kvplan.h): for batches of
// sequences of many lengths, masks and head groups, every unit of every item
// goes to exactly one CTA, the CTAs' walks agree with the owners that the join
// computes, the spans hold every key that some row sees, and no CTA has much
// more than its share.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>

#include "lw_kvplan.h"

using namespace lw;

#define CHECK(x)                                                   \
  do {                                                             \
    if (!(x)) {                                                    \
      std::printf("failed: %s (line %d)\n", #x, __LINE__);         \
      return 1;                                                    \
    }                                                              \
  } while (0)

struct Seq {
  int T, n;
};

static int check(const KvShape& c, const std::vector<Seq>& seqs, int heads, int grid) {
  long long U = 0;
  std::vector<long long> base;
  for (const Seq& s : seqs) {
    base.push_back(U);
    if (s.T) U += heads * kv_head_weight(c, s.T, s.n);
  }
  if (U == 0) return 0;
  const int G = grid < U ? grid : (int)U;
  CHECK(kv_first(U, 0, G) == 0 && kv_first(U, G, G) == U);
  std::map<std::tuple<int, int, int>, std::vector<int>> got;   // item -> owner of each unit
  for (int cta = 0; cta < G; ++cta) {
    KvWalk w{};
    w.x = kv_first(U, cta, G);
    w.xe = kv_first(U, cta + 1, G);
    CHECK(w.x < w.xe);
    CHECK(w.xe - w.x <= (U + G - 1) / G);
    CHECK(kv_owner(w.x, U, G) == cta && kv_owner(w.xe - 1, U, G) == cta);
    CHECK(kv_owner(w.x, U, G) == tc_owner(w.x, U, G));
    int b = 0;
    for (int i = 0; i < (int)seqs.size(); ++i)
      if (seqs[i].T && base[i] <= w.x) b = i;
    w.b = b;
    w.base = base[b];
    w.T = seqs[b].T;
    w.n = seqs[b].n;
    kv_seek(c, w);
    for (;;) {
      if (w.k0 < w.k1) {
        auto& v = got[std::make_tuple(w.b, w.h, w.rt)];
        if (v.empty()) v.assign(w.units, -1);
        CHECK((int)v.size() == w.units);
        for (int k = w.k0; k < w.k1; ++k) {
          CHECK(v[k] == -1);
          v[k] = cta;
          CHECK(kv_owner(w.first + k, U, G) == cta);
        }
      }
      const bool same = kv_next(w, heads);
      if (w.x >= w.xe) break;
      if (!same) {
        w.base = w.x;
        w.h = w.rt = 0;
        do ++w.b;
        while (seqs[w.b].T == 0);
        w.T = seqs[w.b].T;
        w.n = seqs[w.b].n;
      }
      kv_enter(c, w);
    }
  }
  for (int b = 0; b < (int)seqs.size(); ++b) {
    const int T = seqs[b].T, n = seqs[b].n;
    for (int h = 0; h < heads; ++h)
      for (int rt = 0; T && rt < kv_row_tiles(T, c.group, c.RT); ++rt) {
        auto it = got.find(std::make_tuple(b, h, rt));
        CHECK(it != got.end());
        for (int o : it->second) CHECK(o >= 0);
        const KvSpan s = kv_tile_span(T, n, c.group, c.RT, rt, c.causal, c.window);
        CHECK(kv_units(s, c.per) == (int)it->second.size());
        CHECK((long long)it->second.size() * c.per >= s.hi - s.lo && s.lo >= 0 && s.hi * 16 < n + 16);
        for (int r = rt * c.RT; r < (rt + 1) * c.RT && r < T * c.group; ++r) {
          int lo, hi;
          kv_token_keys(T, n, r / c.group, c.causal, c.window, lo, hi);
          for (int j = 0; j < n; j += 1 + n / 50) {   // the keys, from the definition
            const long long pos = (long long)n - T + r / c.group;
            const bool see = (!c.causal || j <= pos) && (!c.window || j > pos - c.window);
            CHECK(see == (j >= lo && j < hi));
          }
          if (lo < hi) CHECK(s.lo * 16 <= lo && hi <= s.hi * 16);
        }
      }
  }
  CHECK(got.size() > 0);
  return 0;
}

int main() {
  int n_checked = 0;
  unsigned rng = 12345;
  const auto next = [&](int m) {
    rng = rng * 1664525u + 1013904223u;
    return (int)(rng >> 8) % m;
  };
  for (int round = 0; round < 300; ++round) {
    const int RTs[] = {8, 16, 128, 256}, pers[] = {4, 8, 16}, extras[] = {0, 3, 8}, grids[] = {1, 7, 152, 304, 608};
    const KvShape c{1 + next(8), RTs[next(4)], pers[next(3)], extras[next(3)], next(2), next(3) ? 0 : 1 + next(300)};
    std::vector<Seq> seqs;
    const int batch = 1 + next(round % 5 ? 6 : 60), big = round % 7 ? 300 : 5000;
    for (int i = 0; i < batch; ++i) {
      const int T = next(4) ? (c.RT < 100 ? next(6) : next(400)) : next(2);
      seqs.push_back(Seq{T, next(5) ? next(big) : next(3)});
    }
    if (check(c, seqs, 1 + next(8), grids[next(5)])) {
      std::printf("round %d: group %d RT %d per %d extra %d causal %d window %d\n", round, c.group, c.RT, c.per,
                  c.extra, c.causal, c.window);
      return 1;
    }
    ++n_checked;
  }
  // past 32 bits
  const long long U = 5000000000ll;
  for (int c = 0; c < 608; ++c) CHECK(kv_owner(kv_first(U, c, 608), U, 608) == c);
  std::printf("ok %d batches\n", n_checked);
  return 0;
}
