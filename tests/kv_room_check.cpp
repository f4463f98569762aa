// The room that eviction and sparse attention give the numbers they choose
// from: it holds every stretch, and takes few sizes whatever the lengths are.
#include <cstdio>
#include <set>

#include "lw_kvroom.h"

using namespace lw;

int main() {
  int n = 0;
  for (int ranks = 1; ranks <= 8; ranks *= 2) {
    std::set<long long> sizes;
    long long before = 0;
    for (long long count = 0; count <= 400000; count += count < 70000 ? 1 : 37) {
      const long long room = kv_select_room(count, ranks);
      const int stretch = kv_select_stretch(count, ranks);
      // the stretches cover the numbers; the room covers a stretch, of fewer numbers too, and wastes less than a step
      if ((long long)stretch * ranks < count || stretch % 32 || room < stretch || room - stretch >= kSelectStep ||
          room < before) {
        std::printf("%lld numbers, %d ranks: stretch %d, room %lld\n", count, ranks, stretch, room);
        return 1;
      }
      before = room;
      sizes.insert(room);
      ++n;
    }
    if ((long long)sizes.size() > 400000 / ranks / kSelectStep + 3) {
      std::printf("%d ranks: %zu sizes\n", ranks, sizes.size());
      return 1;
    }
  }
  std::printf("ok %d counts\n", n);
  return 0;
}
