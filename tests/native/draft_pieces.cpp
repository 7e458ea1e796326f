// Which places of pieces the attention over the draft's cache takes from its
// workspace: those that a split pass can have written, and of other bytes only
// what stays within the workspace.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "internal.h"

int main() {
  int bad = 0;
  auto check = [&](int32_t segment, int32_t first, int32_t count, int32_t ranges, bool want) {
    if (ds::pieces_usable(segment, first, count, ranges) == want) return;
    ++bad;
    std::printf("segment %d, first %d, %d pieces, %d ranges: not %d\n", segment, first,
                count, ranges, want);
  };
  const int32_t most = std::numeric_limits<int32_t>::max(), least = -most - 1;
  for (int32_t segment : {0, 1, 767, 1 << 26})
    for (int32_t ranges : {1, 2, 304, 8192}) {
      const int32_t s = segment;
      check(segment, s, 1, ranges, true);
      check(segment, s, ranges, ranges, true);
      check(segment, s + ranges - 1, 1, ranges, true);
      check(segment, s + ranges - 1, 2, ranges, false);
      check(segment, s, ranges + 1, ranges, false);
      check(segment, s - 1, 1, ranges, false);
      check(segment, s, 0, ranges, false);
      check(segment, s, -1, ranges, false);            // bytes of 255
      check(segment, -1, -1, ranges, false);
      check(segment, s, most, ranges, false);
      check(segment, most, most, ranges, false);
      check(segment, least, 1, ranges, false);
      check(segment, least, least, ranges, false);
      // whatever the bytes are: no piece outside the places of all segments
      uint32_t x = 12345u + (uint32_t)ranges;
      for (int i = 0; i < 100000; ++i) {
        x = x * 1664525u + 1013904223u;
        const int32_t first = (int32_t)x >> (i % 31);
        x = x * 1664525u + 1013904223u;
        const int32_t count = (int32_t)x >> (i % 29);
        if (!ds::pieces_usable(segment, first, count, ranges)) continue;
        if (first < segment || count < 1 || count > ranges ||
            (int64_t)first + count > segment + ranges)
          check(segment, first, count, ranges, false);
      }
    }
  return bad != 0;
}
