// Host check of what attention over shared prefixes counts a tile for
// (branch_cost.h), the code that the kernels divide their work by.  Exit status 0 =
// all hold.
#include <cstdio>
#include <initializer_list>

#include "../bit_quantized_lm_amd/csrc/branch_cost.h"

static int failures = 0;
static void check(bool ok, const char* what, int D, int rows, int groups) {
  if (!ok && ++failures < 20) std::printf("%s: heads of %d, %d rows, %d groups\n", what, D, rows, groups);
}

template <int D>
void tiles() {
  using C = dl::Cost<D>;
  for (int groups : {0, 1, 4, 100, 1 << 20})
    for (int rows = 1; rows <= C::kRows; ++rows) {
      const int cost = C::of(rows, groups);
      const bool wave = C::kStreams && rows <= dl::kStreamRows;   // as the kernels take it
      check((cost == 0) == (groups == 0), "a tile that sees something takes time", D, rows, groups);
      // a workgroup's four waves have a tile each where the tile is a wave's
      const int workgroup = wave ? cost / 4 : cost;
      check(workgroup <= C::of(C::kRows, groups), "a rest takes no longer than a whole tile", D, rows, groups);
      if (!wave && rows <= dl::kSmallRows)
        check(cost == C::of(dl::kSmallRows, groups), "tiles of one kernel take one time", D, rows, groups);
      if (rows > 1 && rows != dl::kStreamRows + 1)
        check(cost >= C::of(rows - 1, groups), "more rows take no less", D, rows, groups);
    }
}

int main() {
  tiles<64>();
  tiles<128>();
  tiles<256>();
  if (failures) return 1;
  std::printf("ok\n");
  return 0;
}
