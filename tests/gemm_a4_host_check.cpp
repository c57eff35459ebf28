// Checks of csrc/gemm_a4_host.h on the host: prints "ok", or what is wrong.
#include "gemm_a4_host.h"

#include <cstdio>
#include <cstdlib>
#include <initializer_list>

using namespace moe::a4;

static void expect(bool ok, const char* what) {
  if (ok) return;
  std::printf("wrong: %s\n", what);
  std::exit(1);
}

// M rows as one group, N columns, 152 SMs: whether the product runs in narrow tiles
static bool narrow(int64_t M, int64_t N) { return narrow_tiles(row_tiles_at_most(M, 1, 128) * ((N + 255) / 256), 4, 152); }

int main() {
  for (int64_t m = 1; m <= 2000; ++m) expect(row_tiles_at_most(m, 1, 128) == (m + 127) / 128, "the tiles of one group");
  // the most tiles that `rows` rows can have in `groups` groups: single rows, and the rest in one
  for (int64_t groups = 1; groups <= 300; groups += 13)
    for (int64_t rows = groups; rows < groups + 700; rows += 3) {
      const int64_t last = rows - (groups - 1);
      expect(row_tiles_at_most(rows, groups, 128) >= groups - 1 + (last + 127) / 128, "a bound for groups");
    }
  // a batch of 128 rows has one row tile, not two: 28 wide tiles, all 112 narrow ones run at once
  expect(narrow(127, 7168) && narrow(128, 7168) && !narrow(129, 7168), "128 x 7168");
  expect(narrow(128, 9728) && !narrow(128, 9729), "128 rows on either side of 152 SMs");
  expect(narrow(256, 4864) && !narrow(256, 4865) && !narrow(257, 4864), "256 rows");
  // a tile of the longest K takes up to 1 us (2100 clocks) for each of its 2^23 blocks
  for (int64_t blocks : {int64_t(1), int64_t(28), int64_t(1) << 20, int64_t(1) << 23})
    expect(wait_limit(blocks) >= 4000000000LL && wait_limit(blocks) >= 2 * 2100 * blocks, "the wait of a long tile");
  std::printf("ok\n");
  return 0;
}
