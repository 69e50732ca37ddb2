// Host check of the fp32 dk, dv plan (cross_plan.h): the blocks that it lets share an SM fit there, for every head
// dimension and every tile that it may choose.
#include <cstdio>

#include "cross_plan.h"

// Bytes of a block of 16 r keys: k, v, 64 rows of q and dO (rows of d floats and 4 or 8 more), scores twice, statistics.
static int bytes(int d, int r) {
  const int ld = d + (r == 4 ? 4 : 8), score_row = (4 / r) * (16 * r + 4);
  return (2 * 16 * r * ld + 2 * 64 * ld + 2 * 16 * r * score_row + 2 * 64 + 16 * r) * 4;
}

int main() {
  unsigned seed = 3;
  auto rnd = [&](int n) {
    seed = seed * 1664525u + 1013904223u;
    return int((seed >> 8) % unsigned(n));
  };
  int most[9] = {};
  for (int t = 0; t < 40000; ++t) {
    const int d = 32 * (1 + rnd(8)), n = 1 + rnd(1 << (1 + rnd(13))), m = 1 + rnd(1 << (1 + rnd(13)));
    const sq::CrossF32Dkdv p = sq::cross_f32_dkdv_plan(1 + rnd(100), 1 + rnd(4), n, m, d);
    // 228 KB of an SM, 1 of them reserved for each block
    if (sq::cross_f32_dkdv_blocks(d) * (bytes(d, p.rows) + 1024) > 228 * 1024) {
      std::printf("FAIL d %d: %d blocks of %d keys, %d bytes each\n", d, sq::cross_f32_dkdv_blocks(d), 16 * p.rows,
                  bytes(d, p.rows));
      return 1;
    }
    if (p.rows > most[d / 32]) most[d / 32] = p.rows;
  }
  for (int i = 1; i <= 8; ++i)  // every tile that is built is chosen somewhere
    if (most[i] != sq::cross_f32_dkdv_rows(32 * i)) {
      std::printf("FAIL d %d: %d rows at most, built for %d\n", 32 * i, most[i], sq::cross_f32_dkdv_rows(32 * i));
      return 1;
    }
  std::printf("ok\n");
  return 0;
}
