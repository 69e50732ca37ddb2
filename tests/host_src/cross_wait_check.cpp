// Host check of cross_wait_ns (cross_plan.h): the limit of a wait covers every block that the busiest CTA of a launch
// works on, at five times the 4 us that a block takes at most, whatever the lengths; beyond it is only the base.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "cross_plan.h"

static int fail(const char* what, long long a, long long b, long long c) {
  std::printf("FAIL %s: %lld %lld %lld\n", what, a, b, c);
  return 1;
}

int main() {
  unsigned seed = 7;
  auto rnd = [&](int n) {
    seed = seed * 1664525u + 1013904223u;
    return int((seed >> 8) % unsigned(n));
  };
  const unsigned long long base = 2000000000ull, block = 20000ull;
  for (int t = 0; t < 3000; ++t) {
    const int B = 1 + rnd(4), hk = 1 + rnd(5), heads = hk * (1 + rnd(4));
    const int n = rnd(3) ? 1 + rnd(700) : 1 + rnd(20000), m = rnd(3) ? 1 + rnd(900) : 1 + rnd(30000);
    const sq::CrossPlan p = sq::make_cross_plan(B, heads, hk, n, m);
    const int sms = rnd(2) ? 148 : 1 + rnd(160), ctas = std::min(p.items, sms);
    std::vector<int> len(B);
    for (int& l : len) l = rnd(2) ? m : rnd(m + 1);
    std::vector<long long> work(ctas, 0);
    for (int i = 0; i < p.items; ++i) {
      const sq::CrossItem it = sq::cross_item(p, heads, i);
      work[i % ctas] += sq::cross_range(p, len[it.b], it.sp[0]).nk;
    }
    const unsigned long long limit = sq::cross_wait_ns(base, p.items, ctas, (p.kblocks + p.splits - 1) / p.splits);
    const long long most = *std::max_element(work.begin(), work.end());
    if (limit < base + block * most) return fail("limit below the work", n, m, most);
  }
  // 9 batch rows of 24 heads, 160,000 queries over 160,000 keys each, every length but the last row's a
  // multiple of 128: the mask warp sleeps through eight rows, 2.3 s
  const sq::CrossPlan p = sq::make_cross_plan(9, 24, 24, 160000, 160000);
  if (sq::cross_wait_ns(base, p.items, 148, p.kblocks) < 5ull * 2600000000ull) return fail("nine rows", p.items, p.kblocks, 0);
  // one key tile over very many: no overflow
  if (sq::cross_wait_ns(base, 1ll << 24, 148, 1ll << 24) < base + block * ((1ull << 48) / 148)) return fail("range", 0, 0, 0);
  std::printf("ok\n");
  return 0;
}
