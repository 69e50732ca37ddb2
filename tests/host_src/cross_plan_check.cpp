// Host check of cross_plan.h: over many shapes, every (batch, head, query tile, key block) is done by
// exactly one job (blocks past the keys excepted, whose keys are all masked), items stay within the
// launch rules the kernel relies on, and the query parts of the dk, dv kernel are in range.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <vector>

#include "cross_plan.h"

static int fail(const char* what, int a, int b, int c, int d) {
  std::printf("FAIL %s: %d %d %d %d\n", what, a, b, c, d);
  return 1;
}

int main() {
  unsigned seed = 1;
  auto rnd = [&](int n) {
    seed = seed * 1664525u + 1013904223u;
    return int((seed >> 8) % unsigned(n));
  };
  for (int t = 0; t < 4000; ++t) {
    const int B = 1 + rnd(3), hk = 1 + rnd(5), heads = hk * (1 + rnd(4));
    const int n = rnd(3) ? 1 + rnd(700) : 1 + rnd(20000), m = rnd(3) ? 1 + rnd(900) : 1 + rnd(30000);
    const sq::CrossPlan p = sq::make_cross_plan(B, heads, hk, n, m);
    if (p.splits != 1 && (p.splits % 2 || p.items > sq::kCrossPlanSms + 1)) return fail("splits", heads, n, m, p.splits);
    const int len = rnd(2) ? m : rnd(m + 1), nb = (len + 127) / 128;
    std::map<long long, int> seen;
    for (int i = 0; i < p.items; ++i) {
      const sq::CrossItem it = sq::cross_item(p, heads, i);
      if (it.b < 0 || it.b >= B || it.h < 0 || it.h >= heads || it.hk != it.h / (heads / hk))
        return fail("item", i, it.b, it.h, it.hk);
      if (p.splits > 1 && it.qt[1] < 0) return fail("split item with one job", i, n, m, p.splits);
      if (p.tiles == 1 && p.splits == 1 && it.qt[1] >= 0) return fail("two jobs", i, n, m, 0);
      int nk = -1;
      for (int x = 0; x < 2; ++x) {
        if (it.qt[x] < 0) continue;
        const sq::CrossRange r = sq::cross_range(p, len, it.sp[x]);
        if (it.qt[x] >= p.qtiles || r.nk < 1 || (nk >= 0 && nk != r.nk)) return fail("job", i, x, it.qt[x], r.nk);
        if (x == 1 && p.splits > 1 && r.k0 != sq::cross_range(p, len, it.sp[0]).k0 + r.nk) return fail("k0", i, x, r.k0, r.nk);
        nk = r.nk;
        for (int k = r.k0; k < r.k0 + r.nk; ++k) {
          if (k >= nb) continue;  // past the length: all masked
          ++seen[(((long long)it.b * heads + it.h) * p.qtiles + it.qt[x]) * 4096 + k];
        }
      }
    }
    if ((long long)seen.size() != (long long)B * heads * p.qtiles * nb) return fail("coverage", n, m, len, int(seen.size()));
    for (auto& kv : seen)
      if (kv.second != 1) return fail("twice", n, m, len, kv.second);
    const int tiles = 1 + rnd(500);
    const int s = sq::cross_dkv_splits(1 + rnd(300), tiles);
    if (s < 1 || s > tiles || s > 64) return fail("dkv splits", tiles, s, 0, 0);
    const int units = 1 + rnd(300), blocks = 1 + rnd(400), ds = sq::cross_dq_splits(units, blocks, rnd(2));
    if (ds < 1 || ds > 64 || (ds > 1 && (ds > blocks / 2 || ds * units > sq::kCrossPlanSms)))
      return fail("dq splits", units, blocks, ds, 0);
    const int d = 32 * (1 + rnd(8));
    const sq::CrossF32Dkdv fp = sq::cross_f32_dkdv_plan((long long)B * hk, heads / hk, n, m, d);
    if ((fp.rows != 1 && fp.rows != 2 && (fp.rows != 4 || d > 160)) || fp.splits < 1 || fp.splits > 64 ||
        fp.splits > (long long)(heads / hk) * ((n + 63) / 64))
      return fail("fp32 dk, dv plan", n, m, fp.rows, fp.splits);
  }
  std::printf("ok\n");
  return 0;
}
