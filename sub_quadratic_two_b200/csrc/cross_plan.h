// cross_plan.h - how a cross-attention forward is cut into work (host and device code).
//
// A job is one 128-query tile over a range of 128-key blocks; an item is two jobs of one
// (batch, head), run side by side on one SM. Where the query tiles fill the SMs, the jobs of
// an item are two neighbouring tiles over all keys, which share the key and value tiles in
// shared memory. Where there are no more tiles than SMs, an item takes one tile alone: a second
// SM is better than a shared tile (24 heads, d = 128, single / pairs: 144 tiles of 768 queries over
// 1,024 keys 20.6 / 22.7 us; 216 tiles of 1,100 over 512 keys 20.6 / 14.5). Where the keys are
// long as well, they are
// split over `splits` jobs, whose partial results a second kernel joins. The join and the fp32
// parts cost 4 to 10 us, more with more rows, and a key block saves 1.5 us at most, so the
// number of key blocks that makes a split worth it grows with the tiles (24 heads, d = 128,
// whole / split: 1 query x 512 keys 12.4 / 13.4 us, x 1,024 18.5 / 14.5, x 27,280 350 / 61;
// 384 x 1,024 18.6 / 20.6, x 4,096 57.5 / 32.9; 768 x 2,048 32.9 / 35.0, x 4,096 59.5 / 49.3).
#pragma once
#include <cstdint>
#include "geometry.h"

namespace sq {

constexpr int kCrossPlanSms = 148;  // the plan depends on sizes alone, so that results do too

struct CrossPlan {
  int qtiles;       // 128-row query tiles per (batch, head)
  int kblocks;      // 128-key blocks of m
  int tiles;        // query tiles per item: 2 (sharing keys) or 1
  int splits;       // jobs that share the keys of a query tile: even, or 1 (not split)
  int per_bh;       // items per (batch, head)
  int items;        // items in all
  FastDiv f_per_bh, f_heads, f_group, f_sp;
};

// (batch, head), query tile and key split of an item's two jobs.
struct CrossItem {
  int b, h, hk;
  int qt[2];   // query tile of each job, -1: none
  int sp[2];   // key split of each job
  bool shared; // both jobs read the same keys
};

inline CrossPlan make_cross_plan(int B, int heads, int kv_heads, int n, int m) {
  CrossPlan p{};
  p.qtiles = (n + 127) / 128;
  p.kblocks = (m + 127) / 128;
  const long long all = (long long)B * heads * p.qtiles;
  p.tiles = all > kCrossPlanSms ? 2 : 1;
  p.splits = 1;
  if (all <= kCrossPlanSms && p.kblocks >= 8 && (long long)p.kblocks * kCrossPlanSms >= 32 * all) {
    long long s = 2 * kCrossPlanSms / all;             // two jobs per SM
    const long long most = p.kblocks / 2;              // at least two blocks per job
    s = s < most ? s : most;
    p.splits = int(s < 64 ? s : 64) & ~1;              // an item holds two of them
    if (p.splits < 2) p.splits = 1;
  }
  if (p.splits > 1)
    p.per_bh = p.qtiles * (p.splits / 2);
  else
    p.per_bh = (p.qtiles + p.tiles - 1) / p.tiles;
  p.items = B * heads * p.per_bh;
  p.f_per_bh = make_fastdiv(uint32_t(p.per_bh));
  p.f_heads = make_fastdiv(uint32_t(heads));
  p.f_group = make_fastdiv(uint32_t(heads / kv_heads));
  p.f_sp = make_fastdiv(uint32_t(p.splits > 1 ? p.splits / 2 : 1));
  return p;
}

SQ_HD CrossItem cross_item(const CrossPlan& p, int heads, int i) {
  CrossItem it;
  const int bh = fdiv(i, p.f_per_bh), r = i - bh * p.per_bh;
  it.b = fdiv(bh, p.f_heads);
  it.h = bh - it.b * heads;
  it.hk = fdiv(it.h, p.f_group);
  if (p.splits > 1) {
    const int qt = fdiv(r, p.f_sp), s = 2 * (r - qt * (p.splits / 2));
    it.qt[0] = it.qt[1] = qt;
    it.sp[0] = s;
    it.sp[1] = s + 1;
    it.shared = false;
  } else {
    it.qt[0] = r * p.tiles;
    it.qt[1] = p.tiles == 2 && it.qt[0] + 1 < p.qtiles ? it.qt[0] + 1 : -1;
    it.sp[0] = it.sp[1] = 0;
    it.shared = it.qt[1] >= 0;
  }
  return it;
}

// Key blocks [k0, k0 + nk) of a job, for `len` keys that may count. nk is the same for every job
// of a batch row and at least 1: a job short of keys runs blocks past the length.
struct CrossRange {
  int k0, nk;
};
SQ_HD CrossRange cross_range(const CrossPlan& p, int len, int sp) {
  const int nb = (len + 127) >> 7;
  CrossRange r;
  r.nk = p.splits > 1 ? (nb + p.splits - 1) / p.splits : nb;
  if (r.nk < 1) r.nk = 1;
  r.k0 = sp * r.nk;
  return r;
}

// The longest that a wait of the tensor-core kernels may last, in ns: `base` and 20 us for every block
// (128 queries x 128 keys, of two jobs in the forward) that a CTA works on, `items` of `blocks` each spread
// over `ctas`. A block takes 1 to 4 us, so the kernel as a whole takes a fifth of it at most, and
// no wait is longer than the kernel: a role may sleep through all of it (the mask warp of a batch in
// which only the last row's length ends inside a block), or through a job of very many keys.
inline uint64_t cross_wait_ns(uint64_t base, long long items, long long ctas, long long blocks) {
  return base + 20000ull * uint64_t((items + ctas - 1) / ctas) * uint64_t(blocks);
}

// How many parts the keys of a query tile are cut into (dq kernels): `tiles` query tiles over
// `blocks` key blocks each. A part per idle SM, two blocks at least to a part. On the tensor cores
// only for long keys, as in the forward's plan (backward of 24 heads of 128, whole / split: 1 query x
// 1,024 keys 28.9 / 25.0 us, x 27,280 397 / 231; 384 x 1,024 37.2 / 41.2, x 2,048 55.1 / 53.6); a block
// of fp32 takes longer than the join (2 heads of 64, 200 x 300: 37.2 / 35.0 us; 8 heads, 100 x 500:
// 43.3 / 35.1, 1 x 4,096: 250 / 70).
inline int cross_dq_splits(long long tiles, int blocks, bool tc) {
  if (2 * tiles > kCrossPlanSms || blocks < (tc ? 8 : 4)) return 1;
  if (tc && (long long)blocks * kCrossPlanSms < 32 * tiles) return 1;
  long long s = kCrossPlanSms / tiles;
  s = s < blocks / 2 ? s : blocks / 2;
  return int(s < 64 ? s : 64);
}

// How many parts the queries of a key tile are cut into (dk, dv kernels): `units` key tiles of
// `tiles` query tiles each over the SMs, in the time of one query tile
// (1.2 to 1.8 us on the tensor cores at d = 128): rounds of units * s over the SMs, each
// ceil(tiles / s) tiles and 1.5 to fill and drain, plus, for s > 1, the join kernel (1.6) and its
// traffic (0.033 for each part of 128 keys). 4 x 8 heads of 128, 2,048 x 226: 31.6 us whole, 29.3 in
// two parts; 3 x 8 heads (4) of 64, 500 x 130: 15.2 and 12.7 in three.
inline int cross_dkv_splits(long long units, int tiles) {
  int best = 1;
  double best_cost = 0;
  for (int s = 1; s <= tiles && s <= 64; ++s) {
    if (s > 1 && units * s > 8 * kCrossPlanSms) break;  // more parts only add to the join
    const double rounds = double((units * s + kCrossPlanSms - 1) / kCrossPlanSms);
    const double cost = rounds * (double((tiles + s - 1) / s) + 1.5) + (s > 1 ? 1.6 + 0.033 * double(units) * s : 0.0);
    if (s == 1 || cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}

// Blocks of the fp32 dk, dv kernel that share an SM, a tile's loads under the other's products: two where the 128
// registers a thread that it leaves cost nothing (24 heads of 96, 300 x 300: 99 in place of 131 us); at d = 128
// they spill.
constexpr int cross_f32_dkdv_blocks(int d) { return d <= 96 ? 2 : 1; }
// The most keys of a block, in 16s: 64, or 32 where the registers (d > 160) or two blocks' shared memory (d = 96:
// 135 KB for 64 keys) do not hold more. One block of 64 keys in place of two of 32, d = 96: 8 heads, 4,096 x 1,024
// backward 1,956 for 1,760 us, 2,000 x 500 517 for 472.
constexpr int cross_f32_dkdv_rows(int d) { return d <= 64 || (d > 96 && d <= 160) ? 4 : 2; }

// The dk, dv kernel in fp32: 16 `rows` keys to a block, and parts of the queries of a key tile.
// The least of, in us (fitted to 12 sizes of 77 to 4,096 rows, to within a quarter): for each
// round of the blocks over the SMs, per 64 queries (1.1 + 2.2 rows) d / 64, and two thirds of that to
// begin and end; where two blocks share an SM together one and a half times as long;
// 2.5 and the parts' traffic where there is something to join. 16 rows and the parts of
// the rule above in its place: 17.1 for 8.3 us at 2 heads of 64, 256 x 77; 76 for 45 at 8 of 32,
// 1,500 x 200; 1,478 for 971 at 8 of 128, 4,096 x 1,024.
struct CrossF32Dkdv {
  int rows, splits;
};
inline CrossF32Dkdv cross_f32_dkdv_plan(long long kv_heads, int group, int n, int m, int d) {
  const long long tiles = (long long)group * ((n + 63) / 64);
  const long long share = cross_f32_dkdv_blocks(d), per = share * kCrossPlanSms;
  CrossF32Dkdv best{1, 1};
  double best_cost = 0;
  for (int r = 1; r <= cross_f32_dkdv_rows(d); r *= 2) {
    const long long units = kv_heads * ((m + 16 * r - 1) / (16 * r));
    const double step = (1.1 + 2.2 * r) * d / 64;
    for (int s = 1; s <= 64 && s <= tiles; ++s) {
      const long long blocks = units * s;
      if (s > 1 && blocks > 4 * per) break;  // more parts only add to the join
      const double rounds = double((blocks + per - 1) / per) * (share > 1 && blocks > kCrossPlanSms ? 1.5 : 1.0);
      const double cost = rounds * step * (double((tiles + s - 1) / s) + 0.67) +
                          (s > 1 ? 2.5 + 16.0 * s * double(kv_heads) * m * d / 4e6 : 0.0);
      if (best_cost == 0 || cost < best_cost) {
        best = CrossF32Dkdv{r, s};
        best_cost = cost;
      }
    }
  }
  return best;
}

}  // namespace sq
