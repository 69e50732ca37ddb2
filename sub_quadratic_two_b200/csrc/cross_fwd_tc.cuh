// cross_fwd_tc.cuh - forward of cross attention on the sm_100a tensor cores (bf16).
//
//   S = Q K^T,  P = exp(s S - max) over the keys that count,  O = P V / sum P
// with the running maximum and sum of each row in fp32. Work is cut by cross_plan.h into
// items of two jobs (a 128-query tile over a range of 128-key blocks); a CTA per SM takes
// items in turn.
//
// Roles (512 threads):
//   warps 0-3, 4-7  softmax of job 0, job 1 (thread = query row = TMEM lane)
//   warps 8-11      epilogue: O / sum -> bf16 -> the job's Q tile (no longer needed) in shared
//                   memory -> TMA store, so the softmax warps go on with the next item
//   warp 12         TMA loads of key and value tiles, one ring in consumption order
//   warp 13         one thread issues every tcgen05.mma
//   warp 14         masks: zeroes the masked rows of key and value tiles before they are used
//                   (what lies there may be NaN or infinite, and P = 0 times NaN is NaN)
//   warp 15         TMA loads of query tiles (four slots: an item ahead)
// TMEM (512 columns): S of job x at [128x, 128x+128), O at [256 + D x, ...). P overwrites S in
// place as packed bf16 and goes to the tensor core in two halves of 64 keys.
// The order of the products is S0(0) S1(0) | PV0(0) S0(1) | PV1(0) S1(1) | ...: while the
// tensor core works on one job, the other job's softmax runs.
// A block of 128 x 128 costs the tensor core 4 x 128 x 128 x D flops (1,024 cycles at D = 128)
// and the multi-function unit 128 x 128 exponentials (1,024 cycles at 16 a cycle): both are
// near their limit at once.
// Rounding: P to bf16 before P V (the tensor core's operand type); sums and statistics in
// fp32; O once at the end. Every wait is bounded (see sm100.cuh).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "cross_plan.h"
#include "cross_tc.cuh"

namespace sq {

constexpr int kCrossThreads = 512;
// Registers per thread: the eight softmax warps hold a whole row of scores (128), the others
// need few. 256 * 184 + 256 * 72 = 512 * 128, the block's share at launch.
constexpr int kCrossSoftmaxRegs = 184, kCrossOtherRegs = 72;

struct alignas(64) CrossMaps {
  CUtensorMap q, k, v, o;
};

struct CrossFwdArgs {
  CrossPlan plan;
  int B, heads, n, m;
  int q_b, q_h, k_b, k_h, v_b, v_h, o_b, o_h;  // 1, or 0 where the map has no such extent
  CrossMask mask;
  float scale_log2;
  float* lse;        // [B, heads, n] or nullptr (not split)
  float* part_o;     // split: [splits][B, heads, n][D] fp32
  float* part_lse;   // split: [splits][B, heads, n], base 2
  int* err;
  uint64_t timeout_ns;
};

template <int D>
struct CrossFwdLayout {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int NQ = 4;
  static constexpr int NKV = D == 128 ? 3 : 8;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = NQ * TILE;
  static constexpr int INV_OFF = KV_OFF + NKV * TILE;  // [job][parity][128] 1 / sum
  static constexpr int BAR_OFF = INV_OFF + 4 * 128 * 4;
  static constexpr int QF = 0, QE = NQ, KVF = 2 * NQ, KVE = KVF + NKV, RDY = KVE + NKV, SF = RDY + NKV, PF = SF + 2,
                       PF2 = PF + 2, OF = PF2 + 2, OE = OF + 2, LF = OE + 2, ST = LF + 4, DRAIN = ST + 1, NBAR = DRAIN + 1;
  static constexpr int BYTES = BAR_OFF + NBAR * 8 + 16;  // + TMEM holder, abort flag
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

// The order of a CTA's key and value tiles: the walk that the loader, the masker and the MMA
// issuer share. on_pv(x, e, first, last, free): P V of job x's pending block, values at ring
// entry e (new: this is the entry's first use; free: its last). on_s(x, e, new, free, it, r, k)
// likewise for the scores of block k.
struct CrossWalk {
  uint32_t entries = 0;
  uint32_t cur_k = 0, cur_v = 0;
  bool pend[2] = {false, false}, pend_first[2], pend_last[2], pend_new[2], pend_free[2];
  int pend_kb[2];
  CrossItem pend_it[2];
  int pend_limit[2];
};

template <int D, bool MASKED>
__global__ void __launch_bounds__(kCrossThreads, 1)
    cross_fwd_tc_kernel(const __grid_constant__ CrossMaps maps, const __grid_constant__ CrossFwdArgs args) {
  using Lay = CrossFwdLayout<D>;
  constexpr int DH = D / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::BAR_OFF + Lay::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::BAR_OFF + Lay::NBAR * 8 + 4);
  float* inv_sum = reinterpret_cast<float*>(smem + Lay::INV_OFF);
  const CrossPlan& plan = args.plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t to = args.timeout_ns;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it; dynamic shared memory starts aligned
    if (threadIdx.x == 0) atomicCAS(args.err, 0, 1);
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::NQ; ++i) {
      mbar_init(&bars[Lay::QF + i], 1);
      mbar_init(&bars[Lay::QE + i], 1);
    }
    for (int i = 0; i < Lay::NKV; ++i) {
      mbar_init(&bars[Lay::KVF + i], 1);
      mbar_init(&bars[Lay::KVE + i], 1);
      mbar_init(&bars[Lay::RDY + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[Lay::SF + i], 1);
      mbar_init(&bars[Lay::PF + i], 4);
      mbar_init(&bars[Lay::PF2 + i], 4);
      mbar_init(&bars[Lay::OF + i], 1);
      mbar_init(&bars[Lay::OE + i], 4);
      mbar_init(&bars[Lay::LF + 2 * i], 4);
      mbar_init(&bars[Lay::LF + 2 * i + 1], 4);
    }
    mbar_init(&bars[Lay::ST], 4);
    mbar_init(&bars[Lay::DRAIN], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == 12 && lane == 0) {
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    prefetch_tmap(&maps.o);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t sbase = smem_u32(smem);

  // Keys of batch row b that may count (the same row is asked for many times in a row).
  int len_b = -1, len_v = 0;
  auto len_of = [&](int b) -> int {
    if (!MASKED) return args.m;
    if (b != len_b) {
      len_v = cross_len(args.mask, b, args.m);
      len_b = b;
    }
    return len_v;
  };
  // Walks the CTA's products in issue order; stops when a visitor returns false.
  auto walk = [&](auto&& on_pv, auto&& on_s) -> bool {
    CrossWalk w;
    auto flush = [&](int x) -> bool {
      if (!w.pend[x]) return true;
      w.pend[x] = false;
      if (w.pend_new[x]) w.cur_v = w.entries++;
      return on_pv(x, w.cur_v, w.pend_new[x], w.pend_free[x], w.pend_first[x], w.pend_last[x], w.pend_it[x],
                   w.pend_kb[x], w.pend_limit[x]);
    };
    for (int i = blockIdx.x; i < plan.items; i += gridDim.x) {
      const CrossItem it = cross_item(plan, args.heads, i);
      const int len = len_of(it.b);
      const CrossRange r0 = cross_range(plan, len, it.sp[0]);
      const CrossRange r1 = it.qt[1] < 0 ? CrossRange{0, 0, 0} : cross_range(plan, len, it.sp[1]);
      const int nk = r0.nk > r1.nk ? r0.nk : r1.nk;
      for (int k = 0; k < nk; ++k) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!flush(x)) return false;
          const CrossRange& r = x ? r1 : r0;
          if (k >= r.nk) continue;
          const bool fresh = !it.shared || x == 0, done = !it.shared || x == 1;
          if (fresh) w.cur_k = w.entries++;
          if (!on_s(x, w.cur_k, fresh, done, k == 0, it, r.k0 + k, r.limit)) return false;
          w.pend[x] = true;
          w.pend_new[x] = fresh;
          w.pend_free[x] = done;
          w.pend_first[x] = k == 0;
          w.pend_last[x] = k == r.nk - 1;
          w.pend_it[x] = it;
          w.pend_kb[x] = r.k0 + k;
          w.pend_limit[x] = r.limit;
        }
      }
    }
    return flush(0) && flush(1);
  };

  if (warp >= 12) {
    regs_give<kCrossOtherRegs>();
    if (warp == 12) {
      // ================================================================ key and value loads
      if (lane == 0) {
        uint32_t issued = 0;
        auto load = [&](uint32_t e, const CUtensorMap* m, int h, int b, int kb) -> bool {
          const uint32_t s = e % Lay::NKV;
          if (!mbar_wait_inline(&bars[Lay::KVE + s], ((e / Lay::NKV) & 1) ^ 1, abort_flag, to)) return false;
          mbar_arrive_expect_tx(&bars[Lay::KVF + s], Lay::TILE);
#pragma unroll
          for (int c = 0; c < DH; ++c)
            tma_load_4d(sbase + Lay::KV_OFF + s * Lay::TILE + c * kCrossBlk, m, &bars[Lay::KVF + s], c * 64, kb * 128, h, b);
          issued = e + 1;
          return true;
        };
        walk(
            [&](int, uint32_t e, bool fresh, bool, bool, bool, const CrossItem& it, int kb, int) -> bool {
              return !fresh || load(e, &maps.v, it.hk * args.v_h, it.b * args.v_b, kb);
            },
            [&](int, uint32_t e, bool fresh, bool, bool, const CrossItem& it, int kb, int) -> bool {
              return !fresh || load(e, &maps.k, it.hk * args.k_h, it.b * args.k_b, kb);
            });
        // let every issued load land before the CTA may exit
        for (uint32_t s = 0; s < uint32_t(Lay::NKV); ++s) {
          const uint32_t uses = issued > s ? (issued - s + Lay::NKV - 1) / Lay::NKV : 0;
          if (uses) mbar_wait_drain(&bars[Lay::KVF + s], (uses - 1) & 1, to);
        }
      }
    } else if (warp == 15) {
      // ================================================================ query loads
      if (lane == 0) {
        uint32_t q = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
          const CrossItem it = cross_item(plan, args.heads, i);
          for (int x = 0; ok && x < 2; ++x) {
            if (it.qt[x] < 0) continue;
            const uint32_t s = q % Lay::NQ;
            if (!(ok = mbar_wait_inline(&bars[Lay::QE + s], ((q / Lay::NQ) & 1) ^ 1, abort_flag, to))) break;
            mbar_arrive_expect_tx(&bars[Lay::QF + s], Lay::TILE);
#pragma unroll
            for (int c = 0; c < DH; ++c)
              tma_load_4d(sbase + Lay::Q_OFF + s * Lay::TILE + c * kCrossBlk, &maps.q, &bars[Lay::QF + s], c * 64,
                          it.qt[x] * 128, it.h * args.q_h, it.b * args.q_b);
            ++q;
          }
        }
        for (uint32_t s = 0; s < uint32_t(Lay::NQ); ++s) {
          const uint32_t uses = q > s ? (q - s + Lay::NQ - 1) / Lay::NQ : 0;
          if (uses) mbar_wait_drain(&bars[Lay::QF + s], (uses - 1) & 1, to);
        }
      }
    } else if (warp == 14) {
      // ================================================================ masked rows to zero
      if (MASKED) {
        auto fix = [&](uint32_t e, const CrossItem& it, int kb, int limit, bool zero) -> bool {
          const uint32_t s = e % Lay::NKV;
          const bool ok = mbar_wait_inline(&bars[Lay::KVF + s], (e / Lay::NKV) & 1, abort_flag, to);
          if (!__all_sync(0xffffffffu, ok)) return false;
          if (zero) {
            uint32_t w[4];
            block_words(limit - kb * 128,
                        args.mask.keys == nullptr ? nullptr : args.mask.keys + it.b * args.mask.stride + kb * 128, lane, w);
            zero_rows<D>(sbase + Lay::KV_OFF + s * Lay::TILE, w, lane);
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&bars[Lay::RDY + s]);
          return true;
        };
        walk(
            [&](int, uint32_t e, bool fresh, bool, bool, bool, const CrossItem& it, int kb, int limit) -> bool {
              return !fresh || fix(e, it, kb, limit, true);
            },
            [&](int, uint32_t e, bool fresh, bool, bool, const CrossItem& it, int kb, int limit) -> bool {
              return !fresh || fix(e, it, kb, limit, false);  // masked scores are replaced, not multiplied
            });
      }
    } else if (warp == 13) {
      // ================================================================ MMA issuer
      if (lane == 0) {
        constexpr uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);
        constexpr uint32_t id_o = idesc_bf16_f32(128, D, 0, 1);
        constexpr int FULL = MASKED ? Lay::RDY : Lay::KVF;
        uint32_t qn = 0;                    // query tiles taken
        uint32_t blocks[2] = {0, 0};        // P V products issued per job slot
        uint32_t jobs[2] = {0, 0};          // jobs begun per job slot
        uint32_t qslot[2] = {0, 0};
        walk(
            [&](int x, uint32_t e, bool, bool done, bool first, bool last, const CrossItem&, int, int) -> bool {
              const uint32_t s = e % Lay::NKV, par = blocks[x] & 1;
              if (!mbar_wait_inline(&bars[FULL + s], (e / Lay::NKV) & 1, abort_flag, to)) return false;
              // the job's first product overwrites O: the epilogue has drained the last job's
              if (first) {
                if (jobs[x] > 0 && !mbar_wait_inline(&bars[Lay::OE + x], (jobs[x] - 1) & 1, abort_flag, to)) return false;
                ++jobs[x];
              }
              if (!mbar_wait_inline(&bars[Lay::PF + x], par, abort_flag, to)) return false;
              tc_fence_after();
              const uint32_t va = sbase + Lay::KV_OFF + s * Lay::TILE;
              const uint32_t o = tmem + 256 + D * x, p = tmem + 128 * x;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ts(o, p + kk * 8, sdesc_sw128(va + kk * 2048, kCrossBlk, 1024), id_o, (!first || kk > 0) ? 1u : 0u);
              if (!mbar_wait_inline(&bars[Lay::PF2 + x], par, abort_flag, to)) return false;
              tc_fence_after();
#pragma unroll
              for (int kk = 4; kk < 8; ++kk)
                mma_ts(o, p + kk * 8, sdesc_sw128(va + kk * 2048, kCrossBlk, 1024), id_o, 1u);
              if (done) tc_commit(&bars[Lay::KVE + s]);
              if (last) tc_commit(&bars[Lay::OF + x]);
              ++blocks[x];
              return true;
            },
            [&](int x, uint32_t e, bool, bool done, bool first, const CrossItem&, int, int) -> bool {
              const uint32_t s = e % Lay::NKV;
              if (!mbar_wait_inline(&bars[FULL + s], (e / Lay::NKV) & 1, abort_flag, to)) return false;
              if (first) {
                qslot[x] = qn % Lay::NQ;
                if (!mbar_wait_inline(&bars[Lay::QF + qslot[x]], (qn / Lay::NQ) & 1, abort_flag, to)) return false;
                ++qn;
              }
              tc_fence_after();
              // S overwrites the columns that this job's previous P V reads P from: the tensor
              // core runs the products of one thread in issue order
              const uint32_t qa = sbase + Lay::Q_OFF + qslot[x] * Lay::TILE, ka = sbase + Lay::KV_OFF + s * Lay::TILE;
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * kCrossBlk + (kk & 3) * 32;
                mma_ss(tmem + 128 * x, sdesc_sw128(qa + off, 16, 1024), sdesc_sw128(ka + off, 16, 1024), id_s,
                       kk > 0 ? 1u : 0u);
              }
              tc_commit(&bars[Lay::SF + x]);
              if (done) tc_commit(&bars[Lay::KVE + s]);
              return true;
            });
        tc_commit(&bars[Lay::DRAIN]);
        mbar_wait_drain(&bars[Lay::DRAIN], 0, to);
      }
    }
  } else if (warp >= 8) {
    // ================================================================ epilogue
    regs_give<kCrossOtherRegs>();
    const int row = threadIdx.x & 127;
    uint32_t q = 0, jobs[2] = {0, 0};
    bool ok = true;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, abort_flag, to)) != 0;
    };
    for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
      const CrossItem it = cross_item(plan, args.heads, i);
#pragma unroll 1
      for (int x = 0; ok && x < 2; ++x) {
        if (it.qt[x] < 0) continue;
        const uint32_t par = jobs[x] & 1, s = q % Lay::NQ;
        // two barriers in turn: the softmax may finish the next job before this wait begins
        if (!(ok = wwait(&bars[Lay::LF + 2 * x + par], (jobs[x] >> 1) & 1))) break;
        ++q;
        ++jobs[x];
        const float inv = inv_sum[(2 * x + par) * 128 + row];
        if (!(ok = wwait(&bars[Lay::OF + x], par))) break;
        tc_fence_after();
        const uint32_t t = tmem + (uint32_t((warp & 3) * 32) << 16) + 256 + D * x;
        const int tok = it.qt[x] * 128 + row;
        if (plan.splits > 1) {
          const long long r = (((long long)it.sp[x] * args.B + it.b) * args.heads + it.h) * args.n + tok;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t v[32];
            tmem_ld32(t + c, v);
            if (tok < args.n) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                float4 f = make_float4(__uint_as_float(v[e]) * inv, __uint_as_float(v[e + 1]) * inv,
                                       __uint_as_float(v[e + 2]) * inv, __uint_as_float(v[e + 3]) * inv);
                if (inv == 0.f) f = make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4*>(args.part_o + r * D + c + e) = f;
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::OE + x]);
          // the Q tile is free once its products are done, which this warp has waited for
          if (threadIdx.x == 256) mbar_arrive(&bars[Lay::QE + s]);
          continue;
        }
        const uint32_t stage = sbase + Lay::Q_OFF + s * Lay::TILE + row * 128;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          tmem_ld32(t + c, v);
          // 1 / sum is 0 for a row without keys; what the products hold there is not looked at
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = inv == 0.f ? 0u
                                : pack_bf16x2(__uint_as_float(v[8 * j + 2 * e]) * inv,
                                              __uint_as_float(v[8 * j + 2 * e + 1]) * inv);
            const int chunk = ((c & 32) >> 3) + j;
            st_shared_v4(stage + (c >> 6) * kCrossBlk + ((chunk ^ (row & 7)) << 4), p[0], p[1], p[2], p[3]);
          }
        }
        tc_fence_before();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[Lay::OE + x]);
          mbar_arrive(&bars[Lay::ST]);
        }
        if (threadIdx.x == 256) {  // stores the tile once all four warps have staged their rows
          ok = mbar_wait_inline(&bars[Lay::ST], (q - 1) & 1, abort_flag, to);
#pragma unroll
          for (int c = 0; ok && c < DH; ++c)
            tma_store_4d(&maps.o, sbase + Lay::Q_OFF + s * Lay::TILE + c * kCrossBlk, c * 64, it.qt[x] * 128,
                         it.h * args.o_h, it.b * args.o_b);
          bulk_commit();
          bulk_wait_read();
          mbar_arrive(&bars[Lay::QE + s]);
        }
        ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
      }
    }
  } else {
    // ================================================================ softmax
    regs_take<kCrossSoftmaxRegs>();
    const int x = warp >> 2, row = threadIdx.x & 127;
    const uint32_t tS = tmem + (uint32_t((warp & 3) * 32) << 16) + 128 * x;
    const uint32_t tO = tmem + (uint32_t((warp & 3) * 32) << 16) + 256 + D * x;
    const float c2 = args.scale_log2;
    const uint64_t c2x2 = f2(c2, c2);
    uint32_t sc = 0, jobs = 0;
    bool ok = true;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, abort_flag, to)) != 0;
    };
    for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
      const CrossItem it = cross_item(plan, args.heads, i);
      const int qt = x ? it.qt[1] : it.qt[0];
      if (qt < 0) continue;
      const CrossRange r = cross_range(plan, len_of(it.b), x ? it.sp[1] : it.sp[0]);
      const int tok = qt * 128 + row;
      // a warp whose rows all lie past the last query has nothing to compute
      const bool idle = qt * 128 + (warp & 3) * 32 >= args.n;
      const unsigned char* keys =
          !MASKED || args.mask.keys == nullptr ? nullptr : args.mask.keys + it.b * args.mask.stride + r.k0 * 128;
      float m_run = -INFINITY, l_run = 0.f;
      for (int k = 0; k < r.nk; ++k, ++sc) {
        const int limit = r.limit - (r.k0 + k) * 128;
        uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
        if (limit < 128 || (MASKED && keys != nullptr))
          block_words(limit, keys == nullptr ? nullptr : keys + k * 128, lane, w);
        if (!(ok = wwait(&bars[Lay::SF + x], sc & 1))) break;
        tc_fence_after();
        if (idle) {
          tc_fence_before();
          if (lane == 0) {
            mbar_arrive(&bars[Lay::PF + x]);
            mbar_arrive(&bars[Lay::PF2 + x]);
          }
          continue;
        }
        // ---- row maximum; masked scores become -inf
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_async(tS + 32 * c, v[c]);
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait(v[c]);
          if (w[c] != ~0u) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((w[c] >> e) & 1u)) v[c][e] = 0xff800000u;
          }
          float a[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = fmaxf(__uint_as_float(v[c][j]), __uint_as_float(v[c][j + 4]));
#pragma unroll
          for (int e = 8; e < 32; e += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = fmax3(a[j], __uint_as_float(v[c][e + j]), __uint_as_float(v[c][e + j + 4]));
          mx = fmax3(mx, fmax3(a[0], a[1], a[2]), a[3]);
        }
        // the first block sets the maximum; a later one moves it only when it grows by more
        // than 2^8 (then O and the sum are rescaled), else its probabilities may exceed 1
        float m_use = mx, alpha = 1.f;
        bool grow = false;
        if (k > 0) {
          grow = (mx - m_run) * c2 > 8.f;
          m_use = grow ? mx : m_run;
          alpha = grow ? ex2_approx((m_run - mx) * c2) : 1.f;
          if (__any_sync(0xffffffffu, grow)) {
            // the previous P V has completed: S of this block was issued behind it
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(tO + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + c, o);
            }
          }
        }
        const float neg = m_use == -INFINITY ? 0.f : -m_use * c2;  // a row without keys: every exponent is -inf
        const uint64_t neg2 = f2(neg, neg);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (w[c] == 0u) {  // no key in this chunk: no exponentials
            tmem_st16_zero(tS + 16 * c);
          } else {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const uint64_t z = ffma2(f2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), c2x2, neg2);
              const float p0 = ex2_approx(f2_lo(z)), p1 = ex2_approx(f2_hi(z));
              sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], f2(p0, p1));
              p[e >> 1] = pack_bf16x2(p0, p1);
            }
            tmem_st16(tS + 16 * c, p);
          }
          if (c & 1) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[(c == 1 ? Lay::PF : Lay::PF2) + x]);
          }
        }
        const uint64_t s2 = fadd2(sum[0], sum[1]);
        l_run = l_run * alpha + (f2_lo(s2) + f2_hi(s2));
        m_run = m_use;
      }
      if (!ok) break;
      const float inv = l_run > 0.f ? 1.f / l_run : l_run == 0.f ? 0.f : l_run;  // NaN stays NaN
      inv_sum[(2 * x + (jobs & 1)) * 128 + row] = inv;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Lay::LF + 2 * x + (jobs & 1)]);
      ++jobs;
      if (tok < args.n) {
        const float l2 = l_run == 0.f ? -INFINITY : m_run * c2 + log2f(l_run);
        const long long rr = ((long long)it.b * args.heads + it.h) * args.n + tok;
        if (plan.splits > 1)
          args.part_lse[(long long)(x ? it.sp[1] : it.sp[0]) * args.B * args.heads * args.n + rr] = l2;
        else if (args.lse != nullptr)
          args.lse[rr] = l2 * 0.69314718055994530942f;
      }
    }
  }

  __syncthreads();
  if (*abort_flag && threadIdx.x == 0 && args.err != nullptr) atomicCAS(args.err, 0, 1);
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the key splits of a row: o = sum_s 2^(l_s - max) o_s / sum_s 2^(l_s - max), with
// l_s = log2 of the split's sum. One warp per row, lanes over the channels.
template <int D>
__global__ void __launch_bounds__(128) cross_join_kernel(const float* __restrict__ part_o,
                                                         const float* __restrict__ part_lse, int splits,
                                                         long long rows, int heads, int n, __nv_bfloat16* o,
                                                         CrossStride so, float* lse) {
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float mx = -INFINITY;
  for (int s = lane; s < splits; s += 32) mx = fmaxf(mx, part_lse[s * rows + row]);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  constexpr int C = D / 32;
  float acc[C], total = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  if (mx != -INFINITY) {
    for (int s = 0; s < splits; ++s) {
      const float wt = exp2f(part_lse[s * rows + row] - mx);
      total += wt;
      const float* p = part_o + (s * rows + row) * D + lane * C;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = fmaf(wt, p[c], acc[c]);
    }
  }
  const float inv = total > 0.f ? 1.f / total : total;
  const long long bh = row / n;
  const int i = int(row - bh * n), b = int(bh / heads), h = int(bh - (long long)b * heads);
  __nv_bfloat16* out = o + b * so.b + h * so.h + i * so.n + lane * C;
#pragma unroll
  for (int c = 0; c < C; c += 2)
    *reinterpret_cast<uint32_t*>(out + c) = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
  if (lse != nullptr && lane == 0) lse[row] = total > 0.f ? (mx + log2f(total)) * 0.69314718055994530942f : mx;
}

}  // namespace sq
