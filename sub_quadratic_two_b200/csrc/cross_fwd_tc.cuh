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
                       OF = PF + 4, OE = OF + 2, LF = OE + 2, ST = LF + 4, DRAIN = ST + 1, NBAR = DRAIN + 1;
  static constexpr int BYTES = BAR_OFF + NBAR * 8 + 16;  // + TMEM holder, abort flag
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

// What a visitor of the walk (below) is told about a product: the ring entry it reads is new,
// is done with, and the product is its job's first or last.
enum { CW_NEW = 1, CW_DONE = 2, CW_FIRST = 4, CW_LAST = 8 };

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
      mbar_init(&bars[Lay::PF + i], 4);      // keys 0-63 of P
      mbar_init(&bars[Lay::PF + 2 + i], 4);  // keys 64-127
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
  // The order of a CTA's products, which the loader, the masker and the MMA issuer share:
  // on_item(item, ranges of its two jobs), then for every block k and job x on_pv(x, entry,
  // flags) of the job's block before, if any, and on_s(x, entry, flags, k). entry counts the
  // key and value tiles in that order. Stops when a visitor returns false. The loops are not
  // unrolled: the code of a role is fetched once.
  auto walk = [&](auto&& on_item, auto&& on_pv, auto&& on_s) -> bool {
    uint32_t entries = 0, cur_k = 0, cur_v = 0;
    uint32_t pend = 0;  // flags of the job's block whose P V is still to come (16: there is one), 8 bits per job
#pragma unroll 1
    for (int i = blockIdx.x;; i += gridDim.x) {
      const bool more = i < plan.items;
      int nk0 = 0, nk1 = 0;
      bool shared = false;
      if (more) {
        const CrossItem it = cross_item(plan, args.heads, i);
        const int len = len_of(it.b);
        const CrossRange r0 = cross_range(plan, len, it.sp[0]);
        CrossRange r1 = r0;
        if (it.qt[1] < 0)
          r1.nk = 0;
        else if (!it.shared)
          r1 = cross_range(plan, len, it.sp[1]);
        nk0 = r0.nk;
        nk1 = r1.nk;
        shared = it.shared;
        on_item(it, r0, r1);
      }
      const int nk = more ? (nk0 > nk1 ? nk0 : nk1) : 1;
#pragma unroll 1
      for (int k = 0; k < nk; ++k) {
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const uint32_t f = (pend >> (8 * x)) & 255u;
          if (f) {
            pend &= ~(255u << (8 * x));
            if (f & CW_NEW) cur_v = entries++;
            if (!on_pv(x, cur_v, f)) return false;
          }
          const int nkx = x ? nk1 : nk0;
          if (k >= nkx) continue;
          const uint32_t g = (shared ? (x ? CW_DONE : CW_NEW) : (CW_DONE | CW_NEW)) | (k == 0 ? CW_FIRST : 0) |
                             (k == nkx - 1 ? CW_LAST : 0);
          if (g & CW_NEW) cur_k = entries++;
          if (!on_s(x, cur_k, g, k)) return false;
          pend |= (g | 16u) << (8 * x);
        }
      }
      if (!more) return true;
    }
  };

  if (warp >= 12) {
    if (warp == 12) {
      // ============================================================== key and value loads
      if (lane == 0) {
        uint32_t issued = 0;
        int kh = 0, kb = 0, vh = 0, vb = 0, k0[2] = {0, 0};
        int pvh[2], pvb[2], prow[2];  // head, batch and first row of each job's pending value tile
        auto load = [&](uint32_t e, const CUtensorMap* m, int row, int h, int b) -> bool {
          const uint32_t s = e % Lay::NKV;
          if (!mbar_wait(&bars[Lay::KVE + s], ((e / Lay::NKV) & 1) ^ 1, abort_flag, to)) return false;
          mbar_arrive_expect_tx(&bars[Lay::KVF + s], Lay::TILE);
#pragma unroll
          for (int c = 0; c < DH; ++c)
            tma_load_4d(sbase + Lay::KV_OFF + s * Lay::TILE + c * kCrossBlk, m, &bars[Lay::KVF + s], c * 64, row, h, b);
          issued = e + 1;
          return true;
        };
        walk(
            [&](const CrossItem& it, const CrossRange& r0, const CrossRange& r1) {
              kh = it.hk * args.k_h;
              kb = it.b * args.k_b;
              vh = it.hk * args.v_h;
              vb = it.b * args.v_b;
              k0[0] = r0.k0;
              k0[1] = r1.k0;
            },
            [&](int x, uint32_t e, uint32_t f) -> bool {
              return !(f & CW_NEW) || load(e, &maps.v, prow[x], pvh[x], pvb[x]);
            },
            [&](int x, uint32_t e, uint32_t f, int k) -> bool {
              prow[x] = (k0[x] + k) * 128;
              pvh[x] = vh;
              pvb[x] = vb;
              return !(f & CW_NEW) || load(e, &maps.k, prow[x], kh, kb);
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
            if (!(ok = mbar_wait(&bars[Lay::QE + s], ((q / Lay::NQ) & 1) ^ 1, abort_flag, to))) break;
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
        int b = 0, pb[2], prow[2], plim[2], k0[2], lim[2];
        // zero: value tiles; masked scores are replaced, so key tiles stay as they are
        auto fix = [&](uint32_t e, int b, int row, int limit, bool zero) -> bool {
          const uint32_t s = e % Lay::NKV;
          const bool ok = mbar_wait(&bars[Lay::KVF + s], (e / Lay::NKV) & 1, abort_flag, to);
          if (!__all_sync(0xffffffffu, ok)) return false;
          if (zero) {
            uint32_t w[4];
            block_words(limit - row, args.mask.keys == nullptr ? nullptr : args.mask.keys + b * args.mask.stride + row,
                        lane, w);
            zero_rows<D>(sbase + Lay::KV_OFF + s * Lay::TILE, w, lane);
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&bars[Lay::RDY + s]);
          return true;
        };
        walk(
            [&](const CrossItem& it, const CrossRange& r0, const CrossRange& r1) {
              b = it.b;
              k0[0] = r0.k0;
              k0[1] = r1.k0;
              lim[0] = r0.limit;
              lim[1] = r1.limit;
            },
            [&](int x, uint32_t e, uint32_t f) -> bool {
              return !(f & CW_NEW) || fix(e, pb[x], prow[x], plim[x], true);
            },
            [&](int x, uint32_t e, uint32_t f, int k) -> bool {
              pb[x] = b;
              prow[x] = (k0[x] + k) * 128;
              plim[x] = lim[x];
              return !(f & CW_NEW) || fix(e, b, prow[x], plim[x], false);
            });
      }
    } else if (warp == 13) {
      // ============================================================== MMA issuer
      if (lane == 0) {
        constexpr uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);
        constexpr uint32_t id_o = idesc_bf16_f32(128, D, 0, 1);
        constexpr int FULL = MASKED ? Lay::RDY : Lay::KVF;
        const uint64_t q0 = sdesc_sw128(sbase + Lay::Q_OFF, 16, 1024), k0 = sdesc_sw128(sbase + Lay::KV_OFF, 16, 1024),
                       v0 = sdesc_sw128(sbase + Lay::KV_OFF, kCrossBlk, 1024);
        uint32_t qn = 0;                  // query tiles taken
        uint32_t qslot = 0;               // query slot of each job, 8 bits each
        uint32_t par = 0, jpar = 0;       // bit x: parity of job slot x's P V products, of its jobs
        uint32_t begun = 0;               // bit x: job slot x has begun a job
        walk([](const CrossItem&, const CrossRange&, const CrossRange&) {},
             [&](int x, uint32_t e, uint32_t f) -> bool {
               const uint32_t s = e % Lay::NKV, p = (par >> x) & 1;
               if (!mbar_wait(&bars[FULL + s], (e / Lay::NKV) & 1, abort_flag, to)) return false;
               // the job's first product overwrites O: the epilogue has drained the last job's
               if (f & CW_FIRST) {
                 if (((begun >> x) & 1) && !mbar_wait(&bars[Lay::OE + x], ((jpar >> x) & 1) ^ 1, abort_flag, to))
                   return false;
                 begun |= 1u << x;
                 jpar ^= 1u << x;
               }
               if (!mbar_wait(&bars[Lay::PF + x], p, abort_flag, to)) return false;
               tc_fence_after();
               const uint64_t va = v0 + s * (Lay::TILE >> 4);
               const uint32_t o = tmem + 256 + D * x, a = tmem + 128 * x;
               mma_ts(o, a, va, id_o, f & CW_FIRST ? 0u : 1u);
#pragma unroll
               for (int kk = 1; kk < 4; ++kk) mma_ts(o, a + kk * 8, va + kk * (2048 >> 4), id_o, 1u);
               if (!mbar_wait(&bars[Lay::PF + 2 + x], p, abort_flag, to)) return false;
               tc_fence_after();
#pragma unroll
               for (int kk = 4; kk < 8; ++kk) mma_ts(o, a + kk * 8, va + kk * (2048 >> 4), id_o, 1u);
               if (f & CW_DONE) tc_commit(&bars[Lay::KVE + s]);
               if (f & CW_LAST) tc_commit(&bars[Lay::OF + x]);
               par ^= 1u << x;
               return true;
             },
             [&](int x, uint32_t e, uint32_t f, int) -> bool {
               const uint32_t s = e % Lay::NKV;
               if (f & CW_FIRST) {
                 const uint32_t z = qn % Lay::NQ;
                 if (!mbar_wait(&bars[Lay::QF + z], (qn / Lay::NQ) & 1, abort_flag, to)) return false;
                 qslot = x ? (qslot & 0xffu) | (z << 8) : (qslot & 0xff00u) | z;
                 ++qn;
               }
               if (!mbar_wait(&bars[FULL + s], (e / Lay::NKV) & 1, abort_flag, to)) return false;
               tc_fence_after();
               // S overwrites the columns that this job's previous P V reads P from: the tensor
               // core runs the products of one thread in issue order
               const uint64_t qa = q0 + ((qslot >> (8 * x)) & 255u) * (Lay::TILE >> 4), ka = k0 + s * (Lay::TILE >> 4);
#pragma unroll
               for (int kk = 0; kk < D / 16; ++kk) {
                 const uint32_t off = ((kk >> 2) * kCrossBlk + (kk & 3) * 32) >> 4;
                 mma_ss(tmem + 128 * x, qa + off, ka + off, id_s, kk > 0 ? 1u : 0u);
               }
               tc_commit(&bars[Lay::SF + x]);
               if (f & CW_DONE) tc_commit(&bars[Lay::KVE + s]);
               return true;
             });
        tc_commit(&bars[Lay::DRAIN]);
        mbar_wait_drain(&bars[Lay::DRAIN], 0, to);
      }
    }
  } else if (warp >= 8) {
    // ================================================================ epilogue
    const int row = threadIdx.x & 127;
    uint32_t q = 0, jobs[2] = {0, 0};
    bool ok = true;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, to)) != 0;
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
          ok = mbar_wait(&bars[Lay::ST], (q - 1) & 1, abort_flag, to);
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
    const int x = warp >> 2, row = threadIdx.x & 127;
    const uint32_t tS = tmem + (uint32_t((warp & 3) * 32) << 16) + 128 * x;
    const uint32_t tO = tmem + (uint32_t((warp & 3) * 32) << 16) + 256 + D * x;
    const float c2 = args.scale_log2;
    const uint64_t c2x2 = f2(c2, c2);
    uint32_t sc = 0, jobs = 0;
    bool ok = true;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, to)) != 0;
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
            mbar_arrive(&bars[Lay::PF + 2 + x]);
          }
          continue;
        }
        // a block that does not count whole: its masked scores become -inf where they lie
        if ((w[0] & w[1] & w[2] & w[3]) != ~0u) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint32_t word = c == 0 ? w[0] : c == 1 ? w[1] : c == 2 ? w[2] : w[3];
            if (word == ~0u) continue;
            uint32_t v[32];
            tmem_ld32(tS + 32 * c, v);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((word >> e) & 1u)) v[e] = 0xff800000u;
            tmem_st32(tS + 32 * c, v);
          }
          tmem_st_wait();
        }
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t v[64];
          tmem_ld64(tS + 64 * c, v);
          float a[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] = fmaxf(__uint_as_float(v[j]), __uint_as_float(v[j + 8]));
#pragma unroll
          for (int e = 16; e < 64; e += 16)
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = fmax3(a[j], __uint_as_float(v[e + j]), __uint_as_float(v[e + j + 8]));
          mx = fmax3(fmax3(mx, a[0], a[1]), fmax3(a[2], a[3], a[4]), fmax3(a[5], a[6], a[7]));
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
        // P of 64 keys at a time, packed over columns [32 c, 32 c + 32), whose scores are done with
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          if ((c ? w[2] | w[3] : w[0] | w[1]) == 0u) {  // no key counts: no exponentials
            tmem_st16_zero(tS + 32 * c);
            tmem_st16_zero(tS + 32 * c + 16);
          } else {
            uint32_t v[64], p[32];
            tmem_ld64(tS + 64 * c, v);
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              const uint64_t z = ffma2(f2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2x2, neg2);
              const float p0 = ex2_approx(f2_lo(z)), p1 = ex2_approx(f2_hi(z));
              sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], f2(p0, p1));
              p[e >> 1] = pack_bf16x2(p0, p1);
            }
            tmem_st32(tS + 32 * c, p);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::PF + 2 * c + x]);
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
