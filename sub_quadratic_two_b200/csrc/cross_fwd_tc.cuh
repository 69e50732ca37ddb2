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
//                   memory -> TMA store, so the softmax warps go on with the next item; their
//                   first thread then loads the job's query tile of the item after next there
//   warp 12         TMA loads of key and value tiles, K(0) V(0) K(1) V(1) ... in a ring (a ring for
//                   each job where the keys are split)
//   warps 13, 15    one thread each issues the tcgen05.mma of job 0, job 1: what a thread spends
//                   between its products (waits, addresses: some 100 cycles each) passes under
//                   the products of the other
//   warp 14         masks: zeroes the masked rows of value tiles before they are used (what lies
//                   there may be NaN or infinite, and P = 0 times NaN is NaN)
// TMEM (512 columns): S of job x at [128x, 128x+128), O at [256 + D x, ...). P overwrites S in
// place as packed bf16 and goes to the tensor core in two halves of 64 keys.
// Each job's products run S(0) | PV(0) S(1) | PV(1) S(2) | ...; while the tensor core works on
// one job, the other job's softmax runs.
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
  static constexpr int NQ = 4;  // query tile of job x of the CTA's j-th item: slot 2 (j & 1) + x
  static constexpr int NKV = D == 128 ? 3 : 8;  // ring of key and value tiles, behind the query tiles
  // Split keys: a CTA has one item, so query slots 2 and 3 are free, and each job takes half of
  // the tiles behind slot 1 as a ring of its own. (With one ring for both, an issuer would not
  // see the phases of the tiles that the other job reads, and a wait by parity needs every phase.)
  static constexpr int NS = (NKV + 2) / 2;
  static constexpr int NB = NKV > 2 * NS ? NKV : 2 * NS;  // ring barriers of each kind
  static constexpr int BAR_OFF = (NQ + NKV) * TILE;
  static constexpr int QF = 0, KVF = QF + NQ, KVE = KVF + NB, RDY = KVE + NB, SF = RDY + NB, PF = SF + 2, OF = PF + 4,
                       OE = OF + 2, LF = OE + 2, ST = LF + 4, DRAIN = ST + 2, NBAR = DRAIN + 2;
  static constexpr int BYTES = BAR_OFF + NBAR * 8 + 16;  // + TMEM holder, abort flag
  static_assert(BYTES <= 232448, "shared memory of one CTA");
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
  const CrossPlan& plan = args.plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t to = args.timeout_ns;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it; dynamic shared memory starts aligned
    if (threadIdx.x == 0) atomicCAS(args.err, 0, 1);
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::NBAR; ++i) {
      // key and value tiles are released by both issuers (or twice by the only one that reads
      // them); the softmax and epilogue warps arrive one by one
      const int count = i >= Lay::KVE && i < Lay::RDY ? 2
                        : (i >= Lay::PF && i < Lay::OF) || (i >= Lay::OE && i < Lay::DRAIN) ? 4 : 1;
      mbar_init(&bars[i], count);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 14) {  // a warp whose lanes stay together: TMEM is taken and given back by whole warps
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

  // Rings of key and value tiles: entry n of job x (or of both) lies in slot(x, n), for the
  // use(n)-th time.
  struct Ring {
    uint32_t size, tile0;
    int count;
    __device__ __forceinline__ uint32_t slot(int x, uint32_t n) const {
      return (count == 2 ? x * size : 0u) + n % size;
    }
    __device__ __forceinline__ uint32_t use(uint32_t n) const { return n / size; }
  };
  const Ring ring = plan.splits > 1 ? Ring{uint32_t(Lay::NS), 2u, 2} : Ring{uint32_t(Lay::NKV), uint32_t(Lay::NQ), 1};

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
  if (warp >= 12) {
    if (warp == 12) {
      // ============================================================== key and value loads
      if (lane == 0) {
        uint32_t e[2] = {0, 0};
        auto load = [&](int x, const CUtensorMap* m, int row, int h, int b) -> bool {
          const uint32_t n = x ? e[1] : e[0], s = ring.slot(x, n);
          if (!mbar_wait(&bars[Lay::KVE + s], (ring.use(n) & 1) ^ 1, abort_flag, to)) return false;
          mbar_arrive_expect_tx(&bars[Lay::KVF + s], Lay::TILE);
#pragma unroll
          for (int c = 0; c < DH; ++c)
            tma_load_4d(sbase + (ring.tile0 + s) * Lay::TILE + c * kCrossBlk, m, &bars[Lay::KVF + s], c * 64, row, h, b);
          x ? ++e[1] : ++e[0];
          return true;
        };
        bool ok = true;
        for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
          const CrossItem it = cross_item(plan, args.heads, i);
          const CrossRange r = cross_range(plan, len_of(it.b), it.sp[0]);
          const int kh = it.hk * args.k_h, kb = it.b * args.k_b, vh = it.hk * args.v_h, vb = it.b * args.v_b;
          // values of block k - 1, then keys of block k
          for (int k = 0; ok && k <= r.nk; ++k)
            for (int x = 0; ok && x < ring.count; ++x) {
              const int row = (r.k0 + x * r.nk + k) * 128;
              if (k > 0) ok = load(x, &maps.v, row - 128, vh, vb);
              if (ok && k < r.nk) ok = load(x, &maps.k, row, kh, kb);
            }
        }
        // let every issued load land before the CTA may exit
        for (int x = 0; x < ring.count; ++x) {
          const uint32_t n = x ? e[1] : e[0];
          for (uint32_t s = 0; s < ring.size; ++s)
            if (n > s) mbar_wait_drain(&bars[Lay::KVF + x * ring.size + s], ((n - 1 - s) / ring.size) & 1, to);
        }
      }
    } else if (warp == 14) {
      // ============================================================== masked value rows to zero
      if (MASKED) {
        uint32_t e[2] = {0, 0};
        // masked scores are replaced, so key tiles are passed on as they are
        auto pass = [&](int x, bool value, int b, int row, int limit) -> bool {
          const uint32_t n = x ? e[1] : e[0], s = ring.slot(x, n);
          const bool ok = mbar_wait(&bars[Lay::KVF + s], ring.use(n) & 1, abort_flag, to);
          if (!__all_sync(0xffffffffu, ok)) return false;
          if (value) {
            uint32_t w[4];
            block_words(limit - row, args.mask.keys == nullptr ? nullptr : args.mask.keys + b * args.mask.stride + row,
                        lane, w);
            zero_rows<D>(sbase + (ring.tile0 + s) * Lay::TILE, w, lane);
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&bars[Lay::RDY + s]);
          x ? ++e[1] : ++e[0];
          return true;
        };
        bool ok = true;
        for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
          const CrossItem it = cross_item(plan, args.heads, i);
          const int len = len_of(it.b);
          const CrossRange r = cross_range(plan, len, it.sp[0]);
          for (int k = 0; ok && k <= r.nk; ++k)
            for (int x = 0; ok && x < ring.count; ++x) {
              const int row = (r.k0 + x * r.nk + k) * 128;
              if (k > 0) ok = pass(x, true, it.b, row - 128, len);
              if (ok && k < r.nk) ok = pass(x, false, it.b, row, len);
            }
        }
      }
    } else if (lane == 0) {
      // ============================================================== MMA issuer of job x
      const int x = warp == 13 ? 0 : 1;
      constexpr uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t id_o = idesc_bf16_f32(128, D, 0, 1);
      constexpr int FULL = MASKED ? Lay::RDY : Lay::KVF;
      const uint64_t q0 = sdesc_sw128(sbase + x * Lay::TILE, 16, 1024),
                     k0 = sdesc_sw128(sbase + ring.tile0 * Lay::TILE, 16, 1024),
                     v0 = sdesc_sw128(sbase + ring.tile0 * Lay::TILE, kCrossBlk, 1024);
      const uint32_t ts = tmem + 128 * x, tacc = tmem + 256 + D * x;
      uint32_t e = 0;                    // key and value tiles of earlier blocks
      uint32_t item = 0;                // items begun
      uint32_t jobs = 0, blocks = 0;    // jobs and P V products of this issuer
      uint32_t quse = 0;                // parity of the two query slots' uses
      uint32_t ve = 0;                  // the pending block: its value tile, place and release
      bool pending = false, pfirst = false, plast = false;
      int i = blockIdx.x, k = 0, nk = 0;
      // Tiles are released by both issuers, also by the one that has no job at an item (it passes
      // over them, so that it sees every phase of their barriers); where one issuer alone reads
      // them (one tile per item, or split keys), it releases them twice.
      const bool alone = plan.tiles == 1 || plan.splits > 1;
      if (x == 1 && plan.tiles == 1 && plan.splits == 1) i = plan.items;  // no jobs in this slot
      for (;;) {
        if (pending) {  // P V
          const uint32_t s = ring.slot(x, ve), p = blocks & 1;
          if (!mbar_wait(&bars[FULL + s], ring.use(ve) & 1, abort_flag, to)) break;
          // the job's first product overwrites O: the epilogue has drained the last job's
          if (pfirst) {
            if (jobs > 0 && !mbar_wait(&bars[Lay::OE + x], (jobs - 1) & 1, abort_flag, to)) break;
            ++jobs;
          }
          const uint64_t va = v0 + s * (Lay::TILE >> 4);
          if (!mbar_wait(&bars[Lay::PF + x], p, abort_flag, to)) break;
          tc_fence_after();
          mma_ts(tacc, ts, va, id_o, pfirst ? 0u : 1u);
#pragma unroll
          for (int kk = 1; kk < 4; ++kk) mma_ts(tacc, ts + kk * 8, va + kk * (2048 >> 4), id_o, 1u);
          if (!mbar_wait(&bars[Lay::PF + 2 + x], p, abort_flag, to)) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 4; kk < 8; ++kk) mma_ts(tacc, ts + kk * 8, va + kk * (2048 >> 4), id_o, 1u);
          tc_commit(&bars[Lay::KVE + s]);
          if (alone) tc_commit(&bars[Lay::KVE + s]);
          if (plast) tc_commit(&bars[Lay::OF + x]);
          ++blocks;
          pending = false;
        }
        // the next block of this job slot: moves on to the next item that has one
        bool ok = true;
        while (ok && k >= nk && i < plan.items) {
          const CrossItem it = cross_item(plan, args.heads, i);
          nk = cross_range(plan, len_of(it.b), it.sp[0]).nk;
          k = 0;
          if (x == 1 && it.qt[1] < 0) {
            for (const uint32_t end = e + 2 * nk; ok && e != end; ++e) {
              const uint32_t s = ring.slot(x, e);
              ok = mbar_wait(&bars[FULL + s], ring.use(e) & 1, abort_flag, to);
              if (ok) mbar_arrive(&bars[Lay::KVE + s]);
            }
            nk = 0;
          }
          i += gridDim.x;
          ++item;
        }
        if (!ok || k >= nk) break;
        // S overwrites the columns that the P V above reads P from: the tensor core runs the
        // products of one thread in issue order
        const uint32_t slot = (item - 1) & 1, s = ring.slot(x, e);
        if (k == 0) {
          if (!mbar_wait(&bars[Lay::QF + 2 * slot + x], (quse >> slot) & 1, abort_flag, to)) break;
          quse ^= 1u << slot;
        }
        if (!mbar_wait(&bars[FULL + s], ring.use(e) & 1, abort_flag, to)) break;
        tc_fence_after();
        const uint64_t qa = q0 + slot * (2 * Lay::TILE >> 4), ka = k0 + s * (Lay::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kCrossBlk + (kk & 3) * 32) >> 4;
          mma_ss(ts, qa + off, ka + off, id_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(&bars[Lay::SF + x]);
        tc_commit(&bars[Lay::KVE + s]);
        if (alone) tc_commit(&bars[Lay::KVE + s]);
        ve = e + 1;
        e += 2;
        pending = true;
        pfirst = k == 0;
        plast = k == nk - 1;
        ++k;
      }
      tc_commit(&bars[Lay::DRAIN + x]);
      mbar_wait_drain(&bars[Lay::DRAIN + x], 0, to);
    }
  } else if (warp >= 8) {
    // ================================================================ epilogue
    const int row = threadIdx.x & 127;
    uint32_t jobs = 0;              // jobs of each slot so far (a byte each, mod 256)
    uint32_t qused = 0, qpar = 0;   // per query slot: ever loaded, parity of its loads
    bool ok = true;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, to)) != 0;
    };
    // the query tile of job x of item i into slot s, where there is such a job
    auto load_q = [&](long long i, int x, uint32_t s) {
      if (i >= plan.items) return;
      const CrossItem it = cross_item(plan, args.heads, int(i));
      const int qt = x ? it.qt[1] : it.qt[0];
      if (qt < 0) return;
      mbar_arrive_expect_tx(&bars[Lay::QF + s], Lay::TILE);
#pragma unroll
      for (int c = 0; c < DH; ++c)
        tma_load_4d(sbase + s * Lay::TILE + c * kCrossBlk, &maps.q, &bars[Lay::QF + s], c * 64, qt * 128,
                    it.h * args.q_h, it.b * args.q_b);
      qused |= 1u << s;
      qpar ^= 1u << s;
    };
    if (threadIdx.x == 256) {
#pragma unroll 1
      for (int s = 0; s < 4; ++s) load_q((long long)blockIdx.x + (s >> 1) * (long long)gridDim.x, s & 1, s);
    }
    __syncwarp();
    uint32_t item = 0;
#pragma unroll 1
    for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x, ++item) {
      const CrossItem it = cross_item(plan, args.heads, i);
#pragma unroll 1
      for (int x = 0; ok && x < 2; ++x) {
        const uint32_t s = 2 * (item & 1) + x;
        const int qt = x ? it.qt[1] : it.qt[0];
        if (qt < 0) {
          if (threadIdx.x == 256) load_q(i + 2ll * gridDim.x, x, s);
          __syncwarp();
          continue;
        }
        const uint32_t job = (jobs >> (8 * x)) & 255u;
        jobs = x ? (jobs & 0xffu) | ((job + 1) & 255u) << 8 : (jobs & 0xff00u) | ((job + 1) & 255u);
        // two barriers in turn: the softmax may finish the next job before this wait begins
        if (!(ok = wwait(&bars[Lay::LF + 2 * x + (job & 1)], (job >> 1) & 1))) break;
        const uint32_t tile = sbase + s * Lay::TILE;
        float m2, l;  // maximum (base 2) and sum of the row
        ld_shared_f2(tile + (row >> 5) * 4096 + lane * 8, m2, l);
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // NaN stays NaN
        const int tok = qt * 128 + row;
        if (tok < args.n) {
          const float l2 = l == 0.f ? -INFINITY : m2 + log2f(l);
          const long long r = ((long long)it.b * args.heads + it.h) * args.n + tok;
          if (plan.splits > 1)
            args.part_lse[(long long)(it.sp[0] + x) * args.B * args.heads * args.n + r] = l2;
          else if (args.lse != nullptr)
            args.lse[r] = l2 * 0.69314718055994530942f;
        }
        __syncwarp();  // the statistics are read before the rows of this warp are staged over them
        if (!(ok = wwait(&bars[Lay::OF + x], job & 1))) break;
        tc_fence_after();
        const uint32_t t = tmem + (uint32_t((warp & 3) * 32) << 16) + 256 + D * x;
        if (plan.splits > 1) {
          const long long r = (((long long)(it.sp[0] + x) * args.B + it.b) * args.heads + it.h) * args.n + tok;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t v[32];
            __syncwarp();  // lanes part below: TMEM is read by whole warps
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
          if (lane == 0) {
            mbar_arrive(&bars[Lay::ST + x]);
            mbar_arrive(&bars[Lay::OE + x]);
          }
          // the statistics of every warp's rows are read before the next query tile comes
          if (threadIdx.x == 256) {
            ok = mbar_wait(&bars[Lay::ST + x], job & 1, abort_flag, to);
            if (ok) load_q(i + 2ll * gridDim.x, x, s);
          }
          ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
          continue;
        }
        const uint32_t stage = tile + row * 128;
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
        // ST before OE: the next job of this slot, and so the next arrivals at its ST, wait for OE,
        // so no warp can arrive for it while another has yet to arrive for this job
        if (lane == 0) {
          mbar_arrive(&bars[Lay::ST + x]);
          mbar_arrive(&bars[Lay::OE + x]);
        }
        if (threadIdx.x == 256) {  // stores the tile once all four warps have staged their rows
          ok = mbar_wait(&bars[Lay::ST + x], job & 1, abort_flag, to);
#pragma unroll
          for (int c = 0; ok && c < DH; ++c)
            tma_store_4d(&maps.o, tile + c * kCrossBlk, c * 64, qt * 128, it.h * args.o_h, it.b * args.o_b);
          bulk_commit();
          bulk_wait_read();
          if (ok) load_q(i + 2ll * gridDim.x, x, s);
        }
        ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
      }
    }
    if (threadIdx.x == 256)
      for (int s = 0; s < 4; ++s)
        if ((qused >> s) & 1u) mbar_wait_drain(&bars[Lay::QF + s], ((qpar >> s) & 1u) ^ 1u, to);
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
    uint32_t item = 0;
    for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x, ++item) {
      const CrossItem it = cross_item(plan, args.heads, i);
      const int qt = x ? it.qt[1] : it.qt[0];
      if (qt < 0) continue;
      const CrossRange r = cross_range(plan, len_of(it.b), x ? it.sp[1] : it.sp[0]);
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
      // the row's statistics for the epilogue, in the query tile that no product reads any more
      st_shared_f2(sbase + (2 * (item & 1) + x) * Lay::TILE + (row >> 5) * 4096 + lane * 8, m_run * c2, l_run);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Lay::LF + 2 * x + (jobs & 1)]);
      ++jobs;
    }
  }

  __syncwarp();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0 && args.err != nullptr) atomicCAS(args.err, 0, 1);
  if (warp == 14) {
    __syncwarp();
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
