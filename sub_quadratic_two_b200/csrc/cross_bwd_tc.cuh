// cross_bwd_tc.cuh - backward of cross attention on the sm_100a tensor cores (bf16).
//
// With P = exp(s S - lse), dP = dO V^T, D = rowsum(dO o O), dS = P o (dP - D):
//   dQ = s dS K,   dK = s dS^T Q,   dV = P^T dO.
// Two kernels, each with its accumulators in TMEM and nothing added across CTAs by atomics
// (so the results repeat bitwise): one holds a query tile and walks the keys (dQ), one holds a
// key tile and walks the queries of its head group (dK, dV). S and dP are computed in both:
// 7 products of 2 n m d flops in place of the 5 of a single kernel, whose dQ parts (one fp32
// [n, d] per 128 keys) would have to be added in memory: at m = 512 four times the bytes of dQ
// in fp32 through L2, more than the two products cost. (With one key block there would be no parts: not
// tried as a kernel of its own.)
//
// Measured at 27,280 x 512, 24 heads of 128, under ncu: dQ 250 us, dK and dV 268 us and 15 to join their
// parts (tensor pipe 54% and 68% busy; replayed back to back 530 in all); together 1,130 TFLOP/s of
// the seven products, 800 of the five.
//
// Rounding: P and dS to bf16 before the products that read them (the tensor core's operand
// type); D, the statistics and the accumulators in fp32; each gradient once at the end.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "cross_tc.cuh"

namespace sq {

constexpr int kCrossBwdThreads = 512;

struct alignas(64) CrossBwdMaps {
  CUtensorMap q, k, v, dout;
};

struct CrossBwdArgs {
  int B, heads, kv_heads, group, n, m;
  int qtiles, kblocks;
  int splits;             // dk, dv kernel: parts of a key tile's queries
  int dq_splits;          // dq kernel: parts of a query tile's keys
  int items;              // dq kernel: (query tile, part) in all; dk, dv kernel: (key tile, part) units
  FastDiv f_dq, f_dq_splits;  // dq items of a (batch, head), of a query tile
  FastDiv f_qtiles, f_heads, f_group, f_kblocks, f_kv_heads;
  int q_b, q_h, k_b, k_h, v_b, v_h, do_b, do_h;  // 1, or 0 where the map has no such extent
  CrossMask mask;
  float scale, scale_log2;
  const __nv_bfloat16 *o, *dout;  // for D
  CrossStride so, sdo, sdq, sdk, sdv;
  const float* lse;       // [B, heads, n]
  float* Drow;            // [B, heads, n]: written by the dq kernel, read by the other
  __nv_bfloat16 *dq, *dk, *dv;
  float* dq_part;         // dq_splits > 1: [part][B, heads, n][D] fp32
  float* part;            // splits > 1: [dk, dv][split][B, kv_heads, kblocks * 128][D] fp32
  int* err;
  uint64_t timeout_ns;
};

// ==================================================================== dQ
//
// Roles (512 threads):
//   warps 0-3, 4-7  key columns 0-63 and 64-127 of each block (thread = query row = TMEM lane)
//   warps 8-11      D of the next tile (from dO and O in memory), then dQ of this one: TMEM -> bf16
//                   rows, 64 bytes of a row per thread and step (there is no room to stage them)
//   warp 12         key tiles and Q;  warp 15: value tiles and dO;  warp 13: tcgen05.mma
//   warp 14         masks: which keys of a block count, for warps 0-7, and zeroes in the masked rows of
//                   key and value tiles
// Where all keys that may count lie in one block, D = sum_j P dP is summed by warps 0-7 instead: it
// costs no read of O, and it is free of O's rounding, which few keys do not average out.
// TMEM: S of block t at [128 (t & 1), ...), dP at [256, 384), dQ at [384, 384 + D). dS replaces
// S in place (packed bf16, each half inside its own columns).
// Per block the tensor core runs S(t+1), dP(t+1), dQ(t); the exponentials of block t+1 run
// while dP(t+1) and dQ(t) do.

template <int D>
struct CrossDqLayout {
  static constexpr int TILE = 128 * D * 2;
  // A key tile stays from S(t) to dQ(t): with two, S(t + 1) waits for dQ(t - 1) and a load.
  static constexpr int NK = D == 128 ? 3 : 4, NV = D == 128 ? 2 : 4;
  static constexpr int Q_OFF = 0;
  static constexpr int DO_OFF = TILE;
  static constexpr int K_OFF = DO_OFF + TILE;
  static constexpr int V_OFF = K_OFF + NK * TILE;
  static constexpr int D_OFF = V_OFF + NV * TILE;  // half sums of D, two tiles in turn
  static constexpr int NW = 8;                     // blocks whose masks are kept
  static constexpr int WORD_OFF = D_OFF + 4 * 128 * 4;
  static constexpr int BAR_OFF = WORD_OFF + NW * 16;
  static constexpr int QF = 0, QE = 1, DOF = 2, DOE = 3, KF = 4, KE = KF + NK, KR = KE + NK, VF = KR + NK, VE = VF + NV,
                       VR = VE + NV, SF = VR + NV, DPF = SF + 2, DSF = DPF + 1, OF = DSF + 1, OE = OF + 1, DF = OE + 1,
                       DE = DF + 2, XD = DE + 2, WF = XD + 4, DRAIN = WF + NW, NBAR = DRAIN + 1;
  static constexpr int BYTES = BAR_OFF + NBAR * 8 + 16;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

template <int D, bool MASKED>
__global__ void __launch_bounds__(kCrossBwdThreads, 1)
    cross_bwd_dq_kernel(const __grid_constant__ CrossBwdMaps maps, const __grid_constant__ CrossBwdArgs args) {
  using Lay = CrossDqLayout<D>;
  constexpr int DH = D / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::BAR_OFF + Lay::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::BAR_OFF + Lay::NBAR * 8 + 4);
  float* half_sum = reinterpret_cast<float*>(smem + Lay::D_OFF);  // [parity][half][row]
  const int warp = int(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint64_t to = args.timeout_ns;
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicCAS(args.err, 0, 1);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::NBAR; ++i) {
      const int warps = i == Lay::DSF || (i >= Lay::DE && i < Lay::DE + 2) ? 8
                        : i == Lay::OE || (i >= Lay::DF && i < Lay::DF + 2) ? 4 : i >= Lay::XD && i < Lay::XD + 4 ? 2 : 1;
      mbar_init(&bars[i], warps);
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
    prefetch_tmap(&maps.dout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t sbase = smem_u32(smem);

  struct Item {
    int b, h, hk, qt, sp;
  };
  auto item_of = [&](int i) -> Item {
    const int bh = fdiv(i, args.f_dq), b = fdiv(bh, args.f_heads), h = bh - b * args.heads;
    const int r = i - bh * args.qtiles * args.dq_splits, qt = fdiv(r, args.f_dq_splits);
    return Item{b, h, fdiv(h, args.f_group), qt, r - qt * args.dq_splits};
  };
  int len_b = -1, len_v = 0;
  auto len_of = [&](int b) -> int {
    if (!MASKED) return args.m;
    if (b != len_b) {
      len_v = cross_len(args.mask, b, args.m);
      len_b = b;
    }
    return len_v;
  };
  // key blocks of an item of batch row b, one at least; a part short of keys runs blocks past the
  // length (all masked), as an item does where no key counts
  auto blocks_of = [&](int b) -> int {
    const int nb = (len_of(b) + 127) >> 7, per = args.dq_splits > 1 ? (nb + args.dq_splits - 1) / args.dq_splits : nb;
    return per > 1 ? per : 1;
  };
  // whether D is summed with dS: the item's one block holds every key
  auto exact_d = [&](int b) -> bool { return args.dq_splits == 1 && blocks_of(b) == 1; };
  auto load = [&](uint32_t dst, const CUtensorMap* m, uint64_t* bar, int row, int h, int b) {
    mbar_arrive_expect_tx(bar, Lay::TILE);
#pragma unroll
    for (int c = 0; c < DH; ++c) tma_load_4d(dst + c * kCrossBlk, m, bar, c * 64, row, h, b);
  };
  // lets the loads issued into a ring land before the CTA may exit
  auto drain_ring = [&](int full, uint32_t slots, uint32_t issued) {
    for (uint32_t s = 0; s < slots; ++s) {
      const uint32_t uses = issued > s ? (issued - s + slots - 1) / slots : 0;
      if (uses) mbar_wait_drain(&bars[full + s], (uses - 1) & 1, to);
    }
  };

  if (warp == 12) {
    if (lane == 0) {  // ---------------------------------------------- key tiles and Q
      uint32_t e = 0, q = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
        const Item it = item_of(i);
        const int nk = blocks_of(it.b);
        // the next tile's Q and dO into L2: their loads come late, behind this tile's last products
        if (i + int(gridDim.x) < args.items) {
          const Item nx = item_of(i + int(gridDim.x));
#pragma unroll
          for (int c = 0; c < DH; ++c) {
            tma_prefetch_4d(&maps.q, c * 64, nx.qt * 128, nx.h * args.q_h, nx.b * args.q_b);
            tma_prefetch_4d(&maps.dout, c * 64, nx.qt * 128, nx.h * args.do_h, nx.b * args.do_b);
          }
        }
        for (int k = 0; ok && k < nk; ++k) {
          const uint32_t s = e % Lay::NK;
          if (!(ok = cross_wait(&bars[Lay::KE + s], ((e / Lay::NK) & 1) ^ 1, abort_flag, to))) break;
          load(sbase + Lay::K_OFF + s * Lay::TILE, &maps.k, &bars[Lay::KF + s], (it.sp * nk + k) * 128, it.hk * args.k_h, it.b * args.k_b);
          ++e;
          if (k == 0) {
            if (!(ok = cross_wait(&bars[Lay::QE], (q & 1) ^ 1, abort_flag, to))) break;
            load(sbase + Lay::Q_OFF, &maps.q, &bars[Lay::QF], it.qt * 128, it.h * args.q_h, it.b * args.q_b);
            ++q;
          }
        }
      }
      drain_ring(Lay::KF, Lay::NK, e);
      drain_ring(Lay::QF, 1, q);
    }
  } else if (warp == 15) {
    if (lane == 0) {  // ---------------------------------------------- value tiles and dO
      uint32_t e = 0, q = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
        const Item it = item_of(i);
        const int nk = blocks_of(it.b);
        for (int k = 0; ok && k < nk; ++k) {
          const uint32_t s = e % Lay::NV;
          if (!(ok = cross_wait(&bars[Lay::VE + s], ((e / Lay::NV) & 1) ^ 1, abort_flag, to))) break;
          load(sbase + Lay::V_OFF + s * Lay::TILE, &maps.v, &bars[Lay::VF + s], (it.sp * nk + k) * 128, it.hk * args.v_h, it.b * args.v_b);
          ++e;
          if (k == 0) {
            if (!(ok = cross_wait(&bars[Lay::DOE], (q & 1) ^ 1, abort_flag, to))) break;
            load(sbase + Lay::DO_OFF, &maps.dout, &bars[Lay::DOF], it.qt * 128, it.h * args.do_h, it.b * args.do_b);
            ++q;
          }
        }
      }
      drain_ring(Lay::VF, Lay::NV, e);
      drain_ring(Lay::DOF, 1, q);
    }
  } else if (warp == 14) {
    if (MASKED) {  // ------------------------------------------------- masks
      uint32_t t = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
        const Item it = item_of(i);
        const int len = len_of(it.b), nk = blocks_of(it.b);
        for (int k = 0; k < nk; ++k, ++t) {
          uint32_t w[4];
          const int key = (it.sp * nk + k) * 128;
          block_words(len - key, args.mask.keys == nullptr ? nullptr : args.mask.keys + it.b * args.mask.stride + key,
                      lane, w);
          const uint32_t sk = t % Lay::NK, sv = t % Lay::NV;
          if (!(ok = cross_warp_wait(&bars[Lay::KF + sk], (t / Lay::NK) & 1, abort_flag, to))) break;
          zero_rows<D>(sbase + Lay::K_OFF + sk * Lay::TILE, w, lane);
          __syncwarp();
          // the block's place is free: K(t) came behind dQ(t - NK), whose dS is written (NK < NW)
          if (lane == 0) {
            if (args.mask.keys != nullptr) {
              st_shared_v4(sbase + Lay::WORD_OFF + (t % Lay::NW) * 16, w[0], w[1], w[2], w[3]);
              mbar_arrive(&bars[Lay::WF + t % Lay::NW]);
            }
            mbar_arrive(&bars[Lay::KR + sk]);
          }
          if (!(ok = cross_warp_wait(&bars[Lay::VF + sv], (t / Lay::NV) & 1, abort_flag, to))) break;
          zero_rows<D>(sbase + Lay::V_OFF + sv * Lay::TILE, w, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::VR + sv]);
        }
      }
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);  // S, dP: both operands K-major
    constexpr uint32_t id_q = idesc_bf16_f32(128, D, 0, 1);    // dQ: A (dS) from TMEM, B (K) MN-major
    constexpr int KREADY = MASKED ? Lay::KR : Lay::KF, VREADY = MASKED ? Lay::VR : Lay::VF;
    const uint32_t el = elect_one(), tm = uniform(tmem);
    const uint64_t q0 = sdesc_sw128(sbase + Lay::Q_OFF, 16, 1024), o0 = sdesc_sw128(sbase + Lay::DO_OFF, 16, 1024),
                   k0 = sdesc_sw128(sbase + Lay::K_OFF, 16, 1024), v0 = sdesc_sw128(sbase + Lay::V_OFF, 16, 1024),
                   kt0 = sdesc_sw128(sbase + Lay::K_OFF, kCrossBlk, 1024);
    auto wait = [&](int bar, uint32_t parity) -> bool {
      return cross_warp_wait(&bars[bar], parity, abort_flag, to);
    };
    // dQ(t) += dS(t) K; the tile's first block overwrites what the epilogue has drained
    auto dq = [&](uint32_t t, uint32_t job, bool first, bool last) -> bool {
      if (first && job > 0 && !wait(Lay::OE, (job - 1) & 1)) return false;
      tc_fence_after();
      const uint32_t s = t % Lay::NK, a = tm + 128 * (t & 1);
      const uint64_t ka = kt0 + s * (Lay::TILE >> 4);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts_by(el, tm + 384, a + (kk >> 2) * 64 + (kk & 3) * 8, ka + kk * (2048 >> 4), id_q,
                  kk == 0 ? (first ? 0u : 1u) : 1u);
      tc_commit_by(el, &bars[Lay::KE + s]);
      if (last) tc_commit_by(el, &bars[Lay::OF]);
      return true;
    };
    uint32_t t = 0, job = 0;
    bool ok = true, prev = false, prev_first = false, prev_last = false;
#pragma unroll 1
    for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x, ++job) {
      const Item it = item_of(i);
      const int nk = int(uniform(uint32_t(blocks_of(it.b))));
#pragma unroll 1
      for (int k = 0; k < nk; ++k, ++t) {
        const bool first = k == 0, last = k == nk - 1;
        const uint32_t sk = t % Lay::NK, sv = t % Lay::NV;
        // S(t) into the columns that dQ(t - 2) read dS from (issued before, so behind it)
        if (!(ok = wait(KREADY + sk, (t / Lay::NK) & 1))) break;
        if (first && !(ok = wait(Lay::QF, job & 1))) break;
        tc_fence_after();
        const uint64_t ka = k0 + sk * (Lay::TILE >> 4), va = v0 + sv * (Lay::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kCrossBlk + (kk & 3) * 32) >> 4;
          mma_ss_by(el, tm + 128 * (t & 1), q0 + off, ka + off, id_s, kk > 0 ? 1u : 0u);
        }
        tc_commit_by(el, &bars[Lay::SF + (t & 1)]);
        if (last) tc_commit_by(el, &bars[Lay::QE]);
        // dS(t - 1) is written, so dP(t - 1) has been read. At a new tile dO has yet to arrive: dQ
        // of the last block goes first. Else the value tile is waited for ahead of dS.
        if (!first && !(ok = wait(VREADY + sv, (t / Lay::NV) & 1))) break;
        if (prev && !(ok = wait(Lay::DSF, (t - 1) & 1))) break;
        if (first) {
          if (prev && !(ok = dq(t - 1, job - 1, prev_first, prev_last))) break;
          if (!(ok = wait(VREADY + sv, (t / Lay::NV) & 1))) break;
          if (!(ok = wait(Lay::DOF, job & 1))) break;
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kCrossBlk + (kk & 3) * 32) >> 4;
          mma_ss_by(el, tm + 256, o0 + off, va + off, id_s, kk > 0 ? 1u : 0u);
        }
        tc_commit_by(el, &bars[Lay::DPF]);
        tc_commit_by(el, &bars[Lay::VE + sv]);
        if (last) tc_commit_by(el, &bars[Lay::DOE]);
        if (!first && !(ok = dq(t - 1, job, prev_first, prev_last))) break;
        prev = true;
        prev_first = first;
        prev_last = last;
      }
    }
    if (ok && prev && wait(Lay::DSF, (t - 1) & 1)) dq(t - 1, job - 1, prev_first, prev_last);
    tc_commit_by(el, &bars[Lay::DRAIN]);
    mbar_wait_drain(&bars[Lay::DRAIN], 0, to);
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ D, dQ
    const int ew = warp & 3, row = threadIdx.x & 127;
    constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes per row, rows per load
    bool ok = true;
    uint32_t made = 0;  // tiles whose D is made
    auto make_d = [&](int i) -> bool {
      const Item it = item_of(i);
      const uint32_t par = made & 1;
      if (!cross_warp_wait(&bars[Lay::DE + par], ((made >> 1) & 1) ^ 1, abort_flag, to)) return false;
      const long long base = ((long long)it.b * args.heads + it.h) * args.n;
      const int r0 = it.qt * 128 + ew * 32 + lane / LPR, c = (lane % LPR) * 8;
#pragma unroll 1
      for (int g = 0; g < 32 / RPI; g += 8) {
        uint4 xa[8], xb[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int tok = r0 + (g + u) * RPI;
          xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
          if (tok < args.n) {
            xa[u] = __ldg(reinterpret_cast<const uint4*>(args.o + it.b * args.so.b + it.h * args.so.h + tok * args.so.n + c));
            xb[u] = __ldg(
                reinterpret_cast<const uint4*>(args.dout + it.b * args.sdo.b + it.h * args.sdo.h + tok * args.sdo.n + c));
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t a[4] = {xa[u].x, xa[u].y, xa[u].z, xa[u].w}, b[4] = {xb[u].x, xb[u].y, xb[u].z, xb[u].w};
          float acc = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), acc);
            acc = fmaf(__uint_as_float(a[e] & 0xffff0000u), __uint_as_float(b[e] & 0xffff0000u), acc);
          }
#pragma unroll
          for (int z = LPR / 2; z > 0; z >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, z);
          const int tok = r0 + (g + u) * RPI;
          if (lane % LPR == 0 && tok < args.n) args.Drow[base + tok] = acc;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Lay::DF + par]);
      ++made;
      return true;
    };
    // D of the tiles whose keys span several blocks (the others' comes with their dS; every part of a
    // tile makes the same D)
    auto make_d_if = [&](int i) -> bool {
      return i >= args.items || exact_d(item_of(i).b) || make_d(i);
    };
    ok = make_d_if(blockIdx.x);
    uint32_t job = 0;
    for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x, ++job) {
      if (!(ok = make_d_if(i + int(gridDim.x)))) break;
      const Item it = item_of(i);
      const int tok = it.qt * 128 + row;
      // a query without keys gets zeros, whatever its dO holds (0 times an infinite dP - D is NaN)
      const float sc = MASKED && tok < args.n &&
                               __ldg(args.lse + ((long long)it.b * args.heads + it.h) * args.n + tok) == -INFINITY
                           ? 0.f
                           : args.scale;
      if (!(ok = cross_warp_wait(&bars[Lay::OF], job & 1, abort_flag, to))) break;
      tc_fence_after();
      const uint32_t t = tmem + (uint32_t(ew * 32) << 16) + 384;
      __nv_bfloat16* out = args.dq + it.b * args.sdq.b + it.h * args.sdq.h + (long long)tok * args.sdq.n;
      float* part = args.dq_part +
                    (((long long)it.sp * args.B * args.heads + (long long)it.b * args.heads + it.h) * args.n + tok) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        __syncwarp();  // lanes part below: TMEM is read by whole warps
        tmem_ld32(t + c, v);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          v[e] = MASKED && sc == 0.f ? 0u : __float_as_uint(__uint_as_float(v[e]) * sc);
        if (args.dq_splits > 1) {
          if (tok < args.n) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + c + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        } else if (tok < args.n) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = pack_bf16x2(__uint_as_float(v[8 * j + 2 * e]), __uint_as_float(v[8 * j + 2 * e + 1]));
            *reinterpret_cast<uint4*>(out + c + 8 * j) = make_uint4(p[0], p[1], p[2], p[3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Lay::OE]);
    }
  } else {
    // ------------------------------------------------------------------ P, dS
    const int g = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const float c2 = args.scale_log2;
    const uint64_t c2x2 = f2(c2, c2);
    uint32_t t = 0, made = 0, summed = 0;  // blocks; tiles with D from the epilogue, and summed here
    bool ok = true;
    for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
      const Item it = item_of(i);
      const int len = len_of(it.b), nk = blocks_of(it.b), tok = it.qt * 128 + row;
      const bool exact = exact_d(it.b);
      const bool idle = it.qt * 128 + (warp & 3) * 32 >= args.n;
      // rows past the last query and rows without keys: P = 2^(s - inf) = 0
      float lse2 = INFINITY;
      if (tok < args.n) {
        const float l = __ldg(args.lse + ((long long)it.b * args.heads + it.h) * args.n + tok);
        lse2 = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
      }
      const uint64_t neg2 = f2(-lse2, -lse2);
      float Dv = 0.f;
      for (int k = 0; k < nk; ++k, ++t) {
        const uint32_t tS = tmem + lanes + 128 * (t & 1) + 64 * g, tP = tmem + lanes + 256 + 64 * g;
        if (!(ok = cross_warp_wait(&bars[Lay::SF + (t & 1)], (t >> 1) & 1, abort_flag, to))) break;
        tc_fence_after();
        // which of this half's keys count
        uint32_t wa, wb;
        if (MASKED && args.mask.keys != nullptr) {
          if (!(ok = cross_warp_wait(&bars[Lay::WF + t % Lay::NW], (t / Lay::NW) & 1, abort_flag, to))) break;
          const uint4 w = ld_shared_v4(sbase + Lay::WORD_OFF + (t % Lay::NW) * 16);
          wa = g ? w.z : w.x;
          wb = g ? w.w : w.y;
        } else {
          uint32_t w[4];
          block_words(len - (it.sp * nk + k) * 128, nullptr, lane, w);
          wa = g ? w[2] : w[0];
          wb = g ? w[3] : w[1];
        }
        float p[64];
        if (!idle) {
          uint32_t v[64];
          tmem_ld64(tS, v);
          if ((wa & wb) != ~0u) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (!(((e < 32 ? wa : wb) >> (e & 31)) & 1u)) v[e] = 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            const uint64_t z = ffma2(f2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2x2, neg2);
            p[e] = ex2_approx(f2_lo(z));
            p[e + 1] = ex2_approx(f2_hi(z));
          }
        }
        if (k == 0 && !exact) {
          if (!(ok = cross_warp_wait(&bars[Lay::DF + (made & 1)], (made >> 1) & 1, abort_flag, to))) break;
          // written by this CTA's epilogue warps, ordered by the barrier (so not read as constant data)
          if (tok < args.n) Dv = *static_cast<volatile float*>(args.Drow + ((long long)it.b * args.heads + it.h) * args.n + tok);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::DE + (made & 1)]);
          ++made;
        }
        if (!(ok = cross_warp_wait(&bars[Lay::DPF], t & 1, abort_flag, to))) break;
        tc_fence_after();
        if (exact && !idle) {
          // D of the row: each half's sum of P dP, exchanged with the warp of the other half
          uint64_t acc = 0ull;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t u[16];
            tmem_ld16_async(tP + 16 * c, u);
            tmem_ld_wait(u);
#pragma unroll
            for (int e = 0; e < 16; e += 2)
              acc = ffma2(f2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])), f2(p[16 * c + e], p[16 * c + e + 1]), acc);
          }
          float* hs = half_sum + (summed & 1) * 256;
          Dv = f2_lo(acc) + f2_hi(acc);
          hs[g * 128 + row] = Dv;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::XD + (warp & 3)]);
          if (!(ok = cross_warp_wait(&bars[Lay::XD + (warp & 3)], summed & 1, abort_flag, to))) break;
          // the same sum on both sides
          const float other = hs[(g ^ 1) * 128 + row];
          Dv = g ? other + Dv : Dv + other;
          if (g == 0 && tok < args.n) args.Drow[((long long)it.b * args.heads + it.h) * args.n + tok] = Dv;
          ++summed;
        }
        if (!idle) {
          const uint64_t nd = f2(-Dv, -Dv);
          uint32_t v[2][16];
          tmem_ld16_async(tP, v[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t(&u)[16] = v[c & 1];
            tmem_ld_wait(u);
            if (c < 3) tmem_ld16_async(tP + 16 * (c + 1), v[(c + 1) & 1]);
            uint32_t d[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const uint64_t z = mul2(fadd2(f2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])), nd),
                                      f2(p[16 * c + e], p[16 * c + e + 1]));
              d[e >> 1] = pack_bf16x2(f2_lo(z), f2_hi(z));
            }
            tmem_st8(tS + 8 * c, d);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Lay::DSF]);
      }
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

// ==================================================================== dK, dV
//
// A unit is a key tile (128 keys of a key head) and a part of the queries of its head group.
// Roles (512 threads):
//   warps 0-3, 4-7  query columns 0-63 and 64-127 of each tile (thread = key row = TMEM lane)
//   warps 8-11      dK and dV of a finished unit: TMEM -> bf16 rows, or fp32 parts
//   warp 12         key and value tiles, query tiles;  warp 15: dO;  warp 13: tcgen05.mma
//   warp 14         -lse log2 e and -D of each query tile into shared memory
// TMEM: S^T [0,128), dP^T [128,256), dV [256, 256 + D), dK [384, 384 + D). P^T and dS^T replace
// S^T and dP^T in place (packed bf16, each half inside its own columns).
// Per query tile the tensor core runs dV(t), S(t+1) once P(t) is there, then dK(t), dP(t+1)
// once dS(t) is there: four products in turn, with the softmax of one under the products of
// the other.

template <int D>
struct CrossDkvLayout {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int NQ = D == 128 ? 3 : 4, NDO = D == 128 ? 2 : 4;
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = TILE;
  static constexpr int Q_OFF = 2 * TILE;
  static constexpr int DO_OFF = Q_OFF + NQ * TILE;
  static constexpr int VEC_OFF = DO_OFF + NDO * TILE;  // two tiles of (-lse, -D)
  static constexpr int BAR_OFF = VEC_OFF + 2 * 256 * 4;
  static constexpr int KF = 0, KE = 1, VF = 2, VE = 3, QF = 4, QE = QF + NQ, DOF = QE + NQ, DOE = DOF + NDO,
                       SF = DOE + NDO, PF = SF + 1, DPF = PF + 1, DSF = DPF + 1, ACCF = DSF + 1, ACCE = ACCF + 1,
                       VECF = ACCE + 1, VECE = VECF + 2, DRAIN = VECE + 2, NBAR = DRAIN + 1;
  static constexpr int BYTES = BAR_OFF + NBAR * 8 + 16;
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

template <int D, bool MASKED>
__global__ void __launch_bounds__(kCrossBwdThreads, 1)
    cross_bwd_dkdv_kernel(const __grid_constant__ CrossBwdMaps maps, const __grid_constant__ CrossBwdArgs args) {
  using Lay = CrossDkvLayout<D>;
  constexpr int DH = D / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::BAR_OFF + Lay::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::BAR_OFF + Lay::NBAR * 8 + 4);
  const int warp = int(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint64_t to = args.timeout_ns;
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicCAS(args.err, 0, 1);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::NBAR; ++i) {
      const int warps = i == Lay::PF || i == Lay::DSF || (i >= Lay::VECE && i < Lay::VECE + 2) ? 8 : i == Lay::ACCE ? 4 : 1;
      mbar_init(&bars[i], warps);
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
    prefetch_tmap(&maps.dout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t sbase = smem_u32(smem);

  struct Unit {
    int b, hk, kb, sp;
    int t0, t1;   // query tiles of the head group (head-major) in this unit
    int limit;    // keys of the tile below it may count
  };
  int len_b = -1, len_v = 0;
  // splits are the slowest index: the key tiles that share query tiles run side by side
  auto unit_of = [&](int i) -> Unit {
    Unit u;
    const int per = args.B * args.kv_heads * args.kblocks;
    u.sp = i / per;
    const int j = i - u.sp * per;
    const int bh = fdiv(j, args.f_kblocks);
    u.kb = j - bh * args.kblocks;
    u.b = fdiv(bh, args.f_kv_heads);
    u.hk = bh - u.b * args.kv_heads;
    if (MASKED && u.b != len_b) {
      len_v = cross_len(args.mask, u.b, args.m);
      len_b = u.b;
    }
    u.limit = (MASKED ? len_v : args.m) - u.kb * 128;
    const int tiles = args.group * args.qtiles, part = (tiles + args.splits - 1) / args.splits;
    u.t0 = u.sp * part;
    u.t1 = u.t0 + part < tiles ? u.t0 + part : tiles;
    if (u.t0 > tiles) u.t0 = tiles;
    if (u.limit <= 0) u.t1 = u.t0;  // no key of the tile counts: nothing to add up
    return u;
  };
  auto load = [&](uint32_t dst, const CUtensorMap* m, uint64_t* bar, int row, int h, int b) {
    mbar_arrive_expect_tx(bar, Lay::TILE);
#pragma unroll
    for (int c = 0; c < DH; ++c) tma_load_4d(dst + c * kCrossBlk, m, bar, c * 64, row, h, b);
  };
  auto drain_ring = [&](int full, uint32_t slots, uint32_t issued) {
    for (uint32_t s = 0; s < slots; ++s) {
      const uint32_t uses = issued > s ? (issued - s + slots - 1) / slots : 0;
      if (uses) mbar_wait_drain(&bars[full + s], (uses - 1) & 1, to);
    }
  };

  if (warp == 12) {
    if (lane == 0) {  // ---------------------------------------------- key, value and query tiles
      uint32_t e = 0, units = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
        const Unit u = unit_of(i);
        if (u.t0 >= u.t1) continue;
        for (int t = u.t0; ok && t < u.t1; ++t) {
          if (t == u.t0) {
            if (!(ok = cross_wait(&bars[Lay::KE], (units & 1) ^ 1, abort_flag, to))) break;
            load(sbase + Lay::K_OFF, &maps.k, &bars[Lay::KF], u.kb * 128, u.hk * args.k_h, u.b * args.k_b);
          }
          const int g = fdiv(t, args.f_qtiles), h = u.hk * args.group + g;
          const uint32_t s = e % Lay::NQ;
          if (!(ok = cross_wait(&bars[Lay::QE + s], ((e / Lay::NQ) & 1) ^ 1, abort_flag, to))) break;
          load(sbase + Lay::Q_OFF + s * Lay::TILE, &maps.q, &bars[Lay::QF + s], (t - g * args.qtiles) * 128,
               h * args.q_h, u.b * args.q_b);
          ++e;
        }
        ++units;
      }
      drain_ring(Lay::KF, 1, units);
      drain_ring(Lay::QF, Lay::NQ, e);
    }
  } else if (warp == 15) {
    if (lane == 0) {  // ---------------------------------------------- value and dO tiles
      uint32_t e = 0, units = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
        const Unit u = unit_of(i);
        if (u.t0 >= u.t1) continue;
        for (int t = u.t0; ok && t < u.t1; ++t) {
          if (t == u.t0) {
            if (!(ok = cross_wait(&bars[Lay::VE], (units & 1) ^ 1, abort_flag, to))) break;
            load(sbase + Lay::V_OFF, &maps.v, &bars[Lay::VF], u.kb * 128, u.hk * args.v_h, u.b * args.v_b);
          }
          const int g = fdiv(t, args.f_qtiles), h = u.hk * args.group + g;
          const uint32_t s = e % Lay::NDO;
          if (!(ok = cross_wait(&bars[Lay::DOE + s], ((e / Lay::NDO) & 1) ^ 1, abort_flag, to))) break;
          load(sbase + Lay::DO_OFF + s * Lay::TILE, &maps.dout, &bars[Lay::DOF + s], (t - g * args.qtiles) * 128,
               h * args.do_h, u.b * args.do_b);
          ++e;
        }
        ++units;
      }
      drain_ring(Lay::VF, 1, units);
      drain_ring(Lay::DOF, Lay::NDO, e);
    }
  } else if (warp == 14) {
    // ------------------------------------------------------------------ statistics of the query tiles
    uint32_t t_all = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
      const Unit u = unit_of(i);
      for (int t = u.t0; t < u.t1; ++t, ++t_all) {
        const int g = fdiv(t, args.f_qtiles), h = u.hk * args.group + g, tok = (t - g * args.qtiles) * 128 + lane * 4;
        const long long base = ((long long)u.b * args.heads + h) * args.n + tok;
        float l[4], d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // queries past the last and queries without keys: P = 2^(s - inf) = 0
          l[e] = -INFINITY;
          d[e] = 0.f;
          if (tok + e < args.n) {
            const float x = __ldg(args.lse + base + e);
            l[e] = x == -INFINITY ? -INFINITY : -x * 1.4426950408889634f;
            d[e] = -__ldg(args.Drow + base + e);
          }
        }
        const uint32_t s = t_all & 1;
        if (!(ok = cross_warp_wait(&bars[Lay::VECE + s], ((t_all >> 1) & 1) ^ 1, abort_flag, to))) break;
        float* vec = reinterpret_cast<float*>(smem + Lay::VEC_OFF) + s * 256;
        *reinterpret_cast<float4*>(vec + lane * 4) = make_float4(l[0], l[1], l[2], l[3]);
        *reinterpret_cast<float4*>(vec + 128 + lane * 4) = make_float4(d[0], d[1], d[2], d[3]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Lay::VECF + s]);
      }
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);
    constexpr uint32_t id_acc = idesc_bf16_f32(128, D, 0, 1);
    const uint32_t el = elect_one(), tm = uniform(tmem);
    const uint64_t ka = sdesc_sw128(sbase + Lay::K_OFF, 16, 1024), va = sdesc_sw128(sbase + Lay::V_OFF, 16, 1024),
                   q0 = sdesc_sw128(sbase + Lay::Q_OFF, 16, 1024), o0 = sdesc_sw128(sbase + Lay::DO_OFF, 16, 1024),
                   qt0 = sdesc_sw128(sbase + Lay::Q_OFF, kCrossBlk, 1024),
                   ot0 = sdesc_sw128(sbase + Lay::DO_OFF, kCrossBlk, 1024);
    auto wait = [&](int bar, uint32_t parity) -> bool {
      return cross_warp_wait(&bars[bar], parity, abort_flag, to);
    };
    // the (unit, tile) pairs in order, with one pair of look-ahead
    struct Step {
      int i, t, t0, t1;
      uint32_t unit;
      bool ok;
    };
    auto seek = [&](int i, uint32_t unit) -> Step {
#pragma unroll 1
      for (; i < args.items; i += gridDim.x) {
        const Unit u = unit_of(i);
        const int t0 = int(uniform(uint32_t(u.t0))), t1 = int(uniform(uint32_t(u.t1)));
        if (t0 < t1) return Step{i, t0, t0, t1, unit, true};
      }
      return Step{i, 0, 0, 0, unit, false};
    };
    // S(e) and dP(e), e: the tile's number over all units
    auto s_mma = [&](const Step& s, uint32_t e) -> bool {
      const uint32_t z = e % Lay::NQ;
      if (s.t == s.t0 && !wait(Lay::KF, s.unit & 1)) return false;
      if (!wait(Lay::QF + z, (e / Lay::NQ) & 1)) return false;
      tc_fence_after();
      const uint64_t qa = q0 + z * (Lay::TILE >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kCrossBlk + (kk & 3) * 32) >> 4;
        mma_ss_by(el, tm, ka + off, qa + off, id_s, kk > 0 ? 1u : 0u);
      }
      tc_commit_by(el, &bars[Lay::SF]);
      if (s.t == s.t1 - 1) tc_commit_by(el, &bars[Lay::KE]);
      return true;
    };
    auto dp_mma = [&](const Step& s, uint32_t e) -> bool {
      const uint32_t z = e % Lay::NDO;
      if (s.t == s.t0 && !wait(Lay::VF, s.unit & 1)) return false;
      if (!wait(Lay::DOF + z, (e / Lay::NDO) & 1)) return false;
      tc_fence_after();
      const uint64_t da = o0 + z * (Lay::TILE >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * kCrossBlk + (kk & 3) * 32) >> 4;
        mma_ss_by(el, tm + 128, va + off, da + off, id_s, kk > 0 ? 1u : 0u);
      }
      tc_commit_by(el, &bars[Lay::DPF]);
      if (s.t == s.t1 - 1) tc_commit_by(el, &bars[Lay::VE]);
      return true;
    };
    uint32_t e = 0;
    Step cur{}, nxt = seek(blockIdx.x, 0);
    bool ok = true;
    // e counts the tiles whose dV and dK are issued; the loop body issues those of tile `cur` (none
    // in the first turn) between S and dP of tile `nxt`
#pragma unroll 1
    while (ok && (cur.ok || nxt.ok)) {
      const bool first = cur.t == cur.t0, last = cur.t == cur.t1 - 1;
      const uint32_t n = cur.ok ? e + 1 : 0;  // number of tile `nxt`
      if (cur.ok) {  // dV += P^T dO (the unit's first overwrites what the epilogue has drained)
        if (first && cur.unit > 0 && !(ok = wait(Lay::ACCE, (cur.unit - 1) & 1))) break;
        if (!(ok = wait(Lay::PF, e & 1))) break;
        tc_fence_after();
        const uint32_t z = e % Lay::NDO;
        const uint64_t da = ot0 + z * (Lay::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_by(el, tm + 256, tm + (kk >> 2) * 64 + (kk & 3) * 8, da + kk * (2048 >> 4), id_acc,
                    kk == 0 ? (first ? 0u : 1u) : 1u);
        tc_commit_by(el, &bars[Lay::DOE + z]);
      }
      if (nxt.ok && !(ok = s_mma(nxt, n))) break;
      if (cur.ok) {  // dK += dS^T Q
        if (!(ok = wait(Lay::DSF, e & 1))) break;
        tc_fence_after();
        const uint32_t z = e % Lay::NQ;
        const uint64_t qa = qt0 + z * (Lay::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_by(el, tm + 384, tm + 128 + (kk >> 2) * 64 + (kk & 3) * 8, qa + kk * (2048 >> 4), id_acc,
                    kk == 0 ? (first ? 0u : 1u) : 1u);
        tc_commit_by(el, &bars[Lay::QE + z]);
        if (last) tc_commit_by(el, &bars[Lay::ACCF]);
      }
      if (nxt.ok && !(ok = dp_mma(nxt, n))) break;
      if (cur.ok) ++e;
      cur = nxt;
      if (cur.ok) {
        if (cur.t + 1 < cur.t1)
          nxt.t = cur.t + 1;
        else
          nxt = seek(cur.i + gridDim.x, cur.unit + 1);
      }
    }
    tc_commit_by(el, &bars[Lay::DRAIN]);
    mbar_wait_drain(&bars[Lay::DRAIN], 0, to);
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ dK, dV
    const int ew = warp & 3, row = threadIdx.x & 127;
    const size_t rows_all = size_t(args.B) * args.kv_heads * args.kblocks * 128;
    uint32_t units = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
      const Unit u = unit_of(i);
      const int key = u.kb * 128 + row;
      bool live = row < u.limit;
      if (MASKED && live && args.mask.keys != nullptr) live = __ldg(args.mask.keys + u.b * args.mask.stride + key) != 0;
      const bool any = u.t0 < u.t1;
      if (!any) live = false;
      if (any) {
        if (!(ok = cross_warp_wait(&bars[Lay::ACCF], units & 1, abort_flag, to))) break;
        tc_fence_after();
      }
      const uint32_t t = tmem + (uint32_t(ew * 32) << 16);
      const size_t prow = size_t(u.sp) * rows_all + (size_t(u.b) * args.kv_heads + u.hk) * args.kblocks * 128 + key;
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {  // 0: dK, 1: dV
        const uint32_t acc = t + (which ? 256 : 384);
        const float sc = which ? 1.f : args.scale;
        const CrossStride& st = which ? args.sdv : args.sdk;
        __nv_bfloat16* out = (which ? args.dv : args.dk) + u.b * st.b + u.hk * st.h + (long long)key * st.n;
        float* part = args.part + (which * size_t(args.splits) * rows_all + prow) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          __syncwarp();  // lanes part below: TMEM is read by whole warps
          if (any) tmem_ld32(acc + c, v);
          // keys that do not count get zeros, whatever the accumulator holds
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = live ? __float_as_uint(__uint_as_float(v[e]) * sc) : 0u;
          if (args.splits > 1) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + c + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          } else if (key < args.m) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(out + c + e) =
                  make_uint4(pack_bf16x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                             pack_bf16x2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                             pack_bf16x2(__uint_as_float(v[e + 4]), __uint_as_float(v[e + 5])),
                             pack_bf16x2(__uint_as_float(v[e + 6]), __uint_as_float(v[e + 7])));
          }
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Lay::ACCE]);
        ++units;
      }
    }
  } else {
    // ------------------------------------------------------------------ P^T, dS^T
    const int g = warp >> 2;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + 64 * g, tP = tmem + lanes + 128 + 64 * g;
    const float c2 = args.scale_log2;
    const uint64_t c2x2 = f2(c2, c2);
    uint32_t e = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
      const Unit u = unit_of(i);
      // a warp whose key rows all lie past the last has nothing to compute; rows that do not
      // count are left to the epilogue, which writes zeros for them
      const bool idle = (warp & 3) * 32 >= u.limit;
      for (int t = u.t0; t < u.t1; ++t, ++e) {
        const uint32_t s = e & 1;
        const uint32_t vec = sbase + Lay::VEC_OFF + s * 1024 + g * 256;
        if (!(ok = cross_warp_wait(&bars[Lay::VECF + s], (e >> 1) & 1, abort_flag, to))) break;
        if (!(ok = cross_warp_wait(&bars[Lay::SF], e & 1, abort_flag, to))) break;
        tc_fence_after();
        float p[64];
        if (!idle) {
          uint32_t v[2][16];
          tmem_ld16_async(tS, v[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t(&x)[16] = v[c & 1];
            tmem_ld_wait(x);
            if (c < 3) tmem_ld16_async(tS + 16 * (c + 1), v[(c + 1) & 1]);
            uint32_t pk[8];
#pragma unroll
            for (int q = 0; q < 16; q += 4) {
              const uint4 l = ld_shared_v4(vec + (16 * c + q) * 4);
              const uint64_t z0 = ffma2(f2(__uint_as_float(x[q]), __uint_as_float(x[q + 1])), c2x2,
                                        f2(__uint_as_float(l.x), __uint_as_float(l.y)));
              const uint64_t z1 = ffma2(f2(__uint_as_float(x[q + 2]), __uint_as_float(x[q + 3])), c2x2,
                                        f2(__uint_as_float(l.z), __uint_as_float(l.w)));
              float* o = p + 16 * c + q;
              o[0] = ex2_approx(f2_lo(z0));
              o[1] = ex2_approx(f2_hi(z0));
              o[2] = ex2_approx(f2_lo(z1));
              o[3] = ex2_approx(f2_hi(z1));
              pk[q >> 1] = pack_bf16x2(o[0], o[1]);
              pk[(q >> 1) + 1] = pack_bf16x2(o[2], o[3]);
            }
            tmem_st8(tS + 8 * c, pk);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Lay::PF]);
        if (!(ok = cross_warp_wait(&bars[Lay::DPF], e & 1, abort_flag, to))) break;
        tc_fence_after();
        if (!idle) {
          uint32_t v[2][16];
          tmem_ld16_async(tP, v[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t(&x)[16] = v[c & 1];
            tmem_ld_wait(x);
            if (c < 3) tmem_ld16_async(tP + 16 * (c + 1), v[(c + 1) & 1]);
            uint32_t d[8];
#pragma unroll
            for (int q = 0; q < 16; q += 4) {
              const uint4 l = ld_shared_v4(vec + 512 + (16 * c + q) * 4);
              const float* o = p + 16 * c + q;
              const uint64_t z0 = mul2(fadd2(f2(__uint_as_float(x[q]), __uint_as_float(x[q + 1])),
                                             f2(__uint_as_float(l.x), __uint_as_float(l.y))),
                                       f2(o[0], o[1]));
              const uint64_t z1 = mul2(fadd2(f2(__uint_as_float(x[q + 2]), __uint_as_float(x[q + 3])),
                                             f2(__uint_as_float(l.z), __uint_as_float(l.w))),
                                       f2(o[2], o[3]));
              d[q >> 1] = pack_bf16x2(f2_lo(z0), f2_hi(z0));
              d[(q >> 1) + 1] = pack_bf16x2(f2_lo(z1), f2_hi(z1));
            }
            tmem_st8(tP + 8 * c, d);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[Lay::DSF]);
          mbar_arrive(&bars[Lay::VECE + s]);
        }
      }
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

// dk, dv = sum of their parts in order of the splits, 4 channels per thread. Rows of the parts:
// mpad for each (b, kv head).
template <typename T>
__global__ void __launch_bounds__(256) cross_join_grads_kernel(const float* __restrict__ part, int splits,
                                                               long long part_rows, int mpad, int kv_heads, int m,
                                                               int D, long long rows, T* dk, CrossStride sdk, T* dv,
                                                               CrossStride sdv) {
  const int C = D / 4;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long r = id / C;  // (b, kv head, key) of the unpadded rows
  if (r >= rows) return;
  const int c = int(id - r * C) * 4, which = blockIdx.y;
  const long long bh = r / m;
  const int j = int(r - bh * m), b = int(bh / kv_heads), h = int(bh - (long long)b * kv_heads);
  const float* p = part + ((which * (long long)splits) * part_rows + bh * mpad + j) * D + c;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < splits; ++s) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p + s * part_rows * D));
    a.x += x.x;
    a.y += x.y;
    a.z += x.z;
    a.w += x.w;
  }
  const CrossStride& st = which ? sdv : sdk;
  T* out = (which ? dv : dk) + b * st.b + h * st.h + j * st.n + c;
  if (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  else
    *reinterpret_cast<float4*>(out) = a;
}

}  // namespace sq
