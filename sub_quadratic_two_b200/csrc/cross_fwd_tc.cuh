// cross_fwd_tc.cuh - forward of cross attention on the sm_100a tensor cores (bf16).
//
//   S = Q K^T,  P = exp(s S - max) over the keys that count,  O = P V / sum P
// with the running maximum and sum of each row in fp32. Work is cut by cross_plan.h into
// items of two jobs (a 128-query tile over a range of 128-key blocks); a CTA per SM takes
// items in turn.
//
// Roles (512 threads):
//   warps 0-3, 4-7  softmax of job 0, job 1 (thread = query row = TMEM lane)
//   warps 8-11      epilogue: O / sum -> bf16 -> one of the warp's two staging buffers (32 rows x 64
//                   channels) -> TMA store, so the softmax warps go on with the next item
//   warp 12         TMA loads of key and value tiles, K(0) V(0) K(1) V(1) ... in a ring (a ring for
//                   each job where the keys are split)
//   warp 15         TMA loads of query tiles: the next item's as soon as a job's last scores are made
//   warp 13         issues every tcgen05.mma (the whole warp runs the loop, one lane's count)
//   warp 14         masks: zeroes the masked rows of value tiles before they are used (what lies there
//                   may be NaN or infinite, and P = 0 times NaN is NaN): those past a length, or, with
//                   a mask of each key, of every tile, key tiles too, and hands the mask to the
//                   tensor core as an operand
// TMEM (512 columns): S of job x at [128x, 128x+128), O at [256 + D x, ...). P overwrites S in
// place as packed bf16.
// The order of the products is S0(0) S1(0) | PV0(0) S0(1) | PV1(0) S1(1) | ...: the jobs take
// turns, and while the tensor core works on one, the other's softmax runs. (An issuing thread
// per job let the two fall in step, products against products and softmax against softmax:
// 232 us against 196 us at 27,280 x 512.)
// A block of 128 x 128 costs the tensor core 4 x 128 x 128 x D flops (1,024 cycles at D = 128)
// and the multi-function unit 128 x 128 exponentials (1,024 cycles at 16 a cycle): both are
// near their limit at once. Measured at 27,280 x 512, 24 heads of 128: 158 us replayed back to back (1,090
// TFLOP/s of the 1,634 that a library product reaches alone), 176 to 187 a call with the L2 flushed;
// tensor pipe 52% and multi-function unit 56% busy. What
// is left is the chain of one block, wait for S, maximum, exponentials, hand P over, which two
// jobs an SM cover only in part; a third does not fit TMEM (S and O of a job take 256 columns).
// A mask of each key is one more product, 0 or -inf times a column of ones on top of S: selects in
// the softmax warps, 128 a row, took 88 us in place of 80 at 4,093 x 1,111, 32 heads of 64.
// Rounding: P to bf16 before P V (the tensor core's operand type); sums and statistics in
// fp32; O once at the end. Every wait is bounded (see sm100.cuh).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>
#include "cross_plan.h"
#include "cross_tc.cuh"

namespace sq {

constexpr int kCrossThreads = 512;
constexpr int kCrossWords = 8;  // blocks whose masks are kept
constexpr int kCrossBias = 4096;  // bytes of a 128 x 16 bf16 operand: 2,048 of columns 0 to 7, then 8 to 15
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

template <int D, int MASK>
struct CrossFwdLayout {
  static constexpr int TILE = 128 * D * 2;
  // Query tile of each job, two staging buffers of 64 channels, the ring of key and value tiles.
  // Four ring tiles at d = 128: with three, a key tile waits for the values of two blocks before
  // (the issuer waited 0.4k cycles a block for it).
  // With a mask of each key the room of one staging buffer (d = 128) or two ring tiles (d = 64) goes
  // to the masks as operands: kCrossBias bytes for the ones and for every other ring slot.
  static constexpr bool BIAS = MASK == 2;
  static constexpr int STAGES = D == 128 && BIAS ? 1 : 2;
  static constexpr int NKV = D == 128 ? 4 : BIAS ? 8 : 10;
  static constexpr int STAGE_OFF = 2 * TILE;
  static constexpr int BIAS_OFF = STAGE_OFF + STAGES * int(kCrossBlk);
  static constexpr int KV_OFF = BIAS_OFF + (BIAS ? (1 + NKV / 2) * kCrossBias : 0);
  // Split keys: each job takes half of the ring as its own. (With one ring for both, the reader of
  // a tile would not see the phases of the tiles that the other job reads, and a wait by parity
  // needs every phase.)
  static constexpr int NS = NKV / 2;
  static constexpr int STAT_OFF = KV_OFF + NKV * TILE;   // (maximum, sum) of each job's rows
  static constexpr int WORD_OFF = STAT_OFF + 2 * 128 * 8;  // masks of eight blocks of each ring
  static constexpr int BAR_OFF = WORD_OFF + 2 * kCrossWords * 16;
  static constexpr int QF = 0, QE = QF + 2, KVF = QE + 2, KVE = KVF + NKV, RDY = KVE + NKV, SF = RDY + NKV, PF = SF + 2,
                       OF = PF + 2, OE = OF + 2, LF = OE + 2, LE = LF + 2, WF = LE + 2, DRAIN = WF + 2 * kCrossWords,
                       NBAR = DRAIN + 1;
  static constexpr int BYTES = BAR_OFF + NBAR * 8 + 16;  // + TMEM holder, abort flag
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

// MASK: which keys count is bounded by 0: m alone, 1: a length for each batch row, 2: a byte for
// each key (and perhaps a length).
template <int D, int MASK>
__global__ void __launch_bounds__(kCrossThreads, 1)
    cross_fwd_tc_kernel(const __grid_constant__ CrossMaps maps, const __grid_constant__ CrossFwdArgs args) {
  using Lay = CrossFwdLayout<D, MASK>;
  constexpr int DH = D / 64;
  constexpr bool MASKED = MASK > 0;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::BAR_OFF);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Lay::BAR_OFF + Lay::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::BAR_OFF + Lay::NBAR * 8 + 4);
  const CrossPlan& plan = args.plan;
  const int warp = int(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint64_t to = args.timeout_ns;
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it; dynamic shared memory starts aligned
    if (threadIdx.x == 0) atomicCAS(args.err, 0, 1);
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::NBAR; ++i) {
      // the softmax and epilogue warps arrive one by one
      const int count = (i >= Lay::PF && i < Lay::OF) || (i >= Lay::OE && i < Lay::WF) ? 4 : 1;
      mbar_init(&bars[i], count);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 14) {  // a warp whose lanes stay together: TMEM is taken and given back by whole warps
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if constexpr (MASK == 2) {  // column 0 of the ones; the masks' columns 1 to 15 stay zero
    for (uint32_t at = threadIdx.x * 16; at < uint32_t(Lay::KV_OFF - Lay::BIAS_OFF); at += kCrossThreads * 16)
      st_shared_v4(smem_u32(smem) + Lay::BIAS_OFF + at, at < 2048u ? 0x3f80u : 0u, 0u, 0u, 0u);
    fence_async_smem();
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
    uint32_t size;
    int count;
    __device__ __forceinline__ uint32_t slot(int x, uint32_t n) const {
      return (count == 2 ? x * size : 0u) + n % size;
    }
    __device__ __forceinline__ uint32_t use(uint32_t n) const { return n / size; }
  };
  const Ring ring = plan.splits > 1 ? Ring{uint32_t(Lay::NS), 2} : Ring{uint32_t(Lay::NKV), 1};

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
    regs_give<kCrossOtherRegs>();
    if (warp == 12) {
      // ============================================================== key and value loads
      if (lane == 0) {
        uint32_t e[2] = {0, 0};
        // cut: a value tile with rows past a length, which the mask warp passes on
        auto load = [&](int x, const CUtensorMap* m, int row, int h, int b, bool cut) -> bool {
          const uint32_t n = x ? e[1] : e[0], s = ring.slot(x, n);
          if (!cross_wait(&bars[Lay::KVE + s], (ring.use(n) & 1) ^ 1, abort_flag, to)) return false;
          uint64_t* full = &bars[(MASK == 1 && cut ? Lay::RDY : Lay::KVF) + s];
          mbar_arrive_expect_tx(full, Lay::TILE);
#pragma unroll
          for (int c = 0; c < DH; ++c)
            tma_load_4d(sbase + Lay::KV_OFF + s * Lay::TILE + c * kCrossBlk, m, full, c * 64, row, h, b);
          x ? ++e[1] : ++e[0];
          return true;
        };
        bool ok = true;
        for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
          const CrossItem it = cross_item(plan, args.heads, i);
          const int len = len_of(it.b);
          const CrossRange r = cross_range(plan, len, it.sp[0]);
          const int kh = it.hk * args.k_h, kb = it.b * args.k_b, vh = it.hk * args.v_h, vb = it.b * args.v_b;
          // values of block k - 1, then keys of block k
          for (int k = 0; ok && k <= r.nk; ++k)
            for (int x = 0; ok && x < ring.count; ++x) {
              const int row = (r.k0 + x * r.nk + k) * 128;
              if (k > 0) ok = load(x, &maps.v, row - 128, vh, vb, row > len);
              if (ok && k < r.nk) ok = load(x, &maps.k, row, kh, kb, false);
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
      if (MASK == 1) {
        // Only the value tiles that a length cuts, in the order of their products: their loads arrive
        // here (RDY), and this warp's arrival stands for the load's at the issuer (KVF). The other tiles
        // go from the loads to the issuer. (Passing every tile on cost 53,680 x 128 with a length 166 us
        // in place of 142, the pair of 512 and 126 states 524 in place of 508: this warp's code is fetched
        // beside that of the softmax warps.)
        uint32_t e[2] = {0, 0}, phase = 0;  // bit s: parity of slot s' cut tiles
        bool ok = true;
#pragma unroll 1
        for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
          const CrossItem it = cross_item(plan, args.heads, i);
          const int len = len_of(it.b);
          const CrossRange r = cross_range(plan, len, it.sp[0]);
          const int cut = len >> 7;  // the first such block; key block k of job x is r.k0 + x nk + k
#pragma unroll 1
          for (int k = cut - (r.k0 + (ring.count - 1) * r.nk) > 0 ? cut - (r.k0 + (ring.count - 1) * r.nk) : 0;
               ok && k < r.nk; ++k)
#pragma unroll 1
            for (int x = 0; ok && x < ring.count; ++x) {
              const int block = r.k0 + x * r.nk + k;
              if (block < cut) continue;
              // a ring holds K(0) V(0) K(1) V(1) ... of an item
              const uint32_t s = ring.slot(x, (x ? e[1] : e[0]) + 2 * k + 1);
              if (!(ok = cross_warp_wait(&bars[Lay::RDY + s], (phase >> s) & 1u, abort_flag, to))) break;
              phase ^= 1u << s;
              uint32_t w[4];
              block_words(len - block * 128, nullptr, lane, w);
              zero_rows<D, true>(sbase + Lay::KV_OFF + s * Lay::TILE, w, lane);
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars[Lay::KVF + s]);
            }
          e[0] += 2 * r.nk;
          e[1] += 2 * r.nk;
        }
      } else if (MASK == 2) {
        uint32_t e[2] = {0, 0}, blocks[2] = {0, 0};
        // a key tile with a mask of each key: masked rows to zero, and the mask as an operand (0 or -inf
        // in column 0), whose product with a column of ones puts masked scores to -inf; the words
        // themselves go to the softmax warps. (A key tile lies in every other ring slot, and has the
        // operand's place as long as the slot.) A block's place among the words is free again: its key
        // tile came into a ring slot that the softmax of at least kCrossWords - 1 - NKV / 2 blocks
        // before is behind.
        auto pass = [&](int x, bool value, const uint32_t (&w)[4]) -> bool {
          const uint32_t n = x ? e[1] : e[0], s = ring.slot(x, n);
          if (!cross_warp_wait(&bars[Lay::KVF + s], ring.use(n) & 1, abort_flag, to)) return false;
          if (value) {
            zero_rows<D>(sbase + Lay::KV_OFF + s * Lay::TILE, w, lane);
          } else {
            const uint32_t at = x * kCrossWords + (x ? blocks[1] : blocks[0]) % kCrossWords;
            zero_rows<D>(sbase + Lay::KV_OFF + s * Lay::TILE, w, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              st_shared_v4(sbase + Lay::BIAS_OFF + (1 + (s >> 1)) * kCrossBias + (32 * j + lane) * 16,
                           (w[j] >> lane) & 1u ? 0u : 0xff80u, 0u, 0u, 0u);
            fence_async_smem();
            if (lane == 0) {
              st_shared_v4(sbase + Lay::WORD_OFF + at * 16, w[0], w[1], w[2], w[3]);
              mbar_arrive(&bars[Lay::WF + at]);
            }
            x ? ++blocks[1] : ++blocks[0];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::RDY + s]);
          x ? ++e[1] : ++e[0];
          return true;
        };
        bool ok = true;
        for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
          const CrossItem it = cross_item(plan, args.heads, i);
          const int len = len_of(it.b);
          const CrossRange r = cross_range(plan, len, it.sp[0]);
          const unsigned char* keys = args.mask.keys + it.b * args.mask.stride;
          uint32_t last[2][4] = {};  // masks of each job's block k - 1, for its values
          for (int k = 0; ok && k <= r.nk; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!ok || x >= ring.count) continue;
              const int row = (r.k0 + x * r.nk + k) * 128;
              uint32_t w[4] = {0u, 0u, 0u, 0u};
              if (k < r.nk) block_words(len - row, keys + row, lane, w);
              if (k > 0) ok = pass(x, true, last[x]);
              if (ok && k < r.nk) ok = pass(x, false, w);
#pragma unroll
              for (int z = 0; z < 4; ++z) last[x][z] = w[z];
            }
        }
      }
    } else if (warp == 15) {
      // ============================================================== query loads
      if (lane == 0) {
        uint32_t n[2] = {0, 0};
        bool ok = true;
        for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
          const CrossItem it = cross_item(plan, args.heads, i);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || it.qt[x] < 0) continue;
            if (!(ok = cross_wait(&bars[Lay::QE + x], (n[x] & 1) ^ 1, abort_flag, to))) continue;
            mbar_arrive_expect_tx(&bars[Lay::QF + x], Lay::TILE);
#pragma unroll
            for (int c = 0; c < DH; ++c)
              tma_load_4d(sbase + x * Lay::TILE + c * kCrossBlk, &maps.q, &bars[Lay::QF + x], c * 64, it.qt[x] * 128,
                          it.h * args.q_h, it.b * args.q_b);
            ++n[x];
          }
          // the next item's into L2: its loads come late, behind this item's last scores
          if (i + int(gridDim.x) < plan.items) {
            const CrossItem nx = cross_item(plan, args.heads, i + int(gridDim.x));
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int c = 0; c < DH; ++c)
                if (nx.qt[x] >= 0)
                  tma_prefetch_4d(&maps.q, c * 64, nx.qt[x] * 128, nx.h * args.q_h, nx.b * args.q_b);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (n[x]) mbar_wait_drain(&bars[Lay::QF + x], (n[x] - 1) & 1, to);
      }
    } else if (warp == 13) {
      // ============================================================== MMA issuer
      constexpr uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t id_o = idesc_bf16_f32(128, D, 0, 1);
      constexpr int FULL = MASK == 2 ? Lay::RDY : Lay::KVF;
      const uint32_t el = elect_one(), tm = uniform(tmem);
      const uint64_t q0 = sdesc_sw128(sbase, 16, 1024), k0 = sdesc_sw128(sbase + Lay::KV_OFF, 16, 1024),
                     v0 = sdesc_sw128(sbase + Lay::KV_OFF, kCrossBlk, 1024),
                     ones = sdesc_plain(sbase + Lay::BIAS_OFF, 2048, 128);
      auto wait = [&](int bar, uint32_t parity) -> bool {
        return cross_warp_wait(&bars[bar], parity, abort_flag, to);
      };
      const bool own = ring.count == 2;
      // ring places as slot | phase << 8, so that no step divides
      uint32_t pos[2] = {0, ring.size};
      auto next = [&](int r) -> uint32_t {
        const uint32_t at = pos[r], first = r ? ring.size : 0u;
        pos[r] = (at & 255u) + 1 == first + ring.size ? first | ((at & 256u) ^ 256u) : at + 1;
        return at;
      };
      // job x: its pending block (scores issued, P V still to come), that block's value tile and
      // place in the job; parity of its P V products; jobs begun
      bool pend[2] = {}, pfirst[2] = {}, plast[2] = {}, pnew[2] = {}, pdone[2] = {};
      uint32_t vpos[2] = {0, 0}, ppar[2] = {0, 0}, jobs[2] = {0, 0}, tiles[2] = {0, 0};
      uint32_t kpos = 0;
      bool ok = true;
      auto step = [&](auto X, bool scores, bool first, bool last, bool two) -> bool {
        constexpr int x = decltype(X)::value;
        const uint32_t ts = tm + 128 * x, tacc = tm + 256 + D * x;
        // everything but P is there by now or comes soon: waited for first, so that the products
        // below follow each other once P is
        const uint32_t sv = vpos[x] & 255u;
        const bool pv = pend[x], first_pv = pfirst[x], last_pv = plast[x], done_pv = pdone[x];
        if (pv) {
          if (pnew[x] && !wait(FULL + sv, vpos[x] >> 8)) return false;
          // the job's first product overwrites O: the epilogue has drained the last job's
          if (first_pv) {
            if (jobs[x] > 0 && !wait(Lay::OE + x, (jobs[x] - 1) & 1)) return false;
            ++jobs[x];
          }
        }
        const bool fresh = own || x == 0, done = own || x == 1 || !two;
        if (scores) {
          if (fresh) {
            kpos = next(own ? x : 0);
            vpos[x] = next(own ? x : 0);
            if (!wait(FULL + (kpos & 255u), kpos >> 8)) return false;
          } else {
            vpos[x] = vpos[0];
          }
          if (first) {
            if (!wait(Lay::QF + x, tiles[x] & 1)) return false;
            ++tiles[x];
          }
        }
        if (pv) {  // P V of the block before
          const uint64_t va = v0 + sv * (Lay::TILE >> 4);
          if (!wait(Lay::PF + x, ppar[x])) return false;
          tc_fence_after();
          mma_ts_by(el, tacc, ts, va, id_o, first_pv ? 0u : 1u);
#pragma unroll
          for (int kk = 1; kk < 8; ++kk) mma_ts_by(el, tacc, ts + kk * 8, va + kk * (2048 >> 4), id_o, 1u);
          if (done_pv) tc_commit_by(el, &bars[Lay::KVE + sv]);
          if (last_pv) tc_commit_by(el, &bars[Lay::OF + x]);
          ppar[x] ^= 1u;
          pend[x] = false;
        }
        if (!scores) return true;
        // S overwrites the columns that the P V above reads P from: the tensor core runs the
        // products of one thread in issue order
        tc_fence_after();
        const uint64_t qa = q0 + x * (Lay::TILE >> 4), ka = k0 + (kpos & 255u) * (Lay::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kCrossBlk + (kk & 3) * 32) >> 4;
          mma_ss_by(el, ts, qa + off, ka + off, id_s, kk > 0 ? 1u : 0u);
        }
        if (MASK == 2)  // 1 times 0 or -inf
          mma_ss_by(el, ts, ones, ones + (1 + ((kpos & 255u) >> 1)) * (kCrossBias >> 4), id_s, 1u);
        tc_commit_by(el, &bars[Lay::SF + x]);
        if (done) tc_commit_by(el, &bars[Lay::KVE + (kpos & 255u)]);
        if (last) tc_commit_by(el, &bars[Lay::QE + x]);
        pend[x] = true;
        pfirst[x] = first;
        plast[x] = last;
        pnew[x] = fresh;
        pdone[x] = done;
        return true;
      };
#pragma unroll 1
      for (int i = blockIdx.x; ok; i += gridDim.x) {
        // past the last item: one turn for the products still pending
        const bool more = i < plan.items;
        int nk = 1;
        bool two = false;
        if (more) {
          const CrossItem it = cross_item(plan, args.heads, i);
          nk = cross_range(plan, int(uniform(uint32_t(len_of(it.b)))), it.sp[0]).nk;
          two = it.qt[1] >= 0;
        }
#pragma unroll 1
        for (int k = 0; ok && k < nk; ++k)
          ok = step(std::integral_constant<int, 0>{}, more, k == 0, k == nk - 1, two) &&
               step(std::integral_constant<int, 1>{}, more && two, k == 0, k == nk - 1, two);
        if (!more) break;
      }
      tc_commit_by(el, &bars[Lay::DRAIN]);
      mbar_wait_drain(&bars[Lay::DRAIN], 0, to);
    }
  } else if (warp >= 8) {
    // ================================================================ epilogue
    regs_give<kCrossOtherRegs>();
    const int row = threadIdx.x & 127;
    uint32_t jobs = 0;    // bit x: parity of job slot x's jobs
    uint32_t halves = 0;  // 64-channel halves staged; half n goes through buffer n & 1
    const int row0 = (warp & 3) * 32;
    bool ok = true;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return cross_warp_wait(bar, parity, abort_flag, to);
    };
#pragma unroll 1
    for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
      const CrossItem it = cross_item(plan, args.heads, i);
#pragma unroll 1
      for (int x = 0; ok && x < 2; ++x) {
        const int qt = x ? it.qt[1] : it.qt[0];
        if (qt < 0) continue;
        const uint32_t job = (jobs >> x) & 1u;
        jobs ^= 1u << x;
        if (!(ok = wwait(&bars[Lay::LF + x], job))) break;
        float m2, l;  // maximum (base 2) and sum of the row
        ld_shared_f2(sbase + Lay::STAT_OFF + (x * 128 + row) * 8, m2, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Lay::LE + x]);
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // NaN stays NaN
        const int tok = qt * 128 + row;
        __syncwarp();
        if (!(ok = wwait(&bars[Lay::OF + x], job))) break;
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
          if (tok < args.n)
            args.part_lse[(long long)(it.sp[0] + x) * args.B * args.heads * args.n +
                          ((long long)it.b * args.heads + it.h) * args.n + tok] = l == 0.f ? -INFINITY : m2 + log2f(l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::OE + x]);
          continue;
        }
#pragma unroll 1
        for (int h = 0; h < DH; ++h, ++halves) {
          const uint32_t stage = sbase + Lay::STAGE_OFF + (halves % Lay::STAGES) * kCrossBlk + row0 * 128;
          // the last store into this buffer has read it
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(Lay::STAGES - 1) : "memory");
          __syncwarp();
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            uint32_t v[32];
            tmem_ld32(t + 64 * h + c, v);
            // 1 / sum is 0 for a row without keys; what the products hold there is not looked at
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t p[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                p[e] = inv == 0.f ? 0u
                                  : pack_bf16x2(__uint_as_float(v[8 * j + 2 * e]) * inv,
                                                __uint_as_float(v[8 * j + 2 * e + 1]) * inv);
              st_shared_v4(stage + lane * 128 + ((((c >> 3) + j) ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
            }
          }
          tc_fence_before();
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (h == DH - 1) mbar_arrive(&bars[Lay::OE + x]);  // O is read
            if (qt * 128 + row0 < args.n)
              tma_store_4d(&maps.o, stage, h * 64, qt * 128 + row0, it.h * args.o_h, it.b * args.o_b);
            bulk_commit();
          }
        }
        // behind the staging, whose fence would wait for it
        if (args.lse != nullptr && tok < args.n)
          args.lse[((long long)it.b * args.heads + it.h) * args.n + tok] =
              l == 0.f ? -INFINITY : (m2 + log2f(l)) * 0.69314718055994530942f;
      }
    }
    if (lane == 0) bulk_wait_read();
  } else {
    // ================================================================ softmax
    regs_take<kCrossSoftmaxRegs>();
    const int x = warp >> 2, row = threadIdx.x & 127;
    const uint32_t tS = tmem + (uint32_t((warp & 3) * 32) << 16) + 128 * x;
    const uint32_t tO = tmem + (uint32_t((warp & 3) * 32) << 16) + 256 + D * x;
    const float c2 = args.scale_log2;
    const uint64_t c2x2 = f2(c2, c2);
    uint32_t sc = 0, jobs = 0;  // blocks and jobs so far
    uint32_t words = 0;         // blocks of the ring so far, also those of items without a job here
    bool ok = true;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return cross_warp_wait(bar, parity, abort_flag, to);
    };
    for (int i = blockIdx.x; ok && i < plan.items; i += gridDim.x) {
      const CrossItem it = cross_item(plan, args.heads, i);
      const int qt = x ? it.qt[1] : it.qt[0];
      const CrossRange r = cross_range(plan, len_of(it.b), x ? it.sp[1] : it.sp[0]);
      if (qt < 0) {
        words += uint32_t(r.nk);
        continue;
      }
      // a warp whose rows all lie past the last query has nothing to compute
      const bool idle = qt * 128 + (warp & 3) * 32 >= args.n;
      float m_run = -INFINITY, l_run = 0.f;
      uint32_t any = MASK == 2 ? 0u : 1u;  // a key counts
      for (int k = 0; k < r.nk; ++k, ++sc) {
        if (!(ok = wwait(&bars[Lay::SF + x], sc & 1))) break;
        tc_fence_after();
        // Which keys count: all below the length; with a mask of each key the scores have it already, and
        // its words tell whether the job has a key at all. The mask warp wrote them before it passed
        // the key tile on, so they are there by now, and the phase is the block's own: its place is
        // taken again eight blocks later, which this job's products hold back.
        uint32_t w[4];
        if (MASK == 2) {
          const uint32_t at = (ring.count == 2 ? x * kCrossWords : 0u) + words % kCrossWords;
          if (!(ok = wwait(&bars[Lay::WF + at], (words / kCrossWords) & 1))) break;
          const uint4 t = ld_shared_v4(sbase + Lay::WORD_OFF + at * 16);
          w[0] = t.x;
          w[1] = t.y;
          w[2] = t.z;
          w[3] = t.w;
          any |= w[0] | w[1] | w[2] | w[3];
          ++words;
        } else {
          block_words((MASKED ? len_of(it.b) : args.m) - (r.k0 + k) * 128, nullptr, lane, w);
        }
        if (idle) {
          tc_fence_before();
          if (lane == 0) {
            mbar_arrive(&bars[Lay::PF + x]);
          }
          continue;
        }
        const bool partial = (w[0] & w[1] & w[2] & w[3]) != ~0u;
        // Without a mask of each key only the last block is partial: its scores past the keys become
        // -inf where they lie, in a short loop (the code below is fetched for every block and has to
        // stay small: selects in registers cost the padded 53,680 pair 3%)
        if (MASK < 2 && partial) {
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
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_async(tS + 32 * c, v[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(v[c]);
        float a[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (c == 0)
              a[j] = fmaxf(__uint_as_float(v[c][j]), __uint_as_float(v[c][j + 8]));
            else
              a[j] = fmax3(a[j], __uint_as_float(v[c][j]), __uint_as_float(v[c][j + 8]));
            a[j] = fmax3(a[j], __uint_as_float(v[c][j + 16]), __uint_as_float(v[c][j + 24]));
          }
        }
        const float mx = fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
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
        // P packed over the columns that the scores lay in, 32 keys at a time, handed over whole (in
        // two halves it took the issuer a wait more: 166.5 against 165 us at 27,280 x 512)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
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
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Lay::PF + x]);
        const uint64_t s2 = fadd2(sum[0], sum[1]);
        l_run = l_run * alpha + (f2_lo(s2) + f2_hi(s2));
        m_run = m_use;
      }
      if (!ok) break;
      if (any == 0u) {  // zeros, whatever the query holds
        m_run = -INFINITY;
        l_run = 0.f;
      }
      // the row's statistics for the epilogue, which has read the last job's
      if (!(ok = wwait(&bars[Lay::LE + x], (jobs & 1) ^ 1))) break;
      st_shared_f2(sbase + Lay::STAT_OFF + (x * 128 + row) * 8, m_run * c2, l_run);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Lay::LF + x]);
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
// l_s = log2 of the split's sum. One warp per row, its lanes over the channels.
template <typename T>
__global__ void __launch_bounds__(128) cross_join_kernel(const float* __restrict__ part_o,
                                                         const float* __restrict__ part_lse, int splits,
                                                         long long rows, int heads, int n, int D, T* o, CrossStride so,
                                                         float* lse) {
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  // lane s holds the weights of splits s and s + 32 (there are at most 64)
  const float l0 = lane < splits ? part_lse[lane * rows + row] : -INFINITY;
  const float l1 = lane + 32 < splits ? part_lse[(lane + 32) * rows + row] : -INFINITY;
  float mx = fmaxf(l0, l1);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  const float ref = mx == -INFINITY ? 0.f : mx;
  const float w0 = exp2f(l0 - ref), w1 = exp2f(l1 - ref);
  float total = w0 + w1;
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
  const float inv = total > 0.f ? 1.f / total : total;
  const long long bh = row / n;
  const int i = int(row - bh * n), b = int(bh / heads), h = int(bh - (long long)b * heads);
  T* out = o + b * so.b + h * so.h + i * so.n;
  for (int c0 = 0; c0 < D; c0 += 128) {
    const int c = c0 + 4 * lane;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float wt = __shfl_sync(0xffffffffu, s < 32 ? w0 : w1, s & 31);
      if (c < D) {
        const float4 p = *reinterpret_cast<const float4*>(part_o + (s * rows + row) * D + c);
        acc.x = fmaf(wt, p.x, acc.x);
        acc.y = fmaf(wt, p.y, acc.y);
        acc.z = fmaf(wt, p.z, acc.z);
        acc.w = fmaf(wt, p.w, acc.w);
      }
    }
    if (c >= D) continue;
    if (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(out + c) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    else
      *reinterpret_cast<float4*>(out + c) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  }
  if (lse != nullptr && lane == 0) lse[row] = total == 0.f ? mx : (mx + log2f(total)) * 0.69314718055994530942f;
}

}  // namespace sq
