// cross_api.cu - C ABI of the operators around the grid attention: cross attention to an
// encoder's states (squad_cross_*) and rotary positions (squad_rotary). Host side only:
// argument checks, plans, tensor maps and launches on the caller's stream.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <utility>

#include "squad.h"
#include "cross_bwd_tc.cuh"
#include "cross_f32.cuh"
#include "cross_fwd_tc.cuh"
#include "geometry.h"
#include "host_state.h"
#include "rotary.cuh"

namespace {

using sq::align256;
using sq::aligned16;

constexpr long long kMaxRows = 1ll << 31;
constexpr int kMaxGridYZ = 65535;

size_t elem_size(int dtype) { return dtype == SQUAD_BF16 ? 2 : 4; }

// Strides a tensor of extents B x h x n may have: multiples of 16 bytes and not negative;
// rows at least d apart; a stride of an extent of 1 is not looked at. broadcast (inputs): batch and
// head strides of 0 are allowed. Else (outputs) no two rows may overlap: the strides in ascending
// order each step over all that the smaller ones reach.
bool stride_ok(const squad_strides& s, int B, int h, int n, int d, size_t elem, bool broadcast) {
  const long long unit = 16 / (long long)elem;
  const long long lo = broadcast ? 0 : d;
  if (n > 1 && (s.n < d || s.n % unit != 0 || s.n >= (1ll << 36))) return false;
  if (h > 1 && (s.h < lo || s.h % unit != 0 || s.h >= (1ll << 36))) return false;
  if (B > 1 && (s.b < lo || s.b % unit != 0 || s.b >= (1ll << 36))) return false;
  if (broadcast) return true;
  long long step[3] = {n > 1 ? s.n : 0, h > 1 ? s.h : 0, B > 1 ? s.b : 0}, size[3] = {n, h, B}, reach = d;
  for (int i = 0; i < 3; ++i) {
    int at = i;
    for (int j = i + 1; j < 3; ++j)
      if (step[j] < step[at]) at = j;
    std::swap(step[i], step[at]);
    std::swap(size[i], size[at]);
    if (size[i] <= 1) continue;
    if (step[i] < reach) return false;
    reach += (size[i] - 1) * step[i];
  }
  return true;
}

bool same_rows(const squad_strides& a, const squad_strides& b, int B, int h, int n) {
  return (B <= 1 || a.b == b.b) && (h <= 1 || a.h == b.h) && (n <= 1 || a.n == b.n);
}

// ---------------------------------------------------------------- cross attention

squad_status check_cross(const squad_cross_desc* d) {
  if (d == nullptr) return SQUAD_ERR_INVALID_ARG;
  if (d->dtype != SQUAD_F32 && d->dtype != SQUAD_BF16) return SQUAD_ERR_INVALID_ARG;
  if (!(d->scale > 0.f) && !(d->scale <= 0.f)) return SQUAD_ERR_INVALID_ARG;  // NaN
  if (d->B <= 0 || d->heads <= 0 || d->kv_heads <= 0 || d->n <= 0 || d->m <= 0 || d->d <= 0) return SQUAD_ERR_SHAPE;
  if (d->heads % d->kv_heads) return SQUAD_ERR_SHAPE;
  const long long rows = (long long)d->B * d->heads, krows = (long long)d->B * d->kv_heads;
  if (rows * d->n >= kMaxRows || krows * d->m >= kMaxRows) return SQUAD_ERR_SHAPE;
  if (d->B > kMaxGridYZ || d->heads > kMaxGridYZ) return SQUAD_ERR_UNSUPPORTED;
  if (d->dtype == SQUAD_BF16 ? (d->d != 64 && d->d != 128) : (d->d % 32 != 0 || d->d > 256))
    return SQUAD_ERR_UNSUPPORTED;
  return SQUAD_OK;
}

squad_status check_cross_strides(const squad_cross_desc* d, bool bwd) {
  const size_t e = elem_size(d->dtype);
  const int B = d->B, h = d->heads, hk = d->kv_heads;
  if (!stride_ok(d->q, B, h, d->n, d->d, e, true) || !stride_ok(d->k, B, hk, d->m, d->d, e, true) ||
      !stride_ok(d->v, B, hk, d->m, d->d, e, true) || !stride_ok(d->o, B, h, d->n, d->d, e, false))
    return SQUAD_ERR_ALIGN;
  if (bwd && (!stride_ok(d->dout, B, h, d->n, d->d, e, true) || !stride_ok(d->dq, B, h, d->n, d->d, e, false) ||
              !stride_ok(d->dk, B, hk, d->m, d->d, e, false) || !stride_ok(d->dv, B, hk, d->m, d->d, e, false)))
    return SQUAD_ERR_ALIGN;
  return SQUAD_OK;
}

sq::CrossStride strides_of(const squad_strides& s) { return {s.b, s.h, s.n}; }

size_t bwd_rowvec_bytes(const squad_cross_desc* d) { return align256(size_t(d->B) * d->heads * d->n * sizeof(float)); }

sq::CrossArgs cross_args(const squad_cross_desc* d, const void* q, const void* k, const void* v, const int* kv_lens,
                         const unsigned char* key_mask) {
  sq::CrossArgs a{};
  a.B = d->B;
  a.heads = d->heads;
  a.kv_heads = d->kv_heads;
  a.group = d->heads / d->kv_heads;
  a.n = d->n;
  a.m = d->m;
  a.d = d->d;
  a.scale = d->scale > 0.f ? d->scale : 1.0f / std::sqrt(float(d->d));
  a.mask = {kv_lens, key_mask, d->mask_stride};
  a.sq = strides_of(d->q);
  a.sk = strides_of(d->k);
  a.sv = strides_of(d->v);
  a.so = strides_of(d->o);
  a.sdo = strides_of(d->dout);
  a.sdq = strides_of(d->dq);
  a.sdk = strides_of(d->dk);
  a.sdv = strides_of(d->dv);
  a.q = q;
  a.k = k;
  a.v = v;
  return a;
}

constexpr int kMaxDevices = 64;

// The attribute is set once per kernel and device; a repeated set by two threads is harmless.
template <typename K>
squad_status allow_smem(K kern, int bytes, const sq::HostDevice& dev, std::atomic<bool>* done) {
  if (!done[dev.device].load(std::memory_order_acquire)) {
    SQ_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    done[dev.device].store(true, std::memory_order_release);
  }
  return SQUAD_OK;
}

// ---------------------------------------------------------------- fp32

struct FwdWs {
  int splits;
  size_t part_lse, total;  // parts of o first
};

// Rows of the fp32 forward and dq tiles, in 16s: 32 where that leaves a block for three quarters of
// the SMs (24 heads of 96, 300 x 300: forward 64 us with 16 rows, 54 with 32; 2 heads of 192, 2,000 x
// 500: 95 and 75; but 2 heads of 64, 256 x 77: 8.6 and 10.7).
int f32_rows(const squad_cross_desc* d) {
  return (long long)d->B * d->heads * ((d->n + 31) / 32) * 4 >= 3 * sq::kCrossPlanSms ? 2 : 1;
}

FwdWs fwd_workspace(const squad_cross_desc* d) {
  FwdWs w{};
  const long long bh = (long long)d->B * d->heads;
  if (d->dtype == SQUAD_BF16) {
    w.splits = sq::make_cross_plan(d->B, d->heads, d->kv_heads, d->n, d->m).splits;
  } else {
    // parts of the keys where the query tiles leave SMs idle, two tiles of keys at least to a part
    const int rows = 16 * f32_rows(d), tiles = (d->m + sq::kF32Cols - 1) / sq::kF32Cols;
    const long long blocks = bh * ((d->n + rows - 1) / rows);
    const long long s = blocks * 2 <= sq::kCrossPlanSms ? sq::kCrossPlanSms / blocks : 1;
    const long long most = tiles / 2 < 64 ? tiles / 2 : 64;
    w.splits = int(s < most ? s : most);
    if (w.splits < 1) w.splits = 1;
  }
  if (w.splits <= 1) return w;
  const size_t rows = size_t(bh) * d->n * w.splits;
  w.part_lse = align256(rows * d->d * sizeof(float));
  w.total = w.part_lse + align256(rows * sizeof(float));
  return w;
}

template <int D, int R>
squad_status f32_cross_fwd(const sq::HostDevice& dev, const sq::CrossArgs& a, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  auto kern = sq::cross_f32_fwd_kernel<D, R>;
  squad_status s = allow_smem(kern, sq::F32Layout<D, R>::FWD, dev, done);
  if (s != SQUAD_OK) return s;
  const dim3 grid(unsigned((a.n + 16 * R - 1) / (16 * R) * a.splits), unsigned(a.heads), unsigned(a.B));
  kern<<<grid, sq::kF32Threads, sq::F32Layout<D, R>::FWD, st>>>(a);
  SQ_CUDA(cudaGetLastError());
  if (a.splits > 1) {
    const long long rows = (long long)a.B * a.heads * a.n;
    sq::cross_join_kernel<float><<<unsigned((rows + 3) / 4), 128, 0, st>>>(
        a.part, a.part_lse, a.splits, rows, a.heads, a.n, D, static_cast<float*>(a.o), a.so, a.lse);
    SQ_CUDA(cudaGetLastError());
  }
  return SQUAD_OK;
}

// dq of queries whose keys were cut into parts
template <typename T>
squad_status join_dq(const float* part, int splits, int B, int heads, int n, int D, T* dq, const sq::CrossStride& sdq,
                     cudaStream_t st) {
  const long long rows = (long long)B * heads * n;
  sq::cross_join_grads_kernel<T><<<unsigned((rows * (D / 4) + 255) / 256), 256, 0, st>>>(part, splits, rows, n, heads, n,
                                                                                         D, rows, dq, sdq, dq, sdq);
  SQ_CUDA(cudaGetLastError());
  return SQUAD_OK;
}

template <int D, int R>
squad_status f32_cross_dq(const sq::HostDevice& dev, const sq::CrossArgs& a, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  auto dq = sq::cross_f32_dq_kernel<D, R>;
  squad_status s;
  if ((s = allow_smem(dq, sq::F32Layout<D, R>::DQ, dev, done)) != SQUAD_OK) return s;
  const dim3 gq(unsigned((a.n + 16 * R - 1) / (16 * R) * a.dq_splits), unsigned(a.heads), unsigned(a.B));
  dq<<<gq, sq::kF32Threads, sq::F32Layout<D, R>::DQ, st>>>(a);
  SQ_CUDA(cudaGetLastError());
  if (a.dq_splits > 1 && (s = join_dq<float>(a.dq_part, a.dq_splits, a.B, a.heads, a.n, D, static_cast<float*>(a.dq),
                                             a.sdq, st)) != SQUAD_OK)
    return s;
  return SQUAD_OK;
}

template <int D, int R>
squad_status f32_cross_dkdv(const sq::HostDevice& dev, const sq::CrossArgs& a, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  // the blocks that the plan counts on (228 KB an SM, 1 of them reserved for each)
  static_assert(sq::cross_f32_dkdv_blocks(D) * (sq::F32Layout<D, R>::DKV + 1024) <= 228 * 1024, "blocks of an SM");
  auto dkv = sq::cross_f32_dkdv_kernel<D, R>;
  squad_status s;
  if ((s = allow_smem(dkv, sq::F32Layout<D, R>::DKV, dev, done)) != SQUAD_OK) return s;
  const dim3 gk(unsigned((a.m + 16 * R - 1) / (16 * R) * a.splits), unsigned(a.kv_heads), unsigned(a.B));
  dkv<<<gk, sq::kF32Threads, sq::F32Layout<D, R>::DKV, st>>>(a);
  SQ_CUDA(cudaGetLastError());
  if (a.splits > 1) {
    const long long rows = (long long)a.B * a.kv_heads * a.m;
    const dim3 grid(unsigned((rows * (D / 4) + 255) / 256), 2);
    sq::cross_join_grads_kernel<float><<<grid, 256, 0, st>>>(a.part, a.splits, rows, a.m, a.kv_heads, a.m, D, rows,
                                                             static_cast<float*>(a.dk), a.sdk,
                                                             static_cast<float*>(a.dv), a.sdv);
    SQ_CUDA(cudaGetLastError());
  }
  return SQUAD_OK;
}

enum F32Kernel { kF32Fwd, kF32Dq, kF32Dkdv };

template <F32Kernel WHICH, int D, int R>
squad_status f32_cross_run(const sq::HostDevice& dev, const sq::CrossArgs& a, cudaStream_t st) {
  if constexpr (WHICH == kF32Fwd) return f32_cross_fwd<D, R>(dev, a, st);
  if constexpr (WHICH == kF32Dq) return f32_cross_dq<D, R>(dev, a, st);
  if constexpr (WHICH == kF32Dkdv) return f32_cross_dkdv<D, R>(dev, a, st);
}

template <F32Kernel WHICH>
squad_status f32_cross(const sq::HostDevice& dev, int r, const sq::CrossArgs& a, cudaStream_t st) {
#define SQ_D(N)                                                                                         \
  case N:                                                                                               \
    return r == 4   ? f32_cross_run<WHICH, N, (WHICH == kF32Dkdv ? sq::cross_f32_dkdv_rows(N) : 2)>(dev, a, st) \
           : r == 2 ? f32_cross_run<WHICH, N, 2>(dev, a, st)                                            \
                    : f32_cross_run<WHICH, N, 1>(dev, a, st)
  switch (a.d) {
    SQ_D(32);
    SQ_D(64);
    SQ_D(96);
    SQ_D(128);
    SQ_D(160);
    SQ_D(192);
    SQ_D(224);
    SQ_D(256);
  }
#undef SQ_D
  return SQUAD_ERR_UNSUPPORTED;
}

// ---------------------------------------------------------------- tensor-core forward (bf16)

// 4-D map (channel, row, head, batch) over a strided tensor, boxes of 64 channels x `rows` rows.
// Extents that are 1 or broadcast (stride 0) are left out: their coordinate is times mb, mh.
squad_status encode_rows(CUtensorMap* map, const sq::HostDevice& dev, const void* base, const squad_strides& st, int B,
                         int h, int n, int d, int* mb, int* mh, uint32_t rows = 128) {
  const uint64_t row = uint64_t(d) * 2;
  *mb = B > 1 && st.b != 0;
  *mh = h > 1 && st.h != 0;
  const uint64_t dims[4] = {uint64_t(d), uint64_t(n), *mh ? uint64_t(h) : 1, *mb ? uint64_t(B) : 1};
  const uint64_t strides[3] = {n > 1 ? uint64_t(st.n) * 2 : row, *mh ? uint64_t(st.h) * 2 : row,
                               *mb ? uint64_t(st.b) * 2 : row};
  const uint32_t box[4] = {64, rows, 1, 1};
  return sq::host_encode_bf16(map, dev.device, 4, base, dims, strides, box);
}

// CTAs of a persistent launch: one an SM takes the items in turn.
int cross_ctas(const sq::HostDevice& dev, int items) { return items < dev.sms ? items : dev.sms; }

template <int D, int MASK>
squad_status launch_cross_fwd(const sq::HostDevice& dev, const sq::CrossMaps& maps, const sq::CrossFwdArgs& a,
                              cudaStream_t st) {
  using Lay = sq::CrossFwdLayout<D, MASK>;
  auto kern = sq::cross_fwd_tc_kernel<D, MASK>;
  static std::atomic<bool> done[kMaxDevices];
  squad_status s = allow_smem(kern, Lay::BYTES, dev, done);
  if (s != SQUAD_OK) return s;
  kern<<<cross_ctas(dev, a.plan.items), sq::kCrossThreads, Lay::BYTES, st>>>(maps, a);
  SQ_CUDA(cudaGetLastError());
  return SQUAD_OK;
}

squad_status tc_cross_fwd(const sq::HostDevice& dev, const squad_cross_desc* d, const sq::CrossArgs& c,
                          cudaStream_t st) {
  sq::CrossMaps maps;
  sq::CrossFwdArgs a{};
  a.plan = sq::make_cross_plan(d->B, d->heads, d->kv_heads, d->n, d->m);
  a.B = d->B;
  a.heads = d->heads;
  a.n = d->n;
  a.m = d->m;
  squad_status s;
  if ((s = encode_rows(&maps.q, dev, c.q, d->q, d->B, d->heads, d->n, d->d, &a.q_b, &a.q_h)) != SQUAD_OK) return s;
  if ((s = encode_rows(&maps.k, dev, c.k, d->k, d->B, d->kv_heads, d->m, d->d, &a.k_b, &a.k_h)) != SQUAD_OK) return s;
  if ((s = encode_rows(&maps.v, dev, c.v, d->v, d->B, d->kv_heads, d->m, d->d, &a.v_b, &a.v_h)) != SQUAD_OK) return s;
  if ((s = encode_rows(&maps.o, dev, c.o, d->o, d->B, d->heads, d->n, d->d, &a.o_b, &a.o_h, 32)) != SQUAD_OK) return s;
  a.mask = c.mask;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  a.lse = c.lse;
  a.err = dev.err;
  a.timeout_ns = sq::cross_wait_ns(sq::kWaitTimeoutNs, a.plan.items, cross_ctas(dev, a.plan.items),
                                   (a.plan.kblocks + a.plan.splits - 1) / a.plan.splits);
  a.part_o = c.part;
  a.part_lse = c.part_lse;
  const int mask = c.mask.keys != nullptr ? 2 : c.mask.lens != nullptr ? 1 : 0;
  if (d->d == 128)
    s = mask == 2   ? launch_cross_fwd<128, 2>(dev, maps, a, st)
        : mask == 1 ? launch_cross_fwd<128, 1>(dev, maps, a, st)
                    : launch_cross_fwd<128, 0>(dev, maps, a, st);
  else
    s = mask == 2   ? launch_cross_fwd<64, 2>(dev, maps, a, st)
        : mask == 1 ? launch_cross_fwd<64, 1>(dev, maps, a, st)
                    : launch_cross_fwd<64, 0>(dev, maps, a, st);
  if (s != SQUAD_OK || a.plan.splits <= 1) return s;
  const long long rows = (long long)d->B * d->heads * d->n;
  const unsigned blocks = unsigned((rows + 3) / 4);
  sq::cross_join_kernel<__nv_bfloat16><<<blocks, 128, 0, st>>>(a.part_o, a.part_lse, a.plan.splits, rows, d->heads, d->n,
                                                              d->d, static_cast<__nv_bfloat16*>(c.o), c.so, c.lse);
  SQ_CUDA(cudaGetLastError());
  return SQUAD_OK;
}

// ---------------------------------------------------------------- tensor-core backward (bf16)

struct BwdWs {
  size_t part, dq_part, total;  // D vector first
  int splits, dq_splits;
  int f32_key_rows;  // of the fp32 dk, dv kernel, in 16s
};

BwdWs bwd_workspace(const squad_cross_desc* d) {
  BwdWs w{};
  w.splits = 1;
  w.part = bwd_rowvec_bytes(d);
  w.total = w.part;
  const bool tc = d->dtype == SQUAD_BF16;
  const long long units = (long long)d->B * d->kv_heads * ((d->m + 127) / 128);
  const long long tiles = (long long)(d->heads / d->kv_heads) * ((d->n + 127) / 128);
  if (tc) {
    w.splits = sq::cross_dkv_splits(units, int(tiles));
  } else {
    const sq::CrossF32Dkdv p =
        sq::cross_f32_dkdv_plan((long long)d->B * d->kv_heads, d->heads / d->kv_heads, d->n, d->m, d->d);
    w.splits = p.splits;
    w.f32_key_rows = p.rows;
  }
  const size_t rows = tc ? size_t(units) * 128 : size_t(d->B) * d->kv_heads * d->m;
  if (w.splits > 1) w.total += align256(size_t(2) * w.splits * rows * d->d * sizeof(float));
  const int qrows = tc ? 128 : 16 * f32_rows(d), kcols = tc ? 128 : sq::kF32Cols;
  w.dq_splits = sq::cross_dq_splits((long long)d->B * d->heads * ((d->n + qrows - 1) / qrows), (d->m + kcols - 1) / kcols,
                                    tc);
  w.dq_part = w.total;
  if (w.dq_splits > 1) w.total += align256(size_t(w.dq_splits) * d->B * d->heads * d->n * d->d * sizeof(float));
  return w;
}

template <int D, bool MASKED>
squad_status launch_cross_bwd(const sq::HostDevice& dev, const sq::CrossBwdMaps& maps, sq::CrossBwdArgs a,
                              cudaStream_t st) {
  squad_status s;
  static std::atomic<bool> done_q[kMaxDevices], done_kv[kMaxDevices];
  auto dq = sq::cross_bwd_dq_kernel<D, MASKED>;
  auto dkv = sq::cross_bwd_dkdv_kernel<D, MASKED>;
  if ((s = allow_smem(dq, sq::CrossDqLayout<D>::BYTES, dev, done_q)) != SQUAD_OK) return s;
  if ((s = allow_smem(dkv, sq::CrossDkvLayout<D>::BYTES, dev, done_kv)) != SQUAD_OK) return s;
  a.items = a.B * a.heads * a.qtiles * a.dq_splits;
  a.timeout_ns = sq::cross_wait_ns(sq::kWaitTimeoutNs, a.items, cross_ctas(dev, a.items),
                                   (a.kblocks + a.dq_splits - 1) / a.dq_splits);
  dq<<<cross_ctas(dev, a.items), sq::kCrossBwdThreads, sq::CrossDqLayout<D>::BYTES, st>>>(maps, a);
  SQ_CUDA(cudaGetLastError());
  if (a.dq_splits > 1 && (s = join_dq<__nv_bfloat16>(a.dq_part, a.dq_splits, a.B, a.heads, a.n, D, a.dq, a.sdq, st)) != SQUAD_OK)
    return s;
  a.items = a.B * a.kv_heads * a.kblocks * a.splits;
  a.timeout_ns = sq::cross_wait_ns(sq::kWaitTimeoutNs, a.items, cross_ctas(dev, a.items),
                                   (a.group * a.qtiles + a.splits - 1) / a.splits);
  dkv<<<cross_ctas(dev, a.items), sq::kCrossBwdThreads, sq::CrossDkvLayout<D>::BYTES, st>>>(maps, a);
  SQ_CUDA(cudaGetLastError());
  if (a.splits > 1) {
    const long long rows = (long long)a.B * a.kv_heads * a.m;
    const dim3 grid(unsigned((rows * (D / 4) + 255) / 256), 2);
    sq::cross_join_grads_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(
        a.part, a.splits, (long long)a.B * a.kv_heads * a.kblocks * 128, a.kblocks * 128, a.kv_heads, a.m, D, rows, a.dk,
        a.sdk, a.dv, a.sdv);
    SQ_CUDA(cudaGetLastError());
  }
  return SQUAD_OK;
}

squad_status tc_cross_bwd(const sq::HostDevice& dev, const squad_cross_desc* d, const sq::CrossArgs& c,
                          const BwdWs& w, void* ws, cudaStream_t st) {
  sq::CrossBwdMaps maps;
  sq::CrossBwdArgs a{};
  a.B = d->B;
  a.heads = d->heads;
  a.kv_heads = d->kv_heads;
  a.group = c.group;
  a.n = d->n;
  a.m = d->m;
  a.qtiles = (d->n + 127) / 128;
  a.kblocks = (d->m + 127) / 128;
  a.splits = w.splits;
  a.dq_splits = w.dq_splits;
  a.f_dq = sq::make_fastdiv(uint32_t(a.qtiles * a.dq_splits));
  a.f_dq_splits = sq::make_fastdiv(uint32_t(a.dq_splits));
  a.f_qtiles = sq::make_fastdiv(uint32_t(a.qtiles));
  a.f_heads = sq::make_fastdiv(uint32_t(a.heads));
  a.f_group = sq::make_fastdiv(uint32_t(a.group));
  a.f_kblocks = sq::make_fastdiv(uint32_t(a.kblocks));
  a.f_kv_heads = sq::make_fastdiv(uint32_t(a.kv_heads));
  squad_status s;
  const int B = d->B, h = d->heads, hk = d->kv_heads, D = d->d;
  if ((s = encode_rows(&maps.q, dev, c.q, d->q, B, h, d->n, D, &a.q_b, &a.q_h)) != SQUAD_OK) return s;
  if ((s = encode_rows(&maps.k, dev, c.k, d->k, B, hk, d->m, D, &a.k_b, &a.k_h)) != SQUAD_OK) return s;
  if ((s = encode_rows(&maps.v, dev, c.v, d->v, B, hk, d->m, D, &a.v_b, &a.v_h)) != SQUAD_OK) return s;
  if ((s = encode_rows(&maps.dout, dev, c.dout, d->dout, B, h, d->n, D, &a.do_b, &a.do_h)) != SQUAD_OK) return s;
  a.mask = c.mask;
  a.scale = c.scale;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  a.o = static_cast<const __nv_bfloat16*>(c.o_in);
  a.dout = static_cast<const __nv_bfloat16*>(c.dout);
  a.so = c.so;
  a.sdo = c.sdo;
  a.sdq = c.sdq;
  a.sdk = c.sdk;
  a.sdv = c.sdv;
  a.lse = c.lse;
  a.Drow = c.Drow;
  a.dq = static_cast<__nv_bfloat16*>(c.dq);
  a.dk = static_cast<__nv_bfloat16*>(c.dk);
  a.dv = static_cast<__nv_bfloat16*>(c.dv);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.part);
  a.dq_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.dq_part);
  a.err = dev.err;
  const bool masked = c.mask.lens != nullptr || c.mask.keys != nullptr;
  if (D == 128)
    return masked ? launch_cross_bwd<128, true>(dev, maps, a, st) : launch_cross_bwd<128, false>(dev, maps, a, st);
  return masked ? launch_cross_bwd<64, true>(dev, maps, a, st) : launch_cross_bwd<64, false>(dev, maps, a, st);
}

}  // namespace

extern "C" {

squad_status squad_cross_workspace_size(const squad_cross_desc* desc, int which, size_t* bytes) {
  if (bytes == nullptr) return SQUAD_ERR_INVALID_ARG;
  squad_status s = check_cross(desc);
  if (s != SQUAD_OK) return s;
  if (which == 0)
    *bytes = fwd_workspace(desc).total;
  else if (which == 1)
    *bytes = bwd_workspace(desc).total;
  else
    return SQUAD_ERR_INVALID_ARG;
  return SQUAD_OK;
}

squad_status squad_cross_fwd(const squad_cross_desc* desc, const void* q, const void* k, const void* v,
                             const int* kv_lens, const unsigned char* key_mask, void* o, float* lse,
                             void* workspace, size_t workspace_bytes, void* stream) {
  squad_status s = check_cross(desc);
  if (s != SQUAD_OK) return s;
  const FwdWs w = fwd_workspace(desc);
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr) return SQUAD_ERR_INVALID_ARG;
  if (key_mask != nullptr && desc->mask_stride != 0 && desc->mask_stride < desc->m) return SQUAD_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, static_cast<const void*>(o), static_cast<const void*>(lse),
                        static_cast<const void*>(workspace)})
    if (!aligned16(p)) return SQUAD_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(kv_lens) & 3u) return SQUAD_ERR_ALIGN;
  if ((s = check_cross_strides(desc, false)) != SQUAD_OK) return s;
  if (w.total > 0 && (workspace == nullptr || workspace_bytes < w.total)) return SQUAD_ERR_WORKSPACE;
  if (o == q || o == k || o == v) return SQUAD_ERR_INVALID_ARG;
  sq::HostDevice dev;
  if ((s = sq::host_device(&dev)) != SQUAD_OK) return s;
  sq::CrossArgs a = cross_args(desc, q, k, v, kv_lens, key_mask);
  a.o = o;
  a.lse = lse;
  a.splits = w.splits;
  a.part = static_cast<float*>(workspace);
  a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.part_lse);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return desc->dtype == SQUAD_BF16 ? tc_cross_fwd(dev, desc, a, st) : f32_cross<kF32Fwd>(dev, f32_rows(desc), a, st);
}

squad_status squad_cross_bwd(const squad_cross_desc* desc, const void* q, const void* k, const void* v,
                             const int* kv_lens, const unsigned char* key_mask, const void* o, const float* lse,
                             const void* dout, void* dq, void* dk, void* dv, void* workspace,
                             size_t workspace_bytes, void* stream) {
  squad_status s = check_cross(desc);
  if (s != SQUAD_OK) return s;
  const BwdWs w = bwd_workspace(desc);
  for (const void* p : {q, k, v, o, static_cast<const void*>(lse), dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv)}) {
    if (p == nullptr) return SQUAD_ERR_INVALID_ARG;
    if (!aligned16(p)) return SQUAD_ERR_ALIGN;
  }
  if (key_mask != nullptr && desc->mask_stride != 0 && desc->mask_stride < desc->m) return SQUAD_ERR_INVALID_ARG;
  if (!aligned16(workspace) || (reinterpret_cast<uintptr_t>(kv_lens) & 3u)) return SQUAD_ERR_ALIGN;
  if ((s = check_cross_strides(desc, true)) != SQUAD_OK) return s;
  if (workspace == nullptr || workspace_bytes < w.total) return SQUAD_ERR_WORKSPACE;
  for (const void* out : {dq, dk, dv})
    for (const void* in : {q, k, v, o, dout})
      if (out == in) return SQUAD_ERR_INVALID_ARG;
  if (dq == dk || dq == dv || dk == dv) return SQUAD_ERR_INVALID_ARG;
  sq::HostDevice dev;
  if ((s = sq::host_device(&dev)) != SQUAD_OK) return s;
  sq::CrossArgs a = cross_args(desc, q, k, v, kv_lens, key_mask);
  a.o_in = o;
  a.lse = const_cast<float*>(lse);
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.Drow = static_cast<float*>(workspace);
  a.splits = w.splits;
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.part);
  a.dq_splits = w.dq_splits;
  a.dq_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.dq_part);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (desc->dtype == SQUAD_BF16) return tc_cross_bwd(dev, desc, a, w, workspace, st);
  if ((s = f32_cross<kF32Dq>(dev, f32_rows(desc), a, st)) != SQUAD_OK) return s;
  return f32_cross<kF32Dkdv>(dev, w.f32_key_rows, a, st);
}

// ---------------------------------------------------------------- rotary positions

squad_status squad_rotary(const squad_rotary_desc* desc, int ntensors, const int* heads, const void* const* x,
                          const squad_strides* xs, void* const* y, const squad_strides* ys, const float* table,
                          void* stream) {
  if (desc == nullptr || heads == nullptr || x == nullptr || xs == nullptr || y == nullptr || ys == nullptr ||
      ntensors < 1 || ntensors > 2)
    return SQUAD_ERR_INVALID_ARG;
  const squad_rotary_desc& d = *desc;
  if (d.dtype != SQUAD_F32 && d.dtype != SQUAD_BF16) return SQUAD_ERR_INVALID_ARG;
  if (d.pairing != SQUAD_ROTARY_ADJACENT && d.pairing != SQUAD_ROTARY_HALF) return SQUAD_ERR_INVALID_ARG;
  if (d.B <= 0 || d.d <= 0 || d.T <= 0 || d.H <= 0 || d.W <= 0) return SQUAD_ERR_SHAPE;
  if (d.cT < 0 || d.cH < 0 || d.cW < 0 || (d.cT | d.cH | d.cW) % 2) return SQUAD_ERR_SHAPE;
  if ((long long)d.cT + d.cH + d.cW > d.d) return SQUAD_ERR_SHAPE;
  const size_t e = elem_size(d.dtype);
  const int per = int(16 / e);  // channels of a 16-byte chunk
  const int r = d.cT + d.cH + d.cW;
  const bool half = d.pairing == SQUAD_ROTARY_HALF;
  if (d.d % per || d.d > 1024 || (half && (r % (2 * per) || (d.d - r) % (2 * per)))) return SQUAD_ERR_UNSUPPORTED;
  const long long n = (long long)d.T * d.H * d.W;
  if (n >= kMaxRows) return SQUAD_ERR_SHAPE;
  if (d.B > kMaxGridYZ) return SQUAD_ERR_UNSUPPORTED;
  const long long entries[3] = {(long long)d.T * (d.cT / 2), (long long)d.H * (d.cH / 2), (long long)d.W * (d.cW / 2)};
  if (entries[0] + entries[1] + entries[2] >= kMaxRows) return SQUAD_ERR_SHAPE;
  if (table == nullptr && r > 0) return SQUAD_ERR_INVALID_ARG;
  sq::RotaryArgs a{};
  long long total = 0;
  for (int i = 0; i < ntensors; ++i) {
    if (heads[i] <= 0) return SQUAD_ERR_SHAPE;
    if (x[i] == nullptr || y[i] == nullptr) return SQUAD_ERR_INVALID_ARG;
    if (!aligned16(x[i]) || !aligned16(y[i])) return SQUAD_ERR_ALIGN;
    if (!stride_ok(xs[i], d.B, heads[i], int(n), d.d, e, true) || !stride_ok(ys[i], d.B, heads[i], int(n), d.d, e, false))
      return SQUAD_ERR_ALIGN;
    total += heads[i];
    const long long es = (long long)e;
    a.t[i] = {static_cast<const uint8_t*>(x[i]), static_cast<uint8_t*>(y[i]), xs[i].b * es, xs[i].h * es,
              xs[i].n * es, ys[i].b * es, ys[i].h * es, ys[i].n * es, heads[i]};
  }
  if (reinterpret_cast<uintptr_t>(table) & 7u) return SQUAD_ERR_ALIGN;
  // an output may be its own input, row for row, and no other tensor
  for (int i = 0; i < ntensors; ++i)
    for (int j = 0; j < ntensors; ++j) {
      if (i != j && (y[i] == y[j] || y[i] == x[j])) return SQUAD_ERR_INVALID_ARG;
      if (i == j && y[i] == x[i] && !same_rows(xs[i], ys[i], d.B, heads[i], int(n))) return SQUAD_ERR_INVALID_ARG;
    }
  const long long groups = (total + sq::kRotaryHeads - 1) / sq::kRotaryHeads;
  if (groups > kMaxGridYZ) return SQUAD_ERR_UNSUPPORTED;
  a.table = reinterpret_cast<const float2*>(table);
  a.n = int(n);
  a.W = d.W;
  a.H = d.H;
  a.pT = d.cT / 2;
  a.pH = d.cH / 2;
  a.pW = d.cW / 2;
  a.offH = int(entries[0]);
  a.offW = int(entries[0] + entries[1]);
  a.lanes = d.d / (half ? 2 * per : per);
  a.rows = sq::kRotaryThreads / a.lanes;
  a.f_lanes = sq::make_fastdiv(uint32_t(a.lanes));
  a.f_w = sq::make_fastdiv(uint32_t(d.W));
  a.f_h = sq::make_fastdiv(uint32_t(d.H));
  a.sign = d.inverse ? -1.f : 1.f;
  sq::HostDevice dev;
  squad_status s = sq::host_device(&dev);
  if (s != SQUAD_OK) return s;
  const dim3 grid(unsigned((n + a.rows - 1) / a.rows), unsigned(groups), unsigned(d.B));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d.dtype == SQUAD_BF16) {
    if (half)
      sq::rotary_kernel<__nv_bfloat16, true><<<grid, sq::kRotaryThreads, 0, st>>>(a);
    else
      sq::rotary_kernel<__nv_bfloat16, false><<<grid, sq::kRotaryThreads, 0, st>>>(a);
  } else {
    if (half)
      sq::rotary_kernel<float, true><<<grid, sq::kRotaryThreads, 0, st>>>(a);
    else
      sq::rotary_kernel<float, false><<<grid, sq::kRotaryThreads, 0, st>>>(a);
  }
  SQ_CUDA(cudaGetLastError());
  return SQUAD_OK;
}

}  // extern "C"
