// cross_simt.cuh - cross attention on the CUDA cores (see squad_cross_fwd).
//
// For P_ij = exp(s <q_i,k_j> - lse_i) over the keys j that count, dP_ij = <dO_i, v_j>,
// D_i = <dO_i, O_i> and dS_ij = P_ij (dP_ij - D_i):
//   o_i = sum_j P_ij v_j,  dq_i = s sum_j dS_ij k_j,  dk_j = s sum_i dS_ij q_i,  dv_j = sum_i P_ij dO_i.
// One warp owns a query row (forward, dq) or a key row (dk, dv); its lanes split the head
// dimension. Masked keys are skipped before they are read.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "geometry.h"
#include "squad_simt.cuh"

namespace sq {

struct CrossStride {
  long long b, h, n;  // elements
};

struct CrossMask {
  const int* lens;             // [B] or nullptr
  const unsigned char* keys;   // one byte per key or nullptr
  long long stride;            // bytes between batch rows of keys
};

// Keys of batch row b below this bound may count.
__device__ __forceinline__ int cross_len(const CrossMask& mk, int b, int m) {
  if (mk.lens == nullptr) return m;
  const int l = __ldg(mk.lens + b);
  return l < 0 ? 0 : l > m ? m : l;
}
__device__ __forceinline__ bool cross_keeps(const CrossMask& mk, int b, int j) {
  return mk.keys == nullptr || __ldg(mk.keys + b * mk.stride + j) != 0;
}

struct CrossArgs {
  int B, heads, kv_heads, group, n, m, d;
  float scale;
  CrossMask mask;
  CrossStride sq, sk, sv, so, sdo, sdq, sdk, sdv;
  const void *q, *k, *v, *o_in, *dout;
  void *o, *dq, *dk, *dv;
  float* lse;   // written by the forward (or nullptr), read by the backward
  float* Drow;  // [B, heads, n], written by the dq kernel for the dk, dv kernel
};

template <typename T>
__device__ __forceinline__ const T* cross_row(const void* base, const CrossStride& s, int b, int h, int i) {
  return static_cast<const T*>(base) + b * s.b + h * s.h + i * s.n;
}
template <typename T>
__device__ __forceinline__ T* cross_row(void* base, const CrossStride& s, int b, int h, int i) {
  return static_cast<T*>(base) + b * s.b + h * s.h + i * s.n;
}

template <typename T, int DPL>
__global__ void __launch_bounds__(kSimtWarps * 32) cross_simt_fwd_kernel(const __grid_constant__ CrossArgs a) {
  const int lane = threadIdx.x & 31, b = blockIdx.z, h = blockIdx.y;
  const int i = blockIdx.x * kSimtWarps + (threadIdx.x >> 5);
  if (i >= a.n) return;
  const T* qr = cross_row<T>(a.q, a.sq, b, h, i);
  float qv[DPL], acc[DPL];
#pragma unroll
  for (int e = 0; e < DPL; ++e) {
    qv[e] = ld_f(qr + lane + 32 * e);
    acc[e] = 0.f;
  }
  float mx = -INFINITY, l = 0.f;
  const int len = cross_len(a.mask, b, a.m);
  for (int j = 0; j < len; ++j) {
    if (!cross_keeps(a.mask, b, j)) continue;
    const T* kr = cross_row<T>(a.k, a.sk, b, h / a.group, j);
    const T* vr = cross_row<T>(a.v, a.sv, b, h / a.group, j);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < DPL; ++e) s = fmaf(qv[e], ld_f(kr + lane + 32 * e), s);
    s = warp_sum(s) * a.scale;
    const float m_new = fmaxf(mx, s);
    const float corr = mx == -INFINITY ? 0.f : expf(mx - m_new);
    const float p = m_new == -INFINITY ? 0.f : expf(s - m_new);
    l = l * corr + p;
#pragma unroll
    for (int e = 0; e < DPL; ++e) acc[e] = fmaf(acc[e], corr, p * ld_f(vr + lane + 32 * e));
    mx = m_new;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  T* orow = cross_row<T>(a.o, a.so, b, h, i);
#pragma unroll
  for (int e = 0; e < DPL; ++e) st_f(orow + lane + 32 * e, acc[e] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[((long long)b * a.heads + h) * a.n + i] = l > 0.f ? mx + logf(l) : -INFINITY;
}

template <typename T, int DPL>
__global__ void __launch_bounds__(kSimtWarps * 32) cross_simt_dq_kernel(const __grid_constant__ CrossArgs a) {
  const int lane = threadIdx.x & 31, b = blockIdx.z, h = blockIdx.y;
  const int i = blockIdx.x * kSimtWarps + (threadIdx.x >> 5);
  if (i >= a.n) return;
  const T* qr = cross_row<T>(a.q, a.sq, b, h, i);
  const T* dr = cross_row<T>(a.dout, a.sdo, b, h, i);
  const T* orow = cross_row<T>(a.o_in, a.so, b, h, i);
  float qv[DPL], dov[DPL], acc[DPL], D = 0.f;
#pragma unroll
  for (int e = 0; e < DPL; ++e) {
    qv[e] = ld_f(qr + lane + 32 * e);
    dov[e] = ld_f(dr + lane + 32 * e);
    D = fmaf(dov[e], ld_f(orow + lane + 32 * e), D);
    acc[e] = 0.f;
  }
  D = warp_sum(D);
  const long long row = ((long long)b * a.heads + h) * a.n + i;
  if (lane == 0) a.Drow[row] = D;
  const float lse = a.lse[row];
  const int len = cross_len(a.mask, b, a.m);
  for (int j = 0; j < len; ++j) {
    if (!cross_keeps(a.mask, b, j)) continue;
    const T* kr = cross_row<T>(a.k, a.sk, b, h / a.group, j);
    const T* vr = cross_row<T>(a.v, a.sv, b, h / a.group, j);
    float s = 0.f, dp = 0.f;
#pragma unroll
    for (int e = 0; e < DPL; ++e) {
      s = fmaf(qv[e], ld_f(kr + lane + 32 * e), s);
      dp = fmaf(dov[e], ld_f(vr + lane + 32 * e), dp);
    }
    const float p = expf(warp_sum(s) * a.scale - lse);
    const float ds = p * (warp_sum(dp) - D);
#pragma unroll
    for (int e = 0; e < DPL; ++e) acc[e] = fmaf(ds, ld_f(kr + lane + 32 * e), acc[e]);
  }
  T* out = cross_row<T>(a.dq, a.sdq, b, h, i);
#pragma unroll
  for (int e = 0; e < DPL; ++e) st_f(out + lane + 32 * e, acc[e] * a.scale);
}

template <typename T, int DPL>
__global__ void __launch_bounds__(kSimtWarps * 32) cross_simt_dkdv_kernel(const __grid_constant__ CrossArgs a) {
  const int lane = threadIdx.x & 31, b = blockIdx.z, kh = blockIdx.y;
  const int j = blockIdx.x * kSimtWarps + (threadIdx.x >> 5);
  if (j >= a.m) return;
  float kv[DPL], vv[DPL], dk[DPL], dv[DPL];
  const bool live = j < cross_len(a.mask, b, a.m) && cross_keeps(a.mask, b, j);
#pragma unroll
  for (int e = 0; e < DPL; ++e) dk[e] = dv[e] = 0.f;
  if (live) {
    const T* kr = cross_row<T>(a.k, a.sk, b, kh, j);
    const T* vr = cross_row<T>(a.v, a.sv, b, kh, j);
#pragma unroll
    for (int e = 0; e < DPL; ++e) {
      kv[e] = ld_f(kr + lane + 32 * e);
      vv[e] = ld_f(vr + lane + 32 * e);
    }
    for (int h = kh * a.group; h < (kh + 1) * a.group; ++h) {
      for (int i = 0; i < a.n; ++i) {
        const T* qr = cross_row<T>(a.q, a.sq, b, h, i);
        const T* dr = cross_row<T>(a.dout, a.sdo, b, h, i);
        const long long row = ((long long)b * a.heads + h) * a.n + i;
        float s = 0.f, dp = 0.f;
#pragma unroll
        for (int e = 0; e < DPL; ++e) {
          s = fmaf(ld_f(qr + lane + 32 * e), kv[e], s);
          dp = fmaf(ld_f(dr + lane + 32 * e), vv[e], dp);
        }
        const float p = expf(warp_sum(s) * a.scale - a.lse[row]);
        const float ds = p * (warp_sum(dp) - a.Drow[row]);
#pragma unroll
        for (int e = 0; e < DPL; ++e) {
          dk[e] = fmaf(ds, ld_f(qr + lane + 32 * e), dk[e]);
          dv[e] = fmaf(p, ld_f(dr + lane + 32 * e), dv[e]);
        }
      }
    }
  }
  T* gk = cross_row<T>(a.dk, a.sdk, b, kh, j);
  T* gv = cross_row<T>(a.dv, a.sdv, b, kh, j);
#pragma unroll
  for (int e = 0; e < DPL; ++e) {
    st_f(gk + lane + 32 * e, dk[e] * a.scale);
    st_f(gv + lane + 32 * e, dv[e]);
  }
}

}  // namespace sq
