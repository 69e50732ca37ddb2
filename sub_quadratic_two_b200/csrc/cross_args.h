// cross_args.h - tensors and masks of a cross-attention call, as the kernels take them.
#pragma once
#include <cstdint>

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
  // fp32: parts of the keys in the forward, of the queries in the dk, dv kernel; their results
  // where there are several
  int splits;
  float *part, *part_lse;
  // dq kernel: parts of the keys, and their results where there are several
  int dq_splits;
  float* dq_part;
};

template <typename T>
__device__ __forceinline__ const T* cross_row(const void* base, const CrossStride& s, int b, int h, int i) {
  return static_cast<const T*>(base) + b * s.b + h * s.h + i * s.n;
}
template <typename T>
__device__ __forceinline__ T* cross_row(void* base, const CrossStride& s, int b, int h, int i) {
  return static_cast<T*>(base) + b * s.b + h * s.h + i * s.n;
}

}  // namespace sq
