// rotary.cuh - rotary positions of the latent grid (squad_rotary).
//
// A token at (t, y, x) has the angles of its axes in the table, one per channel pair; the
// pair (a, b) becomes (a cos - b sin, a sin + b cos), and with the sign of sin changed the
// same kernel turns gradients back. One pass over the data: 2 bytes moved per byte of input
// and 3 flops per element, so it is bound by HBM. The (cos, sin) of a thread's pairs depend
// on the token alone: a thread reads them once (the table is tens of KB and stays in L1/L2)
// and applies them to kRotaryHeads heads, whose 16-byte loads are all in flight at once.
// Measured: q and k of 27,280 tokens, 24 heads of 128 in bf16, token-major in, 108 us: 6.2 TB/s, 94%
// of a plain copy's rate.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "geometry.h"

namespace sq {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryHeads = 8;  // heads per thread

struct RotaryTensor {
  const uint8_t* x;
  uint8_t* y;
  long long xb, xh, xn, yb, yh, yn;  // bytes
  int heads;
};

struct RotaryArgs {
  RotaryTensor t[2];   // the second has no heads when one tensor is given
  const float2* table;
  int n, W, H;
  int pT, pH, pW;      // pairs per axis
  int offH, offW;      // first table entry of the y and x axes
  int lanes;           // threads per row
  int rows;            // rows per block
  FastDiv f_lanes, f_w, f_h;
  float sign;          // 1, or -1 to turn by the opposite angles
};

__device__ __forceinline__ uint4 ld_stream_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// 16 bytes as floats and back.
template <typename T>
struct Chunk;
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// The first `words` words of `done`, the others of `from`: channels past the axes' keep their bits (a product with
// cos 1 and sin 0 would turn the neighbour of an infinity into NaN).
__device__ __forceinline__ uint4 turned_words(int words, const uint4& done, const uint4& from) {
  return make_uint4(words > 0 ? done.x : from.x, words > 1 ? done.y : from.y, words > 2 ? done.z : from.z,
                    words > 3 ? done.w : from.w);
}

// HALF: a thread holds the chunks at channels ca and cb of a row, element e of each being
// one pair; else it holds one chunk with pairs inside it.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int N = Chunk<T>::N;
  constexpr int NP = HALF ? N : N / 2;  // pairs of a thread
  const int r = fdiv(int(threadIdx.x), a.f_lanes), lane = int(threadIdx.x) - r * a.lanes;
  const long long row = (long long)blockIdx.x * a.rows + r;
  if (r >= a.rows || row >= a.n) return;
  const int tok = int(row), b = blockIdx.z;
  const int ty = fdiv(tok, a.f_w), x = tok - ty * a.W, t = fdiv(ty, a.f_h), y = ty - t * a.H;
  const int turned = a.pT + a.pH + a.pW;
  float c[NP], s[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int p = lane * NP + i;
    float2 cs = make_float2(1.f, 0.f);
    if (p < a.pT)
      cs = __ldg(a.table + (long long)t * a.pT + p);
    else if (p < a.pT + a.pH)
      cs = __ldg(a.table + a.offH + (long long)y * a.pH + (p - a.pT));
    else if (p < turned)
      cs = __ldg(a.table + a.offW + (long long)x * a.pW + (p - a.pT - a.pH));
    c[i] = cs.x;
    s[i] = cs.y * a.sign;
  }
  // words of a chunk that are turned (HALF: all or none)
  const int words = HALF ? (lane * N < turned ? 4 : 0) : (turned - lane * NP) * (4 / NP);
  int ca = lane * N, cb = 0;
  if (HALF) {
    if (lane * N < turned) {
      cb = ca + turned;
    } else {  // copied channels, two chunks per thread
      ca = 2 * lane * N;
      cb = ca + N;
    }
  }
  constexpr int ES = int(sizeof(T));
  const int total = a.t[0].heads + a.t[1].heads;
  const int h0 = blockIdx.y * kRotaryHeads;
  const uint8_t* src[kRotaryHeads];
  uint4 va[kRotaryHeads], vb[HALF ? kRotaryHeads : 1];
#pragma unroll
  for (int i = 0; i < kRotaryHeads; ++i) {
    const int hh = h0 + i;
    if (hh >= total) break;
    const bool second = hh >= a.t[0].heads;
    const RotaryTensor& q = second ? a.t[1] : a.t[0];
    src[i] = q.x + b * q.xb + (long long)(second ? hh - a.t[0].heads : hh) * q.xh + tok * q.xn;
    va[i] = ld_stream_v4(src[i] + ca * ES);
    if (HALF) vb[i] = ld_stream_v4(src[i] + cb * ES);
  }
#pragma unroll
  for (int i = 0; i < kRotaryHeads; ++i) {
    const int hh = h0 + i;
    if (hh >= total) break;
    const bool second = hh >= a.t[0].heads;
    const RotaryTensor& q = second ? a.t[1] : a.t[0];
    uint8_t* dst = q.y + b * q.yb + (long long)(second ? hh - a.t[0].heads : hh) * q.yh + tok * q.yn;
    float u[N];
    Chunk<T>::load(va[i], u);
    if (HALF) {
      float w[N];
      Chunk<T>::load(vb[i], w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float p = fmaf(u[e], c[e], -(w[e] * s[e])), z = fmaf(u[e], s[e], w[e] * c[e]);
        u[e] = p;
        w[e] = z;
      }
      *reinterpret_cast<uint4*>(dst + ca * ES) = turned_words(words, Chunk<T>::store(u), va[i]);
      *reinterpret_cast<uint4*>(dst + cb * ES) = turned_words(words, Chunk<T>::store(w), vb[i]);
    } else {
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        const float p = fmaf(u[2 * e], c[e], -(u[2 * e + 1] * s[e]));
        u[2 * e + 1] = fmaf(u[2 * e], s[e], u[2 * e + 1] * c[e]);
        u[2 * e] = p;
      }
      *reinterpret_cast<uint4*>(dst + ca * ES) = turned_words(words, Chunk<T>::store(u), va[i]);
    }
  }
}

}  // namespace sq
