// cross_f32.cuh - cross attention in fp32 on the CUDA cores (see squad_cross_fwd).
//
// For P_ij = exp(s <q_i,k_j> - lse_i) over the keys j that count, dP_ij = <dO_i, v_j>,
// D_i = <dO_i, O_i> and dS_ij = P_ij (dP_ij - D_i):
//   o_i = sum_j P_ij v_j,  dq_i = s sum_j dS_ij k_j,  dk_j = s sum_i dS_ij q_i,  dv_j = sum_i P_ij dO_i.
// Tiles of 16 R rows (queries; keys in the dk, dv kernel) against 64 of the other side live in
// shared memory, rows padded by 16 bytes so that the 16-byte loads of eight lanes fall into
// different banks. 256 threads as 16 x 16: thread (y, x) computes the scores of rows y + 16 i
// (i < R) and columns x + 16 j, and accumulates its rows of the results in 4-channel groups
// x + 16 c. Shared-memory loads bound it (a 16-byte load of a warp takes four passes, shared
// addresses or not): (R + 4) of them for 16 R FMAs. A larger R saves loads, a smaller one gives
// more blocks; forward + backward at 4,096 x 1,024, 8 heads of 128: 5.47 ms with R = 1, 3.28 with 2,
// 2.59 with 4 (28 TFLOP/s forward); at 1,000 x 130, 4 heads of 96: 124 us with 1, 134 with 2.
// Keys that do not count are zero-filled instead of read.
#pragma once
#include <cstdint>
#include "cross_args.h"
#include "geometry.h"

namespace sq {

constexpr int kF32Threads = 256, kF32Cols = 64, kF32P = kF32Cols + 4;

template <int D, int R = 1>
struct F32Layout {
  static constexpr int LD = D + 4;                 // floats between rows of a tile
  static constexpr int NC = (D / 4 + 15) / 16;     // 4-channel groups of a thread
  static constexpr int NR = 16 * R;                // rows of a tile
  static constexpr int ROWS = NR * LD, COLS = kF32Cols * LD, P = NR * kF32P;
  static constexpr int FWD = (ROWS + 2 * COLS + P + kF32Cols) * 4;
  static constexpr int DQ = (2 * ROWS + 2 * COLS + P + kF32Cols) * 4;
  static constexpr int DKV = (2 * ROWS + 2 * COLS + 2 * P + 2 * kF32Cols) * 4;
};

// n rows of D floats (row stride in elements) into a padded tile, by asynchronous copies (every
// load of a tile is in flight at once; a thread that loads and stores by turns waits for each).
// Rows from `valid` on, and rows whose keep entry is 0 (keep may be null), are zero.
template <int D>
__device__ __forceinline__ void f32_load(float* tile, const float* src, long long stride, int n, int valid,
                                         const float* keep) {
  const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(tile));
  for (int i = threadIdx.x; i < n * (D / 4); i += kF32Threads) {
    const int r = i / (D / 4), c = i - r * (D / 4);
    const bool live = r < valid && (keep == nullptr || keep[r] != 0.f);
    // a copy of 0 bytes reads nothing and fills the 16 with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (r * F32Layout<D>::LD + 4 * c) * 4),
                 "l"(live ? src + r * stride + 4 * c : src), "r"(live ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void f32_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for every copy of this thread: none is in flight when a block ends.
__device__ __forceinline__ void f32_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Waits until at most N of this thread's last groups are in flight.
template <int N>
__device__ __forceinline__ void f32_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// s[a][j] += <rows y + 16 a, cols x + 16 j>
template <int D, int R>
__device__ __forceinline__ void f32_dots(const float* rows, const float* cols, int y, int x, float (&s)[R][4]) {
  constexpr int LD = F32Layout<D>::LD;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 a[R], b[4];
#pragma unroll
    for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(rows + (y + 16 * i) * LD + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(cols + (x + 16 * j) * LD + c);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
  }
}

// acc[a][g] += sum_j p[y + 16 a][j] cols[j][channels 4 (x + 16 g) ..]
template <int D, int R>
__device__ __forceinline__ void f32_accumulate(const float* p, const float* cols, int y, int x,
                                               float4 (&acc)[R][F32Layout<D>::NC]) {
  constexpr int LD = F32Layout<D>::LD, NC = F32Layout<D>::NC;
#pragma unroll 2
  for (int j = 0; j < kF32Cols; j += 4) {
    float w[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(p + (y + 16 * i) * kF32P + j);
      w[i][0] = t.x;
      w[i][1] = t.y;
      w[i][2] = t.z;
      w[i][3] = t.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int g = 0; g < NC; ++g) {
        if (D % 64 != 0 && x + 16 * g >= D / 4) continue;
        const float4 v = *reinterpret_cast<const float4*>(cols + (j + e) * LD + 4 * (x + 16 * g));
#pragma unroll
        for (int i = 0; i < R; ++i) {
          acc[i][g].x = fmaf(w[i][e], v.x, acc[i][g].x);
          acc[i][g].y = fmaf(w[i][e], v.y, acc[i][g].y);
          acc[i][g].z = fmaf(w[i][e], v.z, acc[i][g].z);
          acc[i][g].w = fmaf(w[i][e], v.w, acc[i][g].w);
        }
      }
  }
}

// Sum over the 16 threads of a row.
__device__ __forceinline__ float f32_row_sum(float v) {
#pragma unroll
  for (int k = 8; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  return v;
}

// 1 in keep[j] where key j0 + j counts, else 0.
__device__ __forceinline__ void f32_keep(float* keep, int n, const CrossMask& mk, int b, int j0, int len) {
  if (int(threadIdx.x) < n)
    keep[threadIdx.x] = j0 + int(threadIdx.x) < len && cross_keeps(mk, b, j0 + threadIdx.x) ? 1.f : 0.f;
}

// With a.splits > 1 the keys of a query tile are cut into parts (blockIdx.x = query tile * splits +
// part), whose results and log-sums (base 2) go to a.part and a.part_lse, [part][B, heads, n].
template <int D, int R>
__global__ void __launch_bounds__(kF32Threads) cross_f32_fwd_kernel(const __grid_constant__ CrossArgs a) {
  using Lay = F32Layout<D, R>;
  extern __shared__ __align__(16) float f32_smem[];
  float *qs = f32_smem, *ks = qs + Lay::ROWS, *vs = ks + Lay::COLS, *ps = vs + Lay::COLS, *keep = ps + Lay::P;
  const int qt = blockIdx.x / a.splits, sp = blockIdx.x - qt * a.splits;
  const int b = blockIdx.z, h = blockIdx.y, hk = h / a.group, i0 = qt * Lay::NR;
  const int y = threadIdx.x >> 4, x = threadIdx.x & 15, len = cross_len(a.mask, b, a.m);
  // this part's keys: whole tiles of them
  const int tiles = (len + kF32Cols - 1) / kF32Cols, per = (tiles + a.splits - 1) / a.splits * kF32Cols;
  const int k0 = sp * per, k1 = k0 + per < len ? k0 + per : len;
  f32_load<D>(qs, cross_row<float>(a.q, a.sq, b, h, i0), a.sq.n, Lay::NR, a.n - i0, nullptr);
  float4 acc[R][Lay::NC] = {};
  float mx[R], l[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    mx[i] = -INFINITY;
    l[i] = 0.f;
  }
  for (int j0 = k0; j0 < k1; j0 += kF32Cols) {
    __syncthreads();  // the last tile's values are done with
    f32_keep(keep, kF32Cols, a.mask, b, j0, len);
    __syncthreads();
    f32_load<D>(ks, cross_row<float>(a.k, a.sk, b, hk, j0), a.sk.n, kF32Cols, a.m - j0, keep);
    f32_commit();
    f32_load<D>(vs, cross_row<float>(a.v, a.sv, b, hk, j0), a.sv.n, kF32Cols, a.m - j0, keep);
    f32_commit();
    f32_wait<1>();  // the keys (and the queries) are there, the values may still come
    __syncthreads();
    float s[R][4] = {};
    f32_dots<D, R>(qs, ks, y, x, s);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = keep[x + 16 * j] != 0.f ? s[i][j] * a.scale : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float m_new = fmaxf(mx[i], top), ref = m_new == -INFINITY ? 0.f : m_new;
      const float corr = expf(mx[i] - ref);  // 0 before the first key
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = expf(s[i][j] - ref);
        ps[(y + 16 * i) * kF32P + x + 16 * j] = p;
        sum += p;
      }
      l[i] = l[i] * corr + f32_row_sum(sum);
      mx[i] = m_new;
#pragma unroll
      for (int g = 0; g < Lay::NC; ++g) {
        acc[i][g].x *= corr;
        acc[i][g].y *= corr;
        acc[i][g].z *= corr;
        acc[i][g].w *= corr;
      }
    }
    f32_wait<0>();
    __syncthreads();
    f32_accumulate<D, R>(ps, vs, y, x, acc);
  }
  f32_wait_all();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = i0 + y + 16 * i;
    if (r >= a.n) continue;
    const float inv = l[i] > 0.f ? 1.f / l[i] : l[i];
    const long long row = ((long long)b * a.heads + h) * a.n + r, part_row = (long long)sp * a.B * a.heads * a.n + row;
    float* out = a.splits > 1 ? a.part + part_row * D : cross_row<float>(a.o, a.so, b, h, r);
#pragma unroll
    for (int g = 0; g < Lay::NC; ++g) {
      if (D % 64 != 0 && x + 16 * g >= D / 4) continue;
      *reinterpret_cast<float4*>(out + 4 * (x + 16 * g)) =
          make_float4(acc[i][g].x * inv, acc[i][g].y * inv, acc[i][g].z * inv, acc[i][g].w * inv);
    }
    const float lse = l[i] == 0.f ? -INFINITY : mx[i] + logf(l[i]);
    if (x == 0) {
      if (a.splits > 1)
        a.part_lse[part_row] = lse * 1.4426950408889634f;
      else if (a.lse != nullptr)
        a.lse[row] = lse;
    }
  }
}

template <int D, int R>
__global__ void __launch_bounds__(kF32Threads) cross_f32_dq_kernel(const __grid_constant__ CrossArgs a) {
  using Lay = F32Layout<D, R>;
  extern __shared__ __align__(16) float f32_smem[];
  float *qs = f32_smem, *dos = qs + Lay::ROWS, *ks = dos + Lay::ROWS, *vs = ks + Lay::COLS, *ps = vs + Lay::COLS,
        *keep = ps + Lay::P;
  const int b = blockIdx.z, h = blockIdx.y, hk = h / a.group, i0 = blockIdx.x * Lay::NR;
  const int y = threadIdx.x >> 4, x = threadIdx.x & 15, len = cross_len(a.mask, b, a.m);
  f32_load<D>(qs, cross_row<float>(a.q, a.sq, b, h, i0), a.sq.n, Lay::NR, a.n - i0, nullptr);
  f32_load<D>(dos, cross_row<float>(a.dout, a.sdo, b, h, i0), a.sdo.n, Lay::NR, a.n - i0, nullptr);
  f32_commit();
  f32_wait<0>();
  __syncthreads();
  float dd[R], lse[R];
  const long long base = ((long long)b * a.heads + h) * a.n;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = i0 + y + 16 * i;
    float t = 0.f;
    lse[i] = INFINITY;  // rows past the last, and rows without keys: P = 0
    if (r < a.n) {
      const float* o = cross_row<float>(a.o_in, a.so, b, h, r);
      for (int c = x; c < D; c += 16) t = fmaf(dos[(y + 16 * i) * Lay::LD + c], o[c], t);
      const float v = a.lse[base + r];
      lse[i] = v == -INFINITY ? INFINITY : v;
    }
    dd[i] = f32_row_sum(t);
    if (r < a.n && x == 0) a.Drow[base + r] = dd[i];
  }
  float4 acc[R][Lay::NC] = {};
  for (int j0 = 0; j0 < len; j0 += kF32Cols) {
    __syncthreads();
    f32_keep(keep, kF32Cols, a.mask, b, j0, len);
    __syncthreads();
    f32_load<D>(ks, cross_row<float>(a.k, a.sk, b, hk, j0), a.sk.n, kF32Cols, a.m - j0, keep);
    f32_load<D>(vs, cross_row<float>(a.v, a.sv, b, hk, j0), a.sv.n, kF32Cols, a.m - j0, keep);
    f32_commit();
    f32_wait<0>();
    __syncthreads();
    float s[R][4] = {}, dp[R][4] = {};
    f32_dots<D, R>(qs, ks, y, x, s);
    f32_dots<D, R>(dos, vs, y, x, dp);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = keep[x + 16 * j] != 0.f ? expf(s[i][j] * a.scale - lse[i]) : 0.f;
        ps[(y + 16 * i) * kF32P + x + 16 * j] = p * (dp[i][j] - dd[i]);
      }
    __syncthreads();
    f32_accumulate<D, R>(ps, ks, y, x, acc);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = i0 + y + 16 * i;
    if (r >= a.n) continue;
    float* out = cross_row<float>(a.dq, a.sdq, b, h, r);
#pragma unroll
    for (int g = 0; g < Lay::NC; ++g) {
      if (D % 64 != 0 && x + 16 * g >= D / 4) continue;
      *reinterpret_cast<float4*>(out + 4 * (x + 16 * g)) = make_float4(
          acc[i][g].x * a.scale, acc[i][g].y * a.scale, acc[i][g].z * a.scale, acc[i][g].w * a.scale);
    }
  }
}

// A block: 16 R keys and one part of the queries of their head group (blockIdx.x = key tile *
// splits + part); with splits > 1 the parts go to a.part, [dk, dv][split][B, kv_heads, m][D].
template <int D, int R>
__global__ void __launch_bounds__(kF32Threads) cross_f32_dkdv_kernel(const __grid_constant__ CrossArgs a) {
  using Lay = F32Layout<D, R>;
  extern __shared__ __align__(16) float f32_smem[];
  float *ks = f32_smem, *vs = ks + Lay::ROWS, *qs = vs + Lay::ROWS, *dos = qs + Lay::COLS, *ps = dos + Lay::COLS,
        *dss = ps + Lay::P, *lse = dss + Lay::P, *dd = lse + kF32Cols;
  __shared__ float keep[Lay::NR];
  const int b = blockIdx.z, hk = blockIdx.y, kt = blockIdx.x / a.splits, sp = blockIdx.x - kt * a.splits;
  const int j0 = kt * Lay::NR, y = threadIdx.x >> 4, x = threadIdx.x & 15, len = cross_len(a.mask, b, a.m);
  f32_keep(keep, Lay::NR, a.mask, b, j0, len);
  __syncthreads();
  float4 dk[R][Lay::NC] = {}, dv[R][Lay::NC] = {};
  if (j0 < len) {
    f32_load<D>(ks, cross_row<float>(a.k, a.sk, b, hk, j0), a.sk.n, Lay::NR, a.m - j0, keep);
    f32_load<D>(vs, cross_row<float>(a.v, a.sv, b, hk, j0), a.sv.n, Lay::NR, a.m - j0, keep);
    const int qtiles = (a.n + kF32Cols - 1) / kF32Cols, tiles = a.group * qtiles;
    const int per = (tiles + a.splits - 1) / a.splits;
    const int t1 = (sp + 1) * per < tiles ? (sp + 1) * per : tiles;
    for (int t = sp * per; t < t1; ++t) {
      const int g = t / qtiles, h = hk * a.group + g, i0 = (t - g * qtiles) * kF32Cols;
      __syncthreads();
      if (threadIdx.x < kF32Cols) {
        const int r = i0 + threadIdx.x;
        const long long row = ((long long)b * a.heads + h) * a.n + r;
        const float v = r < a.n ? a.lse[row] : INFINITY;
        lse[threadIdx.x] = v == -INFINITY ? INFINITY : v;
        dd[threadIdx.x] = r < a.n ? a.Drow[row] : 0.f;
      }
      f32_load<D>(qs, cross_row<float>(a.q, a.sq, b, h, i0), a.sq.n, kF32Cols, a.n - i0, nullptr);
      f32_load<D>(dos, cross_row<float>(a.dout, a.sdo, b, h, i0), a.sdo.n, kF32Cols, a.n - i0, nullptr);
      f32_commit();
      f32_wait<0>();  // the keys' tiles too, at the first turn
      __syncthreads();
      float s[R][4] = {}, dp[R][4] = {};
      f32_dots<D, R>(ks, qs, y, x, s);
      f32_dots<D, R>(vs, dos, y, x, dp);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = x + 16 * j;
          const float p = keep[y + 16 * i] != 0.f ? expf(s[i][j] * a.scale - lse[c]) : 0.f;
          ps[(y + 16 * i) * kF32P + c] = p;
          dss[(y + 16 * i) * kF32P + c] = p * (dp[i][j] - dd[c]);
        }
      __syncthreads();
      f32_accumulate<D, R>(ps, dos, y, x, dv);
      f32_accumulate<D, R>(dss, qs, y, x, dk);
    }
  }
  f32_wait_all();
  const long long rows = (long long)a.B * a.kv_heads * a.m;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int j = j0 + y + 16 * i;
    if (j >= a.m) continue;
    const long long row = ((long long)b * a.kv_heads + hk) * a.m + j;
    float* ok = a.splits > 1 ? a.part + (sp * rows + row) * D : cross_row<float>(a.dk, a.sdk, b, hk, j);
    float* ov = a.splits > 1 ? a.part + ((a.splits + sp) * rows + row) * D : cross_row<float>(a.dv, a.sdv, b, hk, j);
#pragma unroll
    for (int g = 0; g < Lay::NC; ++g) {
      if (D % 64 != 0 && x + 16 * g >= D / 4) continue;
      const int c = 4 * (x + 16 * g);
      *reinterpret_cast<float4*>(ok + c) =
          make_float4(dk[i][g].x * a.scale, dk[i][g].y * a.scale, dk[i][g].z * a.scale, dk[i][g].w * a.scale);
      *reinterpret_cast<float4*>(ov + c) = dv[i][g];
    }
  }
}

}  // namespace sq
