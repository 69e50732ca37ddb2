// cross_f32.cuh - cross attention in fp32 on the CUDA cores (see squad_cross_fwd).
//
// For P_ij = exp(s <q_i,k_j> - lse_i) over the keys j that count, dP_ij = <dO_i, v_j>,
// D_i = <dO_i, O_i> and dS_ij = P_ij (dP_ij - D_i):
//   o_i = sum_j P_ij v_j,  dq_i = s sum_j dS_ij k_j,  dk_j = s sum_i dS_ij q_i,  dv_j = sum_i P_ij dO_i.
// Tiles of 16 R rows (queries; keys in the dk, dv kernel) against 64 of the other side live in
// shared memory, and shared-memory loads bound the work on them (a 16-byte load of a warp takes
// four passes, shared addresses or not), so a thread always holds 4 x 4 scores (8 loads for 64
// FMAs) or 4 rows of results: the 256 threads are 4 R groups of rows x 16 of columns (or
// channels) x S = 4 / R parts of the sum, along the channels for scores and along the 64 for
// results. The parts of a score are joined by shuffles, those of a result once at the end. (8 x 8
// scores would halve the loads for each FMA; not tried.)
// The loads of a tile are not covered by the products of the one before, but by another block's.
// Forward, 8 heads of 128, 4,096 x 1,024: 703 us with R = 1, 562 with 2 (31 TFLOP/s; the
// shared-memory passes take 0.4 ms of it); 1,000 x 130, 4 heads of 96: 23 and 23 us.
// Keys that do not count are zero-filled instead of read.
#pragma once
#include <cstdint>
#include "cross_args.h"
#include "cross_plan.h"
#include "geometry.h"

namespace sq {

constexpr int kF32Threads = 256, kF32Cols = 64;

template <int D, int R = 1>
struct F32Layout {
  static constexpr int S = 4 / R;                  // parts of a sum
  // Floats between rows of a tile, so that the eight lanes of a pass fall into different banks:
  // eight rows of one chunk (S = 1), or four rows of two chunks in the scores, and four rows of two
  // (S = 4) or two rows two apart of four chunks (S = 2) in the results.
  static constexpr int LD = D + (S == 1 ? 4 : 8);
  static constexpr int NC = (D / 4 + 15) / 16;     // 4-channel groups of a thread
  static constexpr int NR = 16 * R, RG = 4 * R;    // rows of a tile; groups of them, RG apart
  static constexpr int PG = kF32Cols / S + 4, PW = S * PG;  // scores of a part, of a row
  static constexpr int ROWS = NR * LD, COLS = kF32Cols * LD, P = NR * PW;
  static constexpr int FWD = (ROWS + 2 * COLS + P + kF32Cols + NR) * 4;
  static constexpr int DQ = (2 * ROWS + 2 * COLS + P + kF32Cols + 2 * NR) * 4;
  static constexpr int DKV = (2 * ROWS + 2 * COLS + 2 * P + 2 * kF32Cols + NR) * 4;
  // Column j of a score row lies at its part's place: a part's columns are together.
  __device__ static __forceinline__ int place(int j) {
    return S == 4 ? (j & 3) * PG + (j >> 2) : S == 2 ? ((j >> 1) & 1) * PG + (j >> 2) * 2 + (j & 1) : j;
  }
  // The u-th column of part z.
  __device__ static __forceinline__ int column(int z, int u) {
    return S == 4 ? 4 * u + z : S == 2 ? (u >> 1) * 4 + 2 * z + (u & 1) : u;
  }
};

// What a thread does in a tile: rows g + RG i (i < 4); in the scores, columns x + 16 j and part z of
// the channels (the lanes of a part and of four columns alternate); in the results, channel
// groups c + 16 k and part w of the columns.
template <int R>
struct F32Thread {
  int g, x, z, c, w;
  __device__ __forceinline__ F32Thread() {
    constexpr int S = 4 / R;
    const int t = threadIdx.x % (16 * S);
    g = threadIdx.x / (16 * S);
    z = S == 4 ? (t & 1) | ((t >> 2) & 2) : S == 2 ? t & 1 : 0;
    x = S == 4 ? ((t >> 1) & 3) | ((t >> 4) << 2) : S == 2 ? t >> 1 : t;
    c = t / S;
    w = t % S;
  }
  // rows of the joined scores (a < R) and of the joined results
  __device__ __forceinline__ int score_row(int a) const { return g + 4 * R * (z * R + a); }
  __device__ __forceinline__ int result_row(int a) const { return g + 4 * R * (w * R + a); }
};

// n rows of D floats (row stride in elements) into a padded tile, by asynchronous copies (every
// load of a tile is in flight at once; a thread that loads and stores by turns waits for each).
// Rows from `valid` on, and rows whose keep entry is 0 (keep may be null), are zero.
template <int D, int LD>
__device__ __forceinline__ void f32_load(float* tile, const float* src, long long stride, int n, int valid,
                                         const float* keep) {
  const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(tile));
  for (int i = threadIdx.x; i < n * (D / 4); i += kF32Threads) {
    const int r = i / (D / 4), c = i - r * (D / 4);
    const bool live = r < valid && (keep == nullptr || keep[r] != 0.f);
    // a copy of 0 bytes reads nothing and fills the 16 with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (r * LD + 4 * c) * 4),
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

// One half of v to the lane `mask` away, the other half of that lane's added to what stays: the upper
// half stays where `upper`.
template <int N>
__device__ __forceinline__ void f32_halve(float (&v)[2 * N], int mask, bool upper) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float give = upper ? v[i] : v[N + i], keep = upper ? v[N + i] : v[i];
    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, mask);
  }
}

// s[a][j] = <rows t.score_row(a), cols t.x + 16 j>
template <int D, int R>
__device__ __forceinline__ void f32_dots(const float* rows, const float* cols, const F32Thread<R>& t, float (&s)[R][4]) {
  using Lay = F32Layout<D, R>;
  constexpr int LD = Lay::LD, S = Lay::S;
  float p[16] = {};
  const float *ra = rows + t.g * LD + 4 * t.z, *cb = cols + t.x * LD + 4 * t.z;
#pragma unroll 4
  for (int c = 0; c < D; c += 4 * S) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(ra + i * Lay::RG * LD + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(cb + 16 * j * LD + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p[4 * i + j] =
            fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, p[4 * i + j]))));
  }
  if (S == 4) {
    f32_halve<8>(p, 8, t.z & 2);
    f32_halve<4>(reinterpret_cast<float(&)[8]>(p), 1, t.z & 1);
  } else if (S == 2) {
    f32_halve<8>(p, 1, t.z & 1);
  }
#pragma unroll
  for (int a = 0; a < R; ++a)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[a][j] = p[4 * a + j];
}

// acc[4 NC i + 4 k ..] += sum over the columns of part t.w of p[row g + RG i] cols[channels 4 (t.c + 16 k) ..]
template <int D, int R>
__device__ __forceinline__ void f32_accumulate(const float* p, const float* cols, const F32Thread<R>& t,
                                               float (&acc)[16 * F32Layout<D>::NC]) {
  using Lay = F32Layout<D, R>;
  constexpr int LD = Lay::LD, NC = Lay::NC;
  const float* pr = p + t.g * Lay::PW + t.w * Lay::PG;
#pragma unroll 2
  for (int u = 0; u < kF32Cols / Lay::S; u += 4) {
    float w[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(pr + i * Lay::RG * Lay::PW + u);
      w[i][0] = f.x;
      w[i][1] = f.y;
      w[i][2] = f.z;
      w[i][3] = f.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        if (D % 64 != 0 && t.c + 16 * k >= D / 4) continue;
        const float4 v = *reinterpret_cast<const float4*>(cols + Lay::column(t.w, u + e) * LD + 4 * (t.c + 16 * k));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* a = acc + 4 * (NC * i + k);
          a[0] = fmaf(w[i][e], v.x, a[0]);
          a[1] = fmaf(w[i][e], v.y, a[1]);
          a[2] = fmaf(w[i][e], v.z, a[2]);
          a[3] = fmaf(w[i][e], v.w, a[3]);
        }
      }
  }
}
// Joins the parts: afterwards acc[4 NC a + 4 k ..] belongs to row t.result_row(a), a < R.
template <int D, int R>
__device__ __forceinline__ void f32_join(const F32Thread<R>& t, float (&acc)[16 * F32Layout<D>::NC]) {
  constexpr int S = 4 / R, N = 4 * F32Layout<D>::NC;
  if (S == 4) {
    f32_halve<2 * N>(acc, 2, t.w & 2);
    f32_halve<N>(reinterpret_cast<float(&)[2 * N]>(acc), 1, t.w & 1);
  } else if (S == 2) {
    f32_halve<2 * N>(acc, 1, t.w & 1);
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
  constexpr int LD = Lay::LD;
  extern __shared__ __align__(16) float f32_smem[];
  float *qs = f32_smem, *ks = qs + Lay::ROWS, *vs = ks + Lay::COLS, *ps = vs + Lay::COLS, *keep = ps + Lay::P,
        *rowv = keep + kF32Cols;  // of each row: the factor of its results, at the end 1 / sum
  const int qt = blockIdx.x / a.splits, sp = blockIdx.x - qt * a.splits;
  const int b = blockIdx.z, h = blockIdx.y, hk = h / a.group, i0 = qt * Lay::NR;
  const int y = threadIdx.x >> 4, x = threadIdx.x & 15, len = cross_len(a.mask, b, a.m);
  // this part's keys: whole tiles of them
  const int tiles = (len + kF32Cols - 1) / kF32Cols, per = (tiles + a.splits - 1) / a.splits * kF32Cols;
  const int k0 = sp * per, k1 = k0 + per < len ? k0 + per : len;
  f32_load<D, LD>(qs, cross_row<float>(a.q, a.sq, b, h, i0), a.sq.n, Lay::NR, a.n - i0, nullptr);
  const F32Thread<R> th;
  float acc[16 * Lay::NC] = {};
  float mx[R], l[R];  // of rows y + 16 i, in each of a row's 16 threads
#pragma unroll
  for (int i = 0; i < R; ++i) {
    mx[i] = -INFINITY;
    l[i] = 0.f;
  }
  for (int j0 = k0; j0 < k1; j0 += kF32Cols) {
    __syncthreads();  // the last tile's values are done with
    f32_keep(keep, kF32Cols, a.mask, b, j0, len);
    __syncthreads();
    f32_load<D, LD>(ks, cross_row<float>(a.k, a.sk, b, hk, j0), a.sk.n, kF32Cols, a.m - j0, keep);
    f32_commit();
    f32_load<D, LD>(vs, cross_row<float>(a.v, a.sv, b, hk, j0), a.sv.n, kF32Cols, a.m - j0, keep);
    f32_commit();
    f32_wait<1>();  // the keys (and the queries) are there, the values may still come
    __syncthreads();
    float s[R][4];
    f32_dots<D, R>(qs, ks, th, s);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) ps[th.score_row(i) * Lay::PW + Lay::place(th.x + 16 * j)] = s[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float* row = ps + (y + 16 * i) * Lay::PW;
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = keep[x + 16 * j] != 0.f ? row[Lay::place(x + 16 * j)] * a.scale : -INFINITY;
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
        row[Lay::place(x + 16 * j)] = p;
        sum += p;
      }
      l[i] = l[i] * corr + f32_row_sum(sum);
      mx[i] = m_new;
      if (x == 0) rowv[y + 16 * i] = corr;
    }
    f32_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float corr = rowv[th.g + Lay::RG * i];
#pragma unroll
      for (int k = 0; k < 4 * Lay::NC; ++k) acc[4 * Lay::NC * i + k] *= corr;
    }
    f32_accumulate<D, R>(ps, vs, th, acc);
  }
  f32_wait_all();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = i0 + y + 16 * i;
    if (x != 0 || r >= a.n) continue;
    rowv[y + 16 * i] = l[i] > 0.f ? 1.f / l[i] : l[i];
    const long long row = ((long long)b * a.heads + h) * a.n + r;
    const float lse = l[i] == 0.f ? -INFINITY : mx[i] + logf(l[i]);
    if (a.splits > 1)
      a.part_lse[(long long)sp * a.B * a.heads * a.n + row] = lse * 1.4426950408889634f;
    else if (a.lse != nullptr)
      a.lse[row] = lse;
  }
  __syncthreads();
  f32_join<D, R>(th, acc);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = i0 + th.result_row(i);
    if (r >= a.n) continue;
    const float inv = rowv[th.result_row(i)];
    const long long part_row = ((long long)sp * a.B + b) * a.heads * a.n + (long long)h * a.n + r;
    float* out = a.splits > 1 ? a.part + part_row * D : cross_row<float>(a.o, a.so, b, h, r);
#pragma unroll
    for (int k = 0; k < Lay::NC; ++k) {
      if (D % 64 != 0 && th.c + 16 * k >= D / 4) continue;
      const float* v = acc + 4 * (Lay::NC * i + k);
      *reinterpret_cast<float4*>(out + 4 * (th.c + 16 * k)) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    }
  }
}

// Parts of the keys as in the forward: a.dq_splits, their results in a.dq_part.
template <int D, int R>
__global__ void __launch_bounds__(kF32Threads) cross_f32_dq_kernel(const __grid_constant__ CrossArgs a) {
  using Lay = F32Layout<D, R>;
  constexpr int LD = Lay::LD;
  extern __shared__ __align__(16) float f32_smem[];
  float *qs = f32_smem, *dos = qs + Lay::ROWS, *ks = dos + Lay::ROWS, *vs = ks + Lay::COLS, *ps = vs + Lay::COLS,
        *keep = ps + Lay::P, *lse = keep + kF32Cols, *dd = lse + Lay::NR;
  const int qt = blockIdx.x / a.dq_splits, sp = blockIdx.x - qt * a.dq_splits;
  const int b = blockIdx.z, h = blockIdx.y, hk = h / a.group, i0 = qt * Lay::NR;
  const int y = threadIdx.x >> 4, x = threadIdx.x & 15, len = cross_len(a.mask, b, a.m);
  f32_load<D, LD>(qs, cross_row<float>(a.q, a.sq, b, h, i0), a.sq.n, Lay::NR, a.n - i0, nullptr);
  f32_load<D, LD>(dos, cross_row<float>(a.dout, a.sdo, b, h, i0), a.sdo.n, Lay::NR, a.n - i0, nullptr);
  f32_commit();
  f32_wait<0>();
  __syncthreads();
  const long long base = ((long long)b * a.heads + h) * a.n;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = i0 + y + 16 * i;
    float t = 0.f, v = -INFINITY;
    if (r < a.n) {
      const float* o = cross_row<float>(a.o_in, a.so, b, h, r);
      for (int c = x; c < D; c += 16) t = fmaf(dos[(y + 16 * i) * LD + c], o[c], t);
      v = a.lse[base + r];
    }
    t = f32_row_sum(t);
    if (x == 0) {
      lse[y + 16 * i] = v == -INFINITY ? INFINITY : v;  // rows past the last, and rows without keys: P = 0
      dd[y + 16 * i] = t;
      if (r < a.n && sp == 0) a.Drow[base + r] = t;
    }
  }
  const F32Thread<R> th;
  float acc[16 * Lay::NC] = {};
  const int tiles = (len + kF32Cols - 1) / kF32Cols, per = (tiles + a.dq_splits - 1) / a.dq_splits * kF32Cols;
  const int k0 = sp * per, k1 = k0 + per < len ? k0 + per : len;
  for (int j0 = k0; j0 < k1; j0 += kF32Cols) {
    __syncthreads();
    f32_keep(keep, kF32Cols, a.mask, b, j0, len);
    __syncthreads();
    f32_load<D, LD>(ks, cross_row<float>(a.k, a.sk, b, hk, j0), a.sk.n, kF32Cols, a.m - j0, keep);
    f32_load<D, LD>(vs, cross_row<float>(a.v, a.sv, b, hk, j0), a.sv.n, kF32Cols, a.m - j0, keep);
    f32_commit();
    f32_wait<0>();
    __syncthreads();
    float s[R][4], dp[R][4];
    f32_dots<D, R>(qs, ks, th, s);
    f32_dots<D, R>(dos, vs, th, dp);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = th.score_row(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = th.x + 16 * j;
        // 0 for a key that does not count, whatever dO holds
        ps[r * Lay::PW + Lay::place(c)] = keep[c] != 0.f ? expf(s[i][j] * a.scale - lse[r]) * (dp[i][j] - dd[r]) : 0.f;
      }
    }
    __syncthreads();
    f32_accumulate<D, R>(ps, ks, th, acc);
  }
  f32_join<D, R>(th, acc);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = i0 + th.result_row(i);
    if (r >= a.n) continue;
    float* out = a.dq_splits > 1 ? a.dq_part + ((long long)sp * a.B * a.heads * a.n + base + r) * D
                                 : cross_row<float>(a.dq, a.sdq, b, h, r);
#pragma unroll
    for (int k = 0; k < Lay::NC; ++k) {
      if (D % 64 != 0 && th.c + 16 * k >= D / 4) continue;
      const float* v = acc + 4 * (Lay::NC * i + k);
      *reinterpret_cast<float4*>(out + 4 * (th.c + 16 * k)) =
          make_float4(v[0] * a.scale, v[1] * a.scale, v[2] * a.scale, v[3] * a.scale);
    }
  }
}

// A block: 16 R keys and one part of the queries of their head group (blockIdx.x = key tile *
// splits + part); with splits > 1 the parts go to a.part, [dk, dv][split][B, kv_heads, m][D].
template <int D, int R>
__global__ void __launch_bounds__(kF32Threads, cross_f32_dkdv_blocks(D))
    cross_f32_dkdv_kernel(const __grid_constant__ CrossArgs a) {
  using Lay = F32Layout<D, R>;
  constexpr int LD = Lay::LD;
  extern __shared__ __align__(16) float f32_smem[];
  float *ks = f32_smem, *vs = ks + Lay::ROWS, *qs = vs + Lay::ROWS, *dos = qs + Lay::COLS, *ps = dos + Lay::COLS,
        *dss = ps + Lay::P, *lse = dss + Lay::P, *dd = lse + kF32Cols, *keep = dd + kF32Cols;
  const int b = blockIdx.z, hk = blockIdx.y, kt = blockIdx.x / a.splits, sp = blockIdx.x - kt * a.splits;
  const int j0 = kt * Lay::NR, len = cross_len(a.mask, b, a.m);
  const F32Thread<R> th;
  f32_keep(keep, Lay::NR, a.mask, b, j0, len);
  __syncthreads();
  float dk[16 * Lay::NC] = {}, dv[16 * Lay::NC] = {};
  if (j0 < len) {
    f32_load<D, LD>(ks, cross_row<float>(a.k, a.sk, b, hk, j0), a.sk.n, Lay::NR, a.m - j0, keep);
    f32_load<D, LD>(vs, cross_row<float>(a.v, a.sv, b, hk, j0), a.sv.n, Lay::NR, a.m - j0, keep);
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
      f32_load<D, LD>(qs, cross_row<float>(a.q, a.sq, b, h, i0), a.sq.n, kF32Cols, a.n - i0, nullptr);
      f32_load<D, LD>(dos, cross_row<float>(a.dout, a.sdo, b, h, i0), a.sdo.n, kF32Cols, a.n - i0, nullptr);
      f32_commit();
      f32_wait<0>();  // the keys' tiles too, at the first turn
      __syncthreads();
      float s[R][4], dp[R][4];
      f32_dots<D, R>(ks, qs, th, s);
      f32_dots<D, R>(vs, dos, th, dp);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = th.score_row(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = th.x + 16 * j, at = r * Lay::PW + Lay::place(c);
          const float p = keep[r] != 0.f ? expf(s[i][j] * a.scale - lse[c]) : 0.f;
          ps[at] = p;
          dss[at] = p * (dp[i][j] - dd[c]);
        }
      }
      __syncthreads();
      f32_accumulate<D, R>(ps, dos, th, dv);
      f32_accumulate<D, R>(dss, qs, th, dk);
    }
  }
  f32_wait_all();
  f32_join<D, R>(th, dk);
  f32_join<D, R>(th, dv);
  const long long rows = (long long)a.B * a.kv_heads * a.m;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int j = j0 + th.result_row(i);
    if (j >= a.m) continue;
    const bool live = keep[th.result_row(i)] != 0.f;  // else zeros, whatever q and dO hold
    const long long row = ((long long)b * a.kv_heads + hk) * a.m + j;
    float* ok = a.splits > 1 ? a.part + (sp * rows + row) * D : cross_row<float>(a.dk, a.sdk, b, hk, j);
    float* ov = a.splits > 1 ? a.part + ((a.splits + sp) * rows + row) * D : cross_row<float>(a.dv, a.sdv, b, hk, j);
#pragma unroll
    for (int k = 0; k < Lay::NC; ++k) {
      if (D % 64 != 0 && th.c + 16 * k >= D / 4) continue;
      const int c = 4 * (th.c + 16 * k);
      const float *vk = dk + 4 * (Lay::NC * i + k), *vv = dv + 4 * (Lay::NC * i + k);
      float4 gk = make_float4(vk[0] * a.scale, vk[1] * a.scale, vk[2] * a.scale, vk[3] * a.scale);
      float4 gv = make_float4(vv[0], vv[1], vv[2], vv[3]);
      if (!live) gk = gv = make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(ok + c) = gk;
      *reinterpret_cast<float4*>(ov + c) = gv;
    }
  }
}

}  // namespace sq
