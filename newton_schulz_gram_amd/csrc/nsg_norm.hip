// Layer norm and its gradient, on gfx950.  For a row x of C elements,
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),
//   xh = (x - mean) rstd,  y = xh weight + bias
// and for a gradient dy, with g = dy weight,
//   dx = rstd (g - sum g / C - xh sum (g xh) / C),
//   dweight = sum over the rows of dy xh,  dbias = sum over the rows of dy.
//
// Streaming passes over rows that stay in registers, bound by HBM: 16384 rows of 4096 in
// bf16 take 51 us (5.3 TB/s), their gradient 78 (5.2).  All sums are fp32 in an order that
// only the sizes fix; there are no atomics.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nsg_layer.h"
#include "nsg_rows.h"

namespace nsg {

// ---------------------------------------------------------------------------
// A row belongs to LANES lanes; lane l of them has the NV pieces of 16 bytes (j LANES + l)
// of it, 16 elements, in the gradient of more than 8192 in a row 32.  The last piece of a
// row whose length is no multiple of a piece lies over the one before it: its first
// elements are read and stored twice, and left out of sums.
// ---------------------------------------------------------------------------
template <typename T> constexpr int kPiece = 16 / (int)sizeof(T);
constexpr int kNormLane = 16;          // elements of a lane
// Elements of a row in registers: 4096 rows of 16384 in bf16 take 57 us and their gradient 106,
// of 16392, which are read again for each sum, 81 and 173.
constexpr int kNormRegisters = 16384;

template <typename T> struct Piece {
  static constexpr int N = kPiece<T>;
  typedef T vec __attribute__((ext_vector_type(N)));
  typedef vec mem __attribute__((aligned(sizeof(T))));
  vec v;
  __device__ __forceinline__ void load(const T *row, int c) { v = *reinterpret_cast<const mem *>(row + c); }
};
// where piece j of lane l lies, how many of its first elements are another's, whether it is there
template <typename T, int LANES> struct Place {
  static constexpr int N = kPiece<T>;
  int c, skip;
  bool there;
  __device__ __forceinline__ Place(int j, int l, int C) {
    c = (j * LANES + l) * N;
    there = c < C;
    skip = c + N > C ? c + N - C : 0;  // (at least N where it is not there)
    if (skip > 0) c = C - N;
  }
};

// N consecutive elements of a row from c on as fp32, zeros behind its end
template <typename T, int N> __device__ __forceinline__ void load_piece(const T *row, int c, int C, float (&f)[N]) {
  if (c + N <= C) {
    Row<T, N, (int)sizeof(T)>::load(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = c + i < C ? (float)row[c + i] : 0.f;
  }
}
template <typename T, int N> __device__ __forceinline__ void store_piece(T *row, int c, int C, const float (&f)[N]) {
  if (c + N <= C) {
    Row<T, N, (int)sizeof(T)>::store(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < C) row[c + i] = (T)f[i];
  }
}
// weights of any type (`dtype` is the same in all lanes), `none` where there are none
template <int N>
__device__ __forceinline__ void load_weights(const void *w, int dtype, int c, int C, float none, float (&f)[N]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = none;
  } else if (dtype == NSG_F32) {
    load_piece<float, N>((const float *)w, c, C, f);
  } else if (dtype == NSG_BF16) {
    load_piece<__bf16, N>((const __bf16 *)w, c, C, f);
  } else {
    load_piece<_Float16, N>((const _Float16 *)w, c, C, f);
  }
}
__device__ __forceinline__ void store_weight(void *w, int dtype, int64_t c, float v) {
  if (dtype == NSG_F32) ((float *)w)[c] = v;
  else if (dtype == NSG_BF16) ((__bf16 *)w)[c] = (__bf16)v;
  else ((_Float16 *)w)[c] = (_Float16)v;
}

// 1 / sqrt(var + eps) for the mean square m2 of differences whose mean is `rest` (a NaN stays one)
__device__ __forceinline__ float row_rstd(float m2, float rest, float eps) {
  const float var = m2 - rest * rest;
  return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
}

// Sums of a and b over the LANES lanes of a row, the same in all of them.  `sh`: a pair
// for each wave of the workgroup, not in use by an earlier sum.
template <int LANES> __device__ __forceinline__ void row_sum(float &a, float &b, float (*sh)[2]) {
  constexpr int L = LANES < 64 ? LANES : 64, WR = LANES / 64;
  a = group_lanes_sum<L>(a);
  b = group_lanes_sum<L>(b);
  if (WR <= 1) return;
  const int wave = threadIdx.x >> 6, first = wave / (WR > 0 ? WR : 1) * WR;
  if ((threadIdx.x & 63) == 0) {
    sh[wave][0] = a;
    sh[wave][1] = b;
  }
  __syncthreads();
  a = b = 0.f;
#pragma unroll
  for (int w = 0; w < WR; ++w) {
    a += sh[first + w][0];
    b += sh[first + w][1];
  }
}

// This thread's row of the THREADS / LANES that a workgroup takes at a time (the same in a
// wave where a row has that many lanes)
template <int LANES> __device__ __forceinline__ int own_row() {
  return LANES >= 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / LANES) : threadIdx.x / LANES;
}

// weights as fp32 in LDS, where threads have no registers for them
template <int THREADS> __device__ __forceinline__ void weights_to_lds(const void *w, int dtype, int C, float none, float *to) {
#pragma unroll 8
  for (int c = threadIdx.x; c < C; c += THREADS)
    to[c] = w == nullptr       ? none
            : dtype == NSG_F32 ? ((const float *)w)[c]
            : dtype == NSG_BF16 ? (float)((const __bf16 *)w)[c] : (float)((const _Float16 *)w)[c];
}

// A workgroup takes THREADS / LANES rows at a time and keeps the weights; the next rows are
// on their way while it works.
template <typename T, int THREADS, int LANES, int NV>
__global__ void __launch_bounds__(THREADS) layer_norm_kernel(NormArgs p) {
  constexpr int N = kPiece<T>, kRows = THREADS / LANES;
  __shared__ float sh[2][THREADS / 64][2];
  const int l = threadIdx.x % LANES, C = (int)p.C;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t r = (int64_t)blockIdx.x * kRows + own_row<LANES>();
  Piece<T> x[NV];
  auto fetch = [&](int64_t row) {
    if (row >= p.R) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Place<T, LANES> at(j, l, C);
      if (at.there) x[j].load((const T *)p.x + row * p.ldx, at.c);
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) x[j].v = (T)0.f;
  fetch(r);
  float w[NV][N], b[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Place<T, LANES> at(j, l, C);
    if (!at.there) continue;
    load_weights<N>(p.weight, p.w_dtype, at.c, C, 1.f, w[j]);
    load_weights<N>(p.bias, p.w_dtype, at.c, C, 0.f, b[j]);
  }
  const float n = (float)C;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.R; r0 += step, r += step) {
    float f[NV][N], sum = 0.f, sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Place<T, LANES> at(j, l, C);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[j][i] = (float)x[j].v[i];
        sum += i >= at.skip ? f[j][i] : 0.f;
      }
    }
    fetch(r + step);
    row_sum<LANES>(sum, sq, sh[0]);
    const float mean = sum / n;
    sum = sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Place<T, LANES> at(j, l, C);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[j][i] -= mean;
        const float d = i >= at.skip ? f[j][i] : 0.f;
        sum += d;
        sq = fmaf(d, d, sq);
      }
    }
    row_sum<LANES>(sum, sq, sh[1]);
    const float rest = sum / n;  // what rounding left of the mean
    const float rstd = row_rstd(sq / n, rest, p.eps);
    if (r >= p.R) continue;
    if (l == 0) {
      p.stats[r] = mean + rest;
      p.stats[p.R + r] = rstd;
    }
    T *y = (T *)p.out + r * p.C;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Place<T, LANES> at(j, l, C);
      if (!at.there) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) f[j][i] = fmaf((f[j][i] - rest) * rstd, w[j][i], b[j][i]);
      Row<T, N, (int)sizeof(T)>::store(y + at.c, f[j]);
    }
  }
}

// The gradient: dx, and with parts [groups][2][C] this workgroup's sums of dy xh and dy.
// A lane has the same columns of every row, so these sums stay in its registers; those of
// the rows that a workgroup takes at a time are added at the end.
template <typename T, int THREADS, int LANES, int NV, bool KEEP>
__global__ void __launch_bounds__(THREADS) layer_norm_backward_kernel(NormArgs p, float *__restrict__ parts) {
  constexpr int N = kPiece<T>, kRows = THREADS / LANES;
  constexpr int kWide = LANES < 64 ? 64 : LANES, kGroups = THREADS / kWide;  // threads that add in LDS, groups of them
  constexpr int kCols = LANES * NV * N;
  __shared__ float sh[2][THREADS / 64][2];
  __shared__ float joined[kGroups > 1 ? 2 * kCols : 1];
  const int l = threadIdx.x % LANES, C = (int)p.C;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t r = (int64_t)blockIdx.x * kRows + own_row<LANES>();
  Piece<T> x[NV], dy[NV];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t row) {
    if (row >= p.R) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Place<T, LANES> at(j, l, C);
      if (!at.there) continue;
      x[j].load((const T *)p.x + row * p.ldx, at.c);
      dy[j].load((const T *)p.dy + row * p.lddy, at.c);
    }
    mean = p.stats[row];
    rstd = p.stats[p.R + row];
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) x[j].v = dy[j].v = (T)0.f;
  // (else the registers hold no next row: 6096 rows of 11008 102 us so, 3048 in fp32 97; with
  // the next row in them 100 and 139)
  constexpr bool kAhead = KEEP;
  if (kAhead) fetch(r);
  __shared__ float lds[KEEP ? 1 : LANES * NV * N];
  if (!KEEP) {
    weights_to_lds<THREADS>(p.weight, p.w_dtype, C, 1.f, lds);
    __syncthreads();
  }
  float w[KEEP ? NV : 1][N], aw[NV][N], ab[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Place<T, LANES> at(j, l, C);
    if (KEEP && at.there) load_weights<N>(p.weight, p.w_dtype, at.c, C, 1.f, w[KEEP ? j : 0]);
#pragma unroll
    for (int i = 0; i < N; ++i) aw[j][i] = ab[j][i] = 0.f;
  }
  const float n = (float)C;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.R; r0 += step, r += step, turn ^= 1) {
    float xh[NV][N], g[NV][N], a = 0.f, b = 0.f;
    if (!kAhead) fetch(r);
    const float rs = rstd;
    const bool own = r < p.R;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Place<T, LANES> at(j, l, C);
      if (!KEEP && at.there) {
        int c = at.c;
        asm volatile("" : "+v"(c));  // read for each row: kept for all, they would need too many registers
        Row<float, N, 4>::load(lds + c, w[0]);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = (float)dy[j].v[i];
        xh[j][i] = ((float)x[j].v[i] - mean) * rs;
        g[j][i] = at.there ? d * w[KEEP ? j : 0][i] : 0.f;
        if (own) {
          aw[j][i] = fmaf(d, xh[j][i], aw[j][i]);
          ab[j][i] += d;
        }
        if (i >= at.skip) {
          a += g[j][i];
          b = fmaf(g[j][i], xh[j][i], b);
        }
      }
    }
    if (kAhead) fetch(r + step);
    row_sum<LANES>(a, b, sh[turn]);
    a /= n;
    b /= n;
    if (!own) continue;
    T *dx = (T *)p.out + r * p.C;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Place<T, LANES> at(j, l, C);
      if (!at.there) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) g[j][i] = rs * (g[j][i] - a - xh[j][i] * b);
      Row<T, N, (int)sizeof(T)>::store(dx + at.c, g[j]);
    }
  }
  if (parts == nullptr) return;
  // rows of a wave, then of the workgroup
  if (LANES < 64) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int off = LANES; off < 64; off <<= 1) {
          aw[j][i] += __shfl_xor(aw[j][i], off, 64);
          ab[j][i] += __shfl_xor(ab[j][i], off, 64);
        }
      }
  }
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / kWide);
  const bool adds = LANES >= 64 || (threadIdx.x & 63) < LANES;
  for (int k = 1; k < kGroups; ++k) {
    __syncthreads();
    if (group == k && adds) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Row<float, N>::store(joined + (j * LANES + l) * N, aw[j]);
        Row<float, N>::store(joined + kCols + (j * LANES + l) * N, ab[j]);
      }
    }
    __syncthreads();
    if (group == 0 && adds) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[N];
        Row<float, N>::load(joined + (j * LANES + l) * N, v);
#pragma unroll
        for (int i = 0; i < N; ++i) aw[j][i] += v[i];
        Row<float, N>::load(joined + kCols + (j * LANES + l) * N, v);
#pragma unroll
        for (int i = 0; i < N; ++i) ab[j][i] += v[i];
      }
    }
  }
  if (group > 0 || !adds) return;
  float *to = parts + (size_t)blockIdx.x * 2 * p.C;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Place<T, LANES> at(j, l, C);
    if (!at.there) continue;
    Row<float, N, 4>::store(to + at.c, aw[j]);
    Row<float, N, 4>::store(to + p.C + at.c, ab[j]);
  }
}

// Rows that do not fit in registers: read once for each sum and once for the output
template <typename T> __global__ void __launch_bounds__(1024) layer_norm_wide_kernel(NormArgs p) {
  constexpr int N = kPiece<T>;
  __shared__ float sh[2][16][2];
  const float n = (float)p.C;
  for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x) {
    const T *x = (const T *)p.x + r * p.ldx;
    T *y = (T *)p.out + r * p.C;
    float f[N], w[N], b2[N], a = 0.f, b = 0.f;
    for (int c = (int)threadIdx.x * N; c < p.C; c += 1024 * N) {
      load_piece<T, N>(x, c, p.C, f);
#pragma unroll
      for (int i = 0; i < N; ++i) a += f[i];
    }
    row_sum<1024>(a, b, sh[0]);
    float mean = a / n;
    a = b = 0.f;
    for (int c = (int)threadIdx.x * N; c < p.C; c += 1024 * N) {
      load_piece<T, N>(x, c, p.C, f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = c + i < p.C ? f[i] - mean : 0.f;
        a += d;
        b = fmaf(d, d, b);
      }
    }
    row_sum<1024>(a, b, sh[1]);
    const float rest = a / n, rstd = row_rstd(b / n, rest, p.eps);
    if (threadIdx.x == 0) {
      p.stats[r] = mean + rest;
      p.stats[p.R + r] = rstd;
    }
    for (int c = (int)threadIdx.x * N; c < p.C; c += 1024 * N) {
      load_piece<T, N>(x, c, p.C, f);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = (f[i] - mean - rest) * rstd;
      load_weights<N>(p.weight, p.w_dtype, c, p.C, 1.f, w);
      load_weights<N>(p.bias, p.w_dtype, c, p.C, 0.f, b2);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = fmaf(f[i], w[i], b2[i]);
      store_piece<T, N>(y, c, p.C, f);
    }
  }
}
template <typename T> __global__ void __launch_bounds__(1024) layer_norm_wide_dx_kernel(NormArgs p) {
  constexpr int N = kPiece<T>;
  __shared__ float sh[2][16][2];
  int turn = 0;
  for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x, turn ^= 1) {
    const T *x = (const T *)p.x + r * p.ldx, *dy = (const T *)p.dy + r * p.lddy;
    const float mean = p.stats[r], rstd = p.stats[p.R + r];
    float a = 0.f, b = 0.f;
    auto at = [&](int c, float (&f)[N], float (&g)[N]) {
      float w[N];
      load_piece<T, N>(x, c, p.C, f);
      load_piece<T, N>(dy, c, p.C, g);
      load_weights<N>(p.weight, p.w_dtype, c, p.C, 1.f, w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        g[i] *= w[i];
        f[i] = c + i < p.C ? (f[i] - mean) * rstd : 0.f;
      }
    };
    for (int c = (int)threadIdx.x * N; c < p.C; c += 1024 * N) {
      float f[N], g[N];
      at(c, f, g);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        a += g[i];
        b = fmaf(g[i], f[i], b);
      }
    }
    row_sum<1024>(a, b, sh[turn]);
    a /= (float)p.C;
    b /= (float)p.C;
    for (int c = (int)threadIdx.x * N; c < p.C; c += 1024 * N) {
      float f[N], g[N];
      at(c, f, g);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = rstd * (g[i] - a - f[i] * b);
      store_piece<T, N>((T *)p.out + r * p.C, c, p.C, f);
    }
  }
}

// ---------------------------------------------------------------------------
// dweight and dbias: sums of groups of rows, one of the groups after another
// ---------------------------------------------------------------------------
// (256, 512 and 1024 of them: 16384 rows of 4096 84, 85 and 88 us, 131072 of 512 82, 85 and 89)
constexpr int kNormGroups = 256;

// parts [groups][2][C]
template <typename T> __global__ void __launch_bounds__(256) layer_norm_dw_kernel(NormArgs p, int64_t per, float *__restrict__ parts) {
  constexpr int N = kPiece<T>;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * N;
  if (c >= p.C) return;
  const int64_t r0 = (int64_t)blockIdx.y * per, r1 = min(p.R, r0 + per);
  float a[N], b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = b[i] = 0.f;
#pragma unroll 4
  for (int64_t r = r0; r < r1; ++r) {
    const float mean = p.stats[r], rstd = p.stats[p.R + r];
    float f[N], g[N];
    load_piece<T, N>((const T *)p.x + r * p.ldx, c, p.C, f);
    load_piece<T, N>((const T *)p.dy + r * p.lddy, c, p.C, g);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = fmaf(g[i], (f[i] - mean) * rstd, a[i]);
      b[i] += g[i];
    }
  }
  float *to = parts + (size_t)blockIdx.y * 2 * p.C;
  store_piece<float, N>(to, c, p.C, a);
  store_piece<float, N>(to + p.C, c, p.C, b);
}

// 64 columns of the 2 C to a workgroup, its 16 waves share the groups
__global__ void __launch_bounds__(1024) layer_norm_join_kernel(NormArgs p, int groups, const float *__restrict__ parts) {
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float a = 0.f;
  if (c < 2 * p.C) {
#pragma unroll 8
    for (int g = wave; g < groups; g += 16) a += parts[(size_t)g * 2 * p.C + c];
  }
  sh[wave][lane] = a;
  __syncthreads();
  if (wave > 0 || c >= 2 * p.C) return;
  a = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) a += sh[w][lane];
  void *to = c < p.C ? p.dweight : p.dbias;
  if (to != nullptr) store_weight(to, p.w_dtype, c < p.C ? c : c - p.C, a);
}

// ---------------------------------------------------------------------------
// How many lanes a row takes: enough for 16 elements each.  With 8, 16 and 32 of them 16384
// rows of 4096 in bf16 take 52, 46 and 45 us, their gradient 82, 85 and 86; 1003 of 1250 in fp32
// 4.6, 4.7 and 5.5, and 12, 11 and 20; 32768 of 1024 44, 42 and 42, and 78, 80 and 145.  (Calls
// one after the other on the same memory, where the last-level cache takes part of the
// stores; 16384 rows of 4096 with an output of their own for each call: 51 us for 43.)
//
// Rows shorter than a piece go to the kernel for wide ones, which takes any length but has a
// workgroup for each row: 1048576 rows of 7 in bf16 take 7.5 ms and their gradient 13, of 8
// 25 and 41 us.
// ---------------------------------------------------------------------------
template <typename T, class K> static hipError_t by_width(const NormArgs &a, hipStream_t s) {
  constexpr int NV = kNormLane / kPiece<T>;
  if (a.C < kPiece<T>) return K::template wide<T>(a, s);
  if (a.C <= 4 * kNormLane) return K::template rows<T, 4, NV>(a, s);
  if (a.C <= 8 * kNormLane) return K::template rows<T, 8, NV>(a, s);
  if (a.C <= 16 * kNormLane) return K::template rows<T, 16, NV>(a, s);
  if (a.C <= 32 * kNormLane) return K::template rows<T, 32, NV>(a, s);
  if (a.C <= 64 * kNormLane) return K::template rows<T, 64, NV>(a, s);
  if (a.C <= 128 * kNormLane) return K::template rows<T, 128, NV>(a, s);
  if (a.C <= 256 * kNormLane) return K::template rows<T, 256, NV>(a, s);
  if (a.C <= 512 * kNormLane) return K::template rows<T, 512, NV>(a, s);
  if (a.C <= kNormRegisters) return K::template rows<T, K::kLongest, NV * 1024 / K::kLongest>(a, s);
  return K::template wide<T>(a, s);
}
static int64_t fewer(int64_t a, int64_t b) { return a < b ? a : b; }

struct NormForward {
  static constexpr int kLongest = 1024;  // lanes of a row above 8192
  template <typename T, int LANES, int NV> static hipError_t rows(const NormArgs &a, hipStream_t s) {
    constexpr int threads = LANES < 256 ? 256 : LANES, rows = threads / LANES;
    // (1024, 1536 and 4096 workgroups of 256: 16384 rows of 4096 47, 46 and 43 us; 256, 512 and
    // 1024 of 1024 threads: 6096 rows of 11008 61, 63 and 67; calls on the same memory, see below)
    constexpr int most = threads == 1024 ? 256 : 256 * 4096 / threads;
    hipLaunchKernelGGL((layer_norm_kernel<T, threads, LANES, NV>),
                       dim3((unsigned)fewer((a.R + rows - 1) / rows, most)), dim3(threads), 0, s, a);
    return hipGetLastError();
  }
  template <typename T> static hipError_t wide(const NormArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(layer_norm_wide_kernel<T>, dim3((unsigned)fewer(a.R, 1 << 16)), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
};

hipError_t launch_layer_norm(const NormArgs &a, hipStream_t s) {
  switch (a.dtype) {
    case NSG_F16: return by_width<_Float16, NormForward>(a, s);
    case NSG_BF16: return by_width<__bf16, NormForward>(a, s);
    default: return by_width<float, NormForward>(a, s);
  }
}

size_t layer_norm_backward_workspace(int64_t R, int64_t C) { return (size_t)fewer(R, kNormGroups) * 2 * (size_t)C * 4; }

static hipError_t norm_join(const NormArgs &a, int groups, hipStream_t s) {
  if (a.dweight == nullptr && a.dbias == nullptr) return hipSuccess;
  hipLaunchKernelGGL(layer_norm_join_kernel, dim3((unsigned)((2 * a.C + 63) / 64)), dim3(1024), 0, s, a, groups,
                     (const float *)a.workspace);
  return hipGetLastError();
}

struct NormBackward {
  static constexpr int kLongest = 512;  // (of 256 registers: the sums are two more for each element)
  static float *parts(const NormArgs &a) { return a.dweight == nullptr && a.dbias == nullptr ? nullptr : (float *)a.workspace; }
  template <typename T, int LANES, int NV> static hipError_t rows(const NormArgs &a, hipStream_t s) {
    constexpr int threads = LANES < 512 ? 512 : LANES, rows = threads / LANES;
    constexpr bool keep = NV * kPiece<T> == kNormLane;
    const int groups = (int)fewer((a.R + rows - 1) / rows, kNormGroups);
    if (groups > 0) {
      hipLaunchKernelGGL((layer_norm_backward_kernel<T, threads, LANES, NV, keep>),
                         dim3((unsigned)groups), dim3(threads), 0, s, a, parts(a));
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return norm_join(a, groups, s);
  }
  template <typename T> static hipError_t wide(const NormArgs &a, hipStream_t s) {
    const int64_t groups = fewer(a.R, kNormGroups), per = groups ? (a.R + groups - 1) / groups : 0, used = groups ? (a.R + per - 1) / per : 0;
    if (a.R > 0) {
      hipLaunchKernelGGL(layer_norm_wide_dx_kernel<T>, dim3((unsigned)fewer(a.R, 1 << 16)), dim3(1024), 0, s, a);
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      if (parts(a) != nullptr) {
        const dim3 grid((unsigned)((a.C + 256 * kPiece<T> - 1) / (256 * kPiece<T>)), (unsigned)used);
        hipLaunchKernelGGL(layer_norm_dw_kernel<T>, grid, dim3(256), 0, s, a, per, parts(a));
        e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
    }
    return norm_join(a, (int)used, s);
  }
};

hipError_t launch_layer_norm_backward(const NormArgs &a, hipStream_t s) {
  switch (a.dtype) {
    case NSG_F16: return by_width<_Float16, NormBackward>(a, s);
    case NSG_BF16: return by_width<__bf16, NormBackward>(a, s);
    default: return by_width<float, NormBackward>(a, s);
  }
}

}  // namespace nsg
