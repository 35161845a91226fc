// Layer norm and its gradient, on gfx950.  For a row x of C elements,
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),
//   xh = (x - mean) rstd,  y = xh weight + bias
// and for a gradient dy, with g = dy weight,
//   dx = rstd (g - sum g / C - xh sum (g xh) / C),
//   dweight = sum over the rows of dy xh,  dbias = sum over the rows of dy.
//
// Streaming passes over rows that stay in registers, bound by HBM.  All sums are
// fp32 in an order that only the sizes fix; there are no atomics.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nsg_layer.h"
#include "nsg_rows.h"

namespace nsg {

// ---------------------------------------------------------------------------
// A row belongs to WR waves; lane l of them has the NV pieces of 16 bytes
// (j WR 64 + l) of it: at most 16 elements, rows of up to 16384.
// ---------------------------------------------------------------------------
template <typename T> constexpr int kPiece = 16 / (int)sizeof(T);
constexpr int kNormLane = 16;    // elements of a lane
constexpr int kNormWaves = 16;   // waves of a row at most
constexpr int kNormRegisters = kNormLane * kNormWaves * 64;  // elements of a row in registers

// 16 bytes of a row from element c on, zeros behind its end
template <typename T> struct Piece {
  static constexpr int N = kPiece<T>;
  typedef T vec __attribute__((ext_vector_type(N)));
  typedef vec mem __attribute__((aligned(sizeof(T))));
  vec v;
  __device__ __forceinline__ void load(const T *row, int c, int C) {
    if (c + N <= C) {
      v = *reinterpret_cast<const mem *>(row + c);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = c + i < C ? row[c + i] : (T)0.f;
    }
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

// Sums of a and b over the WR waves of a row, the same in all their lanes.  `sh`:
// a pair for each wave of the workgroup, not in use by an earlier sum.
template <int WR> __device__ __forceinline__ void row_sum(float &a, float &b, float (*sh)[2]) {
  a = wave_sum(a);
  b = wave_sum(b);
  if (WR == 1) return;
  const int wave = threadIdx.x >> 6, first = wave / WR * WR;
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

// A workgroup takes WAVES / WR rows at a time and keeps the weights; the next rows are
// on their way while it works.
template <typename T, int WAVES, int WR, int NV>
__global__ void __launch_bounds__(WAVES * 64) layer_norm_kernel(NormArgs p) {
  constexpr int N = kPiece<T>, kRows = WAVES / WR;
  __shared__ float sh[2][WAVES][2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = (wave % WR) * 64 + (threadIdx.x & 63);
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t r = (int64_t)blockIdx.x * kRows + wave / WR;
  Piece<T> x[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j].load((const T *)p.x + row * p.ldx, (j * WR * 64 + l) * N, row < p.R ? (int)p.C : 0);
  };
  constexpr bool kAhead = WR < 16;  // (16 waves have 128 registers each, too few for the next row)
  if (kAhead) fetch(r);
  float w[NV][N], b[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_weights<N>(p.weight, p.w_dtype, (j * WR * 64 + l) * N, p.C, 1.f, w[j]);
    load_weights<N>(p.bias, p.w_dtype, (j * WR * 64 + l) * N, p.C, 0.f, b[j]);
  }
  const float n = (float)p.C;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.R; r0 += step, r += step) {
    float f[NV][N], sum = 0.f, sq = 0.f;
    if (!kAhead) fetch(r);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[j][i] = (float)x[j].v[i];
        sum += f[j][i];
      }
    if (kAhead && r0 + step < p.R) fetch(r + step);
    row_sum<WR>(sum, sq, sh[0]);
    const float mean = sum / n;
    sum = sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = (j * WR * 64 + l) * N + i < p.C ? f[j][i] - mean : 0.f;
        f[j][i] = d;
        sum += d;
        sq = fmaf(d, d, sq);
      }
    row_sum<WR>(sum, sq, sh[1]);
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
      const int c = (j * WR * 64 + l) * N;
      if (c >= p.C) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) f[j][i] = fmaf((f[j][i] - rest) * rstd, w[j][i], b[j][i]);
      store_piece<T, N>(y, c, p.C, f[j]);
    }
  }
}

// The gradient: dx, and with parts [groups][2][C] this workgroup's sums of dy xh and dy.
// A lane has the same columns of every row, so these sums stay in its registers; the
// rows that a workgroup takes at a time are added at the end, in LDS.
template <typename T, int WAVES, int WR, int NV>
__global__ void __launch_bounds__(WAVES * 64) layer_norm_backward_kernel(NormArgs p, float *__restrict__ parts) {
  constexpr int N = kPiece<T>, kRows = WAVES / WR;
  __shared__ float sh[2][WAVES][2];
  __shared__ float joined[kRows > 1 ? 2 * WR * 64 * NV * N : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = (wave % WR) * 64 + (threadIdx.x & 63);
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t r = (int64_t)blockIdx.x * kRows + wave / WR;
  Piece<T> x[NV], dy[NV];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * WR * 64 + l) * N, C = row < p.R ? (int)p.C : 0;
      x[j].load((const T *)p.x + row * p.ldx, c, C);
      dy[j].load((const T *)p.dy + row * p.lddy, c, C);
    }
    mean = row < p.R ? p.stats[row] : 0.f;
    rstd = row < p.R ? p.stats[p.R + row] : 0.f;
  };
  constexpr bool kAhead = WR < 16;
  if (kAhead) fetch(r);
  float w[NV][N], aw[NV][N], ab[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_weights<N>(p.weight, p.w_dtype, (j * WR * 64 + l) * N, p.C, 1.f, w[j]);
#pragma unroll
    for (int i = 0; i < N; ++i) aw[j][i] = ab[j][i] = 0.f;
  }
  const float n = (float)p.C;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.R; r0 += step, r += step, turn ^= 1) {
    float xh[NV][N], g[NV][N], a = 0.f, b = 0.f;
    if (!kAhead) fetch(r);
    const float rs = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = (float)dy[j].v[i];
        xh[j][i] = (j * WR * 64 + l) * N + i < p.C ? ((float)x[j].v[i] - mean) * rs : 0.f;
        aw[j][i] = fmaf(d, xh[j][i], aw[j][i]);
        ab[j][i] += d;
        g[j][i] = d * w[j][i];
        a += g[j][i];
        b = fmaf(g[j][i], xh[j][i], b);
      }
    if (kAhead && r0 + step < p.R) fetch(r + step);
    row_sum<WR>(a, b, sh[turn]);
    a /= n;
    b /= n;
    if (r >= p.R) continue;
    T *dx = (T *)p.out + r * p.C;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * WR * 64 + l) * N;
      if (c >= p.C) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) g[j][i] = rs * (g[j][i] - a - xh[j][i] * b);
      store_piece<T, N>(dx, c, p.C, g[j]);
    }
  }
  if (parts == nullptr) return;
  constexpr int kCols = WR * 64 * NV * N;
  for (int k = 1; k < kRows; ++k) {
    __syncthreads();
    if (wave / WR == k) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Row<float, N>::store(joined + (j * WR * 64 + l) * N, aw[j]);
        Row<float, N>::store(joined + kCols + (j * WR * 64 + l) * N, ab[j]);
      }
    }
    __syncthreads();
    if (wave < WR) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[N];
        Row<float, N>::load(joined + (j * WR * 64 + l) * N, v);
#pragma unroll
        for (int i = 0; i < N; ++i) aw[j][i] += v[i];
        Row<float, N>::load(joined + kCols + (j * WR * 64 + l) * N, v);
#pragma unroll
        for (int i = 0; i < N; ++i) ab[j][i] += v[i];
      }
    }
  }
  if (wave >= WR) return;
  float *to = parts + (size_t)blockIdx.x * 2 * p.C;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * WR * 64 + l) * N;
    if (c >= p.C) continue;
    store_piece<float, N>(to, c, p.C, aw[j]);
    store_piece<float, N>(to + p.C, c, p.C, ab[j]);
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
    row_sum<16>(a, b, sh[0]);
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
    row_sum<16>(a, b, sh[1]);
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
    row_sum<16>(a, b, sh[turn]);
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
constexpr int kNormGroups = 512;

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
// How many waves a row takes and how many pieces a lane of it has
template <typename T, class K> static hipError_t by_width(const NormArgs &a, hipStream_t s) {
  constexpr int NV = kNormLane / kPiece<T>;
  if (a.C <= 512) return K::template rows<T, 1, NV / 2>(a, s);
  if (a.C <= 1024) return K::template rows<T, 1, NV>(a, s);
  if (a.C <= 2048) return K::template rows<T, 2, NV>(a, s);
  if (a.C <= 4096) return K::template rows<T, 4, NV>(a, s);
  if (a.C <= 8192) return K::template rows<T, 8, NV>(a, s);
  if (a.C <= kNormRegisters) return K::template rows<T, 16, NV>(a, s);
  return K::template wide<T>(a, s);
}
static int64_t fewer(int64_t a, int64_t b) { return a < b ? a : b; }

struct NormForward {
  template <typename T, int WR, int NV> static hipError_t rows(const NormArgs &a, hipStream_t s) {
    constexpr int waves = WR < 4 ? 4 : WR, most = 256 * 24 / waves;
    hipLaunchKernelGGL((layer_norm_kernel<T, waves, WR, NV>), dim3((unsigned)fewer((a.R + waves / WR - 1) / (waves / WR), most)),
                       dim3(waves * 64), 0, s, a);
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
  static float *parts(const NormArgs &a) { return a.dweight == nullptr && a.dbias == nullptr ? nullptr : (float *)a.workspace; }
  template <typename T, int WR, int NV> static hipError_t rows(const NormArgs &a, hipStream_t s) {
    constexpr int waves = WR < 8 ? 8 : WR, most = kNormGroups * 8 / waves;
    const int groups = (int)fewer((a.R + waves / WR - 1) / (waves / WR), most);
    if (groups > 0) {
      hipLaunchKernelGGL((layer_norm_backward_kernel<T, waves, WR, NV>), dim3((unsigned)groups), dim3(waves * 64), 0, s, a, parts(a));
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
