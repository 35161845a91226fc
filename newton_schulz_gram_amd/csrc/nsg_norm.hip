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
// (j WR 64 + l) of it.
// ---------------------------------------------------------------------------
template <typename T> constexpr int kPiece = 16 / (int)sizeof(T);

// N consecutive elements of a row from c on, zeros behind its end
template <typename T, int N> __device__ __forceinline__ void load_piece(const T *row, int64_t c, int64_t C, float (&f)[N]) {
  if (c + N <= C) {
    Row<T, N, (int)sizeof(T)>::load(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = c + i < C ? (float)row[c + i] : 0.f;
  }
}
template <typename T, int N> __device__ __forceinline__ void store_piece(T *row, int64_t c, int64_t C, const float (&f)[N]) {
  if (c + N <= C) {
    Row<T, N, (int)sizeof(T)>::store(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < C) row[c + i] = (T)f[i];
  }
}
// the same of weights of any type (`dtype` is the same in all lanes)
template <int N> __device__ __forceinline__ void load_weights(const void *w, int dtype, int64_t c, int64_t C, float (&f)[N]) {
  if (dtype == NSG_F32) load_piece<float, N>((const float *)w, c, C, f);
  else if (dtype == NSG_BF16) load_piece<__bf16, N>((const __bf16 *)w, c, C, f);
  else load_piece<_Float16, N>((const _Float16 *)w, c, C, f);
}
__device__ __forceinline__ void store_weight(void *w, int dtype, int64_t c, float v) {
  if (dtype == NSG_F32) ((float *)w)[c] = v;
  else if (dtype == NSG_BF16) ((__bf16 *)w)[c] = (__bf16)v;
  else ((_Float16 *)w)[c] = (_Float16)v;
}

// f weight + bias, where there are any (w: room)
template <int N> __device__ __forceinline__ void weigh(const NormArgs &p, int64_t c, float (&f)[N], float (&w)[N]) {
  if (p.weight != nullptr) {
    load_weights<N>(p.weight, p.w_dtype, c, p.C, w);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] *= w[i];
  }
  if (p.bias != nullptr) {
    load_weights<N>(p.bias, p.w_dtype, c, p.C, w);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] += w[i];
  }
}

// 1 / sqrt(var + eps) for the mean square m2 of differences whose mean is `rest` (a NaN stays one)
__device__ __forceinline__ float row_rstd(float m2, float rest, float eps) {
  const float var = m2 - rest * rest;
  return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
}

// Sums of a and b over the WR waves of a row, the same in all their lanes.  `sh`:
// a pair for each wave of the workgroup, not in use by an earlier sum.
template <int WR> __device__ __forceinline__ void row_sum(float &a, float &b, float (*sh)[2]) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    a += __shfl_xor(a, off, 64);
    b += __shfl_xor(b, off, 64);
  }
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

template <typename T, int WAVES, int WR, int NV>
__global__ void __launch_bounds__(WAVES * 64) layer_norm_kernel(NormArgs p) {
  constexpr int N = kPiece<T>;
  __shared__ float sh[2][WAVES][2];
  const int wave = threadIdx.x >> 6;
  for (int64_t r0 = (int64_t)blockIdx.x * (WAVES / WR); r0 < p.R; r0 += (int64_t)gridDim.x * (WAVES / WR)) {
  const int64_t r = r0 + wave / WR;
  const bool there = r < p.R;
  const T *x = (const T *)p.x + (there ? r : 0) * p.ldx;
  const int l = (wave % WR) * 64 + (threadIdx.x & 63);
  float f[NV][N], a = 0.f, b = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) load_piece<T, N>(x, (int64_t)(j * WR * 64 + l) * N, p.C, f[j]);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) a += f[j][i];
  row_sum<WR>(a, b, sh[0]);
  const float n = (float)p.C;
  float mean = a / n;
  a = b = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = (j * WR * 64 + l) * N + i < p.C ? f[j][i] - mean : 0.f;
      f[j][i] = d;
      a += d;
      b = fmaf(d, d, b);
    }
  row_sum<WR>(a, b, sh[1]);
  // a / n: what rounding left of the mean
  const float rest = a / n, rstd = row_rstd(b / n, rest, p.eps);
  mean += rest;
  if (!there) continue;
  if (l == 0) {
    p.stats[r] = mean;
    p.stats[p.R + r] = rstd;
  }
  T *y = (T *)p.out + r * p.C;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = (int64_t)(j * WR * 64 + l) * N;
    if (c >= p.C) continue;
    float w[N], v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (f[j][i] - rest) * rstd;
    weigh<N>(p, c, v, w);
    store_piece<T, N>(y, c, p.C, v);
  }
  }
}

template <typename T, int WAVES, int WR, int NV>
__global__ void __launch_bounds__(WAVES * 64) layer_norm_dx_kernel(NormArgs p) {
  constexpr int N = kPiece<T>;
  __shared__ float sh[2][WAVES][2];
  const int wave = threadIdx.x >> 6;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * (WAVES / WR); r0 < p.R; r0 += (int64_t)gridDim.x * (WAVES / WR), turn ^= 1) {
  const int64_t r = r0 + wave / WR;
  const bool there = r < p.R;
  const int64_t row = there ? r : 0;
  const T *x = (const T *)p.x + row * p.ldx, *dy = (const T *)p.dy + row * p.lddy;
  const int l = (wave % WR) * 64 + (threadIdx.x & 63);
  const float mean = p.stats[row], rstd = p.stats[p.R + row];
  float f[NV][N], g[NV][N], a = 0.f, b = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = (int64_t)(j * WR * 64 + l) * N;
    load_piece<T, N>(x, c, p.C, f[j]);
    load_piece<T, N>(dy, c, p.C, g[j]);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = (int64_t)(j * WR * 64 + l) * N;
    float w[N];
    if (p.weight != nullptr) load_weights<N>(p.weight, p.w_dtype, c, p.C, w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (p.weight != nullptr) g[j][i] *= w[i];
      f[j][i] = c + i < p.C ? (f[j][i] - mean) * rstd : 0.f;
      a += g[j][i];
      b = fmaf(g[j][i], f[j][i], b);
    }
  }
  row_sum<WR>(a, b, sh[turn]);
  if (!there) continue;
  a /= (float)p.C;
  b /= (float)p.C;
  T *dx = (T *)p.out + r * p.C;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = (int64_t)(j * WR * 64 + l) * N;
    if (c >= p.C) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) f[j][i] = rstd * (g[j][i] - a - f[j][i] * b);
    store_piece<T, N>(dx, c, p.C, f[j]);
  }
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
    float f[N], w[N], a = 0.f, b = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * N; c < p.C; c += 1024 * N) {
      load_piece<T, N>(x, c, p.C, f);
#pragma unroll
      for (int i = 0; i < N; ++i) a += f[i];
    }
    row_sum<16>(a, b, sh[0]);
    float mean = a / n;
    a = b = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * N; c < p.C; c += 1024 * N) {
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
    for (int64_t c = (int64_t)threadIdx.x * N; c < p.C; c += 1024 * N) {
      load_piece<T, N>(x, c, p.C, f);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = (f[i] - mean - rest) * rstd;
      weigh<N>(p, c, f, w);
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
    auto at = [&](int64_t c, float (&f)[N], float (&g)[N]) {
      float w[N];
      load_piece<T, N>(x, c, p.C, f);
      load_piece<T, N>(dy, c, p.C, g);
      if (p.weight != nullptr) load_weights<N>(p.weight, p.w_dtype, c, p.C, w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (p.weight != nullptr) g[i] *= w[i];
        f[i] = c + i < p.C ? (f[i] - mean) * rstd : 0.f;
      }
    };
    for (int64_t c = (int64_t)threadIdx.x * N; c < p.C; c += 1024 * N) {
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
    for (int64_t c = (int64_t)threadIdx.x * N; c < p.C; c += 1024 * N) {
      float f[N], g[N];
      at(c, f, g);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = rstd * (g[i] - a - f[i] * b);
      store_piece<T, N>((T *)p.out + r * p.C, c, p.C, f);
    }
  }
}

// ---------------------------------------------------------------------------
// dweight and dbias: sums of groups of rows, then of the groups
// ---------------------------------------------------------------------------
constexpr int kNormGroups = 256;
static int64_t norm_groups(int64_t R) { return R < kNormGroups ? R : kNormGroups; }

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
// How many waves a row takes and how many pieces a lane of it has.
template <typename T, class K> static hipError_t by_width(const NormArgs &a, hipStream_t s) {
  const int64_t need = (a.C + 64 * kPiece<T> - 1) / (64 * kPiece<T>);  // pieces of 64 lanes
  if (need <= 1) return K::template rows<T, 4, 1, 1>(a, s);
  if (need <= 2) return K::template rows<T, 4, 1, 2>(a, s);
  if (need <= 4) return K::template rows<T, 4, 4, 1>(a, s);
  if (need <= 8) return K::template rows<T, 4, 4, 2>(a, s);
  if (need <= 16) return K::template rows<T, 4, 4, 4>(a, s);
  if (need <= 64) return K::template rows<T, 16, 16, 4>(a, s);
  return K::template wide<T>(a, s);
}
// workgroups for so many units of work (HIP counts a launch's threads in 32 bits; the kernels loop)
static dim3 norm_grid(int64_t n) { return dim3((unsigned)(n < (1 << 21) ? n : 1 << 21)); }

struct NormForward {
  template <typename T, int WAVES, int WR, int NV> static hipError_t rows(const NormArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((layer_norm_kernel<T, WAVES, WR, NV>), norm_grid((a.R + WAVES / WR - 1) / (WAVES / WR)), dim3(WAVES * 64),
                       0, s, a);
    return hipGetLastError();
  }
  template <typename T> static hipError_t wide(const NormArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(layer_norm_wide_kernel<T>, norm_grid(a.R), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
};
struct NormBackward {
  template <typename T, int WAVES, int WR, int NV> static hipError_t rows(const NormArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((layer_norm_dx_kernel<T, WAVES, WR, NV>), norm_grid((a.R + WAVES / WR - 1) / (WAVES / WR)),
                       dim3(WAVES * 64), 0, s, a);
    return hipGetLastError();
  }
  template <typename T> static hipError_t wide(const NormArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(layer_norm_wide_dx_kernel<T>, norm_grid(a.R), dim3(1024), 0, s, a);
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

size_t layer_norm_backward_workspace(int64_t R, int64_t C) { return (size_t)norm_groups(R) * 2 * (size_t)C * 4; }

template <typename T> static hipError_t backward_t(const NormArgs &a, hipStream_t s) {
  if (a.out != nullptr && a.R > 0) {
    const hipError_t e = by_width<T, NormBackward>(a, s);
    if (e != hipSuccess) return e;
  }
  if (a.dweight == nullptr && a.dbias == nullptr) return hipSuccess;
  float *parts = (float *)a.workspace;
  const int64_t groups = norm_groups(a.R), per = groups ? (a.R + groups - 1) / groups : 0;
  const int64_t used = groups ? (a.R + per - 1) / per : 0;
  if (groups > 0) {
    const dim3 grid((unsigned)((a.C + 256 * kPiece<T> - 1) / (256 * kPiece<T>)), (unsigned)used);
    hipLaunchKernelGGL(layer_norm_dw_kernel<T>, grid, dim3(256), 0, s, a, per, parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(layer_norm_join_kernel, dim3((unsigned)((2 * a.C + 63) / 64)), dim3(1024), 0, s, a, (int)used,
                     (const float *)parts);
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const NormArgs &a, hipStream_t s) {
  switch (a.dtype) {
    case NSG_F16: return backward_t<_Float16>(a, s);
    case NSG_BF16: return backward_t<__bf16>(a, s);
    default: return backward_t<float>(a, s);
  }
}

}  // namespace nsg
