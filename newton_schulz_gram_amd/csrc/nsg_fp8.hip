// 8-bit floating point operands with one fp32 scale for each block of 128, on
// gfx950.
//
//   s = max(amax / F, 2^-126),  q = RNE_8(x (1 / s)),  x ~ q s
// with amax the largest finite |x| of the block and F the type's largest value
// (448 for e4m3, 57344 for e5m2); amax / F, 1 / s and the product are one fp32
// operation each.  |x| (1 / s) exceeds F by 2^-22 relative at most, far less
// than half a step, so nothing saturates.  An infinity or NaN does not take
// part in amax: it becomes NaN (in e5m2 an infinity stays one) and reaches only
// the products it takes part in, while the rest of its block keeps its scale.
//
// A block is 128 elements of a row (activations, as the product contracts
// them), a 128 x 128 tile (weights: the same numbers then serve the product
// with the matrix and with its transpose, which is written in the same pass),
// or 128 rows of a column (operands of the weight gradients, which contract
// over rows; written transposed, each expert's rows starting at a multiple of
// 128 columns).  Rows of q are padded with zeros to a multiple of 128; scales
// are stored block index first, so that a product's tile reads consecutive ones.
//
// All three read x once and write q (1 byte) and s (1/32 byte).  Measured (bytes of the
// definition): rows 16384 x 11008 in 110 us, 5.0 TB/s; tiles with the transposed copy
// 512 x 2048 x 512 in 420 us, 5.1 TB/s, both at the copy rate; columns 131072 x 2048 of
// 512 experts in 212 us, 3.8 TB/s, 32771 x 2048 of 64 in 50 us, 4.1.  What keeps the
// columns from the copy rate is not shown; counted for the latter: 134 MB read, as by the
// definition, and 87 written for 69 (128-byte pieces of q_t's rows, which lie cap apart).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "nsg_expert.h"
#include "nsg_segments.h"

namespace nsg {

template <bool E4M3> __device__ __forceinline__ float f8_scale(float amax) {
  return fmaxf(amax / (E4M3 ? 448.f : 57344.f), 0x1p-126f);
}

// four values to four bytes, rounded to nearest even
template <bool E4M3> __device__ __forceinline__ uint32_t f8_pack(float a, float b, float c, float d) {
  int w = 0;
  if constexpr (E4M3) {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
  }
  return (uint32_t)w;
}

// 8 elements of a row as they are in memory, and their sizes: the bits without the
// sign, which order like the numbers, so that amax takes one `and` and one maximum
// per register (two 16-bit elements).  Sizes from kInf on are infinities and NaN.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
template <typename T> struct Eight {
  static constexpr int N = 4;  // registers
  typedef u16x2 reg;
  static constexpr uint32_t kInf = std::is_same<T, __bf16>::value ? 0x7F80u : 0x7C00u;
  reg d[4];
  static __device__ __forceinline__ reg size(reg v) { return v & (uint16_t)0x7FFF; }
  static __device__ __forceinline__ reg finite(reg v) { return reg{v[0] < kInf ? v[0] : (uint16_t)0, v[1] < kInf ? v[1] : (uint16_t)0}; }
  static __device__ __forceinline__ uint32_t largest(reg v) { return v[0] > v[1] ? v[0] : v[1]; }
  static __device__ __forceinline__ uint32_t of(const reg (&m)[N], int v) { return m[v >> 1][v & 1]; }
  static __device__ __forceinline__ float number(uint32_t bits) { return (float)__builtin_bit_cast(T, (uint16_t)bits); }
  __device__ __forceinline__ float value(int v) const { return number(d[v >> 1][v & 1]); }
  __device__ __forceinline__ void put(int v, T x) { d[v >> 1][v & 1] = __builtin_bit_cast(uint16_t, x); }
};
template <> struct Eight<float> {
  static constexpr int N = 8;
  typedef uint32_t reg;
  static constexpr uint32_t kInf = 0x7F800000u;
  reg d[8];
  static __device__ __forceinline__ reg size(reg v) { return v & 0x7FFFFFFFu; }
  static __device__ __forceinline__ reg finite(reg v) { return v < kInf ? v : 0u; }
  static __device__ __forceinline__ uint32_t largest(reg v) { return v; }
  static __device__ __forceinline__ uint32_t of(const reg (&m)[N], int v) { return m[v]; }
  static __device__ __forceinline__ float number(uint32_t bits) { return __uint_as_float(bits); }
  __device__ __forceinline__ float value(int v) const { return __uint_as_float(d[v]); }
  __device__ __forceinline__ void put(int v, float x) { d[v] = __float_as_uint(x); }
};

// Elements c .. c + 7 of a row of C, zeros behind it.  VEC: rows take 16-byte loads
// and C is a multiple of 8.
template <typename T, bool VEC> __device__ __forceinline__ Eight<T> load8(const T *row, int64_t c, int64_t C) {
  Eight<T> x = {};
  if constexpr (VEC) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if (c < C) {
      constexpr int Q = (int)sizeof(T) / 2;
      u32x4 q[Q];
#pragma unroll
      for (int h = 0; h < Q; ++h) q[h] = reinterpret_cast<const u32x4 *>(row + c)[h];
#pragma unroll
      for (int i = 0; i < Eight<T>::N; ++i) {
        const uint32_t word = q[i / 4][i % 4];  // (a cast of the element itself would take the vector's first)
        x.d[i] = __builtin_bit_cast(typename Eight<T>::reg, word);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < 8; ++v)
      if (c + v < C) x.put(v, row[c + v]);
  }
  return x;
}

// m = larger of m and the sizes of x
template <typename T> __device__ __forceinline__ void grow(typename Eight<T>::reg (&m)[Eight<T>::N], const Eight<T> &x) {
#pragma unroll
  for (int i = 0; i < Eight<T>::N; ++i) m[i] = __builtin_elementwise_max(m[i], Eight<T>::size(x.d[i]));
}
template <typename T> __device__ __forceinline__ uint32_t largest(const typename Eight<T>::reg (&m)[Eight<T>::N]) {
  typename Eight<T>::reg r = m[0];
#pragma unroll
  for (int i = 1; i < Eight<T>::N; ++i) r = __builtin_elementwise_max(r, m[i]);
  return Eight<T>::largest(r);
}
// Sizes of the finite elements of x[0 .. R - 1], column by column.
template <typename T, int R> __device__ __forceinline__ void sizes(typename Eight<T>::reg (&m)[Eight<T>::N], const Eight<T> (&x)[R]) {
#pragma unroll
  for (int i = 0; i < Eight<T>::N; ++i) m[i] = typename Eight<T>::reg(0);
#pragma unroll
  for (int r = 0; r < R; ++r) grow<T>(m, x[r]);
  if (largest<T>(m) >= Eight<T>::kInf) {  // rare: again without the infinities and NaN
#pragma unroll
    for (int i = 0; i < Eight<T>::N; ++i) m[i] = typename Eight<T>::reg(0);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < Eight<T>::N; ++i)
        m[i] = __builtin_elementwise_max(m[i], Eight<T>::finite(Eight<T>::size(x[r].d[i])));
  }
}

// ---------------------------------------------------------------------------
// Rows: 16 lanes per block of 128, 8 elements each; a workgroup takes 16 rows
// (so the scales of one block index leave as 64 bytes) and a.blocks blocks.
// ---------------------------------------------------------------------------
constexpr int kRowBlocks = 8;  // at most

template <typename T, bool VEC, bool E4M3>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs a) {
  const int l = threadIdx.x & 15;
  // x: parts of a row, which are read together (16384 x 11008: 110 us, 138 with the
  // groups of rows first); y and the rest of z: groups of 16 rows
  const int64_t g = blockIdx.z % a.B, r = (blockIdx.z / a.B * 65535 + blockIdx.y) * 16 + (threadIdx.x >> 4);
  if (r >= a.R) return;
  const int64_t Cp = up128(a.C), nb = Cp / kF8Block;
  const T *row = (const T *)a.x + (g * a.R + r) * a.ldx;
  uint8_t *q = (uint8_t *)a.q + (g * a.R + r) * Cp;
  const int64_t b0 = (int64_t)blockIdx.x * a.blocks, b1 = b0 + a.blocks < nb ? b0 + a.blocks : nb;
#pragma unroll 4
  for (int64_t b = b0; b < b1; ++b) {
    const int64_t c = b * kF8Block + l * 8;
    const Eight<T> x[1] = {load8<T, VEC>(row, c, a.C)};
    typename Eight<T>::reg m[Eight<T>::N];
    sizes<T>(m, x);
    uint32_t size = largest<T>(m);
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) size = max(size, (uint32_t)__shfl_xor((int)size, off, 16));
    const float s = f8_scale<E4M3>(Eight<T>::number(size)), inv = 1.f / s;
    float f[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) f[v] = x[0].value(v) * inv;
    uint2 w;
    w.x = f8_pack<E4M3>(f[0], f[1], f[2], f[3]);
    w.y = f8_pack<E4M3>(f[4], f[5], f[6], f[7]);
    *reinterpret_cast<uint2 *>(q + c) = w;
    if (l == 0) a.s[(g * nb + b) * a.R + r] = s;
  }
}

// ---------------------------------------------------------------------------
// Tiles and columns: a workgroup takes a 128 x 128 tile; thread (rg, cc) =
// (t / 16, t % 16) holds rows 8 rg .. + 7 and columns 8 cc .. + 7.  The tile's
// transposed copy goes through LDS (one row of 128 bytes per column, 144 apart
// so that rows keep 16-byte alignment).
// ---------------------------------------------------------------------------
constexpr int kTurnPitch = 144;

// w[i]: the 8 bytes of row 8 rg + i; afterwards o[v]: the 8 bytes of column 8 cc + v
__device__ __forceinline__ void turn8x8(const uint2 (&w)[8], uint2 (&o)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {      // columns 4 h .. 4 h + 3
#pragma unroll
    for (int u = 0; u < 2; ++u) {    // rows 4 u .. 4 u + 3
      const uint32_t r0 = h ? w[4 * u].y : w[4 * u].x, r1 = h ? w[4 * u + 1].y : w[4 * u + 1].x;
      const uint32_t r2 = h ? w[4 * u + 2].y : w[4 * u + 2].x, r3 = h ? w[4 * u + 3].y : w[4 * u + 3].x;
      // v_perm_b32 selects bytes of {first, second}: 0-3 the second's, 4-7 the first's
      const uint32_t a01 = __builtin_amdgcn_perm(r1, r0, 0x05010400u);  // r0.0 r1.0 r0.1 r1.1
      const uint32_t b01 = __builtin_amdgcn_perm(r1, r0, 0x07030602u);  // r0.2 r1.2 r0.3 r1.3
      const uint32_t a23 = __builtin_amdgcn_perm(r3, r2, 0x05010400u);
      const uint32_t b23 = __builtin_amdgcn_perm(r3, r2, 0x07030602u);
      const uint32_t c0 = __builtin_amdgcn_perm(a23, a01, 0x05040100u), c1 = __builtin_amdgcn_perm(a23, a01, 0x07060302u);
      const uint32_t c2 = __builtin_amdgcn_perm(b23, b01, 0x05040100u), c3 = __builtin_amdgcn_perm(b23, b01, 0x07060302u);
      if (u == 0) {
        o[4 * h].x = c0; o[4 * h + 1].x = c1; o[4 * h + 2].x = c2; o[4 * h + 3].x = c3;
      } else {
        o[4 * h].y = c0; o[4 * h + 1].y = c1; o[4 * h + 2].y = c2; o[4 * h + 3].y = c3;
      }
    }
  }
}

// this thread's 8 x 8 bytes into LDS, column by column; then row c of the
// turned tile goes to dst + c ld for the `cols` columns that there are
__device__ __forceinline__ void store_turned(const uint2 (&w)[8], unsigned char *lds, uint8_t *dst, int64_t ld, int cols) {
  const int cc = threadIdx.x & 15, rg = threadIdx.x >> 4;
  uint2 o[8];
  turn8x8(w, o);
#pragma unroll
  for (int v = 0; v < 8; ++v) *reinterpret_cast<uint2 *>(lds + (8 * cc + v) * kTurnPitch + 8 * rg) = o[v];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 8 lanes per row, 16 bytes each
    const int c = i * 32 + (threadIdx.x >> 3), part = threadIdx.x & 7;
    if (c < cols)
      *reinterpret_cast<uint4 *>(dst + c * ld + 16 * part) = *reinterpret_cast<const uint4 *>(lds + c * kTurnPitch + 16 * part);
  }
}

template <typename T, bool VEC, bool E4M3>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const QuantArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char lds[128 * kTurnPitch];
  __shared__ uint32_t wmax[4];
  const int cc = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int64_t tc = blockIdx.x, tr = blockIdx.y, g = blockIdx.z;
  const int64_t Cp = up128(a.C), Rp = up128(a.R), nbc = Cp / kF8Block, nbr = Rp / kF8Block;
  const int64_t r0 = tr * 128 + rg * 8, c = tc * 128 + cc * 8;
  const T *x = (const T *)a.x + g * a.R * a.ldx;
  Eight<T> f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = r0 + i < a.R ? load8<T, VEC>(x + (r0 + i) * a.ldx, c, a.C) : Eight<T>{};
  typename Eight<T>::reg m[Eight<T>::N];
  sizes<T>(m, f);
  uint32_t size = largest<T>(m);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) size = max(size, (uint32_t)__shfl_xor((int)size, off, 64));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = size;
  __syncthreads();
  size = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const float s = f8_scale<E4M3>(Eight<T>::number(size)), inv = 1.f / s;
  uint2 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = f[i].value(k) * inv;
    w[i].x = f8_pack<E4M3>(v[0], v[1], v[2], v[3]);
    w[i].y = f8_pack<E4M3>(v[4], v[5], v[6], v[7]);
    if (r0 + i < a.R) *reinterpret_cast<uint2 *>((uint8_t *)a.q + (g * a.R + r0 + i) * Cp + c) = w[i];
  }
  if (threadIdx.x == 0) {
    a.s[(g * nbc + tc) * nbr + tr] = s;
    if (a.qt) a.st[(g * nbr + tr) * nbc + tc] = s;
  }
  if (a.qt) {
    const int64_t left = a.C - tc * 128;
    store_turned(w, lds, (uint8_t *)a.qt + (g * a.C + tc * 128) * Rp + tr * 128, Rp, left < 128 ? (int)left : 128);
  }
}

// Columns: a workgroup takes one of all experts' blocks of 128 rows and every
// a.share-th of its column tiles; blocks behind the last expert's
// are written as zeros with the smallest scale, as an expert's unused places are.
template <typename T, bool VEC, bool E4M3>
__global__ void __launch_bounds__(256) quantize_columns_kernel(const QuantArgs a) {
  const unsigned blocks = (unsigned)a.blocks;
  __shared__ __attribute__((aligned(16))) unsigned char lds[128 * kTurnPitch];
  __shared__ typename Eight<T>::reg cmax[4][16][Eight<T>::N];
  __shared__ int sh[8];
  // workgroup b runs on XCD b % 8: each XCD takes consecutive blocks, whose rows of
  // q_t are neighbours, and the workgroups that share a block's rows run together
  const unsigned share = (unsigned)a.share, q = blockIdx.x >> 3;
  const unsigned per = (blocks + 7) / 8, block = (blockIdx.x & 7) * per + q / share;
  if (q / share >= per || block >= blocks) return;
  const Segment seg = find_unit<256>(a.offsets, a.E, (int)a.P, kF8Block, (int)block, sh);
  const int cc = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int64_t cap = kF8Block * (int64_t)blocks;
  const int64_t tiles = (a.C + 127) / 128;
  const int left = seg.expert < 0 ? 0 : seg.len - seg.unit * kF8Block;  // rows of this block
  int64_t row[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    row[i] = -1;
    if (rg * 8 + i < left) {
      row[i] = seg.begin + seg.unit * kF8Block + rg * 8 + i;
      if (a.tokens) row[i] = a.tokens[row[i]];
      if (row[i] >= a.R) row[i] = -1;
    }
  }
  for (int64_t tc = q % share; tc < tiles; tc += share) {
    const int64_t c = tc * 128 + cc * 8;
    Eight<T> f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = row[i] >= 0 ? load8<T, VEC>((const T *)a.x + row[i] * a.ldx, c, a.C) : Eight<T>{};
    typename Eight<T>::reg m[Eight<T>::N];
    sizes<T>(m, f);
#pragma unroll
    for (int off = 16; off <= 32; off <<= 1)
#pragma unroll
      for (int i = 0; i < Eight<T>::N; ++i)
        m[i] = __builtin_elementwise_max(
            m[i], __builtin_bit_cast(typename Eight<T>::reg, __shfl_xor(__builtin_bit_cast(int, m[i]), off, 64)));
    if ((threadIdx.x & 63) < 16) {
#pragma unroll
      for (int i = 0; i < Eight<T>::N; ++i) cmax[wave][cc][i] = m[i];
    }
    __syncthreads();  // also: the previous tile's turned rows have left LDS
#pragma unroll
    for (int i = 0; i < Eight<T>::N; ++i)
      m[i] = __builtin_elementwise_max(__builtin_elementwise_max(cmax[0][cc][i], cmax[1][cc][i]),
                                       __builtin_elementwise_max(cmax[2][cc][i], cmax[3][cc][i]));
    float inv[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const float s = f8_scale<E4M3>(Eight<T>::number(Eight<T>::of(m, v)));
      inv[v] = 1.f / s;
      if (rg == 0 && c + v < a.C) a.st[(int64_t)block * a.C + c + v] = s;
    }
    uint2 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = f[i].value(k) * inv[k];
      w[i].x = f8_pack<E4M3>(v[0], v[1], v[2], v[3]);
      w[i].y = f8_pack<E4M3>(v[4], v[5], v[6], v[7]);
    }
    const int64_t cols = a.C - tc * 128;
    store_turned(w, lds, (uint8_t *)a.qt + tc * 128 * cap + (int64_t)block * kF8Block, cap, cols < 128 ? (int)cols : 128);
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// 8 elements of every row take 16-byte loads
static bool vec8(const QuantArgs &a) {
  const int64_t per = a.x_dtype == NSG_F32 ? 4 : 8;
  return reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % per == 0 && a.C % 8 == 0;
}

#define NSG_QUANT(KERNEL, grid)                                                                            \
  do {                                                                                                     \
    const bool vec = vec8(a), e4 = a.f8 == NSG_F8E4M3;                                                     \
    switch (a.x_dtype) {                                                                                   \
      case NSG_F16: NSG_QUANT_T(KERNEL, grid, _Float16); break;                                            \
      case NSG_BF16: NSG_QUANT_T(KERNEL, grid, __bf16); break;                                             \
      default: NSG_QUANT_T(KERNEL, grid, float); break;                                                    \
    }                                                                                                      \
  } while (0)
#define NSG_QUANT_T(KERNEL, grid, T)                                                                       \
  if (vec && e4) hipLaunchKernelGGL((KERNEL<T, true, true>), grid, dim3(256), 0, s, a);                    \
  else if (vec) hipLaunchKernelGGL((KERNEL<T, true, false>), grid, dim3(256), 0, s, a);                    \
  else if (e4) hipLaunchKernelGGL((KERNEL<T, false, true>), grid, dim3(256), 0, s, a);                     \
  else hipLaunchKernelGGL((KERNEL<T, false, false>), grid, dim3(256), 0, s, a)

hipError_t launch_quantize_rows(const QuantArgs &args, hipStream_t s) {
  QuantArgs a = args;
  const int64_t nb = up128(a.C) / kF8Block, groups = (a.R + 15) / 16 * a.B;
  // a block each where there are few: 64 x 4096 in 2.5 us against 5.8
  a.blocks = groups * nb / 1024;
  a.blocks = a.blocks < 1 ? 1 : a.blocks > kRowBlocks ? kRowBlocks : a.blocks;
  const int64_t rows = (a.R + 15) / 16, z = (rows + 65534) / 65535;
  if (z * a.B > 65535) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)((nb + a.blocks - 1) / a.blocks), (unsigned)(rows < 65535 ? rows : 65535), (unsigned)(z * a.B));
  NSG_QUANT(quantize_rows_kernel, grid);
  return hipGetLastError();
}

hipError_t launch_quantize_tiles(const QuantArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)(up128(a.C) / 128), (unsigned)(up128(a.R) / 128), (unsigned)a.B);
  NSG_QUANT(quantize_tiles_kernel, grid);
  return hipGetLastError();
}

hipError_t launch_quantize_columns(const QuantArgs &args, hipStream_t s) {
  QuantArgs a = args;
  a.blocks = a.P / kF8Block + a.E;
  const int64_t tiles = (a.C + 127) / 128;
  // 4 workgroups share a block's column tiles, more where there are few blocks: each
  // has to find its expert (1000 rows of 8 experts, C = 1024: 6.6 us with 8 (all), 9.6 with 4;
  // 131072 rows of 512, C = 2048: 248 us with 16, 211 with 4)
  const int64_t y = (2048 + a.blocks - 1) / a.blocks;
  a.share = y < 4 ? 4 : y;
  if (a.share > tiles) a.share = tiles;
  const dim3 grid((unsigned)((a.blocks + 7) / 8 * 8 * a.share));
  NSG_QUANT(quantize_columns_kernel, grid);
  return hipGetLastError();
}

}  // namespace nsg
