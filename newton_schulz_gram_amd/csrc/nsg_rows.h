// Rows of fp16, bf16 or fp32 elements read and written a few consecutive elements
// to a lane, as fp32.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

namespace nsg {

static inline bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// V consecutive elements.  ALIGN: bytes that they are aligned to (the
// instructions take any).
template <typename T, int V, int ALIGN = V * (int)sizeof(T)> struct Row {
  typedef T vec __attribute__((ext_vector_type(V)));
  typedef vec mem __attribute__((aligned(ALIGN)));
  static __device__ __forceinline__ void load(const T *p, float (&f)[V]) {
    const vec x = *reinterpret_cast<const mem *>(p);
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = (float)x[v];
  }
  static __device__ __forceinline__ void store(T *p, const float (&f)[V]) {
    vec x;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = (T)f[v];
    *reinterpret_cast<mem *>(p) = x;
  }
};
template <typename T, int ALIGN> struct Row<T, 1, ALIGN> {
  static __device__ __forceinline__ void load(const T *p, float (&f)[1]) { f[0] = (float)*p; }
  static __device__ __forceinline__ void store(T *p, const float (&f)[1]) { *p = (T)f[0]; }
};

// ---------------------------------------------------------------------------
// Sums over the 64 lanes, the same in all of them: within rows of 16 lanes, then over
// the rows, by data-parallel moves between lanes (no LDS).
// ---------------------------------------------------------------------------
template <int CTRL, int ROWS> __device__ __forceinline__ float lanes_moved(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, ROWS == 0xf));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += lanes_moved<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8: zeros come in
  v += lanes_moved<0x112, 0xf>(v);
  v += lanes_moved<0x114, 0xf>(v);
  v += lanes_moved<0x118, 0xf>(v);
  v += lanes_moved<0x142, 0xa>(v);  // lane 15 of a row to the next one (rows 1 and 3; the others add 0)
  v += lanes_moved<0x143, 0xc>(v);  // lane 31 to rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Sums over groups of L lanes, L a power of two of at least 4, the same in all lanes of a
// group: both lanes of a pair join the same two values
template <int L> __device__ __forceinline__ float group_lanes_sum(float v) {
  if (L == 64) return wave_sum(v);
  v += lanes_moved<0xB1, 0xf>(v);  // lanes 1, 0, 3, 2 of four
  v += lanes_moved<0x4E, 0xf>(v);  // lanes 2, 3, 0, 1
  if (L >= 8) v += lanes_moved<0x141, 0xf>(v);  // eight lanes mirrored
  if (L >= 16) v += lanes_moved<0x140, 0xf>(v);  // sixteen
  if (L >= 32) {
    const unsigned x = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);  // the values of two rows of 16
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

}  // namespace nsg
