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

}  // namespace nsg
