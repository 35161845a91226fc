// Which expert a workgroup works for: the rows of the experts lie behind each
// other (offsets [E + 1] on the device, so the host knows no lengths), each
// expert's rows are cut into units of `unit` rows, and a launch has as many
// workgroups as there can be units.
//
// Offsets are device data: they are clamped to 0 <= begin <= end <= P here, so
// that no offsets, however wrong, take a kernel out of its buffers.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "nsg.h"

namespace nsg {

struct Segment {
  int expert;  // -1: no such unit
  int begin;   // first row of the expert
  int len;     // its rows
  int unit;    // index of the unit inside the expert
};

__device__ __forceinline__ int seg_clamp(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// the expert's clamped rows
__device__ __forceinline__ void seg_bounds(const int32_t *offsets, int e, int P, int &begin, int &end) {
  begin = seg_clamp(offsets[e], 0, P);
  end = seg_clamp(offsets[e + 1], begin, P);
}

// Sum of v over the threads before this one, and the total (NT threads).
// `sh`: NT / 64 + 1 ints of LDS.
template <int NT> __device__ __forceinline__ int block_before(int v, int *sh, int &total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  if (lane == 63) sh[wave] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    const int t = sh[w];
    if (w < wave) before += t;
    total += t;
  }
  __syncthreads();
  return before + x - v;
}

// The unit `target` of all experts' units, counted through the experts in
// order; with `tail` the rows behind offsets[E] follow as expert E's.  Every
// thread of the workgroup calls it; `sh`: NT / 64 + 4 ints of LDS.
template <int NT>
__device__ __forceinline__ Segment find_unit(const int32_t *offsets, int E, int P, int unit, int target, int *sh,
                                             bool tail = false) {
  // a thread's experts, loaded once, all loads together
  constexpr int kMost = (NSG_MAX_EXPERTS + 1 + NT - 1) / NT;
  const int all = E + (tail ? 1 : 0);
  const int per = (all + NT - 1) / NT, e0 = (int)threadIdx.x * per;
  int begin[kMost], len[kMost], mine = 0;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    begin[i] = len[i] = 0;
    if (i < per && e0 + i < all) {
      int end = P;
      if (e0 + i < E) seg_bounds(offsets, e0 + i, P, begin[i], end);
      else begin[i] = seg_clamp(offsets[E], 0, P);
      len[i] = end - begin[i];
    }
    mine += (len[i] + unit - 1) / unit;
  }
  int *res = sh + NT / 64;
  if (threadIdx.x == 0) res[0] = -1;
  int total;
  int at = block_before<NT>(mine, sh, total);
  if (target >= at && target < at + mine) {
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int u = (len[i] + unit - 1) / unit;
      if (target >= at && target < at + u) {
        res[0] = e0 + i;
        res[1] = begin[i];
        res[2] = len[i];
        res[3] = target - at;
      }
      at += u;
    }
  }
  __syncthreads();
  Segment s;
  s.expert = __builtin_amdgcn_readfirstlane(res[0]);
  s.begin = __builtin_amdgcn_readfirstlane(res[1]);
  s.len = __builtin_amdgcn_readfirstlane(res[2]);
  s.unit = __builtin_amdgcn_readfirstlane(res[3]);
  __syncthreads();
  return s;
}

// Units of the experts before `expert`.  Every thread of the workgroup calls it.
template <int NT>
__device__ __forceinline__ int units_before(const int32_t *offsets, int P, int unit, int expert, int *sh) {
  int mine = 0;
  for (int e = threadIdx.x; e < expert; e += NT) {
    int b, n;
    seg_bounds(offsets, e, P, b, n);
    mine += (n - b + unit - 1) / unit;
  }
  int total;
  block_before<NT>(mine, sh, total);
  return __builtin_amdgcn_readfirstlane(total);
}

}  // namespace nsg
