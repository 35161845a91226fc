// Products of 8-bit operands with a scale for each block of 128, on gfx950:
//
//   out[m, n] = sum_b sa[b, m] sb[b, n] sum_{k in block b} A[m, k] B[n, k]
//
// A holds tokens (or output gradients), B weights (or activations).  The outer
// sum is one fp32 fused multiply-add per block and element, on the VALU, while
// the matrix cores run the next block.  Scales may be any fp32 numbers; what is done
// where the product of two leaves fp32's range stands at not_finite below.
//
// The inner sum of a block starts from zero, in one of two ways:
//   16-bit outputs: one v_mfma_f32_16x16x128_f8f6f4.  Its sums are fp32, but
//     inside each group of 8 consecutive k it first cuts the products off at
//     2^-13 of the largest one's power of two (found by probing pairs of products;
//     the 16x16x32 and 32x32x64 8-bit instructions do the same): an error below
//     7 * 2^-13 of the group's largest product.  On normal values the result is off
//     by 1.3e-5 relative, 1/300 of a bf16 rounding and 1/37 of an f16 one; twice the
//     matrix rate of exact sums is taken for that.  Where large products of different
//     groups cancel the error stays relative to them, as the header says.
//   fp32 outputs: four v_mfma_f32_16x16x32_bf16 on the operands converted to bf16,
//     which holds every 8-bit value: products exact, sums fp32 (1e-8 relative by
//     the same probe), half the matrix rate.
//
// The MFMA's rows are B's rows and its columns A's: a lane then holds one token
// (one scale sa per fragment) and four consecutive n, and with the row order
// that stage loads give B in LDS, 16 consecutive n of its token, which leave as
// 16-byte stores.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "nsg_expert.h"
#include "nsg_segments.h"

namespace nsg {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) unsigned char *lds_u8_t;

// One direct global -> LDS load of 16 (4) bytes per lane: lane l's go to
// lds + 16 l (4 l).  Issued as inline assembly so that the compiler does not
// wait for it before unrelated LDS reads: the kernel waits itself.
// `lds`: byte address in LDS, the same in every lane; nothing is loaded where `on`
// is 0.  The branch is inside the assembly so that the main loop stays one basic
// block, whose instruction order the scheduling barriers keep.
// The source is a 64-bit address in every lane, or a 32-bit offset to a base.
// The two instructions between the write of m0 and the load are the wait state that
// an LDS load needs there; the compiler adds none inside assembly.
#define NSG_DMA(WIDTH)                                                                                           \
  asm volatile("s_mov_b32 m0, %1\n\ts_cmp_eq_u32 %2, 0\n\ts_cbranch_scc1 .Lno%=\n\tglobal_load_lds_" WIDTH       \
               " %0, off\n.Lno%=:" ::"v"(src), "s"(lds), "s"(on) : "memory", "scc", "m0")
#define NSG_DMA_BASE(WIDTH)                                                                                      \
  asm volatile("s_mov_b32 m0, %1\n\ts_cmp_eq_u32 %2, 0\n\ts_cbranch_scc1 .Lno%=\n\tglobal_load_lds_" WIDTH       \
               " %0, %3\n.Lno%=:" ::"v"(off), "s"(lds), "s"(on), "s"(base) : "memory", "scc", "m0")
__device__ __forceinline__ void dma16(const void *src, unsigned lds, int on) { NSG_DMA("dwordx4"); }
__device__ __forceinline__ void dma16(uint64_t base, unsigned off, unsigned lds, int on) { NSG_DMA_BASE("dwordx4"); }
__device__ __forceinline__ void dma4(uint64_t base, unsigned off, unsigned lds, int on) { NSG_DMA_BASE("dword"); }
#undef NSG_DMA
#undef NSG_DMA_BASE
// an address that is the same in every lane, in scalar registers
__device__ __forceinline__ uint64_t uniform(const void *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return (uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((unsigned)(v >> 32)) << 32 |
         (unsigned)__builtin_amdgcn_readfirstlane((unsigned)v);
}
// All but the last N of this wave's loads have landed (all of them where `on` is
// 0) and its LDS reads have returned; then every other wave's too.
template <int N> __device__ __forceinline__ void landed_barrier(int on) {
  asm volatile("s_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 .Lall%=\n\ts_waitcnt vmcnt(%1)\n\ts_branch .Lgo%=\n"
               ".Lall%=:\n\ts_waitcnt vmcnt(0)\n.Lgo%=:\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier"
               ::"s"(on), "n"(N) : "memory", "scc");
}
// This wave's LDS reads have returned, and every other wave's.
__device__ __forceinline__ void read_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A fragment: 16 rows x 128 k, lane l holding 32 k of row l % 16 (the same 32 for
// A and B, so their order does not matter).  F: 1 for e5m2, 0 for e4m3; WIDE:
// held in bf16.
template <int F, bool WIDE> struct Frag {
  i32x8 v;
  __device__ __forceinline__ void set(i32x4 lo, i32x4 hi) { v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
};
template <int F> struct Frag<F, true> {
  bf16x8 v[4];
  static __device__ __forceinline__ bf16x2 pair(int w, bool high) {
    if constexpr (F) return high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.f, true) : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.f, false);
    else return high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true) : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
  }
  static __device__ __forceinline__ bf16x8 eight(int x, int y) {
    const bf16x2 a = pair(x, false), b = pair(x, true), c = pair(y, false), d = pair(y, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  __device__ __forceinline__ void set(i32x4 lo, i32x4 hi) {
    v[0] = eight(lo[0], lo[1]);
    v[1] = eight(lo[2], lo[3]);
    v[2] = eight(hi[0], hi[1]);
    v[3] = eight(hi[2], hi[3]);
  }
};
template <int FA, int FB> __device__ __forceinline__ f32x4 mma(const Frag<FB, false> &b, const Frag<FA, false> &a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, f32x4{0.f, 0.f, 0.f, 0.f}, FB, FA, 0, 0, 0, 0);
}
template <int FA, int FB> __device__ __forceinline__ f32x4 mma(const Frag<FB, true> &b, const Frag<FA, true> &a) {
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[i], a.v[i], d, 0, 0, 0);
  return d;
}

// 8 consecutive elements of an output row, of which the first `cols` exist
template <typename T> __device__ __forceinline__ void store8(T *dst, const float (&v)[8], int64_t cols, bool vec) {
  constexpr int V = 16 / (int)sizeof(T);
  typedef T vec_t __attribute__((ext_vector_type(V)));
  if (vec && cols >= 8) {
#pragma unroll
    for (int h = 0; h < 8 / V; ++h) {
      vec_t x;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = (T)v[h * V + i];
      *reinterpret_cast<vec_t *>(dst + h * V) = x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cols) dst[i] = (T)v[i];
  }
}
__device__ __forceinline__ void store8(void *out, int dtype, int64_t at, const float (&v)[8], int64_t cols, bool vec) {
  if (dtype == NSG_BF16) store8((__bf16 *)out + at, v, cols, vec);
  else if (dtype == NSG_F16) store8((_Float16 *)out + at, v, cols, vec);
  else store8((float *)out + at, v, cols, vec);
}

template <typename T> __device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  typedef T vec_t __attribute__((ext_vector_type(8)));
  vec_t x;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (T)v[i];
  return __builtin_bit_cast(u32x4, x);
}

// 4 consecutive elements, likewise
template <typename T> __device__ __forceinline__ void store4(T *dst, f32x4 v, int64_t cols, bool vec) {
  if (vec) {
    typedef T vec_t __attribute__((ext_vector_type(4)));
    *reinterpret_cast<vec_t *>(dst) = vec_t{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cols) dst[i] = (T)v[i];
  }
}
__device__ __forceinline__ void store4(void *out, int dtype, int64_t at, f32x4 v, int64_t cols, bool vec) {
  if (dtype == NSG_BF16) store4((__bf16 *)out + at, v, cols, vec);
  else if (dtype == NSG_F16) store4((_Float16 *)out + at, v, cols, vec);
  else store4((float *)out + at, v, cols, vec);
}

// What a workgroup computes: BM rows of A from m0 (kExperts: rows m0 .. m1 of
// the output) against rows n0 .. of B, over nkb blocks.
struct Work {
  const uint8_t *A, *B;   // first block
  const float *sa, *sb;   // scales of the first block
  int64_t ka, kb;         // scales of one block index of A, of B
  int64_t m0, m1, n0;     // rows of the output, and behind the last of them
  int64_t out;            // element offset of the output matrix
  int nkb;
  bool zero;              // rows behind the last expert's
};

// Tile order.  Workgroup b runs on XCD b % 8, and each XCD has an L2 of its own.
//   kDense: each XCD takes runs of 32 consecutive tiles; consecutive tiles go
//     down 4 rows of tiles, then on to the next column.
//   kExperts, kWgrad: the tiles that share an expert's rows are on one XCD.
// Returns false where the workgroup has nothing to do.
template <int BM, int BN, int NT>
__device__ __forceinline__ bool find_work(const F8GemmArgs &p, int *sh, Work &w) {
  const int64_t nkb = p.K / kF8Block;
  const unsigned tn_all = (unsigned)((p.N + BN - 1) / BN);
  const unsigned xcd = blockIdx.x & 7, q = blockIdx.x >> 3;
  w.ka = p.a_tile ? (p.M + 127) / 128 : p.M;
  w.kb = p.b_tile ? (p.N + 127) / 128 : p.N;
  w.zero = false;
  w.nkb = (int)nkb;
  if (p.mode == kDense) {
    const unsigned tm_all = (unsigned)((p.M + BM - 1) / BM);
    const unsigned per = tm_all * tn_all, total = per * (unsigned)p.batch;
    const unsigned run = total >= 256 ? 32 : (total + 7) / 8;
    const unsigned o = (q / run) * run * 8 + xcd * run + q % run;
    if (o >= total) return false;
    const unsigned g = o / per, t = o - g * per;
    const unsigned strip = 4 * tn_all, r0 = t / strip * 4, in = t % strip;
    const unsigned h = min(4u, tm_all - r0);
    const unsigned tm = r0 + in % h, tn = in / h;
    w.A = (const uint8_t *)p.A + g * p.M * p.K;
    w.B = (const uint8_t *)p.B + g * p.N * p.K;
    w.sa = p.sa + g * nkb * w.ka;
    w.sb = p.sb + g * nkb * w.kb;
    w.m0 = (int64_t)tm * BM;
    w.m1 = min(p.M, w.m0 + BM);
    w.n0 = (int64_t)tn * BN;
    w.out = (int64_t)g * p.M * p.N;
    return true;
  }
  if (p.mode == kExperts) {
    const unsigned u = q / tn_all * 8 + xcd;
    w.n0 = (int64_t)(q % tn_all) * BN;
    const Segment seg = find_unit<NT>(p.offsets, p.E, (int)p.M, BM, (int)u, sh, true);
    if (seg.expert < 0) return false;
    w.zero = seg.expert == p.E;
    const int64_t e = w.zero ? 0 : seg.expert;
    w.ka = p.a_tile ? (p.T + 127) / 128 : p.T;
    w.A = (const uint8_t *)p.A;
    w.B = (const uint8_t *)p.B + e * p.N * p.K;
    w.sa = p.sa;
    w.sb = p.sb + e * nkb * w.kb;
    w.m0 = seg.begin + (int64_t)seg.unit * BM;
    w.m1 = min((int64_t)seg.begin + seg.len, w.m0 + BM);
    w.out = 0;
    if (w.zero) w.nkb = 0;
    return true;
  }
  const unsigned tm_all = (unsigned)((p.M + BM - 1) / BM), per = tm_all * tn_all;
  const int64_t e = (int64_t)(q / per) * 8 + xcd;
  if (e >= p.E) return false;
  const unsigned t = q % per;
  int begin, end;
  seg_bounds(p.offsets, (int)e, (int)p.T, begin, end);
  const int b0 = units_before<NT>(p.offsets, (int)p.T, kF8Block, (int)e, sh);
  const int64_t first = min((int64_t)b0, nkb);
  w.nkb = (int)min((int64_t)((end - begin + kF8Block - 1) / kF8Block), nkb - first);
  w.A = (const uint8_t *)p.A + first * kF8Block;
  w.B = (const uint8_t *)p.B + first * kF8Block;
  w.sa = p.sa + first * w.ka;
  w.sb = p.sb + first * w.kb;
  w.m0 = (int64_t)(t / tn_all) * BM;
  w.m1 = min(p.M, w.m0 + BM);
  w.n0 = (int64_t)(t % tn_all) * BN;
  w.out = e * p.M * p.N;
  return true;
}

// The row of A behind row m of the output (m below m1), and whether there is one.
__device__ __forceinline__ int64_t row_of_a(const F8GemmArgs &p, int64_t m, bool &there) {
  if (p.mode != kExperts) return m;
  const int64_t r = p.tokens ? p.tokens[m] : m;
  there = r >= 0 && r < p.T;
  return there ? r : 0;
}

// ---------------------------------------------------------------------------
// Scales whose product is past the largest fp32 number.  The kernels below multiply a
// block's sum d by sa sb, formed first: one product serves a row of a tile, and a large
// scale with a small one stays in range.  Where both are so large that sa sb is
// infinite, d = 0 gives NaN and a small d infinity, whatever the result; the output is
// not finite then in any case, since no later block brings it back.  So each kernel
// looks at its outputs once at the end (not_finite), and where one is not finite and
// the scales can be the cause, the wave computes its outputs again with (d sa) sb:
// both factors are above 1 there, so d sa is infinite only where the result is.
// (The looks cost the weight gradients of 512 experts 464 -> 466 us, the others nothing;
// with a NaN in every row 8192 x 4096 x 11008 takes 288 -> 289 us, 8192 x 4096 x 4096
// with row scales of B, where all scales of A are read again, 133 -> 149.
// The loops below are not unrolled: they hardly ever run, and unrolled they changed the
// registers of the kernels around them, 256 x 4096 x 4096 15.6 -> 15.8 us.)
// A product sa sb below 2^-126 is rounded to a multiple of 2^-149 and changes a block's
// part of the output by at most 2^-150 |d|, below 2^-111 (e5m2) or 2^-125 (e4m3).
// ---------------------------------------------------------------------------
// seen = largest size of the values that it was called with, NaN where one was among
// them (one v_maximum3 for two values)
__device__ __forceinline__ void look_at(float a, float b, float &seen) {
  seen = __builtin_elementwise_maximum(__builtin_elementwise_maximum(seen, __builtin_fabsf(a)), __builtin_fabsf(b));
}
__device__ __forceinline__ bool not_finite(float seen) { return __builtin_expect(__any(!(seen < __builtin_inff())), 0); }

// Whether scales of rows m .. m + rows - 1 and n .. n + cols - 1 can have an infinite
// product: first the side with fewer scales, and where none of them is above 1, no.
__device__ __forceinline__ bool scales_overflow(const F8GemmArgs &p, const Work &w, int64_t m, int rows, int64_t n, int cols) {
  const int lane = threadIdx.x & 63;
  float both = 1.f;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const bool of_b = (side == 0) == (p.b_tile != 0), tile = of_b ? p.b_tile : p.a_tile;
    const float *scales = of_b ? w.sb : w.sa;
    const int64_t ld = of_b ? w.kb : w.ka;
    const int first = (int)(of_b ? n : m), last = (int)(of_b ? min(n + cols, p.N) : min(m + rows, w.m1)) - 1;
    float top = 0.f;
    // tile scales: a lane takes every 64th block; row scales: a row
    const int i0 = tile ? min(first, last) >> 7 : first + lane, i1 = tile ? last >> 7 : last;
#pragma unroll 1
    for (int i = i0; i <= i1; i += tile ? 1 : 64) {
      bool there = true;
      const float *s = scales + (tile || of_b ? i : row_of_a(p, i, there));
#pragma unroll 1
      for (int kb = tile ? lane : 0; kb < w.nkb; kb += tile ? 64 : 1) top = fmaxf(top, fabsf(s[kb * ld]));
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    if (!(top > 1.f)) return false;
    both *= top;
  }
  return both > 0x1.fffffep127f;
}

// The 16 x 16 outputs from row m and column n, straight from memory, block by block in
// order as the tile and deep kernels add them.
template <int FA, int FB, bool WIDE>
__device__ __forceinline__ void compute_again(const F8GemmArgs &p, const Work &w, int64_t m, int64_t n) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  bool there = true;
  const int64_t row = row_of_a(p, min(m + r16, w.m1 - 1), there);
  const uint8_t *a = w.A + row * p.K + 16 * g, *b = w.B + min(n + r16, p.N - 1) * p.K + 16 * g;
  m += r16;
  n += 4 * g;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int64_t kb = 0; kb < w.nkb; ++kb) {
    Frag<FA, WIDE> fa;
    Frag<FB, WIDE> fb;
    fa.set(*reinterpret_cast<const i32x4 *>(a + kb * kF8Block), *reinterpret_cast<const i32x4 *>(a + kb * kF8Block + 64));
    fb.set(*reinterpret_cast<const i32x4 *>(b + kb * kF8Block), *reinterpret_cast<const i32x4 *>(b + kb * kF8Block + 64));
    const f32x4 d = mma<FA, FB>(fb, fa);
    const float sa = w.sa[kb * w.ka + (p.a_tile ? row >> 7 : row)];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t c = min(n + v, p.N - 1);
      const float sb = w.sb[kb * w.kb + (p.b_tile ? c >> 7 : c)], x = sa * sb;
      const bool past = __builtin_isinf(x) && !__builtin_isinf(sa) && !__builtin_isinf(sb);
      acc[v] = fmaf(past ? d[v] * sa : d[v], past ? sb : x, acc[v]);
    }
  }
  if (m >= w.m1 || n >= p.N) return;
  if (!there) acc = f32x4{0.f, 0.f, 0.f, 0.f};
  store4(p.out, p.out_dtype, w.out + m * p.N + n, acc, p.N - n, false);
}

// A wave's 16 MF x 16 NF outputs from row m and column n, already stored, of which one was
// not finite.
template <int MF, int NF, int FA, int FB, bool WIDE>
__device__ __forceinline__ void mend(const F8GemmArgs &p, const Work &w, int64_t m, int64_t n) {
  if (!scales_overflow(p, w, m, 16 * MF, n, 16 * NF)) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // other lanes stored what this one stores now
#pragma unroll 1
  for (int f = 0; f < MF * NF; ++f) compute_again<FA, FB, WIDE>(p, w, m + 16 * (f % MF), n + 16 * (f / MF));
}

// ---------------------------------------------------------------------------
// Tile kernel: BM x BN outputs, WGM x WGN waves.  Both operands stream through
// LDS in stages of one block (128 bytes of each row), in two slots, with their
// scales, in three.  LDS rows are 128 bytes; chunk c (16 bytes) of row r sits at
// c ^ ((r >> 1) & 7), so that the 16 rows of a fragment read fall on distinct
// banks.  Row 16 f + r of 32 LDS rows of B holds n = 8 (r / 4) + 4 f + r % 4 of
// those 32.
//
// A wave keeps A's fragments of a stage in registers and takes B's one by one
// (row i of its NF x MF fragments), each read a row ahead.  The multiply-adds of
// an MFMA follow three MFMAs later, so that neither waits for the other.
//
// A load takes longer than a stage's MFMAs (about 1.3 us against 0.9 us), so a
// slot is refilled in parts as soon as each is read: during stage kt
//   row 1          every wave has A's fragments: A (and the scales) of kt + 2
//   row NF / 2 - 1 every wave has the first half of its B rows: that half of
//                  kt + 2; the second half of kt has landed
//   row NF - 1     every wave has the rest: the second half of kt + 2; all of
//                  kt + 1 but its second half has landed, and its first fragments
//                  are read under this row's MFMAs
// with a barrier each, so that every load has about 1.5 stages to land.
// ---------------------------------------------------------------------------
template <int BM, int BN, int WGM, int WGN, int FA, int FB, bool WIDE, bool B_TILE, bool FAR>
__global__ void __launch_bounds__(WGM *WGN * 64, 2) gemm_f8_tile_kernel(const F8GemmArgs p) {
  constexpr int NW = WGM * WGN, NT = NW * 64;
  constexpr int MF = BM / WGM / 16, NF = BN / WGN / 16;  // fragments of a wave
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;      // direct loads of a wave and stage
  constexpr int STAGE = (BM + BN) * 128, SCALES = (BM + BN) * 4;
  static_assert((BM + BN) / 64 == NW, "one load of scales per wave");
  static_assert(NF % 4 == 0 && (!B_TILE || 128 % (BN / WGN) == 0), "a wave's columns share a tile scale");
  static_assert(MF == 4 && LA == 4 && LB == 4, "the schedule of the loads");
  __shared__ __attribute__((aligned(1024))) unsigned char lds[2 * STAGE + 3 * SCALES];
  __shared__ int sh[NW + 4];
  Work w;
  if (!find_work<BM, BN, NT>(p, sh, w)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WGN, wn = wave % WGN;

  // direct-load sources; rows outside the output re-read its last row.  FAR: as
  // addresses, else as offsets to a base that moves from stage to stage.
  const uint8_t *srcA[LA], *srcB[LB];
  unsigned offA[LA], offB[LB];
  bool there = true;
  const int64_t firstA = p.mode == kExperts ? 0 : w.m0;
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int r = (wave + NW * i) * 8 + (lane >> 3), c = ((lane & 7) ^ ((r >> 1) & 7)) << 4;
    const int64_t row = row_of_a(p, min(w.m0 + r, w.m1 - 1), there);
    if (FAR) srcA[i] = w.A + row * p.K + c;
    else offA[i] = (unsigned)((row - firstA) * p.K + c);
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int r = (wave + NW * i) * 8 + (lane >> 3), c = ((lane & 7) ^ ((r >> 1) & 7)) << 4;
    const int n = (r & ~31) + 8 * ((r & 15) >> 2) + 4 * ((r >> 4) & 1) + (r & 3);
    const int64_t row = min(w.n0 + n, p.N - 1);
    if (FAR) srcB[i] = w.B + row * p.K + c;
    else offB[i] = (unsigned)((row - w.n0) * p.K + c);
  }
  uint64_t baseA = uniform(w.A + firstA * p.K), baseB = uniform(w.B + w.n0 * p.K);
  // the wave's 64 scales of a stage: A's, or B's
  unsigned offS;
  if (wave < BM / 64) {
    const int64_t row = row_of_a(p, min(w.m0 + wave * 64 + lane, w.m1 - 1), there);
    offS = (unsigned)(p.a_tile ? row >> 7 : row) * 4;
  } else {
    const int64_t n = min(w.n0 + (wave - BM / 64) * 64 + lane, p.N - 1);
    offS = (unsigned)(p.b_tile ? n >> 7 : n) * 4;
  }
  uint64_t baseS = uniform(wave < BM / 64 ? w.sa : w.sb);
  const uint64_t stepS = uniform(reinterpret_cast<const void *>(4 * (wave < BM / 64 ? w.ka : w.kb)));
  const unsigned lds0 = (unsigned)(size_t)(lds_u8_t)lds;
  // load q of a stage, where `on`, into slot `slot` (scales: `sslot`).  In order:
  // A 0-3, scales 4, the first halves of B's rows 5-6, the second ones 7-8 (a
  // wave's load i fills rows 8 NW i + 8 wave .. + 7, so the first halves are i = 0
  // and 2).
  auto load = [&](int q, int slot, int sslot, int on) {
    const unsigned at = lds0 + slot * STAGE;
    if (q < 4) {
      const unsigned to = at + (wave + NW * q) * 1024;
      if (FAR) dma16(srcA[q], to, on);
      else dma16(baseA, offA[q], to, on);
      if (FAR) srcA[q] += kF8Block;
      else if (q == 3) baseA += kF8Block;
    } else if (q == 4) {
      dma4(baseS, offS, lds0 + 2 * STAGE + sslot * SCALES + wave * 256, on);
      baseS += stepS;
    } else {
      const int i = (q == 5 || q == 7 ? 0 : 2) + (q >= 7 ? 1 : 0);
      const unsigned to = at + BM * 128 + (wave + NW * i) * 1024;
      if (FAR) dma16(srcB[i], to, on);
      else dma16(baseB, offB[i], to, on);
      if (FAR) srcB[i] += kF8Block;
      else if (q == 8) baseB += kF8Block;
    }
  };
  auto flag = [](bool v) { return __builtin_amdgcn_readfirstlane(v ? 1 : 0); };

  const int r16 = lane & 15, g = lane >> 4;
  const int rA = wm * MF * 16 + r16, rB = wn * NF * 16 + r16;
  const int swz = (r16 >> 1) & 7;
  const int c0 = (g ^ swz) << 4, c1 = ((4 + g) ^ swz) << 4;
  Frag<FA, WIDE> a[MF];
  Frag<FB, WIDE> b[2];
  f32x4 t[2];             // B's scales of a row of fragments (row scales)
  float s[MF], sn[MF], tile = 1.f;  // A's scales (times B's, for a tile scale); the next stage's
  auto read_a = [&](const unsigned char *st, int j) {
    const unsigned char *row = st + (rA + 16 * j) * 128;
    a[j].set(*reinterpret_cast<const i32x4 *>(row + c0), *reinterpret_cast<const i32x4 *>(row + c1));
  };
  auto read_b = [&](const unsigned char *st, int i) {
    const unsigned char *row = st + BM * 128 + (rB + 16 * i) * 128;
    b[i & 1].set(*reinterpret_cast<const i32x4 *>(row + c0), *reinterpret_cast<const i32x4 *>(row + c1));
  };
  // (read when the previous row's last multiply-adds, three MFMAs late, are done)
  auto read_t = [&](const unsigned char *sc, int i) {
    if (!B_TILE) t[i & 1] = *reinterpret_cast<const f32x4 *>(sc + (BM + wn * NF * 16 + (i >> 1) * 32 + 8 * g + 4 * (i & 1)) * 4);
  };
  auto read_s = [&](const unsigned char *sc) {
    const float *f = reinterpret_cast<const float *>(sc);
    if (B_TILE) tile = f[BM + wn * NF * 16];
#pragma unroll
    for (int j = 0; j < MF; ++j) sn[j] = f[rA + 16 * j];
  };

  f32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  static_assert(MF == 4 && NF % 4 == 0, "the rings below");
  f32x4 d[4];  // block sums in flight: MFMA number q of a stage writes d[q % 4]
#pragma unroll
  for (int v = 0; v < 4; ++v) d[v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < MF; ++j) s[j] = 0.f;  // for the multiply-adds that come before any MFMA
  t[1] = f32x4{0.f, 0.f, 0.f, 0.f};
  // multiply-adds of MFMA (i, j) with A's scale x
  auto add = [&](int i, int j, float x) {
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(d[j][v], B_TILE ? x : x * t[i & 1][v], acc[i][j][v]);
  };
  constexpr int ROW_A = 1, ROW_H = NF / 2 - 1, ROW_Z = NF - 1;
  static_assert(ROW_A <= ROW_H && ROW_H < ROW_Z, "the order of the loads");
  const unsigned char *scales = lds + 2 * STAGE;
  if (w.nkb > 0) {
    const int two = flag(w.nkb > 1);
#pragma unroll
    for (int q = 0; q < 9; ++q) load(q, 0, 0, 1);
#pragma unroll
    for (int q = 0; q < 9; ++q) load(q, 1, 1, two);
    landed_barrier<11>(two);  // stage 0 but for the second halves
#pragma unroll
    for (int j = 0; j < MF; ++j) read_a(lds, j);
    read_b(lds, 0);
    read_t(scales, 0);
    read_s(scales);
  }
  // the stages of a wave: IDLE where none of its rows or columns is in the output, which
  // then loads and waits like the others and leaves the matrix cores to them
  auto stages = [&](auto idle) {
    constexpr bool IDLE = decltype(idle)::value;
    int s0 = 0;  // kt % 3
    for (int kt = 0; kt < w.nkb; ++kt) {
      const int slot = kt & 1, s1 = s0 == 2 ? 0 : s0 + 1, s2 = s1 == 2 ? 0 : s1 + 1;
      const unsigned char *st = lds + slot * STAGE, *nst = lds + (slot ^ 1) * STAGE;
      const unsigned char *sc = scales + s0 * SCALES, *nsc = scales + s1 * SCALES;
      const int on1 = flag(kt + 1 < w.nkb), on2 = flag(kt + 2 < w.nkb);
      if (!IDLE) s[0] = sn[0] * tile;  // the others once the previous stage's last multiply-adds are done
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        // the second halves of kt were followed by the 9 loads of kt + 1 and, where
        // A's row is an earlier one, 5 of kt + 2; those of kt + 1 up to its first
        // halves by 2 of its own and 7 of kt + 2
        if (i == ROW_H) {
          if (ROW_A < ROW_H) landed_barrier<14>(on2);
          else landed_barrier<9>(on1);
        } else if (i == ROW_A) {
          read_barrier();
        } else if (i == ROW_Z) {
          landed_barrier<9>(on2);
        }
        if (!IDLE) {
          if (i + 1 < NF) {
            read_b(st, i + 1);
          } else {  // (after the last stage: what is read here is not used)
            read_b(nst, 0);
            read_s(nsc);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < MF; ++j) {
          if (!IDLE) {
            d[j] = mma<FA, FB>(b[i & 1], a[j]);
            if (i + 1 == NF) read_a(nst, j);
          }
          const int after = (i - ROW_A) * MF + j;  // MFMAs since A's row
          if (ROW_A < ROW_H) {
            if (after >= 0 && after < 5) load(after, slot, s2, on2);
            if (i == ROW_H && j < 2) load(5 + j, slot, s2, on2);
          } else {
            if (after >= 0 && after < 7) load(after, slot, s2, on2);
          }
          if (i == ROW_Z && j < 2) load(7 + j, slot, s2, on2);
          if (!IDLE) {
            if (j == 3) {
              if (i + 1 < NF) read_t(sc, i + 1);
              else read_t(nsc, 0);
              add(i, 0, s[0]);
            } else if (i > 0) {
              add(i - 1, j + 1, s[j + 1]);
            } else {
              add(NF - 1, j + 1, s[j + 1]);
              s[j + 1] = sn[j + 1] * tile;
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      s0 = s1;
    }
  };
  // only with tile scales of B (weights by expert: 16384 x 8 rows over 512 experts 238 ->
  // 223 us, 2048 x 8 over 64 115 -> 107): with row scales, which weight gradients have,
  // whose tiles are mostly full, the second loop cost 456 -> 467
  if constexpr (B_TILE) {
    if (flag(w.m0 + wm * MF * 16 >= w.m1 || w.n0 + wn * NF * 16 >= p.N)) {
      stages(std::true_type{});
      return;
    }
  }
  stages(std::false_type{});
#pragma unroll
  for (int j = 0; j < 3; ++j) add(NF - 1, j + 1, s[j + 1]);

  float seen = 0.f;
  // row j's outputs, once they are on their way (with a tile scale of B a row has one
  // product of scales for all columns)
  auto look_at_row = [&](int j) {
#pragma unroll
    for (int i = 0; i < (B_TILE ? 1 : NF); ++i) {
      look_at(acc[i][j][0], acc[i][j][1], seen);
      if (!B_TILE) look_at(acc[i][j][2], acc[i][j][3], seen);
    }
  };

  const bool vec = (p.N * (p.out_dtype == NSG_F32 ? 4 : 2)) % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  if (vec && p.out_dtype != NSG_F32 && w.n0 + BN <= p.N) {
    // (large products, past the caches: weight gradients of 512 experts, 1.07 GB, 467 ->
    // 443 us, 16384 x 16384 x 1024 313 -> 294, 8192 x 8192 x 512 49 -> 50)
    constexpr bool STREAM = BM == 256;
    // lanes of neighbouring tokens swap halves of 64 n, so that a store fills
    // whole 128-byte lines: first the even tokens', then the odd ones'
    const bool odd = r16 & 1;
    uint16_t *base = (uint16_t *)p.out + w.out + w.n0 + wn * NF * 16 + 8 * g + (odd ? 32 : 0);
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int64_t m = w.m0 + rA + 16 * j, me = m - odd, mo = me + 1;
      bool there = true;
      if (!w.zero && m < w.m1) row_of_a(p, m, there);
#pragma unroll
      for (int i = 0; i < NF; i += 4) {
        u32x4 h[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = there ? acc[i + 2 * k + (e >> 2)][j][e & 3] : 0.f;
          h[k] = p.out_dtype == NSG_BF16 ? pack8<__bf16>(v) : pack8<_Float16>(v);
        }
        u32x4 get;
#pragma unroll
        for (int e = 0; e < 4; ++e)  // from lane ^ 1
          get[e] = (uint32_t)__builtin_amdgcn_mov_dpp((int)(odd ? h[0][e] : h[1][e]), 0xB1, 0xF, 0xF, true);
        u32x4 *te = reinterpret_cast<u32x4 *>(base + me * p.N + i * 16), *to = reinterpret_cast<u32x4 *>(base + mo * p.N + i * 16);
        const u32x4 ve = odd ? get : h[0], vo = odd ? h[1] : get;
        if constexpr (STREAM) {
          if (me < w.m1) __builtin_nontemporal_store(ve, te);
          if (mo < w.m1) __builtin_nontemporal_store(vo, to);
        } else {
          if (me < w.m1) *te = ve;
          if (mo < w.m1) *to = vo;
        }
      }
      look_at_row(j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int64_t m = w.m0 + rA + 16 * j;
      if (m >= w.m1) continue;
      bool there = true;
      if (!w.zero) row_of_a(p, m, there);
#pragma unroll
      for (int i = 0; i < NF; i += 2) {
        const int64_t n = w.n0 + wn * NF * 16 + i * 16 + 8 * g;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = there ? acc[i + (k >> 2)][j][k & 3] : 0.f;
        store8(p.out, p.out_dtype, w.out + m * p.N + n, v, p.N - n, vec);
      }
      look_at_row(j);
    }
  }
  if (not_finite(seen)) mend<MF, NF, FA, FB, WIDE>(p, w, w.m0 + wm * MF * 16, w.n0 + wn * NF * 16);
}

// ---------------------------------------------------------------------------
// Kernel for few tiles: 64 x 64 outputs, four waves of 32 x 32.  With fewer tiles
// than compute units what counts is how long a tile takes, which in the tile kernel
// is a load's latency for every stage; here NS - 1 of the NS slots are in flight,
// and a stage's fragments are read under the MFMAs of the one before.  Layouts as in
// the tile kernel.
// ---------------------------------------------------------------------------
template <int NS, int FA, int FB, bool WIDE, bool B_TILE>
__global__ void __launch_bounds__(256, 2) gemm_f8_deep_kernel(const F8GemmArgs p) {
  constexpr int BM = 64, BN = 64, STAGE = (BM + BN) * 128 + (BM + BN) * 4;
  constexpr int LOADS = 5;  // of a wave and stage: two of each operand, one of scales
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NS * STAGE];
  __shared__ int sh[8];
  Work w;
  if (!find_work<BM, BN, 256>(p, sh, w)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  unsigned offA[2], offB[2], offS;
  bool there = true;
  const int64_t firstA = p.mode == kExperts ? 0 : w.m0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (wave + 4 * i) * 8 + (lane >> 3), c = ((lane & 7) ^ ((r >> 1) & 7)) << 4;
    const int64_t row = row_of_a(p, min(w.m0 + r, w.m1 - 1), there);
    offA[i] = (unsigned)((row - firstA) * p.K + c);
    const int n = (r & ~31) + 8 * ((r & 15) >> 2) + 4 * ((r >> 4) & 1) + (r & 3);
    offB[i] = (unsigned)((min(w.n0 + n, p.N - 1) - w.n0) * p.K + c);
  }
  uint64_t baseA = uniform(w.A + firstA * p.K), baseB = uniform(w.B + w.n0 * p.K);
  // waves 0 and 2 load A's 64 scales (twice the same), 1 and 3 B's
  if (wn == 0) {
    const int64_t row = row_of_a(p, min(w.m0 + lane, w.m1 - 1), there);
    offS = (unsigned)(p.a_tile ? row >> 7 : row) * 4;
  } else {
    const int64_t n = min(w.n0 + lane, p.N - 1);
    offS = (unsigned)(p.b_tile ? n >> 7 : n) * 4;
  }
  uint64_t baseS = uniform(wn == 0 ? w.sa : w.sb);
  const uint64_t stepS = uniform(reinterpret_cast<const void *>(4 * (wn == 0 ? w.ka : w.kb)));
  const unsigned lds0 = (unsigned)(size_t)(lds_u8_t)lds;
  auto load = [&](int slot, bool some) {
    const int on = __builtin_amdgcn_readfirstlane(some ? 1 : 0);
    const unsigned at = lds0 + slot * STAGE;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      dma16(baseA, offA[i], at + (wave + 4 * i) * 1024, on);
      dma16(baseB, offB[i], at + BM * 128 + (wave + 4 * i) * 1024, on);
    }
    dma4(baseS, offS, at + (BM + BN) * 128 + wn * 256, on);
    baseA += kF8Block;
    baseB += kF8Block;
    baseS += stepS;
  };

  const int r16 = lane & 15, g = lane >> 4, swz = (r16 >> 1) & 7;
  const int c0 = (g ^ swz) << 4, c1 = ((4 + g) ^ swz) << 4;
  const int rA = wm * 32 + r16, rB = wn * 32 + r16;
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  Frag<FA, WIDE> a[2][2];  // of even and odd stages
  Frag<FB, WIDE> b[2][2];
  float s[2][2];
  f32x4 t[2][2];
  auto read = [&](int slot, int o) {
    const unsigned char *st = lds + slot * STAGE;
    const float *sA = reinterpret_cast<const float *>(st + (BM + BN) * 128), *sB = sA + BM + wn * 32;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned char *rowA = st + (rA + 16 * j) * 128, *rowB = st + BM * 128 + (rB + 16 * j) * 128;
      a[o][j].set(*reinterpret_cast<const i32x4 *>(rowA + c0), *reinterpret_cast<const i32x4 *>(rowA + c1));
      b[o][j].set(*reinterpret_cast<const i32x4 *>(rowB + c0), *reinterpret_cast<const i32x4 *>(rowB + c1));
      s[o][j] = sA[rA + 16 * j];
      t[o][j] = B_TILE ? f32x4{sB[0], 0.f, 0.f, 0.f} : *reinterpret_cast<const f32x4 *>(sB + 8 * g + 4 * j);
    }
  };
  int slot = 0;  // kt % NS
  // stage kt, whose fragments are in registers; the next one's are read
  auto stage = [&](int kt, int o) {
    const int next = slot + 1 == NS ? 0 : slot + 1;
    // stage kt + 1 has landed, and every wave has read stage kt, whose slot is refilled
    landed_barrier<LOADS *(NS - 2)>(__builtin_amdgcn_readfirstlane(kt + NS - 1 < w.nkb ? 1 : 0));
    read(next, o ^ 1);  // (after the last stage: not used)
    load(slot, kt + NS < w.nkb);
    slot = next;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x4 d = mma<FA, FB>(b[o][i], a[o][j]);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(d[v], s[o][j] * t[o][i][B_TILE ? 0 : v], acc[i][j][v]);
      }
  };
  if (w.nkb > 0) {
#pragma unroll
    for (int k = 0; k < NS; ++k) load(k, k < w.nkb);
    landed_barrier<LOADS *(NS - 1)>(__builtin_amdgcn_readfirstlane(NS - 1 < w.nkb ? 1 : 0));
    read(0, 0);
  }
  int kt = 0;
  for (; kt + 1 < w.nkb; kt += 2) {
    stage(kt, 0);
    stage(kt + 1, 1);
  }
  if (kt < w.nkb) stage(kt, 0);

  const bool vec = (p.N * (p.out_dtype == NSG_F32 ? 4 : 2)) % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  float seen = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t m = w.m0 + rA + 16 * j, n = w.n0 + wn * 32 + 8 * g;
    if (m >= w.m1) continue;
    there = true;
    if (!w.zero) row_of_a(p, m, there);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = there ? acc[k >> 2][j][k & 3] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; k += 2) look_at(v[k], v[k + 1], seen);
    store8(p.out, p.out_dtype, w.out + m * p.N + n, v, p.N - n, vec);
  }
  if (not_finite(seen)) mend<2, 2, FA, FB, WIDE>(p, w, w.m0 + wm * 32, w.n0 + wn * 32);
}

// ---------------------------------------------------------------------------
// Kernel for few rows of A: a workgroup takes 16 MF rows of A and 16 NF rows of B,
// and its NW waves take the blocks of K in turn.  What bounds it is reading B
// once, so nothing goes through LDS: a wave loads fragments of U blocks straight
// into registers (16 rows x 64 bytes a load), all of them before the first use,
// and K split over the waves keeps enough loads in flight where B has few rows.
// The waves' sums are added in LDS in their order.
// ---------------------------------------------------------------------------
template <int MF, int NF, int NW, int U, int FA, int FB, bool WIDE, bool B_TILE>
__global__ void __launch_bounds__(NW * 64) gemm_f8_rows_kernel(const F8GemmArgs p) {
  __shared__ f32x4 sums[NW][NF * MF][64];
  __shared__ int sh[NW + 4];
  Work w;
  if (!find_work<16 * MF, 16 * NF, NW * 64>(p, sh, w)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const uint8_t *rowA[MF], *rowB[NF];
  const float *scaleA[MF], *scaleB[NF];
  bool there = true;
#pragma unroll
  for (int j = 0; j < MF; ++j) {
    const int64_t row = row_of_a(p, min(w.m0 + 16 * j + r16, w.m1 - 1), there);
    rowA[j] = w.A + row * p.K + 16 * g;
    scaleA[j] = w.sa + (p.a_tile ? row >> 7 : row);
  }
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    rowB[i] = w.B + min(w.n0 + 16 * i + r16, p.N - 1) * p.K + 16 * g;
    // a tile scale is one for the 16 rows; row scales are loaded four times
    scaleB[i] = w.sb + (B_TILE ? min(w.n0 + 16 * i, p.N - 1) >> 7 : 0);
  }
  f32x4 acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int k0 = wave; k0 < w.nkb; k0 += NW * U) {
    i32x4 la[U][MF][2], lb[U][NF][2];
    float sa[U][MF];
    f32x4 sb[U][NF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t kb = min(k0 + u * NW, w.nkb - 1);  // one behind the last is loaded again and not used
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        lb[u][i][0] = *reinterpret_cast<const i32x4 *>(rowB[i] + kb * kF8Block);
        lb[u][i][1] = *reinterpret_cast<const i32x4 *>(rowB[i] + kb * kF8Block + 64);
      }
#pragma unroll
      for (int j = 0; j < MF; ++j) {
        la[u][j][0] = *reinterpret_cast<const i32x4 *>(rowA[j] + kb * kF8Block);
        la[u][j][1] = *reinterpret_cast<const i32x4 *>(rowA[j] + kb * kF8Block + 64);
        sa[u][j] = scaleA[j][kb * w.ka];
      }
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        if (B_TILE) {
          sb[u][i][0] = scaleB[i][kb * w.kb];
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int64_t n = min(w.n0 + 16 * i + 4 * g + v, p.N - 1);
            sb[u][i][v] = scaleB[i][kb * w.kb + (p.b_tile ? n >> 7 : n)];
          }
        }
      }
    }
    asm volatile("" ::: "memory");  // the loads stay above their uses, together
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u * NW >= w.nkb) continue;
      Frag<FA, WIDE> a[MF];
#pragma unroll
      for (int j = 0; j < MF; ++j) a[j].set(la[u][j][0], la[u][j][1]);
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        Frag<FB, WIDE> b;
        b.set(lb[u][i][0], lb[u][i][1]);
#pragma unroll
        for (int j = 0; j < MF; ++j) {
          const f32x4 d = mma<FA, FB>(b, a[j]);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(d[v], sa[u][j] * sb[u][i][B_TILE ? 0 : v], acc[i][j][v]);
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) sums[wave][i * MF + j][lane] = acc[i][j];
  __syncthreads();
  const bool vec = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  for (int f = wave; f < NF * MF; f += NW) {
    f32x4 v = sums[0][f][lane];
#pragma unroll
    for (int k = 1; k < NW; ++k) v += sums[k][f][lane];
    const int64_t m = w.m0 + 16 * (f % MF) + r16, n = w.n0 + 16 * (f / MF) + 4 * g;
    float seen = 0.f;
    look_at(v[0], v[1], seen);
    look_at(v[2], v[3], seen);
    if (m < w.m1 && n < p.N) {
      there = true;
      if (!w.zero) row_of_a(p, m, there);
      if (!there) v = f32x4{0.f, 0.f, 0.f, 0.f};
      store4(p.out, p.out_dtype, w.out + m * p.N + n, v, p.N - n, vec);
    }
    if (not_finite(seen)) mend<1, 1, FA, FB, WIDE>(p, w, m - r16, n - 4 * g);
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// workgroups of a launch: every tile that there can be, rounded up to the order above
template <int BM, int BN> static int64_t grid_of(const F8GemmArgs &a) {
  const int64_t tn = (a.N + BN - 1) / BN;
  if (a.mode == kDense) {
    const int64_t total = a.batch * ((a.M + BM - 1) / BM) * tn;
    const int64_t run = total >= 256 ? 32 : (total + 7) / 8;
    return (total + 8 * run - 1) / (8 * run) * (8 * run);
  }
  if (a.mode == kExperts) {
    // every expert has at most one tile that is not full, and so has the tail
    const int64_t units = a.M / BM + (a.E + 1 < a.M ? a.E + 1 : a.M);
    return (units + 7) / 8 * 8 * tn;
  }
  return ((int64_t)a.E + 7) / 8 * 8 * ((a.M + BM - 1) / BM) * tn;
}

// HIP counts a launch's threads in 32 bits
static bool launchable(int64_t grid, int threads) { return grid * threads <= 0xFFFFFFFFll; }

// Calls launch<FA, FB, B_TILE>() for the types and scales of `a`.
template <typename L> static hipError_t by_type(const F8GemmArgs &a, int64_t grid, int threads, L launch) {
  if (!launchable(grid, threads)) return hipErrorInvalidConfiguration;
  using one = std::integral_constant<int, 1>;
  using zero = std::integral_constant<int, 0>;
  auto scales = [&](auto fa, auto fb) { a.b_tile ? launch(fa, fb, one{}) : launch(fa, fb, zero{}); };
  const bool fa = a.a_dtype == NSG_F8E5M2, fb = a.b_dtype == NSG_F8E5M2;
  if (fa) fb ? scales(one{}, one{}) : scales(one{}, zero{});
  else fb ? scales(zero{}, one{}) : scales(zero{}, zero{});
  return hipGetLastError();
}

// rows of a tile of BN (gathered: all rows of A) are within 32-bit offsets of each other
static bool near_rows(const F8GemmArgs &a, int64_t tile) {
  return (a.mode == kExperts && a.T > tile ? a.T : tile) * a.K <= 0xFFFFFFFFll;
}

template <int BM, int BN, int WGM, int WGN, bool WIDE> static hipError_t launch_tile(const F8GemmArgs &a, hipStream_t s) {
  constexpr int NT = WGM * WGN * 64;
  const int64_t grid = grid_of<BM, BN>(a);
  const bool far = !near_rows(a, BM > BN ? BM : BN);
  return by_type(a, grid, NT, [&](auto fa, auto fb, auto tile) {
    if (far)
      hipLaunchKernelGGL((gemm_f8_tile_kernel<BM, BN, WGM, WGN, fa(), fb(), WIDE, tile() != 0, true>), dim3((unsigned)grid),
                         dim3(NT), 0, s, a);
    else
      hipLaunchKernelGGL((gemm_f8_tile_kernel<BM, BN, WGM, WGN, fa(), fb(), WIDE, tile() != 0, false>), dim3((unsigned)grid),
                         dim3(NT), 0, s, a);
  });
}

template <bool WIDE> static hipError_t launch_deep(const F8GemmArgs &a, hipStream_t s) {
  const int64_t grid = grid_of<64, 64>(a);
  return by_type(a, grid, 256, [&](auto fa, auto fb, auto tile) {
    hipLaunchKernelGGL((gemm_f8_deep_kernel<8, fa(), fb(), WIDE, tile() != 0>), dim3((unsigned)grid), dim3(256), 0, s, a);
  });
}

// whether a launch holds the few-rows kernel's workgroups, 16 NF columns of B each: for
// batches of more than about 2^27 columns in all it does not, and the tile kernel's
// (128 columns for 256 threads) it does
template <int MF, int NF, int NW> static bool rows_launchable(const F8GemmArgs &a) {
  return launchable(grid_of<16 * MF, 16 * NF>(a), NW * 64);
}

template <int MF, int NF, int NW, int U, bool WIDE> static hipError_t launch_rows(const F8GemmArgs &a, hipStream_t s) {
  const int64_t grid = grid_of<16 * MF, 16 * NF>(a);
  return by_type(a, grid, NW * 64, [&](auto fa, auto fb, auto tile) {
    hipLaunchKernelGGL((gemm_f8_rows_kernel<MF, NF, NW, U, fa(), fb(), WIDE, tile() != 0>), dim3((unsigned)grid),
                       dim3(NW * 64), 0, s, a);
  });
}

constexpr int64_t kComputeUnits = 256;  // of an MI355X

// Which kernel.  All but the one for few rows add an output's blocks in the same
// order, so that their results are the same bit for bit.
template <bool WIDE> static hipError_t launch_any(const F8GemmArgs &a, hipStream_t s) {
  // few rows: 16 x 4096 x 4096 in 6.7 us against the deep kernel's 15.1, 32 in 8.5
  // against 15.3; with more rows of B those of A are read too often: 32 x 8192 x 4096 in
  // 13.9 against 15.3, 32 x 11008 x 4096 in 19.6 against 15.6
  if (a.mode == kDense && a.M <= 16 && rows_launchable<1, 1, 8>(a)) return launch_rows<1, 1, 8, 4, WIDE>(a, s);
  if (a.mode == kDense && a.M <= 32 && a.batch * a.N <= 8192) return launch_rows<2, 1, 8, 2, WIDE>(a, s);
  // one or two tokens' experts (K = 2048, N = 512): 1 x 8 rows in 6.2 us against the deep
  // kernel's 10.9, 2 x 8 in 9.5 against 11.6, 4 x 8 in 16.5 against 12.4
  if (a.mode == kExperts && a.M * a.N <= 8192) return launch_rows<1, 1, 8, 4, WIDE>(a, s);
  // no more 64 x 64 tiles than compute units: 256 x 4096 x 4096 (256 tiles) in 15.8 us
  // against 23.0 with 128 x 128 tiles, 128 x 11008 x 4096 (344) in 29.5 against 23.2;
  // weight gradients of 256 x 256 over 4096 rows (128 workgroups) in 16.4 against 28.6,
  // two of 512 x 512 over 300 rows (512) in 9.1 against 6.3
  if (grid_of<64, 64>(a) <= kComputeUnits && near_rows(a, 64)) return launch_deep<WIDE>(a, s);
  // 256 x 256 tiles (8-bit instructions only: their registers are full) need most of
  // the chip's compute units busy, one workgroup each, and mostly full tiles:
  //   1024 x 11008 x 4096 (172 tiles) in 48 us against 53 with 128 x 128 tiles,
  //   2048 x 4096 x 4096 (128) in 47 against 36; experts with tile scales, whose empty
  //   parts of a tile cost least, with 128 rows on average (8192 x 8 over 512, N = 512,
  //   K = 2048) in 155 against 168, with 64 (512 x 8 over 64, N = K = 2048) in 66 against
  //   67; with row scales and 256 rows (2048 x 8 over 64) in 116 against 128, with 128
  //   in 97 against 84; weight gradients of 512 experts of 2048 x 512 in 458 against 611
  if constexpr (!WIDE) {
    const int64_t full = (a.M / 256) * (a.N / 256) * (a.mode == kDense ? a.batch : a.mode == kWgrad ? a.E : 1);
    if (full >= 160 && (a.mode != kExperts || a.M >= (a.b_tile ? 96 : 192) * (int64_t)a.E)) return launch_tile<256, 256, 4, 2, false>(a, s);
  }
  return launch_tile<128, 128, 2, 2, WIDE>(a, s);
}

hipError_t launch_gemm_f8(const F8GemmArgs &a, hipStream_t s) {
  return a.out_dtype == NSG_F32 ? launch_any<true>(a, s) : launch_any<false>(a, s);
}

}  // namespace nsg
