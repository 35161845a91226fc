// Internal interface of the expert-layer operators: tokens sorted by expert
// and back (nsg_expert.hip), 8-bit operands with block scales (nsg_fp8.hip)
// and their products (nsg_fp8_gemm.hip), launched by nsg_expert_api.cpp.
// Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime.h>

#include "nsg.h"

namespace nsg {

constexpr int kF8Block = 128;  // elements of one scale along a row; side of a tile

inline __host__ __device__ int64_t up128(int64_t n) { return (n + kF8Block - 1) / kF8Block * kF8Block; }

// ---- tokens sorted by expert (nsg_expert.hip) -----------------------------
int expert_sort_chunks(int64_t P);  // workgroups of the sort; above 1 it needs a table [chunks][E]
hipError_t launch_expert_sort(const void *ids, int wide, int64_t P, int k, int E, int32_t *offsets, int32_t *rows,
                              int32_t *tokens, int32_t *table, hipStream_t s);
hipError_t launch_expert_dispatch(const void *x, int elem, int64_t T, int64_t C, int64_t ldx, const int32_t *offsets, int E,
                                  const int32_t *rows, int k, void *out, hipStream_t s);
hipError_t launch_expert_combine(const void *y, int dtype, int64_t P, int64_t C, int64_t ldy, const int32_t *rows,
                                 int64_t T, int k, const float *w, void *out, hipStream_t s);
hipError_t launch_expert_combine_backward(const void *dout, int64_t lddo, const void *y, int64_t ldy, int dtype,
                                          int64_t P, int64_t C, const int32_t *offsets, int E, const int32_t *rows,
                                          int64_t T, int k, const float *w, void *dy, float *dw, hipStream_t s);

// ---- 8-bit operands (nsg_fp8.hip) -----------------------------------------
struct QuantArgs {
  const void *x = nullptr;
  int x_dtype = NSG_BF16;
  int f8 = NSG_F8E4M3;
  int64_t B = 0, R = 0, C = 0, ldx = 0;  // x [B][R][ldx]
  void *q = nullptr;                     // [B][R][Cp]
  float *s = nullptr;                    // rows: [B][Cp/128][R]; tiles: [B][Cp/128][ceil(R/128)]
  void *qt = nullptr;                    // tiles: [B][C][Rp]; columns: [C][cap]
  float *st = nullptr;                   // tiles: [B][Rp/128][ceil(C/128)]; columns: [cap/128][C]
  // columns: the rows P of x (through `tokens` where given), by expert
  const int32_t *offsets = nullptr, *tokens = nullptr;
  int E = 0;
  int64_t P = 0;
  // by the launchers.  Rows: blocks of a workgroup; columns: all blocks of 128 rows,
  // and how many workgroups share the column tiles of one
  int64_t blocks = 0, share = 0;
};
hipError_t launch_quantize_rows(const QuantArgs &a, hipStream_t s);
hipError_t launch_quantize_tiles(const QuantArgs &a, hipStream_t s);
hipError_t launch_quantize_columns(const QuantArgs &a, hipStream_t s);

// ---- their products (nsg_fp8_gemm.hip) ------------------------------------
// out[m, n] = sum over K blocks b of sa[b, m] sb[b, n] sum_{k in b} A[m, k] B[n, k].
//   kDense: `batch` products, operands and output one behind the other.
//   kExperts: row p of the output is row tokens[p] (or p) of A against the
//     matrix of B whose expert has p between its offsets; rows behind
//     offsets[E] are zero.
//   kWgrad: output e contracts the K blocks of expert e in the columns layout.
enum F8Mode : int { kDense = 0, kExperts = 1, kWgrad = 2 };
struct F8GemmArgs {
  int mode = kDense;
  int a_dtype = NSG_F8E4M3, b_dtype = NSG_F8E4M3, out_dtype = NSG_BF16;
  int64_t batch = 1;      // kDense
  int64_t M = 0, N = 0;   // rows of A (kExperts: rows P of the output), rows of B
  int64_t K = 0;          // padded row length of the operands, a multiple of 128
  const void *A = nullptr, *B = nullptr;
  const float *sa = nullptr, *sb = nullptr;
  int a_tile = 0, b_tile = 0;  // the scales are one for 128 rows
  const int32_t *offsets = nullptr, *tokens = nullptr;
  int E = 0;
  int64_t T = 0;          // kExperts: rows of A; kWgrad: rows P behind the offsets
  void *out = nullptr;    // [batch | 1 | E][M][N]
};
hipError_t launch_gemm_f8(const F8GemmArgs &a, hipStream_t s);

}  // namespace nsg
