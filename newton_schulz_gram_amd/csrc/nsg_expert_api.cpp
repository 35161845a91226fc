// C entry points of the expert-layer operators (include/nsg.h): argument
// checks, then one or two launches on the caller's stream.  Nothing is
// allocated and the host never waits.
#include <cstdint>

#include "nsg_expert.h"

using namespace nsg;

namespace {

constexpr int64_t kMaxRows = NSG_MAX_ROWS;
constexpr int64_t kMaxSide = NSG_MAX_SIDE;

bool float_dtype(int32_t d) { return d == NSG_F16 || d == NSG_BF16 || d == NSG_F32; }
bool f8_dtype(int32_t d) { return d == NSG_F8E4M3 || d == NSG_F8E5M2; }
int64_t elem_size(int32_t d) { return d == NSG_F32 ? 4 : 2; }
bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// a launcher refuses a grid that HIP cannot hold with hipErrorInvalidConfiguration
nsg_status_t done(hipError_t e) {
  return e == hipSuccess ? NSG_OK : e == hipErrorInvalidConfiguration ? NSG_ERR_SHAPE : NSG_ERR_HIP;
}
hipStream_t hs(void *stream) { return reinterpret_cast<hipStream_t>(stream); }

// P = T k choices of E experts
nsg_status_t check_choices(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || k < 1 || k > kMaxRows || T > kMaxRows / k) return NSG_ERR_SHAPE;
  if (E < 1 || E > NSG_MAX_EXPERTS) return NSG_ERR_SHAPE;
  return NSG_OK;
}
// rows of C elements, ld apart
nsg_status_t check_rows(int64_t n, int64_t C, int64_t ld) {
  if (n < 0 || n > kMaxRows || C < 0 || C > kMaxSide || ld < C || ld > (1ll << 31)) return NSG_ERR_SHAPE;
  return NSG_OK;
}
bool rows_aligned(const void *p, int32_t dtype) { return aligned(p, (uintptr_t)elem_size(dtype)); }

}  // namespace

extern "C" {

// ---- tokens sorted by expert and back ----------------------------------------

nsg_status_t nsg_expert_sort_workspace_size(int64_t T, int64_t k, int64_t E, size_t *bytes) {
  if (bytes == nullptr) return NSG_ERR_INVALID_ARG;
  const nsg_status_t st = check_choices(T, k, E);
  if (st != NSG_OK) return st;
  const int chunks = expert_sort_chunks(T * k);
  *bytes = chunks > 1 ? (size_t)chunks * (size_t)E * 4 : 0;
  return NSG_OK;
}

nsg_status_t nsg_expert_sort(const void *ids, int32_t id_bits, int64_t T, int64_t k, int64_t E, int32_t *offsets,
                             int32_t *rows, int32_t *tokens, void *workspace, size_t workspace_bytes, void *stream) {
  size_t need = 0;
  const nsg_status_t st = nsg_expert_sort_workspace_size(T, k, E, &need);
  if (st != NSG_OK) return st;
  if (id_bits != 32 && id_bits != 64) return NSG_ERR_UNSUPPORTED_DTYPE;
  const int64_t P = T * k;
  if (offsets == nullptr || (P > 0 && (ids == nullptr || rows == nullptr || tokens == nullptr))) return NSG_ERR_INVALID_ARG;
  if (!aligned(ids, (uintptr_t)(id_bits / 8)) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(tokens, 4))
    return NSG_ERR_INVALID_ARG;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 4)))
    return NSG_ERR_WORKSPACE_TOO_SMALL;
  return done(launch_expert_sort(ids, id_bits == 64, P, (int)k, (int)E, offsets, rows, tokens,
                                 reinterpret_cast<int32_t *>(workspace), hs(stream)));
}

nsg_status_t nsg_expert_dispatch(const void *x, int32_t dtype, int64_t T, int64_t C, int64_t ldx, const int32_t *offsets,
                                 int64_t E, const int32_t *rows, int64_t k, void *out, void *stream) {
  if (!float_dtype(dtype)) return NSG_ERR_UNSUPPORTED_DTYPE;
  nsg_status_t st = check_choices(T, k, E);
  if (st == NSG_OK) st = check_rows(T, C, ldx);
  if (st != NSG_OK) return st;
  if (T == 0 || C == 0) return NSG_OK;
  if (x == nullptr || offsets == nullptr || rows == nullptr || out == nullptr) return NSG_ERR_INVALID_ARG;
  if (!rows_aligned(x, dtype) || !rows_aligned(out, dtype) || !aligned(offsets, 4) || !aligned(rows, 4))
    return NSG_ERR_INVALID_ARG;
  return done(launch_expert_dispatch(x, (int)elem_size(dtype), T, C, ldx, offsets, (int)E, rows, (int)k, out, hs(stream)));
}

nsg_status_t nsg_expert_combine(const void *y, int32_t dtype, int64_t P, int64_t C, int64_t ldy, const int32_t *rows,
                                int64_t T, int64_t k, const float *weights, void *out, void *stream) {
  if (!float_dtype(dtype)) return NSG_ERR_UNSUPPORTED_DTYPE;
  nsg_status_t st = check_choices(T, k, 1);
  if (st == NSG_OK) st = check_rows(P, C, ldy);
  if (st != NSG_OK) return st;
  if (T == 0 || C == 0) return NSG_OK;
  if (rows == nullptr || out == nullptr || (P > 0 && y == nullptr)) return NSG_ERR_INVALID_ARG;
  if (!rows_aligned(y, dtype) || !rows_aligned(out, dtype) || !aligned(rows, 4) || !aligned(weights, 4))
    return NSG_ERR_INVALID_ARG;
  return done(launch_expert_combine(y, dtype, P, C, ldy, rows, T, (int)k, weights, out, hs(stream)));
}

nsg_status_t nsg_expert_combine_backward(const void *dout, int64_t lddo, const void *y, int64_t ldy, int32_t dtype,
                                         int64_t P, int64_t C, const int32_t *offsets, int64_t E, const int32_t *rows,
                                         int64_t T, int64_t k, const float *weights, void *dy, float *dw, void *stream) {
  if (!float_dtype(dtype)) return NSG_ERR_UNSUPPORTED_DTYPE;
  nsg_status_t st = check_choices(T, k, E);
  if (st == NSG_OK) st = check_rows(P, C, ldy);
  if (st == NSG_OK) st = check_rows(T, C, lddo);
  if (st != NSG_OK) return st;
  if (P != T * k) return NSG_ERR_SHAPE;
  if (T == 0) return NSG_OK;
  if (offsets == nullptr || rows == nullptr || dw == nullptr || (C > 0 && (dout == nullptr || y == nullptr || dy == nullptr)))
    return NSG_ERR_INVALID_ARG;
  if (!rows_aligned(dout, dtype) || !rows_aligned(y, dtype) || !rows_aligned(dy, dtype) || !aligned(offsets, 4) ||
      !aligned(rows, 4) || !aligned(weights, 4) || !aligned(dw, 4))
    return NSG_ERR_INVALID_ARG;
  return done(launch_expert_combine_backward(dout, lddo, y, ldy, dtype, P, C, offsets, (int)E, rows, T, (int)k, weights, dy,
                                             dw, hs(stream)));
}

// ---- 8-bit operands ------------------------------------------------------------

nsg_status_t nsg_quantize_fp8(const void *x, int32_t x_dtype, int64_t B, int64_t R, int64_t C, int64_t ldx,
                              int32_t block, int32_t q_dtype, void *q, float *scale, void *q_t, float *scale_t,
                              void *stream) {
  if (!float_dtype(x_dtype) || !f8_dtype(q_dtype)) return NSG_ERR_UNSUPPORTED_DTYPE;
  if (block != NSG_BLOCK_ROW && block != NSG_BLOCK_TILE) return NSG_ERR_INVALID_ARG;
  const nsg_status_t st = check_rows(R, C, ldx);
  if (st != NSG_OK) return st;
  // the grid holds a batch in its z and a tile of rows in its y index
  if (B < 0 || B > 65535 || (block == NSG_BLOCK_TILE && R > 128 * 65535)) return NSG_ERR_SHAPE;
  if (block == NSG_BLOCK_ROW && (q_t != nullptr || scale_t != nullptr)) return NSG_ERR_INVALID_ARG;
  if ((q_t == nullptr) != (scale_t == nullptr)) return NSG_ERR_INVALID_ARG;
  if (B == 0 || R == 0 || C == 0) return NSG_OK;
  if (x == nullptr || q == nullptr || scale == nullptr) return NSG_ERR_INVALID_ARG;
  if (!rows_aligned(x, x_dtype) || !aligned(q, 16) || !aligned(q_t, 16) || !aligned(scale, 4) || !aligned(scale_t, 4))
    return NSG_ERR_INVALID_ARG;
  QuantArgs a;
  a.x = x; a.x_dtype = x_dtype; a.f8 = q_dtype;
  a.B = B; a.R = R; a.C = C; a.ldx = ldx;
  a.q = q; a.s = scale; a.qt = q_t; a.st = scale_t;
  return done(block == NSG_BLOCK_ROW ? launch_quantize_rows(a, hs(stream)) : launch_quantize_tiles(a, hs(stream)));
}

nsg_status_t nsg_fp8_columns(int64_t P, int64_t E, int64_t *cap) {
  if (cap == nullptr) return NSG_ERR_INVALID_ARG;
  if (P < 0 || P > kMaxRows || E < 1 || E > NSG_MAX_EXPERTS) return NSG_ERR_SHAPE;
  *cap = kF8Block * (P / kF8Block + E);
  return NSG_OK;
}

nsg_status_t nsg_quantize_fp8_columns(const void *x, int32_t x_dtype, int64_t R, int64_t C, int64_t ldx,
                                      const int32_t *offsets, int64_t E, const int32_t *tokens, int64_t P,
                                      int32_t q_dtype, void *q_t, float *scale, void *stream) {
  if (!float_dtype(x_dtype) || !f8_dtype(q_dtype)) return NSG_ERR_UNSUPPORTED_DTYPE;
  const nsg_status_t st = check_rows(R, C, ldx);
  if (st != NSG_OK) return st;
  if (E < 1 || E > NSG_MAX_EXPERTS || P < 0 || P > kMaxRows || (tokens == nullptr && P > 0 && P != R)) return NSG_ERR_SHAPE;
  if (C == 0) return NSG_OK;
  if (offsets == nullptr || q_t == nullptr || scale == nullptr || (R > 0 && x == nullptr)) return NSG_ERR_INVALID_ARG;
  if (!rows_aligned(x, x_dtype) || !aligned(q_t, 16) || !aligned(scale, 4) || !aligned(offsets, 4) || !aligned(tokens, 4))
    return NSG_ERR_INVALID_ARG;
  QuantArgs a;
  a.x = x; a.x_dtype = x_dtype; a.f8 = q_dtype;
  a.B = 1; a.R = R; a.C = C; a.ldx = ldx;
  a.qt = q_t; a.st = scale;
  a.offsets = offsets; a.tokens = tokens; a.E = (int)E; a.P = P;
  return done(launch_quantize_columns(a, hs(stream)));
}

// ---- their products ------------------------------------------------------------

static nsg_status_t check_product(int32_t a_dtype, int32_t b_dtype, int32_t out_dtype, int64_t M, int64_t N, int64_t K) {
  if (!f8_dtype(a_dtype) || !f8_dtype(b_dtype) || !float_dtype(out_dtype)) return NSG_ERR_UNSUPPORTED_DTYPE;
  if (M < 0 || M > kMaxRows || N < 0 || N > kMaxSide || K < 0 || K > 2 * kMaxRows || K % kF8Block) return NSG_ERR_SHAPE;
  return NSG_OK;
}
static nsg_status_t check_operands(const void *qa, const float *sa, const void *qb, const float *sb, const void *out,
                                   int32_t out_dtype) {
  if (qa == nullptr || sa == nullptr || qb == nullptr || sb == nullptr || out == nullptr) return NSG_ERR_INVALID_ARG;
  if (!aligned(qa, 16) || !aligned(qb, 16) || !aligned(sa, 4) || !aligned(sb, 4) || !rows_aligned(out, out_dtype))
    return NSG_ERR_INVALID_ARG;
  return NSG_OK;
}
static bool block_ok(int32_t b) { return b == NSG_BLOCK_ROW || b == NSG_BLOCK_TILE; }

nsg_status_t nsg_gemm_fp8_nt(int32_t a_dtype, int32_t b_dtype, int32_t out_dtype, int64_t batch, int64_t M, int64_t N,
                             int64_t K, const void *qa, const float *sa, int32_t a_block, const void *qb,
                             const float *sb, int32_t b_block, void *out, void *stream) {
  nsg_status_t st = check_product(a_dtype, b_dtype, out_dtype, M, N, K);
  if (st != NSG_OK) return st;
  if (!block_ok(a_block) || !block_ok(b_block)) return NSG_ERR_INVALID_ARG;
  if (batch < 0 || batch > 65535) return NSG_ERR_SHAPE;
  if (batch == 0 || M == 0 || N == 0) return NSG_OK;
  if (K == 0) return NSG_ERR_SHAPE;
  st = check_operands(qa, sa, qb, sb, out, out_dtype);
  if (st != NSG_OK) return st;
  F8GemmArgs a;
  a.mode = kDense;
  a.a_dtype = a_dtype; a.b_dtype = b_dtype; a.out_dtype = out_dtype;
  a.batch = batch; a.M = M; a.N = N; a.K = K;
  a.A = qa; a.sa = sa; a.a_tile = a_block == NSG_BLOCK_TILE;
  a.B = qb; a.sb = sb; a.b_tile = b_block == NSG_BLOCK_TILE;
  a.out = out;
  return done(launch_gemm_f8(a, hs(stream)));
}

nsg_status_t nsg_expert_gemm_fp8(int32_t a_dtype, int32_t b_dtype, int32_t out_dtype, int64_t T, int64_t P, int64_t E,
                                 int64_t N, int64_t K, const void *qa, const float *sa, const int32_t *tokens,
                                 const void *qb, const float *sb, int32_t b_block, const int32_t *offsets, void *out,
                                 void *stream) {
  nsg_status_t st = check_product(a_dtype, b_dtype, out_dtype, P, N, K);
  if (st != NSG_OK) return st;
  if (!block_ok(b_block)) return NSG_ERR_INVALID_ARG;
  if (E < 1 || E > NSG_MAX_EXPERTS || T < 0 || T > kMaxRows || (tokens == nullptr && P > 0 && T != P)) return NSG_ERR_SHAPE;
  if (P == 0 || N == 0) return NSG_OK;
  if (K == 0 || T == 0) return NSG_ERR_SHAPE;
  st = check_operands(qa, sa, qb, sb, out, out_dtype);
  if (st != NSG_OK) return st;
  if (offsets == nullptr || !aligned(offsets, 4) || !aligned(tokens, 4)) return NSG_ERR_INVALID_ARG;
  F8GemmArgs a;
  a.mode = kExperts;
  a.a_dtype = a_dtype; a.b_dtype = b_dtype; a.out_dtype = out_dtype;
  a.M = P; a.N = N; a.K = K; a.T = T; a.E = (int)E;
  a.A = qa; a.sa = sa; a.tokens = tokens;
  a.B = qb; a.sb = sb; a.b_tile = b_block == NSG_BLOCK_TILE;
  a.offsets = offsets;
  a.out = out;
  return done(launch_gemm_f8(a, hs(stream)));
}

nsg_status_t nsg_expert_wgrad_fp8(int32_t a_dtype, int32_t b_dtype, int32_t out_dtype, int64_t P, int64_t E, int64_t N,
                                  int64_t K, const void *qa_t, const float *sa, const void *qb_t, const float *sb,
                                  const int32_t *offsets, void *out, void *stream) {
  int64_t cap = 0;
  nsg_status_t st = nsg_fp8_columns(P, E, &cap);
  if (st != NSG_OK) return st;
  if (N > kMaxSide) return NSG_ERR_SHAPE;
  st = check_product(a_dtype, b_dtype, out_dtype, N, K, cap);
  if (st != NSG_OK) return st;
  if (N == 0 || K == 0) return NSG_OK;
  st = check_operands(qa_t, sa, qb_t, sb, out, out_dtype);
  if (st != NSG_OK) return st;
  if (offsets == nullptr || !aligned(offsets, 4)) return NSG_ERR_INVALID_ARG;
  F8GemmArgs a;
  a.mode = kWgrad;
  a.a_dtype = a_dtype; a.b_dtype = b_dtype; a.out_dtype = out_dtype;
  a.M = N; a.N = K; a.K = cap; a.T = P; a.E = (int)E;
  a.A = qa_t; a.sa = sa;
  a.B = qb_t; a.sb = sb;
  a.offsets = offsets;
  a.out = out;
  return done(launch_gemm_f8(a, hs(stream)));
}

}  // extern "C"
