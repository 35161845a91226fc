// C entry points of the operators between token ids and the expert layer
// (include/nsg.h): argument checks, then the launches on the caller's stream.
// Nothing is allocated and the host never waits.
#include <cmath>
#include <cstdint>

#include "nsg_layer.h"

using namespace nsg;

namespace {

constexpr int64_t kMaxRows = NSG_MAX_ROWS;
constexpr int64_t kMaxSide = NSG_MAX_SIDE;

bool float_dtype(int32_t d) { return d == NSG_F16 || d == NSG_BF16 || d == NSG_F32; }
bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool elem_aligned(const void *p, int32_t dtype) { return aligned(p, dtype == NSG_F32 ? 4 : 2); }
nsg_status_t done(hipError_t e) { return e == hipSuccess ? NSG_OK : NSG_ERR_HIP; }
hipStream_t hs(void *stream) { return reinterpret_cast<hipStream_t>(stream); }

// rows of C elements, ld apart
nsg_status_t check_rows(int64_t n, int64_t C, int64_t ld) {
  if (n < 0 || n > kMaxRows || C < 0 || C > kMaxSide || ld < C || ld > (1ll << 31)) return NSG_ERR_SHAPE;
  return NSG_OK;
}
// a workspace of `need` bytes
nsg_status_t check_space(const void *workspace, size_t bytes, size_t need) {
  if (need > 0 && (workspace == nullptr || bytes < need || !aligned(workspace, 16))) return NSG_ERR_WORKSPACE_TOO_SMALL;
  return NSG_OK;
}
nsg_status_t check_ids(const void *ids, int32_t id_bits, int64_t T) {
  if (T > 0 && ids == nullptr) return NSG_ERR_INVALID_ARG;
  return aligned(ids, (uintptr_t)(id_bits / 8)) ? NSG_OK : NSG_ERR_INVALID_ARG;
}
nsg_status_t check_router(int32_t dtype, int64_t T, int64_t E, int64_t ld, int64_t k, int32_t score, int32_t normalize, float scale) {
  if (!float_dtype(dtype)) return NSG_ERR_UNSUPPORTED_DTYPE;
  if (E < 1 || E > NSG_MAX_EXPERTS || k < 1 || k > NSG_MAX_CHOICES || k > E) return NSG_ERR_SHAPE;
  if (T < 0 || T > kMaxRows / k || ld < E || ld > (1ll << 31)) return NSG_ERR_SHAPE;
  if (score != NSG_SCORE_SOFTMAX && score != NSG_SCORE_SIGMOID) return NSG_ERR_INVALID_ARG;
  if ((normalize != 0 && normalize != 1) || !std::isfinite(scale)) return NSG_ERR_INVALID_ARG;
  return NSG_OK;
}

}  // namespace

extern "C" {

// ---- embedding -------------------------------------------------------------------

nsg_status_t nsg_embedding(const void *ids, int32_t id_bits, int64_t T, const void *W, int32_t dtype, int64_t V, int64_t C,
                           int64_t ldw, float scale, void *out, void *stream) {
  if (!float_dtype(dtype) || (id_bits != 32 && id_bits != 64)) return NSG_ERR_UNSUPPORTED_DTYPE;
  nsg_status_t st = check_rows(T, C, ldw);
  if (st != NSG_OK) return st;
  if (V < 0 || V > NSG_MAX_VOCAB) return NSG_ERR_SHAPE;
  if (!std::isfinite(scale)) return NSG_ERR_INVALID_ARG;
  if (T == 0 || C == 0) return NSG_OK;
  st = check_ids(ids, id_bits, T);
  if (st != NSG_OK) return st;
  if (out == nullptr || (V > 0 && W == nullptr) || !elem_aligned(W, dtype) || !elem_aligned(out, dtype)) return NSG_ERR_INVALID_ARG;
  EmbedArgs a;
  a.ids = ids; a.wide = id_bits == 64;
  a.T = T; a.V = V; a.C = C;
  a.x = W; a.x_dtype = dtype; a.ld = ldw;
  a.scale = scale;
  a.out = out; a.out_dtype = dtype;
  return done(launch_embedding(a, hs(stream)));
}

nsg_status_t nsg_embedding_backward_workspace_size(int64_t T, int64_t V, int64_t C, size_t *bytes) {
  if (bytes == nullptr) return NSG_ERR_INVALID_ARG;
  const nsg_status_t st = check_rows(T, C, C);
  if (st != NSG_OK) return st;
  if (V < 0 || V > NSG_MAX_VOCAB) return NSG_ERR_SHAPE;
  *bytes = V == 0 ? 0 : embedding_backward_workspace(T, V, C);
  return NSG_OK;
}

nsg_status_t nsg_embedding_backward(const void *dout, int32_t dtype, int64_t T, int64_t C, int64_t lddo, const void *ids,
                                    int32_t id_bits, int64_t V, float scale, void *dW, int32_t dw_dtype, int32_t accumulate,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  if (!float_dtype(dtype) || !float_dtype(dw_dtype) || (id_bits != 32 && id_bits != 64)) return NSG_ERR_UNSUPPORTED_DTYPE;
  size_t need = 0;
  nsg_status_t st = nsg_embedding_backward_workspace_size(T, V, C, &need);
  if (st == NSG_OK) st = check_rows(T, C, lddo);
  if (st != NSG_OK) return st;
  if ((accumulate != 0 && accumulate != 1) || !std::isfinite(scale)) return NSG_ERR_INVALID_ARG;
  if (V == 0 || C == 0 || (T == 0 && accumulate)) return NSG_OK;
  st = check_ids(ids, id_bits, T);
  if (st != NSG_OK) return st;
  if (dW == nullptr || (T > 0 && dout == nullptr) || !elem_aligned(dout, dtype) || !elem_aligned(dW, dw_dtype))
    return NSG_ERR_INVALID_ARG;
  st = check_space(workspace, workspace_bytes, need);
  if (st != NSG_OK) return st;
  EmbedArgs a;
  a.ids = ids; a.wide = id_bits == 64;
  a.T = T; a.V = V; a.C = C;
  a.x = dout; a.x_dtype = dtype; a.ld = lddo;
  a.scale = scale;
  a.out = dW; a.out_dtype = dw_dtype; a.accumulate = accumulate;
  a.workspace = workspace;
  return done(launch_embedding_backward(a, hs(stream)));
}

// ---- layer norm --------------------------------------------------------------------

nsg_status_t nsg_layer_norm(const void *x, int32_t dtype, int64_t R, int64_t C, int64_t ldx, const void *weight,
                            const void *bias, int32_t w_dtype, float eps, void *y, float *stats, void *stream) {
  if (!float_dtype(dtype) || !float_dtype(w_dtype)) return NSG_ERR_UNSUPPORTED_DTYPE;
  const nsg_status_t st = check_rows(R, C, ldx);
  if (st != NSG_OK) return st;
  if (C == 0 && R > 0) return NSG_ERR_SHAPE;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return NSG_ERR_INVALID_ARG;
  if (R == 0) return NSG_OK;
  if (x == nullptr || y == nullptr || stats == nullptr) return NSG_ERR_INVALID_ARG;
  if (!elem_aligned(x, dtype) || !elem_aligned(y, dtype) || !elem_aligned(weight, w_dtype) || !elem_aligned(bias, w_dtype) ||
      !aligned(stats, 4))
    return NSG_ERR_INVALID_ARG;
  NormArgs a;
  a.x = x; a.dtype = dtype;
  a.R = R; a.C = C; a.ldx = ldx;
  a.weight = weight; a.bias = bias; a.w_dtype = w_dtype;
  a.eps = eps;
  a.out = y; a.stats = stats;
  return done(launch_layer_norm(a, hs(stream)));
}

nsg_status_t nsg_layer_norm_backward_workspace_size(int64_t R, int64_t C, size_t *bytes) {
  if (bytes == nullptr) return NSG_ERR_INVALID_ARG;
  const nsg_status_t st = check_rows(R, C, C);
  if (st != NSG_OK) return st;
  *bytes = R == 0 || C == 0 ? 0 : layer_norm_backward_workspace(R, C);
  return NSG_OK;
}

nsg_status_t nsg_layer_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, int32_t dtype, int64_t R,
                                     int64_t C, const float *stats, const void *weight, int32_t w_dtype, void *dx,
                                     void *dweight, void *dbias, void *workspace, size_t workspace_bytes, void *stream) {
  if (!float_dtype(dtype) || !float_dtype(w_dtype)) return NSG_ERR_UNSUPPORTED_DTYPE;
  nsg_status_t st = check_rows(R, C, ldx);
  if (st == NSG_OK) st = check_rows(R, C, lddy);
  if (st != NSG_OK) return st;
  if (C == 0) return R > 0 ? NSG_ERR_SHAPE : NSG_OK;
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (R > 0 && (dy == nullptr || x == nullptr || stats == nullptr || dx == nullptr)) return NSG_ERR_INVALID_ARG;
  if (!elem_aligned(dy, dtype) || !elem_aligned(x, dtype) || !elem_aligned(dx, dtype) || !elem_aligned(weight, w_dtype) ||
      !elem_aligned(dweight, w_dtype) || !elem_aligned(dbias, w_dtype) || !aligned(stats, 4))
    return NSG_ERR_INVALID_ARG;
  size_t need = 0;
  st = nsg_layer_norm_backward_workspace_size(R, C, &need);
  if (st == NSG_OK) st = check_space(workspace, workspace_bytes, sums ? need : 0);
  if (st != NSG_OK) return st;
  if (R == 0 && !sums) return NSG_OK;
  NormArgs a;
  a.x = x; a.dy = dy; a.dtype = dtype;
  a.R = R; a.C = C; a.ldx = ldx; a.lddy = lddy;
  a.weight = weight; a.w_dtype = w_dtype;
  a.out = dx; a.stats = const_cast<float *>(stats);
  a.dweight = dweight; a.dbias = dbias;
  a.workspace = workspace;
  return done(launch_layer_norm_backward(a, hs(stream)));
}

// ---- router --------------------------------------------------------------------------

nsg_status_t nsg_expert_route_workspace_size(int64_t T, int64_t E, size_t *bytes) {
  if (bytes == nullptr) return NSG_ERR_INVALID_ARG;
  if (T < 0 || T > kMaxRows || E < 1 || E > NSG_MAX_EXPERTS) return NSG_ERR_SHAPE;
  *bytes = expert_route_workspace(T, (int)E);
  return NSG_OK;
}

nsg_status_t nsg_expert_route(const void *logits, int32_t dtype, int64_t T, int64_t E, int64_t ld, int64_t k, int32_t score,
                              const float *bias, const uint8_t *mask, int32_t normalize, float scale, int32_t *ids,
                              float *weights, int32_t *counts, float *probs, float *loss, void *workspace,
                              size_t workspace_bytes, void *stream) {
  nsg_status_t st = check_router(dtype, T, E, ld, k, score, normalize, scale);
  if (st != NSG_OK) return st;
  const bool balance = counts != nullptr;
  if ((probs != nullptr) != balance || (loss != nullptr) != balance) return NSG_ERR_INVALID_ARG;
  if (T > 0 && (logits == nullptr || ids == nullptr || weights == nullptr)) return NSG_ERR_INVALID_ARG;
  if (!elem_aligned(logits, dtype) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(counts, 4) ||
      !aligned(probs, 4) || !aligned(loss, 4))
    return NSG_ERR_INVALID_ARG;
  if (balance) st = check_space(workspace, workspace_bytes, expert_route_workspace(T, (int)E));
  if (st != NSG_OK) return st;
  if (T == 0 && !balance) return NSG_OK;
  RouteArgs a;
  a.logits = logits; a.dtype = dtype;
  a.T = T; a.E = (int)E; a.ld = ld;
  a.k = (int)k; a.score = score; a.normalize = normalize; a.scale = scale;
  a.bias = bias; a.mask = mask;
  a.ids = ids; a.weights = weights;
  a.counts = counts; a.probs = probs; a.loss = loss;
  a.workspace = workspace;
  return done(launch_expert_route(a, hs(stream)));
}

nsg_status_t nsg_expert_route_backward(const void *logits, int32_t dtype, int64_t T, int64_t E, int64_t ld, int64_t k,
                                       int32_t score, int32_t normalize, float scale, const int32_t *ids,
                                       const float *dweights, const int32_t *counts, float balance, const float *dloss,
                                       void *dlogits, void *stream) {
  const nsg_status_t st = check_router(dtype, T, E, ld, k, score, normalize, scale);
  if (st != NSG_OK) return st;
  if (!std::isfinite(balance)) return NSG_ERR_INVALID_ARG;
  if (T == 0) return NSG_OK;
  if (logits == nullptr || ids == nullptr || dlogits == nullptr || (dloss != nullptr && counts == nullptr)) return NSG_ERR_INVALID_ARG;
  if (!elem_aligned(logits, dtype) || !elem_aligned(dlogits, dtype) || !aligned(ids, 4) || !aligned(dweights, 4) ||
      !aligned(counts, 4) || !aligned(dloss, 4))
    return NSG_ERR_INVALID_ARG;
  RouteArgs a;
  a.logits = logits; a.dtype = dtype;
  a.T = T; a.E = (int)E; a.ld = ld;
  a.k = (int)k; a.score = score; a.normalize = normalize; a.scale = scale;
  a.ids = const_cast<int32_t *>(ids);
  a.dweights = dweights;
  a.counts = const_cast<int32_t *>(counts);
  a.balance = balance; a.dloss = dloss;
  a.dlogits = dlogits;
  return done(launch_expert_route_backward(a, hs(stream)));
}

}  // extern "C"
