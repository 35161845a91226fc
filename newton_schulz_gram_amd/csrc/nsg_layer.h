// Internal interface of the operators between token ids and the expert layer: the
// embedding (nsg_embed.hip), layer norm (nsg_norm.hip), the router with its balance
// loss (nsg_route.hip), and their gradients, launched by nsg_layer_api.cpp.
// Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <hip/hip_runtime.h>

#include "nsg.h"

namespace nsg {

// ---- embedding (nsg_embed.hip) ----------------------------------------------
struct EmbedArgs {
  const void *ids = nullptr;
  int wide = 0;                // ids are int64, else int32
  int64_t T = 0, V = 0, C = 0;
  const void *x = nullptr;     // W [V][ld], or dout [T][ld]
  int x_dtype = NSG_BF16;
  int64_t ld = 0;
  float scale = 1.f;
  void *out = nullptr;         // [T][C] of x_dtype, or dW [V][C] of out_dtype
  int out_dtype = NSG_BF16;
  int accumulate = 0;          // dW: added to what out holds
  void *workspace = nullptr;   // dW
};
hipError_t launch_embedding(const EmbedArgs &a, hipStream_t s);
size_t embedding_backward_workspace(int64_t T, int64_t V, int64_t C);
hipError_t launch_embedding_backward(const EmbedArgs &a, hipStream_t s);

// ---- layer norm (nsg_norm.hip) ------------------------------------------------
struct NormArgs {
  const void *x = nullptr, *dy = nullptr;  // [R][ldx], [R][lddy]
  int dtype = NSG_BF16;
  int64_t R = 0, C = 0, ldx = 0, lddy = 0;
  const void *weight = nullptr, *bias = nullptr;  // [C] of w_dtype, or NULL
  int w_dtype = NSG_F32;
  float eps = 0.f;
  void *out = nullptr;                     // y or dx [R][C]
  float *stats = nullptr;                  // mean [R], rstd [R]
  void *dweight = nullptr, *dbias = nullptr;  // [C] of w_dtype, or NULL
  void *workspace = nullptr;
};
hipError_t launch_layer_norm(const NormArgs &a, hipStream_t s);
size_t layer_norm_backward_workspace(int64_t R, int64_t C);
hipError_t launch_layer_norm_backward(const NormArgs &a, hipStream_t s);

// ---- router (nsg_route.hip) -----------------------------------------------------
struct RouteArgs {
  const void *logits = nullptr;  // [T][ld]
  int dtype = NSG_F32;
  int64_t T = 0, ld = 0;
  int E = 0, k = 0, score = NSG_SCORE_SOFTMAX, normalize = 0;
  float scale = 1.f;
  const float *bias = nullptr;
  const uint8_t *mask = nullptr;
  int32_t *ids = nullptr;        // [T][k]
  float *weights = nullptr;      // [T][k]
  int32_t *counts = nullptr;     // [E + 1]; with probs [E] and loss [1]
  float *probs = nullptr, *loss = nullptr;
  void *workspace = nullptr;
  // gradient
  const float *dweights = nullptr, *dloss = nullptr;
  float balance = 0.f;
  void *dlogits = nullptr;       // [T][E]
};
size_t expert_route_workspace(int64_t T, int E);  // with the balance loss
hipError_t launch_expert_route(const RouteArgs &a, hipStream_t s);
hipError_t launch_expert_route_backward(const RouteArgs &a, hipStream_t s);

}  // namespace nsg
