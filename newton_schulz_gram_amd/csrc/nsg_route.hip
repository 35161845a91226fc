// The router in front of the experts, on gfx950: scores, choice, weights, balance
// loss, and their gradient.  For the logits l of a token,
//   s = softmax(l) or sigmoid(l),  p = s / sum s
//   choice   the k largest l, with a bias the k largest s + bias (in 64 bits, so
//            that scores next to each other are told apart); equal ones: the lower
//            index; NaN and -inf are never chosen
//   weights  w_j = scale s_j, normalised: scale s_j / sum over the chosen
//   balance  N tokens with a choice, counts[e] choices of expert e, probs[e] the
//            mean of p[e] over the N tokens, loss = E / (k N) sum_e counts[e] probs[e]
//
// L lanes share a token, a lane has N consecutive experts in registers.  The work is
// small (one read of the logits, a few instructions a logit): launches and the k
// rounds of the choice bound it.  Sums over tokens are fp32 in an order that only the
// sizes fix, counts are integers; there are no atomics on memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "nsg_layer.h"
#include "nsg_rows.h"

namespace nsg {

constexpr int kRouteThreads = 256;
constexpr int kRouteBlocks = 256;  // with the balance loss: workgroups whose sums are joined

// N consecutive logits from e on, -inf behind the last expert
template <typename T, int N> __device__ __forceinline__ void load_logits(const T *row, int e, int E, float (&f)[N]) {
  if (e + N <= E) {
    Row<T, N, (int)sizeof(T)>::load(row + e, f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = e + i < E ? (float)row[e + i] : -INFINITY;
  }
}

template <int L> __device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}
template <int L> __device__ __forceinline__ double lanes_max(double v) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) v = fmax(v, __shfl_xor(v, off, 64));
  return v;
}
template <int L, typename F> __device__ __forceinline__ F lanes_sum(F v) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// A score times a factor that is the same for all experts of a token, whose largest
// logit is `top`: no score that matters under- or overflows.  The score itself is
// this times score_factor.
template <typename F> __device__ __forceinline__ F shifted_score(int score, F l, F top) {
  if (score == NSG_SCORE_SIGMOID) return exp(fmin(l, (F)0) - fmin(top, (F)0)) / ((F)1 + exp(-fabs(l)));
  return exp(l - top);
}
__device__ __forceinline__ float sigmoid(float l) { return expf(fminf(l, 0.f)) / (1.f + expf(-fabsf(l))); }

// LDS written by some lanes of a wave is read by others
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The k largest keys of a token, one after the other, to id[j] and their logits to lg[j].
template <int N, int L, typename K>
__device__ __forceinline__ int choose(K (&key)[N], const float (&l)[N], int k, int sub, int32_t *id, float *lg) {
  const int lane = threadIdx.x & 63;
  const uint64_t group = (L == 64 ? ~0ull : (1ull << L) - 1) << (lane - sub);
  int found = 0;
  for (int j = 0; j < k; ++j) {
    K best = key[0];
    int at = 0;
    float mine = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
        mine = l[i];
      }
    const K top = lanes_max<L>(best);
    const bool some = top > -(K)INFINITY;
    const uint64_t who = __ballot(some && best == top) & group;
    const bool won = some && __ffsll((long long)who) - 1 == lane;
    if (won) {
      id[j] = sub * N + at;
      lg[j] = mine;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i == at) key[i] = -(K)INFINITY;
    } else if (!some && sub == 0) {
      id[j] = -1;
      lg[j] = -INFINITY;
    }
    found += some;
  }
  return found;
}

template <typename T, int N, int L, bool BIAS>
__global__ void __launch_bounds__(kRouteThreads) expert_route_kernel(RouteArgs p, float *__restrict__ sums, int32_t *__restrict__ cnts) {
  constexpr int kTokens = kRouteThreads / L;
  constexpr int kMost = N * L < NSG_MAX_CHOICES ? N * L : NSG_MAX_CHOICES;
  __shared__ int32_t id[kTokens][kMost];
  __shared__ float lg[kTokens][kMost];
  __shared__ int32_t count[NSG_MAX_EXPERTS + 1];
  __shared__ float red[kRouteThreads * N];
  const int sub = threadIdx.x % L, token = threadIdx.x / L, e0 = sub * N;
  const bool balance = sums != nullptr;
  if (balance) {
    for (int e = threadIdx.x; e <= p.E; e += kRouteThreads) count[e] = 0;
    __syncthreads();
  }
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < p.T; t0 += (int64_t)gridDim.x * kTokens) {
    const int64_t t = t0 + token;
    const bool there = t < p.T && (p.mask == nullptr || p.mask[t]);
    float l[N];
    if (there) {
      load_logits<T, N>((const T *)p.logits + t * p.ld, e0, p.E, l);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) l[i] = -INFINITY;
    }
    float top = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, l[i]);
    top = lanes_max<L>(top);
    if (!(top > -INFINITY)) top = 0.f;
    float s[N], sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = shifted_score<float>(p.score, l[i], top);
      if (e0 + i >= p.E) s[i] = 0.f;
      sum += s[i];
    }
    sum = lanes_sum<L>(sum);
    int found;
    if (BIAS) {
      double key[N], total = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        key[i] = shifted_score<double>(p.score, (double)l[i], (double)top);
        if (e0 + i < p.E) total += key[i];
      }
      total = p.score == NSG_SCORE_SIGMOID ? exp(fmin((double)top, 0.0)) : 1.0 / lanes_sum<L>(total);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const double v = e0 + i < p.E ? key[i] * total + (double)p.bias[e0 + i] : -(double)INFINITY;
        key[i] = l[i] > -INFINITY && v == v ? v : -(double)INFINITY;
      }
      found = choose<N, L, double>(key, l, p.k, sub, id[token], lg[token]);
    } else {
      float key[N];
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = l[i] == l[i] ? l[i] : -INFINITY;
      found = choose<N, L, float>(key, l, p.k, sub, id[token], lg[token]);
    }
    wave_sync();
    // the weights, a choice to a lane; with softmax a NaN among the logits is in all of them
    const bool softmax = p.score != NSG_SCORE_SIGMOID;
    const float poison = softmax && sum != sum ? sum : 0.f;
    float high = -INFINITY, whole = 0.f;
    if (p.normalize) {
      for (int j = sub; j < found; j += L) high = fmaxf(high, lg[token][j]);
      high = lanes_max<L>(high);
      for (int j = sub; j < found; j += L) whole += shifted_score<float>(p.score, lg[token][j], high);
      whole = lanes_sum<L>(whole);
    }
    if (t < p.T) {
      for (int j = sub; j < p.k; j += L) {
        float w = 0.f;
        if (j < found) {
          const float x = lg[token][j];
          if (p.normalize) w = shifted_score<float>(p.score, x, high) / whole;
          else w = softmax ? expf(x - top) / sum : sigmoid(x);
          w = w * p.scale + poison;
          if (balance) atomicAdd(&count[id[token][j]], 1);
        }
        p.ids[t * p.k + j] = id[token][j];
        p.weights[t * p.k + j] = w;
      }
    }
    if (balance && found > 0) {
      const float inv = 1.f / sum;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(s[i], inv, acc[i]);
      if (sub == 0) atomicAdd(&count[p.E], 1);
    }
    wave_sync();
  }
  if (!balance) return;
#pragma unroll
  for (int i = 0; i < N; ++i) red[token * (N * L) + e0 + i] = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
    float a = 0.f;
    for (int g = 0; g < kTokens; ++g) a += red[g * (N * L) + e];
    sums[(size_t)blockIdx.x * p.E + e] = a;
  }
  for (int e = threadIdx.x; e <= p.E; e += kRouteThreads) cnts[(size_t)blockIdx.x * (p.E + 1) + e] = count[e];
}

// One workgroup: 1024 / wide threads share the blocks' sums of an expert.
__global__ void __launch_bounds__(1024) expert_balance_kernel(RouteArgs p, int blocks, int wide, const float *__restrict__ sums,
                                                              const int32_t *__restrict__ cnts) {
  __shared__ float fs[1024];
  __shared__ int is[1024];
  __shared__ int tokens;
  const int share = 1024 / wide, e = threadIdx.x % wide, g = threadIdx.x / wide;
  float a = 0.f;
  int n = 0, all = 0;
  for (int b = threadIdx.x; b < blocks; b += 1024) all += cnts[(size_t)b * (p.E + 1) + p.E];
  if (e < p.E) {
    for (int b = g; b < blocks; b += share) {
      a += sums[(size_t)b * p.E + e];
      n += cnts[(size_t)b * (p.E + 1) + e];
    }
  }
  if (threadIdx.x == 0) tokens = 0;
  __syncthreads();
  if (all) atomicAdd(&tokens, all);
  fs[threadIdx.x] = a;
  is[threadIdx.x] = n;
  __syncthreads();
  const int N = tokens;
  float part = 0.f;
  if (g == 0 && e < p.E) {
    for (int i = 1; i < share; ++i) {
      a += fs[i * wide + e];
      n += is[i * wide + e];
    }
    a = N > 0 ? a / (float)N : 0.f;
    p.counts[e] = n;
    p.probs[e] = a;
    part = (float)n * a;
  }
  if (threadIdx.x == 0) p.counts[p.E] = N;
  __syncthreads();
  fs[threadIdx.x] = part;
  __syncthreads();
  for (int off = 512; off >= 1; off >>= 1) {
    if ((int)threadIdx.x < off) fs[threadIdx.x] += fs[threadIdx.x + off];
    __syncthreads();
  }
  if (threadIdx.x == 0) *p.loss = N > 0 ? fs[0] * ((float)p.E / ((float)p.k * (float)N)) : 0.f;
}

// ---------------------------------------------------------------------------
// the gradient.  With g_j = scale dw_j of the chosen,
//   softmax             dl_e = p_e (g_e - sum_j g_j p_j)
//   softmax normalised  dl_j = v_j (g_j - sum g v) for the chosen, v_j = s_j / sum of them
//   sigmoid             dl_j = g_j s_j (1 - s_j)
//   sigmoid normalised  dl_j = v_j (1 - s_j) (g_j - sum g v)
// and of the balance loss, c_e = balance dloss E counts[e] / (k N^2), for tokens with a
// choice  dl_e += p_e (c_e - sum p c), with sigmoid times 1 - s_e.
// ---------------------------------------------------------------------------
template <typename T, int N, int L>
__global__ void __launch_bounds__(kRouteThreads) expert_route_backward_kernel(RouteArgs p) {
  constexpr int kTokens = kRouteThreads / L;
  __shared__ float add[kTokens][N * L];  // what the choices of a token add at its experts
  const int sub = threadIdx.x % L, token = threadIdx.x / L, e0 = sub * N;
  const bool softmax = p.score != NSG_SCORE_SIGMOID;
  float c[N];
#pragma unroll
  for (int i = 0; i < N; ++i) c[i] = 0.f;
  if (p.counts != nullptr) {
    const float n = (float)p.counts[p.E];
    const float f = n > 0.f ? p.balance * (p.dloss != nullptr ? *p.dloss : 1.f) * ((float)p.E / (float)p.k) / n / n : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e0 + i < p.E) c[i] = f * (float)p.counts[e0 + i];
  }
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < p.T; t0 += (int64_t)gridDim.x * kTokens) {
    const int64_t t = t0 + token;
    const bool there = t < p.T;
    const T *row = (const T *)p.logits + (there ? t : 0) * p.ld;
    float l[N];
    load_logits<T, N>(row, e0, p.E, l);
#pragma unroll
    for (int i = 0; i < N; ++i) add[token][e0 + i] = 0.f;
    float top = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, l[i]);
    top = lanes_max<L>(top);
    if (!(top > -INFINITY)) top = 0.f;
    float s[N], sum = 0.f, pc = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = shifted_score<float>(p.score, l[i], top);
      if (e0 + i >= p.E) s[i] = 0.f;
      sum += s[i];
      pc = fmaf(s[i], c[i], pc);
    }
    sum = lanes_sum<L>(sum);
    pc = lanes_sum<L>(pc) / sum;
    // the choices, one to a lane at a time
    auto chosen = [&](int j, float &x) {
      const int e = there && j < p.k ? p.ids[t * p.k + j] : -1;
      const bool some = e >= 0 && e < p.E;
      x = some ? (float)row[e] : -INFINITY;
      return some ? e : -1;
    };
    float high = -INFINITY, whole = 0.f, dot = 0.f;
    int found = 0;
    for (int j = sub; j < p.k; j += L) {
      float x;
      found |= chosen(j, x) >= 0;
      high = fmaxf(high, x);
    }
    high = lanes_max<L>(high);
    found = __ballot(found) >> ((threadIdx.x & 63) - sub) & (L == 64 ? ~0ull : (1ull << L) - 1) ? 1 : 0;
    if (!(high > -INFINITY)) high = 0.f;
    if (p.dweights != nullptr) {
      for (int j = sub; j < p.k; j += L) {
        float x;
        if (chosen(j, x) < 0) continue;
        const float g = p.dweights[t * p.k + j] * p.scale;
        const float v = p.normalize ? shifted_score<float>(p.score, x, high) : softmax ? expf(x - top) : 0.f;
        whole += v;
        dot = fmaf(g, v, dot);
      }
      whole = lanes_sum<L>(whole);
      dot = lanes_sum<L>(dot) / (p.normalize ? whole : sum);
      wave_sync();
      for (int j = sub; j < p.k; j += L) {
        float x;
        const int e = chosen(j, x);
        if (e < 0) continue;
        const float g = p.dweights[t * p.k + j] * p.scale;
        float d = g;
        if (p.normalize) d = shifted_score<float>(p.score, x, high) / whole * (g - dot);
        if (!softmax) d *= p.normalize ? sigmoid(-x) : sigmoid(x) * sigmoid(-x);
        if (p.normalize && softmax && sum != sum) d = sum;
        atomicAdd(&add[token][e], d);
      }
      wave_sync();
    }
    if (there && e0 < p.E) {
      float d[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float a = add[token][e0 + i];
        const float pe = s[i] / sum;
        d[i] = softmax && !p.normalize && p.dweights != nullptr ? pe * (a - dot) : a;
        if (p.counts != nullptr) d[i] = fmaf(pe * (softmax ? 1.f : sigmoid(-l[i])), c[i] - pc, d[i]);
        if (!found) d[i] = 0.f;
      }
      T *to = (T *)p.dlogits + t * p.E;
      if (e0 + N <= p.E) {
        Row<T, N, (int)sizeof(T)>::store(to + e0, d);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (e0 + i < p.E) to[e0 + i] = (T)d[i];
      }
    }
    wave_sync();
  }
}

// ---------------------------------------------------------------------------
// workgroups of a launch over T tokens; with the balance loss each adds a row of sums
static int64_t route_blocks(int64_t T, int lanes, bool few) {
  const int64_t tokens = kRouteThreads / lanes, n = (T + tokens - 1) / tokens, most = few ? kRouteBlocks : 1 << 16;
  return n < most ? n : most;
}

// N and L for E experts
template <typename T, class K> static hipError_t by_experts(const RouteArgs &a, hipStream_t s) {
  if (a.E <= 16) return K::template launch<T, 4, 4>(a, s);
  if (a.E <= 64) return K::template launch<T, 4, 16>(a, s);
  if (a.E <= 128) return K::template launch<T, 8, 16>(a, s);
  if (a.E <= 256) return K::template launch<T, 16, 16>(a, s);
  if (a.E <= 512) return K::template launch<T, 16, 32>(a, s);
  return K::template launch<T, 16, 64>(a, s);
}

static size_t route_sums(int E) { return ((size_t)kRouteBlocks * (size_t)E * 4 + 15) / 16 * 16; }
size_t expert_route_workspace(int64_t T, int E) {
  return T == 0 ? 0 : route_sums(E) + (size_t)kRouteBlocks * (size_t)(E + 1) * 4;
}

struct RouteForward {
  template <typename T, int N, int L> static hipError_t launch(const RouteArgs &a, hipStream_t s) {
    const bool balance = a.counts != nullptr;
    float *sums = balance ? (float *)a.workspace : nullptr;
    int32_t *cnts = balance ? (int32_t *)((char *)a.workspace + route_sums(a.E)) : nullptr;
    const int64_t blocks = route_blocks(a.T, L, balance);
    if (blocks > 0) {
      if (a.bias != nullptr)
        hipLaunchKernelGGL((expert_route_kernel<T, N, L, true>), dim3((unsigned)blocks), dim3(kRouteThreads), 0, s, a, sums, cnts);
      else
        hipLaunchKernelGGL((expert_route_kernel<T, N, L, false>), dim3((unsigned)blocks), dim3(kRouteThreads), 0, s, a, sums, cnts);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (!balance) return hipSuccess;
    int wide = 1;
    while (wide < a.E) wide *= 2;
    hipLaunchKernelGGL(expert_balance_kernel, dim3(1), dim3(1024), 0, s, a, (int)blocks, wide, (const float *)sums,
                       (const int32_t *)cnts);
    return hipGetLastError();
  }
};
struct RouteBackward {
  template <typename T, int N, int L> static hipError_t launch(const RouteArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((expert_route_backward_kernel<T, N, L>), dim3((unsigned)route_blocks(a.T, L, false)), dim3(kRouteThreads),
                       0, s, a);
    return hipGetLastError();
  }
};

hipError_t launch_expert_route(const RouteArgs &a, hipStream_t s) {
  switch (a.dtype) {
    case NSG_F16: return by_experts<_Float16, RouteForward>(a, s);
    case NSG_BF16: return by_experts<__bf16, RouteForward>(a, s);
    default: return by_experts<float, RouteForward>(a, s);
  }
}
hipError_t launch_expert_route_backward(const RouteArgs &a, hipStream_t s) {
  switch (a.dtype) {
    case NSG_F16: return by_experts<_Float16, RouteBackward>(a, s);
    case NSG_BF16: return by_experts<__bf16, RouteBackward>(a, s);
    default: return by_experts<float, RouteBackward>(a, s);
  }
}

}  // namespace nsg
