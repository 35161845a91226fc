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
constexpr int kBalanceBlocks = 256;  // with the balance loss: workgroups, whose sums are joined

// N consecutive logits of a row from e on, -inf behind the last expert.  (The type of
// the logits is the same in all lanes: one branch a row instead of three kernels.)
template <typename T, int N> __device__ __forceinline__ void load_as(const T *row, int e, int E, float (&f)[N]) {
  if (e + N <= E) {
    Row<T, N, (int)sizeof(T)>::load(row + e, f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = e + i < E ? (float)row[e + i] : -INFINITY;
  }
}
template <int N> __device__ __forceinline__ void load_logits(const RouteArgs &p, int64_t t, int e, float (&f)[N]) {
  const int64_t at = t * p.ld;
  if (p.dtype == NSG_F32) load_as((const float *)p.logits + at, e, p.E, f);
  else if (p.dtype == NSG_BF16) load_as((const __bf16 *)p.logits + at, e, p.E, f);
  else load_as((const _Float16 *)p.logits + at, e, p.E, f);
}
__device__ __forceinline__ float logit(const RouteArgs &p, int64_t t, int e) {
  const int64_t at = t * p.ld + e;
  if (p.dtype == NSG_F32) return ((const float *)p.logits)[at];
  return p.dtype == NSG_BF16 ? (float)((const __bf16 *)p.logits)[at] : (float)((const _Float16 *)p.logits)[at];
}
template <typename T, int N> __device__ __forceinline__ void store_as(T *row, int e, int E, const float (&f)[N]) {
  if (e + N <= E) {
    Row<T, N, (int)sizeof(T)>::store(row + e, f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e + i < E) row[e + i] = (T)f[i];
  }
}

// ---------------------------------------------------------------------------
// Groups of L lanes, which a token's logits are spread over
// ---------------------------------------------------------------------------
template <int CTRL> __device__ __forceinline__ float lane_swap(float v) {
  const int x = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, true));
}
// The values of two halves of 32 (64) lanes, each in all of them
template <int L> __device__ __forceinline__ void half_swap(float v, float &a, float &b) {
  const unsigned x = __builtin_bit_cast(unsigned, v);
  const auto r = L == 32 ? __builtin_amdgcn_permlane16_swap(x, x, false, false) : __builtin_amdgcn_permlane32_swap(x, x, false, false);
  a = __builtin_bit_cast(float, (unsigned)r[0]);
  b = __builtin_bit_cast(float, (unsigned)r[1]);
}
// op over the group, the same in all its lanes: both lanes of a pair join the same two
// values, so sums are the same too
template <int L, class Op> __device__ __forceinline__ float group_join(float v, Op op) {
  v = op(v, lane_swap<0xB1>(v));  // lanes 1, 0, 3, 2 of four
  v = op(v, lane_swap<0x4E>(v));  // lanes 2, 3, 0, 1
  if (L >= 16) {
    v = op(v, lane_swap<0x141>(v));  // eight lanes mirrored
    v = op(v, lane_swap<0x140>(v));  // sixteen
  }
  float a, b;
  if (L >= 32) {
    half_swap<32>(v, a, b);
    v = op(a, b);
  }
  if (L >= 64) {
    half_swap<64>(v, a, b);
    v = op(a, b);
  }
  return v;
}
template <int L> __device__ __forceinline__ float group_max(float v) {
  return group_join<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L> __device__ __forceinline__ float group_sum(float v) {
  return group_join<L>(v, [](float a, float b) { return a + b; });
}
// lanes of this lane's group among those of the wave
template <int L> __device__ __forceinline__ uint64_t group_lanes() {
  const int lane = threadIdx.x & 63;
  return (L == 64 ? ~0ull : (1ull << L) - 1) << (lane / L * L);
}
// LDS written by some lanes of a wave is read by others
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------
// e^x for x <= 0 within 2 units of its last place, 0 from -104 on: 2^h (1 + r ln 2)
// for x log2 e = h + r, h in fp32 (a fifth of the instructions of expf; NaN stays NaN)
__device__ __forceinline__ float exp_down(float x) {
  x = x < -104.f ? -104.f : x;
  const float h = x * 1.44269502f;  // log2 e = 1.44269502 + 1.9259630e-8
  const float r = fmaf(x, 1.9259630e-8f, fmaf(x, 1.44269502f, -h));
  const float v = __builtin_amdgcn_exp2f(h);
  return fmaf(v, r * 0.693147181f, v);
}
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }  // within 1 unit

// 1 / x for a sum of scores; 0 where nothing has one
__device__ __forceinline__ float inverse_sum(float x) { return x == 0.f ? 0.f : 1.f / x; }

// The score of one logit times e^-shift; of all of a token's logits, see score_shift
template <bool SIGMOID> __device__ __forceinline__ float shifted_score(float l, float shift) {
  if (!SIGMOID) return exp_down(l - shift);
  return exp_down(fminf(l, 0.f) - shift) * inverse(1.f + exp_down(-fabsf(l)));
}
__device__ __forceinline__ float sigmoid(float l) {
  const float e = exp_down(-fabsf(l));
  return (l >= 0.f ? 1.f : e) * inverse(1.f + e);
}

// A token's scores times a factor that they share, so that none that matters under- or
// overflows: softmax e^(l - shift) with shift the largest logit, sigmoid
// sigmoid(l) e^-shift with shift 0 unless the largest logit is far below it.
template <bool SIGMOID> __device__ __forceinline__ float score_shift(float top) {
  return SIGMOID ? (top < -60.f ? top : 0.f) : top;
}
// scores s and their sum; behind the last expert, where l is -inf, they are 0
template <bool SIGMOID, int N, int L> __device__ __forceinline__ float scores(const float (&l)[N], float shift, float (&s)[N]) {
  float sum = 0.f;
  if (SIGMOID && __ballot(shift != 0.f) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = sigmoid(l[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = shifted_score<SIGMOID>(l[i], shift);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) sum += s[i];
  return group_sum<L>(sum);
}

// ---------------------------------------------------------------------------
// choice
// ---------------------------------------------------------------------------
// The k largest of a token's keys, one after the other, equal ones by index: index and
// key to id[j], val[j], -1 and -inf where none is left.  Returns how many there were.
//
// With gap > 0 the keys are off by rounding: two of them are `close` if they are less than
// gap (sizes + 1/8 of the largest size of a key) apart, else their order is right.  Then the
// keys that come next are taken too, at most kNext, until one is not close to the k-th:
// the first k in the right order are among these `taken` ones, unless `more`.
constexpr int kNext = 16;
struct Closeness {
  float gap, sizes;
  bool close, more;
  int taken;
};
template <int N, int L, bool GAPS>
__device__ __forceinline__ int choose(float (&key)[N], int k, int sub, int32_t *id, float *val, Closeness &c) {
  const int lane = threadIdx.x & 63;
  const uint64_t group = group_lanes<L>();
  const int rounds = GAPS ? k + kNext : k;
  int found = 0, taken = 0;
  float first = 0.f, last = INFINITY, kth = 0.f, least = INFINITY;
  bool on = true;
  for (int j = 0; j < rounds; ++j) {
    float best = key[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = fmaxf(best, key[i]);
    const float top = group_max<L>(best);
    const bool some = top > -INFINITY;
    if (GAPS) {
      if (j == 0) first = top;
      const float margin = c.gap * (c.sizes + 0.125f * fmaxf(fabsf(first), fabsf(top)));
      if (j >= k) {
        on = on && some && !(kth - top > margin);
        if (__ballot(on) == 0) break;
      }
      if (some && on && !(last - top > margin)) least = 0.f;
      last = top;
      if (j == k - 1) kth = top;
    }
    const uint64_t who = __ballot(some && best == top) & group;
    if (on && some && __ffsll((unsigned long long)who) - 1 == lane) {
      int at = 0;
      bool hit = false;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool now = key[i] == top && !hit;
        key[i] = now ? -INFINITY : key[i];
        at = now ? i : at;
        hit = hit || now;
      }
      id[j] = sub * N + at;
      val[j] = top;
    } else if (!some && j < k && sub == 0) {
      id[j] = -1;
      val[j] = -INFINITY;
    }
    if (j < k) found += some;
    taken += some && on;
  }
  if (GAPS) {
    c.close = least == 0.f;
    c.taken = taken;
    c.more = c.close && on && taken == k + kNext;
  }
  return found;
}

// The same with keys in 64 bits.
template <int N, int L> __device__ __forceinline__ void choose64(double (&key)[N], int k, int sub, int32_t *id, bool write) {
  const int lane = threadIdx.x & 63;
  const uint64_t group = group_lanes<L>();
  for (int j = 0; j < k; ++j) {
    double best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    double top = best;
#pragma unroll
    for (int off = L / 2; off >= 1; off >>= 1) top = fmax(top, __shfl_xor(top, off, 64));
    const bool some = top > -(double)INFINITY;
    const uint64_t who = __ballot(some && best == top) & group;
    const bool won = some && __ffsll((unsigned long long)who) - 1 == lane;
    if (won) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i == at) key[i] = -(double)INFINITY;
    }
    if (write && (won || (!some && sub == 0))) id[j] = some ? sub * N + at : -1;
  }
}

struct BalanceRow {  // a workgroup's sum and count of an expert; behind the last one, its tokens
  float sum;
  int32_t count;
};
static int64_t balance_pitch(int E) { return (E + 2) / 2 * 2; }

// LDS of a token: the chosen experts and what chose them; with a bias also those that
// come next, their exact keys and the order of these
static __host__ __device__ int route_kept(int k, int E, bool bias) { return bias ? (k + kNext < E ? k + kNext : E) : k; }
static __host__ __device__ int route_room(int k, int E, bool bias) { return route_kept(k, E, bias) * (bias ? 20 : 8); }

template <int N> constexpr int kBalanceThreads = N > 8 ? 512 : 1024;

template <int N, int L, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(kBalanceThreads<N>) expert_route_kernel(RouteArgs p, BalanceRow *__restrict__ rows, int64_t pitch) {
  extern __shared__ __attribute__((aligned(16))) char room[];
  __shared__ int32_t count[NSG_MAX_EXPERTS + 1];
  __shared__ float total[NSG_MAX_EXPERTS];
  const int tokens = blockDim.x / L;
  const int sub = threadIdx.x % L, token = threadIdx.x / L, e0 = sub * N;
  const int kept = route_kept(p.k, p.E, BIAS);
  double *const exact = reinterpret_cast<double *>(room) + (BIAS ? token * kept : 0);
  int32_t *const id = reinterpret_cast<int32_t *>(room + (BIAS ? tokens * kept * 8 : 0)) + token * kept;
  float *const val = reinterpret_cast<float *>(id + tokens * kept);
  int32_t *const sorted = id + 2 * tokens * kept;  // (BIAS)
  constexpr bool softmax = !SIGMOID;
  const bool balance = rows != nullptr;
  if (balance) {
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) count[e] = 0;
    __syncthreads();
  }
  float acc[N], bias[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    acc[i] = 0.f;
    bias[i] = BIAS && e0 + i < p.E ? p.bias[e0 + i] : 0.f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < p.T; t0 += (int64_t)gridDim.x * tokens) {
    const int64_t t = t0 + token;
    const bool there = t < p.T && (p.mask == nullptr || p.mask[t]);
    float l[N];
    if (there) {
      load_logits<N>(p, t, e0, l);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) l[i] = -INFINITY;
    }
    float top = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, l[i]);
    top = group_max<L>(top);
    if (!(top > -INFINITY)) top = 0.f;
    const float shift = score_shift<SIGMOID>(top);
    float s[N], sum = 0.f;
    if (balance || BIAS || softmax) sum = scores<SIGMOID, N, L>(l, shift, s);
    int found;
    if (BIAS) {
      float key[N];
      const float whole = softmax ? inverse(sum) : shift == 0.f ? 1.f : exp_down(shift);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float v = fmaf(s[i], whole, bias[i]);
        key[i] = l[i] > -INFINITY && v == v ? v : -INFINITY;
      }
      // Scores, at most `whole` times the largest shifted one, are off by less than 32
      // roundings of that, with the bias by one of the key.
      Closeness c{64.f * 0x1p-24f, softmax ? whole : 1.f, false, false, 0};
      found = choose<N, L, true>(key, p.k, sub, id, val, c);
      if (__ballot(c.close) != 0) {
        // keys in 64 bits: of the taken experts, or all where the next ones did not end
        double all = 1.0;
        if (softmax) {
          all = 0;
#pragma unroll
          for (int i = 0; i < N; ++i) all += l[i] > -INFINITY ? exp((double)l[i] - (double)top) : 0.0;
#pragma unroll
          for (int off = L / 2; off >= 1; off >>= 1) all += __shfl_xor(all, off, 64);
        }
        auto key64 = [&](float x, float b) {
          const double v = (double)x;
          return (softmax ? exp(v - (double)top) / all : (v >= 0 ? 1.0 : exp(v)) / (1.0 + exp(-fabs(v)))) + (double)b;
        };
        wave_sync();
        if (c.close && !c.more) {
          for (int j = sub; j < c.taken; j += L) exact[j] = key64(logit(p, t, id[j]), p.bias[id[j]]);
        }
        wave_sync();
        if (c.close && !c.more) {
          for (int j = sub; j < c.taken; j += L) {
            int rank = 0;
            for (int i = 0; i < c.taken; ++i) rank += exact[i] > exact[j] || (exact[i] == exact[j] && id[i] < id[j]);
            sorted[rank] = id[j];
          }
        }
        wave_sync();
        if (c.close && !c.more) {
          for (int j = sub; j < found; j += L) id[j] = sorted[j];
        }
        if (__ballot(c.more) != 0) {
          double whole64[N];
#pragma unroll
          for (int i = 0; i < N; ++i) whole64[i] = l[i] > -INFINITY && bias[i] > -INFINITY ? key64(l[i], bias[i]) : -(double)INFINITY;
          wave_sync();
          choose64<N, L>(whole64, p.k, sub, id, c.more);
        }
      }
      wave_sync();
      for (int j = sub; j < found; j += L) val[j] = logit(p, t, id[j]);
    } else {
      float key[N];
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = l[i] == l[i] ? l[i] : -INFINITY;
      Closeness c{};
      found = choose<N, L, false>(key, p.k, sub, id, val, c);
    }
    wave_sync();
    // the weights, a choice to a lane; with softmax a NaN among the logits is in all of them
    float high = -INFINITY, whole = 0.f;
    if (p.normalize) {
      for (int j = sub; j < found; j += L) high = fmaxf(high, val[j]);
      high = score_shift<SIGMOID>(group_max<L>(high));
      for (int j = sub; j < found; j += L) whole += shifted_score<SIGMOID>(val[j], high);
      whole = p.scale / group_sum<L>(whole);
    } else {
      whole = softmax ? p.scale / sum : p.scale;
    }
    if (t < p.T) {
      for (int j = sub; j < p.k; j += L) {
        float w = 0.f;
        if (j < found) {
          const float x = val[j];
          w = whole * (p.normalize ? shifted_score<SIGMOID>(x, high) : softmax ? exp_down(x - top) : sigmoid(x));
          if (softmax && sum != sum) w = sum;
          if (balance) atomicAdd(&count[id[j]], 1);
        }
        p.ids[t * p.k + j] = id[j];
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
  // the groups' sums, one group after the other in a wave, one wave after the other
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float v = acc[i];
#pragma unroll
    for (int off = L; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
    acc[i] = v;
  }
  for (int w = 0; w < (int)blockDim.x / 64; ++w) {
    if ((int)threadIdx.x / 64 == w && (threadIdx.x & 63) < L) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e0 + i < p.E) total[e0 + i] = w == 0 ? acc[i] : total[e0 + i] + acc[i];
    }
    __syncthreads();
  }
  BalanceRow *to = rows + (int64_t)blockIdx.x * pitch;
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) to[e] = BalanceRow{e < p.E ? total[e] : 0.f, count[e]};
}

// One workgroup: groups of `pitch / 2` threads share the rows, a thread two experts of them.
__global__ void __launch_bounds__(1024) expert_balance_kernel(RouteArgs p, int blocks, const BalanceRow *__restrict__ rows,
                                                              int64_t pitch) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  __shared__ float fs[2][1024];
  __shared__ int is[2][1024];
  __shared__ float part[16];
  __shared__ int tokens;
  const int units = (int)pitch / 2, share = 1024 / units, u = (int)threadIdx.x % units, g = (int)threadIdx.x / units;
  float a0 = 0.f, a1 = 0.f;
  int n0 = 0, n1 = 0;
  if (g < share) {
    for (int b0 = g; b0 < blocks; b0 += 16 * share) {
      u32x4 v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int b = b0 + i * share;
        v[i] = b < blocks ? *reinterpret_cast<const u32x4 *>(rows + (int64_t)b * pitch + 2 * u) : u32x4(0);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        a0 += __uint_as_float(v[i][0]);
        n0 += (int)v[i][1];
        a1 += __uint_as_float(v[i][2]);
        n1 += (int)v[i][3];
      }
    }
  }
  fs[0][threadIdx.x] = a0;
  fs[1][threadIdx.x] = a1;
  is[0][threadIdx.x] = n0;
  is[1][threadIdx.x] = n1;
  __syncthreads();
  const bool mine = g == 0 && u < units;
  if (mine) {
    for (int i = 1; i < share; ++i) {
      a0 += fs[0][i * units + u];
      a1 += fs[1][i * units + u];
      n0 += is[0][i * units + u];
      n1 += is[1][i * units + u];
    }
    if (2 * u == p.E) tokens = n0;
    if (2 * u + 1 == p.E) tokens = n1;
  }
  __syncthreads();
  const int N = tokens;
  float v = 0.f;
  if (mine) {
    a0 = N > 0 ? a0 / (float)N : 0.f;
    a1 = N > 0 ? a1 / (float)N : 0.f;
    if (2 * u < p.E) {
      p.counts[2 * u] = n0;
      p.probs[2 * u] = a0;
      v = (float)n0 * a0;
    }
    if (2 * u + 1 < p.E) {
      p.counts[2 * u + 1] = n1;
      p.probs[2 * u + 1] = a1;
      v = fmaf((float)n1, a1, v);
    }
  }
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    p.counts[p.E] = N;
    v = 0.f;
    for (int w = 0; w < 16; ++w) v += part[w];
    *p.loss = N > 0 ? v * ((float)p.E / ((float)p.k * (float)N)) : 0.f;
  }
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
template <int N, int L, bool SIGMOID>
__global__ void __launch_bounds__(kRouteThreads) expert_route_backward_kernel(RouteArgs p) {
  constexpr int kTokens = kRouteThreads / L;
  constexpr int kMost = N * L < NSG_MAX_CHOICES ? N * L : NSG_MAX_CHOICES, kMine = kMost / L;
  // what the choices of a token add at its experts, expert e at (e % N) L + e / N: lanes read
  // next to each other.  It is all zeros between tokens.
  __shared__ float add[kTokens][N * L];
  const int sub = threadIdx.x % L, token = threadIdx.x / L, e0 = sub * N;
  constexpr bool softmax = !SIGMOID;
  const bool weights = p.dweights != nullptr;
  const uint64_t group = group_lanes<L>();
  float c[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    c[i] = 0.f;
    add[token][i * L + sub] = 0.f;
  }
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
    // this lane's choices (j = sub, sub + L, ...), and the logits
    int e[kMine];
    float g[kMine], x[kMine];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int j = sub + m * L;
      const bool in = there && j < p.k;
      e[m] = in ? p.ids[t * p.k + j] : -1;
      if (e[m] >= p.E) e[m] = -1;
      g[m] = in && weights ? p.dweights[t * p.k + j] * p.scale : 0.f;
    }
    float l[N];
    load_logits<N>(p, there ? t : 0, e0, l);
    bool any = false;
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      any = any || e[m] >= 0;
      x[m] = e[m] >= 0 ? logit(p, t, e[m]) : -INFINITY;
    }
    const bool found = (__ballot(any) & group) != 0;
    float top = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, l[i]);
    top = group_max<L>(top);
    if (!(top > -INFINITY)) top = 0.f;
    float s[N], pc = 0.f;
    const float sum = inverse_sum(scores<SIGMOID, N, L>(l, score_shift<SIGMOID>(top), s));
#pragma unroll
    for (int i = 0; i < N; ++i) pc = fmaf(s[i], c[i], pc);
    pc = group_sum<L>(pc) * sum;
    float dot = 0.f;
    if (weights) {
      float high = -INFINITY, whole = 0.f, v[kMine];
#pragma unroll
      for (int m = 0; m < kMine; ++m) high = fmaxf(high, x[m]);
      high = group_max<L>(high);
      high = high > -INFINITY ? score_shift<SIGMOID>(high) : 0.f;
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        v[m] = p.normalize ? shifted_score<SIGMOID>(x[m], high) : softmax ? exp_down(x[m] - top) : 0.f;
        if (e[m] < 0) v[m] = 0.f;
        whole += v[m];
        dot = fmaf(g[m], v[m], dot);
      }
      whole = p.normalize ? inverse_sum(group_sum<L>(whole)) : sum;
      dot = group_sum<L>(dot) * whole;
      wave_sync();
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        if (e[m] < 0) continue;
        float d = g[m];
        if (p.normalize) d = v[m] * whole * (g[m] - dot);
        if (!softmax) d *= p.normalize ? sigmoid(-x[m]) : sigmoid(x[m]) * sigmoid(-x[m]);
        if (p.normalize && softmax && sum != sum) d = sum;
        atomicAdd(&add[token][e[m] % N * L + e[m] / N], d);
      }
      wave_sync();
    }
    float d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = weights ? add[token][i * L + sub] : 0.f;
    if (weights) {
      wave_sync();
#pragma unroll
      for (int m = 0; m < kMine; ++m)
        if (e[m] >= 0) add[token][e[m] % N * L + e[m] / N] = 0.f;
      wave_sync();
    }
    if (there && e0 < p.E) {
      const bool full = softmax && !p.normalize && weights;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float pe = s[i] * sum;
        if (full) d[i] = pe * (d[i] - dot);
        if (p.counts != nullptr) d[i] = fmaf(softmax ? pe : pe * sigmoid(-l[i]), c[i] - pc, d[i]);
        if (!found) d[i] = 0.f;
      }
      const int64_t to = t * p.E;
      if (p.dtype == NSG_F32) store_as((float *)p.dlogits + to, e0, p.E, d);
      else if (p.dtype == NSG_BF16) store_as((__bf16 *)p.dlogits + to, e0, p.E, d);
      else store_as((_Float16 *)p.dlogits + to, e0, p.E, d);
    }
    wave_sync();
  }
}

// ---------------------------------------------------------------------------
// workgroups of `threads` for T tokens of so many lanes, at most `most`
static int64_t route_blocks(int64_t T, int threads, int lanes, int64_t most) {
  const int64_t tokens = threads / lanes, n = (T + tokens - 1) / tokens;
  return n < most ? n : most;
}

// N and L for E experts
template <class K> static hipError_t by_experts(const RouteArgs &a, hipStream_t s) {
  const bool few = a.T <= 1024;
  if (a.E <= 16) return K::template launch<4, 4>(a, s);
  if (a.E <= 64) return few ? K::template launch<1, 64>(a, s) : K::template launch<4, 16>(a, s);
  if (a.E <= 128) return few ? K::template launch<2, 64>(a, s) : K::template launch<8, 16>(a, s);
  if (a.E <= 256) return few ? K::template launch<4, 64>(a, s) : K::template launch<8, 32>(a, s);
  if (a.E <= 512) return K::template launch<8, 64>(a, s);
  return K::template launch<16, 64>(a, s);
}

size_t expert_route_workspace(int64_t T, int E) {
  return T == 0 ? 0 : (size_t)kBalanceBlocks * (size_t)balance_pitch(E) * sizeof(BalanceRow);
}

struct RouteForward {
  template <int N, int L> static hipError_t launch(const RouteArgs &a, hipStream_t s) {
    const bool balance = a.counts != nullptr;
    // with the balance loss as many threads as the choices' LDS allows: few rows to join
    int threads = balance ? kBalanceThreads<N> : kRouteThreads;
    const int room = route_room(a.k, a.E, a.bias != nullptr);
    while (threads > 64 && threads / L * room > 48 << 10) threads /= 2;
    const int64_t pitch = balance_pitch(a.E), blocks = route_blocks(a.T, threads, L, balance ? kBalanceBlocks : 1 << 16);
    BalanceRow *rows = balance ? (BalanceRow *)a.workspace : nullptr;
    if (blocks > 0) {
      const dim3 grid((unsigned)blocks), block(threads);
      const unsigned lds = (unsigned)(threads / L * room);
      if (a.score == NSG_SCORE_SIGMOID && a.bias != nullptr)
        hipLaunchKernelGGL((expert_route_kernel<N, L, true, true>), grid, block, lds, s, a, rows, pitch);
      else if (a.score == NSG_SCORE_SIGMOID)
        hipLaunchKernelGGL((expert_route_kernel<N, L, true, false>), grid, block, lds, s, a, rows, pitch);
      else if (a.bias != nullptr)
        hipLaunchKernelGGL((expert_route_kernel<N, L, false, true>), grid, block, lds, s, a, rows, pitch);
      else
        hipLaunchKernelGGL((expert_route_kernel<N, L, false, false>), grid, block, lds, s, a, rows, pitch);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (!balance) return hipSuccess;
    hipLaunchKernelGGL(expert_balance_kernel, dim3(1), dim3(1024), 0, s, a, (int)blocks, (const BalanceRow *)rows, pitch);
    return hipGetLastError();
  }
};
struct RouteBackward {
  template <int N, int L> static hipError_t launch(const RouteArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)route_blocks(a.T, kRouteThreads, L, 1 << 16)), block(kRouteThreads);
    if (a.score == NSG_SCORE_SIGMOID) hipLaunchKernelGGL((expert_route_backward_kernel<N, L, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((expert_route_backward_kernel<N, L, false>), grid, block, 0, s, a);
    return hipGetLastError();
  }
};

hipError_t launch_expert_route(const RouteArgs &a, hipStream_t s) { return by_experts<RouteForward>(a, s); }
hipError_t launch_expert_route_backward(const RouteArgs &a, hipStream_t s) { return by_experts<RouteBackward>(a, s); }

}  // namespace nsg
