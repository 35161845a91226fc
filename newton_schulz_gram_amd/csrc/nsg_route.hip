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
// small (one read of the logits, some 30 instructions for each): launches and, with many
// tokens, these instructions and the k rounds of the choice bound it.  16384 tokens of 256
// experts, k = 8, take 8.2 us (7.2 of them the counted vector instructions at 2.4 GHz), with a
// bias 14 (10), with the balance loss too 22 in three launches, the gradient of 512 experts
// 12.6 (9.3).  Sums over tokens are fp32 in an order that only the sizes fix, counts are
// integers; there are no atomics on memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nsg_layer.h"
#include "nsg_rows.h"

namespace nsg {

constexpr int kRouteThreads = 256;
// Workgroups at most (131072 tokens, k = 4, of 256 and 512 experts)
constexpr int kRouteBlocks = 8192;         // (1024, 2048, 8192: 44, 40, 37 us and 105, 91, 80)
constexpr int kRouteBackwardBlocks = 2048; // (the same: 33, 33, 40 and 60, 60, 63)
// with the balance loss, whose sums are joined (128, 256, 512: 97, 53, 56 us and 221, 116,
// 120; 16384 tokens 21, 15, 18 and 36, 23, 26)
constexpr int kBalanceBlocks = 256;

// N consecutive numbers of a row from e on, -inf behind the last expert
template <typename T, int N> __device__ __forceinline__ void load_as(const T *row, int e, int E, float (&f)[N]) {
  if (e + N <= E) {
    Row<T, N, (int)sizeof(T)>::load(row + e, f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = e + i < E ? (float)row[e + i] : -INFINITY;
  }
}
// N consecutive logits, loaded as they are and converted when they are used: a conversion
// would wait for the load.  (The type of the logits is the same in all lanes: a branch or two
// for each token instead of three kernels.)
template <int N> struct Logits {
  uint32_t w[N];  // one to a word, or two
  __device__ __forceinline__ void load(const RouteArgs &p, int64_t t, int e) {
    const int64_t at = t * p.ld + e;
    if (p.dtype == NSG_F32) words<uint32_t, N>((const uint32_t *)p.logits + at, e, p.E, 0xff800000u);
    else words<uint16_t, (N + 1) / 2>((const uint16_t *)p.logits + at, e, p.E, p.dtype == NSG_BF16 ? 0xff80ff80u : 0xfc00fc00u);
  }
  __device__ __forceinline__ void get(const RouteArgs &p, float (&f)[N]) const {
    if (p.dtype == NSG_F32) {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
    } else if (p.dtype == NSG_BF16) {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i / 2] >> (16 * (i & 1))));
    }
  }

 private:
  template <typename T, int W> __device__ __forceinline__ void words(const T *row, int e, int E, uint32_t none) {
    constexpr int kIn = sizeof(T) == 2 ? 2 : 1;  // elements of a word
    if (N % kIn == 0 && e + N <= E) {
      typedef uint32_t vec __attribute__((ext_vector_type(W)));
      typedef vec mem __attribute__((aligned(sizeof(T))));
      const vec v = *reinterpret_cast<const mem *>(row);
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = none;
      if (e < E) {
        if (N == 1) {
          w[0] = row[0];  // (kIn 2: the other half is not used)
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (e + i < E) {
              const uint32_t x = row[i];
              if (kIn == 1) w[i] = x;
              else w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | x << 16 : (w[i / 2] & 0xffff0000u) | x;
            }
        }
      }
    }
  }
};
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
// Floats as whole numbers in the same order (a NaN counts as -inf), and back
__device__ __forceinline__ int ordered(float f) {
  const int i = __builtin_bit_cast(int, f == f ? f : -INFINITY);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __builtin_bit_cast(float, i ^ ((i >> 31) & 0x7fffffff)); }
// Largest of the group in whole numbers, which a move between lanes and the comparison
// take one instruction for (floats: three)
template <int L, typename I> __device__ __forceinline__ I group_max_of(I v) {
  auto moved = [](I x, auto ctrl) { return (I)__builtin_amdgcn_update_dpp((int)x, (int)x, decltype(ctrl)::value, 0xf, 0xf, true); };
  v = max(v, moved(v, std::integral_constant<int, 0xB1>()));
  v = max(v, moved(v, std::integral_constant<int, 0x4E>()));
  if (L >= 16) {
    v = max(v, moved(v, std::integral_constant<int, 0x141>()));
    v = max(v, moved(v, std::integral_constant<int, 0x140>()));
  }
  if (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap((unsigned)v, (unsigned)v, false, false);
    v = max((I)r[0], (I)r[1]);
  }
  if (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap((unsigned)v, (unsigned)v, false, false);
    v = max((I)r[0], (I)r[1]);
  }
  return v;
}
template <int L> __device__ __forceinline__ int group_max(int v) { return group_max_of<L, int>(v); }
template <int L> __device__ __forceinline__ uint32_t group_max(uint32_t v) { return group_max_of<L, uint32_t>(v); }
template <int L> __device__ __forceinline__ float group_max(float v) { return unordered(group_max<L>(ordered(v))); }
template <int L> __device__ __forceinline__ float group_sum(float v) {
  return group_join<L>(v, [](float a, float b) { return a + b; });
}
// lanes of this lane's group among those of the wave
template <int L> __device__ __forceinline__ uint64_t group_lanes() {
  const int lane = threadIdx.x & 63;
  return (~0ull >> (64 - L)) << (lane / L * L);
}
// LDS written by some lanes of a wave is read by others
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------
// e^x, mostly for x <= 0, by the hardware's 2^x (within 1 unit): the argument's rounding makes it |x|
// roundings, which for the scores e^(l - top) of a token is less than one of the largest
__device__ __forceinline__ float exp_down(float x) {
  return __builtin_amdgcn_exp2f(fmaf(x, 1.44269502f, x * 1.9259630e-8f));  // the two parts of log2 e
}
__device__ __forceinline__ float inverse(float x) { return __builtin_amdgcn_rcpf(x); }  // within 1 unit

// 1 / x for a sum of scores; 0 where nothing has one
__device__ __forceinline__ float inverse_sum(float x) { return x == 0.f ? 0.f : 1.f / x; }

// The score of one logit times e^-shift; of all of a token's logits, see score_shift
template <bool SIGMOID> __device__ __forceinline__ float shifted_score(float l, float shift) {
  if (!SIGMOID) return exp_down(l - shift);
  return exp_down(fminf(l, 0.f) - shift) * inverse(1.f + exp_down(-fabsf(l)));
}
// (below -88, where e^-l leaves fp32, and the score its normal numbers: 0)
__device__ __forceinline__ float sigmoid(float l) { return inverse(1.f + exp_down(-l)); }

// A token's scores times a factor that they share, so that none that matters under- or
// overflows: softmax e^(l - shift) with shift the largest logit, sigmoid
// sigmoid(l) e^-shift with shift 0 unless the largest logit is far below it.
constexpr float kFar = -60.f;
// The gradient multiplies scores by numbers of any size before it divides by their sum: with
// the largest score at least e^-8 what underflows there is below E 2^-150 e^8 < 2^-126
constexpr float kFarBackward = -8.f;
template <bool SIGMOID> __device__ __forceinline__ float score_shift(float top, float far = kFar) {
  return SIGMOID ? (top < far ? top : 0.f) : top;
}
// The same for those of the chosen, of which a token's weights are shares: the largest becomes
// at least 1/2, so that any scale or gradient may be multiplied by them and by their sum's inverse
template <bool SIGMOID> __device__ __forceinline__ float chosen_shift(float top) { return SIGMOID ? fminf(top, 0.f) : top; }
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
// fp32 keys of scores with a bias are off by rounding: softmax scores, at most `size`, by less
// than 44 roundings of it (5 of the exponential; its sum's 4 + ln 1024 of the terms and 22
// of adding; the quotient's), sigmoid ones by less than 6 of 1 (1.3 of the exponential, which
// s (1 - s) weakens, 1 of the sum, 2 of its inverse, 1 of a product), the keys by one of their
// own.  Two that are further apart than this are in the order of the exact ones.
template <bool SIGMOID> __device__ __forceinline__ float key_margin(float size, float a, float b) {
  return 0x1p-24f * (SIGMOID ? 12.f + 4.f * fmaxf(fabsf(a), fabsf(b)) : fmaf(96.f, size, 4.f * fmaxf(fabsf(a), fabsf(b))));
}
// The key in 64 bits; `all`: the sum of e^(l - top)
template <bool SIGMOID> __device__ __forceinline__ double exact_key(float l, float top, double all, float bias) {
  const double x = (double)l;
  const double s = SIGMOID ? (x >= 0 ? 1.0 : exp(x)) / (1.0 + exp(-fabs(x))) : exp(x - (double)top) / all;
  return s + (double)bias;
}
template <int N, int L> __device__ __forceinline__ double exact_sum(const float (&l)[N], float top) {
  double all = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) all += l[i] > -INFINITY ? exp((double)l[i] - (double)top) : 0.0;
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) all += __shfl_xor(all, off, 64);
  return all;
}
template <int N, bool SIGMOID> __device__ __forceinline__ void exact_keys(const float (&l)[N], const float (&bias)[N], float top,
                                                                          double all, double (&key)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    key[i] = l[i] > -INFINITY ? exact_key<SIGMOID>(l[i], top, all, bias[i]) : -(double)INFINITY;
    if (!(key[i] > -(double)INFINITY)) key[i] = -(double)INFINITY;
  }
}
// fp32 keys: logits, or scores s `whole` with the bias; -inf for what is never chosen
template <int N, bool BIAS> __device__ __forceinline__ void make_keys(const float (&l)[N], const float (&s)[N], float whole,
                                                                      const float (&bias)[N], float (&key)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float v = BIAS ? fmaf(s[i], whole, bias[i]) : l[i];
    key[i] = l[i] > -INFINITY && v == v ? v : -INFINITY;
  }
}

// fp32 keys as whole numbers in the same order (both zeros alike), which take fewer
// instructions; never chosen: kNever
constexpr int kNever = INT32_MIN;
__device__ __forceinline__ int key_of(float f) {
  const int i = __builtin_bit_cast(int, f + 0.f);
  return f > -INFINITY ? i ^ ((i >> 31) & 0x7fffffff) : kNever;
}

__device__ __forceinline__ bool never(int key) { return key == kNever; }
__device__ __forceinline__ bool never(double key) { return !(key > -(double)INFINITY); }
__device__ __forceinline__ void take(int &key) { key = kNever; }
__device__ __forceinline__ void take(double &key) { key = -(double)INFINITY; }
template <int L> __device__ __forceinline__ double group_max(double v) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) {
    const double o = __shfl_xor(v, off, 64);
    v = o > v ? o : v;
  }
  return v;
}

// Whether this lane is the first of its group among those of the wave's mask
template <int L> __device__ __forceinline__ bool first_of_group(uint64_t mask) {
  const unsigned lo = (unsigned)mask, hi = (unsigned)(mask >> 32);
  if (L == 64) return __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0)) == 0;
  const int lane = threadIdx.x & 63;
  const unsigned up_to = (lane < 32 ? lo : hi) << (31 - (lane & 31));  // this lane's bit is the highest
  return (up_to & 0x7fffffffu) >> (31 - lane % L) == 0;
}

// The largest of a token's keys, of equal ones the first, as choice j: its index and (fp32
// keys) itself to id[j] and val[j], if `write`.  It is taken out of the keys.  Returns
// whether there was one.
template <int N, int L, typename K>
__device__ __forceinline__ bool choose_one(K (&key)[N], int j, int sub, int32_t *id, float *val, bool write) {
  K best = key[0];
#pragma unroll
  for (int i = 1; i < N; ++i) best = key[i] > best ? key[i] : best;
  const K top = group_max<L>(best);
  const bool some = !never(top), mine = some && best == top;
  const uint64_t who = __ballot(mine);
  if (mine && first_of_group<L>(who)) {
    int at = N - 1;
#pragma unroll
    for (int i = N - 2; i >= 0; --i) at = key[i] == top ? i : at;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      K gone;
      take(gone);
      key[i] = at == i ? gone : key[i];
    }
    if (write) {
      id[j] = sub * N + at;
      if (sizeof(K) == 4) val[j] = unordered((int)top);
    }
  }
  return some;
}
// The k largest, one after the other; how many there were
template <int N, int L, typename K>
__device__ __forceinline__ int choose(K (&key)[N], int k, int sub, int32_t *id, float *val, bool write) {
  int found = 0;
  for (int j = 0; j < k; ++j) found += choose_one<N, L, K>(key, j, sub, id, val, write);
  return found;
}

// Up to 256 experts: keys of 31 bits, the fp32 key's order in the upper ones and the expert
// in the lowest kIdBits, lower ones first; 0: never chosen.  No two are equal, so the largest
// key below the one before it is the next choice: a subtraction for each and a maximum, about
// 20 instructions a choice of 8 experts a lane; finding the lane and taking the key out are
// 50 (16384 tokens of 256, k = 8: 8.2 us, with a bias 14; so 10.1 and 17.2).  16-bit logits
// keep all of their bits.  Of other keys the last bits are lost: the first k in the right
// order are among the first k and those that come next, until one is too far from the k-th.
// These are taken too (`taken` in all), at most kNext of them; `more`: there are more.
constexpr int kNext = 16;
template <int N, int L> struct Packed {
  static constexpr uint32_t kLast = N * L - 1;
  // -inf and NaN: what is never chosen, below kLeast
  static constexpr uint32_t kLeast = 0x400000;
  static __device__ __forceinline__ uint32_t pack(float key, uint32_t e) {
    const uint32_t i = __builtin_bit_cast(uint32_t, fmaxf(key, -INFINITY));
    return ((i ^ ((uint32_t)((int)i >> 31) | 0x80000000u)) >> 1 & ~kLast) | (kLast - e);
  }
  static __device__ __forceinline__ int expert(uint32_t k) { return (int)(kLast - (k & kLast)); }
  // the fp32 key, of a 16-bit one all, else up to 2 N L steps of fp32 below it
  static __device__ __forceinline__ float key(uint32_t k) {
    const int i = (int)((k & ~kLast) << 1 ^ 0x80000000u);
    return unordered(i < 0 ? i | (int)(2 * kLast + 1) : i);
  }
  uint32_t top;  // the last choice; at first above all keys, or where nothing is chosen 0
  __device__ __forceinline__ explicit Packed(bool counts) : top(counts ? 1u << 31 : 0) {}
  __device__ __forceinline__ bool next(const uint32_t (&keys)[N]) {
    uint32_t best = keys[0] - top;  // of keys below it in the upper half, largest for the largest
#pragma unroll
    for (int i = 1; i < N; ++i) best = max(best, keys[i] - top);
    best = group_max<L>(best);
    const bool below = best >> 31;
    top = below ? top + best : top;
    return below && top >= kLeast;
  }
};
struct Taken {
  int found, taken;  // at most k; with those that come next
  bool more;
};
// The largest keys to list.  `look`: with those that come next, for keys of scores of at most
// `size` with a bias, or of logits, which are near where only lost bits differ.
template <int N, int L, bool SIGMOID, bool BIAS>
__device__ __forceinline__ Taken choose_packed(const uint32_t (&keys)[N], bool counts, int k, int sub, uint32_t *list, bool look,
                                               float size) {
  typedef Packed<N, L> P;
  P r(counts);
  Taken c{0, 0, false};
  for (int j = 0; j < k; ++j) {
    c.found += r.next(keys);
    if (sub == 0) list[j] = r.top;
  }
  c.taken = c.found;
  if (!look) return c;
  const uint32_t kth = r.top;
  // (of the k-th, one that comes next is always taken: the order of neighbours shows how
  // close they are)
  bool on = c.found == k;
  for (int j = k; __ballot(on) != 0; ++j) {
    if (j == k + kNext) {
      c.more = on;
      break;
    }
    on = r.next(keys) && on;
    if (on && sub == 0) list[j] = r.top;
    c.taken += on;
    if (!BIAS) {
      on = on && (kth & ~P::kLast) == (r.top & ~P::kLast);
    } else {
      const float x = P::key(kth), y = P::key(r.top), lost = 0x1p-24f * (4 * P::kLast + 4);
      on = on && !(x - y > key_margin<SIGMOID>(size, x, y) + lost * fmaxf(fabsf(x), fabsf(y)));
    }
  }
  return c;
}

struct BalanceRow {  // a workgroup's sum and count of an expert; behind the last one, its tokens
  float sum;
  int32_t count;
};
static int64_t balance_pitch(int E) { return (E + 2) / 2 * 2; }

// What a workgroup adds up for the balance loss
__device__ __forceinline__ void balance_clear(const RouteArgs &p, int32_t *count) {
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) count[e] = 0;
  __syncthreads();
}
// The groups' sums: one group after the other in a wave, then the waves', whose sums of
// expert e lie at (e % N) L + e / N of their rows of `sums`, so that lanes write next to each other.
template <int N, int L>
__device__ __forceinline__ void balance_store(const RouteArgs &p, float (&acc)[N], const int32_t *count, float *sums, BalanceRow *to) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int off = L; off < 64; off <<= 1) acc[i] += __shfl_xor(acc[i], off, 64);
  }
  __syncthreads();
  const int wave = threadIdx.x / 64, waves = blockDim.x / 64, lane = threadIdx.x & 63;
  if (lane < L) {
#pragma unroll
    for (int i = 0; i < N; ++i) sums[(wave * N + i) * L + lane] = acc[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
    float v = 0.f;
    if (e < p.E)
      for (int w = 0; w < waves; ++w) v += sums[(w * N + e % N) * L + e / N];
    to[e] = BalanceRow{v, count[e]};
  }
}

// The weight of a chosen expert with logit x.  `high`: chosen_shift of the largest chosen
// logit, `whole`: scale / sum of the chosen's shifted scores; not normalised, softmax:
// the largest logit and scale / sum of all.
template <bool SIGMOID> __device__ __forceinline__ float chosen_weight(const RouteArgs &p, float x, float high, float whole) {
  return SIGMOID && !p.normalize ? p.scale * sigmoid(x) : whole * shifted_score<SIGMOID>(x, high);
}

// ---- several tokens to a wave: up to 256 experts ---------------------------------
// LDS of a token: the chosen keys, then experts, and their logits; where keys lose bits
// (`look`) also those that come next, their exact keys, the order of these, and whole keys
static __host__ __device__ bool group_looks(const RouteArgs &p) { return p.bias != nullptr || p.dtype == NSG_F32; }
static __host__ __device__ int group_kept(int k, int E, bool look) { return look ? (k + kNext <= E ? k + kNext : E + 1) : k; }
static __host__ __device__ int group_room(int k, int E, bool look) { return group_kept(k, E, look) * (look ? 24 : 8); }

template <int N, int L, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(1024) expert_route_group_kernel(RouteArgs p, BalanceRow *__restrict__ rows, int64_t pitch) {
  extern __shared__ __attribute__((aligned(16))) char room[];
  __shared__ int32_t count[N * L + 1];
  const int tokens = blockDim.x / L;
  const int sub = threadIdx.x % L, token = threadIdx.x / L, e0 = sub * N;
  const bool look = group_looks(p);
  const int kept = group_kept(p.k, p.E, look);
  double *const exact = reinterpret_cast<double *>(room) + (look ? token * kept : 0);
  int32_t *const id = reinterpret_cast<int32_t *>(room + (look ? tokens * kept * 8 : 0)) + token * kept;
  float *const val = reinterpret_cast<float *>(id + tokens * kept);
  int32_t *const order = id + 2 * tokens * kept;  // (look)
  float *const whole = reinterpret_cast<float *>(id + 3 * tokens * kept);
  const bool balance = rows != nullptr;
  if (balance) balance_clear(p, count);
  float acc[N], bias[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = bias[i] = 0.f;
  // the next tokens' logits are on their way while these are worked on
  const int step = (int)gridDim.x * tokens, T = (int)p.T;  // (at most NSG_MAX_ROWS)
  Logits<N> next;
  int counts = 0;
  auto fetch = [&](int t) {
    counts = t < T && (p.mask == nullptr || p.mask[t]);
    next.load(p, t < T ? t : 0, e0);
  };
  fetch((int)blockIdx.x * tokens + token);
  for (int t0 = (int)blockIdx.x * tokens; t0 < T; t0 += step) {
    const int t = t0 + token;
    float l[N], s[N];
    next.get(p, l);
    if (BIAS) load_as(p.bias, e0, p.E, bias);  // (for each token: there are no registers to keep it in)
    const bool counted = counts;  // (else what follows is computed of no one's logits, and nothing is chosen)
    if (t0 + step < T) fetch(t + step);
    float top = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, l[i]);
    top = group_max<L>(top);
    if (!(top > -INFINITY)) top = 0.f;
    const float shift = score_shift<SIGMOID>(top);
    float sum = 0.f, unit = 1.f;
    if (balance || BIAS || !SIGMOID) sum = scores<SIGMOID, N, L>(l, shift, s);
    if (BIAS) unit = !SIGMOID ? inverse(sum) : shift == 0.f ? 1.f : exp_down(shift);
    typedef Packed<N, L> P;
    uint32_t keys[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float key = fmaf(s[i], unit, bias[i]);
      keys[i] = P::pack(!BIAS ? l[i] + 0.f : l[i] > -INFINITY ? key : -INFINITY, e0 + i);  // (+ 0: both zeros alike)
    }
    const Taken c = choose_packed<N, L, SIGMOID, BIAS>(keys, counted, p.k, sub, reinterpret_cast<uint32_t *>(id), look, unit);
    const int found = c.found;
    bool moved = false;  // choice j lies at order[j]
    wave_sync();
    // a choice to a lane: its logit and whole key
    for (int j = sub; j < c.taken; j += L) {
      const uint32_t k = (uint32_t)id[j];
      const int e = P::expert(k);
      const float x = look ? logit(p, t, e) : P::key(k);
      id[j] = e;
      val[j] = x;
      if (look) whole[j] = BIAS ? fmaf(shifted_score<SIGMOID>(x, shift), unit, p.bias[e]) : x;
    }
    if (look) {
      wave_sync();
      bool off = false;  // not in order, or too near to tell
      for (int j = sub; j + 1 < c.taken; j += L) {
        const float x = whole[j], y = whole[j + 1];
        off = off || !(BIAS ? x - y > key_margin<SIGMOID>(unit, x, y) : x >= y);
      }
      const uint64_t group = group_lanes<L>();
      const bool sort = (__ballot(off) & group) != 0 || c.more;
      if (__builtin_expect(__ballot(sort) != 0, 0)) {
        // the order of the whole keys, of those that are too near by their 64 bits, or of all
        // experts' where those that come next did not end
        moved = sort && !c.more;
        // `which` of this lane's choices, a bit for each; those that are near another
        auto set_order = [&](uint32_t which, auto *key, bool loose) {
          wave_sync();
          uint32_t near = 0;
          for (int j = sub; j < c.taken; j += L) {
            const uint32_t bit = 1u << (j / L);
            if (!(which & bit)) continue;
            const auto x = key[j];
            int rank = 0;
            for (int i = 0; i < c.taken; ++i) {
              const auto y = key[i];
              rank += y > x || (y == x && id[i] < id[j]);
              if (loose && i != j && !(fabsf((float)(x - y)) > key_margin<SIGMOID>(unit, (float)x, (float)y))) near |= bit;
            }
            order[rank] = j;
          }
          wave_sync();
          return near;
        };
        const uint32_t near = set_order(moved ? ~0u : 0, whole, BIAS);
        if (BIAS && __ballot(near != 0 || c.more) != 0) {
          const double all = SIGMOID ? 1.0 : exact_sum<N, L>(l, top);
          for (int j = sub; moved && j < c.taken; j += L)
            exact[j] = near >> (j / L) & 1 ? exact_key<SIGMOID>(val[j], top, all, p.bias[id[j]]) : (double)whole[j];
          set_order(near, exact, false);
          if (__ballot(c.more) != 0) {
            double key64[N];
            exact_keys<N, SIGMOID>(l, bias, top, all, key64);
            choose<N, L, double>(key64, p.k, sub, id, val, c.more);
          }
        }
        if (!BIAS && __ballot(c.more) != 0) {
          int key[N];
#pragma unroll
          for (int i = 0; i < N; ++i) key[i] = key_of(l[i]);
          choose<N, L, int>(key, p.k, sub, id, val, c.more);
        }
        wave_sync();
        for (int j = sub; c.more && j < found; j += L) val[j] = logit(p, t, id[j]);
      }
    }
    wave_sync();
    // a choice to a lane
    float high = top, factor = 0.f;
    if (p.normalize) {
      if (BIAS) {
        high = -INFINITY;
        for (int j = sub; j < found; j += L) high = fmaxf(high, val[moved ? order[j] : j]);
        high = group_max<L>(high);
      }
      high = chosen_shift<SIGMOID>(high);
      for (int j = sub; j < found; j += L) factor += shifted_score<SIGMOID>(val[moved ? order[j] : j], high);
      factor = p.scale * inverse_sum(group_sum<L>(factor));
    } else if (!SIGMOID) {
      factor = p.scale * inverse_sum(sum);
    }
    if (t < T) {
      for (int j = sub; j < p.k; j += L) {
        float w = 0.f;
        int e = -1;
        if (j < found) {
          const int at = moved ? order[j] : j;
          e = id[at];
          w = chosen_weight<SIGMOID>(p, val[at], high, factor);
          if (!SIGMOID && sum != sum) w = sum;  // with softmax a NaN among the logits is in all weights
          if (balance) atomicAdd(&count[e], 1);
        }
        const int64_t to = (int64_t)t * p.k + j;
        p.ids[to] = e;
        p.weights[to] = w;
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
  if (balance) balance_store<N, L>(p, acc, count, reinterpret_cast<float *>(room), rows + (int64_t)blockIdx.x * pitch);
}

// ---- a token to a wave -----------------------------------------------------------
__device__ __forceinline__ int wave_max(int v) { return __builtin_amdgcn_readfirstlane(group_max<64>(v)); }
__device__ __forceinline__ float wave_max(float v) { return unordered(wave_max(ordered(v))); }

// What a wave chooses from: the keys of at least `from`, their experts and logits
struct Candidate {
  float key;
  int32_t id;
  float logit;
};
constexpr int kCandidates = 64;  // one to a lane
// How many of the n candidates, one to a lane, come before this lane's
__device__ __forceinline__ int candidate_rank(const Candidate &mine, int n) {
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const float key = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mine.key), j));
    const int id = __builtin_amdgcn_readlane(mine.id, j);
    rank += key > mine.key || (key == mine.key && id < mine.id);
  }
  return rank;
}

// A bound that at least `need` and hardly more of the lanes' largest keys are not below: so
// many keys, and a few more, are not below it.  -inf where no more than `need` lanes have a key.
__device__ __forceinline__ float candidate_bound(float best, float top, int need) {
  int lo = ~wave_max(best > -INFINITY ? ~ordered(best) : INT32_MIN);  // the smallest
  if (__popcll(__ballot(best > -INFINITY)) <= need) return -INFINITY;
  int hi = ordered(top) + 1;  // (of +inf too)
  while ((unsigned)hi - (unsigned)lo > 1u) {  // at least `need` are not below lo, fewer not below hi
    const int mid = (int)((unsigned)lo + ((unsigned)hi - (unsigned)lo) / 2);
    const int n = __popcll(__ballot(best >= unordered(mid)));
    if (n < need) {
      hi = mid;
    } else {
      lo = mid;
      if (n <= need + 4) break;
    }
  }
  return unordered(lo);
}
template <int N>
__device__ __forceinline__ int gather_candidates(const float (&key)[N], const float (&l)[N], int e0, float from, Candidate *c) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool in = key[i] > -INFINITY && !(key[i] < from);
    const uint64_t who = __ballot(in);
    if (who != 0) {
      const int at = n + (int)__builtin_amdgcn_mbcnt_hi((unsigned)(who >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)who, 0));
      if (in && at < kCandidates) c[at] = Candidate{key[i], e0 + i, l[i]};
      n += __popcll(who);
    }
  }
  return n;
}

// threads of a workgroup, by the registers that a thread needs
template <int N, bool BIAS> constexpr int kWaveThreads() { return N > (BIAS ? 4 : 8) ? 512 : 1024; }

template <int N, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__((kWaveThreads<N, BIAS>())) expert_route_kernel(RouteArgs p, BalanceRow *__restrict__ rows, int64_t pitch) {
  extern __shared__ float sums[];  // the waves' sums
  __shared__ Candidate cands[kWaveThreads<N, BIAS>() / 64][kCandidates];
  __shared__ int32_t ids[kWaveThreads<N, BIAS>() / 64][kCandidates];
  __shared__ float vals[kWaveThreads<N, BIAS>() / 64][kCandidates];  // the chosen's logits
  __shared__ float sorted[BIAS ? kWaveThreads<N, BIAS>() / 64 : 1][kCandidates];  // and keys
  __shared__ double exact[BIAS ? kWaveThreads<N, BIAS>() / 64 : 1][kCandidates];
  __shared__ int32_t count[NSG_MAX_EXPERTS + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), e0 = lane * N;
  Candidate *const cand = cands[wave];
  int32_t *const id = ids[wave];
  float *const val = vals[wave];
  float *const skey = sorted[BIAS ? wave : 0];
  double *const key64 = exact[BIAS ? wave : 0];
  const bool balance = rows != nullptr;
  if (balance) balance_clear(p, count);
  float acc[N], bias[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = bias[i] = 0.f;
  if (BIAS) load_as(p.bias, e0, p.E, bias);
  // the next token's logits are on their way while one is worked on
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / 64);
  Logits<N> next;
  int counts = 1;
  auto fetch = [&](int64_t t) {
    if (p.mask != nullptr) counts = p.mask[t];
    next.load(p, t, e0);
  };
  // A token's results are stored in the next one's turn: what waits for the logits would wait
  // for these stores too.
  int64_t done = -1;
  int32_t out_id = 0;
  float out_weight = 0.f;
  auto store = [&]() {
    if (done >= 0 && lane < p.k) {
      p.ids[done * p.k + lane] = out_id;
      p.weights[done * p.k + lane] = out_weight;
    }
  };
  int64_t t = (int64_t)blockIdx.x * (blockDim.x / 64) + wave;
  if (t < p.T) fetch(t);
  for (; t < p.T; t += step) {
    float l[N], s[N], key[N];
    next.get(p, l);
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = counts ? l[i] : -INFINITY;
    store();
    if (t + step < p.T) fetch(t + step);
    float best = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = fmaxf(best, l[i]);
    float top = wave_max(best);
    if (!(top > -INFINITY)) top = 0.f;
    const float shift = score_shift<SIGMOID>(top);
    float sum = 0.f, unit = 1.f;
    if (balance || BIAS || !SIGMOID) sum = scores<SIGMOID, N, 64>(l, shift, s);
    if (BIAS) unit = !SIGMOID ? inverse(sum) : shift == 0.f ? 1.f : exp_down(shift);
    make_keys<N, BIAS>(l, s, unit, bias, key);
    best = key[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = fmaxf(best, key[i]);
    const float first = BIAS ? wave_max(best) : top;
    const int need = BIAS ? p.k + 1 : p.k;  // one more, to see how close it is
    int n = gather_candidates<N>(key, l, e0, candidate_bound(best, first, need), cand);
    int found = n < p.k ? n : p.k;
    wave_sync();
    if (n <= kCandidates) {
      // the candidates in order, one to a lane
      Candidate mine = cand[lane < n ? lane : 0];
      int rank = candidate_rank(mine, n);
      if (lane < n) {
        id[rank] = mine.id;
        val[rank] = mine.logit;
        if (BIAS) skey[rank] = mine.key;
      }
      if (BIAS) {
        wave_sync();
        const int last = n < need ? n - 1 : p.k;
        const float margin = n > 1 ? key_margin<SIGMOID>(unit, skey[0], skey[last]) : 0.f;
        const int at = lane < last ? lane : 0;
        const uint64_t close = __ballot(lane < last && !(skey[at] - skey[at + 1 < 64 ? at + 1 : 63] > margin));
        if (close != 0) {
          // exact keys: of all that may be among the first k, if they are no more than the lanes
          if (last == p.k && (close >> (p.k - 1) & 1)) {
            const float from = skey[p.k - 1] - 2.f * margin;
            wave_sync();
            n = gather_candidates<N>(key, l, e0, from, cand);
            wave_sync();
          }
          const double all = SIGMOID ? 1.0 : exact_sum<N, 64>(l, top);
          if (n <= kCandidates) {
            mine = cand[lane < n ? lane : 0];
            const double x = exact_key<SIGMOID>(mine.logit, top, all, p.bias[mine.id]);
            if (lane < n) key64[lane] = x;
            wave_sync();
            rank = 0;
            for (int j = 0; j < n; ++j) rank += key64[j] > x || (key64[j] == x && cand[j].id < mine.id);
            if (lane < n && rank < p.k) {
              id[rank] = mine.id;
              val[rank] = mine.logit;
            }
          } else {
            double keys64[N];
            exact_keys<N, SIGMOID>(l, bias, top, all, keys64);
            choose<N, 64, double>(keys64, p.k, lane, id, val, true);
            wave_sync();
            if (lane < found) val[lane] = logit(p, t, id[lane]);
          }
        }
      }
    } else if (BIAS) {  // many equal or nearly equal keys, or k near 64
      double keys64[N];
      exact_keys<N, SIGMOID>(l, bias, top, SIGMOID ? 1.0 : exact_sum<N, 64>(l, top), keys64);
      found = choose<N, 64, double>(keys64, p.k, lane, id, val, true);
      wave_sync();
      if (lane < found) val[lane] = logit(p, t, id[lane]);
    } else {
      int whole_key[N];
#pragma unroll
      for (int i = 0; i < N; ++i) whole_key[i] = key_of(key[i]);
      found = choose<N, 64, int>(whole_key, p.k, lane, id, val, true);
    }
    wave_sync();
    // a choice to a lane
    const bool in = lane < found;
    const float x = in ? val[lane] : -INFINITY;
    float high = top, whole = 0.f;
    if (p.normalize) {
      high = chosen_shift<SIGMOID>(BIAS ? wave_max(x) : top);
      whole = p.scale / wave_sum(in ? shifted_score<SIGMOID>(x, high) : 0.f);
    } else if (!SIGMOID) {
      whole = p.scale / sum;
    }
    done = t;
    out_id = in ? id[lane] : -1;
    out_weight = in ? chosen_weight<SIGMOID>(p, x, high, whole) : 0.f;
    if (!SIGMOID && in && sum != sum) out_weight = sum;  // with softmax a NaN among the logits is in all weights
    if (balance) {
      if (in) atomicAdd(&count[out_id], 1);
      if (found > 0) {
        const float inv = 1.f / sum;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(s[i], inv, acc[i]);
        if (lane == 0) atomicAdd(&count[p.E], 1);
      }
    }
    wave_sync();
  }
  store();
  if (balance) balance_store<N, 64>(p, acc, count, sums, rows + (int64_t)blockIdx.x * pitch);
}

// Sums of the rows of experts 2 u and 2 u + 1 (behind the last one, the tokens): `units`
// threads side by side, 1024 / units of them for a unit, which share the rows and join
// their sums in halves.  In the first ones' results.
struct BalancePair {
  float a0, a1;
  int n0, n1;
};
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ BalancePair balance_sum(const BalanceRow *__restrict__ rows, int blocks, int64_t pitch, int unit,
                                                   int units, BalancePair *sh) {
  const int share = 1024 / units, g = (int)threadIdx.x / units;
  BalancePair r{0.f, 0.f, 0, 0};
  if (g < share) {
    for (int b0 = g; b0 < blocks; b0 += 16 * share) {
      u32x4 v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int b = b0 + i * share;
        v[i] = b < blocks ? *reinterpret_cast<const u32x4 *>(rows + (int64_t)b * pitch + 2 * unit) : u32x4(0);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        r.a0 += __uint_as_float(v[i][0]);
        r.n0 += (int)v[i][1];
        r.a1 += __uint_as_float(v[i][2]);
        r.n1 += (int)v[i][3];
      }
    }
  }
  for (int n = share; n > 1;) {
    const int half = (n + 1) / 2;
    if (g < n) sh[threadIdx.x] = r;
    __syncthreads();
    if (g + half < n) {
      const BalancePair o = sh[threadIdx.x + half * units];
      r.a0 += o.a0;
      r.a1 += o.a1;
      r.n0 += o.n0;
      r.n1 += o.n1;
    }
    __syncthreads();
    n = half;
  }
  return r;
}

// 16 experts to a workgroup, which has 128 threads for each two of them: one row of the
// rows' sums
__global__ void __launch_bounds__(1024) expert_balance_rows_kernel(int blocks, const BalanceRow *__restrict__ rows, int64_t pitch,
                                                                   BalanceRow *__restrict__ out) {
  __shared__ BalancePair sh[16][8];
  const int wave = threadIdx.x / 64, unit = (int)blockIdx.x * 8 + (int)threadIdx.x % 8, units = (int)pitch / 2;
  BalancePair r{0.f, 0.f, 0, 0};
  if (unit < units) {
    u32x4 v[kBalanceBlocks / 128];
#pragma unroll
    for (int i = 0; i < kBalanceBlocks / 128; ++i) {
      const int b = (int)threadIdx.x / 8 + i * 128;
      v[i] = b < blocks ? *reinterpret_cast<const u32x4 *>(rows + (int64_t)b * pitch + 2 * unit) : u32x4(0);
    }
#pragma unroll
    for (int i = 0; i < kBalanceBlocks / 128; ++i) {
      r.a0 += __uint_as_float(v[i][0]);
      r.n0 += (int)v[i][1];
      r.a1 += __uint_as_float(v[i][2]);
      r.n1 += (int)v[i][3];
    }
  }
#pragma unroll
  for (int off = 8; off < 64; off <<= 1) {
    r.a0 += __shfl_xor(r.a0, off, 64);
    r.n0 += __shfl_xor(r.n0, off, 64);
    r.a1 += __shfl_xor(r.a1, off, 64);
    r.n1 += __shfl_xor(r.n1, off, 64);
  }
  if ((threadIdx.x & 63) < 8) sh[wave][threadIdx.x & 63] = r;
  __syncthreads();
  if (threadIdx.x < 8 && unit < units) {
#pragma unroll
    for (int w = 1; w < 16; ++w) {
      const BalancePair o = sh[w][threadIdx.x];
      r.a0 += o.a0;
      r.n0 += o.n0;
      r.a1 += o.a1;
      r.n1 += o.n1;
    }
    out[2 * unit] = BalanceRow{r.a0, r.n0};
    out[2 * unit + 1] = BalanceRow{r.a1, r.n1};
  }
}

// One workgroup: counts, probs and loss
__global__ void __launch_bounds__(1024) expert_balance_kernel(RouteArgs p, int blocks, const BalanceRow *__restrict__ rows,
                                                              int64_t pitch) {
  __shared__ BalancePair sh[1024];
  __shared__ float part[16];
  __shared__ int tokens;
  const int units = (int)pitch / 2, u = (int)threadIdx.x % units;
  BalancePair r = balance_sum(rows, blocks, pitch, u, units, sh);
  const bool mine = (int)threadIdx.x < units;
  if (mine && 2 * u == p.E) tokens = r.n0;
  if (mine && 2 * u + 1 == p.E) tokens = r.n1;
  __syncthreads();
  const int N = tokens;
  float v = 0.f;
  if (mine) {
    r.a0 = N > 0 ? r.a0 / (float)N : 0.f;
    r.a1 = N > 0 ? r.a1 / (float)N : 0.f;
    if (2 * u < p.E) {
      p.counts[2 * u] = r.n0;
      p.probs[2 * u] = r.a0;
      v = (float)r.n0 * r.a0;
    }
    if (2 * u + 1 < p.E) {
      p.counts[2 * u + 1] = r.n1;
      p.probs[2 * u + 1] = r.a1;
      v = fmaf((float)r.n1, r.a1, v);
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
    load_as(p.counts, e0, p.E, c);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = e0 + i < p.E ? f * c[i] : 0.f;
  }
  // a token's logits and this lane's choices (j = sub, sub + L, ...); the next ones are on
  // their way while these are worked on
  const int64_t step = (int64_t)gridDim.x * kTokens;
  Logits<N> next_l;
  float next_g[kMine];
  int next_e[kMine];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int j = sub + m * L;
      const bool in = t < p.T && j < p.k;
      next_e[m] = in ? p.ids[t * p.k + j] : -1;
      next_g[m] = in && weights ? p.dweights[t * p.k + j] : 0.f;
    }
    next_l.load(p, t < p.T ? t : 0, e0);
  };
  // a token's gradient is stored in the next one's turn: what waits for the logits would
  // wait for these stores too
  int64_t done = -1;
  float out[N];
  auto store = [&]() {
    if (done < 0 || e0 >= p.E) return;
    const int64_t to = done * p.E;
    if (p.dtype == NSG_F32) store_as((float *)p.dlogits + to, e0, p.E, out);
    else if (p.dtype == NSG_BF16) store_as((__bf16 *)p.dlogits + to, e0, p.E, out);
    else store_as((_Float16 *)p.dlogits + to, e0, p.E, out);
  };
  fetch((int64_t)blockIdx.x * kTokens + token);
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < p.T; t0 += step) {
    const int64_t t = t0 + token;
    const bool there = t < p.T;
    int e[kMine];
    float l[N], g[kMine], x[kMine];
    bool any = false;
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      e[m] = next_e[m] < p.E ? next_e[m] : -1;
      g[m] = e[m] >= 0 ? next_g[m] * p.scale : 0.f;  // (what stands at no choice may be NaN)
      any = any || e[m] >= 0;
      x[m] = e[m] >= 0 ? logit(p, t, e[m]) : -INFINITY;
    }
    next_l.get(p, l);
    store();
    if (t0 + step < p.T) fetch(t + step);
    const bool found = (__ballot(any) & group) != 0;
    float top = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, l[i]);
    top = group_max<L>(top);
    if (!(top > -INFINITY)) top = 0.f;
    float s[N], pc = 0.f;
    const float sum = inverse_sum(scores<SIGMOID, N, L>(l, score_shift<SIGMOID>(top, kFarBackward), s));
#pragma unroll
    for (int i = 0; i < N; ++i) pc = fmaf(s[i], c[i], pc);
    pc = group_sum<L>(pc) * sum;
    float dot = 0.f;
    if (weights) {
      float high = -INFINITY, whole = 0.f, v[kMine];
#pragma unroll
      for (int m = 0; m < kMine; ++m) high = fmaxf(high, x[m]);
      high = group_max<L>(high);
      high = high > -INFINITY ? chosen_shift<SIGMOID>(high) : 0.f;
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
    const bool full = softmax && !p.normalize && weights;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float pe = s[i] * sum;
      if (full) d[i] = pe * (d[i] - dot);
      if (p.counts != nullptr) d[i] = fmaf(softmax ? pe : pe * sigmoid(-l[i]), c[i] - pc, d[i]);
      out[i] = found ? d[i] : 0.f;
    }
    done = there ? t : -1;
    wave_sync();
  }
  store();
}

// ---------------------------------------------------------------------------
size_t expert_route_workspace(int64_t T, int E) {
  return T == 0 ? 0 : (size_t)(kBalanceBlocks + 1) * (size_t)balance_pitch(E) * sizeof(BalanceRow);
}

struct RouteForward {
  // Many rows are summed by as many workgroups as there are 16 experts first: one that reads
  // them all takes 8 us for 256 rows of 256 experts, 14 of 512 and 25 of 1024.
  static hipError_t join(const RouteArgs &a, int blocks, BalanceRow *rows, int64_t pitch, hipStream_t s) {
    if (blocks * pitch > 8192) {
      BalanceRow *sums = rows + kBalanceBlocks * pitch;
      hipLaunchKernelGGL(expert_balance_rows_kernel, dim3((unsigned)((pitch / 2 + 7) / 8)), dim3(1024), 0, s, blocks,
                         (const BalanceRow *)rows, pitch, sums);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      rows = sums;
      blocks = 1;
    }
    hipLaunchKernelGGL(expert_balance_kernel, dim3(1), dim3(1024), 0, s, a, blocks, (const BalanceRow *)rows, pitch);
    return hipGetLastError();
  }
  template <class F> static hipError_t with_kernel(const RouteArgs &a, F kernel) {
    const bool g = a.score == NSG_SCORE_SIGMOID, b = a.bias != nullptr;
    return g ? b ? kernel(std::true_type(), std::true_type()) : kernel(std::true_type(), std::false_type())
             : b ? kernel(std::false_type(), std::true_type()) : kernel(std::false_type(), std::false_type());
  }
  // threads of a workgroup and the tokens that it takes at a time
  template <class F> static hipError_t launch(const RouteArgs &a, int threads, int tokens, hipStream_t s, F kernel) {
    const bool balance = a.counts != nullptr;
    const int64_t pitch = balance_pitch(a.E), need = (a.T + tokens - 1) / tokens, most = balance ? kBalanceBlocks : kRouteBlocks;
    const int blocks = (int)(need < most ? need : most);
    BalanceRow *rows = balance ? (BalanceRow *)a.workspace : nullptr;
    if (blocks > 0) {
      kernel(dim3((unsigned)blocks), dim3((unsigned)threads), rows, pitch);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return balance ? join(a, blocks, rows, pitch, s) : hipSuccess;
  }
  template <int N, int L> static hipError_t group(const RouteArgs &a, hipStream_t s) {
    return with_kernel(a, [&](auto sigmoid, auto bias) {
      constexpr bool S = decltype(sigmoid)::value, B = decltype(bias)::value;
      const bool balance = a.counts != nullptr;
      // with the balance loss as many threads as their LDS allows: few rows to join
      int threads = balance ? 1024 : kRouteThreads;
      const int room = group_room(a.k, a.E, group_looks(a));
      while (threads > 64 && threads / L * room > 60 << 10) threads /= 2;
      unsigned lds = threads / L * room;
      if (balance && lds < threads / 64 * N * L * 4u) lds = threads / 64 * N * L * 4u;  // the waves' sums
      return launch(a, threads, threads / L, s, [&](dim3 grid, dim3 block, BalanceRow *rows, int64_t pitch) {
        hipLaunchKernelGGL((expert_route_group_kernel<N, L, S, B>), grid, block, lds, s, a, rows, pitch);
      });
    });
  }
  template <int N> static hipError_t wave(const RouteArgs &a, hipStream_t s) {
    return with_kernel(a, [&](auto sigmoid, auto bias) {
      constexpr bool S = decltype(sigmoid)::value, B = decltype(bias)::value;
      const bool balance = a.counts != nullptr;
      const int threads = balance ? kWaveThreads<N, B>() : kRouteThreads;
      const unsigned lds = balance ? threads * N * 4 : 0;
      return launch(a, threads, threads / 64, s, [&](dim3 grid, dim3 block, BalanceRow *rows, int64_t pitch) {
        hipLaunchKernelGGL((expert_route_kernel<N, S, B>), grid, block, lds, s, a, rows, pitch);
      });
    });
  }
};

// Lanes and experts of a lane: with few experts a wave of its own for each token has too
// little to do (16384 tokens, k = 8, of 64 / 128 / 256 experts: 4.6 / 5.3 / 8.2 us, a wave each
// 14 / 15 / 16), with many the groups' k rounds go over too many (512 / 1024: 24 / 35 us, a wave
// each, which chooses among few candidates, 15 / 21).  Of 16 experts 2 and 8 lanes take 3.6 us
// for 4.0 with k = 8, but 4.9 for 3.7 with 65536 tokens and k = 1; of 256, 16 and 16 lanes 20 us
// for 25 with 65536 tokens, but 20 for 16 with a bias and fp64 keys to settle.
hipError_t launch_expert_route(const RouteArgs &a, hipStream_t s) {
  if (a.E <= 16) return RouteForward::group<4, 4>(a, s);
  if (a.E <= 64) return RouteForward::group<4, 16>(a, s);
  if (a.E <= 128) return RouteForward::group<8, 16>(a, s);
  if (a.E <= 256) return RouteForward::group<8, 32>(a, s);
  if (a.E <= 512) return RouteForward::wave<8>(a, s);
  return RouteForward::wave<16>(a, s);
}

template <int N, int L> static hipError_t route_backward(const RouteArgs &a, hipStream_t s) {
  constexpr int tokens = kRouteThreads / L;
  const int64_t need = (a.T + tokens - 1) / tokens;
  const dim3 grid((unsigned)(need < kRouteBackwardBlocks ? need : kRouteBackwardBlocks)), block(kRouteThreads);
  if (a.score == NSG_SCORE_SIGMOID) hipLaunchKernelGGL((expert_route_backward_kernel<N, L, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((expert_route_backward_kernel<N, L, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Few tokens leave the chip empty: a wave for each is done sooner (1024 / 2048 / 4096 tokens of
// 256 experts: 4.0 / 4.4 / 5.4 us, 16 lanes each 5.2 / 5.4 / 5.6; of 64: 3.6 / 4.0 / 4.5 and
// 4.1 / 4.2 / 4.4).
hipError_t launch_expert_route_backward(const RouteArgs &a, hipStream_t s) {
  const bool few = a.T <= 2048;
  if (a.E <= 16) return route_backward<4, 4>(a, s);
  if (a.E <= 64) return few ? route_backward<1, 64>(a, s) : route_backward<4, 16>(a, s);
  if (a.E <= 128) return few ? route_backward<2, 64>(a, s) : route_backward<8, 16>(a, s);
  if (a.E <= 256) return few ? route_backward<4, 64>(a, s) : route_backward<16, 16>(a, s);
  if (a.E <= 512) return few ? route_backward<8, 64>(a, s) : route_backward<16, 32>(a, s);
  return route_backward<16, 64>(a, s);
}

}  // namespace nsg
