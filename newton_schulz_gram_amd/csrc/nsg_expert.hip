// Tokens sorted by expert and back, on gfx950.
//
//   sort      a stable counting sort of the P = T k choices by expert:
//             offsets[e] = choices of the experts below e; rows[p] = offsets[id]
//             + earlier choices of the same expert, -1 for an id outside 0 .. E-1;
//             tokens[rows[p]] = p / k, -1 behind offsets[E].
//   dispatch  out[rows[t, j]] = x[t], 0 behind offsets[E]
//   combine   out[t] = sum_j w[t, j] y[rows[t, j]] (w = 1 where not given, which
//             is dispatch's gradient), in fp32, j in order, rounded once
//   combine's gradient  dy[rows[t, j]] = w[t, j] dout[t],
//             dw[t, j] = <dout[t], y[rows[t, j]]> in fp32
//
// The sort touches 16 bytes a choice and is bound by latency; the others are
// streaming passes, bound by HBM.  No atomics on memory: counts are integers,
// sums have a fixed order, so every result is reproducible bit for bit.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nsg_expert.h"
#include "nsg_segments.h"

namespace nsg {

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
static_assert(NSG_MAX_EXPERTS <= kSortThreads, "thread e scans expert e");
constexpr int kSortKept = 4;         // steps of 64 choices whose experts a wave keeps in registers
constexpr int kSortChunk = kSortThreads * kSortKept;  // choices of one workgroup, then
constexpr int kSortMaxChunks = 128;  // every workgroup of the second pass reads the whole table

// Choices of one workgroup, a multiple of 1024: up to kSortChunk choices take one
// workgroup and one launch; more, about 64 workgroups (4099 x 8 choices of 512
// experts: 9.0 us, with workgroups of kSortChunk 11.2) until they are of kSortChunk,
// then workgroups of that until there are kSortMaxChunks, which grow from there on
// (and read the ids twice).
static int64_t sort_chunk(int64_t P) {
  int64_t c = P;
  if (P > kSortChunk) {
    c = (P + 63) / 64;
    if (c > kSortChunk) c = kSortChunk;
    const int64_t least = (P + kSortMaxChunks - 1) / kSortMaxChunks;
    if (c < least) c = least;
  }
  return c == 0 ? kSortThreads : (c + kSortThreads - 1) / kSortThreads * kSortThreads;
}
int expert_sort_chunks(int64_t P) { return P == 0 ? 1 : (int)((P + sort_chunk(P) - 1) / sort_chunk(P)); }

// the expert of choice i, or -1
template <typename TI> __device__ __forceinline__ int expert_of(const TI *ids, int64_t i, int E) {
  const TI v = ids[i];
  return v >= 0 && v < (TI)E ? (int)v : -1;
}

// choices of each expert in each chunk
template <typename TI>
__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const TI *__restrict__ ids, int64_t P, int64_t chunk,
                                                                    int E, int32_t *__restrict__ table) {
  __shared__ int count[NSG_MAX_EXPERTS];
  for (int e = threadIdx.x; e < E; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * chunk, i1 = min(P, i0 + chunk);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) {
    const int e = expert_of(ids, i, E);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) table[(size_t)blockIdx.x * E + e] = count[e];
}

// Place the choices of chunk blockIdx.x.  at[w][e]: where the next choice of
// expert e in wave w's part of the chunk goes.  A wave takes its part 64 choices
// at a time: the lanes with the same expert find each other by ballots over the
// bits of the id, so their order is that of the choices.
template <typename TI, bool KEPT>
__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const TI *__restrict__ ids, int64_t P, int64_t chunk,
                                                                    int chunks, int k, int E, int bits,
                                                                    const int32_t *__restrict__ table,
                                                                    int32_t *__restrict__ offsets,
                                                                    int32_t *__restrict__ rows,
                                                                    int32_t *__restrict__ tokens) {
  __shared__ int at[kSortWaves * NSG_MAX_EXPERTS];
  __shared__ int sh[kSortWaves + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t i0 = (int64_t)blockIdx.x * chunk, i1 = min(P, i0 + chunk);
  const int64_t part = chunk / kSortWaves;  // a multiple of 64
  const int64_t w0 = i0 + wave * part, w1 = min(i1, w0 + part);
  int kept[kSortKept];
  if (KEPT) {
#pragma unroll
    for (int u = 0; u < kSortKept; ++u) {
      const int64_t p = w0 + u * 64 + lane;
      kept[u] = p < w1 ? expert_of(ids, p, E) : -1;
    }
  }
  for (int i = threadIdx.x; i < kSortWaves * E; i += kSortThreads) at[i] = 0;
  __syncthreads();
  if (KEPT) {
#pragma unroll
    for (int u = 0; u < kSortKept; ++u)
      if (kept[u] >= 0) atomicAdd(&at[wave * E + kept[u]], 1);
  } else {
    for (int64_t i = w0 + lane; i < w1; i += 64) {
      const int e = expert_of(ids, i, E);
      if (e >= 0) atomicAdd(&at[wave * E + e], 1);
    }
  }
  __syncthreads();
  // thread e: all of expert e's choices, and those before this chunk
  const int e = threadIdx.x;
  int total = 0, before = 0;
  if (e < E) {
    if (chunks == 1) {
      for (int w = 0; w < kSortWaves; ++w) total += at[w * E + e];
    } else {
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const int n = table[(size_t)c * E + e];
        total += n;
        before += c < (int)blockIdx.x ? n : 0;
      }
    }
  }
  int all;
  const int first = block_before<kSortThreads>(total, sh, all);
  if (e < E) {
    int next = first + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = at[w * E + e];
      at[w * E + e] = next;
      next += n;
    }
    if (blockIdx.x == 0) {
      offsets[e] = first;
      if (e == E - 1) offsets[E] = all;
    }
  }
  __syncthreads();
  volatile int *mine = at + wave * E;
  auto place = [&](int64_t p, int id) {
    uint64_t same = __ballot(id >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t one = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? one : ~one;
    }
    if (id >= 0) {
      const int rank = __popcll(same & ((1ull << lane) - 1)), n = __popcll(same);
      const int base = mine[id];
      __builtin_amdgcn_wave_barrier();
      if (rank == n - 1) mine[id] = base + n;
      rows[p] = base + rank;
      tokens[base + rank] = (int32_t)((uint32_t)p / (uint32_t)k);
    } else if (p < w1) {
      rows[p] = -1;
    }
    __builtin_amdgcn_wave_barrier();
  };
  if (KEPT) {
#pragma unroll
    for (int u = 0; u < kSortKept; ++u)
      if (w0 + u * 64 < w1) place(w0 + u * 64 + lane, kept[u]);
  } else {
    for (int64_t i = w0; i < w1; i += 64) place(i + lane, i + lane < w1 ? expert_of(ids, i + lane, E) : -1);
  }
  for (int64_t p = i0 + threadIdx.x; p < i1; p += kSortThreads)
    if (p >= all) tokens[p] = -1;
}

template <typename TI>
static hipError_t sort_t(const void *ids, int64_t P, int k, int E, int32_t *offsets, int32_t *rows, int32_t *tokens,
                         int32_t *table, hipStream_t s) {
  const int64_t chunk = sort_chunk(P);
  const int chunks = expert_sort_chunks(P);
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  if (chunks > 1) {
    hipLaunchKernelGGL(expert_count_kernel<TI>, dim3((unsigned)chunks), dim3(kSortThreads), 0, s,
                       (const TI *)ids, P, chunk, E, table);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (chunk <= kSortChunk)
    hipLaunchKernelGGL((expert_place_kernel<TI, true>), dim3((unsigned)chunks), dim3(kSortThreads), 0, s, (const TI *)ids, P,
                       chunk, chunks, k, E, bits, (const int32_t *)table, offsets, rows, tokens);
  else
    hipLaunchKernelGGL((expert_place_kernel<TI, false>), dim3((unsigned)chunks), dim3(kSortThreads), 0, s, (const TI *)ids, P,
                       chunk, chunks, k, E, bits, (const int32_t *)table, offsets, rows, tokens);
  return hipGetLastError();
}

hipError_t launch_expert_sort(const void *ids, int wide, int64_t P, int k, int E, int32_t *offsets, int32_t *rows,
                              int32_t *tokens, int32_t *table, hipStream_t s) {
  return wide ? sort_t<int64_t>(ids, P, k, E, offsets, rows, tokens, table, s)
              : sort_t<int32_t>(ids, P, k, E, offsets, rows, tokens, table, s);
}

// ---------------------------------------------------------------------------
// dispatch: one wave per 64 x 16 bytes of a token (a part; see Parts), read once and stored to the rows of the token's choices; rows behind the last
// expert's are cleared by the choices of the same numbers.  Elements are moved as
// they are, so only their size matters.
// ---------------------------------------------------------------------------
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Outputs up to this size (the last-level cache holds 256 MB) stay there for what
// reads them next; larger ones are streamed past it: 134 MB in 24 us kept and 26
// streamed, 197 MB in 39.5 both, 268 MB in 56 and 53, 537 MB in 121 and 104.
constexpr int64_t kDispatchKept = 224 << 20;

// Four waves of a workgroup take 1 << lp parts of 4 >> lp tokens: a row's parts are
// read and written together (one token's four parts to a workgroup instead of four
// tokens' first parts, 16384 x 8 rows of 4 KB: dispatch 153 -> 104 us, combine 155 ->
// 120, 4.9 and 5.0 TB/s).
struct Parts {
  int64_t t, part;
  __device__ __forceinline__ explicit Parts(int lp) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    t = (int64_t)blockIdx.x * (4 >> lp) + (wave >> lp);
    part = ((int64_t)blockIdx.y << lp) + (wave & ((1 << lp) - 1));
  }
};
// lp and the grid for T tokens of so many parts (HIP counts a launch's threads in 32 bits)
static int parts_log(int64_t T, int64_t parts) { return T > (1 << 23) || parts < 2 ? 0 : parts < 4 ? 1 : 2; }
static dim3 parts_grid(int64_t T, int64_t parts, int lp) {
  return dim3((unsigned)((T + (4 >> lp) - 1) / (4 >> lp)), (unsigned)((parts + (1 << lp) - 1) >> lp));
}

template <typename V, bool STREAM>
__global__ void __launch_bounds__(256) expert_dispatch_kernel(const V *__restrict__ x, int64_t T, int64_t n, int64_t ldx,
                                                              const int32_t *__restrict__ offsets, int E,
                                                              const int32_t *__restrict__ rows, int k,
                                                              int lp, V *__restrict__ out) {
  const Parts at(lp);
  const int64_t t = at.t, c = at.part * 64 + (threadIdx.x & 63);
  if (t >= T || c >= n) return;
  const int64_t P = T * k, all = seg_clamp(offsets[E], 0, (int)P);
  const V v = x[t * ldx + c];
#pragma unroll 4
  for (int64_t p = t * k; p < (t + 1) * k; ++p) {
    const int64_t r = rows[p];
    if (r >= 0 && r < P) {
      if (STREAM) __builtin_nontemporal_store(v, out + r * n + c);
      else out[r * n + c] = v;
    }
    if (p >= all) out[p * n + c] = V(0);
  }
}

static bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename V>
static hipError_t dispatch_t(const void *x, int64_t T, int64_t n, int64_t ldx, const int32_t *offsets, int E,
                             const int32_t *rows, int k, void *out, hipStream_t s) {
  const int64_t parts = (n + 63) / 64;
  const int lp = parts_log(T, parts);
  const dim3 grid = parts_grid(T, parts, lp);
  if (T * k * n * (int64_t)sizeof(V) > kDispatchKept)
    hipLaunchKernelGGL((expert_dispatch_kernel<V, true>), grid, dim3(256), 0, s, (const V *)x, T, n, ldx, offsets, E, rows, k,
                       lp, (V *)out);
  else
    hipLaunchKernelGGL((expert_dispatch_kernel<V, false>), grid, dim3(256), 0, s, (const V *)x, T, n, ldx, offsets, E, rows, k,
                       lp, (V *)out);
  return hipGetLastError();
}

hipError_t launch_expert_dispatch(const void *x, int elem, int64_t T, int64_t C, int64_t ldx, const int32_t *offsets, int E,
                                  const int32_t *rows, int k, void *out, hipStream_t s) {
  const int64_t per = 16 / elem;
  if (aligned16(x) && aligned16(out) && C % per == 0 && ldx % per == 0)
    return dispatch_t<u32x4>(x, T, C / per, ldx / per, offsets, E, rows, k, out, s);
  if (elem == 4) return dispatch_t<uint32_t>(x, T, C, ldx, offsets, E, rows, k, out, s);
  return dispatch_t<uint16_t>(x, T, C, ldx, offsets, E, rows, k, out, s);
}

// ---------------------------------------------------------------------------
// combine and its gradient.  A lane owns V consecutive elements of a row: 16
// bytes of them, or one element where rows do not take 16-byte accesses.
// ---------------------------------------------------------------------------
// ALIGN: bytes that the elements are aligned to (the instructions take any).
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

// One wave per 64 V elements of a token (a part).
template <typename T, int V>
__global__ void __launch_bounds__(256) expert_combine_kernel(const T *__restrict__ y, int64_t P, int64_t C, int64_t ldy,
                                                             const int32_t *__restrict__ rows, int64_t ntok, int k,
                                                             const float *__restrict__ w, int lp, T *__restrict__ out) {
  const Parts at(lp);
  const int64_t t = at.t, c = (at.part * 64 + (threadIdx.x & 63)) * V;
  if (t >= ntok || c >= C) return;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int64_t r = rows[t * k + j];
    if (r < 0 || r >= P) continue;
    const float g = w ? w[t * k + j] : 1.f;
    float f[V];
    Row<T, V>::load(y + r * ldy + c, f);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(g, f[v], acc[v]);
  }
  Row<T, V>::store(out + t * C + c, acc);
}

// One wave per choice; a token's choices are neighbours, so dout comes from cache
// for all but one.  Whether a lane takes V elements at once goes by C alone, so that
// neither alignment nor pitch changes the order of dw's sum.
template <typename T, int V>
__global__ void __launch_bounds__(256) expert_combine_backward_kernel(
    const T *__restrict__ dout, int64_t lddo, const T *__restrict__ y, int64_t ldy, int64_t P, int64_t C,
    const int32_t *__restrict__ offsets, int E, const int32_t *__restrict__ rows, int k, const float *__restrict__ w,
    T *__restrict__ dy, float *__restrict__ dw) {
  const int lane = threadIdx.x & 63;
  const int64_t p = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (p >= P) return;
  const int64_t t = (uint32_t)p / (uint32_t)k;
  const int64_t r = rows[p];
  const bool there = r >= 0 && r < P;
  float dot = 0.f;
  if (there) {
    const float g = w ? w[p] : 1.f;
    const T *d = dout + t * lddo, *f = y + r * ldy;
    T *out = dy + r * C;
#pragma unroll 4
    for (int64_t c = (int64_t)lane * V; c < C; c += 64 * V) {
      float u[V], v[V];
      Row<T, V, (int)sizeof(T)>::load(d + c, u);
      Row<T, V, (int)sizeof(T)>::load(f + c, v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dot = fmaf(u[i], v[i], dot);
        u[i] *= g;
      }
      Row<T, V, (int)sizeof(T)>::store(out + c, u);
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) dot += __shfl_xor(dot, off, 64);
  if (lane == 0) dw[p] = there ? dot : 0.f;
  if (p >= seg_clamp(offsets[E], 0, (int)P)) {  // a row behind the last expert's
    float z[V];
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = 0.f;
    for (int64_t c = (int64_t)lane * V; c < C; c += 64 * V) Row<T, V, (int)sizeof(T)>::store(dy + p * C + c, z);
  }
}

template <typename T, int V>
static hipError_t combine_v(const void *y, int64_t P, int64_t C, int64_t ldy, const int32_t *rows, int64_t ntok, int k,
                            const float *w, void *out, hipStream_t s) {
  const int64_t parts = (C + 64 * V - 1) / (64 * V);
  const int lp = parts_log(ntok, parts);
  hipLaunchKernelGGL((expert_combine_kernel<T, V>), parts_grid(ntok, parts, lp), dim3(256), 0, s, (const T *)y, P, C, ldy,
                     rows, ntok, k, w, lp, (T *)out);
  return hipGetLastError();
}

template <typename T>
static hipError_t combine_t(const void *y, int64_t P, int64_t C, int64_t ldy, const int32_t *rows, int64_t ntok, int k,
                            const float *w, void *out, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (aligned16(y) && aligned16(out) && C % V == 0 && ldy % V == 0)
    return combine_v<T, V>(y, P, C, ldy, rows, ntok, k, w, out, s);
  return combine_v<T, 1>(y, P, C, ldy, rows, ntok, k, w, out, s);
}

hipError_t launch_expert_combine(const void *y, int dtype, int64_t P, int64_t C, int64_t ldy, const int32_t *rows,
                                 int64_t T, int k, const float *w, void *out, hipStream_t s) {
  switch (dtype) {
    case NSG_F16: return combine_t<_Float16>(y, P, C, ldy, rows, T, k, w, out, s);
    case NSG_BF16: return combine_t<__bf16>(y, P, C, ldy, rows, T, k, w, out, s);
    default: return combine_t<float>(y, P, C, ldy, rows, T, k, w, out, s);
  }
}

template <typename T>
static hipError_t backward_t(const void *dout, int64_t lddo, const void *y, int64_t ldy, int64_t P, int64_t C,
                             const int32_t *offsets, int E, const int32_t *rows, int k, const float *w, void *dy,
                             float *dw, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const dim3 grid((unsigned)((P + 3) / 4));
  if (C % V == 0)
    hipLaunchKernelGGL((expert_combine_backward_kernel<T, V>), grid, dim3(256), 0, s, (const T *)dout, lddo,
                       (const T *)y, ldy, P, C, offsets, E, rows, k, w, (T *)dy, dw);
  else
    hipLaunchKernelGGL((expert_combine_backward_kernel<T, 1>), grid, dim3(256), 0, s, (const T *)dout, lddo,
                       (const T *)y, ldy, P, C, offsets, E, rows, k, w, (T *)dy, dw);
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const void *dout, int64_t lddo, const void *y, int64_t ldy, int dtype,
                                          int64_t P, int64_t C, const int32_t *offsets, int E, const int32_t *rows,
                                          int64_t T, int k, const float *w, void *dy, float *dw, hipStream_t s) {
  switch (dtype) {
    case NSG_F16: return backward_t<_Float16>(dout, lddo, y, ldy, P, C, offsets, E, rows, k, w, dy, dw, s);
    case NSG_BF16: return backward_t<__bf16>(dout, lddo, y, ldy, P, C, offsets, E, rows, k, w, dy, dw, s);
    default: return backward_t<float>(dout, lddo, y, ldy, P, C, offsets, E, rows, k, w, dy, dw, s);
  }
}

}  // namespace nsg
