// Embedding of token ids and its gradient, on gfx950.
//
//   forward   out[t] = scale W[ids[t]], zeros for an id outside 0 .. V - 1
//   gradient  dW[v] = scale sum of dout[t] over the tokens with ids[t] = v
//
// Both are streaming passes, bound by HBM: 16384 rows of 4096 in bf16 take 43 us (5.1 TB/s by
// the rows that are read and written), the gradient of 65536, over 128000 of them, 355 (4.5;
// half of it is clearing).  The gradient sorts the tokens by id
// (stably, in one or two digits) and sums the runs of equal ids.  The sorted list is
// cut into chunks of a length that only the sizes fix; what a run has inside one
// chunk is summed in token order, and a run over several chunks is joined from their
// sums, in order.  No atomics on memory: every result is reproducible bit for bit.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nsg_layer.h"
#include "nsg_rows.h"
#include "nsg_segments.h"

namespace nsg {

// ---------------------------------------------------------------------------
// Rows in pieces of 16 bytes.  Long ones: one wave per 64 pieces (a part), four waves of a
// workgroup take 1 << lp parts of 4 >> lp rows.  Rows of at most 32 pieces (SHORT): 1 << lp
// lanes a row, several rows to a wave (524288 rows of 64 in bf16: 81 us, so 18).
// ---------------------------------------------------------------------------
template <bool SHORT> struct Lane {
  int64_t t, piece;
  __device__ __forceinline__ explicit Lane(int lp) {
    if (SHORT) {
      t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lp;
      piece = threadIdx.x & ((1 << lp) - 1);
    } else {
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      t = (int64_t)blockIdx.x * (4 >> lp) + (wave >> lp);
      piece = (((int64_t)blockIdx.y << lp) + (wave & ((1 << lp) - 1))) * 64 + (threadIdx.x & 63);
    }
  }
};
// (HIP counts a launch's threads in 32 bits)
struct LaneGrid {
  bool is_short;
  int lp;
  dim3 grid;
  LaneGrid(int64_t rows, int64_t pieces) {
    is_short = pieces <= 32;
    const int64_t parts = (pieces + 63) / 64;
    if (is_short) {
      lp = 0;
      while ((1 << lp) < pieces) ++lp;
      grid = dim3((unsigned)(((rows << lp) + 255) / 256));
    } else {
      lp = rows > (1 << 23) || parts < 2 ? 0 : parts < 4 ? 1 : 2;
      grid = dim3((unsigned)((rows + (4 >> lp) - 1) / (4 >> lp)), (unsigned)((parts + (1 << lp) - 1) >> lp));
    }
  }
};

// N elements of a row from c on, zeros behind its end
template <typename T, int N> struct Cells {
  typedef T vec __attribute__((ext_vector_type(N)));
  typedef vec mem __attribute__((aligned(sizeof(T))));
  vec v;
  __device__ __forceinline__ void load(const T *row, int64_t c, int64_t C) {
    if (c + N <= C) {
      v = *reinterpret_cast<const mem *>(row + c);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = c + i < C ? row[c + i] : (T)0.f;
    }
  }
};
template <typename T, int N> __device__ __forceinline__ void store_cells(T *row, int64_t c, int64_t C, const float (&f)[N]) {
  if (c + N <= C) {
    Row<T, N, (int)sizeof(T)>::store(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < C) row[c + i] = (T)f[i];
  }
}
// A last piece that is not whole lies over the one before it: two lanes write the same there
template <int N> __device__ __forceinline__ int64_t piece_at(int64_t piece, int64_t C) {
  const int64_t c = piece * N;
  return c + N > C && C >= N ? C - N : c;
}

// id i, or -1 where it is none of 0 .. V - 1
__device__ __forceinline__ int id_at(const void *ids, int wide, int64_t i, int64_t V) {
  const int64_t v = wide ? reinterpret_cast<const int64_t *>(ids)[i] : reinterpret_cast<const int32_t *>(ids)[i];
  return v >= 0 && v < V ? (int)v : -1;
}

template <typename T, bool SHORT>
__global__ void __launch_bounds__(256) embedding_kernel(const void *__restrict__ ids, int wide, int64_t ntok,
                                                        const T *__restrict__ W, int64_t V, int64_t C, int64_t ldw,
                                                        float scale, int lp, T *__restrict__ out) {
  constexpr int N = 16 / (int)sizeof(T);
  const Lane<SHORT> at(lp);
  if (at.t >= ntok || at.piece * N >= C) return;
  const int64_t c = piece_at<N>(at.piece, C);
  const int v = id_at(ids, wide, at.t, V);
  Cells<T, N> row;
  if (v >= 0) row.load(W + (int64_t)v * ldw, c, C);
  float f[N];
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = v >= 0 ? (float)row.v[i] * scale : 0.f;
  store_cells<T, N>(out + at.t * C, c, C, f);
}

template <typename T> static hipError_t embedding_t(const EmbedArgs &a, hipStream_t s) {
  constexpr int N = 16 / (int)sizeof(T);
  const LaneGrid g(a.T, (a.C + N - 1) / N);
  if (g.is_short)
    hipLaunchKernelGGL((embedding_kernel<T, true>), g.grid, dim3(256), 0, s, a.ids, a.wide, a.T, (const T *)a.x, a.V, a.C, a.ld,
                       a.scale, g.lp, (T *)a.out);
  else
    hipLaunchKernelGGL((embedding_kernel<T, false>), g.grid, dim3(256), 0, s, a.ids, a.wide, a.T, (const T *)a.x, a.V, a.C, a.ld,
                       a.scale, g.lp, (T *)a.out);
  return hipGetLastError();
}

hipError_t launch_embedding(const EmbedArgs &a, hipStream_t s) {
  switch (a.x_dtype) {
    case NSG_F16: return embedding_t<_Float16>(a, s);
    case NSG_BF16: return embedding_t<__bf16>(a, s);
    default: return embedding_t<float>(a, s);
  }
}

// ---------------------------------------------------------------------------
// Clearing dW.  The sort waits for its own memory accesses most of the time and keeps few
// CUs busy, so its launches have more workgroups, which clear a share of dW each.
// ---------------------------------------------------------------------------
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct Clear {
  u32x4 *mid = nullptr;             // n units of 16 bytes
  int64_t n = 0;
  uint16_t *head = nullptr, *tail = nullptr;  // what lies before and behind them: less than 16 bytes each
  int nhead = 0, ntail = 0;
  int blocks = 0;                   // workgroups that share it, behind those of the sort
  bool stream = false;              // past the caches
  __device__ __forceinline__ void run(int block) const {
    const int64_t per = (n + blocks - 1) / blocks, i1 = min(n, (block + 1) * per);
    if (stream) {
      for (int64_t i = block * per + threadIdx.x; i < i1; i += blockDim.x) __builtin_nontemporal_store(u32x4(0), mid + i);
    } else {
      for (int64_t i = block * per + threadIdx.x; i < i1; i += blockDim.x) mid[i] = u32x4(0);
    }
    if (block == 0 && (int)threadIdx.x < nhead) head[threadIdx.x] = 0;
    if (block == 0 && (int)threadIdx.x < ntail) tail[threadIdx.x] = 0;
  }
};
// A dW that the last-level cache (256 MB) holds is cleared in it, a larger one past it: the
// gradient of 4099 tokens (98 MB) takes 27 us, streamed 32; of 65536 (1.05 GB) 372, streamed 354.
constexpr int64_t kClearKept = 224 << 20;

// share i of `shares` of `bytes` bytes at p
static Clear clear_share(void *p, int64_t bytes, int i, int shares) {
  Clear c;
  if (bytes == 0) return c;
  char *b = (char *)p;
  int64_t head = (16 - reinterpret_cast<uintptr_t>(p) % 16) % 16;
  if (head > bytes) head = bytes;
  const int64_t n = (bytes - head) / 16, i0 = n * i / shares;
  c.mid = (u32x4 *)(b + head) + i0;
  c.n = n * (i + 1) / shares - i0;
  if (i == 0) {
    c.head = (uint16_t *)b;
    c.nhead = (int)(head / 2);
    c.tail = (uint16_t *)(b + head + n * 16);
    c.ntail = (int)((bytes - head - n * 16) / 2);
  }
  const int64_t blocks = (c.n + 4095) / 4096;  // 64 KB or more to a workgroup
  c.blocks = blocks > 1024 ? 1024 : blocks < 1 ? 1 : (int)blocks;
  c.stream = bytes > kClearKept;
  return c;
}
__global__ void __launch_bounds__(1024) embed_clear_kernel(Clear c) { c.run((int)blockIdx.x); }

// ---------------------------------------------------------------------------
// the gradient's sort: a stable counting sort of the tokens by their id, by its low
// digit and then by its high one (ids of up to 10 bits: one digit).  Tokens without an
// id are left out: keys behind the last token that has one are -1.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortBits = 10;
constexpr int kSortBins = 1 << kSortBits;
// steps of 64 tokens that a wave keeps in registers (131072 and 524288 tokens: the call takes
// 41.6 and 69 us so, 42.5 and 71 with the tokens read again)
constexpr int kSortKept = 4;
constexpr int kSortChunk = kSortThreads * kSortKept;   // tokens of one workgroup, then
constexpr int kSortMaxChunks = 128;                    // every workgroup reads the whole table
// Steps of a sort by one workgroup, in LDS: 8192 tokens take 16 us, in four launches 17 (1024: 7)
constexpr int kSortAlone = 8;
static_assert(NSG_MAX_VOCAB <= kSortBins * kSortBins, "two digits");

struct SortPlan {
  int64_t chunk;
  int chunks, digits, bits;  // bits of a digit
};
static SortPlan sort_plan(int64_t N, int64_t V) {
  SortPlan p;
  p.chunk = N;
  if (N > kSortThreads * kSortAlone) {
    p.chunk = (N + 63) / 64;
    if (p.chunk > kSortChunk) p.chunk = kSortChunk;
    const int64_t least = (N + kSortMaxChunks - 1) / kSortMaxChunks;
    if (p.chunk < least) p.chunk = least;
  }
  p.chunk = (p.chunk + kSortThreads - 1) / kSortThreads * kSortThreads;
  p.chunks = N == 0 ? 1 : (int)((N + p.chunk - 1) / p.chunk);
  int bits = 1;
  while ((1ll << bits) < V) ++bits;
  p.digits = bits <= kSortBits ? 1 : 2;
  p.bits = (bits + p.digits - 1) / p.digits;
  return p;
}

struct Pair {  // a token and its id, -1 behind the last token that has one
  int key, tok;
};
// the tokens before a digit's pass: the ids as they are, or the pairs of the pass before
struct SortInput {
  const void *ids;
  int wide;
  int64_t V;
  const Pair *pairs;  // NULL: ids
  __device__ __forceinline__ Pair operator()(int64_t i) const { return pairs ? pairs[i] : Pair{id_at(ids, wide, i, V), (int)i}; }
};

// tokens of each value of the digit in each chunk
__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(SortInput in, int64_t N, int64_t chunk, int shift, int bits,
                                                                   int32_t *__restrict__ table, int chunks, Clear c) {
  if ((int)blockIdx.x >= chunks) return c.run((int)blockIdx.x - chunks);
  __shared__ int count[kSortBins];
  const int bins = 1 << bits;
  for (int e = threadIdx.x; e < bins; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * chunk, i1 = min(N, i0 + chunk);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) {
    const int k = in(i).key;
    if (k >= 0) atomicAdd(&count[(k >> shift) & (bins - 1)], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += kSortThreads) table[(size_t)blockIdx.x * bins + e] = count[e];
}

// Place the tokens of chunk `block`: get(i) reads pair i, put(i, pair) writes it.
// at[w][d]: where the next token with digit d in wave w's part of the chunk goes.  A wave
// takes its part 64 tokens at a time: the lanes with the same digit find each other by
// ballots over its bits, so their order is that of the tokens.  KEPT: steps of 64 tokens a
// wave keeps, 0: it reads them again.
template <int KEPT, class Get, class Put>
__device__ __forceinline__ void place_chunk(Get get, Put put, int64_t N, int64_t chunk, int chunks, int block, int shift, int bits,
                                            const int32_t *__restrict__ table, int *at, int *sh) {
  const int bins = 1 << bits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t i0 = (int64_t)block * chunk, i1 = min(N, i0 + chunk);
  const int64_t part = chunk / kSortWaves;  // a multiple of 64, with KEPT at most KEPT 64
  const int64_t w0 = i0 + wave * part, w1 = min(i1, w0 + part);
  const Pair none{-1, 0};
  Pair kept[KEPT > 0 ? KEPT : 1];
  if (KEPT > 0) {
#pragma unroll
    for (int u = 0; u < KEPT; ++u) {
      const int64_t p = w0 + u * 64 + lane;  // (w1: also the end of the wave's part)
      kept[u] = none;
      if (p < w1) kept[u] = get(p);
    }
  }
  for (int i = threadIdx.x; i < kSortWaves * bins; i += kSortThreads) at[i] = 0;
  __syncthreads();
  if (KEPT > 0) {
#pragma unroll
    for (int u = 0; u < KEPT; ++u)
      if (kept[u].key >= 0) atomicAdd(&at[wave * bins + ((kept[u].key >> shift) & (bins - 1))], 1);
  } else {
    for (int64_t i = w0 + lane; i < w1; i += 64) {
      const int k = get(i).key;
      if (k >= 0) atomicAdd(&at[wave * bins + ((k >> shift) & (bins - 1))], 1);
    }
  }
  __syncthreads();
  // thread e: all tokens with digit e, and those before this chunk
  const int e = threadIdx.x;
  int total = 0, before = 0, own[kSortWaves];
  if (e < bins) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) own[w] = at[w * bins + e];
    if (chunks == 1) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) total += own[w];
    } else {
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const int n = table[(size_t)c * bins + e];
        total += n;
        before += c < block ? n : 0;
      }
    }
  }
  int all;
  const int first = block_before<kSortThreads>(total, sh, all);
  if (e < bins) {
    int next = first + before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      at[w * bins + e] = next;
      next += own[w];
    }
  }
  __syncthreads();
  int *const mine = at + wave * bins;
  auto wave_sync = [] {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  auto place = [&](Pair v) {
    const int d = (v.key >> shift) & (bins - 1);
    const uint64_t there = __ballot(v.key >= 0);
    unsigned lo = (unsigned)there, hi = (unsigned)(there >> 32);
    auto match = [&](int b) {  // (bits that no digit has change nothing)
      const int set = (d << (31 - b)) >> 31;  // all bits of it
      const uint64_t one = __ballot(set);
      lo = __builtin_amdgcn_bitop3_b32(lo, (unsigned)one, (unsigned)set, 0x90);  // lo & ~(one ^ set)
      hi = __builtin_amdgcn_bitop3_b32(hi, (unsigned)(one >> 32), (unsigned)set, 0x90);
    };
#pragma unroll
    for (int b = 0; b < 8; ++b) match(b);
    if (bits > 8) {
#pragma unroll
      for (int b = 8; b < kSortBits; ++b) match(b);
    }
    if (v.key >= 0) {
      const int rank = (int)__builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0)), n = __popc(lo) + __popc(hi);
      const int base = mine[d];
      wave_sync();
      if (rank == n - 1) mine[d] = base + n;
      put(base + rank, v);
    }
    wave_sync();
  };
  if (KEPT > 0) {
#pragma unroll
    for (int u = 0; u < KEPT; ++u)
      if (w0 + u * 64 < w1) place(kept[u]);
  } else {
    for (int64_t i = w0; i < w1; i += 64) {
      Pair v = none;
      if (i + lane < w1) v = get(i + lane);
      place(v);
    }
  }
  for (int64_t p = i0 + threadIdx.x; p < i1; p += kSortThreads)
    if (p >= all) put(p, none);
}

template <int KEPT>
__global__ void __launch_bounds__(kSortThreads) embed_place_kernel(SortInput in, int64_t N, int64_t chunk, int chunks, int shift,
                                                                   int bits, const int32_t *__restrict__ table,
                                                                   Pair *__restrict__ pairs, Clear c) {
  if ((int)blockIdx.x >= chunks) return c.run((int)blockIdx.x - chunks);
  __shared__ int at[kSortWaves * kSortBins];
  __shared__ int sh[kSortWaves + 1];
  place_chunk<KEPT>(in, [&](int64_t i, Pair v) { pairs[i] = v; }, N, chunk, chunks, (int)blockIdx.x, shift, bits, table, at, sh);
}

// All digits by one workgroup.  The pairs stay in LDS between the passes, where stores to
// scattered places cost less than in memory (a cache line each).
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(SortInput in, int64_t N, int64_t chunk, int digits, int bits,
                                                                  Pair *__restrict__ pairs, Clear c) {
  if (blockIdx.x > 0) return c.run((int)blockIdx.x - 1);
  __shared__ int at[kSortWaves * kSortBins];
  __shared__ int sh[kSortWaves + 1];
  __shared__ Pair list[kSortThreads * kSortAlone];
  auto put = [&](int64_t i, Pair v) { list[i] = v; };
  place_chunk<kSortAlone>(in, put, N, chunk, 1, 0, 0, bits, nullptr, at, sh);
  __syncthreads();
  if (digits == 2) {
    // (every thread has read its pairs before the first barrier in there, so they may be overwritten)
    place_chunk<kSortAlone>([&](int64_t i) { return list[i]; }, put, N, chunk, 1, 0, bits, bits, nullptr, at, sh);
    __syncthreads();
  }
  for (int64_t i = threadIdx.x; i < N; i += kSortThreads) pairs[i] = list[i];
}

// ---------------------------------------------------------------------------
// the gradient's sums
// ---------------------------------------------------------------------------
constexpr int kRunUnroll = 8;

// Sorted tokens of a chunk: enough rows on their way to keep the memory busy, at least one
// round of loads, and few sums of parts of runs (524288 rows of 64 in bf16, chunks of 16,
// 32 and 64: sums 18, 25 and 42 us, joining them 15, 9 and 6; 262144 in fp32: 19, 17, 24 and 12, 8, 5).
static int64_t run_chunk(int64_t N, int64_t C) {
  int64_t S = kRunUnroll;
  while (S < 64 && N / (2 * S) * C >= 2048 * 512) S *= 2;
  return S;
}
static int64_t run_chunks(int64_t N, int64_t C) { return (N + run_chunk(N, C) - 1) / run_chunk(N, C); }

// where the sums of parts of runs lie: two rows of fp32 for each chunk, what its first
// run has here if it began before, and what its last one has if it began here and goes on
static int64_t part_pitch(int64_t C) { return (C + 3) / 4 * 4; }

// a chunk's runs
struct Chunk {
  int64_t p0, p1;
  int last;  // its last run
  bool before, after, whole;  // the first run began in an earlier chunk; the last one goes on; they are one
  __device__ __forceinline__ Chunk(const Pair *pairs, int64_t N, int64_t S, int64_t c) {
    p0 = c * S;
    p1 = min(N, p0 + S);
    // (all four loads at once)
    const int first = pairs[p0].key, prev = pairs[p0 > 0 ? p0 - 1 : 0].key;
    last = pairs[p1 - 1].key;
    const int next = pairs[p1 < N ? p1 : p1 - 1].key;
    before = p0 > 0 && first >= 0 && prev == first;
    after = p1 < N && last >= 0 && next == last;
    whole = before && first == last;
  }
};

// A lane sums its piece of a chunk's rows.  With ADD a run's row of dW is read together with
// its first row of dout.
template <typename T, typename O, bool ADD, bool SHORT>
__global__ void __launch_bounds__(256) embed_runs_kernel(const Pair *__restrict__ pairs, int64_t ntok, int64_t S, int64_t chunks, const T *__restrict__ dout,
                                                         int64_t ld, int64_t C, float scale, int lp,
                                                         O *__restrict__ out, float *__restrict__ parts, int64_t pitch) {
  constexpr int N = 16 / (int)sizeof(T);
  const Lane<SHORT> at(lp);
  if (at.t >= chunks || at.piece * N >= C) return;
  // (with ADD no element may be read and written by two lanes)
  const int64_t c = ADD ? at.piece * N : piece_at<N>(at.piece, C);
  const Chunk ch(pairs, ntok, S, at.t);
  float acc[N];
  Cells<O, N> old;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    acc[i] = 0.f;
    if (ADD) old.v[i] = (O)0.f;
  }
  int run = -1;
  bool began = ch.before;  // the present run began in an earlier chunk
  auto close = [&](bool goes_on) {
    if (began || goes_on) {
      store_cells<float, N>(parts + (at.t * 2 + (began ? 0 : 1)) * pitch, c, C, acc);
    } else {
      float f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = ADD ? fmaf(acc[i], scale, (float)old.v[i]) : acc[i] * scale;
      store_cells<O, N>(out + (int64_t)run * C, c, C, f);
    }
  };
  int last = -1;
  for (int64_t p = ch.p0; p < ch.p1; p += kRunUnroll) {
    int key[kRunUnroll];
    Cells<T, N> row[kRunUnroll];
    Cells<O, N> was[ADD ? kRunUnroll : 1];
#pragma unroll
    for (int u = 0; u < kRunUnroll; ++u) {
      const Pair v = p + u < ch.p1 ? pairs[p + u] : Pair{-1, 0};  // keys of -1 are the last ones
      key[u] = v.key;
      if (key[u] >= 0) {
        row[u].load(dout + (int64_t)v.tok * ld, c, C);
        if (ADD && key[u] != last) was[ADD ? u : 0].load(out + (int64_t)key[u] * C, c, C);
      }
      last = key[u];
    }
#pragma unroll
    for (int u = 0; u < kRunUnroll; ++u) {
      if (key[u] < 0) continue;
      if (key[u] != run) {
        if (run >= 0) {
          close(false);
          began = false;
        }
        run = key[u];
        if (ADD) old = was[ADD ? u : 0];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += (float)row[u].v[i];
    }
  }
  if (run >= 0) close(ch.after);
}

// The run that begins in chunk t and goes on: its parts in the order of the chunks.  A wave
// takes 256 elements of it, a workgroup as many of 16 chunks.  A run of many parts (a
// padding token's; at most one begins in a workgroup's chunks) is summed by all its waves,
// wave w every 16th part from w on: one of 8192 parts of 1024 takes 134 us, by one wave 609;
// joining the runs of 65536 tokens of 4096, half of which are the same, 33 us, by one wave each 73.
constexpr int kJoinWaves = 16;
// Parts of a run that one wave sums, more by all (65536 tokens of 1024, 2000 of an id, so 32
// parts: the call takes 50 us where one wave sums them, 48 where all do)
constexpr int kJoinAlone = 16;
static_assert(kJoinAlone >= kJoinWaves, "one run of many parts in a workgroup");
template <typename O>
__global__ void __launch_bounds__(kJoinWaves * 64) embed_join_kernel(const Pair *__restrict__ pairs, int64_t ntok, int64_t S,
                                                                     int64_t chunks, int64_t C, float scale, bool add,
                                                                     O *__restrict__ out, const float *__restrict__ parts,
                                                                     int64_t pitch) {
  __shared__ int many[kJoinWaves];  // parts of a wave's run that all waves sum, 0: none
  __shared__ float sums[kJoinWaves][256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (int64_t)blockIdx.x * kJoinWaves, t = t0 + wave, c = (int64_t)blockIdx.y * 256 + lane * 4;
  int run = -1;
  int64_t more = 0;  // chunks that the run goes on in
  if (t < chunks) {
    const Chunk ch(pairs, ntok, S, t);
    if (ch.after && !ch.whole) run = ch.last;
  }
  if (run >= 0) {
    // chunks behind t that begin with it: the first so many of `left`
    for (int64_t left = chunks - 1 - t, unit = 1; left > 0; unit = (left + 63) / 64) {
      const int64_t q = more + (lane + 1) * unit;
      const uint64_t on = __ballot(q <= more + left && pairs[(q <= more + left ? t + q : t) * S].key == run);
      const int n = on == ~0ull ? 64 : __ffsll((long long)~on) - 1;
      more += n * unit;
      left = min(left - n * unit, n == 64 ? left : unit - 1);
    }
  }
  if (lane == 0) many[wave] = more > kJoinAlone ? (int)more : 0;
  __syncthreads();
  // parts i, i + step, ... of the run that begins in chunk `from`
  auto add_parts = [&](int64_t from, int64_t i, int64_t step, int64_t n, float(&acc)[4]) {
    if (c >= C) return;
#pragma unroll 8
    for (; i <= n; i += step) {
      float f[4];
      Row<float, 4>::load(parts + (from + i) * 2 * pitch + c, f);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] += f[v];
    }
  };
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (run >= 0 && c < C) Row<float, 4>::load(parts + (t * 2 + 1) * pitch + c, acc);
  if (more <= kJoinAlone) add_parts(t, 1, 1, more, acc);
  const uint64_t shared = __ballot(many[lane % kJoinWaves] > 0);
  if (shared != 0) {
    const int who = __ffsll((long long)shared) - 1;  // whose run that is
    float own[4] = {0.f, 0.f, 0.f, 0.f};
    add_parts(t0 + who, 1 + wave, kJoinWaves, many[who], own);
    Row<float, 4>::store(&sums[wave][lane * 4], own);
    __syncthreads();
    if (wave == who) {
#pragma unroll
      for (int i = 0; i < kJoinWaves; ++i) {
        float f[4];
        Row<float, 4>::load(&sums[i][lane * 4], f);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] += f[v];
      }
    }
  }
  if (run < 0 || c >= C) return;
  O *row = out + (int64_t)run * C;
  Cells<O, 4> old;
  if (add) old.load(row, c, C);
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] = add ? fmaf(acc[v], scale, (float)old.v[v]) : acc[v] * scale;
  store_cells<O, 4>(row, c, C, acc);
}

// Two lists of pairs (one where one workgroup sorts), the sort's table, the sums of parts of runs
struct EmbedSpace {
  size_t pairs1, pairs, table, parts, bytes;
  EmbedSpace(int64_t T, int64_t V, int64_t C) {
    const SortPlan p = sort_plan(T, V);
    const size_t list = ((size_t)T * sizeof(Pair) + 15) / 16 * 16;
    pairs = 0;
    pairs1 = list;
    table = pairs1 + (p.chunks > 1 ? list : 0);
    parts = table + (p.chunks > 1 ? (size_t)p.chunks * (size_t)(4 << p.bits) : 0);
    parts = (parts + 15) / 16 * 16;
    bytes = parts + (size_t)run_chunks(T, C) * 2 * (size_t)part_pitch(C) * 4;
  }
};
size_t embedding_backward_workspace(int64_t T, int64_t V, int64_t C) { return T == 0 || C == 0 ? 0 : EmbedSpace(T, V, C).bytes; }

template <typename T, typename O> static hipError_t runs_to(const EmbedArgs &a, const EmbedSpace &sp, hipStream_t s) {
  constexpr int N = 16 / (int)sizeof(T);
  char *ws = (char *)a.workspace;
  const Pair *pairs = (const Pair *)(ws + sp.pairs);
  float *parts = (float *)(ws + sp.parts);
  const int64_t S = run_chunk(a.T, a.C), chunks = run_chunks(a.T, a.C), pitch = part_pitch(a.C);
  const LaneGrid g(chunks, (a.C + N - 1) / N);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, g.grid, dim3(256), 0, s, pairs, a.T, S, chunks, (const T *)a.x, a.ld, a.C, a.scale, g.lp, (O *)a.out,
                       parts, pitch);
  };
  if (a.accumulate) g.is_short ? go(embed_runs_kernel<T, O, true, true>) : go(embed_runs_kernel<T, O, true, false>);
  else g.is_short ? go(embed_runs_kernel<T, O, false, true>) : go(embed_runs_kernel<T, O, false, false>);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks < 2) return e;
  const dim3 grid((unsigned)((chunks + kJoinWaves - 1) / kJoinWaves), (unsigned)((a.C + 255) / 256));
  hipLaunchKernelGGL((embed_join_kernel<O>), grid, dim3(kJoinWaves * 64), 0, s, pairs, a.T, S, chunks, a.C, a.scale,
                     a.accumulate != 0, (O *)a.out, parts, pitch);
  return hipGetLastError();
}
template <typename T> static hipError_t runs_t(const EmbedArgs &a, const EmbedSpace &sp, hipStream_t s) {
  switch (a.out_dtype) {
    case NSG_F16: return runs_to<T, _Float16>(a, sp, s);
    case NSG_BF16: return runs_to<T, __bf16>(a, sp, s);
    default: return runs_to<T, float>(a, sp, s);
  }
}

hipError_t launch_embedding_backward(const EmbedArgs &a, hipStream_t s) {
  const int64_t bytes = a.accumulate ? 0 : a.V * a.C * (a.out_dtype == NSG_F32 ? 4 : 2);
  if (a.T == 0) {
    const Clear c = clear_share(a.out, bytes, 0, 1);
    if (c.blocks > 0) hipLaunchKernelGGL(embed_clear_kernel, dim3((unsigned)c.blocks), dim3(1024), 0, s, c);
    return hipGetLastError();
  }
  const EmbedSpace sp(a.T, a.V, a.C);
  const SortPlan p = sort_plan(a.T, a.V);
  char *ws = (char *)a.workspace;
  Pair *pairs1 = (Pair *)(ws + sp.pairs1), *pairs = (Pair *)(ws + sp.pairs);
  int32_t *table = (int32_t *)(ws + sp.table);
  SortInput in{a.ids, a.wide, a.V, nullptr};
  hipError_t e = hipSuccess;
  if (p.chunks == 1) {
    const Clear c = clear_share(a.out, bytes, 0, 1);
    hipLaunchKernelGGL(embed_sort_kernel, dim3(1 + (unsigned)c.blocks), dim3(kSortThreads), 0, s, in, a.T, p.chunk, p.digits,
                       p.bits, pairs, c);
    e = hipGetLastError();
  } else {
    for (int d = 0; d < p.digits && e == hipSuccess; ++d) {
      const bool last = d == p.digits - 1;
      Pair *to = last ? pairs : pairs1;
      Clear c = clear_share(a.out, bytes, 2 * d, 2 * p.digits);
      hipLaunchKernelGGL(embed_count_kernel, dim3((unsigned)(p.chunks + c.blocks)), dim3(kSortThreads), 0, s, in, a.T, p.chunk,
                         d * p.bits, p.bits, table, p.chunks, c);
      e = hipGetLastError();
      if (e != hipSuccess) break;
      c = clear_share(a.out, bytes, 2 * d + 1, 2 * p.digits);
      if (p.chunk <= kSortChunk)
        hipLaunchKernelGGL(embed_place_kernel<kSortKept>, dim3((unsigned)(p.chunks + c.blocks)), dim3(kSortThreads), 0, s, in, a.T,
                           p.chunk, p.chunks, d * p.bits, p.bits, (const int32_t *)table, to, c);
      else
        hipLaunchKernelGGL(embed_place_kernel<0>, dim3((unsigned)(p.chunks + c.blocks)), dim3(kSortThreads), 0, s, in, a.T, p.chunk,
                           p.chunks, d * p.bits, p.bits, (const int32_t *)table, to, c);
      e = hipGetLastError();
      in.pairs = pairs1;
    }
  }
  if (e != hipSuccess) return e;
  switch (a.x_dtype) {
    case NSG_F16: return runs_t<_Float16>(a, sp, s);
    case NSG_BF16: return runs_t<__bf16>(a, sp, s);
    default: return runs_t<float>(a, sp, s);
  }
}

}  // namespace nsg
