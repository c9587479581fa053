// Token rows sorted by expert, and back:
//
//   key(r) = the expert of route r = t * K + k, or E where the route is skipped
//   rows in the order of (key, r); place(r) = #{s : (key(s), s) < (key(r), r)}
//   rows[place(r)] = x[t],  zeros where key(r) = E
//   y[t] = sum_k w[t][k] * rows[place(t, k)]
// and y's gradient: drows[place(r)] = w[r] * dy[t], dw[r] = <dy[t], rows[place(r)]>.
// The order is a stable counting sort, so every result has one value.
//
// Bound: HBM for the rows (a token's row is read once and written K times, or
// the other way round); launches for a few tokens.  At 16384 tokens of 7168 bf16
// with 8 of 256 experts each: the order 15 us, rows written 427 to 431 us (4.9 TB/s,
// as a copy), read and summed 344 to 362 (5.8 to 6.1), read and written with both
// gradients 775 to 809 (4.9 to 5.1 for 3.99 GB): medians of several runs, which differ
// by where the buffers lie (single launches from 372, 334 and 662); one token 4.3.
#include <type_traits>

#include "mm_device.hpp"
#include "mm_elements_dev.hpp"
#include "mm_ops_internal.hpp"

namespace mm {

namespace {

constexpr int kThreads = 256;
constexpr int kPlaceThreads = 1024;
constexpr int kMaxThreads = 512;     // of k_combine_backward
constexpr int kMaxTopk = 64;
constexpr int kMost = 8;             // slots of a token that are in flight together
// Most routes of the single launch, where every workgroup reads all of them once
// for each eight slots of its token.  us, one launch / three, rows of 7168 bf16,
// top-8: 1 token 4.0 / 10, 64 tokens 5.4 / 12, 256 tokens 11 / 16, 512 tokens 20 / 22,
// 1024 tokens 36 / 34; top-4 of 4096: 2048 tokens 28 / 23; top-64 of 1024: 128 tokens 85 / 21.
// The bound leaves the number of workgroups out; within it that cost 1 us at
// most where measured (one behind the other, rows of 7168 bf16): top-1 1024 tokens 8.3 / 14, 2048 tokens 15 / 20,
// 4096 tokens 31 / 30; top-2 1024 tokens 11 / 17, 2048 tokens 21 / 25; top-4 1024 tokens 19 / 23;
// top-8 512 tokens 20 / 23.
constexpr int64_t kFewRoutes = 4096;

__device__ __forceinline__ int key_of(const SortArgs& a, int64_t r) {
  const int e = a.ids[r];
  const bool on = a.active == nullptr || a.active[(uint32_t)r / (uint32_t)a.K] != 0;   // (routes are below 2^30)
  return on && (uint32_t)e < (uint32_t)a.E ? e : a.E;
}

// Exclusive prefix of v over the workgroup's threads; `all` gets the sum.
// Every thread takes part; `part` holds one number a wave.
template <int NT>
__device__ __forceinline__ int32_t block_prefix(int32_t v, int32_t* part, int32_t& all) {
  const int l = threadIdx.x % 64, w = threadIdx.x / 64;
  int32_t p = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(p, d, 64);
    if (l >= d) p += o;
  }
  __syncthreads();                   // (part may still be read from the last call)
  if (l == 63) part[w] = p;
  __syncthreads();
  int32_t before = 0;
  all = 0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) {
    before += i < w ? part[i] : 0;
    all += part[i];
  }
  return before + p - v;
}

// counts and offsets from the experts' totals (tot[0 .. E], tot[E] the skipped)
template <int NT>
__device__ void write_offsets(const SortArgs& a, const int32_t* tot, int32_t* part) {
  int32_t base = 0;
  for (int e0 = 0; e0 <= a.E; e0 += NT) {
    const int e = e0 + (int)threadIdx.x;
    const int32_t v = e < a.E ? tot[e] : 0;
    int32_t all;
    const int32_t p = base + block_prefix<NT>(v, part, all);
    if (e < a.E) a.counts[e] = v;
    if (e <= a.E) a.offsets[e] = p;
    base += all;
  }
}

// How a workgroup's threads share narrow rows: `cx` of them (a power of two)
// go along a row, the others take further tokens.
struct Split {
  int cx, c, ty, sub;
};
__device__ __forceinline__ Split split_of(int64_t chunks) {
  int cx = 1;
  while (cx < 64 && cx < chunks) cx <<= 1;
  return Split{cx, (int)threadIdx.x & (cx - 1), kThreads / cx, (int)threadIdx.x / cx};
}

// A value of an array that no kernel writes while this one runs.  UNIFORM: the
// same address in all lanes, through the scalar unit.
template <bool UNIFORM, typename T>
__device__ __forceinline__ T slot(const T* p) {
  if constexpr (UNIFORM) return *(const __attribute__((address_space(4))) T*)reinterpret_cast<uintptr_t>(p);
  return *p;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// f(t, c): every vector c of every token t, by the whole grid.  WIDE (rows of 64
// vectors and more): a wave takes 64 neighbours of one token.
template <bool WIDE, typename F>
__device__ __forceinline__ void for_vectors(int64_t tokens, int64_t chunks, const F& f) {
  if constexpr (WIDE) {
    const uint32_t per = (uint32_t)((chunks + 63) / 64);          // (a tensor has fewer than 2^32 such pieces)
    const uint32_t total = (uint32_t)tokens * per, step = gridDim.x * (kThreads / 64);
    for (uint32_t u = blockIdx.x * (kThreads / 64) + (uint32_t)uniform(threadIdx.x / 64); u < total; u += step) {
      const int64_t c = (int64_t)(u % per) * 64 + threadIdx.x % 64;
      if (c < chunks) f((int64_t)(u / per), c);
    }
  } else {
    const Split s = split_of(chunks);
    for (int64_t t = (int64_t)blockIdx.x * s.ty + s.sub; t < tokens; t += (int64_t)gridDim.x * s.ty)
      for (int64_t c = s.c; c < chunks; c += s.cx) f(t, c);
  }
}

// what is read or written once
template <typename V>
__device__ __forceinline__ V stream_in(const V* p) { return __builtin_nontemporal_load(p); }
template <typename V>
__device__ __forceinline__ void stream_out(void* p, const V& v) { __builtin_nontemporal_store(v, static_cast<V*>(p)); }

}  // namespace

// A few routes: each workgroup finds the places of one token's routes by
// counting the routes before them, so that one launch does it all; one
// workgroup more counts the experts' routes.
template <int V>
__global__ __launch_bounds__(kThreads) void k_sort_few(SortArgs a) {
  typedef typename Bytes<V>::type vec;
  constexpr int kWaves = kThreads / 64;
  __shared__ int32_t cnt[kWaves][kMost], place[kMaxTopk];
  const int tid = threadIdx.x, w = tid / 64, R = (int)a.R;
  const int64_t t = blockIdx.x;
  // the order of (key, route): routes are below 2^13 (kFewRoutes), keys at most 2^10
  auto rank_of = [&](int r) { return (uint32_t)key_of(a, r) << 13 | (uint32_t)r; };
  if (t == a.T) {
    __shared__ int32_t hist[1025], part[kWaves];
    if (blockIdx.y > 0) return;
    for (int e = tid; e <= a.E; e += kThreads) hist[e] = 0;
    __syncthreads();
    for (int r = tid; r < R; r += kThreads) atomicAdd(&hist[key_of(a, r)], 1);
    __syncthreads();
    write_offsets<kThreads>(a, hist, part);
    return;
  }
  for (int k0 = 0; k0 < a.K; k0 += kMost) {
    const int r0 = (int)t * a.K + k0;
    uint32_t mine[kMost];
    int before[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) mine[i] = k0 + i < a.K ? rank_of(r0 + i) : 0, before[i] = 0;
    for (int j = 0; j < R; j += kThreads) {
      const uint32_t other = j + tid < R ? rank_of(j + tid) : ~0u;
#pragma unroll
      for (int i = 0; i < kMost; ++i) before[i] += __popcll(ballot(other < mine[i]));
    }
    if (tid % 64 == 0) {
#pragma unroll
      for (int i = 0; i < kMost; ++i) cnt[w][i] = before[i];
    }
    __syncthreads();
    if (tid < kMost && k0 + tid < a.K) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) n += cnt[i][tid];
      const bool skip = key_of(a, r0 + tid) == a.E;
      place[k0 + tid] = skip ? ~n : n;
      if (blockIdx.y == 0) {
        a.row_of_route[r0 + tid] = skip ? -1 : n;
        a.route_of_row[n] = skip ? -1 : r0 + tid;
      }
    }
    __syncthreads();
  }
  if (a.rows == nullptr) return;
  const int64_t chunks = a.row_bytes / V;
  for (int64_t c = (int64_t)blockIdx.y * kThreads + tid; c < chunks; c += (int64_t)gridDim.y * kThreads) {
    const vec v = *reinterpret_cast<const vec*>(a.x + t * a.row_bytes + c * V);
    for (int k = 0; k < a.K; ++k) {
      const int p = place[k];
      *reinterpret_cast<vec*>(a.rows + (int64_t)(p < 0 ? ~p : p) * a.row_bytes + c * V) = p < 0 ? vec{} : v;
    }
  }
}

// Many routes, first launch: experts' routes of each chunk.
__global__ __launch_bounds__(kThreads) void k_sort_count(SortArgs a) {
  __shared__ int32_t hist[1025];
  for (int e = threadIdx.x; e <= a.E; e += kThreads) hist[e] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * a.chunk, hi = lo + a.chunk < a.R ? lo + a.chunk : a.R;
  for (int64_t r = lo + threadIdx.x; r < hi; r += kThreads) atomicAdd(&hist[key_of(a, r)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kThreads) a.hist[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// Second launch: where the chunk's first route of each expert goes, from all
// chunks' counts, then the places of its routes, 1024 at a time in order: the
// routes of an expert in a wave by comparing keys bit by bit over the wave.
__global__ __launch_bounds__(kPlaceThreads) void k_sort_place(SortArgs a) {
  constexpr int W = kPlaceThreads / 64;
  extern __shared__ int32_t dyn[];
  __shared__ int32_t part[W];
  const int E1 = a.E + 1, tid = threadIdx.x, l = tid % 64, w = tid / 64;
  int32_t *base = dyn, *tot = dyn + E1;                               // [E1] each
  uint16_t* of_wave = reinterpret_cast<uint16_t*>(dyn + 2 * E1);      // [W][E1] routes of a wave, at most 64
  for (int e = tid; e < 2 * E1; e += kPlaceThreads) dyn[e] = 0;
  __syncthreads();
  // threads share (expert, part of the chunks)
  int groups = 1;
  while (groups < W && groups * 2 * a.E <= kPlaceThreads) groups *= 2;
  const int per = kPlaceThreads / groups, g = tid / per;
  for (int e = tid % per; e < a.E; e += per) {
    int32_t pre = 0, all = 0;
#pragma unroll 8
    for (int c = g; c < a.chunks; c += groups) {
      const int32_t v = a.hist[(int64_t)c * a.E + e];
      all += v;
      pre += c < (int)blockIdx.x ? v : 0;
    }
    if (pre) atomicAdd(&base[e], pre);
    if (all) atomicAdd(&tot[e], all);
  }
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * a.chunk, hi = lo + a.chunk < a.R ? lo + a.chunk : a.R;
  int32_t kept = 0, earlier = 0;         // kept routes of all chunks, and of those before this one
  for (int e0 = 0; e0 < a.E; e0 += kPlaceThreads) {
    const int e = e0 + tid;
    const int32_t pre = e < a.E ? base[e] : 0;
    int32_t all;
    block_prefix<kPlaceThreads>(pre, part, all);
    earlier += all;
    const int32_t p = kept + block_prefix<kPlaceThreads>(e < a.E ? tot[e] : 0, part, all);
    if (e < a.E) base[e] = pre + p;
    kept += all;
  }
  if (tid == 0) base[a.E] = kept + (int32_t)lo - earlier;
  if (blockIdx.x == 0) write_offsets<kPlaceThreads>(a, tot, part);
  int bits = 1;
  while ((1 << bits) <= a.E) ++bits;
  for (int64_t r0 = lo; r0 < hi; r0 += kPlaceThreads) {
    for (int e = tid; e < W * E1; e += kPlaceThreads) of_wave[e] = 0;
    __syncthreads();
    const int64_t r = r0 + tid;
    const bool in = r < hi;
    const int key = in ? key_of(a, r) : 0;
    uint64_t same = ballot(in);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? m : ~m;
    }
    const int rank = __popcll(same & lanemask_lt());
    if (in && rank == 0) of_wave[w * E1 + key] = (uint16_t)__popcll(same);
    __syncthreads();
    if (in) {
      int32_t p = base[key] + rank;
#pragma unroll
      for (int i = 0; i < W; ++i) p += i < w ? of_wave[i * E1 + key] : 0;
      a.row_of_route[r] = key == a.E ? -1 : p;
      a.route_of_row[p] = key == a.E ? -1 : (int32_t)r;
    }
    __syncthreads();
    for (int e = tid; e < E1; e += kPlaceThreads) {
      int32_t n = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) n += of_wave[i * E1 + e];
      base[e] += n;
    }
    __syncthreads();
  }
}

// rows[row_of_route[t][k]] = x[t]; who brings token t also clears those of the
// rows t * K .. t * K + K - 1 that no route fills.  WIDE: a workgroup a token, or
// several where there are few (16384 tokens of 7168 bf16 to 8 experts each: a
// wave per 64 vectors instead, as k_combine_tokens has it, 2% more).
template <int V, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_sort_rows(SortArgs a) {
  typedef typename Bytes<V>::type vec;
  const int64_t kept = slot<true>(a.offsets + a.E), chunks = a.row_bytes / V;
  auto one = [&](int64_t t, int64_t c) {
    const vec v = *reinterpret_cast<const vec*>(a.x + t * a.row_bytes + c * V);
    for (int k = 0; k < a.K; ++k) {
      const int64_t p = slot<WIDE>(a.row_of_route + t * a.K + k);
      if (p >= 0 && p < a.R) stream_out(a.rows + p * a.row_bytes + c * V, v);
    }
    for (int64_t p = t * a.K > kept ? t * a.K : kept; p < (t + 1) * a.K; ++p)
      stream_out(a.rows + p * a.row_bytes + c * V, vec{});
  };
  if constexpr (WIDE) {
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x)
      for (int64_t c = (int64_t)blockIdx.y * kThreads + threadIdx.x; c < chunks; c += (int64_t)gridDim.y * kThreads) one(t, c);
  } else {
    for_vectors<false>(a.T, chunks, one);
  }
}

namespace {

// Slots k0 .. k0 + SLOTS - 1 of token t: their rows, -1 for one that is skipped or
// past K, and their weights.  No load is under a condition: the compiler would
// wait for the loads in flight at each.
template <int SLOTS, bool UNIFORM>
__device__ __forceinline__ void load_slots(const CombineTokensArgs& a, int64_t t, int k0, int64_t (&p)[SLOTS], float (&w)[SLOTS]) {
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int64_t at = t * a.K + (k0 + i < a.K ? k0 + i : k0);
    p[i] = slot<UNIFORM>(a.row_of_route + at);
    w[i] = slot<UNIFORM>(a.weights != nullptr ? a.weights + at : reinterpret_cast<const float*>(a.row_of_route + at));
  }
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    if (a.weights == nullptr) w[i] = 1.0f;
    if (k0 + i >= a.K || p[i] >= a.R) p[i] = -1;
  }
}

}  // namespace

// y[t] = sum_k w[t][k] * rows[row_of_route[t][k]] in float32, in the order of k,
// SLOTS rows in flight.  A skipped slot reads row 0 and adds nothing, whatever
// its weight.  WIDE: a wave takes 64 neighbouring vectors of a token, its rows'
// places and weights come through the scalar unit (a workgroup a token, places by
// lane, 478 us in place of 344 at 16384 x 8 rows of 7168 bf16).
template <typename E, int N, int SLOTS, bool WIDE>
__global__ __launch_bounds__(kThreads) void k_combine_tokens(CombineTokensArgs a) {
  typedef Elems<E, N> el;
  const E* rows = static_cast<const E*>(a.rows);
  for_vectors<WIDE>(a.T, a.H / N, [&](int64_t t, int64_t c) {
    float acc[N] = {};
    for (int k0 = 0; k0 < a.K; k0 += SLOTS) {
      int64_t p[SLOTS];
      float w[SLOTS];
      typename el::vec v[SLOTS];
      load_slots<SLOTS, WIDE>(a, t, k0, p, w);
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) v[i] = stream_in(reinterpret_cast<const typename el::vec*>(rows + (p[i] < 0 ? 0 : p[i]) * a.H + c * N));
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        float f[N];
        el::unpack(v[i], f);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = p[i] < 0 ? acc[j] : fmaf(w[i], f[j], acc[j]);
      }
    }
    el::store(static_cast<E*>(a.y) + t * a.H + c * N, acc);
  });
}

// drows[p] = w * dy[t] and dw = <dy[t], rows[p]> for the token's rows p, SLOTS at
// a time.  A token has a wave, or (WIDE) a workgroup whose size the launch fits
// to the row.  The sums' order is fixed.
template <typename E, int N, int SLOTS, bool WIDE>
__global__ __launch_bounds__(kMaxThreads) void k_combine_backward(CombineTokensArgs a) {
  typedef Elems<E, N> el;
  typedef typename el::vec vec;
  __shared__ float red[kMaxThreads / 64][SLOTS];
  const int64_t chunks = a.H / N;
  const int waves = blockDim.x / 64, w = uniform(threadIdx.x / 64), l = threadIdx.x % 64;
  const int at = WIDE ? threadIdx.x : l, per = WIDE ? blockDim.x : 64;
  const E *rows = static_cast<const E*>(a.rows), *dy = static_cast<const E*>(a.dy);
  E* drows = static_cast<E*>(a.drows);
  const int64_t kept = slot<true>(a.offsets + a.E);
  const int64_t step = WIDE ? gridDim.x : (int64_t)gridDim.x * waves;
  for (int64_t t = WIDE ? blockIdx.x : (int64_t)blockIdx.x * waves + w; t < a.T; t += step) {
    for (int k0 = 0; k0 < a.K; k0 += SLOTS) {
      int64_t p[SLOTS];
      float wt[SLOTS], dot[SLOTS];
      load_slots<SLOTS, true>(a, t, k0, p, wt);
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) dot[i] = 0.0f;
      for (int64_t c = at; c < chunks; c += per) {
        float d[N];
        vec v[SLOTS];
        const vec raw = *reinterpret_cast<const vec*>(dy + t * a.H + c * N);
        if (a.dweights != nullptr) {
#pragma unroll
          for (int i = 0; i < SLOTS; ++i) v[i] = stream_in(reinterpret_cast<const vec*>(rows + (p[i] < 0 ? 0 : p[i]) * a.H + c * N));
        }
        el::unpack(raw, d);
        if (drows != nullptr) {
#pragma unroll
          for (int i = 0; i < SLOTS; ++i) {
            float o[N];
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] = wt[i] * d[j];
            if (p[i] >= 0) stream_out(drows + p[i] * a.H + c * N, el::pack(o));
          }
        }
        if (a.dweights != nullptr) {
#pragma unroll
          for (int i = 0; i < SLOTS; ++i) {
            float f[N];
            el::unpack(v[i], f);
#pragma unroll
            for (int j = 0; j < N; ++j) dot[i] = fmaf(d[j], f[j], dot[i]);
          }
        }
      }
      if (a.dweights != nullptr) {
        float mine = 0.0f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
          const float sum = p[i] < 0 ? 0.0f : wave_sum(dot[i]);
          mine = l == i ? sum : mine;
        }
        if constexpr (WIDE) {
          __syncthreads();             // (the last slots' sums have been read)
          if (l < SLOTS) red[w][l] = mine;
          __syncthreads();
          if (w == 0 && l < SLOTS) {
            mine = 0.0f;
            for (int i = 0; i < waves; ++i) mine += red[i][l];
          }
        }
        if ((!WIDE || w == 0) && l < SLOTS && k0 + l < a.K) a.dweights[t * a.K + k0 + l] = mine;
      }
    }
    if (drows != nullptr) {
      for (int64_t q = t * a.K > kept ? t * a.K : kept; q < (t + 1) * a.K; ++q)
        for (int64_t c = at; c < chunks; c += per) stream_out(drows + q * a.H + c * N, vec{});
    }
  }
}

namespace {

// widest power of two up to 16 that divides a row
int vector_bytes(int64_t row_bytes) {
  const int64_t v = row_bytes & -row_bytes;
  return (int)(v < 16 ? v : 16);
}

// workgroups of for_vectors
bool is_wide(int64_t chunks) { return chunks >= 64; }
unsigned vector_grid(int64_t tokens, int64_t chunks) {
  int64_t cx = 1;
  while (cx < 64 && cx < chunks) cx <<= 1;
  const int64_t pieces = is_wide(chunks) ? tokens * ((chunks + 63) / 64) * 64 : tokens * cx;
  const int64_t n = (pieces + kThreads - 1) / kThreads;
  return (unsigned)(n < (1 << 20) ? n : (1 << 20));
}

// a workgroup brings 256 vectors of a row at a time; few tokens' rows are shared by several, up to 1024 in all
unsigned slices_of(int64_t chunks, int64_t tokens) {
  const int64_t turns = (chunks + kThreads - 1) / kThreads, most = 1024 / tokens > 1 ? 1024 / tokens : 1;
  return (unsigned)(turns < most ? turns : most);
}

template <int V>
hipError_t sort_rows(const SortArgs& a, hipStream_t s) {
  const int64_t chunks = a.row_bytes / V, most = 1 << 20;
  if (is_wide(chunks))
    hipLaunchKernelGGL((k_sort_rows<V, true>), dim3((unsigned)(a.T < most ? a.T : most), slices_of(chunks, a.T)), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_sort_rows<V, false>), dim3(vector_grid(a.T, chunks)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int V>
hipError_t sort_few(const SortArgs& a, hipStream_t s) {
  const unsigned slices = a.rows == nullptr ? 1 : slices_of(a.row_bytes / V, a.T);
  hipLaunchKernelGGL(k_sort_few<V>, dim3((unsigned)(a.T + 1), slices), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename E, int N, int SLOTS>
hipError_t combine(const CombineTokensArgs& a, hipStream_t s) {
  const int64_t chunks = a.H / N;
  const dim3 grid(vector_grid(a.T, chunks));
  if (is_wide(chunks)) hipLaunchKernelGGL((k_combine_tokens<E, N, SLOTS, true>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_combine_tokens<E, N, SLOTS, false>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename E, int N, int SLOTS>
hipError_t combine_backward(const CombineTokensArgs& a, hipStream_t s) {
  const int64_t chunks = a.H / N, most = 1 << 20;
  if (chunks <= 64) {
    const int64_t n = (a.T + 3) / 4;
    hipLaunchKernelGGL((k_combine_backward<E, N, SLOTS, false>), dim3((unsigned)(n < most ? n : most)), dim3(256), 0, s, a);
  } else {
    // the fewest turns along a row, and for them the fewest waves
    const int64_t turns = (chunks + kMaxThreads - 1) / kMaxThreads, threads = ((chunks + turns - 1) / turns + 63) / 64 * 64;
    hipLaunchKernelGGL((k_combine_backward<E, N, SLOTS, true>), dim3((unsigned)(a.T < most ? a.T : most)), dim3((unsigned)threads), 0, s, a);
  }
  return hipGetLastError();
}

// f(E, N, SLOTS) for the element type, the widest vector that divides a row and
// the slots of a token that are in flight together
template <typename F>
hipError_t for_elements(const CombineTokensArgs& a, const F& f) {
  const int v = vector_bytes(a.H * (a.element == MM_ELEMENT_F32 ? 4 : 2));
  auto slots = [&](auto e, auto n) {
    return a.K > 4 ? f(e, n, std::integral_constant<int, kMost>{}) : f(e, n, std::integral_constant<int, 4>{});
  };
  if (a.element == MM_ELEMENT_F32) {
    if (v == 16) return slots(float{}, std::integral_constant<int, 4>{});
    if (v == 8) return slots(float{}, std::integral_constant<int, 2>{});
    return slots(float{}, std::integral_constant<int, 1>{});
  }
  auto half = [&](auto e) {
    if (v == 16) return slots(e, std::integral_constant<int, 8>{});
    if (v == 8) return slots(e, std::integral_constant<int, 4>{});
    if (v == 4) return slots(e, std::integral_constant<int, 2>{});
    return slots(e, std::integral_constant<int, 1>{});
  };
  return a.element == MM_ELEMENT_BF16 ? half(__bf16{}) : half(_Float16{});
}

}  // namespace

int sort_chunk(int64_t routes) {
  // at most 512 chunks of whole turns of k_sort_place
  const int64_t even = (routes + 511) / 512;
  return (int)((even + kPlaceThreads - 1) / kPlaceThreads * kPlaceThreads);
}

bool sort_in_one(int64_t routes, int64_t topk) { return routes * ((topk + kMost - 1) / kMost) <= kFewRoutes; }

hipError_t launch_sort_order(const SortArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_sort_count, dim3((unsigned)a.chunks), dim3(kThreads), 0, s, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const size_t lds = (size_t)(a.E + 1) * (2 * 4 + kPlaceThreads / 64 * 2);
  hipLaunchKernelGGL(k_sort_place, dim3((unsigned)a.chunks), dim3(kPlaceThreads), lds, s, a);
  return hipGetLastError();
}

hipError_t launch_sort_few(const SortArgs& a, hipStream_t s) {
  switch (vector_bytes(a.row_bytes)) {
    case 16: return sort_few<16>(a, s);
    case 8: return sort_few<8>(a, s);
    case 4: return sort_few<4>(a, s);
    case 2: return sort_few<2>(a, s);
    default: return sort_few<1>(a, s);
  }
}

hipError_t launch_sort_rows(const SortArgs& a, hipStream_t s) {
  switch (vector_bytes(a.row_bytes)) {
    case 16: return sort_rows<16>(a, s);
    case 8: return sort_rows<8>(a, s);
    case 4: return sort_rows<4>(a, s);
    case 2: return sort_rows<2>(a, s);
    default: return sort_rows<1>(a, s);
  }
}

hipError_t launch_combine_tokens(const CombineTokensArgs& a, hipStream_t s) {
  return for_elements(a, [&](auto e, auto n, auto k) { return combine<decltype(e), n.value, k.value>(a, s); });
}

hipError_t launch_combine_backward(const CombineTokensArgs& a, hipStream_t s) {
  return for_elements(a, [&](auto e, auto n, auto k) { return combine_backward<decltype(e), n.value, k.value>(a, s); });
}

}  // namespace mm
