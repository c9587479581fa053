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
// the other way round); launches for a few tokens.
#include <type_traits>

#include "mm_device.hpp"
#include "mm_elements_dev.hpp"
#include "mm_ops_internal.hpp"

namespace mm {

namespace {

constexpr int kThreads = 256;
constexpr int kPlaceThreads = 1024;
constexpr int kMaxTopk = 64;
constexpr int kMost = 8;             // slots of a token that are in flight together

__device__ __forceinline__ int key_of(const SortArgs& a, int64_t r) {
  const int e = a.ids[r];
  if ((uint32_t)e >= (uint32_t)a.E) return a.E;
  if (a.active != nullptr && a.active[(uint32_t)r / (uint32_t)a.K] == 0) return a.E;   // (routes are below 2^30)
  return e;
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

// How a workgroup's threads share rows: `cx` of them (a power of two) go
// along a row, the others take further tokens.
struct Split {
  int cx, c, ty, sub;
};
__device__ __forceinline__ Split split_of(int64_t chunks) {
  int cx = 1;
  while (cx < kThreads && cx < chunks) cx <<= 1;
  return Split{cx, (int)threadIdx.x & (cx - 1), kThreads / cx, (int)threadIdx.x / cx};
}

}  // namespace

// A few routes: each workgroup finds the places of one token's routes by
// counting the routes before them, so that one launch does it all.
template <int V>
__global__ __launch_bounds__(kThreads) void k_sort_few(SortArgs a) {
  typedef typename Bytes<V>::type vec;
  __shared__ int32_t hist[1025], part[kThreads / 64], cnt[kThreads / 64][kMost], place[kMaxTopk];
  __shared__ uint8_t skip[kMaxTopk];
  const int tid = threadIdx.x, w = tid / 64, R = (int)a.R;
  const int64_t t = blockIdx.x;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int e = tid; e <= a.E; e += kThreads) hist[e] = 0;
    __syncthreads();
    for (int r = tid; r < R; r += kThreads) atomicAdd(&hist[key_of(a, r)], 1);
    __syncthreads();
    write_offsets<kThreads>(a, hist, part);
  }
  for (int k0 = 0; k0 < a.K; k0 += kMost) {
    const int r0 = (int)t * a.K + k0;
    int key[kMost], before[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) key[i] = k0 + i < a.K ? key_of(a, r0 + i) : -1, before[i] = 0;
    for (int r = tid; r < R; r += kThreads) {
      const int e = key_of(a, r);
#pragma unroll
      for (int i = 0; i < kMost; ++i) before[i] += e < key[i] || (e == key[i] && r < r0 + i) ? 1 : 0;
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int n = wave_sum(before[i]);
      if (tid % 64 == 0) cnt[w][i] = n;
    }
    __syncthreads();
    if (tid < kMost && k0 + tid < a.K) {
      int n = 0, mine = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 64; ++i) n += cnt[i][tid];
#pragma unroll
      for (int i = 0; i < kMost; ++i) mine = i == tid ? key[i] : mine;
      place[k0 + tid] = n;
      skip[k0 + tid] = mine == a.E;
      if (blockIdx.y == 0) {
        a.row_of_route[r0 + tid] = mine == a.E ? -1 : n;
        a.route_of_row[n] = mine == a.E ? -1 : r0 + tid;
      }
    }
    __syncthreads();
  }
  if (a.rows == nullptr) return;
  const int64_t chunks = a.row_bytes / V;
  for (int64_t c = (int64_t)blockIdx.y * kThreads + tid; c < chunks; c += (int64_t)gridDim.y * kThreads) {
    const vec v = *reinterpret_cast<const vec*>(a.x + t * a.row_bytes + c * V);
    const vec zero = {};
    for (int k = 0; k < a.K; ++k)
      *reinterpret_cast<vec*>(a.rows + (int64_t)place[k] * a.row_bytes + c * V) = skip[k] ? zero : v;
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

// rows[row_of_route[t][k]] = x[t]; the workgroup of token t also clears those of
// the rows t * K .. t * K + K - 1 that no route fills.
template <int V>
__global__ __launch_bounds__(kThreads) void k_sort_rows(SortArgs a) {
  typedef typename Bytes<V>::type vec;
  const int64_t chunks = a.row_bytes / V;
  const Split s = split_of(chunks);
  const int64_t kept = a.offsets[a.E];
  for (int64_t t = (int64_t)blockIdx.x * s.ty + s.sub; t < a.T; t += (int64_t)gridDim.x * s.ty) {
    const int32_t* to = a.row_of_route + t * a.K;
    for (int64_t c = s.c; c < chunks; c += s.cx) {
      const vec v = *reinterpret_cast<const vec*>(a.x + t * a.row_bytes + c * V);
      for (int k = 0; k < a.K; ++k) {
        const int64_t p = to[k];
        if (p >= 0 && p < a.R) *reinterpret_cast<vec*>(a.rows + p * a.row_bytes + c * V) = v;
      }
    }
    for (int64_t p = t * a.K > kept ? t * a.K : kept; p < (t + 1) * a.K; ++p)
      for (int64_t c = s.c; c < chunks; c += s.cx) *reinterpret_cast<vec*>(a.rows + p * a.row_bytes + c * V) = vec{};
  }
}

// y[t] = sum_k w[t][k] * rows[row_of_route[t][k]] in float32, in the order of k,
// eight rows in flight.
template <typename E, int N>
__global__ __launch_bounds__(kThreads) void k_combine_tokens(CombineTokensArgs a) {
  typedef Elems<E, N> el;
  const int64_t chunks = a.H / N;
  const Split s = split_of(chunks);
  const E* rows = static_cast<const E*>(a.rows);
  for (int64_t t = (int64_t)blockIdx.x * s.ty + s.sub; t < a.T; t += (int64_t)gridDim.x * s.ty) {
    int32_t p[kMost];
    float w[kMost];
    auto slots = [&](int k0) {
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        const bool in = k0 + i < a.K;
        p[i] = in ? a.row_of_route[t * a.K + k0 + i] : -1;
        w[i] = in && a.weights != nullptr ? a.weights[t * a.K + k0 + i] : 1.0f;
        if (p[i] >= a.R) p[i] = -1;
      }
    };
    if (a.K <= kMost) slots(0);
    for (int64_t c = s.c; c < chunks; c += s.cx) {
      float acc[N] = {};
      for (int k0 = 0; k0 < a.K; k0 += kMost) {
        if (a.K > kMost) slots(k0);
        float v[kMost][N];
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
#pragma unroll
          for (int j = 0; j < N; ++j) v[i][j] = 0.0f;
          if (p[i] >= 0) el::load(rows + p[i] * a.H + c * N, v[i]);
        }
        // a skipped slot adds nothing, whatever its weight
#pragma unroll
        for (int i = 0; i < kMost; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j) acc[j] = p[i] >= 0 ? fmaf(w[i], v[i][j], acc[j]) : acc[j];
      }
      el::store(static_cast<E*>(a.y) + t * a.H + c * N, acc);
    }
  }
}

// drows[p] = w * dy[t] and dw = <dy[t], rows[p]> for the token's rows p, eight
// slots at a time; 64 or 256 threads a token.  The sums' order is fixed.
template <typename E, int N, int PER>
__global__ __launch_bounds__(kThreads) void k_combine_backward(CombineTokensArgs a) {
  typedef Elems<E, N> el;
  constexpr int kTokens = kThreads / PER;
  __shared__ float red[kThreads / 64][kMost];
  const int64_t chunks = a.H / N;
  const int sub = threadIdx.x / PER, at = threadIdx.x % PER, w = threadIdx.x / 64, l = threadIdx.x % 64;
  const E *rows = static_cast<const E*>(a.rows), *dy = static_cast<const E*>(a.dy);
  E* drows = static_cast<E*>(a.drows);
  const int64_t kept = a.offsets[a.E];
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < a.T; t0 += (int64_t)gridDim.x * kTokens) {
    const int64_t t = t0 + sub;
    const bool live = t < a.T;
    const int32_t* from = a.row_of_route + t * a.K;
    for (int k0 = 0; k0 < a.K; k0 += kMost) {
      int32_t p[kMost];
      float wt[kMost], dot[kMost];
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        const int32_t q = live && k0 + i < a.K ? from[k0 + i] : -1;
        p[i] = q < a.R ? q : -1;
        wt[i] = p[i] >= 0 ? a.weights[t * a.K + k0 + i] : 0.0f;
        dot[i] = 0.0f;
      }
      for (int64_t c = at; live && c < chunks; c += PER) {
        float d[N];
        el::load(dy + t * a.H + c * N, d);
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          if (p[i] < 0) continue;
          if (a.dweights != nullptr) {
            float v[N];
            el::load(rows + p[i] * a.H + c * N, v);
#pragma unroll
            for (int j = 0; j < N; ++j) dot[i] = fmaf(d[j], v[j], dot[i]);
          }
          if (drows != nullptr) {
            float o[N];
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] = wt[i] * d[j];
            el::store(drows + p[i] * a.H + c * N, o);
          }
        }
      }
      if (a.dweights != nullptr) {
#pragma unroll
        for (int i = 0; i < kMost; ++i) dot[i] = wave_sum(dot[i]);
        if constexpr (PER > 64) {
          __syncthreads();             // (the last slots' sums have been read)
          if (l == 0) {
#pragma unroll
            for (int i = 0; i < kMost; ++i) red[w][i] = dot[i];
          }
          __syncthreads();
          if (at < kMost && live && k0 + at < a.K) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER / 64; ++i) sum += red[i][at];
            a.dweights[t * a.K + k0 + at] = sum;
          }
        } else {
          float mine = dot[0];
#pragma unroll
          for (int i = 1; i < kMost; ++i) mine = l == i ? dot[i] : mine;
          if (l < kMost && live && k0 + l < a.K) a.dweights[t * a.K + k0 + l] = mine;
        }
      }
    }
    if (drows != nullptr && live) {
      for (int64_t q = t * a.K > kept ? t * a.K : kept; q < (t + 1) * a.K; ++q)
        for (int64_t c = at; c < chunks; c += PER) {
          const float zero[N] = {};
          el::store(drows + q * a.H + c * N, zero);
        }
    }
  }
}

namespace {

// widest power of two up to 16 that divides a row
int vector_bytes(int64_t row_bytes) {
  const int64_t v = row_bytes & -row_bytes;
  return (int)(v < 16 ? v : 16);
}

int64_t tokens_a_group(int64_t chunks) {
  int64_t cx = 1;
  while (cx < kThreads && cx < chunks) cx <<= 1;
  return kThreads / cx;
}

unsigned grid_of(int64_t groups) { return (unsigned)(groups < (1 << 20) ? groups : (1 << 20)); }

template <int V>
hipError_t sort_rows(const SortArgs& a, hipStream_t s) {
  const int64_t ty = tokens_a_group(a.row_bytes / V);
  hipLaunchKernelGGL(k_sort_rows<V>, dim3(grid_of((a.T + ty - 1) / ty)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int V>
hipError_t sort_few(const SortArgs& a, hipStream_t s) {
  // a workgroup brings 4 KiB of a row at a time; up to 1024 of them
  const int64_t turns = a.rows == nullptr ? 1 : (a.row_bytes / V + kThreads - 1) / kThreads;
  const int64_t most = 1024 / a.T > 1 ? 1024 / a.T : 1;
  hipLaunchKernelGGL(k_sort_few<V>, dim3((unsigned)a.T, (unsigned)(turns < most ? turns : most)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename E, int N>
hipError_t combine(const CombineTokensArgs& a, hipStream_t s) {
  const int64_t ty = tokens_a_group(a.H / N);
  hipLaunchKernelGGL((k_combine_tokens<E, N>), dim3(grid_of((a.T + ty - 1) / ty)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename E, int N>
hipError_t combine_backward(const CombineTokensArgs& a, hipStream_t s) {
  if (a.H / N <= 64)
    hipLaunchKernelGGL((k_combine_backward<E, N, 64>), dim3(grid_of((a.T + 3) / 4)), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_combine_backward<E, N, kThreads>), dim3(grid_of(a.T)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

// f(E, N) for the element type and the widest vector that divides a row
template <typename F>
hipError_t for_elements(int element, int64_t H, const F& f) {
  const int v = vector_bytes(H * (element == MM_ELEMENT_F32 ? 4 : 2));
  if (element == MM_ELEMENT_F32) {
    if (v == 16) return f(float{}, std::integral_constant<int, 4>{});
    if (v == 8) return f(float{}, std::integral_constant<int, 2>{});
    return f(float{}, std::integral_constant<int, 1>{});
  }
  auto half = [&](auto e) {
    if (v == 16) return f(e, std::integral_constant<int, 8>{});
    if (v == 8) return f(e, std::integral_constant<int, 4>{});
    if (v == 4) return f(e, std::integral_constant<int, 2>{});
    return f(e, std::integral_constant<int, 1>{});
  };
  return element == MM_ELEMENT_BF16 ? half(__bf16{}) : half(_Float16{});
}

}  // namespace

int sort_chunk(int64_t routes) {
  // at most 512 chunks of whole turns of k_sort_place
  const int64_t even = (routes + 511) / 512;
  return (int)((even + kPlaceThreads - 1) / kPlaceThreads * kPlaceThreads);
}

bool sort_in_one(int64_t routes) { return routes <= 8192; }

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
  return for_elements(a.element, a.H, [&](auto e, auto n) { return combine<decltype(e), n.value>(a, s); });
}

hipError_t launch_combine_backward(const CombineTokensArgs& a, hipStream_t s) {
  return for_elements(a.element, a.H, [&](auto e, auto n) { return combine_backward<decltype(e), n.value>(a, s); });
}

}  // namespace mm
