// Products of 8-bit integers with a float32 scale per row of x and per row
// (output channel) of w, dense or over groups of rows:
//
//   y[m][n] = float(sum_k q[m][k] * w[n][k]) * ws[n] * s[m]
//
// and the quantiser of the rows:
//   s[m] = max(max_k|x[m][k]| / 127, 1e-8),  q = round-half-even(x / s), in [-127, 127].
//
// The sums are exact (int32, K up to 131056), so tiles, slices of K and the
// number of rows have no part in a result.
#include <type_traits>

#include "mm_device.hpp"
#include "mm_elements_dev.hpp"
#include "mm_ops_internal.hpp"
#include "mm_tiles_dev.hpp"

namespace mm {

namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kStep = 128;           // K-values (bytes) of a row that a part of a stage holds
constexpr int kFewRows = 16;         // most rows that are streamed together
constexpr int kFewCols = 16;
// Most rows of a product that are streamed; us one behind the other, weights from HBM, streamed / tiles of 32 x 32:
// 4096 x 7168: 1 row 10.3 / 11.5, 4 rows 10.6 / 11.6, 8 rows 11.0 / 11.6 (another run: 16 rows 11.2 / 10.3, where 1 row
// took 8.4 / 10.1).  The rule goes by the rows alone, which suits that shape: the tiles are faster from one row on where
// K is short (7168 x 2048: 7.1 / 6.3, 8 rows 8.2 / 6.4), and from four on at 16384 x 4096 (18.6 / 19.2, 4 rows 19.6 / 19.2,
// 8 rows 21.1 / 19.2).
constexpr int kStreamRows = 8;
constexpr int kQuantThreads = 512;
constexpr uint32_t kOutside = 0x7fffff00u;   // an offset beyond every descriptor: arrives as zeros

// 16 x 16 outputs, 64 K-values: each lane supplies 16 bytes of its A row and B
// column (lane % 16); element i of lane l is C[4 * (l / 16) + i][l % 16].
__device__ __forceinline__ void mfma64(i32x4& c, const u32x4& a, const u32x4& b) {
  c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// four neighbouring columns n .. n + 3 of a row of y [..][N]
template <typename E>
__device__ __forceinline__ void put4(void* y, int N, int64_t row, int n, const float (&v)[4]) {
  E* p = static_cast<E*>(y) + row * N + n;
  if (N % 4 == 0) {
    if (n < N) Elems<E, 4>::store(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) p[i] = (E)v[i];
  }
}

// their scales, from a group's row (16-byte aligned where N % 4 is 0)
__device__ __forceinline__ void scales4(const float* p, int N, int n, float (&v)[4]) {
  if (N % 4 == 0) {
    Elems<float, 4>::load(p + (n < N ? n : 0), v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p[n + i < N ? n + i : N - 1];
  }
}

__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const uint8_t*>((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

// One tile: WM x WN waves of 16 * MT rows x 16 * NT columns; D stages of LDS,
// each P parts of 128 K-values, filled by LDS-DMA D - 1 stages ahead.  Weights
// are the MFMA's A operand, so a lane's four sums are four columns of one row.
// Bound, at 256 x 256: copies and LDS.  16384 x 4096 x 7168 runs at 2.2 to 2.5 POPS
// (a large library product at 2.36); its products without copies at 3.05, its
// copies alone take as long as at 2.84; LDS moves 192 KiB of operands and 64 of
// copies a stage, 2048 cycles for 2048 of products.
// SPREAD: copies that go out between two column tiles' products (0: all of a
// stage's before its first product).
template <typename E, int WM, int WN, int MT, int NT, int D, int P, int SPREAD>
__device__ __forceinline__ void int8_tile(const Int8Args& a, const TileAt& at, uint8_t* const (&slot)[D]) {
  constexpr int W = WM * WN, BM = 16 * MT * WM, BN = 16 * NT * WN, kPart = (BM + BN) * kStep;
  constexpr int kGroups = (BM + BN) / 8, kOfA = BM / 8, kCopies = P * kGroups / W;
  static_assert(kOfA % W == 0 && kGroups % W == 0 && W % 2 == 0, "a wave's copies are of one operand each");
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));   // nothing derived from it is kept across tiles
  // (the arguments' fields in registers: a tile of this size outgrows what the
  // compiler follows through the reference)
  const int K = uniform(a.K), N = uniform(a.N);
  const TileAt t = uniform_tile(at);
  const int w = uniform(tid / 64), l = tid % 64, r = l % 16, g = l / 16, wm = w % WM, wn = w / WM;
  const int KB = (K + kStep - 1) / kStep, stages = (KB + P - 1) / P;
  const int rows = t.rows, cols = N - t.n0 < BN ? N - t.n0 : BN;
  // One instruction moves 8 rows of 128 bytes, lane i to byte 16 * i; the chunk
  // at place p of row x is p ^ (x / 2 % 8), so that 16 rows read at one chunk
  // hit 16 different bank groups.  Rows past the last one, chunks past K and
  // stages past the end are beyond the descriptor: zeros without an access.
  const int chunk = (l % 8) ^ ((4 * (w % 2) + l / 16) % 8);
  const uint32_t voff = (uint32_t)(l / 8) * K + chunk * 16;
  const uint32_t vlast = chunk * 16 < K - (KB - 1) * kStep ? voff : kOutside;
  const uint8_t* ab = uniform_ptr(a.a + t.m0 * K);
  const uint8_t* bb = uniform_ptr(a.b + ((int64_t)t.group * N + t.n0) * K);
  auto copy = [&](int i, int s, uint8_t* to) __attribute__((always_inline)) {
    const int item = W * i, p = item / kGroups, grp = item % kGroups;      // (compile-time), + w
    const bool of_a = grp < kOfA;
    const int kb = s * P + p;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(of_a ? ab : bb), (short)0, kb < KB ? (of_a ? rows : cols) * K : 0, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(to + p * kPart + (grp + w) * 1024), 16,
                                             kb + 1 < KB ? voff : vlast, ((of_a ? grp : grp - kOfA) + w) * 8 * K + kb * kStep, 0, 0);
  };
  const int sw = (r / 2) % 8;
  const int o0 = (g ^ sw) * 16 + r * kStep, o1 = ((g + 4) ^ sw) * 16 + r * kStep;
  i32x4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
  auto turn = [&]() __attribute__((always_inline)) {
    // the stage's products stay before the wait: nothing else ties them to it
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) asm volatile("" : "+v"(acc[j][i]));
    __builtin_amdgcn_sched_barrier(0);
    stage_barrier<(D - 2) * kCopies>();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto stage = [&](int s, const uint8_t* from, uint8_t* to) __attribute__((always_inline)) {
    int next = 0;
    if constexpr (SPREAD == 0) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) copy(i, s + D - 1, to);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (P > 1 && s * P + p >= KB) break;
      const uint8_t *sa = from + p * kPart, *sb = sa + BM * kStep;
      // The first 64 K-values of all columns, then the other 64: one half's rows
      // are in registers while the other half's arrive, a few before each column.
      u32x4 af[2][MT], b[2];
      auto rows_of = [&](int h, int i) __attribute__((always_inline)) { af[h][i] = *reinterpret_cast<const u32x4*>(sa + (wm * MT + i) * 16 * kStep + (h ? o1 : o0)); };
      auto cols_of_half = [&](int at) __attribute__((always_inline)) {
        b[at % 2] = *reinterpret_cast<const u32x4*>(sb + (wn * NT + at % NT) * 16 * kStep + (at / NT ? o1 : o0));
      };
      cols_of_half(0);
#pragma unroll
      for (int i = 0; i < MT; ++i) rows_of(0, i);
#pragma unroll
      for (int at = 0; at < 2 * NT; ++at) {
        const int h = at / NT, j = at % NT;
        if (at + 1 < 2 * NT) cols_of_half(at + 1);
        if (h == 0) {
#pragma unroll
          for (int i = j * MT / NT; i < (j + 1) * MT / NT; ++i) rows_of(1, i);
        }
        if constexpr (SPREAD > 0) {
#pragma unroll
          for (int c = 0; c < SPREAD; ++c)
            if (next < kCopies) copy(next++, s + D - 1, to);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) mfma64(acc[j][i], b[at % 2], af[h][i]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    turn();
  };
#pragma unroll
  for (int u = 0; u < D - 1; ++u)
#pragma unroll
    for (int i = 0; i < kCopies; ++i) copy(i, u, slot[u]);
  turn();
  // (a break inside the loop would be a path on which the compiler sees a slot
  // filled one stage ago, and waits for it)
  int s = 0;
  for (; s + D <= stages; s += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) stage(s + u, slot[u], slot[(u + D - 1) % D]);
  }
#pragma unroll
  for (int u = 0; u < D - 1; ++u) {
    if (s + u >= stages) break;
    stage(s + u, slot[u], slot[(u + D - 1) % D]);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);              // no copy outlives the tile
  void* const y = a.y;
  const float *as = a.as + t.m0, *bs = a.bs + (int64_t)t.group * N;
  // all scales before the first store: a load behind stores waits for them too
  float ws[NT][4], sa[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) scales4(bs, N, t.n0 + (wn * NT + j) * 16 + 4 * g, ws[j]);
#pragma unroll
  for (int i = 0; i < MT; ++i) sa[i] = as[(wm * MT + i) * 16 + r < rows ? (wm * MT + i) * 16 + r : 0];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int row = (wm * MT + i) * 16 + r;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = (float)acc[j][i][k] * ws[j][k] * sa[i];
      if (row < rows) put4<E>(y, N, t.m0 + row, t.n0 + (wn * NT + j) * 16 + 4 * g, v);
    }
  }
  __syncthreads();      // the next tile of this workgroup writes the stages again
}

}  // namespace

// Products whose large tiles would leave most CUs without one: tiles of class c.
template <typename E, int C, int WM, int WN, int MT, int NT, int D>
__global__ __launch_bounds__(64 * WM * WN) void k_int8_ring(Int8Args a) {
  constexpr int kBytes = 16 * (MT * WM + NT * WN) * kStep * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kBytes], s1[kBytes], s2[D > 2 ? kBytes : 16], s3[D > 2 ? kBytes : 16];
  const int x = blockIdx.x % 8, step = gridDim.x / 8;
  const int64_t total = count_blocks(a, C) * ((a.N + cols_of(C) - 1) / cols_of(C));
  const int64_t first = total * x / 8, n = total * (x + 1) / 8 - first;
  for (int64_t k = blockIdx.x / 8; k < n; k += step) {
    TileAt t;
    if (!find_tile(a, C, first + k, t)) break;
    if constexpr (D == 4) {
      uint8_t* const slot[4] = {s0, s1, s2, s3};
      int8_tile<E, WM, WN, MT, NT, 4, 2, 0>(a, t, slot);
    } else {
      uint8_t* const slot[2] = {s0, s1};
      int8_tile<E, WM, WN, MT, NT, 2, 2, 2>(a, t, slot);
    }
  }
}

namespace {

constexpr int kDeep = 4;

// The weights of 16 columns from memory, `kDeep` steps of 128 K-values in
// flight a wave, the W waves taking steps in turn.  Returns a wave's sums.
template <int W, typename Rows>
__device__ __forceinline__ i32x4 stream_columns(const Int8Args& a, int n0, int w, int l, const Rows& rows) {
  const int r = l % 16, g = l / 16, K = a.K, KB = (K + kStep - 1) / kStep;
  const uint8_t* bp = a.b + (int64_t)(n0 + r < a.N ? n0 + r : a.N - 1) * K;
  u32x4 b[kDeep][2];
  typename Rows::Ahead x[kDeep][2];
  // past the end: the last step again, unused (a load under a condition would
  // make the compiler wait for all of them); past K inside the last step: the
  // row's first values, which meet zeros
  auto load = [&](int d, int kb) {
    kb = kb < KB ? kb : KB - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = kb * kStep + g * 32 + h * 16;
      b[d][h] = *reinterpret_cast<const u32x4*>(bp + (k < K ? k : 0));
      rows.ask(x[d][h], k < K ? k : 0);
    }
  };
#pragma unroll
  for (int d = 0; d < kDeep; ++d) load(d, w + d * W);
  rows.bring();
  i32x4 acc = {0, 0, 0, 0};
  for (int k0 = w; k0 < KB; k0 += kDeep * W) {
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int kb = k0 + d * W;
      if (kb < KB) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = kb * kStep + g * 32 + h * 16;
          mfma64(acc, b[d][h], rows.at(x[d][h], k, k < K));
        }
      }
      load(d, kb + kDeep * W);
    }
  }
  return acc;
}

// sums of the waves, scaled and written
template <typename E, int W>
__device__ __forceinline__ void finish_columns(const Int8Args& a, const i32x4& acc, int n0, int64_t m0, int rows, float sa,
                                               i32x4 (*red)[64]) {
  const int tid = threadIdx.x, w = tid / 64, l = tid % 64, r = l % 16, g = l / 16;
  red[w][l] = acc;
  __syncthreads();
  if (tid < 64 && r < rows) {
    i32x4 sum = red[0][l];
#pragma unroll
    for (int i = 1; i < W; ++i) sum += red[i][l];
    float ws[4], v[4];
    scales4(a.bs, a.N, n0 + 4 * g, ws);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = (float)sum[k] * ws[k] * sa;
    put4<E>(a.y, a.N, m0 + r, n0 + 4 * g, v);
  }
  __syncthreads();      // the next columns write `red` again
}

// rows of codes in memory, asked for with the weights of their step
struct RowsOfCodes {
  typedef u32x4 Ahead;
  const uint8_t* p;
  __device__ void bring() const {}
  __device__ void ask(u32x4& x, int k) const { x = *reinterpret_cast<const u32x4*>(p + k); }
  __device__ u32x4 at(const u32x4& x, int, bool in) const { return in ? x : u32x4{0u, 0u, 0u, 0u}; }
};

// The rows behind a.M, up to 16 (a.tail): 16 columns a workgroup at a time, weights
// straight from memory into the operands.
template <typename E, int W>
__device__ __forceinline__ void stream_tail(const Int8Args& a, i32x4 (*red)[64]) {
  const int l = threadIdx.x % 64, w = uniform(threadIdx.x / 64), units = (a.N + kFewCols - 1) / kFewCols;
  const int64_t row = a.M + (l % 16 < a.tail ? l % 16 : 0);
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const i32x4 acc = stream_columns<W>(a, u * kFewCols, w, l, RowsOfCodes{a.a + row * a.K});
    finish_columns<E, W>(a, acc, u * kFewCols, a.M, a.tail, a.as[row], red);
  }
}

}  // namespace

// A few rows of codes.
template <typename E>
__global__ __launch_bounds__(256) void k_int8_few(Int8Args a) {
  __shared__ i32x4 red[4][64];
  stream_tail<E, 4>(a, red);
}

// Products with many rows, or too many columns for small tiles: 256 x 256 tiles, and
// 128 x 256 for a group's rest; up to 16 rows behind the tiles of one matrix (which
// may have no tile) are streamed by who is done.
// One workgroup a CU; XCD x takes an eighth of each class's list (neighbours
// share an L2), and its workgroups take every n-th tile of it in turn.
template <typename E>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_int8_mma(Int8Args a) {
  // separate arrays: the compiler then sees that a stage's reads and the other
  // stage's copies do not meet, and does not wait for the copies
  __shared__ __attribute__((aligned(1024))) uint8_t s0[(kBM + kBN) * kStep], s1[(kBM + kBN) * kStep];
  uint8_t* const slot[2] = {s0, s1};
  const int x = blockIdx.x % 8, step = gridDim.x / 8;
  int64_t n[2], first[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int64_t total = count_blocks(a, c) * ((a.N + kBN - 1) / kBN);
    first[c] = total * x / 8;
    n[c] = total * (x + 1) / 8 - first[c];
  }
  for (int64_t k = blockIdx.x / 8; k < n[0] + n[1]; k += step) {
    TileAt t;
    if (k < n[0]) {
      if (!find_tile(a, kFull, first[0] + k, t)) break;
      int8_tile<E, 4, 2, 4, 8, 2, 1, 1>(a, t, slot);
    } else {
      if (!find_tile(a, kHalf, first[1] + k - n[0], t)) break;
      int8_tile<E, 4, 2, 2, 8, 2, 1, 1>(a, t, slot);
    }
  }
  if (a.tail > 0) stream_tail<E, 8>(a, reinterpret_cast<i32x4(*)[64]>(s0));
}

namespace {

// most values of the rows that every workgroup quantises for itself
constexpr int kRowValues = 8 * 1024;

// Rows of x, quantised into LDS by the whole workgroup: values in registers, a
// maximum per row, then the codes.
template <typename X, int THREADS>
struct RowsOfX {
  struct Ahead {};
  const Int8Args& a;
  uint8_t* codes;              // [M][pitch], zeros from K to the step's end
  float* scale;                // [M]
  uint32_t* amax;              // [M]
  int pitch, row;
  __device__ void bring() const {
    constexpr int kTurns = kRowValues / 8 / THREADS;
    const int tid = threadIdx.x, M = (int)a.M, per = a.K / 8, pad = (pitch - a.K) / 8;
    const X* x = static_cast<const X*>(a.x);
    float v[kTurns][8];
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const int i = tid + u * THREADS;
      if (i < M * per) load_elems(x + (int64_t)i * 8, v[u]);
    }
    if (tid < M) amax[tid] = 0;
    for (int i = tid; i < M * pad; i += THREADS)
      *reinterpret_cast<u32x2*>(codes + i / pad * pitch + a.K + i % pad * 8) = u32x2{0u, 0u};
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const int i = tid + u * THREADS;
      if (i - tid % 64 >= M * per) break;            // (the same in all lanes of a wave)
      uint32_t m = 0;
      const int mine = i < M * per ? i / per : -1;
      if (mine >= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m = amax_of(v[u][j], m);
      }
      const int first = uniform(mine);
      if (ballot(mine == first || mine < 0) == ~0ull) {
        m = wave_max(m);
        if (tid % 64 == 0) atomicMax(&amax[first], m);
      } else if (mine >= 0) {
        atomicMax(&amax[mine], m);
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const int i = tid + u * THREADS;
      if (i >= M * per) break;
      *reinterpret_cast<u32x2*>(codes + i / per * pitch + i % per * 8) = int8_codes(v[u], int8_scale(amax[i / per]));
    }
    if (tid < M) scale[tid] = int8_scale(amax[tid]);
    __syncthreads();
  }
  __device__ void ask(Ahead&, int) const {}
  __device__ u32x4 at(const Ahead&, int k, bool) const { return *reinterpret_cast<const u32x4*>(codes + row * pitch + k); }
};

}  // namespace

// A few floating rows (a decoded token's projection): 16 columns a workgroup;
// the first weights are asked for, the rows are quantised into LDS meanwhile.
// Bound: latency; 1 row x 7168 x 2048 7.8 us for 14.7 MB of weights (3 at the copy's
// rate), 11.5 with a quantising launch before it.
template <typename E, typename X, int W>
__global__ __launch_bounds__(64 * W) void k_int8_rows(Int8Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ i32x4 red[W][64];
  __shared__ float scale[kFewRows];
  __shared__ uint32_t amax[kFewRows];
  const int l = threadIdx.x % 64, w = uniform(threadIdx.x / 64), n0 = (int)blockIdx.x * kFewCols, M = (int)a.M;
  const int pitch = (a.K + kStep - 1) / kStep * kStep + 16;      // rows of one column of chunks in different banks
  const int row = l % 16 < M ? l % 16 : 0;
  const i32x4 acc = stream_columns<W>(a, n0, w, l, RowsOfX<X, 64 * W>{a, dyn, scale, amax, pitch, row});
  finish_columns<E, W>(a, acc, n0, 0, M, scale[row], red);
}

// Codes and scales of rows: a wave a row (GROUP false), or a workgroup whose size
// the launch fits to the row; TURNS chunks of 8 values a thread in registers, as
// they are in memory; longer rows are read twice.  Bound: HBM; 16384 x 7168 bf16 74
// us (4.8 TB/s; with the values as float32 in registers 99).
template <typename X, bool GROUP, int TURNS>
__global__ __launch_bounds__(kQuantThreads) void k_int8_quantize(const X* x, int64_t rows, int K, uint8_t* q, float* s) {
  __shared__ uint32_t red[kQuantThreads / 64];
  const int waves = blockDim.x / 64, w = threadIdx.x / 64, per = K / 8;
  const int at = GROUP ? threadIdx.x : threadIdx.x % 64, step = GROUP ? blockDim.x : 64, rows_at_once = GROUP ? 1 : waves;
  for (int64_t m0 = (int64_t)blockIdx.x * rows_at_once; m0 < rows; m0 += (int64_t)gridDim.x * rows_at_once) {
    int64_t m = GROUP ? m0 : m0 + w;
    m = m < rows ? m : rows - 1;             // (past the end: the last row again)
    const X* p = x + m * K;
    Raw8<X> v[TURNS];
    uint32_t big = 0;
#pragma unroll
    for (int u = 0; u < TURNS; ++u) v[u].load(p + (at + u * step < per ? at + u * step : 0) * 8);
#pragma unroll
    for (int u = 0; u < TURNS; ++u) {
      float f[8];
      v[u].unpack(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) big = amax_of(f[j], big);
    }
    for (int c = at + TURNS * step; c < per; c += step) {
      float f[8];
      load_elems(p + c * 8, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) big = amax_of(f[j], big);
    }
    big = wave_max(big);
    if constexpr (GROUP) {
      __syncthreads();                      // (the last row's maximum has been read)
      if (threadIdx.x % 64 == 0) red[w] = big;
      __syncthreads();
      for (int i = 0; i < waves; ++i) big = red[i] > big ? red[i] : big;
    }
    const float sc = int8_scale(big);
    if (at == 0) s[m] = sc;
#pragma unroll
    for (int u = 0; u < TURNS; ++u) {
      float f[8];
      v[u].unpack(f);
      const u32x2 o = int8_codes(f, sc);
      if (at + u * step < per) *reinterpret_cast<u32x2*>(q + m * K + (at + u * step) * 8) = o;
    }
    for (int c = at + TURNS * step; c < per; c += step) {
      float f[8];
      load_elems(p + c * 8, f);
      *reinterpret_cast<u32x2*>(q + m * K + c * 8) = int8_codes(f, sc);
    }
  }
}

namespace {

template <typename F>
hipError_t for_type(int element, const F& f) {
  return element == MM_ELEMENT_BF16 ? f(__bf16{}) : element == MM_ELEMENT_F16 ? f(_Float16{}) : f(float{});
}

template <typename E>
hipError_t gemm(const Int8Args& args, int num_cus, hipStream_t s) {
  Int8Args a = args;
  const unsigned units = (unsigned)((a.N + kFewCols - 1) / kFewCols);
  if (a.x != nullptr) {
    const size_t lds = (size_t)a.M * ((a.K + kStep - 1) / kStep * kStep + 16);
    return for_type(a.x_element, [&](auto x) {
      // eight waves where each then has all its steps in flight (1 row, us, four / eight waves: 7168 x 2048 7.7 / 9.7,
      // 16384 x 4096 18.4 / 21.0, 4096 x 7168 13.8 / 12.1)
      if (a.K <= 32 * kStep) hipLaunchKernelGGL((k_int8_rows<E, decltype(x), 4>), dim3(units), dim3(256), lds, s, a);
      else hipLaunchKernelGGL((k_int8_rows<E, decltype(x), 8>), dim3(units), dim3(512), lds, s, a);
      return hipGetLastError();
    });
  }
  // The smallest tiles that give a CU at most one, then those of 128 x 128 for up
  // to two rounds, then the large ones.  us with weights from HBM, 32 x 32 / 64 x 32 /
  // 64 x 64 / 128 x 64 / 128 x 128 / large, 4096 x 7168: 64 rows 11 / 15 / 20 / 25 / 30 /
  // 49, 128 rows 20 / 15 / 20 / 28 / 34 / 53, 256 rows 36 / 27 / 21 / 28 / 34 / 73, 512 rows
  // 72 / 54 / 41 / 38 / 46 / 90, 1024 rows - / - / 83 / 74 / 50 / 92, 1280 rows (320 tiles of
  // 128 x 128) 79 / 93, 2048 rows (512) 94 / 96, 2560 rows (640) 117 / 97; 2048 to 7168: 64
  // rows 10 / 7.7 / 9.9 / 11 / 13 / 20, 256 rows 29 / 23 / 18 / 12 / 15 / 31, 512 rows - / - / 32 /
  // 21 / 16 / 32, 1024 rows (448) 29 / 33, 1536 rows (672) 43 / 34.
  // Groups count as evenly filled, the empty ones too (which have rows is known on the
  // device alone): right for a prefill; a decoded batch over few of many groups gets
  // larger tiles than its rows fill (8 rows to 8 of 32 groups, 4096 x 7168, 83 us; to 8
  // of 8 55; 48 for the weights at a copy's rate).
  const int64_t even = a.M / a.G > 0 ? a.M / a.G : 1;
  const unsigned cus = (unsigned)((num_cus + 7) / 8 * 8);
  auto count = [&](int c) { return (even + most_rows(c) - 1) / most_rows(c) * a.G * ((a.N + cols_of(c) - 1) / cols_of(c)); };
  if (a.offsets == nullptr && a.M <= kStreamRows) {
    a.tail = (int)a.M;
    a.M = 0;
    hipLaunchKernelGGL(k_int8_few<E>, dim3(units), dim3(256), 0, s, a);
  } else if (count(k32x32) <= num_cus) {
    hipLaunchKernelGGL((k_int8_ring<E, k32x32, 2, 2, 1, 1, 4>), dim3(cus), dim3(256), 0, s, a);
  } else if (count(k64x32) <= num_cus) {
    hipLaunchKernelGGL((k_int8_ring<E, k64x32, 2, 2, 2, 1, 4>), dim3(cus), dim3(256), 0, s, a);
  } else if (count(k64x64) <= num_cus) {
    hipLaunchKernelGGL((k_int8_ring<E, k64x64, 2, 2, 2, 2, 4>), dim3(cus), dim3(256), 0, s, a);
  } else if (count(kMid) <= num_cus) {
    hipLaunchKernelGGL((k_int8_ring<E, kMid, 4, 2, 2, 2, 2>), dim3(cus), dim3(512), 0, s, a);
  } else if (count(k128x128) <= 2 * num_cus) {
    hipLaunchKernelGGL((k_int8_ring<E, k128x128, 4, 2, 2, 4, 2>), dim3(cus), dim3(512), 0, s, a);
  } else {
    // one matrix: up to 16 rows beyond the blocks of 256 are streamed, in place of a
    // round more (16388 x 4096 x 2048: 2.6 us for the last four rows; 4097 x 4096 x 7168,
    // whose tiles all end together: 4.6).  9 to 16 rows of more columns than 128 x 128
    // tiles take in two rounds (65536 on 256 CUs) come here too: all of them are such
    // rows, and there is no tile
    const int64_t rest = a.offsets == nullptr ? a.M % kBM : 0;
    if (rest <= kFewRows) {
      a.tail = (int)rest;
      a.M -= rest;
    }
    hipLaunchKernelGGL(k_int8_mma<E>, dim3(cus), dim3(512), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

bool int8_from_x(const Int8Args& a) { return a.offsets == nullptr && a.M <= kFewRows && a.M * a.K <= kRowValues; }

hipError_t launch_int8_gemm(const Int8Args& a, int num_cus, hipStream_t s) {
  return for_type(a.y_element, [&](auto e) { return gemm<decltype(e)>(a, num_cus, s); });
}

hipError_t launch_int8_quantize(const void* x, int element, int64_t rows, int cols, uint8_t* q, float* s, hipStream_t st) {
  return for_type(element, [&](auto e) {
    typedef decltype(e) X;
    const int chunks = cols / 8;
    auto run = [&](auto group, auto turns, int threads) {
      const int64_t n = decltype(group)::value ? rows : (rows + 3) / 4;
      hipLaunchKernelGGL((k_int8_quantize<X, decltype(group)::value, decltype(turns)::value>),
                         dim3((unsigned)(n < (1 << 20) ? n : (1 << 20))), dim3((unsigned)threads), 0, st,
                         static_cast<const X*>(x), rows, cols, q, s);
      return hipGetLastError();
    };
    typedef std::integral_constant<int, 2> Two;
    typedef std::integral_constant<int, 4> Four;
    // a wave a row up to 2048 columns; beyond, two chunks a thread while a workgroup has enough of them
    if (chunks <= 2 * 64) return run(std::false_type{}, Two{}, 256);
    if (chunks <= 4 * 64) return run(std::false_type{}, Four{}, 256);
    if (chunks <= 2 * kQuantThreads) return run(std::true_type{}, Two{}, (chunks + 127) / 128 * 64);
    return run(std::true_type{}, Four{}, kQuantThreads);
  });
}

}  // namespace mm
