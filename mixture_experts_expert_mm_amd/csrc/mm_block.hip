// Products of e4m3 matrices with one float32 scale per 128 values of an
// activation row and per 128 x 128 block of a weight:
//
//   y[m][n] = sum_kb sa[m][kb] * sb[n / 128][kb] * sum_{k in kb} qa[m][k] * qb[n][k]
//
// and the quantiser that makes qa and sa from bf16 rows:
//   sa = max(max|group| / 448, 1e-8),  qa = round-half-even(x / sa), saturating.
//
// Each group of 128 K-values is one 16 x 16 x 128 MFMA per 16 x 16 outputs,
// started from zero; its float32 result is scaled into float32 accumulators.
#include <type_traits>

#include "mm_device.hpp"
#include "mm_ops_internal.hpp"

namespace mm {

namespace {

constexpr int kBlock = 128;

__device__ __forceinline__ f32x4 mfma128(const u32x4& a0, const u32x4& a1, const u32x4& b0, const u32x4& b1) {
  const i32x8 a = __builtin_bit_cast(i32x8, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7));
  const i32x8 b = __builtin_bit_cast(i32x8, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
  const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 127, 0, 127);
}

// largest magnitude of the 8 bf16 of v and m, as float bits: integer order is
// magnitude order, and a NaN is above infinity
__device__ __forceinline__ uint32_t amax_bits(const u32x4& v, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (v[i] << 16) & 0x7fffffffu, hi = v[i] & 0x7fff0000u;
    m = lo > m ? lo : m;
    m = hi > m ? hi : m;
  }
  return m;
}

__device__ __forceinline__ float block_scale(uint32_t amax) {
  const float s = __uint_as_float(amax) / 448.0f;
  return s < 1e-8f ? 1e-8f : s;        // NaN stays
}

__device__ __forceinline__ float sat448(float v) { return v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v; }

// 8 bf16 -> 8 e4m3 codes of x / s (the IEEE quotient)
__device__ __forceinline__ u32x2 quant8(const u32x4& v, float s) {
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w = 0;
    const uint32_t a = v[2 * h], b = v[2 * h + 1];
    w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(sat448(__uint_as_float(a << 16) / s),
                                                  sat448(__uint_as_float(a & 0xffff0000u) / s), (int)w, false);
    w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(sat448(__uint_as_float(b << 16) / s),
                                                  sat448(__uint_as_float(b & 0xffff0000u) / s), (int)w, true);
    o[h] = w;
  }
  return o;
}

}  // namespace

// 16 lanes per group of 128, 8 values a lane.  Bound: HBM.
__global__ __launch_bounds__(256) void k_block_quantize(const uint8_t* x, int64_t chunks, uint8_t* q, float* s) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < chunks; i += stride) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(x + i * 16);
    uint32_t m = amax_bits(v, 0);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const uint32_t w = (uint32_t)__shfl_xor((int)m, o, 64);
      m = w > m ? w : m;
    }
    const float sc = block_scale(m);
    *reinterpret_cast<u32x2*>(q + i * 8) = quant8(v, sc);
    if (i % 16 == 0) s[i / 16] = sc;
  }
}

hipError_t launch_block_quantize(const void* x, int64_t rows, int cols, uint8_t* q, float* s, hipStream_t st) {
  const int64_t chunks = rows * (cols / 8);       // a multiple of 16: a group never straddles two rounds
  const int64_t blocks = (chunks + 255) / 256;
  hipLaunchKernelGGL(k_block_quantize, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st,
                     static_cast<const uint8_t*>(x), chunks, q, s);
  return hipGetLastError();
}

namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kThreads = 512, kWaves = 8;
constexpr int kBM = 256, kBN = 256;       // the large tile
constexpr int kMidBM = 128, kMidBN = 64;  // the small tile
constexpr int kFewRows = 16;              // most rows of a streaming unit
constexpr int kFewCols = 16;
constexpr int kRing = 4;                  // stages of the smallest tiles
constexpr int kLargeTiles = 96;           // fewest large tiles of a product that is cut into them
constexpr int kGroupM = 6;                // M-blocks that a run of tiles goes through before the next N-block

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// rows of group gi, clipped to the matrix
__device__ __forceinline__ void group_rows(const BlockArgs& a, int gi, int64_t& lo, int64_t& n) {
  if (a.offsets == nullptr) {
    lo = 0, n = a.M;
    return;
  }
  lo = a.offsets[gi];
  int64_t hi = lo + a.counts[gi];
  lo = lo < 0 ? 0 : lo;
  hi = hi > a.M ? a.M : hi;
  n = hi > lo ? hi - lo : 0;
}

// How the rows of a group are cut: into blocks of 256 rows, a rest of up to
// 128 rows being a half block (half the products), listed after the full
// ones.  kMid: blocks of 128 rows and 64 columns; the others as they say.
enum Class : int { kFull = 0, kHalf = 1, kMid = 2, k64x64 = 3, k64x32 = 4, k32x32 = 5, k32x16 = 6, k128x128 = 7 };

__host__ __device__ __forceinline__ int cols_of(int c) { return c <= kHalf ? kBN : c == k128x128 ? 128 : c <= k64x64 ? kMidBN : c == k32x16 ? 16 : 32; }
__host__ __device__ __forceinline__ int most_rows(int c) { return c <= kHalf ? kBM : c == kMid || c == k128x128 ? kMidBM : c >= k32x32 ? 32 : 64; }

// M-blocks of class c in a group of n rows
__device__ __forceinline__ int64_t blocks_of(int c, int64_t n) {
  const int rest = (int)(n % kBM);
  if (c >= kMid) return (n + most_rows(c) - 1) / most_rows(c);
  if (c == kHalf) return rest > 0 && rest <= kBM / 2 ? 1 : 0;
  return n / kBM + (rest > kBM / 2 ? 1 : 0);
}
__device__ __forceinline__ int64_t first_block_row(int c, int64_t n, int64_t mb) {
  return c == kHalf ? n / kBM * kBM : mb * most_rows(c);
}

// M-blocks of class c over all groups (every lane of the wave takes part)
__device__ int64_t count_blocks(const BlockArgs& a, int c) {
  if (a.offsets == nullptr) return blocks_of(c, a.M);
  int64_t sum = 0;
  for (int g = lane_id(); g < a.G; g += 64) {
    int64_t lo, n;
    group_rows(a, g, lo, n);
    sum += blocks_of(c, n);
  }
  return wave_sum(sum);
}

struct TileAt {
  int64_t m0;          // first row
  int rows, group, n0;
};

// in scalar registers, where the copies' descriptors need it (rows are below 2^24)
__device__ __forceinline__ TileAt uniform_tile(const TileAt& t) {
  return TileAt{(int64_t)(uint32_t)uniform((int)t.m0), uniform(t.rows), uniform(t.group), uniform(t.n0)};
}

// Tile `at` of class c in the order (group, 6 M-blocks, N-block, M-block): the
// 32 tiles of an XCD then read 6 row panels and 5 or 6 weight panels.  A CU's
// requests wait 500 cycles on average, and how many find L2 decides the rate:
// 16384 x 4096 x 7168 takes 424 us (482 with 64 M-blocks first), 16384 x 7168 x
// 2048 270 us (280 with 8, 292 with 64).
__device__ bool find_tile(const BlockArgs& a, int c, int64_t at, TileAt& o) {
  const int bn = cols_of(c), nb = (a.N + bn - 1) / bn;
  int l = lane_id();
  asm volatile("" : "+v"(l));
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    int64_t lo = 0, n = 0;
    if (g0 + l < a.G) group_rows(a, g0 + l, lo, n);
    const int64_t mine = blocks_of(c, n) * nb;
    int64_t pre = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t v = __shfl_up(pre, d, 64);
      if (l >= d) pre += v;
    }
    const int64_t all = __shfl(pre, 63, 64);
    if (at < all) {
      const int src = __ffsll((unsigned long long)ballot(at < pre)) - 1;
      const int64_t first = __shfl(pre - mine, src, 64), rows = __shfl(n, src, 64), row0 = __shfl(lo, src, 64);
      const int64_t mb = blocks_of(c, rows), k = at - first;
      const int64_t chunk = k / (kGroupM * nb), m0 = chunk * kGroupM, in = k - m0 * nb;
      const int64_t gm = mb - m0 < kGroupM ? mb - m0 : kGroupM;
      const int64_t m = first_block_row(c, rows, m0 + in % gm);
      const int64_t most = most_rows(c);
      o.group = g0 + src;
      o.n0 = (int)(in / gm) * bn;
      o.m0 = row0 + m;
      o.rows = (int)(rows - m < most ? rows - m : most);
      return true;
    }
    at -= all;
  }
  return false;
}

// Large tile: 64 * MT rows x 256 columns, 8 waves (2 along N, 4 along M) of
// 16 * MT rows x 128 columns, one group of 128 K-values per stage, two LDS
// stages filled by LDS-DMA.  Weights are the MFMA's A operand, so a lane's
// four accumulators are four columns of one row: its scale is one number per
// row tile, and its result one 8-byte store.
// Bound: the copies.  Products alone take 1.03 us a stage, copies that always
// hit the same lines 1.0 us, the real ones 1.65 us: 64 KiB a stage with a
// mean latency of 500 cycles, of which a CU has about 64 lines in flight.
// 16384 x 4096 x 7168 ran at 2.27 PFLOP/s; a large e4m3 library product reaches
// 2.67 here.
// PAIR (small tiles): two groups of 128 a stage, in four slots of LDS, for
// half as many waits.
template <int WN, int NT, int MT, bool PAIR, int SR>
__device__ __forceinline__ void mma_tile(const BlockArgs& a, const TileAt& at, uint8_t* sa0, uint8_t* sa1, uint8_t* sb0,
                                         uint8_t* sb1, uint8_t* sa2, uint8_t* sa3, uint8_t* sb2, uint8_t* sb3,
                                         float (*ssc)[2][SR]) {
  constexpr int WM = kWaves / WN, BM = 16 * MT * WM, BN = 16 * NT * WN;
  static_assert(BM <= SR && BM % 64 == 0 && BN % 64 == 0 && (kBlock % (16 * NT) == 0), "whole copies, one weight scale a wave");
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));   // nothing derived from it is kept across tiles: the registers are full
  const TileAt t = uniform_tile(at);
  const int w = uniform(tid / 64), l = tid % 64, r = l % 16, g = l / 16;
  const int wm = w % WM, wn = w / WM, KB = a.K / kBlock;
  const int rows = t.rows, cols = a.N - t.n0 < BN ? a.N - t.n0 : BN;
  // one instruction moves 8 rows of 128 bytes, lane i to byte 16 * i; the
  // chunk at place p of row x is p ^ (x / 2 % 8), so that 16 rows read at one
  // chunk hit 16 different bank groups.  Rows past the last one are beyond the
  // descriptor and arrive as zeros without a memory access.
  const uint32_t voff = (uint32_t)(l / 8) * a.K + (((l % 8) ^ ((4 * (w % 2) + l / 16) % 8)) * 16);
  const uint8_t *ab = a.a + t.m0 * a.K, *bb = a.b + ((int64_t)t.group * a.N + t.n0) * a.K;
  constexpr int kCopies = (BM + BN) / 64;   // instructions of a wave and stage
  auto copy = [&](int i, int kb, uint8_t* sa, uint8_t* sb) {
    const bool of_a = i < BM / 64;
    const int grp = w + 8 * (of_a ? i : i - BM / 64);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)(of_a ? ab : bb), (short)0, (of_a ? rows : cols) * a.K, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)((of_a ? sa : sb) + grp * 1024), 16, voff, grp * 8 * a.K + kb * kBlock, 0, 0);
  };
  const int nb = (t.n0 + wn * NT * 16) / kBlock, nblocks = (a.N + kBlock - 1) / kBlock;
  const float* bsp = a.bs + ((int64_t)t.group * nblocks + (nb < nblocks ? nb : nblocks - 1)) * KB;
  const int sw = (r / 2) % 8;
  // a lane group takes chunks g and g + 4 of both operands: each read then
  // covers four neighbouring chunks (2g and 2g + 1 met in the same banks:
  // half of the LDS cycles were conflicts)
  const int c0 = (g ^ sw) * 16 + r * kBlock, c1 = ((g + 4) ^ sw) * 16 + r * kBlock;
  // Row scales of two stages at a time through LDS, one a thread: a wave's own
  // gather of its 64 rows' scales, each in a line of its own, cost a fifth of
  // the time (780 against 612 us without them at 16384 x 4096 x 7168).
  // Beyond the rows the descriptor gives 0, beyond a row's end its neighbour's
  // scale, which no product takes.
  const float* asb = a.as + t.m0 * KB;
  const int srow = tid / 2;
  auto ask = [&](int kb) {
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)asb, (short)0, rows * KB * 4, 0x00020000);
    return __builtin_amdgcn_raw_buffer_load_b32(rs, (srow * KB + tid % 2) * 4, kb * 4, 0);
  };
  auto keep = [&](int pair, uint32_t v) {
    if (srow < SR) ssc[pair % 2][tid % 2][srow] = __uint_as_float(v);
  };
  f32x4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // The copies of stage kn go out two at a time between the first products:
  // all at once they hold up each wave's issue until the address unit has taken
  // them, and copies and products add up; one at a time, over the whole stage,
  // the last ones are waited for (32 groups of 512 rows, 4096 x 7168: two 602 us,
  // three 604, one 630; 4097 x 7168 x 4096 109, 112, 117).
  auto compute = [&](auto more, const uint8_t* sa, const uint8_t* sb, const float* ss, float scb, int kn, uint8_t* na, uint8_t* nbuf) {
    constexpr int need = (kCopies + NT - 1) / NT, per = decltype(more)::value ? (need > 2 ? need : 2) : 0;
    u32x4 af[MT][2], b[2][2];
    float sc[MT];
    f32x4 sum[2][MT];
    auto weights = [&](int j) {
      b[j % 2][0] = *reinterpret_cast<const u32x4*>(sb + (wn * NT + j) * 16 * kBlock + c0);
      b[j % 2][1] = *reinterpret_cast<const u32x4*>(sb + (wn * NT + j) * 16 * kBlock + c1);
    };
    weights(0);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      af[i][0] = *reinterpret_cast<const u32x4*>(sa + (wm * MT + i) * 16 * kBlock + c0);
      af[i][1] = *reinterpret_cast<const u32x4*>(sa + (wm * MT + i) * 16 * kBlock + c1);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sc[i] = ss[(wm * MT + i) * 16 + r] * scb;
    // products of tile j while tile j - 1 is scaled and tile j + 1 is read;
    // issue order: the reads, then a product and four scalings in turn
#pragma unroll
    for (int j = 0; j <= NT; ++j) {
      if (j + 1 < NT) weights(j + 1);
      if (j < NT) {
#pragma unroll
        for (int q = 0; q < per; ++q)
          if (j * per + q < kCopies) copy(j * per + q, kn, na, nbuf);
#pragma unroll
        for (int i = 0; i < MT; ++i) sum[j % 2][i] = mfma128(b[j % 2][0], b[j % 2][1], af[i][0], af[i][1]);
      }
      if (j > 0) {
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j - 1][i] += sum[(j - 1) % 2][i] * sc[i];
      }
      if (j > 0 && j < NT) {
        if (j + 1 < NT) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        if (j * per < kCopies && per > 0) __builtin_amdgcn_sched_group_barrier(0x010, per, 0);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto turn = [&]() {
    // the stage's products stay before the wait: nothing else ties them to it
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) asm volatile("" : "+v"(acc[j][i]));
    __builtin_amdgcn_sched_barrier(0);
    stage_barrier<0>();
    __builtin_amdgcn_sched_barrier(0);
  };
  if constexpr (PAIR) {
    auto last = [&](int kb) { return kb < KB ? kb : KB - 1; };   // past the end: the last group again, unused
    float sc0 = bsp[0], sc1 = bsp[last(1)];
    {
      const uint32_t v = ask(0);
#pragma unroll
      for (int i = 0; i < kCopies; ++i) copy(i, 0, sa0, sb0);
#pragma unroll
      for (int i = 0; i < kCopies; ++i) copy(i, last(1), sa1, sb1);
      keep(0, v);
    }
    turn();
    auto stage = [&](int kb, int pair, uint8_t* a0, uint8_t* a1, uint8_t* b0, uint8_t* b1, uint8_t* na0, uint8_t* na1,
                     uint8_t* nb0, uint8_t* nb1) {
      const uint32_t v = ask(kb + 2);
      const float n0 = bsp[last(kb + 2)], n1 = bsp[last(kb + 3)];
      __builtin_amdgcn_sched_barrier(0);
      compute(std::true_type{}, a0, b0, ssc[pair % 2][0], sc0, last(kb + 2), na0, nb0);
      if (kb + 1 < KB) compute(std::true_type{}, a1, b1, ssc[pair % 2][1], sc1, last(kb + 3), na1, nb1);
      keep(pair + 1, v);
      turn();
      sc0 = n0, sc1 = n1;
    };
    for (int kb = 0, pair = 0; kb < KB; kb += 4, pair += 2) {
      stage(kb, pair, sa0, sa1, sb0, sb1, sa2, sa3, sb2, sb3);
      if (kb + 2 >= KB) break;
      stage(kb + 2, pair + 1, sa2, sa3, sb2, sb3, sa0, sa1, sb0, sb1);
    }
  } else {
    {
      const uint32_t v = ask(0);
#pragma unroll
      for (int i = 0; i < kCopies; ++i) copy(i, 0, sa0, sb0);
      keep(0, v);
    }
    float scb = bsp[0];
    turn();
    int kb = 0, pair = 0;
    for (; kb + 1 < KB; kb += 2, ++pair) {
      // loads that the next stages need go out before the copies: a wait for
      // them leaves the copies in flight
      const uint32_t v = ask(kb + 2);
      const float scb1 = bsp[kb + 1];
      __builtin_amdgcn_sched_barrier(0);
      compute(std::true_type{}, sa0, sb0, ssc[pair % 2][0], scb, kb + 1, sa1, sb1);
      turn();
      const int nx = kb + 2 < KB ? kb + 2 : KB - 1;   // past the end: the last stage again, unused
      scb = bsp[nx];
      __builtin_amdgcn_sched_barrier(0);
      keep(pair + 1, v);
      compute(std::true_type{}, sa1, sb1, ssc[pair % 2][1], scb1, nx, sa0, sb0);
      turn();
    }
    if (kb < KB) compute(std::false_type{}, sa0, sb0, ssc[pair % 2][0], scb, 0, sa1, sb1);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int n = t.n0 + (wn * NT + j) * 16 + 4 * g;
      const int row = (wm * MT + i) * 16 + r;
      if (row < rows && n < a.N)
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + (t.m0 + row) * a.N + n) =
            u32x2{pack_bf16x2(acc[j][i][0], acc[j][i][1]), pack_bf16x2(acc[j][i][2], acc[j][i][3])};
    }
  __syncthreads();      // the next tile of this workgroup writes the stages again
}

}  // namespace

// Products with many rows.  One workgroup a CU; XCD x takes an eighth of
// each class's list (neighbours share an L2), and its workgroups take
// every n-th tile of it in turn.
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_block_mma(BlockArgs a) {
  // separate arrays: the compiler then sees that a stage's reads and the other
  // stage's copies do not meet, and does not wait for the copies
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[kBM * kBlock], sa1[kBM * kBlock], sb0[kBN * kBlock], sb1[kBN * kBlock];
  __shared__ float ssc[2][2][kBM];
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
      mma_tile<2, 8, 4, false>(a, t, sa0, sa1, sb0, sb1, nullptr, nullptr, nullptr, nullptr, ssc);
    } else {
      if (!find_tile(a, kHalf, first[1] + k - n[0], t)) break;
      mma_tile<2, 8, 2, false>(a, t, sa0, sa1, sb0, sb1, nullptr, nullptr, nullptr, nullptr, ssc);
    }
  }
}

// Products whose large tiles would leave most CUs without one: 128 rows x 32 * NT
// columns, one workgroup a CU with two groups of 128 a stage, or (PAIR false)
// three with one.
template <int NT, bool PAIR>
__global__ __launch_bounds__(kThreads) void k_block_mid(BlockArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[kMidBM * kBlock], sa1[kMidBM * kBlock];
  __shared__ __attribute__((aligned(1024))) uint8_t sb0[32 * NT * kBlock], sb1[32 * NT * kBlock];
  __shared__ float ssc[2][2][kMidBM];
  constexpr int c = NT == 2 ? kMid : k128x128;
  const int x = blockIdx.x % 8, step = gridDim.x / 8;
  const int64_t total = count_blocks(a, c) * ((a.N + 32 * NT - 1) / (32 * NT));
  const int64_t first = total * x / 8, n = total * (x + 1) / 8 - first;
  for (int64_t k = blockIdx.x / 8; k < n; k += step) {
    TileAt t;
    if (!find_tile(a, c, first + k, t)) break;
    if constexpr (PAIR) {
      __shared__ __attribute__((aligned(1024))) uint8_t sa2[kMidBM * kBlock], sa3[kMidBM * kBlock];
      __shared__ __attribute__((aligned(1024))) uint8_t sb2[32 * NT * kBlock], sb3[32 * NT * kBlock];
      mma_tile<2, NT, 2, true>(a, t, sa0, sa1, sb0, sb1, sa2, sa3, sb2, sb3, ssc);
    } else {
      mma_tile<2, NT, 2, false>(a, t, sa0, sa1, sb0, sb1, nullptr, nullptr, nullptr, nullptr, ssc);
    }
  }
}

// Products with few tiles of any size: 32 * MT rows x 32 * NT columns by four
// waves (2 x 2), two groups of 128 K-values a stage, four stages of LDS.
// NT = 0: 16 columns; two waves take a stage's first group, two its second.
// Bound: the stages in turn: 17 rows x 4096 x 7168 takes 12.5 us with weights from
// HBM (29 MB, 6 us at the copy rate): its copies alone 11.7, its products alone
// 9.8; with one stage ahead instead of three 24.  Six or eight stages: the same
// or worse (more to fill first).
template <int MT, int NT>
__device__ __forceinline__ void ring_tile(const BlockArgs& a, const TileAt& at, uint8_t* const (&slot)[kRing],
                                          float* const (&scale)[kRing]) {
  constexpr int D = kRing;
  constexpr bool SPLIT = NT == 0;
  constexpr int BM = 32 * MT, BN = SPLIT ? 16 : 32 * NT, kPart = (BM + BN) * kBlock, kGroups = (BM + BN) / 8;
  constexpr int kCopies = 2 * kGroups / 4 + 1;    // instructions of a wave and stage
  constexpr int NC = SPLIT ? 1 : NT;              // column tiles of a wave
  const int tid = threadIdx.x;
  const TileAt t = uniform_tile(at);
  const int w = uniform(tid / 64), l = tid % 64, r = l % 16, g = l / 16, wm = w % 2, wn = w / 2;
  const int KB = a.K / kBlock, stages = (KB + 1) / 2, rows = t.rows, cols = a.N - t.n0 < BN ? a.N - t.n0 : BN;
  // as mma_tile: 8 rows of 128 bytes an instruction, chunks swapped by row, zeros beyond the rows
  const uint32_t voff = (uint32_t)(l / 8) * a.K + (((l % 8) ^ ((4 * (w % 2) + l / 16) % 8)) * 16);
  const uint8_t *ab = a.a + t.m0 * a.K, *bb = a.b + ((int64_t)t.group * a.N + t.n0) * a.K;
  // row scales by the same path: lane i of wave w brings group i % 2 of row 32 * w + i / 2
  const uint32_t svo = w < MT ? (uint32_t)((32 * w + l / 2) * KB + l % 2) * 4 : 0x7fffff00u;
  const float* asb = a.as + t.m0 * KB;
  const int nb = t.n0 / kBlock, nblocks = (a.N + kBlock - 1) / kBlock;   // BN columns lie in one block
  const float* bsp = a.bs + ((int64_t)t.group * nblocks + nb) * KB;
  const int sw = (r / 2) % 8;
  const int o0 = (g ^ sw) * 16 + r * kBlock, o1 = ((g + 4) ^ sw) * 16 + r * kBlock;
  auto block = [&](int kb) { return kb < KB ? kb : KB - 1; };   // past the end: the last group again, unused
  // (stages past the end are copied from nothing: without a memory access)
  auto copy = [&](int s, uint8_t* to, float* sc) {
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)ab, (short)0, s < stages ? rows * a.K : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void*)bb, (short)0, s < stages ? cols * a.K : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)asb, (short)0, s < stages ? rows * KB * 4 : 0, 0x00020000);
    if constexpr (SPLIT) {
#pragma unroll
      for (int i = 0; i < 2 * kGroups / 4; ++i) {
        const int item = w + 4 * i, p = item / kGroups, grp = item % kGroups;   // rows of a, then of b
        const bool of_a = grp < BM / 8;
        const int at = block(2 * s + p) * kBlock + (of_a ? grp : grp - BM / 8) * 8 * a.K;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(of_a ? ra : rb, (lds_ptr_t)(to + p * kPart + grp * 1024), 16, voff, at, 0, 0);
      }
    } else {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int at = block(2 * s + p) * kBlock;
#pragma unroll
        for (int i = 0; i < NT; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(to + p * kPart + BM * kBlock + (w + 4 * i) * 1024), 16, voff, (w + 4 * i) * 8 * a.K + at, 0, 0);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(to + p * kPart + (w + 4 * i) * 1024), 16, voff, (w + 4 * i) * 8 * a.K + at, 0, 0);
      }
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(sc + w * 64), 4, svo, s * 8, 0, 0);
  };
  f32x4 acc[NC][MT];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto turn = [&]() {
    // the stage's products stay before the wait: nothing else ties them to it
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) asm volatile("" : "+v"(acc[j][i]));
    __builtin_amdgcn_sched_barrier(0);
    stage_barrier<(D - 2) * kCopies>();           // all but the next stage's copies may be in flight
    __builtin_amdgcn_sched_barrier(0);
  };
  // Weight scales by lane, the next CB blocks' asked for CB blocks ahead: a load
  // that a stage waits for would wait for the copies before it too.
  constexpr int CB = 8 * D;
  float cur = bsp[block(l)], nxt = bsp[block(CB + l)];
  int base = 0;
  auto refresh = [&](int s) {
    if (2 * s - base != CB) return;
    base += CB;
    cur = nxt;
    nxt = bsp[block(base + CB + l)];
  };
  __builtin_amdgcn_sched_barrier(0);
  auto stage = [&](int s, const uint8_t* from, const float* sc, uint8_t* to, float* nsc) {
    copy(s + D - 1, to, nsc);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < (SPLIT ? 1 : 2); ++u) {
      const int p = SPLIT ? wn : u;
      if (p == 0 || 2 * s + 1 < KB) {
        u32x4 af[MT][2], bf[NC][2];
        float sa[MT];
        const float sb = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(cur), 2 * s + p - base));
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          const uint8_t* q = from + p * kPart + BM * kBlock + (wn * NT + j) * 16 * kBlock;
          bf[j][0] = *reinterpret_cast<const u32x4*>(q + o0);
          bf[j][1] = *reinterpret_cast<const u32x4*>(q + o1);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint8_t* q = from + p * kPart + (wm * MT + i) * 16 * kBlock;
          af[i][0] = *reinterpret_cast<const u32x4*>(q + o0);
          af[i][1] = *reinterpret_cast<const u32x4*>(q + o1);
          sa[i] = sc[((wm * MT + i) * 16 + r) * 2 + p] * sb;
        }
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[j][i] += mfma128(bf[j][0], bf[j][1], af[i][0], af[i][1]) * sa[i];
      }
    }
    turn();
  };
#pragma unroll
  for (int u = 0; u < D - 1; ++u) copy(u, slot[u], scale[u]);
  turn();
  // (a break inside the loop would be a path on which the compiler sees a slot
  // filled one stage ago, and waits for it)
  auto at_slot = [&](int s, int u) { stage(s + u, slot[u], scale[u], slot[(u + D - 1) % D], scale[(u + D - 1) % D]); };
  int s = 0;
  for (; s + D <= stages; s += D) {
    refresh(s);
#pragma unroll
    for (int u = 0; u < D; ++u) at_slot(s, u);
  }
  refresh(s);
#pragma unroll
  for (int u = 0; u < D - 1; ++u) {
    if (s + u >= stages) break;
    at_slot(s, u);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);              // no copy outlives the tile
  if constexpr (SPLIT) {
    __syncthreads();                               // nobody reads or fills a stage any more
    f32x4* half = reinterpret_cast<f32x4*>(slot[0]);
    if (wn == 1) {
#pragma unroll
      for (int i = 0; i < MT; ++i) half[(wm * MT + i) * 64 + l] = acc[0][i];
    }
    __syncthreads();
    if (wn == 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[0][i] += half[(wm * MT + i) * 64 + l];
    }
  }
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (SPLIT && wn != 0) break;
      const int n = t.n0 + (wn * NT + j) * 16 + 4 * g;
      const int row = (wm * MT + i) * 16 + r;
      if (row < rows && n < a.N)
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + (t.m0 + row) * a.N + n) =
            u32x2{pack_bf16x2(acc[j][i][0], acc[j][i][1]), pack_bf16x2(acc[j][i][2], acc[j][i][3])};
    }
  __syncthreads();      // the next tile of this workgroup writes the stages again
}

template <int MT, int NT>
__global__ __launch_bounds__(256) void k_block_ring(BlockArgs a) {
  constexpr int c = NT == 0 ? k32x16 : MT == 1 ? k32x32 : NT == 1 ? k64x32 : k64x64;
  constexpr int kBytes = (32 * MT + (NT == 0 ? 16 : 32 * NT)) * kBlock * 2;
  // separate arrays, as in k_block_mma
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kBytes], s1[kBytes], s2[kBytes], s3[kBytes];
  __shared__ float c0[256], c1[256], c2[256], c3[256];   // a float a thread, whatever the rows
  uint8_t* const slot[kRing] = {s0, s1, s2, s3};
  float* const scale[kRing] = {c0, c1, c2, c3};
  const int x = blockIdx.x % 8, step = gridDim.x / 8;
  const int64_t total = count_blocks(a, c) * ((a.N + cols_of(c) - 1) / cols_of(c));
  const int64_t first = total * x / 8, n = total * (x + 1) / 8 - first;
  for (int64_t k = blockIdx.x / 8; k < n; k += step) {
    TileAt t;
    if (!find_tile(a, c, first + k, t)) break;
    ring_tile<MT, NT>(a, t, slot, scale);
  }
}

// The last rows of one matrix, up to 16 (a.m_first and on): 16 columns a workgroup.
// Each weight byte goes straight from memory into an operand; the 8 waves
// share the K-blocks, D of them in flight a wave, and meet in LDS.
__global__ __launch_bounds__(kThreads) void k_block_few(BlockArgs a) {
  constexpr int D = 4;
  __shared__ f32x4 red[kWaves][64];
  const int tid = threadIdx.x, w = uniform(tid / 64), l = tid % 64, r = l % 16, g = l / 16;
  const int KB = a.K / kBlock, n0 = (int)blockIdx.x * kFewCols, rows = (int)(a.M - a.m_first);
  const uint8_t* bp = a.b + (int64_t)(n0 + r) * a.K + g * 32;
  const float* bsp = a.bs + (int64_t)(n0 / kBlock) * KB;
  const int64_t row = a.m_first + (r < rows ? r : 0);
  const uint8_t* ap = a.a + row * a.K + g * 32;
  const float* asp = a.as + row * KB;
  struct Stage {
    u32x4 b[2], x[2];
    float sa, sb;
  } st[D];
  // Past the end the last block again, unused: a load under a condition would
  // make the compiler wait for every load in flight before each product.
  auto load = [&](Stage& s, int kb) {
    kb = kb < KB ? kb : KB - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) s.b[h] = *reinterpret_cast<const u32x4*>(bp + (int64_t)kb * kBlock + h * 16);
    s.sb = bsp[kb];
#pragma unroll
    for (int h = 0; h < 2; ++h) s.x[h] = *reinterpret_cast<const u32x4*>(ap + (int64_t)kb * kBlock + h * 16);
    s.sa = asp[kb];
  };
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int d = 0; d < D; ++d) load(st[d], w + d * kWaves);
  for (int kb = w; kb < KB; kb += D * kWaves) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int k = kb + d * kWaves;
      if (k < KB) acc += mfma128(st[d].b[0], st[d].b[1], st[d].x[0], st[d].x[1]) * (st[d].sa * st[d].sb);
      load(st[d], k + D * kWaves);
    }
  }
  red[w][l] = acc;
  __syncthreads();
  if (tid < 64 && r < rows) {
    f32x4 v = red[0][l];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) v += red[k][l];
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + row * a.N + n0 + 4 * g) =
        u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

// A few rows (a decoded token's projection): 16 columns a workgroup of 4 waves.
// The first weights are asked for, the rows are brought into LDS meanwhile, from
// codes or quantised from bf16 (the same codes and scales as k_block_quantize,
// by the same code), then the waves stream their K-blocks.  Bound: latency: one row x
// 7168 x 2048 takes 7.1 us for 14.7 MB of weights (3 us at the copy rate);
// a quantising kernel before it took 2.5 us and a launch more.
constexpr int kRowThreads = 256, kRowWaves = 4;
// Most codes in LDS; us with weights from HBM, these / the smallest tiles: 4 rows
// x 4096 x 7168 11.5 / 12.0, 8 rows 14.4 / 11.9; 8 rows x 2048 x 4096 7.4 / 7.7, 16
// rows 9.6 / 7.7.
constexpr int64_t kRowBytes = 32 * 1024;

template <bool FROM_X>
__global__ __launch_bounds__(kRowThreads) void k_block_rows(BlockArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ f32x4 red[kRowWaves][64];
  const int tid = threadIdx.x, w = uniform(tid / 64), l = tid % 64, r = l % 16, g = l / 16;
  const int KB = a.K / kBlock, M = (int)a.M, n0 = (int)blockIdx.x * kFewCols;
  const int pitch = a.K + 16;                   // rows of one column of chunks in different banks
  uint8_t* codes = dyn;                         // [M][pitch]
  float* scales = reinterpret_cast<float*>(dyn + M * pitch);   // [M][KB]
  constexpr int D = 4;
  const uint8_t* bp = a.b + (int64_t)(n0 + r) * a.K + g * 32;
  const float* bsp = a.bs + (int64_t)(n0 / kBlock) * KB;
  u32x4 b[D][2];
  float sb[D];
  // past the end: the last block again, unused (a load under a condition would
  // make the compiler wait for all of them)
  auto load = [&](int d, int kb) {
    kb = kb < KB ? kb : KB - 1;
    b[d][0] = *reinterpret_cast<const u32x4*>(bp + (int64_t)kb * kBlock);
    b[d][1] = *reinterpret_cast<const u32x4*>(bp + (int64_t)kb * kBlock + 16);
    sb[d] = bsp[kb];
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, w + d * kRowWaves);
  if constexpr (!FROM_X) {
    const int per = a.K / 16;
    for (int i = tid; i < M * per; i += kRowThreads)
      *reinterpret_cast<u32x4*>(codes + i / per * pitch + i % per * 16) = *reinterpret_cast<const u32x4*>(a.a + (int64_t)i * 16);
    for (int i = tid; i < M * KB; i += kRowThreads) scales[i] = a.as[i];
  }
  const int per = a.K / 8;
  for (int i = tid; FROM_X && i < M * per; i += kRowThreads) {   // 16 lanes a group; a whole number of groups a round
    const int row = i / per, c = i % per;
    const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.x) + (int64_t)i * 16);
    uint32_t m = amax_bits(v, 0);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const uint32_t x = (uint32_t)__shfl_xor((int)m, o, 64);
      m = x > m ? x : m;
    }
    const float s = block_scale(m);
    *reinterpret_cast<u32x2*>(codes + row * pitch + c * 8) = quant8(v, s);
    if (c % 16 == 0) scales[row * KB + c / 16] = s;
  }
  __syncthreads();
  const int row = r < M ? r : 0;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = w; k0 < KB; k0 += D * kRowWaves) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int kb = k0 + d * kRowWaves;
      if (kb < KB) {
        const uint8_t* q = codes + row * pitch + kb * kBlock + g * 32;
        acc += mfma128(b[d][0], b[d][1], *reinterpret_cast<const u32x4*>(q), *reinterpret_cast<const u32x4*>(q + 16)) *
               (scales[row * KB + kb] * sb[d]);
      }
      load(d, kb + D * kRowWaves);
    }
  }
  red[w][l] = acc;
  __syncthreads();
  if (tid < 64 && r < M) {
    const f32x4 v = red[0][l] + red[1][l] + red[2][l] + red[3][l];
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + (int64_t)r * a.N + n0 + 4 * g) =
        u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

bool block_in_lds(const BlockArgs& a) { return a.offsets == nullptr && a.M <= 16 && a.M * a.K <= kRowBytes; }
// bf16 rows are quantised by every workgroup for itself, against a launch more
// (1 row x 7168 x 2048 7.1 against 9.2 us, 4 rows 9.6 / 9.2, 8 rows 13.1 / 9.2; 2 rows x
// 4096 x 7168 15.4 / 13.6)
constexpr int64_t kRowValues = 8 * 1024;
bool block_from_x(const BlockArgs& a) { return block_in_lds(a) && a.M * a.K <= kRowValues; }

hipError_t launch_block_gemm(const BlockArgs& args, int num_cus, hipStream_t s) {
  BlockArgs a = args;
  const int64_t units = a.N / kFewCols;
  if (block_in_lds(a)) {
    const size_t lds = (size_t)(a.M * (a.K + 16 + a.K / kBlock * 4));
    if (a.x != nullptr) hipLaunchKernelGGL(k_block_rows<true>, dim3((unsigned)units), dim3(kRowThreads), lds, s, a);
    else hipLaunchKernelGGL(k_block_rows<false>, dim3((unsigned)units), dim3(kRowThreads), lds, s, a);
    return hipGetLastError();
  }
  // The smallest tiles that give a CU at most one: us with weights from HBM, 128 x
  // 64 / 64 x 64, 64 x 32 or 32 x 32 / 32 x 16, 4096 x 7168: 17 rows 34 / 15.3 / 12.5, 64
  // rows 36 / 15, 128 rows 43 / 21, 256 rows 42 / 27; 2048 x 4096: 17 rows 17.5 / 9.0 /
  // 7.7, 256 rows 18.6 / 12; 7168 x 2048: 17 rows 12.3 / 6.9 / -, 256 rows 15.5 / 15.3.
  // Then, at 4096 x 7168, 512 rows: large tiles / 128 x 64 / 128 x 64 with two groups a
  // stage 81 / 40 / 33.  128 x 64 / 128 x 128 where a CU gets at most one of these:
  // 1024 x 4096 x 7168 63 / 52, 320 x 7168 x 2048 21 / 18, 2048 x 2048 x 4096 37 / 30.
  // Large tiles from 96 of them on (large / 128 x 64: 4096 x 7168 80 tiles 85 / 89,
  // 96 tiles 88 / 99, 112 tiles 89 / 101, 128 tiles 89 / 111; 2048 x 4096 72 tiles 50 /
  // 49, 96 tiles 51 / 50, 104 tiles 51 / 55; 7168 x 2048 84 tiles 32 / 28, 112 tiles 33 /
  // 33, 140 tiles 33 / 42; 32 groups of 16 rows, 512 half tiles, 182 / 277).
  const int64_t even = a.M / a.G > 0 ? a.M / a.G : 1;
  const int64_t tiles = (even + kBM - 1) / kBM * a.G * ((a.N + kBN - 1) / kBN);
  const unsigned cus = (unsigned)((num_cus + 7) / 8 * 8);
  auto count = [&](int c) { return (even + most_rows(c) - 1) / most_rows(c) * a.G * ((a.N + cols_of(c) - 1) / cols_of(c)); };
  if (count(k32x16) <= num_cus) hipLaunchKernelGGL((k_block_ring<1, 0>), dim3(cus), dim3(256), 0, s, a);
  else if (count(k32x32) <= num_cus) hipLaunchKernelGGL((k_block_ring<1, 1>), dim3(cus), dim3(256), 0, s, a);
  else if (count(k64x32) <= num_cus) hipLaunchKernelGGL((k_block_ring<2, 1>), dim3(cus), dim3(256), 0, s, a);
  else if (count(k64x64) <= num_cus) hipLaunchKernelGGL((k_block_ring<2, 2>), dim3(cus), dim3(256), 0, s, a);
  else if (tiles < kLargeTiles && count(kMid) <= num_cus) hipLaunchKernelGGL((k_block_mid<2, true>), dim3(cus), dim3(kThreads), 0, s, a);
  else if (count(k128x128) <= num_cus) hipLaunchKernelGGL((k_block_mid<4, true>), dim3(cus), dim3(kThreads), 0, s, a);
  else if (tiles < kLargeTiles) hipLaunchKernelGGL((k_block_mid<2, false>), dim3(3 * cus), dim3(kThreads), 0, s, a);
  else {
    // one matrix: up to 16 rows beyond the blocks of 256 are streamed (4097 rows,
    // 115 us; 147 with a half tile for the last row).  17 to 128 rows beyond, and
    // those of groups, are a half tile, which copies 48 of a full one's 64 KiB a
    // stage; where the full tiles fill the CUs' last round it takes one more.
    const int64_t rest = a.offsets == nullptr ? a.M % kBM : 0;
    if (rest <= kFewRows) a.M -= rest;
    hipLaunchKernelGGL(k_block_mma, dim3(cus), dim3(kThreads), 0, s, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.M == args.M) return err;
    a.m_first = a.M;
    a.M = args.M;
    hipLaunchKernelGGL(k_block_few, dim3((unsigned)units), dim3(kThreads), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace mm
