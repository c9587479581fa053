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

struct TileAt {
  int64_t m0, rows;    // first row of the tile, rows of its group from there
  int group, n0;
};

// Finds tile `at` of the list (group, N-block, M-block: M fastest) among the
// groups, 64 at a time; every lane of the wave takes part.  Returns false
// past the end.
template <int BM, int BN>
__device__ bool find_tile(const BlockArgs& a, int64_t at, TileAt& o) {
  const int nb = (a.N + BN - 1) / BN;
  const int l = lane_id();
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    int64_t lo = 0, n = 0;
    if (g0 + l < a.G) group_rows(a, g0 + l, lo, n);
    const int64_t mine = (n + BM - 1) / BM * nb;
    int64_t pre = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t v = __shfl_up(pre, d, 64);
      if (l >= d) pre += v;
    }
    const int64_t all = __shfl(pre, 63, 64);
    if (at < all) {
      const uint64_t m = ballot(at < pre);
      const int src = __ffsll((unsigned long long)m) - 1;
      const int64_t first = __shfl(pre - mine, src, 64), rows = __shfl(n, src, 64), row0 = __shfl(lo, src, 64);
      const int64_t mb = (rows + BM - 1) / BM, k = at - first;
      o.group = g0 + src;
      o.n0 = (int)(k / mb) * BN;
      o.m0 = row0 + (k % mb) * BM;
      o.rows = rows - (k % mb) * BM;
      return true;
    }
    at -= all;
  }
  return false;
}

}  // namespace

// 128 rows x 128 columns, 4 waves of 64 x 64, one group of 128 K-values per
// stage, two LDS stages.
__global__ __launch_bounds__(256) void k_block_tile(BlockArgs a) {
  constexpr int BM = 128, BN = 128;
  __shared__ __attribute__((aligned(16))) u32x4 sa[2][BM * 8], sb[2][BN * 8];
  const int tid = threadIdx.x, w = tid / 64, l = tid % 64, r = l % 16, g = l / 16;
  const int wm = w % 2, wn = w / 2, KB = a.K / kBlock;
  for (int64_t at = blockIdx.x;; at += gridDim.x) {
    TileAt t;
    if (!find_tile<BM, BN>(a, at, t)) break;
    const uint8_t *ap[4], *bp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 32 + tid / 8;
      ap[i] = a.a + (t.m0 + (row < t.rows ? row : 0)) * a.K + (tid % 8) * 16;
      const int n = t.n0 + row;
      bp[i] = a.b + ((int64_t)t.group * a.N + (n < a.N ? n : a.N - 1)) * a.K + (tid % 8) * 16;
    }
    const float* asp[4];
    int64_t tok[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = wm * 64 + i * 16 + r;
      tok[i] = row < t.rows ? t.m0 + row : -1;
      asp[i] = a.as + (t.m0 + (row < t.rows ? row : 0)) * KB;
    }
    const int nb = (t.n0 + wn * 64) / kBlock, nblocks = (a.N + kBlock - 1) / kBlock;
    const float* bsp = a.bs + ((int64_t)t.group * nblocks + (nb < nblocks ? nb : nblocks - 1)) * KB;
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 ra[4], rb[4];
    auto fetch = [&](int kb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ra[i] = *reinterpret_cast<const u32x4*>(ap[i] + (int64_t)kb * kBlock);
        rb[i] = *reinterpret_cast<const u32x4*>(bp[i] + (int64_t)kb * kBlock);
      }
    };
    auto put = [&](int st) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i * 32 + tid / 8, c = (tid % 8) ^ (row % 8);
        sa[st][row * 8 + c] = ra[i];
        sb[st][row * 8 + c] = rb[i];
      }
    };
    fetch(0);
    put(0);
    __syncthreads();
    for (int kb = 0; kb < KB; ++kb) {
      if (kb + 1 < KB) fetch(kb + 1);
      float sc[4];
      const float bscale = bsp[kb];
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = asp[i][kb] * bscale;
      const u32x4 *A = sa[kb & 1], *B = sb[kb & 1];
      u32x4 bf[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = wn * 64 + j * 16 + r;
        bf[j][0] = B[row * 8 + ((2 * g) ^ (row % 8))];
        bf[j][1] = B[row * 8 + ((2 * g + 1) ^ (row % 8))];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = wm * 64 + i * 16 + r;
        const u32x4 a0 = A[row * 8 + ((2 * g) ^ (row % 8))], a1 = A[row * 8 + ((2 * g + 1) ^ (row % 8))];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += mfma128(bf[j][0], bf[j][1], a0, a1) * sc[i];
      }
      if (kb + 1 < KB) put((kb + 1) & 1);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = t.n0 + wn * 64 + j * 16 + 4 * g;
        if (tok[i] >= 0 && n < a.N)
          *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + tok[i] * a.N + n) =
              u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
      }
  }
}

hipError_t launch_block_gemm(const BlockArgs& a, int num_cus, hipStream_t s) {
  const int64_t tiles = ((a.M + 127) / 128 + (a.offsets ? a.G : 0)) * ((a.N + 127) / 128);
  const int64_t most = 2 * (int64_t)num_cus;
  hipLaunchKernelGGL(k_block_tile, dim3((unsigned)(tiles < most ? tiles : most)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mm
