// How the products cut their rows and columns into tiles and find them: one
// matrix, or groups of rows with a matrix each.  Args: offsets, counts, M, N, G
// as in BlockArgs and Int8Args.
#pragma once
#include "mm_device.hpp"

namespace mm {
namespace {

constexpr int kBM = 256, kBN = 256;       // the large tile
constexpr int kMidBM = 128, kMidBN = 64;  // the small tile
constexpr int kGroupM = 6;                // M-blocks that a run of tiles goes through before the next N-block


__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// rows of group gi, clipped to the matrix
template <typename Args>
__device__ __forceinline__ void group_rows(const Args& a, int gi, int64_t& lo, int64_t& n) {
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
template <typename Args>
__device__ int64_t count_blocks(const Args& a, int c) {
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
// requests wait 500 cycles on average, and how many find L2 decides the rate
// (block-scaled product):
// 16384 x 4096 x 7168 takes 424 us (482 with 64 M-blocks first), 16384 x 7168 x
// 2048 270 us (280 with 8, 292 with 64).
template <typename Args>
__device__ bool find_tile(const Args& a, int c, int64_t at, TileAt& o) {
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

}  // namespace
}  // namespace mm
