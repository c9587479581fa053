// Router: scores of every expert for every token, then each token's top-k.
//
//   z = x . Wr^T            (bf16 operands, float32 sums on the bf16 MFMA)
//   softmax: z += bias,  score = softmax(z),  ranking by z
//   sigmoid: score = 1 / (1 + e^-z),  ranking by score + bias (by z without)
//
// Two kernels: k_router_scores writes partial scores (the hidden dimension
// cut into KS slices so that a single token still occupies many CUs), and
// k_router_select adds them and selects, one wave per token.
//
// The order of two experts is decided by their 64-bit scores, and a float32
// score carries a bound on its error.  The MFMA takes 8 products at a time: it
// cuts each below 2^-24 of the power of two of the largest one (7 * 2^-24 of that
// one at most) and adds the eight to the accumulator with one rounding, of at
// most 2^-24 of the sum that results.  The roundings need not be independent:
// where a large partial sum takes in small products of one sign, all go the same
// way (a value of 1, then eights just below half of its ulp: 446 steps of 2^-23
// are lost at hidden 7168).  So they are added up.  With m_z the largest partial
// sum of a token and tile of experts that the kernels saw in slice z: 4 roundings
// an MFMA of the m_z, and those of the sums over waves and slices.  A partial
// sum between two looks is off the nearer one by at most half of the products
// between them: 4 * (MFMAs between looks) / 2 of |x| |w|, beside the 7 of the
// cut products (launch_router_select).  No partial sum is above |x| |w|, which
// takes the place of the m_z where a NaN or an infinity of another expert of the
// tile hides them.  Where two experts are closer than their bounds, both are
// summed again in 64 bits.
#include <type_traits>

#include "mm_router_dev.hpp"

namespace mm {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kRouterStep = 64;       // hidden values per step of a wave (two MFMAs)

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float sumsq(const u32x4& v, float acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = v[i];     // a value: the cast of a vector's element takes the vector's first
    acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, u), __builtin_bit_cast(bf16x2, u), acc, false);
  }
  return acc;
}

// The larger of two magnitudes by their bits, among which a NaN is the largest:
// the selection has to learn that it hides the others (fmaxf would drop it).
__device__ __forceinline__ float larger(float a, float b) {
  const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  return x > y ? a : b;
}

// The largest magnitude of many floats from their bits: the largest positive
// one in signed order, the largest negative one in unsigned order, half an
// instruction a value each.
struct Largest {
  int32_t pos = 0;
  uint32_t neg = 0x80000000u;
  __device__ __forceinline__ void see(const f32x4& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = v[i];
      const int32_t b = __builtin_bit_cast(int32_t, f);
      pos = b > pos ? b : pos;
      neg = (uint32_t)b > neg ? (uint32_t)b : neg;
    }
  }
  __device__ __forceinline__ float value() const { return larger(__uint_as_float((uint32_t)pos), __uint_as_float(neg & 0x7fffffffu)); }
};

}  // namespace

// TT x ET tiles of 16 tokens x 16 experts a wave; the 8 waves share the hidden
// dimension and are added in LDS in a fixed order.
// Lane l of a tile holds 8 consecutive hidden values of expert (A) and token
// (B) l % 16; accumulator i is expert 4 * (l / 16) + i of token l % 16.
template <int TT, int ET>
__global__ __launch_bounds__(kThreads) void k_router_scores(RouterArgs a) {
  constexpr int KW = kWaves, kSlots = KW / 2;
  __shared__ f32x4 red[kSlots][TT * ET][64];
  __shared__ float xn[KW][TT * 16], xm[KW][TT * 16], wn[KW][ET * 16];
  const int kw = threadIdx.x / 64, l = threadIdx.x % 64, r = l % 16, g = l / 16;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * TT);
  const int e0 = (int)blockIdx.y * (16 * ET);
  const uint8_t *xp[TT], *wp[ET];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int64_t t = t0 + 16 * i + r;
    xp[i] = static_cast<const uint8_t*>(a.x) + (t < a.T ? t : a.T - 1) * a.H * 2 + g * 32;
  }
#pragma unroll
  for (int j = 0; j < ET; ++j) {
    const int e = e0 + 16 * j + r;
    wp[j] = static_cast<const uint8_t*>(a.w) + (int64_t)(e < a.E ? e : a.E - 1) * a.H * 2 + g * 32;
  }
  f32x4 acc[TT][ET];
  float xs[TT], ws[ET];
  Largest most[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) xs[i] = 0.0f;
  auto look = [&]() {
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int j = 0; j < ET; ++j) most[i].see(acc[i][j]);
  };
#pragma unroll
  for (int j = 0; j < ET; ++j) ws[j] = 0.0f;
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int j = 0; j < ET; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const bool do_x = blockIdx.y == 0, do_w = blockIdx.x == 0;
  const int steps = a.H / kRouterStep, q = (int)blockIdx.z * KW + kw, Q = KW * a.KS;
  for (int s = q; s < steps; s += Q) {
    u32x4 xv[TT][2], wv[ET][2];
#pragma unroll
    for (int j = 0; j < ET; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) wv[j][h] = *reinterpret_cast<const u32x4*>(wp[j] + (int64_t)s * (kRouterStep * 2) + h * 16);
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) xv[i][h] = *reinterpret_cast<const u32x4*>(xp[i] + (int64_t)s * (kRouterStep * 2) + h * 16);
    look();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < ET; ++j) acc[i][j] = mfma16(wv[j][h], xv[i][h], acc[i][j]);
    if (do_x) {
#pragma unroll
      for (int i = 0; i < TT; ++i) xs[i] = sumsq(xv[i][1], sumsq(xv[i][0], xs[i]));
    }
    if (do_w) {
#pragma unroll
      for (int j = 0; j < ET; ++j) ws[j] = sumsq(wv[j][1], sumsq(wv[j][0], ws[j]));
    }
  }
  look();
  // squared norms and largest partial sums: the four lane groups of a row, then the KW waves
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    float v = xs[i], m = most[i].value();
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    m = larger(m, __shfl_xor(m, 16, 64));
    m = larger(m, __shfl_xor(m, 32, 64));
    if (g == 0) xn[kw][16 * i + r] = v, xm[kw][16 * i + r] = m;
  }
#pragma unroll
  for (int j = 0; j < ET; ++j) {
    float v = ws[j];
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    if (g == 0) wn[kw][j * 16 + r] = v;
  }
#pragma unroll
  for (int h = KW / 2; h >= 1; h /= 2) {
    if (kw >= h && kw < 2 * h) {
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < ET; ++j) red[kw - h][i * ET + j][l] = acc[i][j];
    }
    __syncthreads();
    if (kw < h) {
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < ET; ++j) acc[i][j] += red[kw][i * ET + j][l];
    }
    __syncthreads();
  }
  float* part = a.part + (int64_t)blockIdx.z * a.T * a.Ep;
  if (kw == 0) {
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int64_t t = t0 + 16 * i + r;
#pragma unroll
      for (int j = 0; j < ET; ++j) {
        const int e = e0 + 16 * j + 4 * g;
        if (t < a.T && e < a.Ep) *reinterpret_cast<f32x4*>(part + t * a.Ep + e) = acc[i][j];
      }
    }
  }
  if ((int)threadIdx.x < 16 * TT && t0 + threadIdx.x < a.T) {
    float v = 0.0f, m = 0.0f;
#pragma unroll
    for (int k = 0; k < KW; ++k) v += xn[k][threadIdx.x], m = larger(m, xm[k][threadIdx.x]);
    if (blockIdx.y == 0) a.xnorm[(int64_t)blockIdx.z * a.T + t0 + threadIdx.x] = v;
    a.xmost[((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * a.T + t0 + threadIdx.x] = m;
  }
  if (do_w && (int)threadIdx.x < ET * 16) {
    const int e = (int)blockIdx.y * (16 * ET) + threadIdx.x;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < KW; ++k) v += wn[k][threadIdx.x];
    if (e < a.Ep) a.wnorm[(int64_t)blockIdx.z * a.Ep + e] = v;
  }
}

typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kTileE = 256;

// The same for many tokens and experts: 32 * TT tokens x 256 experts a
// workgroup (8 waves of 16 * TT x 64), stages of 64 hidden values filled by
// LDS-DMA two stages ahead, in three slots (TT = 8: Wr, which mostly comes from
// L2, one stage ahead in two; tokens one stage ahead: 70 for 67 us).
// Bound: the copies, of which a CU takes 36 to 40 bytes a ns: 2.8 MB a CU with
// TT = 4 at 16384 x 256 x 7168, 1.9 MB with 8, where the 64 tiles take four slices
// for two and twice the partial scores, 67 MB, are written behind the last
// stage (69 / 71 us; in one slice, 33000 x 256, 227 / 195).  Looking for the largest
// partial sum costs 5 of 72 us at every third stage, 12 of 79 at each.
template <int TT>
__device__ __forceinline__ void router_tile(const RouterArgs& a, uint8_t* x0, uint8_t* w0, uint8_t* x1, uint8_t* w1,
                                            uint8_t* x2, uint8_t* w2) {
  constexpr int kTileT = 32 * TT;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid / 64), l = tid % 64, r = l % 16, g = l / 16;
  const int wt = w % 2, we = w / 2;              // wave's 16 * TT tokens and 64 experts
  // workgroup b runs on XCD b % 8: an XCD keeps to one slice of the hidden
  // dimension, so that slice of Wr stays in its L2
  const int per = 8 / a.KS, z = (int)(blockIdx.x % 8) / per;
  const int64_t tile = (int64_t)(blockIdx.x / 8) * per + blockIdx.x % per;
  const int64_t t0 = tile * kTileT;
  if (t0 >= a.T) return;
  const int e0 = (int)blockIdx.y * kTileE;
  const int rows = (int)(a.T - t0 < kTileT ? a.T - t0 : kTileT), cols = a.E - e0 < kTileE ? a.E - e0 : kTileE;
  const int steps = a.H / 64, s0 = steps * z / a.KS, s1 = steps * (z + 1) / a.KS;
  const int pitch = a.H * 2;
  // one instruction moves 8 rows of 128 bytes; the chunk at place p of row y is p ^ (y / 2 % 8)
  const uint32_t voff = (uint32_t)(l / 8) * pitch + (((l % 8) ^ ((4 * (w % 2) + l / 16) % 8)) * 16);
  const uint8_t *xb = static_cast<const uint8_t*>(a.x) + t0 * pitch, *wb = static_cast<const uint8_t*>(a.w) + (int64_t)e0 * pitch;
  constexpr int kCopies = (kTileT + kTileE) / 64;
  auto copy = [&](int i, int s, uint8_t* xs, uint8_t* ws) {
    const int at = (s < s1 ? s : s1 - 1) * 128;  // past the end: the last stage again, unused
    const bool of_x = i < kTileT / 64;
    const int grp = w + 8 * (of_x ? i : i - kTileT / 64);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)(of_x ? xb : wb), (short)0, (of_x ? rows : cols) * pitch, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)((of_x ? xs : ws) + grp * 1024), 16, voff, grp * 8 * pitch + at, 0, 0);
  };
  f32x4 acc[4][TT];                              // [expert tile][token tile]
  float xs2[TT / 4], ws2[4];
  Largest most[TT];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ws2[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
#pragma unroll
  for (int j = 0; j < TT / 4; ++j) xs2[j] = 0.0f;
  // squared norms: of the tokens a quarter by each of the four waves that hold them
  const bool do_x = blockIdx.y == 0, do_w = tile == 0 && wt == 0;
  const int sw = (r / 2) % 8;
  // the copies of stages nsx (x) and nsw (Wr) go out two at a time among the first products, Wr's before x's
  auto compute = [&](const uint8_t* xs, const uint8_t* ws, int nsx, uint8_t* nx, int nsw, uint8_t* nw) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = ((4 * h + g) ^ sw) * 16 + r * 128;
      u32x4 xf[TT], wf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) wf[i] = *reinterpret_cast<const u32x4*>(ws + (we * 4 + i) * 2048 + c);
#pragma unroll
      for (int i = 0; i < TT; ++i) xf[i] = *reinterpret_cast<const u32x4*>(xs + (wt * TT + i) * 2048 + c);
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        if (h == 0 && 2 * j < kCopies) {
          const int i = (2 * j + kTileT / 64) % kCopies;
          copy(i, i < kTileT / 64 ? nsx : nsw, nx, nw);
          copy(i + 1, i < kTileT / 64 ? nsx : nsw, nx, nw);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = mfma16(wf[i], xf[j], acc[i][j]);
        if (do_x && j / (TT / 4) == we) xs2[j % (TT / 4)] = sumsq(xf[j], xs2[j % (TT / 4)]);
      }
      if (do_w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ws2[i] = sumsq(wf[i], ws2[i]);
      }
    }
  };
  // `look`: every third stage, six MFMAs
  const std::true_type yes;
  const std::false_type no;
  auto turn = [&](auto look) {
    // the stage's products stay before the wait: nothing else ties them to it
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) asm volatile("" : "+v"(acc[i][j]));
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (decltype(look)::value) {
#pragma unroll
      for (int j = 0; j < TT; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) most[j].see(acc[i][j]);
        asm volatile("" : "+v"(most[j].pos), "+v"(most[j].neg));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // all copies but the newest stage's (TT = 8: its x)
    stage_barrier<TT == 4 ? kCopies : kTileT / 64>();
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int i = 0; i < kCopies; ++i) copy(i, s0, x0, w0);
#pragma unroll
  for (int i = 0; i < (TT == 4 ? kCopies : kTileT / 64); ++i) copy(i, s0 + 1, x1, w1);
  turn(no);
  if constexpr (TT == 4) {
    // (a break inside the loop would be a path on which the compiler sees a
    // slot filled one stage ago, and waits for it)
    int s = s0;
    for (; s + 2 < s1; s += 3) {
      compute(x0, w0, s + 2, x2, s + 2, w2);
      turn(no);
      compute(x1, w1, s + 3, x0, s + 3, w0);
      turn(no);
      compute(x2, w2, s + 4, x1, s + 4, w1);
      turn(yes);
    }
    if (s < s1) {
      compute(x0, w0, s + 2, x2, s + 2, w2);
      turn(yes);
    }
    if (s + 1 < s1) {
      compute(x1, w1, s + 3, x0, s + 3, w0);
      turn(yes);
    }
  } else {
    int s = s0;
    for (; s + 5 < s1; s += 6) {
      compute(x0, w0, s + 2, x2, s + 1, w1);
      turn(no);
      compute(x1, w1, s + 3, x0, s + 2, w0);
      turn(no);
      compute(x2, w0, s + 4, x1, s + 3, w1);
      turn(yes);
      compute(x0, w1, s + 5, x2, s + 4, w0);
      turn(no);
      compute(x1, w0, s + 6, x0, s + 5, w1);
      turn(no);
      compute(x2, w1, s + 7, x1, s + 6, w0);
      turn(yes);
    }
    if (s < s1) {
      compute(x0, w0, s + 2, x2, s + 1, w1);
      turn(yes);
    }
    if (s + 1 < s1) {
      compute(x1, w1, s + 3, x0, s + 2, w0);
      turn(yes);
    }
    if (s + 2 < s1) {
      compute(x2, w0, s + 4, x1, s + 3, w1);
      turn(yes);
    }
    if (s + 3 < s1) {
      compute(x0, w1, s + 5, x2, s + 4, w0);
      turn(yes);
    }
    if (s + 4 < s1) {
      compute(x1, w0, s + 6, x0, s + 5, w1);
      turn(yes);
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);            // no copy outlives the workgroup
  __syncthreads();                               // the stages are free
  float* xm = reinterpret_cast<float*>(x0);      // [4][kTileT]: largest partial sums
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    float m = most[j].value();
    m = larger(m, __shfl_xor(m, 16, 64));
    m = larger(m, __shfl_xor(m, 32, 64));
    if (g == 0) xm[we * kTileT + (wt * TT + j) * 16 + r] = m;
  }
  __syncthreads();
  if (tid < rows)
    a.xmost[((int64_t)z * gridDim.y + blockIdx.y) * a.T + t0 + tid] =
        larger(larger(xm[tid], xm[kTileT + tid]), larger(xm[2 * kTileT + tid], xm[3 * kTileT + tid]));
  float* part = a.part + (int64_t)z * a.T * a.Ep;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int t = (wt * TT + j) * 16 + r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + (we * 4 + i) * 16 + 4 * g;
      if (t < rows && e < a.Ep) *reinterpret_cast<f32x4*>(part + (t0 + t) * a.Ep + e) = acc[i][j];
    }
  }
  if (do_x) {
#pragma unroll
    for (int j = 0; j < TT / 4; ++j) {
      float v = xs2[j];
      v += __shfl_xor(v, 16, 64);
      v += __shfl_xor(v, 32, 64);
      const int t = (wt * TT + we * (TT / 4) + j) * 16 + r;
      if (g == 0 && t < rows) a.xnorm[(int64_t)z * a.T + t0 + t] = v;
    }
  }
  if (do_w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = ws2[i];
      v += __shfl_xor(v, 16, 64);
      v += __shfl_xor(v, 32, 64);
      const int e = e0 + (we * 4 + i) * 16 + r;
      if (g == 0 && e < a.Ep) a.wnorm[(int64_t)z * a.Ep + e] = v;
    }
  }
}

// separate arrays: the compiler then sees that a stage's reads and the next
// stages' copies do not meet, and does not wait for the copies
__global__ __launch_bounds__(kThreads) void k_router_tile128(RouterArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t x0[128 * 128], x1[128 * 128], x2[128 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t w0[kTileE * 128], w1[kTileE * 128], w2[kTileE * 128];
  router_tile<4>(a, x0, w0, x1, w1, x2, w2);
}
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_router_tile256(RouterArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t x0[256 * 128], x1[256 * 128], x2[256 * 128], w0[kTileE * 128], w1[kTileE * 128];
  router_tile<8>(a, x0, w0, x1, w1, x2, nullptr);
}

// One wave per token.  (Four tokens a wave in turn, the next one's scores
// asked for meanwhile, took 58 against 43 us at 16384 x 256: a token that needs
// 64-bit sums then holds up three others.)  Bound: issue, about 500
// instructions a token, and the latency of the scores: 50 us at 16384 x 256
// (20 without the turns that select, 33 without the 64-bit sums of one token in
// 20).
template <int NV, int KM>
__global__ __launch_bounds__(256, NV <= 4 ? 4 : 1) void k_router_select(RouterArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  if (t >= a.T) return;
  RouterExperts<NV> ex;
  RouterToken<NV> tok;
  router_load_token<NV, KM>(a, t, tok);
  router_load_experts<NV, KM>(a, ex);
  int id;
  float w;
  router_select_token<NV>(a, t, ex, tok, id, w);
  const int l = lane_id();
  if (l < a.K) {
    a.ids[t * a.K + l] = id;
    a.weights[t * a.K + l] = w;
  }
}

// With few tokens or few scores in all, the scores are a stream of Wr: 16 x 16
// tiles over as many workgroups as the hidden dimension gives (us for both
// kernels, 16 x 16 / 64 x 64 a wave, hidden 7168: 333 tokens x 32 experts
// 18 / 23, 500 x 64 22 / 25, 1000 x 32 24 / 25, 1000 x 64 28 / 25, 4000 x 32
// 43 / 33).  Beyond, with up to 64 experts, a wave holds 64 x 64 and the waves
// share the hidden dimension; with more experts the LDS tiles (64 x 64 a wave /
// tiles of 128 x 256: 16384 x 32 83 / 87, 16384 x 64 93 / 91, 2000 x 128 40 / 37,
// 16384 x 128 152 / 98).  Tiles of 256 x 256 where those of 128 x 256 fill half of
// the CUs in one slice and each of theirs gets 24 stages or more (tiles of 128 /
// 256 rows, hidden 7168: 2000 x 256 44 / 57, 10000 x 256 95 / 98, 16384 x 128
// 99 / 102, 16384 x 256 117 / 125, 20000 x 256 165 / 160, 33000 x 256 309 / 275,
// 65536 x 128 334 / 316; hidden 4096: 16384 x 256 84 / 97, 33000 x 256 200 / 184,
// 8192 x 512 81 / 103; hidden 2048: 33000 x 128 117 / 110, 65536 x 128 169 / 172).
// The counts are those of a device of 256 CUs.
RouterShape router_shape(int64_t T, int H, int E) {
  RouterShape s{};
  const int steps = H / kRouterStep;
  s.ep = (E + 15) / 16 * 16;
  s.eb = 16;
  if (T <= 64 || T * E <= 32768) {
    s.wide = 0;
    s.ks = steps / (kWaves * 2);   // two steps a wave, four: 9.4, 10.1 us for both kernels at 1 x 32 x 7168
    s.ks = s.ks < 1 ? 1 : s.ks > 8 ? 8 : s.ks;
    return s;
  }
  // slices that fill the CUs with `tiles`, of `least` steps at least
  auto slices = [&](int64_t tiles, int least) {
    int64_t n = 256 / tiles;
    n = n < steps / least ? n : steps / least;
    return (int)(n < 1 ? 1 : n > 8 ? 8 : n);
  };
  if (E <= 64) {
    s.wide = 1;
    s.eb = 64;
    s.ks = slices((T + 63) / 64, 2 * kWaves);
    return s;
  }
  s.eb = kTileE;
  const int64_t cols = (E + kTileE - 1) / kTileE;
  for (s.wide = 3;; s.wide = 2) {
    const int rows = s.wide == 3 ? 256 : 128;
    const int64_t tiles = (T + rows - 1) / rows * cols;
    const int n = slices(tiles, 8);
    s.ks = n >= 8 ? 8 : n >= 4 ? 4 : n >= 2 ? 2 : 1;   // whole XCDs to a slice
    if (s.wide == 2 || ((T + 127) / 128 * cols > 128 && steps / s.ks >= 24)) return s;
  }
}

hipError_t launch_router_scores(const RouterArgs& a, hipStream_t s) {
  const RouterShape sh = router_shape(a.T, a.H, a.E);
  if (sh.wide == 0) {
    const dim3 grid((unsigned)((a.T + 15) / 16), (unsigned)(a.Ep / 16), (unsigned)a.KS);
    hipLaunchKernelGGL((k_router_scores<1, 1>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  if (sh.wide >= 2) {
    const int rows = sh.wide == 3 ? 256 : 128;
    const int64_t tiles = (a.T + rows - 1) / rows, per = 8 / a.KS;
    const dim3 grid((unsigned)((tiles + per - 1) / per * 8), (unsigned)((a.E + kTileE - 1) / kTileE));
    if (sh.wide == 3) hipLaunchKernelGGL(k_router_tile256, grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(k_router_tile128, grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_router_scores<4, 4>), dim3((unsigned)((a.T + 63) / 64), 1, (unsigned)a.KS), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

namespace {

template <int NV>
hipError_t run_select(const RouterArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + 3) / 4));
  if (a.KS <= 2) hipLaunchKernelGGL((k_router_select<NV, 2>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_router_select<NV, 8>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_router_select(const RouterArgs& args, hipStream_t s) {
  RouterArgs a = args;
  const int steps = a.H / kRouterStep;           // of two MFMAs
  if (a.EB == kTileE) {
    // a slice is one chain; the slices are added one after the other
    a.of_sums = (float)(8 * ((steps + a.KS - 1) / a.KS) + a.KS - 1);
    a.of_products = 8 + 2 * 6;                   // a look every six MFMAs
  } else {
    // a slice is eight chains, added in pairs (4 sums of 2 m, 2 of 4 m, one of 8 m)
    a.of_sums = (float)(8 * kWaves * ((steps + kWaves * a.KS - 1) / (kWaves * a.KS)) + 24 + kWaves * (a.KS - 1));
    a.of_products = 8 + 2 * 2;                   // a look every two
  }
  if (a.E <= 64) return run_select<1>(a, s);
  if (a.E <= 128) return run_select<2>(a, s);
  if (a.E <= 256) return run_select<4>(a, s);
  if (a.E <= 512) return run_select<8>(a, s);
  return run_select<16>(a, s);
}

}  // namespace mm
