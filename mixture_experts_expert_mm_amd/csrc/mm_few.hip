// The routed-expert layer for at most 64 tokens: kernels that stream the live
// experts' weights from HBM into MFMA operands.
//
//   Linear1: A[r] = SwiGLU(x_t . W1[e]) for every route r = (t, k), e = id(r)
//   Linear2: y[t] = sum over t's routes of g_r * (A[r] . W2[e])
//
// Weights are the A operand of the 16 x 16 x 32 MFMA (16 weight rows), up to
// 16 routes of one expert its B operand, so a weight byte is read once
// whatever the number of tokens (twice in Linear2 of a float32 y, for an expert
// with more than 32 routes).  e4m3 weights are widened exactly to bf16
// (activations are not quantised); float32 accumulators.  A is held in bf16
// parts: one when y is bf16, whose own rounding is as large; three, the whole
// float, when y is float32.
// Up to 16 tokens k_few_l1 and k_few_l2 stream the weights into registers;
// with more, or (Linear2) a float32 y, k_few_tile brings them through LDS and
// k_few_combine adds a token's contributions.  Bound: HBM.
#include <type_traits>

#include "mm_device.hpp"
#include "mm_ops_internal.hpp"

namespace mm {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxT = 64, kMaxE = 1024, kMaxK = 32;
constexpr int kStreamT = 16;           // most tokens of the streaming kernels: one MFMA of routes an expert
constexpr int kStage = 128;            // K-values per stage of a wave

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// 8 e4m3 -> 8 bf16, exact
__device__ __forceinline__ u32x4 widen8(uint32_t w0, uint32_t w1) {
#define CVT(x, hi_) __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((x), 1.0f, (hi_)))
  return u32x4{CVT(w0, false), CVT(w0, true), CVT(w1, false), CVT(w1, true)};
#undef CVT
}

// The tokens of each expert as bit masks, by every workgroup for itself: a
// few thousand ids at most, which cost less than a kernel of their own.
// Returns whether some token names an expert twice.
__device__ __forceinline__ bool mark_tokens(const FewArgs& a, unsigned long long* tokens, int32_t& twice) {
  const int tid = threadIdx.x, Et = a.E + a.S, n = a.T * a.K;
  for (int e = tid; e < Et; e += kThreads) tokens[e] = 0;
  if (tid == 0) twice = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int t = i / a.K, id = a.ids[i];
    if (id >= 0 && id < a.E && (a.active == nullptr || a.active[t] != 0) &&
        (atomicOr(&tokens[id], 1ull << t) >> t & 1))
      twice = 1;
  }
  if (a.S && tid < a.T && (a.active == nullptr || a.active[tid] != 0)) atomicOr(&tokens[a.E], 1ull << tid);
  __syncthreads();
  return twice != 0;
}

// Whether (t, k) is the route of its expert: the first k of t that names it.
// Its weight is then the sum over all k that do, in their order.
__device__ __forceinline__ bool first_route(const FewArgs& a, bool twice, int t, int k, int id, float& gate) {
  gate = a.weights[t * a.K + k];
  if (!twice) return true;
  for (int j = 0; j < a.K; ++j)
    if (j != k && a.ids[t * a.K + j] == id) {
      if (j < k) return false;
      gate += a.weights[t * a.K + j];
    }
  return true;
}

// The routes of a batch grouped by expert, in LDS.
struct Lists {
  unsigned long long tokens[kMaxE];            // tokens of each expert, one bit each
  int32_t route[kStreamT * (kMaxK + 1)];       // list: route t * (K + S) + k, by expert and token
  float gate[kStreamT * (kMaxK + 1)];
  int16_t token[kStreamT * (kMaxK + 1)];
  int16_t expert[kMaxE];       // live experts, ascending
  int16_t start[kMaxE + 1];    // first list entry of each live expert
  int16_t first[kMaxE];        // first list entry of expert e
  int32_t live, twice;
};

// A route's place among its expert's is the number of earlier tokens in the
// expert's mask: the order does not depend on how the atomics arrive.
__device__ void build_lists(const FewArgs& a, Lists& L) {
  const int tid = threadIdx.x, Et = a.E + a.S, n = a.T * a.K;
  const bool twice = mark_tokens(a, L.tokens, L.twice);
  if (tid < 64) {
    int live = 0, at = 0;
    for (int e0 = 0; e0 < Et; e0 += 64) {
      const int e = e0 + tid, c = e < Et ? __popcll(L.tokens[e]) : 0;
      const uint64_t m = ballot(c > 0);
      int pre = c;             // routes of the experts up to this one
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(pre, o, 64);
        if (tid >= o) pre += v;
      }
      if (c > 0) {
        const int p = live + __popcll((unsigned long long)(m & lanemask_lt()));
        L.expert[p] = (int16_t)e;
        L.start[p] = L.first[e] = (int16_t)(at + pre - c);
      }
      live += __popcll((unsigned long long)m);
      at += __shfl(pre, 63, 64);
    }
    if (tid == 0) {
      L.live = live;
      L.start[live] = (int16_t)at;
    }
  }
  __syncthreads();
  auto place = [&](int e, int t, int k, float gate) {
    const int p = L.first[e] + __popcll(L.tokens[e] & ((1ull << t) - 1));
    L.route[p] = t * (a.K + a.S) + k;
    L.gate[p] = gate;
    L.token[p] = (int16_t)t;
  };
  for (int i = tid; i < n; i += kThreads) {
    const int t = i / a.K, id = a.ids[i];
    float gate;
    if (id >= 0 && id < a.E && (a.active == nullptr || a.active[t] != 0) && first_route(a, twice, t, i % a.K, id, gate))
      place(id, t, i % a.K, gate);
  }
  if (a.S && tid < a.T && (a.active == nullptr || a.active[tid] != 0)) place(a.E, tid, a.K, 1.0f);
  __syncthreads();
}

// One stage of a wave: WT tiles of 16 weight rows and 16 routes in P parts,
// 128 K-values.  A lane's 16-byte pieces of a weight row and of a route's row
// cover the same K-values in the same order.
template <int F, int WT, int P>
struct Stage {
  static constexpr int WL = F == MM_FEW_BF16 ? 4 : 2;
  u32x4 w[WT][WL];
  u32x4 b[P][4];
  float s[WT];
};

template <int F> constexpr int weight_bytes() { return F == MM_FEW_BF16 ? 2 : 1; }
// byte offset of a weight row's piece j of lane group g inside a stage
__device__ __forceinline__ int w_piece(int g, int j) { return 64 * j + 16 * g; }
// bf16 operand piece j (of MFMA j) of lane group g: the K-values that the
// weight piece covers
template <int F> __device__ __forceinline__ int b_piece(int g, int j) {
  return F == MM_FEW_BF16 ? 64 * j + 16 * g : 128 * (j / 2) + 32 * g + 16 * (j % 2);
}

template <int F, int WT, int P>
__device__ __forceinline__ void load_weights(Stage<F, WT, P>& st, const uint8_t* const (&wp)[WT], int64_t off, int g) {
#pragma unroll
  for (int i = 0; i < WT; ++i)
#pragma unroll
    for (int j = 0; j < Stage<F, WT, P>::WL; ++j)
      st.w[i][j] = *reinterpret_cast<const u32x4*>(wp[i] + off + w_piece(g, j));
}

template <int F, int WT, int P>
__device__ __forceinline__ void multiply(const Stage<F, WT, P>& st, f32x4 (&acc)[WT]) {
#pragma unroll
  for (int i = 0; i < WT; ++i) {
    f32x4 sum = F == MM_FEW_FP8_BLOCK ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 w = F == MM_FEW_BF16 ? st.w[i][F == MM_FEW_BF16 ? j : 0]
                                       : widen8(st.w[i][F == MM_FEW_BF16 ? 0 : j / 2][2 * (j % 2)], st.w[i][F == MM_FEW_BF16 ? 0 : j / 2][2 * (j % 2) + 1]);
#pragma unroll
      for (int p = 0; p < P; ++p) sum = mfma16(w, st.b[p][j], sum);
    }
    acc[i] = F == MM_FEW_FP8_BLOCK ? acc[i] + sum * st.s[i] : sum;
  }
}

template <int WT>
__device__ __forceinline__ void clear(f32x4 (&acc)[WT]) {
#pragma unroll
  for (int i = 0; i < WT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

__device__ __forceinline__ float swiglu(float g, float u, float clamp) {
  // a NaN stays one (a clamp by min and max would replace it)
  g = g > clamp ? clamp : g < -clamp ? -clamp : g;
  u = u > clamp ? clamp : u < -clamp ? -clamp : u;
  return g / (1.0f + expf(-g)) * u;
}

// bf16 parts of a float whose sum is the float to P * 8 bits
template <int P>
__device__ __forceinline__ void split_bf16(float v, uint16_t (&o)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    o[p] = f32_to_bf16_bits(v);
    const float h = bf16_bits_to_f32(o[p]);
    v = p + 1 < P && h - h == 0.0f ? v - h : 0.0f;   // inf and NaN sit in the first part
  }
}

}  // namespace

// Linear1.  A unit is 16 columns of A of one live expert (16 gate and 16 up
// rows of W1) for all of its routes; the 8 waves share the hidden dimension,
// stage by stage, and their sums meet in LDS.  D stages of a wave are in
// flight, across units.  One token, 7168 x 2048, 8 + 1 experts: 53 us for the
// 264 MB of e4m3 weights (5.0 TB/s), 88 us for bf16 (5.3 TB/s with 8 experts); a
// large copy moves 4.9 TB/s in both directions together.
template <int F, int P, int D>
__global__ __launch_bounds__(kThreads) void k_few_l1(FewArgs a) {
  __shared__ Lists L;
  // two buffers: a unit's sums are read while the next unit's are written
  __shared__ f32x4 red[2][kWaves][2][64];
  build_lists(a, L);
  const int w = uniform(threadIdx.x / 64), l = threadIdx.x % 64, r = l % 16, g = l / 16;
  constexpr int WB = weight_bytes<F>();
  const int nst = a.H / kStage, nsw = (nst + kWaves - 1) / kWaves, cols = a.I / 16;
  const int units = uniform(L.live) * cols;
  const int64_t R = (int64_t)a.T * (a.K + a.S);

  // the next stage to load: stage j of unit u
  struct Cursor {
    int u, j;
    int e, c, n0, n;
    const uint8_t* wp[2];
    const uint8_t* bp;
    const float* sp[2];
  };
  if ((int)blockIdx.x >= units) return;
  // Past the last unit a cursor keeps its pointers: its loads go on, into
  // stages that nothing multiplies.  A load under a condition would make the
  // compiler wait for every load in flight before each product.
  auto aim = [&](Cursor& cu) {
    if (cu.u >= units) return;
    const int le = cu.u / cols;
    cu.c = cu.u % cols;
    cu.e = uniform(L.expert[le]);
    cu.n0 = uniform(L.start[le]);
    cu.n = uniform(L.start[le + 1]) - cu.n0;
    const int row = 64 * (cu.c / 2) + 16 * (cu.c % 2) + r;
    cu.wp[0] = a.w1 + ((int64_t)cu.e * 2 * a.I + row) * a.H * WB;
    cu.wp[1] = cu.wp[0] + (int64_t)32 * a.H * WB;
    cu.bp = static_cast<const uint8_t*>(a.x) + (int64_t)L.token[cu.n0 + (r < cu.n ? r : 0)] * a.H * 2;
    if constexpr (F == MM_FEW_FP8_BLOCK) {
      cu.sp[0] = a.s1 + ((int64_t)cu.e * (2 * a.I / 128) + cu.c / 8) * nst;
      cu.sp[1] = cu.sp[0] + (int64_t)(a.I / 128) * nst;
    }
  };
  auto step = [&](Cursor& cu) {
    if (++cu.j < nsw) return;
    cu.j = 0;
    cu.u += gridDim.x;
    aim(cu);
  };
  auto load = [&](const Cursor& cu, Stage<F, 2, 1>& st) {
    const int js = cu.j * kWaves + w, s = js < nst ? js : nst - 1;
    load_weights<F, 2, 1>(st, cu.wp, (int64_t)s * (kStage * WB), g);
#pragma unroll
    for (int j = 0; j < 4; ++j) st.b[0][j] = *reinterpret_cast<const u32x4*>(cu.bp + (int64_t)s * (kStage * 2) + b_piece<F>(g, j));
    if constexpr (F == MM_FEW_FP8_BLOCK) st.s[0] = cu.sp[0][s], st.s[1] = cu.sp[1][s];
  };

  Cursor ld{}, cu{};
  ld.u = cu.u = blockIdx.x;
  aim(ld);
  aim(cu);
  Stage<F, 2, 1> st[D];
  f32x4 acc[2];
  clear(acc);
  int side = 0;
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load(ld, st[d]);
    if (ld.u < units) step(ld);
  }
  while (cu.u < units) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (cu.u < units && cu.j * kWaves + w < nst) multiply<F, 2, 1>(st[d], acc);
      load(ld, st[d]);
      if (ld.u < units) step(ld);
      if (cu.u < units) {
        if (cu.j + 1 == nsw) {
          // the unit's sums: 8 waves' parts, SwiGLU, A
          red[side][w][0][l] = acc[0];
          red[side][w][1][l] = acc[1];
          clear(acc);
          __syncthreads();
          const float* rf = reinterpret_cast<const float*>(red[side]);
          side ^= 1;
          for (int i = threadIdx.x; i < 16 * cu.n; i += kThreads) {
            // column c of list entry m: accumulator c % 4 of lane 16 * (c / 4) + m
            const int c = i % 16, m = i / 16, at = (16 * (c / 4) + m) * 4 + c % 4;
            float hg = 0.0f, hu = 0.0f;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) {
              hg += rf[k * 512 + at];
              hu += rf[k * 512 + 256 + at];
            }
            const int col = cu.c * 16 + c;
            if constexpr (F == MM_FEW_FP8) {
              hg *= a.s1[(int64_t)cu.e * 2 * a.I + col];
              hu *= a.s1[(int64_t)cu.e * 2 * a.I + a.I + col];
            }
            uint16_t o[P];
            split_bf16<P>(swiglu(hg, hu, a.clamp), o);
            const int64_t route = L.route[cu.n0 + m];
#pragma unroll
            for (int p = 0; p < P; ++p) a.a[(p * R + route) * a.I + col] = o[p];
          }
        }
        step(cu);
      }
    }
  }
}

// Linear2.  A unit is 16 * WT columns of y over every live expert; its
// stages (expert, 128 values of I) are cut into 8 runs, one a wave.  A wave
// adds gate * sum to its own copy of the unit's y in LDS at the end of an
// expert, and the 8 copies are added in order.  One token, 7168 x 2048, 8 + 1
// experts: 29 us for the 132 MB of e4m3 weights, 53 us for bf16 with 8 experts.
template <int F, int WT, int D>
__global__ __launch_bounds__(kThreads) void k_few_l2(FewArgs a) {
  __shared__ Lists L;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  f32x4* ys = reinterpret_cast<f32x4*>(dyn);   // [2][kWaves][T][4 * WT]: one of the two is added and cleared while the other fills
  const int ylen = kWaves * a.T * 4 * WT;
  build_lists(a, L);
  const int w = uniform(threadIdx.x / 64), l = threadIdx.x % 64, r = l % 16, g = l / 16;
  constexpr int WB = weight_bytes<F>();
  const int nst = a.I / kStage;
  const int units = a.H / (16 * WT);
  const int total = uniform(L.live) * nst, nsw = total > kWaves ? (total + kWaves - 1) / kWaves : 1;
  for (int i = threadIdx.x; i < 2 * ylen; i += kThreads) ys[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();

  if (total == 0) {          // no route at all
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.T * a.H; i += gridDim.x * kThreads)
      static_cast<uint16_t*>(a.y)[i] = 0;
    return;
  }
  // this wave's first stage (the last stage for a wave without any: its loads have to go somewhere)
  const int f0 = w * nsw < total ? w * nsw : total - 1;

  struct Cursor {
    int u, j;                  // unit, stage of this wave's run
    int s, le;                 // stage inside the expert, live expert
    int e, n0, n;
    const uint8_t* wp[WT];
    const uint8_t* bp;
    const float* sp[WT];
  };
  auto valid = [&](const Cursor& cu) { return w * nsw + cu.j < total; };
  auto aim = [&](Cursor& cu) {
    if (cu.u >= units) return;
    cu.e = uniform(L.expert[cu.le]);
    cu.n0 = uniform(L.start[cu.le]);
    cu.n = uniform(L.start[cu.le + 1]) - cu.n0;
    const uint8_t* base = a.w2 + (int64_t)cu.e * a.H * a.I * WB;
#pragma unroll
    for (int i = 0; i < WT; ++i) {
      cu.wp[i] = base + (int64_t)((cu.u * WT + i) * 16 + r) * a.I * WB;
      if constexpr (F == MM_FEW_FP8_BLOCK)
        cu.sp[i] = a.s2 + ((int64_t)cu.e * (a.H / 128) + (cu.u * WT + i) / 8) * nst;
    }
    cu.bp = reinterpret_cast<const uint8_t*>(a.a) + (int64_t)L.route[cu.n0 + (r < cu.n ? r : 0)] * a.I * 2;
  };
  auto first = [&](Cursor& cu) {
    cu.j = 0;
    cu.s = f0 % nst;
    cu.le = f0 / nst;
    aim(cu);
  };
  auto step = [&](Cursor& cu) {
    if (++cu.j == nsw) {
      cu.u += gridDim.x;
      first(cu);
    } else if (valid(cu) && ++cu.s == nst) {
      cu.s = 0;
      ++cu.le;
      aim(cu);
    }
  };
  auto load = [&](const Cursor& cu, Stage<F, WT, 1>& st) {
    load_weights<F, WT, 1>(st, cu.wp, (int64_t)cu.s * (kStage * WB), g);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st.b[0][j] = *reinterpret_cast<const u32x4*>(cu.bp + (int64_t)cu.s * (kStage * 2) + b_piece<F>(g, j));
    if constexpr (F == MM_FEW_FP8_BLOCK) {
#pragma unroll
      for (int i = 0; i < WT; ++i) st.s[i] = cu.sp[i][cu.s];
    }
  };

  Cursor ld{}, cu{};
  ld.u = cu.u = blockIdx.x;
  first(ld);
  first(cu);
  Stage<F, WT, 1> st[D];
  f32x4 acc[WT];
  clear(acc);
  int side = 0;
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load(ld, st[d]);
    if (ld.u < units) step(ld);
  }
  while (cu.u < units) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (cu.u < units && valid(cu)) multiply<F, WT, 1>(st[d], acc);
      load(ld, st[d]);
      if (ld.u < units) step(ld);
      if (cu.u < units) {
        const bool last = cu.j + 1 == nsw;
        if (valid(cu) && (last || cu.s + 1 == nst || w * nsw + cu.j + 1 == total)) {
          // end of this wave's part of an expert: gate * sum into its copy of y
          if (r < cu.n) {
            const float gate = L.gate[cu.n0 + r];
            f32x4* y = ys + side * ylen + ((int64_t)w * a.T + L.token[cu.n0 + r]) * (4 * WT) + g;
#pragma unroll
            for (int k = 0; k < WT; ++k) {
              f32x4 v = acc[k];
              if constexpr (F == MM_FEW_FP8)
                v *= *reinterpret_cast<const f32x4*>(a.s2 + (int64_t)cu.e * a.H + (cu.u * WT + k) * 16 + 4 * g);
              y[4 * k] += v * gate;
            }
          }
          clear(acc);
        }
        if (last) {
          __syncthreads();
          // thread: 4 columns of a token
          f32x4* yu = ys + side * ylen;
          side ^= 1;
          for (int i = threadIdx.x; i < a.T * 4 * WT; i += kThreads) {
            f32x4 v = yu[i];
            yu[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 1; k < kWaves; ++k) {
              v += yu[(int64_t)k * a.T * 4 * WT + i];
              yu[(int64_t)k * a.T * 4 * WT + i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            const int64_t at = (int64_t)(i / (4 * WT)) * a.H + cu.u * 16 * WT + (i % (4 * WT)) * 4;
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
          }
        }
        step(cu);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// More tokens: tiles through LDS.  With several routes an expert, the kernels
// above read a route's row again for every 16 columns, and those reads, not
// the weights, fill the vector memory path (64 tokens, e4m3, 32 experts:
// Linear1 264 us for 0.94 GB of weights).  Here a workgroup takes 256 weight
// rows of one expert, 32 a wave, and all of the expert's routes; both come by
// LDS-DMA, 128 bytes of a weight row a stage, two stages ahead (one where
// three stages do not fit LDS).  64 tokens, 7168 x 2048, 32 experts in e4m3:
// Linear1 173 us for 940 MB, Linear2 101 us for 470 MB and the slots, combine 7.5 us.
// Bound: HBM.  (Waiting for every copy at each stage's barrier: 185, 107, 7.5.)
// ---------------------------------------------------------------------------
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kTileRows = 256;         // weight rows of a workgroup

// One live expert of the batch and its routes.
struct ExpertRoutes {
  unsigned long long tokens[kMaxE];
  int32_t route[kMaxT];
  int32_t token[kMaxT];
  float gate[kMaxT];
  int32_t expert, n, twice;
};

// The `index`-th live expert (n = 0 if there are fewer); as build_lists.
__device__ void find_expert(const FewArgs& a, ExpertRoutes& X, int index) {
  const int tid = threadIdx.x, Et = a.E + a.S, n = a.T * a.K;
  if (tid < kMaxT) X.route[tid] = 0, X.token[tid] = 0, X.gate[tid] = 0.0f;
  if (tid == 0) X.n = 0, X.expert = 0;
  const bool twice = mark_tokens(a, X.tokens, X.twice);
  if (tid < 64) {
    int before = 0;
    for (int e0 = 0; e0 < Et; e0 += 64) {
      const bool on = e0 + tid < Et && X.tokens[e0 + tid] != 0;
      const uint64_t m = ballot(on);
      if (on && before + __popcll((unsigned long long)(m & lanemask_lt())) == index) {
        X.expert = e0 + tid;
        X.n = __popcll(X.tokens[e0 + tid]);
      }
      before += __popcll((unsigned long long)m);
    }
  }
  __syncthreads();
  if (X.n == 0) return;
  const int e = X.expert;
  const unsigned long long mine = X.tokens[e];
  auto place = [&](int t, int k, float gate) {
    const int p = __popcll(mine & ((1ull << t) - 1));
    X.route[p] = t * (a.K + a.S) + k;
    X.gate[p] = gate;
    X.token[p] = t;
  };
  if (e < a.E) {
    for (int i = tid; i < n; i += kThreads) {
      const int t = i / a.K;
      float gate;
      if (a.ids[i] == e && (mine >> t & 1) && first_route(a, twice, t, i % a.K, e, gate)) place(t, i % a.K, gate);
    }
  } else if (tid < a.T && (mine >> tid & 1)) {
    place(tid, a.K, 1.0f);
  }
  __syncthreads();
}

// MODE 1: Linear1, A = SwiGLU(x . W1) in P parts; MODE 2: Linear2, gate * (A .
// W2) of every route into its slot, A in P parts.  NT: route tiles of 16 held
// at once (an expert with more goes round again).
template <int F, int MODE, int P, int NT>
__device__ __forceinline__ void few_tile(const FewArgs& a) {
  constexpr int WB = weight_bytes<F>();
  constexpr int VK = 128 / WB;                 // K-values a stage
  constexpr int PB = MODE == 1 ? 1 : P;        // parts of the routes' operand
  constexpr int RB = VK * 2;                   // bytes of a route's row a stage: 256 (e4m3), 128 (bf16)
  constexpr int S = PB * NT <= 4 ? 3 : 2;      // stages in LDS
  constexpr int XB = PB * NT * 16 * RB;        // bytes of the routes' operand a stage
  __shared__ __attribute__((aligned(1024))) uint8_t w0[kTileRows * 128], w1[kTileRows * 128], w2[S == 3 ? kTileRows * 128 : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t x0[XB], x1[XB], x2[S == 3 ? XB : 16];
  __shared__ ExpertRoutes X;
  find_expert(a, X, blockIdx.y);
  const int total = uniform(X.n);
  if (total == 0) return;
  const int tid = threadIdx.x, w = uniform(tid / 64), l = tid % 64, r = l % 16, g = l / 16;
  const int e = uniform(X.expert), Kd = MODE == 1 ? a.H : a.I, N = MODE == 1 ? 2 * a.I : a.H;
  const int row0 = (int)blockIdx.x * kTileRows, steps = Kd / VK;
  const int64_t R = (int64_t)a.T * (a.K + a.S);
  const uint8_t* wb = (MODE == 1 ? a.w1 : a.w2) + ((int64_t)e * N + row0) * Kd * WB;
  const int wpitch = Kd * WB;                  // N is a multiple of 256: every tile is whole
  // weight rows: the chunk at place p of row y is p ^ (y / 2 % 8)
  const uint32_t wvo = (uint32_t)(l / 8) * wpitch + (((l % 8) ^ ((4 * (w % 2) + l / 16) % 8)) * 16);
  // the wave's two tiles: gate and up of 16 columns (groups of 32 rows), or 32 columns
  const int t0 = MODE == 1 ? 64 * (w / 2) + 16 * (w % 2) : 32 * w, t1 = t0 + (MODE == 1 ? 32 : 16);
  const int sw = (r / 2) % 8;
  const int wc0 = (g ^ sw) * 16 + r * 128, wc1 = ((g + 4) ^ sw) * 16 + r * 128;
  const int sx = RB == 256 ? 8 * (r & 1) + (r >> 1) : sw;
  const float *sp0 = nullptr, *sp1 = nullptr;  // block scales of the two tiles
  if constexpr (F == MM_FEW_FP8_BLOCK) {
    const int nb = Kd / 128;
    if constexpr (MODE == 1) {
      const int c = (row0 / 2 + 16 * w) / 128;
      sp0 = a.s1 + ((int64_t)e * (N / 128) + c) * nb;
      sp1 = sp0 + (int64_t)(a.I / 128) * nb;
    } else {
      sp0 = sp1 = a.s2 + ((int64_t)e * (N / 128) + (row0 + t0) / 128) * nb;
    }
  }

  for (int q0 = 0; q0 < total; q0 += 16 * NT) {
    const int n = total - q0 < 16 * NT ? total - q0 : 16 * NT, nt = (n + 15) / 16;
    // A route's row in LDS: e4m3 weights take 16 K-values a lane and piece, two
    // chunks of it; chunk c = 8j + 2g + h sits at place (8j + 4h + g) ^ sx(row),
    // so that a read covers neighbouring places over g.  One instruction
    // moves 1024 / RB rows.
    constexpr int RPI = 1024 / RB, XI = NT * 16 / RPI;   // rows an instruction; instructions a part
    constexpr int XW = (PB * XI + kWaves - 1) / kWaves;  // a wave (those past the last repeat one)
    uint32_t xvo[XW];
#pragma unroll
    for (int i = 0; i < XW; ++i) {
      const int at = (w + kWaves * i) % (PB * XI), part = at / XI, y = at % XI * RPI + l / (RB / 16), pos = l % (RB / 16);
      int c;
      if constexpr (RB == 256) {
        const int v = pos ^ (8 * (y & 1) + (y % 16 >> 1));
        c = (v & 8) | (v & 3) << 1 | (v >> 2 & 1);
      } else {
        c = pos ^ (y / 2 % 8);
      }
      const int64_t line = MODE == 1 ? X.token[q0 + y < total ? q0 + y : 0] : part * R + X.route[q0 + y < total ? q0 + y : 0];
      xvo[i] = q0 + y < total ? (uint32_t)(line * Kd * 2 + c * 16) : 0x7fffff00u;   // beyond the descriptor: zeros, no access
    }
    const uint8_t* xb = MODE == 1 ? static_cast<const uint8_t*>(a.x) : reinterpret_cast<const uint8_t*>(a.a);
    const int xbytes = (int)((MODE == 1 ? (int64_t)a.T : PB * R) * Kd * 2);
    auto copy = [&](int s, uint8_t* ws, uint8_t* xs) {
      s = s < steps ? s : steps - 1;           // past the end: the last stage again, unused
      const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc((void*)wb, (short)0, kTileRows * wpitch, 0x00020000);
      const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc((void*)xb, (short)0, xbytes, 0x00020000);
#pragma unroll
      for (int i = 0; i < kTileRows / 64; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr_t)(ws + (w + 8 * i) * 1024), 16, wvo, (w + 8 * i) * 8 * wpitch + s * 128, 0, 0);
#pragma unroll
      for (int i = 0; i < XW; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)(xs + (w + kWaves * i) % (PB * XI) * 1024), 16, xvo[i], s * RB, 0, 0);
    };
    constexpr int kCopies = kTileRows / 64 + XW;
    f32x4 acc[2][NT];
    clear(acc[0]);
    clear(acc[1]);
    auto compute = [&](const uint8_t* ws, const uint8_t* xs, float s0, float s1) {
      f32x4 sum[2][NT];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < NT; ++m) sum[i][m] = F == MM_FEW_FP8_BLOCK ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][m];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4 wa = *reinterpret_cast<const u32x4*>(ws + t0 * 128 + (j ? wc1 : wc0));
        const u32x4 wc = *reinterpret_cast<const u32x4*>(ws + t1 * 128 + (j ? wc1 : wc0));
#pragma unroll
        for (int h = 0; h < 3 - WB; ++h) {     // e4m3: two operands of 8 values
          const u32x4 oa = WB == 2 ? wa : widen8(wa[2 * h], wa[2 * h + 1]);
          const u32x4 ob = WB == 2 ? wc : widen8(wc[2 * h], wc[2 * h + 1]);
#pragma unroll
          for (int m = 0; m < NT; ++m)
            if (m == 0 || m < nt) {
#pragma unroll
              for (int p = 0; p < PB; ++p) {
                const int place = (RB == 256 ? 8 * j + 4 * h + g : 4 * j + g) ^ sx;
                const u32x4 b = *reinterpret_cast<const u32x4*>(xs + ((p * NT + m) * 16 + r) * RB + place * 16);
                sum[0][m] = mfma16(oa, b, sum[0][m]);
                sum[1][m] = mfma16(ob, b, sum[1][m]);
              }
            }
        }
      }
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        acc[0][m] = F == MM_FEW_FP8_BLOCK ? acc[0][m] + sum[0][m] * s0 : sum[0][m];
        acc[1][m] = F == MM_FEW_FP8_BLOCK ? acc[1][m] + sum[1][m] * s1 : sum[1][m];
      }
    };
    auto turn = [&]() {
      // the stage's products stay before the wait: nothing else ties them to it
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < NT; ++m) asm volatile("" : "+v"(acc[i][m]));
      __builtin_amdgcn_sched_barrier(0);
      // all copies but the newest stage's (S == 3) have landed
      stage_barrier<S == 3 ? kCopies : 0>();
      __builtin_amdgcn_sched_barrier(0);
    };
    auto scales = [&](int s, float& s0, float& s1) {
      if constexpr (F == MM_FEW_FP8_BLOCK) s0 = sp0[s < steps ? s : steps - 1], s1 = sp1[s < steps ? s : steps - 1];
    };
    float sa[2] = {1.0f, 1.0f}, sn[2] = {1.0f, 1.0f};
    auto stage = [&](int s, const uint8_t* ws, const uint8_t* xs, uint8_t* nw, uint8_t* nx) {
      scales(s + 1, sn[0], sn[1]);
      __builtin_amdgcn_sched_barrier(0);
      copy(s + S - 1, nw, nx);
      compute(ws, xs, sa[0], sa[1]);
      turn();
      sa[0] = sn[0], sa[1] = sn[1];
    };
    scales(0, sa[0], sa[1]);
    copy(0, w0, x0);
    if constexpr (S == 3) copy(1, w1, x1);
    turn();
    if constexpr (S == 3) {
      // (a break inside the loop would be a path on which the compiler sees a
      // slot filled one stage ago, and waits for it)
      int s = 0;
      for (; s + 2 < steps; s += 3) {
        stage(s, w0, x0, w2, x2);
        stage(s + 1, w1, x1, w0, x0);
        stage(s + 2, w2, x2, w1, x1);
      }
      if (s < steps) stage(s, w0, x0, w2, x2);
      if (s + 1 < steps) stage(s + 1, w1, x1, w0, x0);
    } else {
      for (int s = 0; s < steps; s += 2) {
        stage(s, w0, x0, w1, x1);
        if (s + 1 >= steps) break;
        stage(s + 1, w1, x1, w0, x0);
      }
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);        // no copy outlives the round
    __syncthreads();
    if constexpr (MODE == 1) {
      const int col = row0 / 2 + 16 * w + 4 * g;
      f32x4 sg, su;
      if constexpr (F == MM_FEW_FP8) {
        sg = *reinterpret_cast<const f32x4*>(a.s1 + (int64_t)e * 2 * a.I + col);
        su = *reinterpret_cast<const f32x4*>(a.s1 + (int64_t)e * 2 * a.I + a.I + col);
      }
#pragma unroll
      for (int m = 0; m < NT; ++m)
        if (16 * m + r < n) {
          f32x4 hg = acc[0][m], hu = acc[1][m];
          if constexpr (F == MM_FEW_FP8) hg *= sg, hu *= su;
          uint16_t o[4][P];
#pragma unroll
          for (int i = 0; i < 4; ++i) split_bf16<P>(swiglu(hg[i], hu[i], a.clamp), o[i]);
          const int64_t route = X.route[q0 + 16 * m + r];
#pragma unroll
          for (int p = 0; p < P; ++p)
            *reinterpret_cast<u32x2*>(a.a + (p * R + route) * a.I + col) =
                u32x2{o[0][p] | (uint32_t)o[1][p] << 16, o[2][p] | (uint32_t)o[3][p] << 16};
        }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = row0 + t0 + 16 * i + 4 * g;
        f32x4 sc;
        if constexpr (F == MM_FEW_FP8) sc = *reinterpret_cast<const f32x4*>(a.s2 + (int64_t)e * a.H + col);
#pragma unroll
        for (int m = 0; m < NT; ++m)
          if (16 * m + r < n) {
            f32x4 v = acc[i][m];
            if constexpr (F == MM_FEW_FP8) v *= sc;
            *reinterpret_cast<f32x4*>(a.slot + (int64_t)X.route[q0 + 16 * m + r] * a.H + col) = v * X.gate[q0 + 16 * m + r];
          }
      }
    }
  }
}

}  // namespace

template <int F, int MODE, int P, int NT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_few_tile(FewArgs a) {
  few_tile<F, MODE, P, NT>(a);
}

// y[t]: the slots of t's routes in the order of k.  A slot is one that Linear2
// wrote: a valid id that no earlier k of the token names.
__global__ __launch_bounds__(256) void k_few_combine(FewArgs a) {
  const int t = blockIdx.y, c = ((int)blockIdx.x * 256 + threadIdx.x) * 4, Ks = a.K + a.S;
  __shared__ int32_t ids[kMaxK];
  const bool on = a.active == nullptr || a.active[t] != 0;
  if (threadIdx.x < a.K) ids[threadIdx.x] = a.ids[t * a.K + threadIdx.x];
  __syncthreads();
  if (c >= a.H) return;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (on) {
    for (int k = 0; k < Ks; ++k) {
      if (k < a.K) {
        const int id = ids[k];
        bool first = id >= 0 && id < a.E;
        for (int j = 0; j < k; ++j) first = first && ids[j] != id;
        if (!first) continue;
      }
      v += *reinterpret_cast<const f32x4*>(a.slot + ((int64_t)t * Ks + k) * a.H + c);
    }
  }
  const int64_t at = (int64_t)t * a.H + c;
  if (a.y_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + at) = v;
  else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

namespace {

template <int F, int P, int D>
hipError_t run_l1(const FewArgs& a, int num_cus, hipStream_t s) {
  const int64_t routes = (int64_t)a.T * a.K + (a.S ? a.T : 0);
  const int64_t live = routes < a.E + a.S ? routes : a.E + a.S;
  const int64_t units = live * (a.I / 16);
  const int grid = (int)(units < num_cus ? units : num_cus);
  hipLaunchKernelGGL((k_few_l1<F, P, D>), dim3(grid), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int F, int WT, int D>
hipError_t run_l2(const FewArgs& a, int num_cus, hipStream_t s) {
  const int units = a.H / (16 * WT);
  const size_t lds = (size_t)2 * kWaves * a.T * 4 * WT * 16;
  static_assert(2 * kWaves * kStreamT * 4 * 2 * 16 + sizeof(Lists) <= 65536, "LDS without an attribute");
  hipLaunchKernelGGL((k_few_l2<F, WT, D>), dim3(units < num_cus ? units : num_cus), dim3(kThreads), lds, s, a);
  return hipGetLastError();
}

template <int F, int MODE, int P>
hipError_t run_tile(const FewArgs& a, hipStream_t s) {
  const int64_t routes = (int64_t)a.T * a.K, most = routes < a.E ? routes : a.E;   // live routed experts at most
  const int N = MODE == 1 ? 2 * a.I : a.H;
  const dim3 grid((unsigned)((N + kTileRows - 1) / kTileRows), (unsigned)(most + a.S));
  hipLaunchKernelGGL((k_few_tile<F, MODE, P, MODE == 2 && P == 3 ? 2 : 4>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int F, int P>
hipError_t run_l1_f(const FewArgs& a, int num_cus, hipStream_t s) {
  // us for the whole layer with streaming / tile Linear1 and a bf16 y.  32 experts of
  // 7168 x 2048, top-8, e4m3: 1 token 77 / 85, 4 tokens 171 / 190, 8 tokens 229 / 230, 16
  // tokens 264 / 257, bf16 503 / 497; 64 experts of 2048 x 1408, top-6, e4m3: 1 token
  // 30 / 31, 4 tokens 58 / 52, 8 tokens 80 / 83, 16 tokens 119 / 132, bf16 211 / 234.  16
  // experts of 4096 x 1408, top-4, favour the tiles in e4m3 from 4 tokens on (51 / 49;
  // 16 tokens 69 / 59; bf16 123 / 126): several routes an expert, whose rows the
  // streaming kernel reads again for every 16 columns.  One MFMA of routes is its limit.
  if (a.T > kStreamT) return run_tile<F, 1, P>(a, s);
  return run_l1<F, P, 3>(a, num_cus, s);
}
template <int F, int P>
hipError_t run_l2_f(const FewArgs& a, int num_cus, hipStream_t s) {
  if (few_slots(a.T, a.y_f32)) {
    const hipError_t err = run_tile<F, 2, P>(a, s);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(k_few_combine, dim3((unsigned)((a.H + 1023) / 1024), (unsigned)a.T), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if constexpr (P == 1) {
    // 32 columns a unit where that still gives most CUs one: half the control
    // per weight byte (e4m3, one token: 30 against 37 us; bf16, at 5.9 TB/s
    // within a unit, loses by the missing units: 56 against 51 us)
    if constexpr (F != MM_FEW_BF16)
      if (a.H / 32 >= num_cus * 3 / 4) return run_l2<F, 2, 3>(a, num_cus, s);
    return run_l2<F, 1, 4>(a, num_cus, s);
  } else {
    return hipErrorInvalidValue;               // float32 y always takes the tiles
  }
}
template <int P>
hipError_t run_l1_p(const FewArgs& a, int num_cus, hipStream_t s) {
  switch (a.format) {
    case MM_FEW_BF16: return run_l1_f<MM_FEW_BF16, P>(a, num_cus, s);
    case MM_FEW_FP8: return run_l1_f<MM_FEW_FP8, P>(a, num_cus, s);
    default: return run_l1_f<MM_FEW_FP8_BLOCK, P>(a, num_cus, s);
  }
}
template <int P>
hipError_t run_l2_p(const FewArgs& a, int num_cus, hipStream_t s) {
  switch (a.format) {
    case MM_FEW_BF16: return run_l2_f<MM_FEW_BF16, P>(a, num_cus, s);
    case MM_FEW_FP8: return run_l2_f<MM_FEW_FP8, P>(a, num_cus, s);
    default: return run_l2_f<MM_FEW_FP8_BLOCK, P>(a, num_cus, s);
  }
}

}  // namespace

// Linear2 through slots (tiles and a combine), or streaming.  The three parts
// of A that a float32 y takes cost the streaming kernel a read each per 16
// columns (us for the whole layer, streaming / tiles, 7168 x 2048 in e4m3: 1 token
// 99 / 82, 4 tokens 214 / 172, 16 tokens 360 / 258).  With a bf16 y, the sizes above:
// 1 token 77 / 78, 4 tokens 171 / 187, 16 tokens 264 / 275; smaller matrices with
// several routes an expert favour the tiles (2048 x 1408, 4 tokens 58 / 49, 16 tokens
// 119 / 98; 4096 x 1408, 16 tokens 69 / 63), one token does not (30 / 32, 30 / 33).
bool few_slots(int64_t T, int y_f32) { return y_f32 || T > kStreamT; }

hipError_t launch_few_l1(const FewArgs& a, int num_cus, hipStream_t s) {
  return a.y_f32 ? run_l1_p<3>(a, num_cus, s) : run_l1_p<1>(a, num_cus, s);
}
hipError_t launch_few_l2(const FewArgs& a, int num_cus, hipStream_t s) {
  return a.y_f32 ? run_l2_p<3>(a, num_cus, s) : run_l2_p<1>(a, num_cus, s);
}

}  // namespace mm
