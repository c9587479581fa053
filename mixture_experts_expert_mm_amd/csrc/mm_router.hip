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
// The order of two experts is decided by their 64-bit scores.  The float32
// sum of a score is off by at most about sqrt(steps) * 2^-23 * |x| |w| (every
// step rounds a partial sum that Cauchy-Schwarz bounds by |x| |w|; the
// roundings are independent), so the selection carries that bound per
// expert, and where the best and another expert are closer than their
// bounds, both are summed again in 64 bits.  A few in a hundred tokens need
// it, for two experts each.
#include "mm_device.hpp"
#include "mm_ops_internal.hpp"

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
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v[i]), __builtin_bit_cast(bf16x2, v[i]), acc, false);
  return acc;
}

}  // namespace

// TT x ET tiles of 16 tokens x 16 experts a wave; EW waves along the experts,
// KW = 8 / EW along the hidden dimension, added in LDS in a fixed order.
// Lane l of a tile holds 8 consecutive hidden values of expert (A) and token
// (B) l % 16; accumulator i is expert 4 * (l / 16) + i of token l % 16.
template <int TT, int ET, int EW>
__global__ __launch_bounds__(kThreads) void k_router_scores(RouterArgs a) {
  constexpr int KW = kWaves / EW;
  constexpr int kSlots = KW > 1 ? KW / 2 * EW : 1;
  __shared__ f32x4 red[kSlots][TT * ET][64];
  __shared__ float xn[KW][TT * 16], wn[KW][EW * ET * 16];
  const int w = threadIdx.x / 64, l = threadIdx.x % 64, r = l % 16, g = l / 16;
  const int ew = w % EW, kw = w / EW;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * TT);
  const int e0 = (int)blockIdx.y * (16 * ET * EW) + ew * (16 * ET);
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
#pragma unroll
  for (int i = 0; i < TT; ++i) xs[i] = 0.0f;
#pragma unroll
  for (int j = 0; j < ET; ++j) ws[j] = 0.0f;
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int j = 0; j < ET; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const bool do_x = blockIdx.y == 0 && ew == 0, do_w = blockIdx.x == 0;
  const int steps = a.H / kRouterStep, q = (int)blockIdx.z * KW + kw, Q = KW * a.KS;
#pragma unroll 2
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
  // squared norms: the four lane groups of a row, then the KW waves
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    float v = xs[i];
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    if (ew == 0 && g == 0) xn[kw][16 * i + r] = v;
  }
#pragma unroll
  for (int j = 0; j < ET; ++j) {
    float v = ws[j];
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    if (g == 0) wn[kw][(ew * ET + j) * 16 + r] = v;
  }
#pragma unroll
  for (int h = KW / 2; h >= 1; h /= 2) {
    if (kw >= h && kw < 2 * h) {
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < ET; ++j) red[(kw - h) * EW + ew][i * ET + j][l] = acc[i][j];
    }
    __syncthreads();
    if (kw < h) {
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int j = 0; j < ET; ++j) acc[i][j] += red[kw * EW + ew][i * ET + j][l];
    }
    __syncthreads();
  }
  if constexpr (KW == 1) __syncthreads();
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
  if (blockIdx.y == 0 && (int)threadIdx.x < 16 * TT && t0 + threadIdx.x < a.T) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < KW; ++k) v += xn[k][threadIdx.x];
    a.xnorm[(int64_t)blockIdx.z * a.T + t0 + threadIdx.x] = v;
  }
  if (do_w && (int)threadIdx.x < EW * ET * 16) {
    const int e = (int)blockIdx.y * (16 * ET * EW) + threadIdx.x;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < KW; ++k) v += wn[k][threadIdx.x];
    if (e < a.Ep) a.wnorm[(int64_t)blockIdx.z * a.Ep + e] = v;
  }
}

// x_t . w_e in 64 bits by one wave (every lane gets the sum)
__device__ double router_dot64(const RouterArgs& a, int64_t t, int e) {
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + t * a.H * 2;
  const uint8_t* w = static_cast<const uint8_t*>(a.w) + (int64_t)e * a.H * 2;
  double s = 0.0;
  for (int k = lane_id() * 8; k < a.H; k += 512) {
    const u32x4 xv = *reinterpret_cast<const u32x4*>(x + k * 2), wv = *reinterpret_cast<const u32x4*>(w + k * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // bf16 x bf16 is exact in float32's exponent range or beyond it: multiply in 64 bits
      s += (double)bf16_bits_to_f32(xv[i] & 0xffffu) * (double)bf16_bits_to_f32(wv[i] & 0xffffu);
      s += (double)__uint_as_float(xv[i] & 0xffff0000u) * (double)__uint_as_float(wv[i] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  return s;
}

// One wave per token; lane l holds experts l, l + 64, ...  Keys are doubles:
// the selection value of each expert, NaN below every number, -inf taken out.
template <int NV>
__global__ __launch_bounds__(256) void k_router_select(RouterArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  if (t >= a.T) return;
  const int l = threadIdx.x % 64;
  int my_id = -1;
  double my_z = 0.0;          // lane k: score argument z of the k-th selection
  double zmax = -__builtin_huge_val();
  float zsum = 0.0f;
  if (a.active == nullptr || a.active[t] != 0) {
    const bool sig = a.scoring == MM_ROUTER_SIGMOID;
    float xx = 0.0f;
    for (int z = 0; z < a.KS; ++z) xx += a.xnorm[(int64_t)z * a.T + t];
    const int steps = a.H / 32 + a.KS + kWaves;
    const float unit = 1.1920929e-7f * sqrtf((float)steps) * sqrtf(xx);
    double z[NV], key[NV];
    float err[NV];
    uint32_t live = 0;
    auto key_of = [&](double zz, float b) -> double {
      if (!sig || a.bias == nullptr) return zz;
      return 1.0 / (1.0 + exp(-zz)) + (double)b;
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = l + 64 * v;
      z[v] = 0.0, key[v] = 0.0, err[v] = 0.0f;
      if (e < a.E) {
        float s = 0.0f, ww = 0.0f;
        for (int k = 0; k < a.KS; ++k) {
          s += a.part[((int64_t)k * a.T + t) * a.Ep + e];
          ww += a.wnorm[(int64_t)k * a.Ep + e];
        }
        const float b = a.bias ? a.bias[e] : 0.0f;
        float d = unit * sqrtf(ww) + 1e-36f;
        z[v] = sig ? (double)s : (double)s + (double)b;
        if (sig && a.bias) {
          // float32 sigmoid: its own rounding, and the slope of at most 1/4
          key[v] = (double)(1.0f / (1.0f + expf(-s))) + (double)b;
          d = 0.25f * d + 2.4e-7f;
        } else {
          key[v] = z[v];
        }
        if (!(fabs(key[v]) <= 3.0e38) && d < __builtin_huge_valf()) {
          // +-inf or NaN: exact unless the float32 sum overflowed
          if (xx < 1e36f && ww < 1e36f) d = 0.0f;
        }
        err[v] = d != d ? 0.0f : d;
        if (key[v] != -__builtin_huge_val() || err[v] > 0.0f) live |= 1u << v;
        if (b == -__builtin_huge_valf()) live &= ~(1u << v), err[v] = 0.0f;
      }
      if (key[v] != key[v]) key[v] = -1.7976931348623157e308;
    }
    for (int k = 0; k < a.K; ++k) {
      double best = 0.0;
      int be = -1;
      for (;;) {
        // the largest key, ties to the lowest expert
        best = -__builtin_huge_val();
        be = 1 << 30;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if ((live >> v & 1u) && (key[v] > best || be == 1 << 30)) best = key[v], be = l + 64 * v;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
          const double ob = __shfl_xor(best, o, 64);
          const int oe = __shfl_xor(be, o, 64);
          if (oe < (1 << 30) && (be == 1 << 30 || ob > best || (ob == best && oe < be))) best = ob, be = oe;
        }
        if (be == 1 << 30) break;
        float bd = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (be == l + 64 * v) bd = err[v];
        bd = __shfl(bd, be % 64, 64);
        bool again = false;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int e = l + 64 * v;
          // contested: not surely below the best (inf - inf compares false)
          const bool c = (live >> v & 1u) && e != be && (err[v] > 0.0f || bd > 0.0f) &&
                         !(key[v] + (double)err[v] < best - (double)bd);
          const uint64_t any = ballot(c);
          if (any != 0) again = true;
          uint64_t todo = ballot(c && err[v] > 0.0f);
          while (todo != 0) {
            const int src = __ffsll((unsigned long long)todo) - 1;
            todo &= todo - 1;
            const int ce = src + 64 * v;
            const double dz = router_dot64(a, t, ce);
            if (l == src) {
              const float b = a.bias ? a.bias[ce] : 0.0f;
              z[v] = sig ? dz : dz + (double)b;
              key[v] = key_of(z[v], b);
              if (key[v] == -__builtin_huge_val()) live &= ~(1u << v);
              if (key[v] != key[v]) key[v] = -1.7976931348623157e308;
              err[v] = 0.0f;
            }
          }
        }
        if (!again) {
          if (bd > 0.0f && !(fabs(best) <= 3.0e38)) again = true;   // overflowed in float32, alone at the top
          else break;
        }
        if (bd > 0.0f) {
          const double dz = router_dot64(a, t, be);
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            if (be == l + 64 * v) {
              const float b = a.bias ? a.bias[be] : 0.0f;
              z[v] = sig ? dz : dz + (double)b;
              key[v] = key_of(z[v], b);
              if (key[v] == -__builtin_huge_val()) live &= ~(1u << v);
              if (key[v] != key[v]) key[v] = -1.7976931348623157e308;
              err[v] = 0.0f;
            }
          }
        }
      }
      if (be == 1 << 30) break;
      double zb = 0.0;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (be == l + 64 * v) zb = z[v], live &= ~(1u << v);
      zb = __shfl(zb, be % 64, 64);
      if (l == k) my_id = be, my_z = zb;
    }
    if (!sig) {
      // softmax over every expert
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (l + 64 * v < a.E) zmax = z[v] > zmax || z[v] != z[v] ? z[v] : zmax;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) {
        const double w = __shfl_xor(zmax, o, 64);
        zmax = w > zmax || w != w ? w : zmax;
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (l + 64 * v < a.E) zsum += expf((float)(z[v] - zmax));
      zsum = wave_sum(zsum);
    }
  }
  float wgt = 0.0f;
  if (my_id >= 0)
    wgt = a.scoring == MM_ROUTER_SIGMOID ? (float)(1.0 / (1.0 + exp(-my_z))) : expf((float)(my_z - zmax)) / zsum;
  if (a.renormalize) {
    float s = l < a.K ? wgt : 0.0f;
    s = wave_sum(s);
    wgt = wgt / (s + 1e-20f);
  }
  if (l < a.K) {
    a.ids[t * a.K + l] = my_id;
    a.weights[t * a.K + l] = wgt * a.scale;
  }
}

// Measured rules.  Up to 64 tokens the scores are a stream of Wr: 16 x 16
// tiles over as many workgroups as the hidden dimension gives.  Beyond, a
// wave holds 64 x 64 so that a token row is read once per 256 experts.
RouterShape router_shape(int64_t T, int H, int E) {
  RouterShape s{};
  const int steps = H / kRouterStep;
  s.ep = (E + 15) / 16 * 16;
  s.wide = T > 64;
  if (!s.wide) {
    s.ew = 1;
    s.ks = steps / (kWaves * 4);
  } else {
    s.ew = E <= 64 ? 1 : E <= 128 ? 2 : 4;
    const int64_t tiles = (T + 63) / 64 * ((E + 64 * s.ew - 1) / (64 * s.ew));
    const int64_t want = 256 / tiles, most = steps / (2 * (kWaves / s.ew));
    s.ks = (int)(want < most ? want : most);
  }
  s.ks = s.ks < 1 ? 1 : s.ks > 8 ? 8 : s.ks;
  return s;
}

hipError_t launch_router_scores(const RouterArgs& a, hipStream_t s) {
  const RouterShape sh = router_shape(a.T, a.H, a.E);
  if (!sh.wide) {
    const dim3 grid((unsigned)((a.T + 15) / 16), (unsigned)(a.Ep / 16), (unsigned)a.KS);
    hipLaunchKernelGGL((k_router_scores<1, 1, 1>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  const int per = 64 * sh.ew;
  const dim3 grid((unsigned)((a.T + 63) / 64), (unsigned)((a.E + per - 1) / per), (unsigned)a.KS);
  if (sh.ew == 1) hipLaunchKernelGGL((k_router_scores<4, 4, 1>), grid, dim3(kThreads), 0, s, a);
  else if (sh.ew == 2) hipLaunchKernelGGL((k_router_scores<4, 4, 2>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_router_scores<4, 4, 4>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_router_select(const RouterArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + 3) / 4));
  if (a.E <= 64) hipLaunchKernelGGL(k_router_select<1>, grid, dim3(256), 0, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL(k_router_select<4>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_router_select<16>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mm
