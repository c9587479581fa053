// Selection of one token's experts from its partial scores, by one wave (the
// router's second kernel).
#pragma once
#include "mm_device.hpp"
#include "mm_ops_internal.hpp"

namespace mm {

// x_t . w_e in 64 bits for two experts by one wave (every lane gets the sums)
__device__ __forceinline__ void router_dot64(const RouterArgs& a, int64_t t, int e0, int e1, double& d0, double& d1) {
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + t * a.H * 2;
  const uint8_t *w0 = static_cast<const uint8_t*>(a.w) + (int64_t)e0 * a.H * 2, *w1 = static_cast<const uint8_t*>(a.w) + (int64_t)e1 * a.H * 2;
  double s0 = 0.0, s1 = 0.0;
  constexpr int kAhead = 4;    // pieces of 512 values asked for at once: one wait of memory, not one each
  for (int k0 = lane_id() * 8; k0 < a.H; k0 += 512 * kAhead) {
    u32x4 xv[kAhead], wv[kAhead], vv[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + 512 * u < a.H ? k0 + 512 * u : k0;
      xv[u] = *reinterpret_cast<const u32x4*>(x + k * 2);
      wv[u] = *reinterpret_cast<const u32x4*>(w0 + k * 2);
      vv[u] = *reinterpret_cast<const u32x4*>(w1 + k * 2);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (k0 + 512 * u < a.H) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double lo = bf16_bits_to_f32(xv[u][i] & 0xffffu), hi = __uint_as_float(xv[u][i] & 0xffff0000u);
          s0 += lo * (double)bf16_bits_to_f32(wv[u][i] & 0xffffu);
          s0 += hi * (double)__uint_as_float(wv[u][i] & 0xffff0000u);
          s1 += lo * (double)bf16_bits_to_f32(vv[u][i] & 0xffffu);
          s1 += hi * (double)__uint_as_float(vv[u][i] & 0xffff0000u);
        }
      }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s0 += __shfl_xor(s0, o, 64), s1 += __shfl_xor(s1, o, 64);
  d0 = s0, d1 = s1;
}

// whether every value of token t is zero
__device__ __forceinline__ bool router_zero_row(const RouterArgs& a, int64_t t) {
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + t * a.H * 2;
  uint32_t any = 0;
  for (int k = lane_id() * 8; k < a.H; k += 512) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(x + k * 2);
    any |= v[0] | v[1] | v[2] | v[3];
  }
  return ballot((any & 0x7fff7fffu) != 0) == 0;
}

// largest value of the wave: four shifts inside the rows of 16 lanes, two
// broadcasts across them; lane 63 ends with it
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#define MM_STEP(ctrl, rows)                                                                          \
  {                                                                                                  \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false);      \
    v = o > v ? o : v;                                                                               \
  }
  MM_STEP(0x111, 0xf) MM_STEP(0x112, 0xf) MM_STEP(0x114, 0xf) MM_STEP(0x118, 0xf) MM_STEP(0x142, 0xa) MM_STEP(0x143, 0xc)
#undef MM_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// floats as integers of the same order; NaN is 1, below every number, and 0
// is an expert that cannot be taken
__device__ __forceinline__ uint32_t rank_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return f != f ? 1u : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float rank_value(uint32_t k) {
  return k == 1u ? __builtin_nanf("") : __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// KM: most slices of the hidden dimension (2 or 8).  Up to 32 partial scores a
// lane are asked for at once (16 experts a lane and 8 slices together did not
// fit the registers: 8192 x 512 141 against 86 us).

// What does not change from token to token: lane l holds experts l, l + 64, ...
template <int NV>
struct RouterExperts {
  float norm[NV], bias[NV];      // |w|; bias
};
// One token: |x|^2, the float32 scores, the largest partial sums beside them.
template <int NV>
struct RouterToken {
  float xx, score[NV], most[NV];   // most: summed over the slices
  int active;
};

template <int NV, int KM>
__device__ __forceinline__ void router_load_experts(const RouterArgs& a, RouterExperts<NV>& x) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = lane_id() + 64 * v < a.E ? lane_id() + 64 * v : 0;
    x.bias[v] = a.bias != nullptr ? a.bias[e] : 0.0f;
    float p[KM], s;
#pragma unroll
    for (int k = 0; k < KM; ++k)
      if (k == 0 || k < a.KS) p[k] = a.wnorm[(int64_t)k * a.Ep + e];
    s = p[0];
#pragma unroll
    for (int k = 1; k < KM; ++k)
      if (k < a.KS) s += p[k];
    x.norm[v] = __builtin_amdgcn_sqrtf(s + 2e-34f);
  }
}

template <int NV, int KM>
__device__ __forceinline__ void router_load_token(const RouterArgs& a, int64_t t, RouterToken<NV>& x) {
  constexpr int KC = KM * NV <= 32 ? KM : 32 / NV;
  x.active = a.active == nullptr ? 1 : a.active[t];
  x.xx = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) x.score[v] = x.most[v] = 0.0f;
  const int Y = (a.E + a.EB - 1) / a.EB;
  for (int k0 = 0; k0 < (KC == KM ? 1 : a.KS); k0 += KC) {
    float xx[KC], part[NV][KC], most[NV][KC];
#pragma unroll
    for (int k = 0; k < KC; ++k)
      if (k == 0 || k0 + k < a.KS) {
        xx[k] = a.xnorm[(int64_t)(k0 + k) * a.T + t];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int e = lane_id() + 64 * v < a.E ? lane_id() + 64 * v : 0;
          part[v][k] = a.part[((int64_t)(k0 + k) * a.T + t) * a.Ep + e];
          most[v][k] = a.xmost[((int64_t)(k0 + k) * Y + e / a.EB) * a.T + t];
        }
      }
#pragma unroll
    for (int k = 0; k < KC; ++k)
      if (k == 0 || k0 + k < a.KS) {
        x.xx += xx[k];
#pragma unroll
        for (int v = 0; v < NV; ++v) x.score[v] += part[v][k], x.most[v] += most[v][k];
      }
  }
}

// Lane k returns the k-th expert of token t and its weight (-1 and 0 where
// none is left).  The largest float32 ranks are taken in turn; where one is
// above the next by more than both may be off, their order is that of the
// 64-bit ranks.  The others form runs of neighbours (one token of random data
// in 20 has one with 128 experts or more, one in 80 with 32; mostly of two): the
// members of a run get their 64-bit ranks and are put in order among themselves.  Tokens whose float32 sums left their range, and
// runs past 64 positions, are selected again one expert at a time.
template <int NV>
__device__ __forceinline__ void router_select_token(const RouterArgs& a, int64_t t, const RouterExperts<NV>& ex,
                                                    const RouterToken<NV>& tok, int& id, float& weight) {
  const int l = lane_id();
  id = -1;
  weight = 0.0f;
  if (tok.active == 0) return;
  const bool sig = a.scoring == MM_ROUTER_SIGMOID, biased = a.bias != nullptr;
  const float xx = tok.xx;
  float z[NV], err[NV];        // score argument; bound on the rank's error
  uint32_t key[NV];
  // bounds of the float32 sums (the rule stands at the scores' kernels), with a
  // hundredth for the norms' own roundings; squares below float32's range leave
  // at most 16384 * 2^-126 = 2e-34 out of a norm
  const float sums = 1.01f * 5.9604645e-8f * a.of_sums;
  const float products = 1.01f * 5.9604645e-8f * a.of_products, xn = __builtin_amdgcn_sqrtf(xx + 2e-34f);
  float most = 0.0f;           // the largest bound of this lane
  bool lost = false;           // some float32 sum left its range
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    z[v] = 0.0f, err[v] = 0.0f, key[v] = 0;
    if (l + 64 * v >= a.E) continue;
    const float s = tok.score[v], b = ex.bias[v], wn = ex.norm[v];
    const float norms = xn * wn;
    float d = products * norms + sums * fminf(tok.most[v], norms) + 1e-36f, rank;    // (a NaN is the larger one)
    if (sig) {
      z[v] = s;
      rank = s;
      if (biased) {
        // float32 sigmoid: a slope of at most 1/4, and its own rounding
        rank = __builtin_amdgcn_rcpf(1.0f + __expf(-s)) + b;
        d = 0.25f * d + 1e-6f;
      }
    } else {
      z[v] = rank = s + b;
    }
    d += 2.4e-7f * fabsf(rank);
    if (b == -__builtin_huge_valf()) continue;             // switched off
    key[v] = rank_key(rank);
    if (!(fabsf(rank) <= 3.0e38f) && !(xx < 1e36f && wn < 1e18f) && xx == xx && wn == wn) {
      lost = true;
      err[v] = __builtin_huge_valf();
    } else {
      err[v] = fabsf(rank) <= 3.0e38f ? d : 0.0f;
      if (rank == -__builtin_huge_valf()) key[v] = 0;      // -inf: never taken
    }
    most = err[v] > most ? err[v] : most;
  }
  // bounds are not negative: their bits are in order
  const float gap = 2.0f * __uint_as_float(wave_max_u32(__float_as_uint(most)));
  // the expert at (bl, bv) leaves the ranking and becomes the k-th
  uint32_t left[NV];
  auto take = [&](int k, int bl, int bv) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v == bv && l == bl) left[v] = 0;
    if (l == k) id = bl + 64 * bv;
  };
  // the largest key left, 0 if none; (bl, bv): the lowest expert that has it
  auto largest = [&](int& bl, int& bv) {
    uint32_t m = left[0];
#pragma unroll
    for (int v = 1; v < NV; ++v) m = left[v] > m ? left[v] : m;
    const uint32_t best = wave_max_u32(m);
#pragma unroll
    for (int v = NV - 1; v >= 0; --v) {
      const uint64_t at = ballot(left[v] == best);
      if (at != 0) bv = v, bl = __ffsll((unsigned long long)at) - 1;
    }
    return best;
  };
  // the 64-bit rank of a 64-bit score argument
  auto rank_of = [&](double z, int e) {
    const double b = biased ? (double)a.bias[e] : 0.0;
    return !sig ? z + b : biased ? 1.0 / (1.0 + exp(-z)) + b : z;
  };
  bool sure = ballot(lost) == 0;
  uint64_t chained = 0;        // position k is not surely below position k - 1
  // whether position k with key `best` after `before` ends the list; 2: too long
  uint32_t before = 0;
  auto ends = [&](int k, uint32_t best) {
    const float r = rank_value(best);
    const bool doubt = k > 0 && best > 1u && r - r == 0.0f && !(rank_value(before) - r > gap);
    if (best == 0 || (k >= a.K && !doubt)) return true;
    if (k == 64) {
      sure = false;
      return true;
    }
    chained |= (uint64_t)doubt << k;
    before = best;
    return false;
  };
  if constexpr (NV <= 4) {
    // each lane's keys in descending order, equal ones by expert: a turn looks
    // at the first one only (256 experts: 33 against 60 instructions a turn)
    uint32_t at[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) left[v] = key[v], at[v] = (uint32_t)(l + 64 * v);
#pragma unroll
    for (int n = NV - 1; n > 0; --n)
#pragma unroll
      for (int v = 0; v < n; ++v) {
        const bool swap = left[v + 1] > left[v];
        const uint32_t hk = swap ? left[v + 1] : left[v], lk = swap ? left[v] : left[v + 1];
        const uint32_t ha = swap ? at[v + 1] : at[v], la = swap ? at[v] : at[v + 1];
        left[v] = hk, left[v + 1] = lk, at[v] = ha, at[v + 1] = la;
      }
    for (int k = 0; sure; ++k) {
      const uint32_t best = wave_max_u32(left[0]);
      if (ends(k, best)) break;
      const uint64_t who = ballot(left[0] == best);
      int e = __builtin_amdgcn_readlane((int)at[0], __ffsll((unsigned long long)who) - 1);
      if ((who & (who - 1)) != 0) e = (int)~wave_max_u32(left[0] == best ? ~at[0] : 0u);   // equal ones: the lowest
      if (l == k) id = e;
      if (l == e % 64) {
#pragma unroll
        for (int v = 0; v + 1 < NV; ++v) left[v] = left[v + 1], at[v] = at[v + 1];
        left[NV - 1] = 0;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) left[v] = key[v];
    for (int k = 0; sure; ++k) {
      int bl = 0, bv = 0;
      const uint32_t best = largest(bl, bv);
      if (ends(k, best)) break;
      take(k, bl, bv);
    }
  }
  // a token of zeros: every float32 score is exact, and a long run of equal ones likely
  const bool zero = (chained != 0 || !sure) && xx == 0.0f && router_zero_row(a, t);
  if (sure && !zero && chained != 0) {
    // 64-bit ranks of the positions in runs, two at a time: memory is waited for
    const uint64_t runs = chained | chained >> 1;
    double mine = 0.0;
    for (uint64_t todo = runs; todo != 0;) {
      const int p0 = __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      const int p1 = todo != 0 ? __ffsll((unsigned long long)todo) - 1 : p0;
      todo &= todo - 1;
      double d0, d1;
      const int e0 = __builtin_amdgcn_readlane(id, p0), e1 = __builtin_amdgcn_readlane(id, p1);
      router_dot64(a, t, e0, e1, d0, d1);
      if (l == p0 || l == p1) mine = rank_of(l == p0 ? d0 : d1, id);
      // the weights from the same sums: they fall in the order that these decide
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const double b = sig ? 0.0 : (double)ex.bias[v];
        if (l + 64 * v == e0) z[v] = (float)(d0 + b);
        if (l + 64 * v == e1) z[v] = (float)(d1 + b);
      }
    }
    // each moves within its run by those that it was wrongly before or behind
    const int run = __popcll((unsigned long long)(~chained & ((2ull << l) - 1)));
    int place = l;
    for (uint64_t todo = runs; todo != 0; todo &= todo - 1) {
      const int q = __ffsll((unsigned long long)todo) - 1;
      const double other = __shfl(mine, q, 64);
      const int e = __builtin_amdgcn_readlane(id, q);
      const bool above = other > mine || (other == mine && e < id);
      if (__builtin_amdgcn_readlane(run, q) == run && q != l) place += q > l ? (above ? 1 : 0) : (above ? 0 : -1);
    }
    id = __builtin_amdgcn_ds_permute(4 * place, id);
  }
  if (!sure || zero) {
    // one expert at a time, each with a bound of its own
    double exact[NV];          // the 64-bit rank of an expert in `known`
    uint32_t known = 0;
    id = -1;
#pragma unroll
    for (int v = 0; v < NV; ++v) left[v] = key[v], exact[v] = 0.0;
    auto learn = [&](int v, double zz) {
      const double rank = rank_of(zz, l + 64 * v);
      float e = 2.4e-7f * fabsf((float)rank);
      if (!(e <= 3.0e38f)) e = 0.0f;
      const uint32_t kk = rank == -__builtin_huge_val() ? 0u : rank_key((float)rank);
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (u == v) z[u] = (float)(sig || !biased ? zz : rank), exact[u] = rank, left[u] = kk, err[u] = e;
      known |= 1u << v;
    };
    if (zero) {
      for (int v = 0; v < NV; ++v) {
        float zv = 0.0f;
        uint32_t kv = 0;
#pragma unroll
        for (int u = 0; u < NV; ++u)
          if (u == v) zv = z[u], kv = key[u];
        // a weight that is not finite has made its score NaN, which stays last
        if (kv > 1u && zv - zv == 0.0f) learn(v, 0.0);
      }
    }
    for (int k = 0; k < a.K; ++k) {
      int bl = 0, bv = 0;
      bool none = false;
      for (;;) {
        const uint32_t best = largest(bl, bv);
        none = best == 0;
        if (none) break;
        float be = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (v == bv) be = err[v];
        be = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(be), bl));
        const float floor = rank_value(best) - be;
        // experts whose bound reaches the best one's (the best one among them)
        uint32_t near = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (left[v] != 0 && (!(err[v] <= 3.0e38f) || (left[v] > 1u && rank_value(left[v]) + err[v] >= floor))) near |= 1u << v;
        uint64_t others = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const uint64_t n = ballot(near >> v & 1u);
          others |= v == bv && err[v] <= 3.0e38f ? n & ~(1ull << bl) : n;
        }
        if (ballot(others != 0) == 0) break;
        // their 64-bit ranks, each kept by its lane
        bool grew = false;
        for (int v = 0; v < NV; ++v)
          for (uint64_t todo = ballot((near & ~known) >> v & 1u); todo != 0; todo &= todo - 1) {
            const int src = __ffsll((unsigned long long)todo) - 1;
            double d0, d1;
            router_dot64(a, t, src + 64 * v, src + 64 * v, d0, d1);
            grew = true;
            if (l == src) learn(v, d0);
          }
        if (grew) continue;
        // all known: the largest 64-bit rank, ties to the lowest expert
        double top = -__builtin_huge_val();
        int te = 1 << 30;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if ((near >> v & 1u) && (te == 1 << 30 || exact[v] > top)) top = exact[v], te = l + 64 * v;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
          const double ot = __shfl_xor(top, o, 64);
          const int oe = __shfl_xor(te, o, 64);
          if (oe < (1 << 30) && (te == 1 << 30 || ot > top || (ot == top && oe < te))) top = ot, te = oe;
        }
        te = __builtin_amdgcn_readfirstlane(te);
        bl = te % 64, bv = te / 64;
        break;
      }
      if (none) break;
      take(k, bl, bv);
    }
  }
  if (l >= a.K) id = -1;
  // the selected experts' score arguments, from their lanes
  float my_z = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const float zz = __shfl(z[v], id & 63, 64);
    if (id / 64 == v) my_z = zz;
  }
  if (sig) {
    weight = id >= 0 ? 1.0f / (1.0f + expf(-my_z)) : 0.0f;
  } else {
    // softmax over every expert
    float zmax = -__builtin_huge_valf(), zsum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (l + 64 * v < a.E) zmax = z[v] > zmax || z[v] != z[v] ? z[v] : zmax;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const float w = __shfl_xor(zmax, o, 64);
      zmax = w > zmax || w != w ? w : zmax;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (l + 64 * v < a.E) zsum += expf(z[v] - zmax);
    zsum = wave_sum(zsum);
    weight = id >= 0 ? expf(my_z - zmax) / zsum : 0.0f;
  }
  if (a.renormalize) {
    const float s = wave_sum(weight);
    weight = weight / (s + 1e-20f);
  }
  weight *= a.scale;
}

}  // namespace mm
