// The activation between an expert's two products, and its gradient from a
// copy of its input in 8 bits:
//
//   a = g / (1 + e^-g) * u,  h = [g | u], both clamped to [-c, c] if asked
//   the copy: each half of a row in groups of 128, s = max(max|group| / 127, 1e-8),
//   q = round-half-even(h / s) in [-127, 127], decided in IEEE float32
//   backward at h~ = q * s:  dg = da * u * sig * (1 + g * (1 - sig)) where |g~| <= c,
//                            du = da * g * sig                       where |u~| <= c
//
// h's columns are [g | u], or gate and up columns in turns of `turn` (as the rows
// of a prepared W1 lie); the groups are of neighbouring gates, or ups, either way.
//
// Bound: HBM; every value is read and written once.  65536 rows of 2 x 2048 bf16, one
// launch behind the other on the same buffers: forward with the copy 231 us (1.08
// GB, 4.7 TB/s), backward 191 (5.7; a copy 4.9); with other inputs in turn, traced one
// by one, 235 to 289 and 180 to 204.
#include <type_traits>

#include "mm_device.hpp"
#include "mm_elements_dev.hpp"
#include "mm_ops_internal.hpp"

namespace mm {

namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 128, kLanes = 16, kPer = kGroup / kLanes;   // a group's lanes, a lane's values

// NaN stays, as it does in the formula
__device__ __forceinline__ float clamped(float v, float c) { return v > c ? c : v < -c ? -c : v; }

// 1 / (1 + e^-z).  The 16-bit types take the fast exponential and reciprocal:
// relative error below 2^-16 from z = -87.3 on, against a rounding of 2^-8 or 2^-11;
// below, where the value is under 2^-126, the reciprocal gives 0 (off by at most
// 2^-126, before the factors of gate and up).  float32 takes the accurate ones: 0
// only where e^-z is beyond float32, below z = -88.7.
template <typename E>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(E) == 4) return 1.0f / (1.0f + expf(-z));
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// A lane's eight values of a group: neighbours, where rows are whole vectors
// (WIDE: I % 8 == 0); else every 16th.
template <bool WIDE>
__device__ __forceinline__ int place(int lane, int i) { return WIDE ? lane * kPer + i : i * kLanes + lane; }

// Where a group's gates lie in h; its up values are ups_from behind them.  For a
// lane of the TURN form (always WIDE): its place less what load8 and the like add.
// A form of its own: with halves as one turn of I, the same code for both, halves
// take longer on the same buffers (forward with the copy and backward, us, this /
// that: 65536 rows of 2048 231 + 191 / 243 + 193, 8192 rows 32.3 + 25.0 / 33.1 + 25.2,
// 1333 rows of 1408 float16 6.5 + 4.8 / 6.7 + 4.9; in two turns each, 1 % apart).
template <bool TURN>
__device__ __forceinline__ int64_t gate_at(const SwigluArgs& a, uint32_t row, uint32_t grp, int lane) {
  const int64_t base = (int64_t)row * 2 * a.I;
  if constexpr (TURN) {
    const uint32_t mine = grp * kGroup + lane * kPer, t = (uint32_t)a.turn;
    return base + mine + mine / t * t - lane * kPer;
  }
  return base + grp * kGroup;
}
template <bool TURN>
__device__ __forceinline__ int ups_from(const SwigluArgs& a) { return TURN ? a.turn : a.I; }

template <typename E, bool WIDE>
__device__ __forceinline__ void load8(const E* p, int lane, int n, float (&v)[kPer]) {
  if constexpr (WIDE) {
    if (lane * kPer < n) {
      load_elems(p + lane * kPer, v);
      return;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = place<false>(lane, i) < n ? (float)p[place<false>(lane, i)] : 0.0f;
  }
}

template <typename E, bool WIDE>
__device__ __forceinline__ void store8(E* p, int lane, int n, const float (&v)[kPer]) {
  if constexpr (WIDE) {
    if (lane * kPer < n) store_elems(p + lane * kPer, v);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (place<false>(lane, i) < n) p[place<false>(lane, i)] = (E)v[i];
  }
}

// the group's scale, and the lane's codes
template <bool WIDE>
__device__ __forceinline__ float keep8(const float (&v)[kPer], int8_t* q, int lane, int n) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = amax_of(v[i], m);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    const uint32_t w = (uint32_t)__shfl_xor((int)m, o, 64);
    m = w > m ? w : m;
  }
  const float s = int8_scale(m);
  if constexpr (WIDE) {
    if (lane * kPer < n) *reinterpret_cast<u32x2*>(q + lane * kPer) = int8_codes(v, s);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (place<false>(lane, i) < n) q[place<false>(lane, i)] = (int8_t)int8_code(v[i], s);
  }
  return s;
}

template <bool WIDE>
__device__ __forceinline__ void kept8(const int8_t* q, float s, int lane, int n, float (&v)[kPer]) {
  if constexpr (WIDE) {
    u32x2 w = {0u, 0u};
    if (lane * kPer < n) w = *reinterpret_cast<const u32x2*>(q + lane * kPer);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = (float)(int8_t)(w[i / 4] >> (8 * (i % 4))) * s;
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = place<false>(lane, i) < n ? (float)q[place<false>(lane, i)] * s : 0.0f;
  }
}

}  // namespace

// 16 lanes take a group of the gate and the same group of the up half.
template <typename E, bool WIDE, bool TURN, bool KEEP>
__global__ __launch_bounds__(kThreads) void k_swiglu(SwigluArgs a) {
  const int lane = threadIdx.x % kLanes;
  const uint32_t per_row = (uint32_t)((a.I + kGroup - 1) / kGroup), total = (uint32_t)a.groups;
  const E* h = static_cast<const E*>(a.h);
  E* out = static_cast<E*>(a.a);
  for (uint32_t at = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes; at < total; at += gridDim.x * (kThreads / kLanes)) {
    const uint32_t row = at / per_row, grp = at % per_row;
    const int n = a.I - (int)grp * kGroup;               // values from here to the row's end
    const int64_t gate = gate_at<TURN>(a, row, grp, lane), up = gate + ups_from<TURN>(a);
    float g[kPer], u[kPer], o[kPer];
    load8<E, WIDE>(h + gate, lane, n, g);
    load8<E, WIDE>(h + up, lane, n, u);
    if constexpr (KEEP) {
      const float sg = keep8<WIDE>(g, a.q + gate, lane, n), su = keep8<WIDE>(u, a.q + up, lane, n);
      float* s = a.s + (int64_t)row * 2 * per_row + grp;
      if (lane == 0) s[0] = sg;
      if (lane == 1) s[per_row] = su;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float gc = clamped(g[i], a.clamp);
      o[i] = gc * sigmoid<E>(gc) * clamped(u[i], a.clamp);
    }
    store8<E, WIDE>(out + (int64_t)row * a.I + grp * kGroup, lane, n, o);
  }
}

template <typename E, bool WIDE, bool TURN>
__global__ __launch_bounds__(kThreads) void k_swiglu_backward(SwigluArgs a) {
  const int lane = threadIdx.x % kLanes;
  const uint32_t per_row = (uint32_t)((a.I + kGroup - 1) / kGroup), total = (uint32_t)a.groups;
  const E* da = static_cast<const E*>(a.da);
  E* dh = static_cast<E*>(a.dh);
  for (uint32_t at = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes; at < total; at += gridDim.x * (kThreads / kLanes)) {
    const uint32_t row = at / per_row, grp = at % per_row;
    const int n = a.I - (int)grp * kGroup;
    const int64_t gate = gate_at<TURN>(a, row, grp, lane), up = gate + ups_from<TURN>(a);
    const float* s = a.s + (int64_t)row * 2 * per_row + grp;
    float g[kPer], u[kPer], d[kPer];
    load8<E, WIDE>(da + (int64_t)row * a.I + grp * kGroup, lane, n, d);
    kept8<WIDE>(a.q + gate, s[0], lane, n, g);
    kept8<WIDE>(a.q + up, s[per_row], lane, n, u);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float gc = clamped(g[i], a.clamp), uc = clamped(u[i], a.clamp), sig = sigmoid<E>(gc);
      // (a NaN is in no interval's outside: it stays)
      const bool gout = fabsf(g[i]) > a.clamp, uout = fabsf(u[i]) > a.clamp;
      g[i] = gout ? 0.0f : d[i] * uc * sig * (1.0f + gc * (1.0f - sig));
      u[i] = uout ? 0.0f : d[i] * gc * sig;
    }
    store8<E, WIDE>(dh + gate, lane, n, g);
    store8<E, WIDE>(dh + up, lane, n, u);
  }
}

namespace {

template <typename F>
hipError_t for_type(const SwigluArgs& a, const F& f) {
  auto wide = [&](auto e) {
    if (a.turn) return f(e, std::true_type{}, std::true_type{});        // of 8s, so I is too
    return a.I % kPer == 0 ? f(e, std::true_type{}, std::false_type{}) : f(e, std::false_type{}, std::false_type{});
  };
  return a.element == MM_ELEMENT_BF16 ? wide(__bf16{}) : a.element == MM_ELEMENT_F16 ? wide(_Float16{}) : wide(float{});
}

unsigned grid_of(int64_t groups) {
  const int64_t n = (groups + kThreads / kLanes - 1) / (kThreads / kLanes);
  return (unsigned)(n < (1 << 20) ? n : (1 << 20));
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s) {
  return for_type(a, [&](auto e, auto w, auto t) {
    typedef decltype(e) E;
    constexpr bool W = decltype(w)::value, T = decltype(t)::value;
    if (a.q != nullptr) hipLaunchKernelGGL((k_swiglu<E, W, T, true>), dim3(grid_of(a.groups)), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((k_swiglu<E, W, T, false>), dim3(grid_of(a.groups)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_swiglu_backward(const SwigluArgs& a, hipStream_t s) {
  return for_type(a, [&](auto e, auto w, auto t) {
    hipLaunchKernelGGL((k_swiglu_backward<decltype(e), decltype(w)::value, decltype(t)::value>), dim3(grid_of(a.groups)),
                       dim3(kThreads), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace mm
