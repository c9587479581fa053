// Values of the element types (bf16, float16, float32) as float32, and codes
// of 8 bits with a scale.
#pragma once
#include "mm_device.hpp"

namespace mm {
namespace {

template <int V> struct Bytes;
template <> struct Bytes<16> { typedef u32x4 type; };
template <> struct Bytes<8> { typedef u32x2 type; };
template <> struct Bytes<4> { typedef uint32_t type; };
template <> struct Bytes<2> { typedef uint16_t type; };
template <> struct Bytes<1> { typedef uint8_t type; };

// N values of an element type as float32, and back with one rounding
template <typename E, int N>
struct Elems {
  typedef typename Bytes<sizeof(E) * N>::type vec;
  union Both { vec v; E e[N]; };
  static __device__ __forceinline__ void unpack(const vec& v, float (&f)[N]) {
    Both u;
    u.v = v;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = (float)u.e[i];
  }
  static __device__ __forceinline__ vec pack(const float (&f)[N]) {
    Both u;
#pragma unroll
    for (int i = 0; i < N; ++i) u.e[i] = (E)f[i];
    return u.v;
  }
  static __device__ __forceinline__ void load(const void* p, float (&f)[N]) { unpack(*reinterpret_cast<const vec*>(p), f); }
  static __device__ __forceinline__ void store(void* p, const float (&f)[N]) { *reinterpret_cast<vec*>(p) = pack(f); }
};

// eight neighbours, at an address of their own size
template <typename E>
__device__ __forceinline__ void load_elems(const E* p, float (&f)[8]) {
  if constexpr (sizeof(E) == 2) {
    Elems<E, 8>::load(p, f);
  } else {
    float a[4], b[4];
    Elems<E, 4>::load(p, a);
    Elems<E, 4>::load(p + 4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
  }
}
template <typename E>
__device__ __forceinline__ void store_elems(E* p, const float (&f)[8]) {
  if constexpr (sizeof(E) == 2) {
    Elems<E, 8>::store(p, f);
  } else {
    const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
    Elems<E, 4>::store(p, a);
    Elems<E, 4>::store(p + 4, b);
  }
}

// eight neighbours as they are in memory
template <typename E>
struct Raw8 {
  u32x4 v[sizeof(E) / 2];
  __device__ __forceinline__ void load(const E* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(E) / 2; ++i) v[i] = reinterpret_cast<const u32x4*>(p)[i];
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    if constexpr (sizeof(E) == 2) {
      Elems<E, 8>::unpack(v[0], f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i / 4][i % 4]);
    }
  }
};

// Largest magnitude so far, as float bits: integer order is magnitude order,
// and a NaN is above infinity.
__device__ __forceinline__ uint32_t amax_of(float v, uint32_t m) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b > m ? b : m;
}

// Scale and code of symmetric 8-bit integers, decided in IEEE float32.  With a
// NaN or an infinity among the values the scale is one too, codes are 0, and
// code * scale is NaN.
__device__ __forceinline__ float int8_scale(uint32_t amax) {
  const float s = __uint_as_float(amax) / 127.0f;
  return s < 1e-8f ? 1e-8f : s;        // NaN stays
}
__device__ __forceinline__ int int8_code(float v, float s) {
  const float q = __builtin_rintf(v / s);
  return q >= -127.0f ? (int)(q > 127.0f ? 127.0f : q) : q < -127.0f ? -127 : 0;
}

// Eight codes at once, the same ones: a product with the reciprocal is within
// 2^-15 of the quotient (three roundings of at most 127 * 2^-24 and one more of
// the quotient's own), so it rounds to the same integer unless it is that near
// to the middle between two; only then are the quotients taken.  (Sixteen IEEE
// divisions a lane: 320 us for the copy of 65536 x 4096 bf16 values with its
// activation; this way 280.)
// t + 1.5 * 2^23 has the rounded integer in its low bits.
__device__ __forceinline__ u32x2 int8_codes(const float (&v)[8], float s) {
  constexpr float kShift = 12582912.0f;
  const float r = 1.0f / s;
  uint32_t bits[8];
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = v[i] * r, u = t + kShift;
    bits[i] = __float_as_uint(u);
    most = fmaxf(most, fabsf(t - (u - kShift)));
  }
  if (most > 0.5f - 0x1p-14f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) bits[i] = (uint32_t)int8_code(v[i], s);
  }
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(bits[4 * h + 1], bits[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(bits[4 * h + 3], bits[4 * h + 2], 0x04000c0cu);
    o[h] = s < INFINITY ? lo | hi : 0u;      // (no codes beside a scale that is no number)
  }
  return o;
}

}  // namespace
}  // namespace mm
