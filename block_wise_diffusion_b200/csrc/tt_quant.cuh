// Rounding to 8-bit codes with a scale, shared by the kernels that write them.
//
// The code of x under scale s is x / s rounded to the nearest code, ties to
// even, as if the quotient were exact.  The quotient is taken as x * (1 / s):
// two roundings, at most 2^-22.4 relative off.  That decides the nearest code
// unless it lies next to the middle of two codes; there (about one value in
// a thousand) the sign of x - h s decides, h being the middle: a product of
// a short and a 24-bit significand less x, so one FMA rounds it without
// losing the sign, and 0 is a true tie.
#pragma once
#include <stdint.h>

#include "tt_ptx.cuh"

namespace tt {

constexpr float kScaleFloor = 8.673617379884035e-19f;  // 2^-60

// Largest code of a cache or row type, and the scale of a group whose largest
// magnitude has the bf16 bits `amax` (sign cleared).  NaN and infinity have
// the largest bit patterns, so an integer maximum over the magnitudes keeps
// them; they give the scale NaN.
template <int TYPE>
__device__ __forceinline__ float q8_scale(uint32_t amax) {
  if (amax >= 0x7F80u) return __uint_as_float(0x7FFFFFFFu);
  constexpr float kInv = 1.f / (TYPE == TT_Q8_INT8 ? 127.f : 448.f);
  return fmaxf(__fmul_rn(bf16_value((uint16_t)amax), kInv), kScaleFloor);
}

// Nearest of a grid of spacing `step` (a power of two) to y / s, ties to even
// multiples, given t within 2^-22 relative of y / s; y, s > 0.
__device__ __forceinline__ float round_exact(float y, float s, float t, float step) {
  const float k2 = rintf(2.f * t / step);  // in half steps (exact scaling)
  const float lo = floorf(0.5f * k2);      // grid index at or below
  if (k2 == 2.f * lo) return lo * step;    // nearer to a grid point than to a middle
  const float r = fmaf(-(lo + 0.5f) * step, s, y);
  const float even = 2.f * rintf(0.5f * lo) == lo ? lo : lo + 1.f;
  return (r > 0.f ? lo + 1.f : r < 0.f ? lo : even) * step;
}

// int8 code of x (|x| <= 127 s up to the rounding of s), inv = 1 / s.
__device__ __forceinline__ int q8_int8(float x, float s, float inv) {
  const float t = x * inv;
  float n = rintf(t);
  // |t| <= 127.0001 and its error is below 127 * 2^-22 < 2^-15
  if (fabsf(t - n) > 0.49996f) n = copysignf(round_exact(fabsf(x), s, fabsf(t), 1.f), x);
  return (int)fminf(fmaxf(n, -127.f), 127.f);
}

__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The e4m3 value nearest to x / s as a float: exact near the middle of two
// codes (the 20 bits below a normal's third mantissa bit near 0x80000) and
// for the subnormal codes, whose spacing is 2^-9; x / s itself elsewhere (the
// conversion rounds it).
__device__ __forceinline__ float e4m3_near(float x, float s, float inv) {
  const float t = x * inv;
  const uint32_t u = __float_as_uint(t) & 0x7FFFFFFFu;
  const uint32_t d = (u & 0xFFFFFu) - (0x80000u - 16u);
  if (d > 32u && u >= 0x3C800000u) return t;  // 0x3C800000: 2^-6
  if (u == 0u) return t;
  const int e = max((int)(u >> 23) - 127, -6);
  const float step = __uint_as_float((uint32_t)(e - 3 + 127) << 23);
  return copysignf(round_exact(fabsf(x), s, fabsf(t), step), x);
}

// Four codes as bytes, lowest first.
template <int TYPE>
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d, float s,
                                             float inv) {
  if constexpr (TYPE == TT_Q8_INT8) {
    return (uint32_t)(q8_int8(a, s, inv) & 255) | (uint32_t)(q8_int8(b, s, inv) & 255) << 8 |
           (uint32_t)(q8_int8(c, s, inv) & 255) << 16 | (uint32_t)(q8_int8(d, s, inv) & 255) << 24;
  } else {
    return cvt_e4m3x2(e4m3_near(a, s, inv), e4m3_near(b, s, inv)) |
           cvt_e4m3x2(e4m3_near(c, s, inv), e4m3_near(d, s, inv)) << 16;
  }
}

// Eight bf16 values (one 16-byte vector) to eight codes.
template <int TYPE>
__device__ __forceinline__ uint2 q8_pack8(const uint4& v, float s, float inv) {
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  return make_uint2(q8_pack4<TYPE>(lo(v.x), hi(v.x), lo(v.y), hi(v.y), s, inv),
                    q8_pack4<TYPE>(lo(v.z), hi(v.z), lo(v.w), hi(v.w), s, inv));
}

// Largest magnitude of eight bf16 values, merged into two running 16-bit
// maxima (packed).
__device__ __forceinline__ uint32_t absmax8(uint32_t m, const uint4& v) {
  m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
  return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t absmax_fold(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

// An older code under a new, larger scale: the nearest code of c * s_old /
// s_new.  c * s_old is exact in 64 bits and the quotient of two numbers of
// at most 32 significant bits is, unless it is a middle itself, further than
// 2^-34 relative from any middle of two codes, so the 64-bit quotient decides.
template <int TYPE>
__device__ __forceinline__ uint32_t q8_recode(uint32_t byte, float s_old, float s_new) {
  if constexpr (TYPE == TT_Q8_INT8) {
    const double t = (double)(int)(int8_t)byte * (double)s_old / (double)s_new;
    return (uint32_t)((int)fmin(fmax(rint(t), -127.0), 127.0)) & 255u;
  } else {
    if ((byte & 0x7Fu) == 0x7Fu) return byte;  // NaN stays
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)byte));
    const uint32_t h = h2 & 0xFFFFu;
    // e4m3 magnitudes are fp16 numbers: widen by hand (normal or zero; the
    // smallest, 2^-9, is a normal fp16 number)
    const uint32_t mag = h & 0x7FFFu;
    const float c = mag == 0 ? 0.f : __uint_as_float((mag << 13) + ((127u - 15u) << 23));
    const double t = (double)c * (double)s_old / (double)s_new;
    if (t == 0.0) return byte & 0x80u;
    const int e = max((int)((__double2hiint(t) >> 20) & 0x7FF) - 1023, -6);
    const double step = __hiloint2double((e - 3 + 1023) << 20, 0);
    const float r = (float)(rint(t / step) * step);  // a code: exact
    return (cvt_e4m3x2(r, 0.f) & 0x7Fu) | (byte & 0x80u);
  }
}

}  // namespace tt
