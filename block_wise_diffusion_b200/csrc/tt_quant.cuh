// Rounding to 8-bit codes with a scale, shared by the kernels that write them.
//
// The code of x under scale s is x / s rounded to the nearest code, ties to
// even, as if the quotient were exact.  The quotient is taken as t = x * (1 /
// s): two roundings, at most two units of its last place off.  t gives the two
// codes around x / s and the middle h between them (next to a code itself it
// may give the wrong pair, but then the same nearest code), and the sign of
// x - h s decides: h has a short significand, so one FMA rounds that
// difference without losing its sign, and 0 is a true tie.
// Such quotients are no rarity: half a group's largest value always lies within
// a rounding of a middle of int8 codes (63.5), and one value in 200 of normal
// data is that near to one of e4m3, half of them on it, which a third of a warp's
// vectors meet.  So nothing here takes a long path for them.
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

__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}

// Eight bf16 values (one 16-byte vector) to eight codes; inv = 1 / s.
template <int TYPE>
__device__ __forceinline__ uint2 q8_pack8(const uint4& v, float s, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint2 r;
  if constexpr (TYPE == TT_Q8_INT8) {
    // Rounded down by adding 1.5 * 2^23 (the integer's two's complement is then
    // in the low byte), and up by one where x lies above the middle.
    uint32_t m[8];
    float tie = 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
      const float k = __fadd_rd(x * inv, 12582912.f);
      const float d = fmaf(-((k - 12582912.f) + 0.5f), s, x);
      m[i] = __float_as_uint(k) + 1u + (uint32_t)(__float_as_int(d) >> 31);
      tie = fminf(tie, fabsf(d));
    }
    r = make_uint2(prmt(prmt(m[0], m[1], 0x40), prmt(m[2], m[3], 0x40), 0x5410),
                   prmt(prmt(m[4], m[5], 0x40), prmt(m[6], m[7], 0x40), 0x5410));
    if (tie == 0.f) {  // true ties, above: an odd code down to the even one
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const uint32_t wi = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        const float x = __uint_as_float(i & 1 ? wi & 0xFFFF0000u : wi << 16);
        const float k = __fadd_rd(x * inv, 12582912.f);
        const uint32_t odd = fmaf(-((k - 12582912.f) + 0.5f), s, x) == 0.f ? 1u << (8 * (i & 3)) : 0u;
        if (i < 4)
          r.x &= ~odd;
        else
          r.y &= ~odd;
      }
    }
  } else {
    // The conversion rounds t; where t a little smaller and a little larger
    // (2^-22 relative, more than its error) give the same code, x / s does too.
    // Else, pair by pair, the codes around t by its upper bits (below 2^-6,
    // where codes are 2^-9 apart: of t + 2^-6, whose spacing is theirs), up by
    // one above the middle, or on it from an odd code.
    const float lo = inv * (1.f - 0x1p-22f), hi = inv * (1.f + 0x1p-22f);
    uint32_t c[4], d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xFFFF0000u);
      c[i] = cvt_e4m3x2(x0 * lo, x1 * lo);
      d[i] = cvt_e4m3x2(x0 * hi, x1 * hi);
    }
    r = make_uint2(prmt(c[0], c[1], 0x5410), prmt(c[2], c[3], 0x5410));
    const uint32_t dx = r.x ^ prmt(d[0], d[1], 0x5410), dy = r.y ^ prmt(d[2], d[3], 0x5410);
    uint32_t open = 0;
    if ((dx | dy) != 0)
      open = ((dx & 0xFFFFu) != 0) | ((dx >> 16) != 0) << 1 | ((dy & 0xFFFFu) != 0) << 2 |
             ((dy >> 16) != 0) << 3;
    // (a loop, not four copies: code that few lanes run should not fill the
    // instruction cache)
#pragma unroll 1
    for (; open != 0; open &= open - 1) {
      const int i = __ffs(open) - 1;
      const uint32_t wi = i < 2 ? (i ? v.y : v.x) : (i == 2 ? v.z : v.w);
      uint32_t code = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float x = __uint_as_float(k ? wi & 0xFFFF0000u : wi << 16), u = fabsf(x * inv);
        const bool sub = u < 0.015625f;
        const float o = sub ? 0.015625f : 0.f;
        const uint32_t y = __float_as_uint(u + o);
        const float h = __uint_as_float((y & 0xFFF00000u) | 0x80000u) - o;
        const float e = fmaf(-h, s, fabsf(x));
        const uint32_t low = (y >> 20) - (sub ? 968u : 960u);
        const bool up = e > 0.f || (e == 0.f && (low & 1u) != 0);
        code |= ((low + (up ? 1u : 0u)) | (__float_as_uint(x) >> 24 & 0x80u)) << (8 * k);
      }
      const uint32_t sel = i & 1 ? 0x5410u : 0x3254u;
      uint32_t& half = i < 2 ? r.x : r.y;
      half = prmt(half, code, sel);
    }
  }
  return r;
}

// The scale of a group is nearly always that of its own largest magnitude A.  Then
// x / s = q / (1 + e) with q = x qmax / A and |e| < 2^-23, e the rounding of s
// alone, and a q that is no middle of two codes is further than 2^-17 from any:
// q and a middle h are ratios of integers below 2^16 (x and A have 8 bits, qmax 7,
// h at most 8), so they differ by at least 2^-16 of h.  Every quotient near a
// middle therefore lies on the same side of it, above for e < 0 and below for e >
// 0, and x * (1 / s) moved by 2^-22 to that side (more than its three roundings)
// rounds to the same code.  Returns that factor, or 0 where the group needs
// q8_pack8: e = 0 (true ties) or the scale is the floor.
template <int TYPE>
__device__ __forceinline__ float q8_own_factor(uint32_t amax, float s) {
  constexpr float kMax = TYPE == TT_Q8_INT8 ? 127.f : 448.f;
  const float e = fmaf(s, kMax, -bf16_value((uint16_t)amax));
  const float f = (1.f / s) * (e > 0.f ? 1.f - 0x1p-22f : 1.f + 0x1p-22f);
  return e == 0.f || !(s > kScaleFloor) ? 0.f : f;
}
// Eight values to codes with that factor.
template <int TYPE>
__device__ __forceinline__ uint2 q8_pack8_own(const uint4& v, float f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xFFFF0000u);
    if constexpr (TYPE == TT_Q8_INT8) {
      // (the low byte of 1.5 * 2^23 + n is n's)
      m[2 * i] = __float_as_uint(fmaf(x0, f, 12582912.f));
      m[2 * i + 1] = __float_as_uint(fmaf(x1, f, 12582912.f));
    } else {
      m[i] = cvt_e4m3x2(x0 * f, x1 * f);
    }
  }
  if constexpr (TYPE == TT_Q8_INT8)
    return make_uint2(prmt(prmt(m[0], m[1], 0x40), prmt(m[2], m[3], 0x40), 0x5410),
                      prmt(prmt(m[4], m[5], 0x40), prmt(m[6], m[7], 0x40), 0x5410));
  else
    return make_uint2(prmt(m[0], m[1], 0x5410), prmt(m[2], m[3], 0x5410));
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
