// What the 8-bit attention kernels share: the schedule, code conversion and
// the exact handling of ranges.
//
// Schedule.  A unit is (sequence, KV head, query tile); all units of a
// sequence have the same number of key tiles (one with the block's own keys, the
// others with 128 context keys each), so the tile sequence is described by prefix
// sums over the B sequences alone, and every CTA computes them itself from
// ctx_len instead of waiting for a planning kernel.  CTA c takes the tiles
// [c T / P, (c + 1) T / P) of the T tiles; its part of unit u (a segment) has
// the partial record u + c, which no other segment has.  T < 2^31 is checked
// on the host: the arithmetic is 32-bit, and the whole prologue small, because
// every launch pays for it.
#pragma once
#include "tt_q8.h"
#include "tt_ptx.cuh"

namespace tt {

// One position in the tile sequence and what is left of the CTA's range.
struct TileWalk {
  const int* ctx_len;
  int left;         // tiles of the range not yet handed out
  int B, L_cap, U;  // U: units per sequence
  int b, k;         // sequence, unit within it
  int off;          // tile within the unit
  int len;          // sequence b's context length, loaded when b is reached
  // The next segment: unit (b, k), local tiles [a, e), context length L.
  __host__ __device__ __forceinline__ bool next(int& sb, int& sk, int& a, int& e, int& L) {
    if (left <= 0) return false;
    L = min(max(len, 0), L_cap);
    const int n = 1 + (L + kAttnBN - 1) / kAttnBN;
    sb = b;
    sk = k;
    a = off;
    e = min(n, off + left);
    left -= e - a;
    off = 0;
    if (++k == U) {
      k = 0;
      ++b;
      len = b < B ? ctx_len[b] : 0;
    }
    return true;
  }
};

struct PlanSmem {
  int warp_tot[32];
  int b, pre;
};

// First tile of CTA c, floor(c T / P) (P <= 1024: no product leaves 32 bits).
__host__ __device__ __forceinline__ int cta_first(int c, int T, int P) {
  const int base = T / P;
  return c * base + c * (T - base * P) / P;
}

// Every thread of the CTA: the CTA's walk.  CTA 0 also starts the error word (an
// out-of-range length is clamped and recorded).  NT: threads of the CTA.
template <int NT>
__device__ __forceinline__ TileWalk plan_walk(const AttnQ8Args& a, PlanSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  auto tiles = [&](int b, int& bad) {
    const int L = a.ctx_len[b];
    bad |= L < 0 || L > a.L_cap;
    return 1 + (min(max(L, 0), a.L_cap) + kAttnBN - 1) / kAttnBN;
  };
  int sum = 0, bad = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) sum += tiles(b, bad);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm.warp_tot[warp] = incl;
  bad = __syncthreads_or(bad);
  const int mine = lane < NT / 32 ? sm.warp_tot[lane] : 0;
  const int total = __reduce_add_sync(0xffffffffu, mine);
  int pre = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
  const int U = a.Hkv * a.n_qtiles, T = total * U;
  const int lo = cta_first(blockIdx.x, T, a.n_ctas);
  if (blockIdx.x == 0 && tid == 0) {
    a.err[0] = bad ? (int)TT_ERR_INVALID_ARG : 0;
    a.err[1] = 0;
  }
  if (lo >= pre * U && lo < (pre + sum) * U) {  // exactly one thread
    int b = b0, x = 0;
#pragma unroll 1
    for (;; ++b) {
      const int n = tiles(b, x);
      if (lo < (pre + n) * U) break;
      pre += n;
    }
    sm.b = b;
    sm.pre = pre;
  }
  __syncthreads();
  TileWalk w;
  w.ctx_len = a.ctx_len;
  w.B = a.B;
  w.L_cap = a.L_cap;
  w.U = U;
  w.left = cta_first(blockIdx.x + 1, T, a.n_ctas) - lo;
  w.b = sm.b;
  w.len = a.ctx_len[w.b];
  const int n = 1 + (min(max(w.len, 0), a.L_cap) + kAttnBN - 1) / kAttnBN;
  const int rem = lo - sm.pre * U;
  w.k = rem / n;
  w.off = rem - w.k * n;
  return w;
}

// Recorded for the merge by the CTAs that hold a unit's first and last tile: all
// CTAs between have a record (an empty range inside the unit an empty one).
__host__ __device__ __forceinline__ void put_span(int2* unit_span, size_t u, int cta, bool first,
                                                  bool last) {
  if (first) unit_span[u].x = cta;
  if (last) unit_span[u].y = cta;
}
// The spans of all segments of a CTA's walk.
__host__ __device__ __forceinline__ void put_spans(int2* unit_span, TileWalk walk, int cta) {
  int b, k, lo, hi, L;
  while (walk.next(b, k, lo, hi, L))
    put_span(unit_span, (size_t)b * walk.U + k, cta, lo == 0, hi == 1 + (L + kAttnBN - 1) / kAttnBN);
}
// What a merge may read of a launch of n_ctas CTAs.
__host__ __device__ __forceinline__ bool span_in_range(int2 s, int n_ctas) {
  return s.x >= 0 && s.x <= s.y && s.y < n_ctas;
}

// 2^e, e in [-126, 127]
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Exponent e with amax 2^-e in [2^14, 2^15), for the bf16 magnitude bits amax
// (clamped so that 2^e and 2^-e are normal; 0 for zero and for non-finite).
__device__ __forceinline__ int norm_exp(uint32_t amax) {
  const int e = (int)(amax >> 7);
  return amax == 0 || e == 255 ? 0 : min(max(e - 127 - 14, -126), 126);
}

// Factor of a row's scores with a group of keys: the row's c times the keys' scale
// k, held above 0, because a masked score is -inf and -inf * 0 is NaN.  2^-126
// stands for anything below: the products that it multiplies are below 2^38.
// (Positive floats and the NaN of a product are ordered as integers are.)
__device__ __forceinline__ float score_factor(float c, float k) {
  return __int_as_float(max(__float_as_int(c * k), 0x00800000));
}

// Probabilities are fp16 numbers up to 2^kTop: m is set to a new maximum less kPeak, and
// again when a later one passes m + kTop.  The lower kPeak, the sooner a small
// probability is a subnormal fp16 number and then 0 (below 2^-25), and its key is
// missing from the product that the row sum counts; the higher, the more often O is
// rescaled.  (kPeak 7, 10, 12, 13: 80.3, 80.4, 82.3 and 89.5 us for 4 sequences of 65536
// int8 keys, 221, 221, 227 and 245 for 48 of up to 32768.)
constexpr float kTop = 15.f, kPeak = 10.f;

// Ranges.  With m that reference of s_j + log2 w_j, a key's part of the row
// sum is 2^(s_j - m) = p_j / w_j.  Three things keep it what it is:
//  - w >= 2^-100 (the cache's scales are at least 2^-60, the own values' exponent
//    is held there: values below 2^-114 lose bits, below 2^-125 they are 0), so that
//    the sum stays below 2^127;
//  - p_j is 0 below 2^-126, where p_j / w_j may still count, so w is also held at
//    2^-100 of the largest so far: m <= max s + max log2 w leaves every key of weight
//    2^-26 and more a p that is a number, and what is held moves a value by
//    2^-85 of the largest at most;
//  - a new maximum can move the sum by 2^-220, which is no number either: by its
//    square root, twice.
// A record is a segment's own normalised output with log2 of its sum, m + log2 l,
// in which w no longer occurs.
constexpr int kOwnLow = -100;
__device__ __forceinline__ int own_value_exp(uint32_t amax) { return max(norm_exp(amax), kOwnLow); }
// (NaN stays NaN)
__device__ __forceinline__ float value_scale(float w, float top) {
  const float low = top * 0x1p-100f;
  return w < low ? low : w;
}
// Two running maxima (packed) of bf16 magnitudes.
__device__ __forceinline__ uint32_t absmax_bf16x8(uint32_t m, const uint4& v) {
  m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
  return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// bf16 pair times a power of two, as an fp16 pair
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float f) {
  return pack_f16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
}

// Two codes in the low 16 bits (after int8 codes had their sign bits flipped)
// to an fp16 pair.  int8: the flipped byte is the code + 128, which as the
// low byte of 0x64xx makes 1024 + 128 + code.
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// Four codes to two fp16 pairs.
template <int TYPE>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (TYPE == TT_Q8_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    lo = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

}  // namespace tt
