// Block-denoise attention over an 8-bit cache for at most 16 query rows per
// KV head (the autoregressive step: one position and up to 16 heads).
//
// With so few rows the work is streaming the cache: 2 dh bytes per key
// against 16 rows of arithmetic, far below the tensor cores' rate, so what
// matters is bytes in flight and instructions per byte.  The codes go from
// global memory straight into the operand registers of warp-level matrix
// instructions (m16n8k16, fp16): no shared memory and no barrier on the way.
// That works because the order of dh inside a product is free:
//   S = Q K^T   lane (n, c) = (lane / 4, lane % 4) loads two runs of dh/8 codes
//               of key n (one from each half of the row, so that the lanes of
//               a key read whole sectors); its word j is exactly the operand
//               of step j;
//   O += P V    lane (n, c) loads dh/8 consecutive codes (columns n dh/8 ..) of
//               the keys 2c, 2c+1, 2c+8, 2c+9; byte j of a pair of keys is the
//               operand of column tile j.
// Each warp takes every 8th group of 32 keys with a running maximum and sum
// of its own (the formulas of tt_attn_q8.cu) and refills a register buffer as
// soon as the products have read it.  The 8 warps' results are joined through
// shared memory at a segment's end.
// What bounds it: latency.  248 registers leave two warps to a scheduler, and a
// warp's next keys are requested when the products have read its registers: 0.30
// instructions per cycle and scheduler, no pipe above 28 %, DRAM at 35 %, the stalls
// are loads and fixed latencies.  64 sequences of up to 8192 keys, 2 KV heads of 16
// queries, dh 128, with the merge: e4m3 48 us (2.9 TB/s), int8, whose conversion is
// longer, 52.
#include <math.h>

#include "tt_attn_q8.cuh"

namespace tt {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int NG = 2, kGroup = 16 * NG;  // keys per step of a warp

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// N (2 or 4) words of codes from global memory, not kept in L1.
template <int N>
__device__ __forceinline__ void load_words(uint32_t* x, const uint8_t* p) {
  if constexpr (N == 2)
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                 : "=r"(x[0]), "=r"(x[1])
                 : "l"(p));
  else
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "l"(p));
}
// Where the i-th vector of 8 values of a lane's dh/4 lies: its first run of dh/8
// is in the first half of the row, the second in the other.
template <int DH>
__device__ __forceinline__ constexpr int run_at(int i) {
  return i < DH / 64 ? 8 * i : DH / 2 + 8 * (i - DH / 64);
}

template <int TYPE, int DH>
__global__ void __launch_bounds__(kThreads, 1) attn_q8_rows_kernel(const AttnQ8Args a) {
  griddep_launch();
  griddep_wait();
  extern __shared__ __align__(16) float sm_o[];  // [warp][16][DH + 4]
  __shared__ PlanSmem plan;
  __shared__ float sm_lse[kWarps][16], sm_inv[kWarps][16];
  constexpr int KW = DH / 16;  // words of a key per lane (K side), steps of Q K^T
  constexpr int VW = DH / 32;  // words of a key per lane (V side)
  constexpr int NT = DH / 8;   // column tiles of O
  constexpr int LDO = DH + 4;
  TileWalk walk = plan_walk<kThreads>(a, plan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n8 = lane >> 2, c4 = lane & 3;
  const int rows = a.rows_per_half;
  if (walk.left == 0) {
    if (walk.off > 0) {  // an empty range inside a unit: an empty record
      const size_t slot = (size_t)walk.b * a.Hkv + walk.k + blockIdx.x;
      if (threadIdx.x < 16) a.part_lse[slot * 16 + threadIdx.x] = -INFINITY;
    }
    return;
  }
  int ub, ug, sa, sb, L;
  while (walk.next(ub, ug, sa, sb, L)) {
    const size_t pair = (size_t)ub * a.Hkv + ug;
    uint32_t q[KW][4];
    float c_row[2];
    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, w_top = 0.f;

    // Softmax of NTILE 8-key tiles of scores (16 keys share a scale) and its
    // product with V: `vfrag(t16, j, b0, b1)` gives the operands of keys
    // t16*16.. and column tiles j .. j + 3.  nv: valid keys.
    auto finish = [&](auto& s, const float* sk, const float* lw, const float* iw, int nv,
                      auto&& vfrag) {
      constexpr int N16 = sizeof(s) / sizeof(s[0]) / 2;
      if (nv < 16 * N16) {
#pragma unroll
        for (int t = 0; t < 2 * N16; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (t * 8 + c4 * 2 + e >= nv) s[t][e] = s[t][2 + e] = -INFINITY;
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int g = 0; g < N16; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float y = fmaxf(fmaxf(s[2 * g][2 * h], s[2 * g][2 * h + 1]),
                                fmaxf(s[2 * g + 1][2 * h], s[2 * g + 1][2 * h + 1]));
          mx[h] = fmaxf(mx[h], fmaf(y, score_factor(c_row[h], sk[g]), lw[g]));
        }
      bool need = false;
      float alpha[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        alpha[h] = 1.f;
        if (mx[h] > m[h] + kTop) {
          const float half = ex2(0.5f * (m[h] - (mx[h] - kPeak)));
          alpha[h] = half * half;
          l[h] = l[h] * half * half;
          m[h] = mx[h] - kPeak;
          need = true;
        }
      }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][0] *= alpha[0];
          o[j][1] *= alpha[0];
          o[j][2] *= alpha[1];
          o[j][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int g = 0; g < N16; ++g) {
        uint32_t p[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float cg = score_factor(c_row[h], sk[g]), off = lw[g] - m[h];
          const float p0 = ex2(fmaf(s[2 * g][2 * h], cg, off));
          const float p1 = ex2(fmaf(s[2 * g][2 * h + 1], cg, off));
          const float p2 = ex2(fmaf(s[2 * g + 1][2 * h], cg, off));
          const float p3 = ex2(fmaf(s[2 * g + 1][2 * h + 1], cg, off));
          l[h] = fmaf((p0 + p1) + (p2 + p3), iw[g], l[h]);
          p[h] = pack_f16x2(p0, p1);
          p[2 + h] = pack_f16x2(p2, p3);
        }
#pragma unroll
        for (int j = 0; j < NT; j += 4) {
          uint32_t b0[4], b1[4];
          vfrag(g, j, b0, b1);
#pragma unroll
          for (int i = 0; i < 4; ++i) mma16816(o[j + i], p, b0[i], b1[i]);
        }
      }
    };

    // ---- the context keys of the segment, group by group
    const int key_lo = (max(sa, 1) - 1) * kAttnBN, key_hi = min((sb - 1) * kAttnBN, L);
    const uint8_t* kp = a.k_ctx + pair * a.L_cap * DH + (size_t)n8 * DH + c4 * (DH / 8);
    const uint8_t* vp = a.v_ctx + pair * a.L_cap * DH + (size_t)(2 * c4) * DH + n8 * (DH / 8);
    const float* ksp = a.k_scale + pair * a.n_blocks;
    const float* vsp = a.v_scale + pair * a.n_blocks;
    uint32_t kr[2 * NG][KW], vr[4 * NG][VW];
    // Keys past the segment's end read its last key instead (their scores are
    // masked): no branch and no zero fill between the loads.
    const int kb = key_hi - 1 - n8, vb = key_hi - 1 - 2 * c4;
    auto load_k = [&](int key0) {
#pragma unroll
      for (int t = 0; t < 2 * NG; ++t) {
        const uint8_t* p = kp + (ptrdiff_t)min(key0 + t * 8, kb) * DH;
        load_words<KW / 2>(&kr[t][0], p);
        load_words<KW / 2>(&kr[t][KW / 2], p + DH / 2);
      }
    };
    // vr[4 g + i]: key 16 g + 2 c4 + {0, 1, 8, 9}[i]
    auto load_v = [&](int key0) {
#pragma unroll
      for (int i = 0; i < 4 * NG; ++i) {
        const int at = (i >> 2) * 16 + (i & 1) + ((i >> 1) & 1) * 8;
        load_words<VW>(vr[i], vp + (ptrdiff_t)min(key0 + at, vb) * DH);
      }
    };
    float nks[NG], nvs[NG];
    auto load_scales = [&](int key0) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int pos = key0 + 16 * g;
        nks[g] = pos < key_hi ? __ldg(ksp + (pos >> a.block_shift)) : 1.f;
        nvs[g] = pos < key_hi ? __ldg(vsp + (pos >> a.block_shift)) : 1.f;
      }
    };
    int key0 = key_lo + warp * kGroup;
    if (key0 < key_hi) {
      load_k(key0);
      load_v(key0);
      load_scales(key0);
    }
    // ---- Q: rows n8 and n8 + 8, each brought into fp16 range by a power of two
    // (the first codes are on their way)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = n8 + 8 * h;
      uint4 x[DH / 32];
      uint32_t mx = 0;
      // row r = position r / G of the block, head r % G
      const uint16_t* p = a.q + (((size_t)ub * a.S + r / a.G) * a.Hq + ug * a.G + r % a.G) * DH +
                          c4 * (DH / 8);
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        x[i] = r < rows ? *reinterpret_cast<const uint4*>(p + run_at<DH>(i)) : make_uint4(0, 0, 0, 0);
        mx = absmax_bf16x8(mx, x[i]);
      }
      mx = max(mx & 0xFFFFu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = norm_exp(mx);
      const float f = pow2i(-e);
      c_row[h] = a.scale_log2 * pow2i(e);
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        q[2 * i][h] = bf16x2_to_f16x2(x[i].x, f);
        q[2 * i][2 + h] = bf16x2_to_f16x2(x[i].y, f);
        q[2 * i + 1][h] = bf16x2_to_f16x2(x[i].z, f);
        q[2 * i + 1][2 + h] = bf16x2_to_f16x2(x[i].w, f);
      }
    }
    // ---- the block's own keys (at most 16), by one warp while the others start
    if (sa == 0 && warp == kWarps - 1) {
      const int S = a.S;
      uint32_t bk[2][2 * KW], bv[4][2 * VW];  // bf16
      uint32_t mk = 0, mv = 0;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = t * 8 + n8;
        const uint16_t* p = a.k_blk + (((size_t)ub * S + key) * a.Hkv + ug) * DH + c4 * (DH / 8);
#pragma unroll
        for (int i = 0; i < KW / 2; ++i) {
          const uint4 x =
              key < S ? *reinterpret_cast<const uint4*>(p + run_at<DH>(i)) : make_uint4(0, 0, 0, 0);
          mk = absmax_bf16x8(mk, x);
          bk[t][4 * i] = x.x, bk[t][4 * i + 1] = x.y, bk[t][4 * i + 2] = x.z, bk[t][4 * i + 3] = x.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 2 * c4 + (i & 1) + (i >> 1) * 8;
        const uint16_t* p = a.v_blk + (((size_t)ub * S + key) * a.Hkv + ug) * DH + n8 * (DH / 8);
#pragma unroll
        for (int w = 0; w < VW / 2; ++w) {
          const uint4 x = key < S ? reinterpret_cast<const uint4*>(p)[w] : make_uint4(0, 0, 0, 0);
          mv = absmax_bf16x8(mv, x);
          bv[i][4 * w] = x.x, bv[i][4 * w + 1] = x.y, bv[i][4 * w + 2] = x.z, bv[i][4 * w + 3] = x.w;
        }
      }
      const int ek = norm_exp(__reduce_max_sync(0xffffffffu, max(mk & 0xFFFFu, mk >> 16)));
      const int ev = own_value_exp(__reduce_max_sync(0xffffffffu, max(mv & 0xFFFFu, mv >> 16)));
      const float fk = pow2i(-ek), fv = pow2i(-ev);
      w_top = pow2i(ev);
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int j = 0; j < KW; ++j)
          mma16816(s[t], q[j], bf16x2_to_f16x2(bk[t][2 * j], fk),
                   bf16x2_to_f16x2(bk[t][2 * j + 1], fk));
      }
      const float sk[1] = {pow2i(ek)}, lw[1] = {(float)ev}, iw[1] = {pow2i(-ev)};
      finish(s, sk, lw, iw, S, [&](int, int j, uint32_t(&b0)[4], uint32_t(&b1)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // value j + i of each key: half a word
          auto v = [&](int k) {
            const uint32_t w = bv[k][(j + i) >> 1];
            return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16) * fv;
          };
          b0[i] = pack_f16x2(v(0), v(1));
          b1[i] = pack_f16x2(v(2), v(3));
        }
      });
    }
    for (; key0 < key_hi; key0 += kWarps * kGroup) {
      const int next = key0 + kWarps * kGroup;
      float sk[NG], lw[NG], iw[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        w_top = fmaxf(w_top, nvs[g]);  // (1 past the end: harmless)
        const float w = value_scale(nvs[g], w_top);
        sk[g] = nks[g];
        lw[g] = log2f(w);
        iw[g] = 1.f / w;
      }
      float s[2 * NG][4];
#pragma unroll
      for (int t = 0; t < 2 * NG; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
      for (int j = 0; j < KW; ++j)
#pragma unroll
        for (int t = 0; t < 2 * NG; ++t) {
          uint32_t b0, b1;
          codes4<TYPE>(kr[t][j], b0, b1);
          mma16816(s[t], q[j], b0, b1);
        }
      if (next < key_hi) {
        load_k(next);
        load_scales(next);
      }
      finish(s, sk, lw, iw, key_hi - key0, [&](int g, int j, uint32_t(&b0)[4], uint32_t(&b1)[4]) {
        // four codes of a pair of keys, interleaved: (k0, k1) of each column
        const uint32_t w0 = vr[4 * g][j >> 2], w1 = vr[4 * g + 1][j >> 2];
        const uint32_t w8 = vr[4 * g + 2][j >> 2], w9 = vr[4 * g + 3][j >> 2];
        codes4<TYPE>(__byte_perm(w0, w1, 0x5140), b0[0], b0[1]);
        codes4<TYPE>(__byte_perm(w0, w1, 0x7362), b0[2], b0[3]);
        codes4<TYPE>(__byte_perm(w8, w9, 0x5140), b1[0], b1[1]);
        codes4<TYPE>(__byte_perm(w8, w9, 0x7362), b1[2], b1[3]);
      });
      if (next < key_hi) load_v(next);
    }

    // the next unit's first keys to L2, while this one's results are joined
    if (threadIdx.x < 2 && walk.left > 0) {
      const int nL = min(max(walk.len, 0), a.L_cap);
      const int nk = min(min(nL, (walk.left - 1) * kAttnBN), kWarps * kGroup);
      if (nk > 0)
        prefetch_l2_bulk((threadIdx.x ? a.v_ctx : a.k_ctx) +
                             ((size_t)walk.b * a.Hkv + walk.k) * a.L_cap * DH,
                         (uint32_t)nk * DH);
    }
    // ---- the warps' results: o[j] holds columns (2 c4 + {0, 1}) DH/8 + j of
    // rows n8 (first two) and n8 + 8
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (c4 == 0) {
        sm_lse[warp][n8 + 8 * h] = m[h] + log2f(l[h]);  // -inf without keys
        sm_inv[warp][n8 + 8 * h] = 1.f / l[h];
      }
      float* dst = sm_o + (size_t)(warp * 16 + n8 + 8 * h) * LDO + 2 * c4 * (DH / 8);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < NT; j += 4)
          *reinterpret_cast<float4*>(dst + e * (DH / 8) + j) =
              make_float4(o[j][2 * h + e], o[j + 1][2 * h + e], o[j + 2][2 * h + e],
                          o[j + 3][2 * h + e]);
    }
    __syncthreads();
    const size_t slot = pair + blockIdx.x;
    const bool ends = sb == 1 + (L + kAttnBN - 1) / kAttnBN, whole = sa == 0 && ends;
    if (threadIdx.x == 0) put_span(a.unit_span, pair, blockIdx.x, sa == 0, ends);
    for (int i = threadIdx.x; i < rows * (DH / 4); i += kThreads) {
      const int r = i / (DH / 4), col = (i - r * (DH / 4)) * 4;
      float mr = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mr = fmaxf(mr, sm_lse[w][r]);
      float den = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (sm_lse[w][r] == -INFINITY) continue;  // this warp had no keys
        const float f0 = ex2(sm_lse[w][r] - mr), f = f0 * sm_inv[w][r];
        const float4 x = *reinterpret_cast<const float4*>(sm_o + (size_t)(w * 16 + r) * LDO + col);
        den += f0;
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
      }
      const float inv = 1.f / den;
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (whole) {
        uint16_t* dst = a.out + (((size_t)ub * a.S + r / a.G) * a.Hq + ug * a.G + r % a.G) * DH + col;
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
      } else {
        reinterpret_cast<float4*>(a.part_o)[(slot * 16 + r) * (DH / 4) + col / 4] = acc;
        if (col == 0) a.part_lse[slot * 16 + r] = mr + log2f(den);
      }
    }
    __syncthreads();  // before the next segment's results
  }
}

// CTA = unit, thread = (row, 4 columns): joins the partial records of a unit that
// several CTAs hold, the loads of four records in flight together.
__global__ void __launch_bounds__(512) attn_q8_rows_merge_kernel(const AttnQ8Args a) {
  griddep_launch();
  griddep_wait();
  const int u = blockIdx.x;
  const int2 uc = a.unit_span[u];
  if (uc.x == uc.y) return;  // written by its CTA
  const int b = u / a.Hkv, g = u - b * a.Hkv, dv_log = a.dh == 64 ? 4 : 5;
  const int r = threadIdx.x >> dv_log, v = threadIdx.x & ((1 << dv_log) - 1);
  if (r >= a.rows_per_half) return;
  float mr = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = uc.x; c0 <= uc.y; c0 += 4) {
    float lse[4];
    float4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const size_t rec = ((size_t)u + min(c0 + k, uc.y)) * 16 + r;
      lse[k] = __ldcg(a.part_lse + rec);
      x[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (rec << dv_log) + v);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // past the last record, or one without keys (its output was never written)
      if (c0 + k > uc.y || lse[k] == -INFINITY) continue;
      const float mn = lse[k] > mr ? lse[k] : mr;
      const float f0 = ex2(mr - mn), f1 = ex2(lse[k] - mn);
      mr = mn;
      den = fmaf(den, f0, f1);
      acc.x = fmaf(acc.x, f0, x[k].x * f1);
      acc.y = fmaf(acc.y, f0, x[k].y * f1);
      acc.z = fmaf(acc.z, f0, x[k].z * f1);
      acc.w = fmaf(acc.w, f0, x[k].w * f1);
    }
  }
  const float inv = 1.f / den;
  uint16_t* dst = a.out + (((size_t)b * a.S + r / a.G) * a.Hq + g * a.G + r % a.G) * a.dh + v * 4;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                                              pack_bf16x2(acc.z * inv, acc.w * inv));
}

template <int TYPE, int DH>
cudaError_t launch_rows(const AttnQ8Args& a, cudaStream_t st) {
  constexpr size_t smem = (size_t)kWarps * 16 * (DH + 4) * sizeof(float);
  const cudaError_t e = allow_smem<attn_q8_rows_kernel<TYPE, DH>>(smem);
  if (e != cudaSuccess) return e;
  return launch_k(attn_q8_rows_kernel<TYPE, DH>, dim3(a.n_ctas), dim3(kThreads), smem, st, a);
}

}  // namespace

cudaError_t launch_attn_q8_rows(const AttnQ8Args& a, int type, cudaStream_t st) {
  if (type == TT_Q8_INT8)
    return a.dh == 64 ? launch_rows<TT_Q8_INT8, 64>(a, st) : launch_rows<TT_Q8_INT8, 128>(a, st);
  return a.dh == 64 ? launch_rows<TT_Q8_E4M3, 64>(a, st) : launch_rows<TT_Q8_E4M3, 128>(a, st);
}
cudaError_t launch_attn_q8_rows_merge(const AttnQ8Args& a, cudaStream_t st) {
  return launch_k(attn_q8_rows_merge_kernel, dim3((unsigned)a.units), dim3(4 * a.dh), 0, st, a);
}

}  // namespace tt
