// Block-denoise attention over an 8-bit context cache.
//
// Per query row, with s_j = q . k_j / sqrt(dh) (log2 units), v scale w_j and
// codes c_j:  out = sum_j 2^(s_j) w_j c_j / sum_j 2^(s_j).
// One pass: p_j = 2^(s_j + log2 w_j - m) with m a running maximum of s_j +
// log2 w_j less kPeak, O = sum p_j c_j, l = sum p_j / w_j, out = O / l.  The key
// scale multiplies a score and the value scale adds log2 w_j to its exponent, both
// per group of 16 keys, so neither costs an instruction per element; p_j <= 2^15
// and the row's largest at least 2^10, whatever the scales, which lets P be fp16:
// its rounding is an eighth of the output's for keys down to 2^-24 of the largest
// product, absolute below (2^-35 of it) (tt_attn_q8.cuh has the constants).
//
// Both products run on the tensor cores in fp16 (kind::f16): every int8 and
// e4m3 code is an fp16 number; a query row and the block's own bf16 keys and
// values are brought into fp16 range by a power of two per row (per tile),
// which is exact down to 2^-28 of the largest magnitude.
//
// Inside a CTA (tt_attn_q8.cuh has the schedule) two chains run side by side,
// each with 128 query rows and dh TMEM columns of O:
//   S = Q . K(tile)^T -> softmax -> O += P . V(tile) -> next S ...
// With more than 128 rows per KV head the chains take the two halves of the
// rows and every tile; otherwise they share the rows and take every other
// tile.  The softmax (thread = row) moves the 128 scores of its row to
// registers at once, so ONE S buffer serves both chains by turns, the other
// 128 columns hold a P of its own for each chain, and the next S does not
// wait for this tile's softmax and P . V: with S and P in the same columns
// (two S buffers) every tile paid S, softmax and P . V one after the other,
// 4,900 cycles for the two chains where this order takes 3,500 to 3,900.
// The block's own keys are a unit's last tile: their conversion from bf16 (two
// passes, 13,000 cycles when nothing hides them) then runs under the softmax of
// the tiles before (48 sequences of up to 32768 keys: 221 us; as first tile 20 more).
// What bounds it: a tile of both chains is 2,050 cycles of tensor work and as many
// of exponentials, but the hand-overs between the roles (S twice per tile through
// one buffer, P to its product, the codes' reload and conversion) are loops of about
// 3,200 cycles each: without exponentials, conversion and all but one MMA of eight,
// the time falls by a quarter only.  4 sequences of 65536 int8 keys, S = 16, 2 KV heads of 16
// queries and dh 128, with the merge: 80 us, 860 TFLOP/s and 1.7 TB/s of cache.
// Few tiles per CTA pay the start instead: 8 x 4096 keys, 32 us.
// Roles (16 warps; registers are moved to the softmax by setmaxnreg):
//   warps 0-3 / 4-7   softmax of chain 0 / 1;
//   warps 8-11        codes of one tile in shared memory to fp16 in the swizzled
//                     K and V rings;
//   warps 12, 13      issue of S and of P . V for both chains (12 owns TMEM);
//   warp 14           codes from global to shared memory;
//   warp 15           the tiles' scales.
#include <math.h>

#include "tt_attn_q8.cuh"

namespace tt {

namespace {

constexpr int kThreads = 512;
constexpr int kConv = 128;                  // converter threads
constexpr int kSlots = 2;                   // depth of the K and of the V ring
constexpr uint32_t kSub = kAttnBN * 128;    // 128 rows x 64 fp16: 16 KB

struct Smem {
  uint32_t q, k, v, raw, scales, bars, total;
};
__host__ __device__ constexpr Smem smem_layout(int dh) {
  Smem s{};
  const uint32_t nsub = (uint32_t)dh / 64;
  s.q = 0;
  s.k = s.q + 2 * nsub * kSub;
  s.v = s.k + kSlots * nsub * kSub;
  s.raw = s.v + kSlots * nsub * kSub;    // codes of one K and one V tile
  s.scales = s.raw + 2 * kAttnBN * dh;  // [slot][key scale, log2 w, 1 / w][8 groups]
  s.bars = (s.scales + kSlots * 24 * 4 + 63) / 64 * 64;
  s.total = s.bars + 320;
  return s;
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// Valid keys of local tile t: 128 context keys each, then the block's own S keys.
__device__ __forceinline__ bool is_context(int t, int L) { return t * kAttnBN < L; }
__device__ __forceinline__ int tile_keys(int t, int L, int S) {
  return is_context(t, L) ? min(kAttnBN, L - t * kAttnBN) : S;
}

// Pairs of fp32 in one 64-bit register: one instruction for two.
__device__ __forceinline__ uint64_t pack2u(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  return pack2u(__float_as_uint(x), __float_as_uint(y));
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// TMEM, 8 columns of the thread's lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
               "r"(r[7])
               : "memory");
}

// `bytes` (a multiple of 16) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Row `r` of a 128-byte-swizzled fp16 tile of dh columns: address of 16-byte
// chunk c (8 values).
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)(c >> 3) * kSub + (uint32_t)r * 128 + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Scales of 16 keys (group g) of a tile: key scale, log2 and inverse of the
// value scale.
__device__ __forceinline__ void put_scales(float* sc, int g, float kf, float lw, float iw,
                                           uint64_t* full) {
  sc[g] = kf;
  sc[8 + g] = lw;
  sc[16 + g] = iw;
  mbar_arrive(full);
}
__device__ __forceinline__ void lds4f(uint32_t addr, float (&v)[4]) {
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(addr));
}

// 16 of a row's scores to probabilities, as fp16 pairs, and their part of the
// row sum.  kf: the row's score factor, lw: log2 of the value scale, iw: its inverse.
__device__ __forceinline__ void exps16(const uint32_t* s, float kf, float lw, float iw, float m,
                                       float& l, uint32_t (&p)[8]) {
  const float off = lw - m;
  const uint64_t c2 = pack2(kf, kf), o2 = pack2(off, off);
  uint64_t sum = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float x0, x1;
    unpack2(fma2(pack2u(s[2 * j], s[2 * j + 1]), c2, o2), x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    sum = add2(sum, pack2(p0, p1));
    p[j] = pack_f16x2(p0, p1);
  }
  float e0, e1;
  unpack2(sum, e0, e1);
  l = fmaf(e0 + e1, iw, l);
}

template <int TYPE, int DH>
__global__ void __launch_bounds__(kThreads, 1) attn_q8_kernel(const AttnQ8Args a) {
  griddep_launch();
  griddep_wait();
  extern __shared__ uint8_t smem_raw[];
  __shared__ PlanSmem plan;
  TileWalk walk = plan_walk<kThreads>(a, plan);
  const int U = a.Hkv * a.n_qtiles;
  if (walk.left == 0) {
    if (walk.off > 0) {  // an empty range inside a unit: an empty record
      const size_t slot = (size_t)walk.b * U + walk.k + blockIdx.x;
      for (int i = threadIdx.x; i < 256; i += kThreads)
        a.part_lse[slot * 256 + i] = -INFINITY;
    }
    return;
  }
  constexpr int NSUB = DH / 64;
  constexpr Smem SL = smem_layout(DH);
  uint8_t* base = align1024(smem_raw);
  float* scales = reinterpret_cast<float*>(base + SL.scales);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + SL.bars);
  uint64_t* q_full = bars;               // [chain] query rows written
  uint64_t* s_full = q_full + 2;         // [chain] S holds the chain's scores
  uint64_t* s_free = s_full + 2;         // S is in registers
  uint64_t* p_full = s_free + 1;         // [chain] P written, O corrected
  uint64_t* pv_done = p_full + 2;        // [chain] P . V done
  uint64_t* full = pv_done + 2;          // [K, V][slot]
  uint64_t* empty = full + 2 * kSlots;   // [K, V][slot]
  uint64_t* sc_full = empty + 2 * kSlots;  // [slot]
  uint64_t* rk_full = sc_full + kSlots;  // [K, V] a tile of codes has landed
  uint64_t* rk_empty = rk_full + 2;      // [K, V] it has been converted
  uint64_t* own_full = rk_empty + 2;     // [slot] the own keys' and values' exponents
  int2* own_exp = reinterpret_cast<int2*>(own_full + kSlots);  // [slot]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(own_exp + kSlots);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  uint32_t* red = tmem_slot + 2;  // [8] converter reduction

  // (the shuffle tells the compiler that the index is the same in all lanes)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const bool split = a.halves == 1;  // the chains share the rows and split the tiles
  if (threadIdx.x == 0) {
    mbar_init(s_free, 128);
    for (int c = 0; c < 2; ++c) {
      mbar_init(&q_full[c], 128);
      mbar_init(&s_full[c], 1);
      mbar_init(&p_full[c], 128);
      mbar_init(&pv_done[c], 1);
      mbar_init(&rk_full[c], 1);
      mbar_init(&rk_empty[c], kConv);
    }
    for (int s = 0; s < kSlots; ++s) {
      for (int kv = 0; kv < 2; ++kv) {
        mbar_init(&full[2 * kv + s], kConv);
        mbar_init(&empty[2 * kv + s], 1);
      }
      mbar_init(&sc_full[s], 8);
      mbar_init(&own_full[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int ub, uk, sa, sb, L;  // current segment: sequence, unit in it, local tiles [sa, sb), length

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    reg_inc<192>();
    const int ch = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off, tP = tmem + kAttnBN + ch * 64 + lane_off;
    const uint32_t tO = tmem + 2 * kAttnBN + ch * DH + lane_off;
    const uint32_t sQ = smem_u32(base + SL.q) + ch * NSUB * kSub;
    const bool valid = r < a.rows_per_half;
    const bool busy = (warp & 3) * 32 < a.rows_per_half;  // the warp has a row
    int kt = 0, pt = 0;                                   // tiles of the CTA, turns
    bool ok = true;
    if (!busy) {
      // no rows in this warp: its part of the barriers alone
      while (ok && walk.next(ub, uk, sa, sb, L)) {
        const int step = split ? 2 : 1, first = sa + (split ? ch : 0);
        if (first >= sb) continue;
        mbar_arrive(&q_full[ch]);
        for (int i = first; i < sb; i += step, ++pt) {
          ok = mbar_wait_inline(&s_full[ch], (uint32_t)pt & 1u, a.err, abort_flag,
                                WHERE_ATTN_SOFTMAX);
          if (!ok) break;
          mbar_arrive(s_free);
          mbar_arrive(&p_full[ch]);
          ok = mbar_wait_inline(&pv_done[ch], (uint32_t)pt & 1u, a.err, abort_flag,
                                WHERE_ATTN_SOFTMAX);
          if (!ok) break;
        }
      }
    }
    for (; busy && ok && walk.next(ub, uk, sa, sb, L); kt += sb - sa) {
      const int ug = uk / a.n_qtiles, qt = uk - ug * a.n_qtiles;
      const size_t slot = (size_t)ub * U + uk + blockIdx.x;
      const int step = split ? 2 : 1, first = sa + (split ? ch : 0);
      float m = -INFINITY, l = 0.f;
      // block positions (times heads) of the chain's rows
      const size_t pos0 =
          (size_t)ub * a.S + qt * a.halves * a.s_per_half + (split ? 0 : ch * a.s_per_half);
      const size_t qrow = (pos0 + (r >> a.g_shift)) * a.Hq + ug * a.G + (r & (a.G - 1));
      if (first < sb) {
        // The warp's 32 query rows, each by a power of two in fp16 range: a row
        // to DH / 8 lanes, so that loads are whole lines (a row to a thread
        // took 8,000 cycles), eight in flight: all sixteen of dh 128 at once
        // unroll to more instructions than they save (+7 % on long caches).  The
        // previous segment's last S of this chain has been waited for below.
        float c_row = 0.f;
        {
          constexpr int LPR = DH / 8, RPL = 32 / LPR;  // lanes per row, rows per load
          const int rl = lane / LPR, cl = lane % LPR;
          const int r0 = (warp & 3) * 32;
#pragma unroll 1
          for (int i0 = 0; i0 < LPR; i0 += 8) {
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = r0 + (i0 + i) * RPL + rl;
              x[i] = make_uint4(0, 0, 0, 0);
              if (rr < a.rows_per_half)
                x[i] = *reinterpret_cast<const uint4*>(
                    a.q + ((size_t)(pos0 + (rr >> a.g_shift)) * a.Hq + ug * a.G + (rr & (a.G - 1))) * DH +
                    cl * 8);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = r0 + (i0 + i) * RPL + rl;
              uint32_t mx = absmax_bf16x8(0, x[i]);
              mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
              for (int o = LPR / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              const int e = norm_exp(mx);
              const float f = pow2i(-e);
              sts128(sQ + chunk_at(rr, cl), bf16x2_to_f16x2(x[i].x, f), bf16x2_to_f16x2(x[i].y, f),
                     bf16x2_to_f16x2(x[i].z, f), bf16x2_to_f16x2(x[i].w, f));
              const int mine = __shfl_sync(0xffffffffu, e, (lane % RPL) * LPR);
              if (lane / RPL == i0 + i) c_row = a.scale_log2 * pow2i(mine);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&q_full[ch]);

        for (int i = first; i < sb; i += step, ++pt) {
          const int t = kt + i - sa, ts = split ? ch : t & 1;
          if (!mbar_wait_inline(&sc_full[ts], (uint32_t)(split ? pt : t >> 1) & 1u, a.err,
                                abort_flag, WHERE_ATTN_SOFTMAX)) {
            ok = false;
            break;
          }
          const uint32_t sc = smem_u32(scales + ts * 24);
          float kf[8], lw[8], iw[8];
          lds4f(sc, *reinterpret_cast<float(*)[4]>(&kf[0]));
          lds4f(sc + 16, *reinterpret_cast<float(*)[4]>(&kf[4]));
          lds4f(sc + 32, *reinterpret_cast<float(*)[4]>(&lw[0]));
          lds4f(sc + 48, *reinterpret_cast<float(*)[4]>(&lw[4]));
          lds4f(sc + 64, *reinterpret_cast<float(*)[4]>(&iw[0]));
          lds4f(sc + 80, *reinterpret_cast<float(*)[4]>(&iw[4]));
#pragma unroll
          for (int g = 0; g < 8; ++g) kf[g] = score_factor(c_row, kf[g]);
          if (!mbar_wait_inline(&s_full[ch], (uint32_t)pt & 1u, a.err, abort_flag,
                                WHERE_ATTN_SOFTMAX)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t s[128];
          tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
          tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
          tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
          tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(s_free);
          float alpha = 1.f;
          bool need = false;
          uint32_t p0[8], p1[8];
          const int nv = tile_keys(i, L, a.S);
          if (nv < kAttnBN) {
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (j >= nv) s[j] = __float_as_uint(-INFINITY);
          }
          float mx = -INFINITY;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            {
              const uint32_t* x = s + 16 * g;
              float y0 = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
              float y1 = fmaxf(__uint_as_float(x[2]), __uint_as_float(x[3]));
#pragma unroll
              for (int j = 4; j < 16; j += 4) {
                y0 = fmax3(y0, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                y1 = fmax3(y1, __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
              }
              mx = fmaxf(mx, fmaf(fmaxf(y0, y1), kf[g], lw[g]));
            }
          }
          need = mx > m + kTop;
          if (need) {
            const float half = ex2(0.5f * (m - (mx - kPeak)));
            alpha = half * half;
            l = l * half * half;
            m = mx - kPeak;
          }
          exps16(s, kf[0], lw[0], iw[0], m, l, p0);
          exps16(s + 16, kf[1], lw[1], iw[1], m, l, p1);
          // P and O are the tensor core's until P . V of the turn before has run
          if (i > first && !mbar_wait_inline(&pv_done[ch], (uint32_t)(pt - 1) & 1u, a.err,
                                             abort_flag, WHERE_ATTN_SOFTMAX)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // O to the new maximum before P . V adds to it; a segment's first
          // P . V overwrites O
          if (i > first && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
            for (int c0 = 0; c0 < DH; c0 += 8) {
              uint32_t o[8];
              tmem_ld8(tO + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st8(tO + c0, o);
            }
          }
          tmem_st8(tP, p0);
          tmem_st8(tP + 8, p1);
          exps16(s + 32, kf[2], lw[2], iw[2], m, l, p0);
          tmem_st8(tP + 16, p0);
          exps16(s + 48, kf[3], lw[3], iw[3], m, l, p1);
          tmem_st8(tP + 24, p1);
          exps16(s + 64, kf[4], lw[4], iw[4], m, l, p0);
          tmem_st8(tP + 32, p0);
          exps16(s + 80, kf[5], lw[5], iw[5], m, l, p1);
          tmem_st8(tP + 40, p1);
          exps16(s + 96, kf[6], lw[6], iw[6], m, l, p0);
          tmem_st8(tP + 48, p0);
          exps16(s + 112, kf[7], lw[7], iw[7], m, l, p1);
          tmem_st8(tP + 56, p1);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&p_full[ch]);
        }
        if (!ok) break;
        if (!mbar_wait_inline(&pv_done[ch], (uint32_t)(pt - 1) & 1u, a.err, abort_flag,
                              WHERE_ATTN_SOFTMAX)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      // A unit that this CTA holds alone, in rows of its own, is done; other
      // segments leave a record: their output (tile-major [dh/4][256 rows][4],
      // a warp's store is 512 contiguous bytes) and log2 of their sum.
      const int r256 = ch * 128 + r;
      const bool ends = sb == 1 + (L + kAttnBN - 1) / kAttnBN;
      const bool whole = !split && sa == 0 && ends;
      if (first < sb) {
        float* po = a.part_o + slot * DH * 256 + (size_t)r256 * 4;
        const float inv = 1.f / l;
#pragma unroll 1
        for (int c0 = 0; c0 < DH; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c0, o);
          tmem_wait_ld();
          if (valid && whole) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[j] = pack_bf16x2(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
#pragma unroll
            for (int v = 0; v < 4; ++v)
              *reinterpret_cast<uint4*>(a.out + qrow * DH + c0 + 8 * v) =
                  make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
          } else if (valid) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              *reinterpret_cast<float4*>(po + (size_t)(c0 / 4 + v) * 1024) =
                  make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                              __uint_as_float(o[4 * v + 2]) * inv,
                              __uint_as_float(o[4 * v + 3]) * inv);
          }
        }
      }
      if (valid && !whole) a.part_lse[slot * 256 + r256] = m + log2f(l);
    }
  } else if (warp < 12) {
    // ---------------------------------------------- codes to fp16 tiles
    reg_dec<64>();
    const int tid = threadIdx.x - 256;
    constexpr int NV = kAttnBN * DH / 16 / kConv;  // 16-code chunks per thread
    // The thread's chunks: column `col` of rows row0, row0 + kConv * 16 / DH,
    // ...  Eight lanes that access shared memory together read 128 different
    // bytes of the codes (128-byte rows: columns 0-3 of an even row with 4-7
    // of the odd one beside it) and, by the swizzle, write eight different
    // 16-byte bank groups (even ones for an even row, odd ones for an odd).
    const int half = (tid >> 2) & 1;
    const int row0 = DH == 64 ? tid >> 2 : ((tid >> 4) << 1) + half;
    const int col = DH == 64 ? tid & 3 : (tid & 3) + 4 * (half ^ ((tid >> 3) & 1));
    const uint32_t sK = smem_u32(base + SL.k), rK = smem_u32(base + SL.raw);  // V behind K
    auto convert = [&](uint32_t src, uint32_t dst, int nv) {
      // rows 32 (dh 64) or 16 apart: the swizzle (row & 7) is the same for all
      const uint32_t d0 = dst + chunk_at(row0, 2 * col), d1 = dst + chunk_at(row0, 2 * col + 1);
      const uint32_t s0 = src + row0 * DH + col * 16;
#pragma unroll 1
      for (int i0 = 0; i0 < NV; i0 += 4) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lds128(s0 + (i0 + i) * (kConv * 16));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = row0 + (i0 + i) * (kConv * 16 / DH);
          uint4 x = v[i];
          if (row >= nv) x = make_uint4(0, 0, 0, 0);  // behind the context: zeros
          uint32_t w[8];
          codes4<TYPE>(x.x, w[0], w[1]);
          codes4<TYPE>(x.y, w[2], w[3]);
          codes4<TYPE>(x.z, w[4], w[5]);
          codes4<TYPE>(x.w, w[6], w[7]);
          const uint32_t at = (uint32_t)(i0 + i) * (kConv * 16 / DH) * 128;
          sts128(d0 + at, w[0], w[1], w[2], w[3]);
          sts128(d1 + at, w[4], w[5], w[6], w[7]);
        }
      }
    };
    // The block's own keys or values (kv) [S, Hkv, dh] (bf16) by a power of two
    // in fp16 range; the exponents go to warp 15.  Rows past S are zero.
    int ek = 0;
    auto block_rows = [&](const uint16_t* p, uint32_t dst, int kv, int slot) {
      constexpr int NB = kAttnBN * DH / 8 / kConv;
      uint32_t mx = 0;
      const int c0 = tid % (DH / 8), r0 = tid / (DH / 8);
#pragma unroll 4
      for (int i = 0; i < NB; ++i) {
        const int row = r0 + i * (kConv / (DH / 8));
        if (row < a.S) {
          const uint4 x = *reinterpret_cast<const uint4*>(p + (size_t)row * a.Hkv * DH + c0 * 8);
          mx = absmax_bf16x8(mx, x);
        }
      }
      mx = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
      named_bar_sync(1, kConv);  // the previous use of red is over
      if (lane == 0) red[(warp - 8) + 4 * kv] = mx;
      named_bar_sync(1, kConv);
      const uint32_t* rd = red + 4 * kv;
      const uint32_t top = max(max(rd[0], rd[1]), max(rd[2], rd[3]));
      const int e = kv ? own_value_exp(top) : norm_exp(top);
      if (tid == 0 && kv) {
        own_exp[slot] = make_int2(ek, e);
        mbar_arrive(&own_full[slot]);
      }
      ek = e;
      const float f = pow2i(-e);
#pragma unroll 4
      for (int i = 0; i < NB; ++i) {
        const int row = r0 + i * (kConv / (DH / 8));
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row < a.S)
          x = *reinterpret_cast<const uint4*>(p + (size_t)row * a.Hkv * DH + c0 * 8);
        sts128(dst + chunk_at(row, c0), bf16x2_to_f16x2(x.x, f), bf16x2_to_f16x2(x.y, f),
               bf16x2_to_f16x2(x.z, f), bf16x2_to_f16x2(x.w, f));
      }
    };
    int kt = 0, used0 = 0, used1 = 0;  // tiles, uses of each slot
    int raw = 0;                       // context tiles so far
    bool ok = true;
    while (ok && walk.next(ub, uk, sa, sb, L)) {
      const int ug = uk / a.n_qtiles;
      for (int tl = sa; tl < sb; ++tl, ++kt) {
        // the ring: slots by turns, or one slot per chain (each barrier then
        // has one reader that sees its phases in order)
        const int slot = split ? (tl - sa) & 1 : kt & 1;
        const uint32_t par = ((uint32_t)(slot ? used1++ : used0++) & 1u) ^ 1u;
        const int nv = tile_keys(tl, L, a.S);
        const bool ctx = is_context(tl, L);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {  // K, then V
          if ((ctx && !mbar_wait_inline(&rk_full[kv], (uint32_t)raw & 1u, a.err, abort_flag,
                                           WHERE_ATTN_PRODUCER)) ||
              !mbar_wait_inline(&empty[2 * kv + slot], par, a.err, abort_flag,
                                WHERE_ATTN_PRODUCER)) {
            ok = false;
            break;
          }
          const uint32_t dst = sK + (kv * kSlots + slot) * NSUB * kSub;
          if (!ctx) {
            block_rows((kv ? a.v_blk : a.k_blk) + ((size_t)ub * a.S * a.Hkv + ug) * DH, dst, kv,
                       slot);
          } else {
            convert(rK + kv * kAttnBN * DH, dst, nv);
            mbar_arrive(&rk_empty[kv]);
            raw += kv;
          }
          fence_proxy_async_smem();
          mbar_arrive(&full[2 * kv + slot]);
        }
        if (!ok) break;
      }
    }
  } else {
    reg_dec<64>();
    if (warp == 14) {
      // ----------------------------------------- codes to shared memory
      // One K and one V tile of codes (contiguous in memory) ahead of the
      // converters.  (Tiles further ahead brought into L2 cost more, in the
      // first tiles, than they saved.)
      // The spans by a lane that waits for nothing: a wait that gives up must not
      // leave the merge with spans of another call.  (By a warp that issues products,
      // or by the softmax warps segment by segment: 81 to 82.5 us for 4 sequences of
      // 65536 keys against 80.5.)
      if (lane == 1) put_spans(a.unit_span, walk, blockIdx.x);
      if (lane == 0) {
        const uint32_t rK = smem_u32(base + SL.raw), rV = rK + kAttnBN * DH;
        int raw = 0;
        bool ok = true;
        while (ok && walk.next(ub, uk, sa, sb, L)) {
          const size_t pair = (size_t)ub * a.Hkv + uk / a.n_qtiles;
          const uint8_t* kp = a.k_ctx + pair * a.L_cap * DH;
          const uint8_t* vp = a.v_ctx + pair * a.L_cap * DH;
          for (int tl = sa; tl < sb; ++tl) {
            if (!is_context(tl, L)) break;  // the unit's last tile
            const size_t at = (size_t)tl * kAttnBN * DH;
            const uint32_t n = (uint32_t)tile_keys(tl, L, a.S) * DH;
            const uint32_t par = ((uint32_t)raw & 1u) ^ 1u;
            ok = mbar_wait_inline(&rk_empty[0], par, a.err, abort_flag, WHERE_ATTN_PRODUCER);
            if (!ok) break;
            mbar_arrive_expect_tx(&rk_full[0], n);
            bulk_load(rK, kp + at, n, &rk_full[0]);
            ok = mbar_wait_inline(&rk_empty[1], par, a.err, abort_flag, WHERE_ATTN_PRODUCER);
            if (!ok) break;
            mbar_arrive_expect_tx(&rk_full[1], n);
            bulk_load(rV, vp + at, n, &rk_full[1]);
            ++raw;
          }
        }
      }
    } else if (warp == 15) {
      // -------------------------------------------- scales of the tiles
      // Lane g < 8: 16 keys.  A tile's scales go with its V slot: once P . V of
      // the tile that had the slot before has run, its softmax is done.  A value
      // scale is held at 2^-100 of the segment's largest so far (tt_attn_q8.cuh).
      int kt = 0, used0 = 0, used1 = 0, own0 = 0, own1 = 0;
      bool ok = true;
      while (ok && walk.next(ub, uk, sa, sb, L)) {
        const size_t pair = (size_t)ub * a.Hkv + uk / a.n_qtiles;
        const float* ksp = a.k_scale + pair * a.n_blocks;
        const float* vsp = a.v_scale + pair * a.n_blocks;
        float nk = 1.f, nw = 1.f, top = 0.f;  // a tile ahead
        bool in = false;
        auto load = [&](int tl) {
          const int pos = tl * kAttnBN + lane * 16;
          in = lane < 8 && tl < sb && pos < L;
          nk = in ? __ldg(ksp + (pos >> a.block_shift)) : 1.f;
          nw = in ? __ldg(vsp + (pos >> a.block_shift)) : 1.f;
        };
        load(sa);
        for (int tl = sa; tl < sb; ++tl, ++kt) {
          const int slot = split ? (tl - sa) & 1 : kt & 1;
          const uint32_t par = ((uint32_t)(slot ? used1++ : used0++) & 1u) ^ 1u;
          float w = in ? nw : 0.f;
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
          top = fmaxf(top, w);
          float kf = nk, lw = log2f(value_scale(nw, top)), iw = 1.f / value_scale(nw, top);
          load(tl + 1);
          ok = mbar_wait_inline(&empty[2 + slot], par, a.err, abort_flag, WHERE_ATTN_PRODUCER);
          if (!ok) break;
          if (!is_context(tl, L)) {
            ok = mbar_wait_inline(&own_full[slot], (uint32_t)(slot ? own1++ : own0++) & 1u, a.err,
                                  abort_flag, WHERE_ATTN_PRODUCER);
            if (!ok) break;
            const int2 e = own_exp[slot];
            w = value_scale(pow2i(e.y), top);
            kf = pow2i(e.x);
            lw = log2f(w);
            iw = 1.f / w;
          }
          if (lane < 8) put_scales(scales + slot * 24, lane, kf, lw, iw, &sc_full[slot]);
          __syncwarp();
        }
      }
    } else if (warp == 12) {
      // -------------------------------------------- S = Q . K^T, both chains
      constexpr uint32_t idS = idesc_f16(128, kAttnBN, false);
      const uint64_t dQ0 = sdesc_sw128(smem_u32(base + SL.q), 16, 1024);
      const uint64_t dK0 = sdesc_sw128(smem_u32(base + SL.k), 16, 1024);
      int kt = 0, n = 0, used0 = 0, used1 = 0;  // tiles, products, uses of each slot
      int qs0 = 0, qs1 = 0;                     // segments of each chain
      bool ok = true;
      while (ok && walk.next(ub, uk, sa, sb, L)) {
        for (int i = sa; ok && i < sb; ++i, ++kt) {
          const int slot = split ? (i - sa) & 1 : kt & 1;
          const uint32_t par = (uint32_t)(slot ? used1++ : used0++) & 1u;
          if (!mbar_wait_inline(&full[slot], par, a.err, abort_flag, WHERE_ATTN_MMA)) {
            ok = false;
            break;
          }
          for (int c = split ? slot : 0; c < (split ? slot + 1 : 2); ++c, ++n) {
            if (i == (split ? sa + c : sa) &&
                !mbar_wait_inline(&q_full[c], (uint32_t)(c ? qs1++ : qs0++) & 1u, a.err,
                                  abort_flag, WHERE_ATTN_MMA)) {
              ok = false;
              break;
            }
            if (n > 0 && !mbar_wait_inline(s_free, (uint32_t)(n - 1) & 1u, a.err, abort_flag,
                                           WHERE_ATTN_MMA)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              const uint64_t dQ = dQ0 + (uint64_t)((uint32_t)(c * NSUB) * (kSub >> 4));
              const uint64_t dK = dK0 + (uint64_t)((uint32_t)(slot * NSUB) * (kSub >> 4));
#pragma unroll
              for (int k = 0; k < DH / 16; ++k) {
                const uint64_t off = (uint64_t)(((k >> 2) * kSub + (k & 3) * 32) >> 4);
                umma_bf16_ss(tmem, dQ + off, dK + off, idS, k > 0);
              }
              umma_commit(&s_full[c]);
              if (split || c == 1) umma_commit(&empty[slot]);
            }
            __syncwarp();
          }
        }
      }
    } else if (warp == 13) {
      // ---------------------------------------------- O += P . V, both chains
      constexpr uint32_t idO = idesc_f16(128, DH, true);
      const uint64_t dV0 = sdesc_sw128(smem_u32(base + SL.v), kSub, 1024);
      int kt = 0, used0 = 0, used1 = 0, pt0 = 0, pt1 = 0;
      bool ok = true;
      while (ok && walk.next(ub, uk, sa, sb, L)) {
        for (int i = sa; ok && i < sb; ++i, ++kt) {
          const int slot = split ? (i - sa) & 1 : kt & 1;
          const uint32_t par = (uint32_t)(slot ? used1++ : used0++) & 1u;
          const int ksteps = (tile_keys(i, L, a.S) + 15) >> 4;
          if (!mbar_wait_inline(&full[2 + slot], par, a.err, abort_flag, WHERE_ATTN_MMA)) {
            ok = false;
            break;
          }
          for (int c = split ? slot : 0; c < (split ? slot + 1 : 2); ++c) {
            if (!mbar_wait_inline(&p_full[c], (uint32_t)(c ? pt1++ : pt0++) & 1u, a.err,
                                  abort_flag, WHERE_ATTN_MMA)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              const uint32_t tP = tmem + kAttnBN + c * 64, tO = tmem + 2 * kAttnBN + c * DH;
              const uint32_t more = i > (split ? sa + c : sa) ? 1u : 0u;
              const uint64_t dV = dV0 + (uint64_t)((uint32_t)(slot * NSUB) * (kSub >> 4));
#pragma unroll
              for (int k = 0; k < kAttnBN / 16; ++k)
                if (k < ksteps)
                  umma_bf16_ts(tO, tP + k * 8, dV + (uint64_t)(k * (2048 >> 4)), idO,
                               k > 0 ? 1u : more);
              umma_commit(&pv_done[c]);
              if (split || c == 1) umma_commit(&empty[2 + slot]);
            }
            __syncwarp();
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The records of a unit that several CTAs hold (two per segment where the chains
// split the tiles) into the bf16 output: sum_c 2^(lse_c) o_c / sum_c 2^(lse_c).
// Block = (unit, 32 query rows, 1 / parts of the columns), lane = row, NG groups
// of 4 columns to a warp, whose loads are 512 contiguous bytes.  One pass with a
// running maximum; the loads of KB records are in flight together, for latency
// is all there is.
template <int NG, int KB>
__global__ void __launch_bounds__(256) attn_q8_merge_kernel(const AttnQ8Args a) {
  griddep_launch();
  griddep_wait();
  const int row_blocks = a.halves * 4, ngrp = a.dh / 4, parts = ngrp / (8 * NG);
  const int part = blockIdx.x % parts, rb = blockIdx.x / parts % row_blocks;
  const int u = blockIdx.x / (parts * row_blocks);
  const int2 uc = a.unit_span[u];
  const int per = a.halves == 1 ? 2 : 1;  // records per segment
  if (!span_in_range(uc, a.n_ctas)) return;
  if (per == 1 && uc.x == uc.y) return;   // written by its CTA
  const int lane = threadIdx.x & 31, row = rb * 32 + lane, h = row >> 7, r = row & 127;
  if (rb * 32 - h * 128 >= a.rows_per_half) return;  // no rows in this block
  const int n = (uc.y - uc.x + 1) * per;
  const size_t slot0 = (size_t)u + uc.x;
  const float* lse = a.part_lse + slot0 * 256;
  const float4* po = reinterpret_cast<const float4*>(a.part_o) + slot0 * ngrp * 256;
  // record c: row of the segment's 256 (its chain's 128 where the chains split)
  auto at = [&](int c) { return per == 2 ? (c & 1) * 128 + r : row; };
  auto rec = [&](int c) { return (size_t)(per == 2 ? c >> 1 : c); };
  const int g0 = (part * 8 + (threadIdx.x >> 5)) * NG;
  float mx = -INFINITY, den = 0.f;
  float4 acc[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int c0 = 0; c0 < n; c0 += KB) {
    float x[KB];
    float4 o[KB][NG];
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int c = min(c0 + k, n - 1);
      x[k] = __ldg(lse + rec(c) * 256 + at(c));
#pragma unroll
      for (int g = 0; g < NG; ++g) o[k][g] = __ldcg(po + (rec(c) * ngrp + g0 + g) * 256 + at(c));
    }
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      // past the last record, or one without keys (its output was never written)
      if (c0 + k >= n || x[k] == -INFINITY) continue;
      const float mn = x[k] > mx ? x[k] : mx;
      const float f0 = ex2(mx - mn), f1 = ex2(x[k] - mn);
      mx = mn;
      den = fmaf(den, f0, f1);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        acc[g].x = fmaf(acc[g].x, f0, o[k][g].x * f1);
        acc[g].y = fmaf(acc[g].y, f0, o[k][g].y * f1);
        acc[g].z = fmaf(acc[g].z, f0, o[k][g].z * f1);
        acc[g].w = fmaf(acc[g].w, f0, o[k][g].w * f1);
      }
    }
  }
  const float inv = 1.f / den;
  if (r >= a.rows_per_half) return;
  const int U = a.Hkv * a.n_qtiles;
  const int b = u / U, uk = u - b * U, ug = uk / a.n_qtiles, qt = uk - ug * a.n_qtiles;
  const int s = qt * a.halves * a.s_per_half + h * a.s_per_half + r / a.G;
  uint16_t* dst = a.out + (((size_t)b * a.S + s) * a.Hq + ug * a.G + r % a.G) * a.dh + g0 * 4;
#pragma unroll
  for (int g = 0; g < NG; ++g)
    *reinterpret_cast<uint2*>(dst + 4 * g) =
        make_uint2(pack_bf16x2(acc[g].x * inv, acc[g].y * inv),
                   pack_bf16x2(acc[g].z * inv, acc[g].w * inv));
}

template <int TYPE, int DH>
cudaError_t launch_main(const AttnQ8Args& a, cudaStream_t st) {
  constexpr size_t smem = smem_layout(DH).total + 1024;
  static_assert(smem <= 232448, "shared memory per CTA");
  const cudaError_t e = allow_smem<attn_q8_kernel<TYPE, DH>>(smem);
  if (e != cudaSuccess) return e;
  return launch_k(attn_q8_kernel<TYPE, DH>, dim3(a.n_ctas), dim3(kThreads), smem, st, a);
}

}  // namespace

cudaError_t launch_attn_q8(const AttnQ8Args& a, int type, cudaStream_t st) {
  if (type == TT_Q8_INT8)
    return a.dh == 64 ? launch_main<TT_Q8_INT8, 64>(a, st) : launch_main<TT_Q8_INT8, 128>(a, st);
  return a.dh == 64 ? launch_main<TT_Q8_E4M3, 64>(a, st) : launch_main<TT_Q8_E4M3, 128>(a, st);
}

cudaError_t launch_attn_q8_merge(const AttnQ8Args& a, cudaStream_t st) {
  // Few units (many records each): a quarter (dh 128) or half of a row to a
  // block, so that the whole GPU reads, and ten records at a time.  Many units
  // have two or three records: whole rows, which share the weights' arithmetic.
  const int blocks = a.units * a.halves * 4;
  if (blocks < 4 * num_sms())
    return launch_k(attn_q8_merge_kernel<1, 10>, dim3(blocks * (a.dh / 32)), dim3(256), 0, st, a);
  if (a.dh == 64)
    return launch_k(attn_q8_merge_kernel<2, 4>, dim3(blocks), dim3(256), 0, st, a);
  return launch_k(attn_q8_merge_kernel<4, 3>, dim3(blocks), dim3(256), 0, st, a);
}

}  // namespace tt
