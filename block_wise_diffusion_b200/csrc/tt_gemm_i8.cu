// tcgen05 integer GEMM: C = A[M, K] . B[N, K]^T with int8 operands and exact
// 32-bit integer sums (kind::i8), for the 8-bit linear update and the 8-bit
// vocabulary projection.
//
// A 128-byte-swizzled K-major tile is the same bytes whatever the element, so
// the pipeline is that of the bf16 GEMM with 128 values of K per stage where
// that has 64: warp 0 issues TMA, warp 1 tcgen05.mma (M = 128, N = BN, K = 32)
// into TMEM, warps 2..5 drain it.  The scales enter in the epilogue: a row's
// and a column's, in fp32.  A K that is no multiple of 128 ends in a box whose
// missing bytes TMA fills with zeros.
//
// gemm_i8_kernel is persistent over output tiles (two accumulators, the
// epilogue of one under the products of the next), gemm_i8_pair_kernel the same
// with two CTAs to a tile.  gemm_i8_split_kernel is
// for few tiles: a cluster of CTAs shares one tile and splits K, so that all
// SMs stream weights; each CTA then sends the others their columns of its
// partial sums through distributed shared memory and finishes its own.
// Integer sums do not depend on that order.
//
// What bounds them: few rows, the weights' bytes from HBM (77 masked rows, V =
// 131072, H = 4096: 92 us with quantisation and commit, 5.8 TB/s; 128 x 4608, K =
// 4096, is too short for that: 10.4 us, 2 of them the rows' quantisation); many
// rows, the tensor cores at the clock that the power limit leaves (1024 rows of the
// same vocabulary step: 380 us, 2.9 PFLOP/s of integer products).
//
// The kernel before either of these quantises the rows of A and starts its
// dependent only once everything before itself is complete, so the weights may
// be read before griddepcontrol.wait: the first stages of B are in flight while
// A is still being written.
#include <math.h>

#include "tt_q8.h"
#include "tt_ptx.cuh"

namespace tt {

namespace {

constexpr uint32_t kStageA = kI8BM * kI8BK;  // 16 KB

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// D(tmem) (+)= A(smem desc) * B(smem desc), int8 inputs, int32 accumulate.
__device__ __forceinline__ void umma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::i8: signed A and B, int32 D, K-major.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (publishes nothing but what a fence before it has)
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A tile's column scales to the warp's own shared memory, 0 past the last column:
// before the sums are ready, so that the epilogue does not wait for them chunk by
// chunk.
template <int COLS>
__device__ __forceinline__ void stage_scales(float* cs, const float* b_scale, int ncols) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = lane; c < COLS; c += 32) cs[c] = c < ncols ? __ldg(b_scale + c) : 0.f;
  __syncwarp();
}

// One row's 32 columns (or `lim` of them): integer sums r to bf16, times the
// row's scale rs and the columns' cs; dst: the row's first of them.  vec: 32- or
// 16-byte stores where every row is that aligned (2, 1).  Other N (0): through the
// warp's own `stage`, so that a store is a run of one or two rows (2048 x 4607, K =
// 4096: 45 us; single values, a lane to a row, took 121).  All lanes take part, row0
// is the first lane's row.
constexpr int kStageWords = 32 * 17;  // a row to 17 words: no bank conflicts
__device__ __forceinline__ int store_width(const uint16_t* C, int N) {
  return (N & 15) == 0 && (reinterpret_cast<uintptr_t>(C) & 31) == 0 ? 2 : (N & 7) == 0 ? 1 : 0;
}
__device__ __forceinline__ void store_row32(const uint32_t (&r)[32], float rs, const float* cs,
                                            uint16_t* dst, int lim, int row0, int M, int N, int vec,
                                            uint32_t* stage) {
  const int lane = threadIdx.x & 31;
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 c = *reinterpret_cast<const float4*>(cs + j);
    w[j / 2] = pack_bf16x2((float)(int)r[j] * (rs * c.x), (float)(int)r[j + 1] * (rs * c.y));
    w[j / 2 + 1] = pack_bf16x2((float)(int)r[j + 2] * (rs * c.z), (float)(int)r[j + 3] * (rs * c.w));
  }
  if (vec == 0) {
#pragma unroll
    for (int j = 0; j < 16; ++j) stage[lane * 17 + j] = w[j];
    __syncwarp();
    uint16_t* d0 = dst - (ptrdiff_t)lane * N;  // row0's
    const int rows = min(32, M - row0);
    if ((N & 1) == 0) {
      for (int i = lane >> 4; i < rows; i += 2)
        if (2 * (lane & 15) < lim)
          *reinterpret_cast<uint32_t*>(d0 + (ptrdiff_t)i * N + 2 * (lane & 15)) =
              stage[i * 17 + (lane & 15)];
    } else {
      for (int i = 0; i < rows; ++i)
        if (lane < lim)
          d0[(ptrdiff_t)i * N + lane] = (uint16_t)(stage[i * 17 + (lane >> 1)] >> ((lane & 1) * 16));
    }
    __syncwarp();
    return;
  }
  if (row0 + lane >= M) return;
  if (vec == 2) {
#pragma unroll
    for (int v = 0; v < 2; ++v)
      if (v * 16 < lim)
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + v * 16),
                     "r"(w[8 * v]), "r"(w[8 * v + 1]), "r"(w[8 * v + 2]), "r"(w[8 * v + 3]),
                     "r"(w[8 * v + 4]), "r"(w[8 * v + 5]), "r"(w[8 * v + 6]), "r"(w[8 * v + 7])
                     : "memory");
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (v * 8 < lim)
        reinterpret_cast<uint4*>(dst)[v] =
            make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
  }
}

// Row `row` of an accumulator tile at TMEM address tbase, columns col0 .. + ncols
// with the scales cs: its statistics (EPI 0) or its bf16 values (EPI 1).
template <int EPI>
__device__ __forceinline__ void drain_tile(const GemmI8Args& a, uint32_t tbase, int row, int M,
                                           float rs, const float* cs, int n, int num_n, int col0,
                                           int ncols, uint32_t* stage) {
  const int nchunks = (ncols + 31) >> 5;
  if constexpr (EPI == 0) {
    // Per row: the maximum of sum * column scale, the sum of exponentials
    // relative to it (differences first, so large logits lose nothing),
    // and the lowest column that attains it.
    const float c = row_factor(a.scale_log2, rs);
    float best = -INFINITY, z = 0.f;
    int bidx = 0;
    for (int ch = 0; ch < nchunks; ++ch) {
      uint32_t r[32];
      tmem_ld32(tbase + ch * 32, r);
      tmem_wait_ld();
      const int lim = ncols - ch * 32;
      float cm = -INFINITY;
      int ci = 0;
#pragma unroll
      for (int j4 = 0; j4 < 32; j4 += 4) {
        const float4 c4 = *reinterpret_cast<const float4*>(cs + ch * 32 + j4);
        const float sc[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = j4 + i;
          const float v = (float)(int)r[j] * sc[i];
          r[j] = __float_as_uint(v);
          if (j < lim && v > cm) {
            cm = v;
            ci = j;
          }
        }
      }
      if (cm > best) {
        z *= ex2((best - cm) * c);  // 0 at the first chunk
        best = cm;
        bidx = ch * 32 + ci;
      }
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float e = ex2((__uint_as_float(r[j]) - best) * c);
        s += (j < lim) ? e : 0.f;
      }
      z += s;
    }
    if (row < M)
      a.stats[(size_t)row * num_n + n] = make_float4(best, z, __int_as_float(col0 + bidx), 0.f);
  } else {
    const int vec = store_width(a.C, a.N);
    uint16_t* dst = a.C + (size_t)row * a.N + col0;
    for (int ch = 0; ch < nchunks; ++ch) {
      uint32_t r[32];
      tmem_ld32(tbase + ch * 32, r);
      tmem_wait_ld();
      store_row32(r, rs, cs + ch * 32, dst + ch * 32, ncols - ch * 32, row - (threadIdx.x & 31), M,
                  a.N, vec, stage);
    }
  }
}

// EPI 0: vocabulary statistics, 1: bf16 store.
template <int EPI, int BN, int STAGES>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const GemmI8Args a) {
  griddep_launch();
  extern __shared__ uint8_t smem_raw[];
  const int num_n = (a.N + BN - 1) / BN;
  constexpr uint32_t kStageB = BN * kI8BK;
  const int nkb = (a.K + kI8BK - 1) / kI8BK;
  // With one row tile a CTA's first tile does not depend on the row count:
  // its first B stages are requested before the rows of A are ready.
  const int early = a.M_alloc <= kI8BM ? min(nkb, STAGES) : 0;
  const uint32_t a_bytes = (uint32_t)a.a_box * kI8BK;

  uint8_t* base = align1024(smem_raw);
  uint8_t* sA = base;
  uint8_t* sB = base + STAGES * kStageA;
  uint8_t* bars = sB + STAGES * kStageB;
  uint64_t* full = reinterpret_cast<uint64_t*>(bars);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;
  uint64_t* acce = accf + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  float* scales = reinterpret_cast<float*>(bars + 256);  // of a tile, by each epilogue warp

  // (the shuffle tells the compiler that the index is the same in all lanes)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp == 0 && lane == 0 && early > 0) {
    const uint64_t once = policy_evict_first();
    for (int kb = 0; kb < early; ++kb) {
      mbar_arrive_expect_tx(&full[kb], a_bytes + kStageB);
      tma_load_2d_hint(sB + kb * kStageB, &tmB, &full[kb], kb * kI8BK, blockIdx.x * BN, once);
    }
  }
  griddep_wait();
  const int M = a.M_dev != nullptr ? min(*a.M_dev, a.M_alloc) : a.M_alloc;
  const int num_m = (M + kI8BM - 1) / kI8BM;
  const int tiles = num_m * num_n;

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      const uint64_t keep = policy_evict_last(), once = policy_evict_first();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      if (tiles == 0) {
        // no rows after all: the copies in flight end before the CTA does
        for (int kb = 0; kb < early; ++kb)
          tma_load_2d_hint(sA + kb * kStageA, &tmA, &full[kb], kb * kI8BK, 0, keep);
        for (int kb = 0; kb < early; ++kb)
          mbar_wait(&full[kb], 0, a.err, abort_flag, WHERE_GEMM_PRODUCER);
      }
      int ahead = early;  // stages whose B is already on its way
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const int m = t % num_m, n = t / num_m;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, a.err, abort_flag, WHERE_GEMM_PRODUCER)) {
            ok = false;
            break;
          }
          if (ahead == 0) mbar_arrive_expect_tx(&full[stage], a_bytes + kStageB);
          tma_load_2d_hint(sA + stage * kStageA, &tmA, &full[stage], kb * kI8BK, m * kI8BM, keep);
          if (ahead == 0)
            tma_load_2d_hint(sB + stage * kStageB, &tmB, &full[stage], kb * kI8BK, n * BN,
                             num_m > 1 ? keep : once);
          else
            --ahead;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = idesc_i8(kI8BM, BN);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      if (!mbar_wait(&acce[acc], acc_phase ^ 1, a.err, abort_flag, WHERE_GEMM_MMA)) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * BN;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait(&full[stage], phase, a.err, abort_flag, WHERE_GEMM_MMA)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a0 = sdesc_sw128(smem_u32(sA + stage * kStageA), 16, 1024);
          const uint64_t b0 = sdesc_sw128(smem_u32(sB + stage * kStageB), 16, 1024);
#pragma unroll
          for (int k = 0; k < kI8BK / 32; ++k)
            umma_i8_ss(d, a0 + k * 2, b0 + k * 2, idesc, (kb | k) != 0);
          umma_commit(&empty[stage]);
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) umma_commit(&accf[acc]);
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    float* cs = scales + q * BN;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const int m = t % num_m, n = t / num_m;
      const int row = m * kI8BM + q * 32 + lane;
      const int col0 = n * BN, ncols = min(BN, a.N - col0);
      const float rs = row < M ? a.a_scale[row] : 0.f;
      stage_scales<BN>(cs, a.b_scale + col0, ncols);
      if (!mbar_wait(&accf[acc], acc_phase, a.err, abort_flag, WHERE_GEMM_EPI)) break;
      tc_fence_after();
      const uint32_t tbase = tmem + acc * BN + ((uint32_t)(q * 32) << 16);
      drain_tile<EPI>(a, tbase, row, M, rs, cs, n, num_n, col0, ncols,
                      reinterpret_cast<uint32_t*>(scales + 4 * BN) + q * kStageWords);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- the same with two CTAs to a 256-row tile (tcgen05 cta_group::2)
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// Box to this CTA's shared memory, counted on the (mapped) barrier of CTA 0.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* m, uint32_t bar,
                                                 int x, int y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
      "l"(m), "r"(bar), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both CTAs when the MMAs issued so far are complete.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// Each CTA loads its 128 rows of A and half of the tile's rows of B; the products
// that CTA 0 issues read both halves of B and leave 128 x BN sums in each CTA's
// TMEM, so a tile costs each SM two thirds of the operand bytes of a 128 x 256
// tile of its own.  (2048 x 4608, K = 4096: 24 us from the first products to the
// last, 17 of them the tensor cores' own; then 3 us for the last tile's epilogue.
// A column's scale read from global memory for each chunk, and stores of half
// sectors, made that epilogue 7 us.)
template <int BN, int STAGES>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_i8_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB, const GemmI8Args a) {
  griddep_launch();
  extern __shared__ uint8_t smem_raw[];
  const int num_n = (a.N + BN - 1) / BN;
  constexpr uint32_t kStageB = BN / 2 * kI8BK;
  const int nkb = (a.K + kI8BK - 1) / kI8BK;
  uint8_t* base = align1024(smem_raw);
  uint8_t* sA = base;
  uint8_t* sB = base + STAGES * kStageA;
  uint8_t* bars = sB + STAGES * kStageB;
  uint64_t* full = reinterpret_cast<uint64_t*>(bars);  // CTA 0's, for both
  uint64_t* empty = full + STAGES;                     // each CTA's own
  uint64_t* accf = empty + STAGES;                     // each CTA's own
  uint64_t* acce = accf + 2;                           // CTA 0's, for both
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  float* scales = reinterpret_cast<float*>(bars + 256);  // of a tile, by each epilogue warp

  // (the shuffle tells the compiler that the index is the same in all lanes)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 8);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  // An allocation for a pair needs both CTAs running, and a product or a copy both
  // CTAs' TMEM and barriers ready.
  __syncthreads();
  cluster_arrive_relaxed();
  cluster_wait();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int M = a.M_alloc;
  const int num_m = (M + 2 * kI8BM - 1) / (2 * kI8BM);
  const int tiles = num_m * num_n, t0 = blockIdx.x >> 1, dt = gridDim.x >> 1;
  const int early = min(nkb, STAGES);  // the first B stages do not wait for A
  const uint32_t full0 = map_rank(full, 0);
  if (warp == 0 && lane == 0) {
    const uint64_t keep = policy_evict_last();
    for (int kb = 0; kb < early; ++kb) {
      if (rank == 0) mbar_arrive_expect_tx(&full[kb], 2 * (kStageA + kStageB));
      tma_load_2d_pair(sB + kb * kStageB, &tmB, full0 + kb * 8, kb * kI8BK,
                       t0 / num_m * BN + rank * (BN / 2), keep);
    }
  }
  griddep_wait();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      const uint64_t keep = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int ahead = early;  // stages whose B is already on its way
      for (int t = t0; ok && t < tiles; t += dt) {
        const int m = t % num_m, n = t / num_m;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, a.err, abort_flag, WHERE_GEMM_PRODUCER)) {
            ok = false;
            break;
          }
          // (bytes that arrive before they are expected are counted all the same:
          // the phase cannot end before this arrival)
          if (rank == 0 && ahead == 0) mbar_arrive_expect_tx(&full[stage], 2 * (kStageA + kStageB));
          tma_load_2d_pair(sA + stage * kStageA, &tmA, full0 + stage * 8, kb * kI8BK,
                           (2 * m + rank) * kI8BM, keep);
          if (ahead == 0)
            tma_load_2d_pair(sB + stage * kStageB, &tmB, full0 + stage * 8, kb * kI8BK,
                             n * BN + rank * (BN / 2), keep);
          else
            --ahead;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // the last arrivals on this CTA's barriers, before it may end
      for (int i = 0; ok && i < STAGES; ++i) {
        ok = mbar_wait(&empty[stage], phase ^ 1, a.err, abort_flag, WHERE_GEMM_PRODUCER);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // -------------------------------------- MMA issuer, for both CTAs
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_i8(2 * kI8BM, BN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = t0; ok && t < tiles; t += dt) {
        if (!mbar_wait(&acce[acc], acc_phase ^ 1, a.err, abort_flag, WHERE_GEMM_MMA)) break;
        asm volatile("fence.acq_rel.cluster;" ::: "memory");  // the other CTA's epilogue
        tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&full[stage], phase, a.err, abort_flag, WHERE_GEMM_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t a0 = sdesc_sw128(smem_u32(sA + stage * kStageA), 16, 1024);
            const uint64_t b0 = sdesc_sw128(smem_u32(sB + stage * kStageB), 16, 1024);
#pragma unroll
            for (int k = 0; k < kI8BK / 32; ++k)
              umma_i8_pair(d, a0 + k * 2, b0 + k * 2, idesc, (kb | k) != 0);
            umma_commit_pair(&empty[stage]);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit_pair(&accf[acc]);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    float* cs = scales + q * BN;
    const uint32_t acce0 = map_rank(acce, 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = t0; t < tiles; t += dt) {
      const int m = t % num_m, n = t / num_m;
      const int row = (2 * m + rank) * kI8BM + q * 32 + lane;
      const int col0 = n * BN, ncols = min(BN, a.N - col0);
      const float rs = row < M ? a.a_scale[row] : 0.f;
      stage_scales<BN>(cs, a.b_scale + col0, ncols);
      if (!mbar_wait(&accf[acc], acc_phase, a.err, abort_flag, WHERE_GEMM_EPI)) break;
      tc_fence_after();
      drain_tile<1>(a, tmem + acc * BN + ((uint32_t)(q * 32) << 16), row, M, rs, cs, n, num_n, col0,
                      ncols,
                    reinterpret_cast<uint32_t*>(scales + 4 * BN) + q * kStageWords);
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         acce0 + acc * 8)
                     : "memory");
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();  // neither CTA's memory is used any more
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// One 128 x BN tile to a cluster, whose CTAs each take a range of K (splits = 1:
// to a CTA).
template <int BN>
struct SplitShape {
  static constexpr int kStages = BN == 128 ? 5 : BN == 64 ? 7 : 9;
  static constexpr uint32_t kStageB = BN * kI8BK;
  // partial sums of the other CTAs for this one's columns: [source][column
  // group of 4][128 rows][4]; splits <= BN / 16
  static constexpr uint32_t kRecv = 128 * BN * 4 * (BN / 16 - 1) / (BN / 16);
  static constexpr size_t kSmem = kStages * (kStageA + kStageB) + kRecv + 1024 + 256 + 4 * BN * 4;
};

// 16 bytes to the same shared-memory address of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster(uint32_t saddr, uint32_t rank, uint32_t x, uint32_t y,
                                           uint32_t z, uint32_t w) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(saddr), "r"(rank));
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(remote), "r"(x), "r"(y),
               "r"(z), "r"(w)
               : "memory");
}

template <int BN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_i8_split_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB, const GemmI8Args a,
                         const int splits) {
  griddep_launch();
  using Shape = SplitShape<BN>;
  constexpr int STAGES = Shape::kStages;
  constexpr uint32_t kStageB = Shape::kStageB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = align1024(smem_raw);
  uint8_t* sA = base;
  uint8_t* sB = base + STAGES * kStageA;
  uint8_t* recv = sB + STAGES * kStageB;
  uint8_t* bars = recv + Shape::kRecv;
  uint64_t* full = reinterpret_cast<uint64_t*>(bars);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  float* scales = reinterpret_cast<float*>(bars + 256);  // of a tile, by each epilogue warp
  // (the shuffle tells the compiler that the index is the same in all lanes)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = splits > 1 ? (int)cluster_rank() : 0;
  const int num_m = (a.M_alloc + kI8BM - 1) / kI8BM;
  const int tile = blockIdx.x / splits, m = tile % num_m, n = tile / num_m;
  const int nkb = (a.K + kI8BK - 1) / kI8BK;
  const int kb0 = rank * nkb / splits, kb1 = (rank + 1) * nkb / splits;
  const uint32_t a_bytes = (uint32_t)a.a_box * kI8BK;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(accf, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);  // (32 columns are read at a time, from 112 at the last)
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (splits > 1) cluster_arrive_relaxed();  // this CTA runs: its memory may be written

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t keep = policy_evict_last();
      // (a fresh ring: the first STAGES stages need no wait)
      const int early = min(kb1 - kb0, STAGES);
      for (int i = 0; i < early; ++i) {
        mbar_arrive_expect_tx(&full[i], a_bytes + kStageB);
        tma_load_2d_hint(sB + i * kStageB, &tmB, &full[i], (kb0 + i) * kI8BK, n * BN, keep);
      }
      griddep_wait();
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1, a.err, abort_flag, WHERE_GEMM_PRODUCER)) break;
        if (kb - kb0 >= early) {
          mbar_arrive_expect_tx(&full[stage], a_bytes + kStageB);
          tma_load_2d_hint(sB + stage * kStageB, &tmB, &full[stage], kb * kI8BK, n * BN,
                           keep);
        }
        tma_load_2d_hint(sA + stage * kStageA, &tmA, &full[stage], kb * kI8BK, m * kI8BM, keep);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_i8(kI8BM, BN);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(&full[stage], phase, a.err, abort_flag, WHERE_GEMM_MMA)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint64_t a0 = sdesc_sw128(smem_u32(sA + stage * kStageA), 16, 1024);
        const uint64_t b0 = sdesc_sw128(smem_u32(sB + stage * kStageB), 16, 1024);
#pragma unroll
        for (int k = 0; k < kI8BK / 32; ++k)
          umma_i8_ss(tmem, a0 + k * 2, b0 + k * 2, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
        umma_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (ok && elect_one()) umma_commit(accf);
    __syncwarp();
  }
  const int q = warp & 3, row128 = q * 32 + lane;
  const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
  const int part = BN / splits;  // columns this CTA finishes: rank * part ..
  const int row = m * kI8BM + row128;
  float* cs = scales + q * BN;
  float rs = 0.f;
  if (warp >= 2) {
    const int col = n * BN + rank * part;
    stage_scales<BN>(cs, a.b_scale + col, min(part, a.N - col));
    griddep_wait();  // the rows' scales
    if (row < a.M_alloc) rs = a.a_scale[row];
  }
  __syncwarp();
  if (splits > 1) cluster_wait();  // all CTAs of the cluster run
  bool ok = warp >= 2 && mbar_wait(accf, 0, a.err, abort_flag, WHERE_GEMM_EPI);
  if (ok) tc_fence_after();
  if (ok && splits > 1) {
#pragma unroll 1
    for (int c0 = 0; c0 < BN; c0 += 16) {
      const int to = c0 / part;
      if (to == rank) continue;
      uint32_t r[16];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
          "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
          : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
            "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
            "=r"(r[14]), "=r"(r[15])
          : "r"(tbase + c0));
      tmem_wait_ld();
      // this CTA is source (rank - 1 - to mod splits) of CTA `to`
      const int src = (rank - to - 1 + splits) % splits;
      const uint32_t at = smem_u32(recv) + (uint32_t)(src * (part / 4) + (c0 - to * part) / 4) * 2048 +
                          row128 * 16;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        st_cluster(at + v * 2048, to, r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
    }
  }
  // every thread of the cluster arrives, whatever happened above
  if (splits > 1) {
    __syncthreads();
    cluster_arrive();
    cluster_wait();
  }
  if (ok) {
    const int vec = store_width(a.C, a.N);
#pragma unroll 1
    for (int c0 = 0; c0 < part; c0 += 32) {
      const int col = n * BN + rank * part + c0;
      const int lim = min(min(32, part - c0), a.N - col);
      if (lim <= 0) break;
      uint32_t r[32];
      tmem_ld32(tbase + rank * part + (part < 32 ? 0 : c0), r);
      tmem_wait_ld();
#pragma unroll 1
      for (int src = 0; src < splits - 1; ++src) {
        const uint4* p = reinterpret_cast<const uint4*>(recv + (size_t)(src * (part / 4) + c0 / 4) * 2048 +
                                                        row128 * 16);
#pragma unroll
        for (int v = 0; v < 8; ++v)
          if (v * 4 < part) {
            const uint4 x = p[v * 128];
            r[4 * v] += x.x;
            r[4 * v + 1] += x.y;
            r[4 * v + 2] += x.z;
            r[4 * v + 3] += x.w;
          }
      }
      // (the ring is free by now)
      store_row32(r, rs, cs + c0, a.C + (size_t)row * a.N + col, lim, row - lane, a.M_alloc, a.N, vec,
                  reinterpret_cast<uint32_t*>(sA) + q * kStageWords);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <int EPI, int BN, int STAGES>
cudaError_t launch_gemm_i8(const CUtensorMap& tmA, const CUtensorMap& tmB, const GemmI8Args& a,
                           int grid, cudaStream_t st) {
  constexpr size_t smem = (size_t)STAGES * (kI8BM + BN) * kI8BK + 1024 + 256 + 4 * BN * 4 +
                          (EPI == 1 ? 4 * kStageWords * 4 : 0);
  static_assert(smem <= 232448, "shared memory per CTA");
  static_assert(2 * BN <= 512, "two accumulators must fit TMEM");
  const cudaError_t e = allow_smem<gemm_i8_kernel<EPI, BN, STAGES>>(smem);
  if (e != cudaSuccess) return e;
  return launch_k(gemm_i8_kernel<EPI, BN, STAGES>, dim3(grid), dim3(kGemmThreads), smem, st, tmA,
                  tmB, a);
}

}  // namespace

// `cluster` CTAs (more than one) to a cluster, with the dependent-launch attribute.
template <class Kern, class... Args>
static cudaError_t launch_cluster(Kern kern, int grid, int cluster, size_t smem, cudaStream_t st,
                                  const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <int BN, int STAGES>
static cudaError_t launch_gemm_i8_pair(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                       const GemmI8Args& a, int pairs, cudaStream_t st) {
  constexpr size_t smem = (size_t)STAGES * (kI8BM + BN / 2) * kI8BK + 1024 + 256 + 4 * BN * 4 +
                          4 * kStageWords * 4;
  static_assert(smem <= 232448, "shared memory per CTA");
  static_assert(2 * BN <= 512, "two accumulators must fit TMEM");
  const cudaError_t e = allow_smem<gemm_i8_pair_kernel<BN, STAGES>>(smem);
  if (e != cudaSuccess) return e;
  return launch_cluster(gemm_i8_pair_kernel<BN, STAGES>, 2 * pairs, 2, smem, st, tmA, tmB, a);
}

cudaError_t launch_gemm_i8_vocab(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                 const GemmI8Args& a, int grid, cudaStream_t st) {
  return launch_gemm_i8<0, kI8VocabBN, kI8VocabStages>(tmA, tmB, a, grid, st);
}
cudaError_t launch_gemm_i8_linear(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                  const GemmI8Args& a, bool pair, int grid, cudaStream_t st) {
  if (pair) return launch_gemm_i8_pair<kI8BN, kI8PairStages>(tmA, tmB, a, grid, st);
  return launch_gemm_i8<1, kI8BN, kI8Stages>(tmA, tmB, a, grid, st);
}

template <int BN>
static cudaError_t launch_split(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                const GemmI8Args& a, int splits, cudaStream_t st) {
  constexpr size_t smem = SplitShape<BN>::kSmem;
  static_assert(smem <= 232448, "shared memory per CTA");
  const cudaError_t e = allow_smem<gemm_i8_split_kernel<BN>>(smem);
  if (e != cudaSuccess) return e;
  const int tiles = ((a.M_alloc + kI8BM - 1) / kI8BM) * ((a.N + BN - 1) / BN);
  if (splits == 1)
    return launch_k(gemm_i8_split_kernel<BN>, dim3(tiles), dim3(kGemmThreads), smem, st, tmA, tmB,
                    a, 1);
  return launch_cluster(gemm_i8_split_kernel<BN>, tiles * splits, splits, smem, st, tmA, tmB, a,
                        splits);
}
cudaError_t launch_gemm_i8_split(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                 const GemmI8Args& a, int bn, int splits, cudaStream_t st) {
  if (bn == 32) return launch_split<32>(tmA, tmB, a, splits, st);
  if (bn == 64) return launch_split<64>(tmA, tmB, a, splits, st);
  return launch_split<128>(tmA, tmB, a, splits, st);
}

}  // namespace tt
