// Persistent tcgen05 integer GEMM: C = A[M, K] . B[N, K]^T with int8 operands
// and exact 32-bit integer sums (kind::i8), for the 8-bit linear update and
// the 8-bit vocabulary projection.
//
// A 128-byte-swizzled K-major tile is the same bytes whatever the element, so
// the pipeline is that of the bf16 GEMM with 128 values of K per stage where
// that has 64: warp 0 issues TMA, warp 1 tcgen05.mma (M = 128, N = BN, K = 32)
// into one of two BN-column accumulators in TMEM, warps 2..5 drain the other.
// The scales enter in the epilogue: a row's and a column's, in fp32.
// A K that is no multiple of 128 ends in a box whose missing bytes TMA fills
// with zeros.
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

// EPI 0: vocabulary statistics, 1: bf16 store.
template <int EPI, int BN, int STAGES>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const GemmI8Args a) {
  griddep_launch();
  griddep_wait();
  extern __shared__ uint8_t smem_raw[];
  const int M = a.M_dev != nullptr ? min(*a.M_dev, a.M_alloc) : a.M_alloc;
  if (M <= 0) return;
  const int num_m = (M + kI8BM - 1) / kI8BM, num_n = (a.N + BN - 1) / BN;
  const int tiles = num_m * num_n;
  if ((int)blockIdx.x >= tiles) return;
  constexpr uint32_t kStageB = BN * kI8BK;
  const int nkb = (a.K + kI8BK - 1) / kI8BK;

  uint8_t* base = align1024(smem_raw);
  uint8_t* sA = base;
  uint8_t* sB = base + STAGES * kStageA;
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + STAGES * kStageB);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;
  uint64_t* acce = accf + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      const uint64_t keep = policy_evict_last(), once = policy_evict_first();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const int m = t % num_m, n = t / num_m;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, a.err, abort_flag, WHERE_GEMM_PRODUCER)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], kStageA + kStageB);
          tma_load_2d_hint(sA + stage * kStageA, &tmA, &full[stage], kb * kI8BK, m * kI8BM, keep);
          tma_load_2d_hint(sB + stage * kStageB, &tmB, &full[stage], kb * kI8BK, n * BN,
                           num_m > 1 ? keep : once);
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
        if (lane == 0) {
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
      if (lane == 0) umma_commit(&accf[acc]);
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const int m = t % num_m, n = t / num_m;
      const int row = m * kI8BM + q * 32 + lane;
      const int col0 = n * BN, ncols = min(BN, a.N - col0);
      const int nchunks = (ncols + 31) >> 5;
      const float rs = row < M ? a.a_scale[row] : 0.f;
      if (!mbar_wait(&accf[acc], acc_phase, a.err, abort_flag, WHERE_GEMM_EPI)) break;
      tc_fence_after();
      const uint32_t tbase = tmem + acc * BN + ((uint32_t)(q * 32) << 16);
      // The 32 column scales of a chunk, one per lane (0 past the last column).
      auto col_scale = [&](int ch) {
        const int c = ch * 32 + lane;
        return c < ncols ? __ldg(a.b_scale + col0 + c) : 0.f;
      };
      if constexpr (EPI == 0) {
        // Per row: the maximum of sum * column scale, the sum of exponentials
        // relative to it (differences first, so large logits lose nothing),
        // and the lowest column that attains it.
        const float c = a.scale_log2 * rs;
        float best = -INFINITY, z = 0.f;
        int bidx = 0;
        for (int ch = 0; ch < nchunks; ++ch) {
          uint32_t r[32];
          tmem_ld32(tbase + ch * 32, r);
          const float cs = col_scale(ch);
          tmem_wait_ld();
          const int lim = ncols - ch * 32;
          float cm = -INFINITY;
          int ci = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float v = (float)(int)r[j] * __shfl_sync(0xffffffffu, cs, j);
            r[j] = __float_as_uint(v);
            if (j < lim && v > cm) {
              cm = v;
              ci = j;
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
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acce[acc]);
        if (row < M)
          a.stats[(size_t)row * num_n + n] = make_float4(best, z, __int_as_float(col0 + bidx), 0.f);
      } else {
        for (int ch = 0; ch < nchunks; ++ch) {
          uint32_t r[32];
          tmem_ld32(tbase + ch * 32, r);
          const float cs = col_scale(ch);
          tmem_wait_ld();
          const int lim = ncols - ch * 32;
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float v0 = (float)(int)r[j] * (rs * __shfl_sync(0xffffffffu, cs, j));
            const float v1 = (float)(int)r[j + 1] * (rs * __shfl_sync(0xffffffffu, cs, j + 1));
            w[j >> 1] = pack_bf16x2(v0, v1);
          }
          if (row < M) {
            uint16_t* dst = a.C + (size_t)row * a.N + col0 + ch * 32;
            if ((a.N & 7) == 0) {  // every row 16-byte aligned, lim a multiple of 8
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (v * 8 < lim)
                  reinterpret_cast<uint4*>(dst)[v] =
                      make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j < lim) dst[j] = (uint16_t)(w[j >> 1] >> ((j & 1) * 16));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acce[acc]);
      }
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

template <int EPI, int BN, int STAGES>
cudaError_t launch_gemm_i8(const CUtensorMap& tmA, const CUtensorMap& tmB, const GemmI8Args& a,
                           int grid, cudaStream_t st) {
  constexpr size_t smem = (size_t)STAGES * (kI8BM + BN) * kI8BK + 1024 + 256;
  static_assert(smem <= 232448, "shared memory per CTA");
  static_assert(2 * BN <= 512, "two accumulators must fit TMEM");
  cudaError_t e = cudaFuncSetAttribute(gemm_i8_kernel<EPI, BN, STAGES>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_k(gemm_i8_kernel<EPI, BN, STAGES>, dim3(grid), dim3(kGemmThreads), smem, st, tmA,
                  tmB, a);
}

}  // namespace

cudaError_t launch_gemm_i8_vocab(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                 const GemmI8Args& a, int grid, cudaStream_t st) {
  return launch_gemm_i8<0, kI8VocabBN, kI8VocabStages>(tmA, tmB, a, grid, st);
}
cudaError_t launch_gemm_i8_linear(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                  const GemmI8Args& a, int grid, cudaStream_t st) {
  return launch_gemm_i8<1, kI8BN, kI8Stages>(tmA, tmB, a, grid, st);
}

}  // namespace tt
