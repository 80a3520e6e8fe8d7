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
// epilogue of one under the products of the next).  gemm_i8_split_kernel is
// for few tiles: a cluster of CTAs shares one tile and splits K, so that all
// SMs stream weights; each CTA then sends the others their columns of its
// partial sums through distributed shared memory and finishes its own.
// Integer sums do not depend on that order.
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

// One row's 32 columns (or `lim` of them): integer sums r to bf16, times the
// row's scale rs and the columns' cs (lane j holds column j's).  16-byte
// stores where every row is 16-byte aligned (N a multiple of 8).
__device__ __forceinline__ void store_row32(const uint32_t (&r)[32], float rs, float cs,
                                            uint16_t* dst, int lim, bool valid, bool vec) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float v0 = (float)(int)r[j] * (rs * __shfl_sync(0xffffffffu, cs, j));
    const float v1 = (float)(int)r[j + 1] * (rs * __shfl_sync(0xffffffffu, cs, j + 1));
    w[j >> 1] = pack_bf16x2(v0, v1);
  }
  if (!valid) return;
  if (vec) {
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
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + STAGES * kStageB);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;
  uint64_t* acce = accf + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

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
        const float c = row_factor(a.scale_log2, rs);
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
          store_row32(r, rs, cs, a.C + (size_t)row * a.N + col0 + ch * 32, ncols - ch * 32,
                      row < M, (a.N & 7) == 0);
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

// One 128 x BN tile to a cluster, whose CTAs each take a range of K (splits = 1:
// to a CTA).
template <int BN>
struct SplitShape {
  static constexpr int kStages = BN == 128 ? 5 : BN == 64 ? 7 : 9;
  static constexpr uint32_t kStageB = BN * kI8BK;
  // partial sums of the other CTAs for this one's columns: [source][column
  // group of 4][128 rows][4]; splits <= BN / 16
  static constexpr uint32_t kRecv = 128 * BN * 4 * (BN / 16 - 1) / (BN / 16);
  static constexpr size_t kSmem = kStages * (kStageA + kStageB) + kRecv + 1024 + 256;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
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
  uint64_t* full = reinterpret_cast<uint64_t*>(recv + Shape::kRecv);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
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
  if (splits > 1) cluster_arrive();  // this CTA runs: its memory may be written

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
    griddep_wait();  // the rows' scales
    const int row = m * kI8BM + row128;
    const float rs = row < a.M_alloc ? a.a_scale[row] : 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < part; c0 += 32) {
      const int col = n * BN + rank * part + c0;
      const int lim = min(min(32, part - c0), a.N - col);
      if (lim <= 0) break;
      uint32_t r[32];
      tmem_ld32(tbase + rank * part + (part < 32 ? 0 : c0), r);
      const float cs = lane < lim ? __ldg(a.b_scale + col + lane) : 0.f;
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
      store_row32(r, rs, cs, a.C + (size_t)row * a.N + col, lim, row < a.M_alloc, (a.N & 7) == 0);
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
  constexpr size_t smem = (size_t)STAGES * (kI8BM + BN) * kI8BK + 1024 + 256;
  static_assert(smem <= 232448, "shared memory per CTA");
  static_assert(2 * BN <= 512, "two accumulators must fit TMEM");
  const cudaError_t e = allow_smem<gemm_i8_kernel<EPI, BN, STAGES>>(smem);
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
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tiles * splits);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = splits;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, gemm_i8_split_kernel<BN>, tmA, tmB, a, splits);
}
cudaError_t launch_gemm_i8_split(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                 const GemmI8Args& a, int bn, int splits, cudaStream_t st) {
  if (bn == 32) return launch_split<32>(tmA, tmB, a, splits, st);
  if (bn == 64) return launch_split<64>(tmA, tmB, a, splits, st);
  return launch_split<128>(tmA, tmB, a, splits, st);
}

}  // namespace tt
