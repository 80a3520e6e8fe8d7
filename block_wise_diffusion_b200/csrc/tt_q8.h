// Internal definitions of the 8-bit serving operators.
#pragma once
#include <atomic>

#include "tt_internal.h"

namespace tt {

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per context: a call
// of these operators can be shorter than the attribute call is.
template <auto Kern>
inline cudaError_t allow_smem(size_t bytes) {
  static std::atomic<unsigned long long> done{0};  // context it was last set for
  unsigned long long id = 0;
  const bool known = current_context_id(&id);
  if (known && done.load(std::memory_order_relaxed) == id) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && known) done.store(id, std::memory_order_relaxed);
  return e;
}

// ------------------------------------------------------------ cache append
struct AppendQ8Args {
  int B, Hkv, dh, L_cap, n, n_blocks;  // n_blocks: scales per (sequence, head)
  int block_shift;                     // 2^block_shift positions per scale
  int groups;                          // of cache blocks that a CTA takes side by side
  const int* new_len;                         // optional [B]
  const uint16_t *k_new, *v_new;
  long long stride_b, stride_t, stride_h;     // elements
  uint8_t *k_ctx, *v_ctx;
  float *k_scale, *v_scale;
  int* ctx_len;
  int* err;
};
cudaError_t launch_append_q8(const AppendQ8Args& a, int type, cudaStream_t st);
// ctx_len and the error word, after launch_append_q8.
cudaError_t launch_append_q8_len(const AppendQ8Args& a, cudaStream_t st);

// Row r < rows (or < *M_dev) of x, or row rowlist[r] of it: int8 codes q[r, :]
// and scale[r].
// err: an error word to clear first (optional).
cudaError_t launch_quant_rows(const uint16_t* x, int K, int8_t* q, float* scale,
                              const int* rowlist, const int* M_dev, int rows, int* err,
                              cudaStream_t st);

// The masked rows of x, compacted and quantised; writes rowlist (as PlanArgs
// has it), ctrl[CTRL_M], and clears the error words and seqcnt[0 .. rows / S).
cudaError_t launch_masked_rows(const uint16_t* x, int K, int8_t* q, float* scale,
                               const uint8_t* masked, int rows, int S, int* rowlist, int* ctrl,
                               int* seqcnt, cudaStream_t st);

// ------------------------------------------------------- integer products
// C = A[M, K] . B[N, K]^T, both int8 and K-major, 128 rows x 128 bytes of K
// per tile.
constexpr int kI8BM = 128, kI8BK = 128;
constexpr int kI8VocabBN = kVocabBN, kI8VocabStages = 5;
constexpr int kI8BN = 256, kI8Stages = 4, kI8PairStages = 6;
struct GemmI8Args {
  int M_alloc;           // rows of A
  int a_box;             // rows of a TMA box of A: fewer than 128 when A has fewer (the
                         // tile's other rows stay as they are and are never stored)
  const int* M_dev;      // device row count (nullptr: M_alloc)
  int N, K;
  const float* a_scale;  // [M]
  const float* b_scale;  // [N]
  float4* stats;         // vocabulary: [row][ceil(N / kI8VocabBN)], as GemmArgs::stats
  float scale_log2;      // vocabulary: logit_scale * log2(e)
  uint16_t* C;           // linear: bf16 [M, N]
  int* err;
};
cudaError_t launch_gemm_i8_vocab(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                 const GemmI8Args& a, int grid, cudaStream_t st);
// grid: CTAs, or pairs of CTAs with `pair` (256-row tiles; tmB's box then has half
// a tile's columns).
cudaError_t launch_gemm_i8_linear(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                  const GemmI8Args& a, bool pair, int grid, cudaStream_t st);
// Few tiles: `splits` CTAs (a power of two, at most bn / 16) to a 128 x bn tile,
// bn 32, 64 or 128.
cudaError_t launch_gemm_i8_split(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                 const GemmI8Args& a, int bn, int splits, cudaStream_t st);

// --------------------------------------------------------------- attention
// Units, query tiles and the partition of key tiles are those of the bf16
// call; see tt_attn_q8.cuh for the schedule.
struct AttnQ8Args {
  int B, S, Hq, Hkv, dh, G, L_cap, block_shift, n_blocks;  // 2^block_shift positions per scale
  const uint16_t *q, *k_blk, *v_blk;
  const uint8_t *k_ctx, *v_ctx;
  const float *k_scale, *v_scale;
  const int* ctx_len;
  float scale_log2;  // log2(e) / sqrt(dh)
  uint16_t* out;
  int s_per_half, rows_per_half, halves, n_qtiles, units, n_ctas;
  int g_shift;      // G = 2^g_shift
  int2* unit_span;  // [units] first and last CTA that hold tiles of the unit
  float* part_o;    // [units + n_ctas - 1] outputs of segments:
                    // [dh/4][256 rows][4], or [16 rows][dh] (at most 16 rows)
  float* part_lse;  // [units + n_ctas - 1][256 or 16 rows]: log2 of the segment's sum of
                    // 2^score; -inf without keys (its output is then never written)
  int* err;
};
cudaError_t launch_attn_q8(const AttnQ8Args& a, int type, cudaStream_t st);
cudaError_t launch_attn_q8_merge(const AttnQ8Args& a, cudaStream_t st);
// At most kRowsMax query rows per KV head.
constexpr int kRowsMax = 16;
cudaError_t launch_attn_q8_rows(const AttnQ8Args& a, int type, cudaStream_t st);
cudaError_t launch_attn_q8_rows_merge(const AttnQ8Args& a, cudaStream_t st);

// Query packing and CTA count of an attention call, as the bf16 call has them.
struct AttnShape {
  int G, s_per_half, rows_per_half, halves, n_qtiles, units, n_ctas;
};
AttnShape attn_shape(const tt_dims& d);

// Workspace bytes of the 8-bit calls of tt_workspace_bytes (d already checked).
size_t q8_workspace_bytes(const tt_dims& d, int which);

// 2-D map of bytes, 128-byte swizzle.
bool make_tmap_2d_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                     uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer);

}  // namespace tt
