// C ABI of the 8-bit serving operators: argument checks, workspace layout and
// kernel sequence.  The kernels are in tt_attn_q8.cu, tt_cache_q8.cu and
// tt_gemm_i8.cu; planning and commit are those of the bf16 step.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "tt_q8.h"

namespace tt {

namespace {

#define Q8_CHECK(x)             \
  do {                          \
    tt_status s_ = (x);         \
    if (s_ != TT_OK) return s_; \
  } while (0)

#define Q8_CUDA(call)                                                                  \
  do {                                                                                 \
    cudaError_t e_ = (call);                                                           \
    if (e_ != cudaSuccess)                                                             \
      return set_errorf(TT_ERR_CUDA, "%s failed: %s (%s:%d)", #call,                   \
                        cudaGetErrorString(e_), __FILE__, __LINE__);                   \
  } while (0)

#define Q8_LAUNCH(kind, st, call) \
  do {                            \
    prof_begin((kind), (st));     \
    Q8_CUDA(call);                \
    prof_end((kind), (st));       \
  } while (0)

tt_status check_ptr(const void* p, const char* name, unsigned align) {
  if (p == nullptr) return set_errorf(TT_ERR_INVALID_ARG, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0)
    return set_errorf(TT_ERR_INVALID_ARG, "%s is not %u-byte aligned", name, align);
  return TT_OK;
}

tt_status check_fmt(const tt_q8* f) {
  if (f == nullptr) return set_errorf(TT_ERR_INVALID_ARG, "format is NULL");
  if (f->type != TT_Q8_INT8 && f->type != TT_Q8_E4M3)
    return set_errorf(TT_ERR_UNSUPPORTED, "cache type %d is neither TT_Q8_INT8 nor TT_Q8_E4M3",
                      f->type);
  if (f->block != 16 && f->block != 32 && f->block != 64 && f->block != 128)
    return set_errorf(TT_ERR_UNSUPPORTED, "block=%d not in {16,32,64,128}", f->block);
  return TT_OK;
}

// Positions rounded up to a whole tile or block stay in 32 bits.
tt_status check_cache(const tt_dims* d, const tt_q8* f) {
  Q8_CHECK(check_dims_public(d));
  Q8_CHECK(check_fmt(f));
  if (d->L_cap > 0x7fffff00) return set_errorf(TT_ERR_UNSUPPORTED, "L_cap=%d too large", d->L_cap);
  return TT_OK;
}

int block_shift(const tt_q8& f) { return f.block == 16 ? 4 : f.block == 32 ? 5 : f.block == 64 ? 6 : 7; }

tt_status check_ws_ptr(void* ws, size_t have, size_t need) {
  Q8_CHECK(check_ptr(ws, "ws", 256));
  if (have < need)
    return set_errorf(TT_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return TT_OK;
}

struct Carver {
  uint8_t* base;
  size_t off = 0;
  template <class T>
  T* take(size_t bytes) {
    off = (off + 255) & ~size_t(255);
    T* p = base != nullptr ? reinterpret_cast<T*>(base + off) : nullptr;
    off += bytes;
    return p;
  }
  size_t total() const { return (off + 255) & ~size_t(255); }
};

// -------------------------------------------------------------- attention
struct AttnQ8Ws {
  int* ctrl;
  int2* unit_span;
  float *part_o, *part_lse;
  size_t total;
};
AttnQ8Ws carve_attn(const tt_dims& d, const AttnShape& g, void* ws) {
  Carver c{reinterpret_cast<uint8_t*>(ws)};
  AttnQ8Ws w;
  const size_t rows = d.S * g.G <= kRowsMax ? kRowsMax : 256;
  const size_t slots = (size_t)g.units + g.n_ctas - 1;
  w.ctrl = c.take<int>(kCtrlBytes);
  w.unit_span = c.take<int2>((size_t)g.units * sizeof(int2));
  w.part_o = c.take<float>(slots * rows * d.dh * sizeof(float));
  w.part_lse = c.take<float>(slots * rows * sizeof(float));
  w.total = c.total();
  return w;
}

// ------------------------------------------------------------- vocabulary
struct VocabWs {
  int *ctrl, *seqcnt, *rowlist;
  size_t clear;
  float* tvec;
  int8_t* yq;
  float* ys;
  float4* stats;
  float2* rowres;
  size_t total;
};
VocabWs carve_vocab(const tt_dims& d, void* ws) {
  Carver c{reinterpret_cast<uint8_t*>(ws)};
  const size_t rows = (size_t)d.B * d.S;
  VocabWs w;
  w.ctrl = c.take<int>(kCtrlBytes);
  w.seqcnt = c.take<int>((size_t)d.B * sizeof(int));
  w.clear = c.off;
  w.rowlist = c.take<int>(2 * rows * sizeof(int));
  w.tvec = c.take<float>((size_t)d.B * sizeof(float));
  w.yq = c.take<int8_t>(rows * d.H);
  w.ys = c.take<float>(rows * sizeof(float));
  w.stats = c.take<float4>(rows * ((d.V + kI8VocabBN - 1) / kI8VocabBN) * sizeof(float4));
  w.rowres = c.take<float2>(rows * sizeof(float2));
  w.total = c.total();
  return w;
}

// ----------------------------------------------------------------- linear
struct LinearWs {
  int* ctrl;
  int8_t* xq;
  float* xs;
  size_t total;
};
LinearWs carve_linear(int rows, int K, void* ws) {
  Carver c{reinterpret_cast<uint8_t*>(ws)};
  LinearWs w;
  w.ctrl = c.take<int>(kCtrlBytes);
  w.xq = c.take<int8_t>((size_t)rows * K);
  w.xs = c.take<float>((size_t)rows * sizeof(float));
  w.total = c.total();
  return w;
}

// Tile width and K split of the linear update.  Where 128-row tiles of 32, 64 or
// 128 columns are no more than the SMs, each tile goes to a cluster of `splits`
// CTAs that share its K: of the shapes that fit, the one whose CTAs read the
// fewest bytes, an exchange of partial sums counted as 200 KB (about 1 us).
// 128 x 4608, K = 4096: 72 tiles of 64 in pairs 10.6 us, 144 of 32 alone 12.2,
// 36 of 128 in fours 16.3 (clusters of four leave SMs of a GPC over, so not
// all 36 run at once: more than two CTAs only within 7/8 of the SMs).  64 x 1024, K =
// 8192: 11.3, the best shape 10.6; 384 x 2304, K = 4096: 12.2, the best.  Clusters of
// eight need more room than that bound leaves: 128 x 2048, K = 2048 takes 14.0 us with
// 16 of them, 7.1 as 64 pairs on 32 columns; 256 x 1024, K = 4096 16.1 and 9.5.
// splits = 0: more tiles than SMs; 256-wide tiles, one CTA each in turn, which
// read A less often.
struct I8Shape {
  int bn, splits;
};
I8Shape i8_shape(int rows, int N, int K) {
  const long long m_tiles = (rows + kI8BM - 1ll) / kI8BM;
  const int sms = num_sms(), nkb = (K + kI8BK - 1) / kI8BK;
  I8Shape best{kI8BN, 0};
  double least = 0;
  for (int bn = 32; bn <= 128; bn *= 2) {
    const long long tiles = m_tiles * ((N + bn - 1ll) / bn);
    if (tiles > sms) continue;
    int s = 1;
    while (2 * s <= bn / 16 && 4 * s <= nkb && tiles * 2 * s <= (s == 1 ? sms : sms * 7 / 8))
      s *= 2;
    const double bytes = (double)K / s * (kI8BM + bn) + (s > 1 ? 200e3 : 0);
    if (best.splits == 0 || bytes < least) {
      best = I8Shape{bn, s};
      least = bytes;
    }
  }
  return best;
}

// The persistent linear update: pairs of CTAs on 256-row tiles where there is more
// than one 128-row tile (K = 4096; 2048 x 4608: 34.3 us against 37.4 for CTAs on
// their own; 1024 x 6400: 31 against 35; 200 x 40000: 46 against 51; 16384 x 4608: 252
// against 293), also where the last pair has one 128-row tile and half of its work is
// idle, which costs up to 10 % (300 x 40000: 63 against 61; 384 x 20000: 40 against
// 36; 640 x 20000: 51 against 49).  The vocabulary step, whose row count only the GPU
// knows, keeps CTAs on their own: pairs gain 3 % at 1024 rows of 1024 and lose 20 %
// when 100 of them are masked.
bool i8_pair(int rows) { return rows > kI8BM; }

constexpr int kMaxRows = 1 << 24, kMaxK = 131072;
tt_status check_rows_k(int rows, int K) {
  if (rows < 1) return set_errorf(TT_ERR_INVALID_ARG, "rows=%d", rows);
  if (rows >= kMaxRows) return set_errorf(TT_ERR_UNSUPPORTED, "rows=%d not below 2^24", rows);
  if (K < 1) return set_errorf(TT_ERR_INVALID_ARG, "K=%d", K);
  if (K % 16 != 0 || K > kMaxK)
    return set_errorf(TT_ERR_UNSUPPORTED, "K=%d must be a multiple of 16 and <= %d", K, kMaxK);
  return TT_OK;
}
tt_status check_linear(int rows, int N, int K) {
  Q8_CHECK(check_rows_k(rows, K));
  if (N < 1) return set_errorf(TT_ERR_INVALID_ARG, "N=%d", N);
  if (N >= kMaxRows) return set_errorf(TT_ERR_UNSUPPORTED, "N=%d not below 2^24", N);
  const long long tiles = ((rows + kI8BM - 1ll) / kI8BM) * ((N + kI8BN - 1ll) / kI8BN);
  if (tiles >= (1ll << 31) - 1024) return set_errorf(TT_ERR_UNSUPPORTED, "problem too large");
  return TT_OK;
}

}  // namespace

bool make_tmap_2d_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                     uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer) {
  return make_tmap_2d_type(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, inner, outer, row_bytes,
                           box_inner, box_outer);
}

size_t q8_workspace_bytes(const tt_dims& d, int which) {
  if (which == TT_WS_VOCAB_I8) return carve_vocab(d, nullptr).total;
  if (which == TT_WS_ATTN_Q8) return carve_attn(d, attn_shape(d), nullptr).total;
  return kCtrlBytes;
}

}  // namespace tt

using namespace tt;

extern "C" {

tt_status tt_block_denoise_attn_q8(const tt_dims* d, const tt_q8* f, const tt_bf16* q_blk,
                                   const tt_bf16* k_blk, const tt_bf16* v_blk, const void* k_ctx,
                                   const void* v_ctx, const float* k_scale, const float* v_scale,
                                   const int32_t* ctx_len, tt_bf16* out, void* ws,
                                   size_t ws_bytes, void* stream) {
  Q8_CHECK(check_cache(d, f));
  Q8_CHECK(check_ptr(q_blk, "q_blk", 16));
  Q8_CHECK(check_ptr(k_blk, "k_blk", 16));
  Q8_CHECK(check_ptr(v_blk, "v_blk", 16));
  if (d->L_cap > 0) {  // without room for a context there is no cache to point to
    Q8_CHECK(check_ptr(k_ctx, "k_ctx", 16));
    Q8_CHECK(check_ptr(v_ctx, "v_ctx", 16));
    Q8_CHECK(check_ptr(k_scale, "k_scale", 4));
    Q8_CHECK(check_ptr(v_scale, "v_scale", 4));
  }
  Q8_CHECK(check_ptr(ctx_len, "ctx_len", 4));
  Q8_CHECK(check_ptr(out, "out", 16));
  const AttnShape g = attn_shape(*d);
  if ((long long)d->B * d->Hkv * g.n_qtiles * (1ll + (d->L_cap + kAttnBN - 1) / kAttnBN) >=
      (1ll << 31) - 2048)
    return set_errorf(TT_ERR_UNSUPPORTED, "problem too large");
  const AttnQ8Ws w = carve_attn(*d, g, ws);
  Q8_CHECK(check_ws_ptr(ws, ws_bytes, w.total));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  AttnQ8Args a{};
  a.B = d->B;
  a.S = d->S;
  a.Hq = d->Hq;
  a.Hkv = d->Hkv;
  a.dh = d->dh;
  a.G = d->Hq / d->Hkv;
  a.L_cap = d->L_cap;
  a.block_shift = block_shift(*f);
  a.n_blocks = (d->L_cap + f->block - 1) / f->block;
  a.q = q_blk;
  a.k_blk = k_blk;
  a.v_blk = v_blk;
  a.k_ctx = static_cast<const uint8_t*>(k_ctx);
  a.v_ctx = static_cast<const uint8_t*>(v_ctx);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.ctx_len = ctx_len;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d->dh));
  a.out = out;
  a.s_per_half = g.s_per_half;
  while ((1 << a.g_shift) < g.G) ++a.g_shift;
  a.rows_per_half = g.rows_per_half;
  a.halves = g.halves;
  a.n_qtiles = g.n_qtiles;
  a.units = g.units;
  a.n_ctas = g.n_ctas;
  a.unit_span = w.unit_span;
  a.part_o = w.part_o;
  a.part_lse = w.part_lse;
  a.err = w.ctrl;
  if (d->S * g.G <= kRowsMax) {
    Q8_LAUNCH(TT_K_ATTN_Q8, st, launch_attn_q8_rows(a, f->type, st));
    Q8_LAUNCH(TT_K_MERGE_Q8, st, launch_attn_q8_rows_merge(a, st));
  } else {
    Q8_LAUNCH(TT_K_ATTN_Q8, st, launch_attn_q8(a, f->type, st));
    Q8_LAUNCH(TT_K_MERGE_Q8, st, launch_attn_q8_merge(a, st));
  }
  return TT_OK;
}

tt_status tt_append_ctx_q8(const tt_dims* d, const tt_q8* f, int32_t n, const int32_t* new_len,
                           const tt_bf16* k_new, const tt_bf16* v_new,
                           const tt_row_strides* strides, void* k_ctx, void* v_ctx,
                           float* k_scale, float* v_scale, int32_t* ctx_len, void* ws,
                           size_t ws_bytes, void* stream) {
  Q8_CHECK(check_cache(d, f));
  if (n < 1 || n > d->L_cap)
    return set_errorf(TT_ERR_INVALID_ARG, "n=%d not in [1, L_cap=%d]", n, d->L_cap);
  if (strides == nullptr) return set_errorf(TT_ERR_INVALID_ARG, "strides is NULL");
  if (((strides->batch | strides->token | strides->head) & 7) != 0)
    return set_errorf(TT_ERR_INVALID_ARG, "strides must be multiples of 8 elements");
  if (new_len != nullptr) Q8_CHECK(check_ptr(new_len, "new_len", 4));
  Q8_CHECK(check_ptr(k_new, "k_new", 16));
  Q8_CHECK(check_ptr(v_new, "v_new", 16));
  Q8_CHECK(check_ptr(k_ctx, "k_ctx", 16));
  Q8_CHECK(check_ptr(v_ctx, "v_ctx", 16));
  Q8_CHECK(check_ptr(k_scale, "k_scale", 4));
  Q8_CHECK(check_ptr(v_scale, "v_scale", 4));
  Q8_CHECK(check_ptr(ctx_len, "ctx_len", 4));
  Q8_CHECK(check_ws_ptr(ws, ws_bytes, q8_workspace_bytes(*d, TT_WS_APPEND_Q8)));
  if (2ll * d->Hkv * d->B >= (1ll << 31))
    return set_errorf(TT_ERR_UNSUPPORTED, "problem too large");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  AppendQ8Args a{};
  a.B = d->B;
  a.Hkv = d->Hkv;
  a.dh = d->dh;
  a.L_cap = d->L_cap;
  a.n = n;
  a.block_shift = block_shift(*f);
  a.n_blocks = (d->L_cap + f->block - 1) / f->block;
  a.new_len = new_len;
  a.k_new = k_new;
  a.v_new = v_new;
  a.stride_b = strides->batch;
  a.stride_t = strides->token;
  a.stride_h = strides->head;
  a.k_ctx = static_cast<uint8_t*>(k_ctx);
  a.v_ctx = static_cast<uint8_t*>(v_ctx);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.ctx_len = ctx_len;
  a.err = static_cast<int*>(ws);
  Q8_LAUNCH(TT_K_APPEND_Q8, st, launch_append_q8(a, f->type, st));
  Q8_LAUNCH(TT_K_APPEND_Q8, st, launch_append_q8_len(a, st));
  return TT_OK;
}

tt_status tt_quantize_rows_i8(int32_t rows, int32_t K, const tt_bf16* x, int8_t* q, float* scale,
                              void* stream) {
  Q8_CHECK(check_rows_k(rows, K));
  Q8_CHECK(check_ptr(x, "x", 16));
  Q8_CHECK(check_ptr(q, "q", 16));
  Q8_CHECK(check_ptr(scale, "scale", 4));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Q8_LAUNCH(TT_K_QUANT_I8, st, launch_quant_rows(x, K, q, scale, nullptr, nullptr, rows, nullptr, st));
  return TT_OK;
}

size_t tt_linear_i8_workspace_bytes(int32_t rows, int32_t N, int32_t K) {
  if (check_linear(rows, N, K) != TT_OK) return 0;
  return carve_linear(rows, K, nullptr).total;
}

tt_status tt_linear_i8(int32_t rows, int32_t N, int32_t K, const tt_bf16* x, const int8_t* w_q,
                       const float* w_scale, tt_bf16* out, void* ws, size_t ws_bytes,
                       void* stream) {
  Q8_CHECK(check_linear(rows, N, K));
  Q8_CHECK(check_ptr(x, "x", 16));
  Q8_CHECK(check_ptr(w_q, "w_q", 16));
  Q8_CHECK(check_ptr(w_scale, "w_scale", 16));
  Q8_CHECK(check_ptr(out, "out", 16));
  const LinearWs w = carve_linear(rows, K, ws);
  Q8_CHECK(check_ws_ptr(ws, ws_bytes, w.total));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const I8Shape sh = i8_shape(rows, N, K);
  const bool pair = sh.splits == 0 && i8_pair(rows);
  CUtensorMap tmA, tmB;
  const int a_box = std::min(rows, kI8BM);
  if (!make_tmap_2d_u8(&tmA, w.xq, K, rows, K, kI8BK, a_box) ||
      !make_tmap_2d_u8(&tmB, w_q, K, N, K, kI8BK, pair ? sh.bn / 2 : sh.bn))
    return set_errorf(TT_ERR_CUDA, "cuTensorMapEncodeTiled failed for the 8-bit linear update");
  GemmI8Args a{};
  a.M_alloc = rows;
  a.a_box = a_box;
  a.N = N;
  a.K = K;
  a.a_scale = w.xs;
  a.b_scale = w_scale;
  a.C = out;
  a.err = w.ctrl;
  Q8_LAUNCH(TT_K_QUANT_I8, st,
            launch_quant_rows(x, K, w.xq, w.xs, nullptr, nullptr, rows, w.ctrl, st));
  if (sh.splits) {
    Q8_LAUNCH(TT_K_GEMM_I8, st, launch_gemm_i8_split(tmA, tmB, a, sh.bn, sh.splits, st));
  } else {
    const long long bm = pair ? 2 * kI8BM : kI8BM;
    const long long tiles = ((rows + bm - 1) / bm) * ((N + kI8BN - 1ll) / kI8BN);
    const int grid = (int)std::min<long long>(tiles, pair ? num_sms() / 2 : num_sms());
    Q8_LAUNCH(TT_K_GEMM_I8, st, launch_gemm_i8_linear(tmA, tmB, a, pair, grid, st));
  }
  return TT_OK;
}

tt_status tt_vocab_confidence_commit_i8(const tt_dims* d, const tt_bf16* y, const int8_t* w_q,
                                        const float* w_scale, float gamma, float logit_scale,
                                        int32_t* tokens, uint8_t* masked, float* conf_out,
                                        int32_t* argmax_out, int32_t* n_committed, void* ws,
                                        size_t ws_bytes, void* stream) {
  Q8_CHECK(check_vocab_args(d, y, reinterpret_cast<const tt_bf16*>(w_q), gamma, logit_scale,
                            tokens, masked));
  Q8_CHECK(check_ptr(w_scale, "w_scale", 16));
  const VocabWs w = carve_vocab(*d, ws);
  Q8_CHECK(check_ws_ptr(ws, ws_bytes, w.total));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int rows = d->B * d->S;
  const int* M_dev = w.ctrl + CTRL_M;
  CUtensorMap tmA, tmB;
  const int a_box = std::min(rows, kI8BM);
  if (!make_tmap_2d_u8(&tmA, w.yq, d->H, rows, d->H, kI8BK, a_box) ||
      !make_tmap_2d_u8(&tmB, w_q, d->H, d->V, d->H, kI8BK, kI8VocabBN))
    return set_errorf(TT_ERR_CUDA, "cuTensorMapEncodeTiled failed for the 8-bit vocabulary GEMM");
  // Each row counts the masked rows before it; beyond some thousands of rows
  // (32 MB of flags read for 8192) a plan does it once instead.
  if (rows <= 8192) {
    Q8_LAUNCH(TT_K_QUANT_I8, st,
              launch_masked_rows(y, d->H, w.yq, w.ys, masked, rows, d->S, w.rowlist, w.ctrl,
                                 w.seqcnt, st));
  } else {
    Q8_CUDA(cudaMemsetAsync(w.ctrl, 0, w.clear, st));
    PlanArgs p{d->B, d->S, masked, w.rowlist, w.tvec, w.ctrl, 0};
    Q8_LAUNCH(TT_K_PLAN, st, launch_plan(p, st));
    Q8_LAUNCH(TT_K_QUANT_I8, st,
              launch_quant_rows(y, d->H, w.yq, w.ys, w.rowlist, M_dev, rows, nullptr, st));
  }
  GemmI8Args a{};
  a.M_alloc = rows;
  a.a_box = a_box;
  a.M_dev = M_dev;
  a.N = d->V;
  a.K = d->H;
  a.a_scale = w.ys;
  a.b_scale = w_scale;
  a.stats = w.stats;
  a.scale_log2 = (float)(logit_scale * 1.4426950408889634);
  a.err = w.ctrl;
  const int n_vt = (d->V + kI8VocabBN - 1) / kI8VocabBN;
  const long long tiles = ((rows + kI8BM - 1ll) / kI8BM) * n_vt;
  Q8_LAUNCH(TT_K_GEMM_VOCAB_I8, st,
            launch_gemm_i8_vocab(tmA, tmB, a, (int)std::min<long long>(tiles, num_sms()), st));
  CommitArgs c{};
  c.B = d->B;
  c.S = d->S;
  c.n_vt = n_vt;
  c.stats = w.stats;
  c.row_scale = w.ys;
  c.scale_log2 = a.scale_log2;
  c.gamma = gamma;
  c.rowlist = w.rowlist;
  c.rowres = w.rowres;
  c.seqcnt = w.seqcnt;
  c.M_dev = M_dev;
  c.tokens = tokens;
  c.masked = masked;
  c.ctrl = w.ctrl;
  c.conf_out = conf_out;
  c.argmax_out = argmax_out;
  c.n_committed = n_committed;
  Q8_LAUNCH(TT_K_COMMIT, st, launch_commit(c, st));
  return TT_OK;
}

}  // extern "C"
