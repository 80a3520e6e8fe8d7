// Writers of 8-bit data: rows joining an 8-bit context cache, and rows
// quantised one by one for the integer products.  Both read each bf16 value
// once (a group stays in registers between its maximum and its rounding): 2
// bytes in and 1 byte out per value, all that HBM has to carry.  16 prompts of up to
// 8192 tokens, 2 KV heads of dh 128, blocks of 64, take 36 us as e4m3 (4.1 TB/s): the
// schedulers issue in 78 % of the cycles (ALU 56 %, DRAM 45 %), so instructions bound
// it, with the loads' latency behind them.  16 rows onto each of 64 sequences take 6.5
// us, most of it the two launches, where the blocks' scales stay, and 16 where they
// grow: the older rows are then rounded again by 64-bit quotients.
#include <algorithm>

#include "tt_q8.h"
#include "tt_quant.cuh"

namespace tt {

namespace {

// A thread holds kVec vectors of 8 values of one cache block, so a block of
// block * dh values takes 32 (16 x 64) to 512 (128 x 128) threads.  A CTA has at
// least 128 threads, several blocks side by side where they are small.  (With
// 8 vectors: 40 us against 36 for 16 prompts of up to 8192 tokens; with 2: 60.)
constexpr int kVec = 4;

// How many rows sequence b gets, or -1 when its lengths are out of range.
__device__ __forceinline__ int append_rows(const AppendQ8Args& a, int b, int L) {
  const int m = a.new_len != nullptr ? a.new_len[b] : a.n;
  return (m < 0 || m > a.n || L < 0 || L > a.L_cap - m) ? -1 : m;
}

// CTA (x, y): pair x of (b, g, K or V), and of the groups of cache blocks that
// sequence b's new rows may touch, counted from the block that holds its end,
// y, y + gridDim.y, ..., so that neighbouring CTAs read neighbouring columns of
// the same rows.  NT: threads of a block.
template <int TYPE, int NT>
__global__ void __launch_bounds__(NT < 128 ? 128 : NT, NT == 512 ? 2 : NT == 256 ? 5 : 10) append_q8_kernel(const AppendQ8Args a) {
  constexpr int kCta = NT < 128 ? 128 : NT;
  griddep_launch();
  griddep_wait();
  __shared__ uint32_t red[kCta / 32];
  const int tid = threadIdx.x % NT;
  const int pair = blockIdx.x, is_v = pair & 1, b = (pair >> 1) / a.Hkv;
  const int g = (pair >> 1) - b * a.Hkv;
  const int L = a.ctx_len[b], m = append_rows(a, b, L);
  for (int group = blockIdx.y; group < a.groups; group += gridDim.y) {
    const int bi = group * (kCta / NT) + threadIdx.x / NT;
    const int blk = (max(L, 0) >> a.block_shift) + bi;
    const long long p0 = (long long)blk << a.block_shift;  // first position of the block
    const bool mine = m > 0 && p0 < (long long)L + m;
    if (kCta == NT && !mine) continue;
    const int n_old = mine ? max(0, (int)(L - p0)) : 0;  // older rows in the block
    const int n_end = mine ? (int)min(1ll << a.block_shift, L + m - p0) : 0;
    // A thread's vectors: one column of 8 values, rows row0, row0 + step, .. of the
    // block, of which n_old .. n_end - 1 are new.
    const int dv_log = a.dh == 64 ? 3 : 4, step = NT >> dv_log;
    const int row0 = tid >> dv_log, col = tid & ((1 << dv_log) - 1);
    const uint16_t* src = (is_v ? a.v_new : a.k_new) + (long long)b * a.stride_b +
                          (long long)g * a.stride_h + (p0 - L + row0) * a.stride_t + col * 8;
    const long long src_step = (long long)step * a.stride_t;
    uint4 x[kVec];
    uint32_t mx = 0;
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const int row = row0 + k * step;
      x[k] = make_uint4(0, 0, 0, 0);
      if (row >= n_old && row < n_end) x[k] = *reinterpret_cast<const uint4*>(src);
      src += src_step;
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k) mx = absmax8(mx, x[k]);
    mx = __reduce_max_sync(0xffffffffu, absmax_fold(mx));
    if constexpr (NT > 32) {
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
      __syncthreads();
      const int w0 = threadIdx.x / NT * (NT / 32);
      mx = red[w0];
#pragma unroll
      for (int w = 1; w < NT / 32; ++w) mx = max(mx, red[w0 + w]);
    }
    uint8_t* dst = (is_v ? a.v_ctx : a.k_ctx) + ((long long)(b * a.Hkv + g) * a.L_cap + p0) * a.dh;
    float* sp = (is_v ? a.v_scale : a.k_scale) + (long long)(b * a.Hkv + g) * a.n_blocks + blk;
    const float s_own = q8_scale<TYPE>(mx);
    float s = s_own, s_old = s;
    if (n_old > 0) s_old = *sp;
    // every thread has read the scale before it is written, and `red` before the
    // next group
    if constexpr (NT > 32)
      __syncthreads();
    else
      __syncwarp();
    if (!mine) continue;
    if (s_old >= s || s_old != s_old) {
      s = s_old;  // NaN stays NaN
    } else if (s != s_old) {
      // the older rows of the block under the larger (or NaN) scale
      for (int i = tid; i < n_old * a.dh / 4; i += NT) {
        uint32_t w = reinterpret_cast<uint32_t*>(dst)[i], r = 0;
        if (s == s) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) r |= q8_recode<TYPE>((w >> e) & 255u, s_old, s) << e;
        }
        reinterpret_cast<uint32_t*>(dst)[i] = r;
      }
    }
    const float own = s == s_own ? q8_own_factor<TYPE>(mx, s) : 0.f;
    if (own != 0.f) {
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        const int row = row0 + k * step;
        if (row >= n_old && row < n_end)
          *reinterpret_cast<uint2*>(dst + (k * NT + tid) * 8) = q8_pack8_own<TYPE>(x[k], own);
      }
    } else {
      const float inv = 1.f / s;
      const bool ok = s == s;
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        const int row = row0 + k * step;
        if (row >= n_old && row < n_end)
          *reinterpret_cast<uint2*>(dst + (k * NT + tid) * 8) =
              ok ? q8_pack8<TYPE>(x[k], s, inv) : make_uint2(0, 0);
      }
    }
    if (tid == 0) *sp = s;
  }
}

// After every block is written: ctx_len[b] += rows appended, and the error
// word (one CTA: it reports for all sequences).
__global__ void __launch_bounds__(256) append_len_kernel(const AppendQ8Args a) {
  griddep_launch();
  griddep_wait();
  int bad = 0;
  for (int b = threadIdx.x; b < a.B; b += 256) {
    const int L = a.ctx_len[b];
    const int m = append_rows(a, b, L);
    bad |= m < 0;
    if (m > 0) a.ctx_len[b] = L + m;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    a.err[0] = bad ? (int)TT_ERR_INVALID_ARG : 0;
    a.err[1] = 0;
  }
}

// A row of K values to int8 codes and a scale, by the whole CTA.  A row of up
// to 8192 values stays in registers, a longer one is read again (from L2).
constexpr int kQuantThreads = 256, kQuantVec = 4;
__device__ __forceinline__ void quant_row(const uint4* __restrict__ src, int K,
                                          uint2* __restrict__ dst, float* __restrict__ scale) {
  __shared__ uint32_t red[kQuantThreads / 32];
  const int nv = K >> 3;
  uint4 v[kQuantVec];
  uint32_t mx = 0;
#pragma unroll
  for (int k = 0; k < kQuantVec; ++k) {
    const int i = k * kQuantThreads + threadIdx.x;
    if (i < nv) {
      v[k] = src[i];
      mx = absmax8(mx, v[k]);
    }
  }
  for (int i = kQuantVec * kQuantThreads + threadIdx.x; i < nv; i += kQuantThreads)
    mx = absmax8(mx, src[i]);
  mx = __reduce_max_sync(0xffffffffu, absmax_fold(mx));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
  __syncthreads();
  mx = 0;
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) mx = max(mx, red[w]);
  const float s = q8_scale<TT_Q8_INT8>(mx), inv = 1.f / s;
  const float own = q8_own_factor<TT_Q8_INT8>(mx, s);
  const bool ok = s == s;
  auto codes = [&](const uint4& x) {
    return own != 0.f ? q8_pack8_own<TT_Q8_INT8>(x, own)
           : ok       ? q8_pack8<TT_Q8_INT8>(x, s, inv)
                      : make_uint2(0, 0);
  };
#pragma unroll
  for (int k = 0; k < kQuantVec; ++k) {
    const int i = k * kQuantThreads + threadIdx.x;
    if (i < nv) dst[i] = codes(v[k]);
  }
  for (int i = kQuantVec * kQuantThreads + threadIdx.x; i < nv; i += kQuantThreads)
    dst[i] = codes(src[i]);
  if (threadIdx.x == 0) *scale = s;
}

// CTA r: row r of x (row rowlist[r] of it with a row list, *M_dev rows).
// These kernels wait before they let their dependent start: what that reads
// before its own wait (weights) is complete then.
__global__ void __launch_bounds__(kQuantThreads)
    quant_rows_kernel(const uint16_t* __restrict__ x, int K, int8_t* __restrict__ q,
                      float* __restrict__ scale, const int* __restrict__ rowlist,
                      const int* __restrict__ M_dev, int rows, int* err) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x;
  if (err != nullptr && r == 0 && threadIdx.x < 2) err[threadIdx.x] = 0;
  if (M_dev != nullptr && r >= min(*M_dev, rows)) return;
  quant_row(reinterpret_cast<const uint4*>(x + (long long)(rowlist != nullptr ? rowlist[r] : r) * K),
            K, reinterpret_cast<uint2*>(q + (long long)r * K), scale + r);
}

// The vocabulary step's rows without a planning launch: CTA r finds the place of
// its masked row among the masked rows by counting those before it, and
// quantises it there.  Also what a plan would leave: the row lists, the row
// count (the last CTA), cleared error words and commit counters.
__global__ void __launch_bounds__(kQuantThreads)
    masked_rows_kernel(const uint16_t* __restrict__ x, int K, int8_t* __restrict__ q,
                       float* __restrict__ scale, const uint8_t* __restrict__ masked, int rows,
                       int S, int* __restrict__ rowlist, int* __restrict__ ctrl,
                       int* __restrict__ seqcnt) {
  griddep_wait();
  griddep_launch();
  const int r = blockIdx.x;
  if (r == 0 && threadIdx.x < 2) ctrl[threadIdx.x] = 0;
  if (threadIdx.x == 0 && r % S == 0) seqcnt[r / S] = 0;
  const int mine = masked[r] != 0;
  if (!mine && r != rows - 1) return;
  int j = 0;
  for (int i0 = 0; i0 < r; i0 += kQuantThreads) {
    const int i = i0 + threadIdx.x;
    j += __syncthreads_count(i < r && masked[i] != 0);
  }
  if (threadIdx.x == 0) {
    if (r == rows - 1) ctrl[CTRL_M] = j + mine;
    if (mine) {
      rowlist[j] = r;
      rowlist[rows + r] = j;
    }
  }
  if (mine)
    quant_row(reinterpret_cast<const uint4*>(x + (long long)r * K), K,
              reinterpret_cast<uint2*>(q + (long long)j * K), scale + j);
}

}  // namespace

template <int TYPE, int NT>
static cudaError_t launch_append(const AppendQ8Args& a, cudaStream_t st) {
  constexpr int kCta = NT < 128 ? 128 : NT, kPer = kCta / NT;
  const int nb = ((a.n - 1) >> a.block_shift) + 2;  // blocks n rows may touch
  AppendQ8Args args = a;
  args.groups = (nb + kPer - 1) / kPer;
  const dim3 grid((unsigned)(2 * a.Hkv * a.B), (unsigned)std::min(args.groups, 65535));
  return launch_k(append_q8_kernel<TYPE, NT>, grid, dim3(kCta), 0, st, args);
}
template <int TYPE>
static cudaError_t launch_append_type(const AppendQ8Args& a, cudaStream_t st) {
  switch ((a.dh << a.block_shift) / (8 * kVec)) {
    case 32: return launch_append<TYPE, 32>(a, st);
    case 64: return launch_append<TYPE, 64>(a, st);
    case 128: return launch_append<TYPE, 128>(a, st);
    case 256: return launch_append<TYPE, 256>(a, st);
    default: return launch_append<TYPE, 512>(a, st);
  }
}

cudaError_t launch_append_q8(const AppendQ8Args& a, int type, cudaStream_t st) {
  return type == TT_Q8_INT8 ? launch_append_type<TT_Q8_INT8>(a, st)
                            : launch_append_type<TT_Q8_E4M3>(a, st);
}
cudaError_t launch_append_q8_len(const AppendQ8Args& a, cudaStream_t st) {
  return launch_k(append_len_kernel, dim3(1), dim3(256), 0, st, a);
}

cudaError_t launch_quant_rows(const uint16_t* x, int K, int8_t* q, float* scale,
                              const int* rowlist, const int* M_dev, int rows, int* err,
                              cudaStream_t st) {
  return launch_k(quant_rows_kernel, dim3(rows), dim3(kQuantThreads), 0, st, x, K, q, scale,
                  rowlist, M_dev, rows, err);
}

cudaError_t launch_masked_rows(const uint16_t* x, int K, int8_t* q, float* scale,
                               const uint8_t* masked, int rows, int S, int* rowlist, int* ctrl,
                               int* seqcnt, cudaStream_t st) {
  return launch_k(masked_rows_kernel, dim3(rows), dim3(kQuantThreads), 0, st, x, K, q, scale,
                  masked, rows, S, rowlist, ctrl, seqcnt);
}

}  // namespace tt
