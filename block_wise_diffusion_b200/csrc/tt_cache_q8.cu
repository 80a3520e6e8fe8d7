// Writers of 8-bit data: rows joining an 8-bit context cache, and rows
// quantised one by one for the integer products.  Both read each bf16 value
// once (a group stays in registers between its maximum and its rounding) and
// are bound by HBM: 2 bytes in and 1 byte out per value.
#include "tt_q8.h"
#include "tt_quant.cuh"

namespace tt {

namespace {

constexpr int kAppendThreads = 256;

// How many rows sequence b gets, or -1 when its lengths are out of range.
__device__ __forceinline__ int append_rows(const AppendQ8Args& a, int b, int L) {
  const int m = a.new_len != nullptr ? a.new_len[b] : a.n;
  return (m < 0 || m > a.n || L < 0 || L > a.L_cap - m) ? -1 : m;
}

// CTA (b, g, K or V, i), i fastest: the i-th cache block that sequence b's new
// rows may touch, counted from the block that holds its end.  A thread holds vectors
// of 8 values (at most 8: a block has at most 128 x 128 values).
template <int TYPE>
__global__ void __launch_bounds__(kAppendThreads) append_q8_kernel(const AppendQ8Args a) {
  griddep_launch();
  griddep_wait();
  __shared__ uint32_t red[kAppendThreads / 32];
  const int nb = (a.n + a.block - 1) / a.block + 1;
  const int pair = blockIdx.x / nb, bi = blockIdx.x - pair * nb;
  const int is_v = pair & 1, b = (pair >> 1) / a.Hkv, g = (pair >> 1) - b * a.Hkv;
  const int L = a.ctx_len[b];
  const int m = append_rows(a, b, L);
  if (m < 0) {
    if (threadIdx.x == 0 && bi == 0 && g == 0 && is_v == 0)
      atomicCAS(a.err, 0, (int)TT_ERR_INVALID_ARG);
    return;
  }
  const int blk = L / a.block + bi;
  const long long p0 = (long long)blk * a.block;  // first position of the block
  if (m == 0 || p0 >= (long long)L + m) return;
  const int n_old = max(0, (int)(L - p0));         // older rows in the block
  const int n_end = (int)min((long long)a.block, L + m - p0);
  const int dv = a.dh >> 3;                        // vectors per row
  const int lo = n_old * dv, hi = n_end * dv;      // new vectors of the block
  const uint16_t* src = (is_v ? a.v_new : a.k_new) + (long long)b * a.stride_b +
                        (long long)g * a.stride_h + (p0 - L) * a.stride_t;
  uint8_t* dst = (is_v ? a.v_ctx : a.k_ctx) + ((long long)(b * a.Hkv + g) * a.L_cap + p0) * a.dh;
  float* sp = (is_v ? a.v_scale : a.k_scale) + (long long)(b * a.Hkv + g) * a.n_blocks + blk;

  uint4 x[8];
  uint32_t mx = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = lo + k * kAppendThreads + threadIdx.x;
    if (i < hi) {
      const int t = i / dv;
      x[k] = *reinterpret_cast<const uint4*>(src + (long long)t * a.stride_t + (i - t * dv) * 8);
      mx = absmax8(mx, x[k]);
    }
  }
  mx = __reduce_max_sync(0xffffffffu, absmax_fold(mx));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
  __syncthreads();
  mx = 0;
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) mx = max(mx, red[w]);
  float s = q8_scale<TYPE>(mx);
  if (n_old > 0) {
    const float s_old = *sp;
    __syncthreads();  // every thread has read the scale before it is written
    if (s_old >= s || s_old != s_old) {
      s = s_old;  // NaN stays NaN
    } else if (s != s_old) {
      // the older rows of the block under the larger (or NaN) scale
      for (int i = threadIdx.x; i < n_old * a.dh / 4; i += kAppendThreads) {
        uint32_t w = reinterpret_cast<uint32_t*>(dst)[i], r = 0;
        if (s == s) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) r |= q8_recode<TYPE>((w >> e) & 255u, s_old, s) << e;
        }
        reinterpret_cast<uint32_t*>(dst)[i] = r;
      }
    }
  }
  const float inv = 1.f / s;
  const bool ok = s == s;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = lo + k * kAppendThreads + threadIdx.x;
    if (i < hi)
      *reinterpret_cast<uint2*>(dst + (long long)i * 8) =
          ok ? q8_pack8<TYPE>(x[k], s, inv) : make_uint2(0, 0);
  }
  if (threadIdx.x == 0) *sp = s;
}

// ctx_len[b] += rows appended, after every block of the sequence is written.
__global__ void __launch_bounds__(256) append_len_kernel(const AppendQ8Args a) {
  griddep_launch();
  griddep_wait();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= a.B) return;
  const int L = a.ctx_len[b];
  const int m = append_rows(a, b, L);
  if (m > 0) a.ctx_len[b] = L + m;
}

// Row r of x (row rowlist[r] of it with a row list) to int8 codes and a
// scale.  One CTA per row; a row of up to 8192 values stays in registers, a
// longer one is read again (from L2).
constexpr int kQuantThreads = 256, kQuantVec = 4;
__global__ void __launch_bounds__(kQuantThreads)
    quant_rows_kernel(const uint16_t* __restrict__ x, int K, int8_t* __restrict__ q,
                      float* __restrict__ scale, const int* __restrict__ rowlist,
                      const int* __restrict__ M_dev, int rows) {
  griddep_launch();
  griddep_wait();
  __shared__ uint32_t red[kQuantThreads / 32];
  const int r = blockIdx.x;
  if (M_dev != nullptr && r >= min(*M_dev, rows)) return;
  const int nv = K >> 3;
  const uint4* src =
      reinterpret_cast<const uint4*>(x + (long long)(rowlist != nullptr ? rowlist[r] : r) * K);
  uint2* dst = reinterpret_cast<uint2*>(q + (long long)r * K);
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
  const bool ok = s == s;
#pragma unroll
  for (int k = 0; k < kQuantVec; ++k) {
    const int i = k * kQuantThreads + threadIdx.x;
    if (i < nv) dst[i] = ok ? q8_pack8<TT_Q8_INT8>(v[k], s, inv) : make_uint2(0, 0);
  }
  for (int i = kQuantVec * kQuantThreads + threadIdx.x; i < nv; i += kQuantThreads)
    dst[i] = ok ? q8_pack8<TT_Q8_INT8>(src[i], s, inv) : make_uint2(0, 0);
  if (threadIdx.x == 0) scale[r] = s;
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Args& a, int type, cudaStream_t st) {
  const dim3 grid((unsigned)(((a.n + a.block - 1) / a.block + 1) * 2ll * a.Hkv * a.B));
  cudaError_t e = type == TT_Q8_INT8
                      ? launch_k(append_q8_kernel<TT_Q8_INT8>, grid, dim3(kAppendThreads), 0, st, a)
                      : launch_k(append_q8_kernel<TT_Q8_E4M3>, grid, dim3(kAppendThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  return launch_k(append_len_kernel, dim3((a.B + 255) / 256), dim3(256), 0, st, a);
}

cudaError_t launch_quant_rows(const uint16_t* x, int K, int8_t* q, float* scale,
                              const int* rowlist, const int* M_dev, int rows, cudaStream_t st) {
  return launch_k(quant_rows_kernel, dim3(rows), dim3(kQuantThreads), 0, st, x, K, q, scale,
                  rowlist, M_dev, rows);
}

}  // namespace tt
