// Block-denoise attention over an 8-bit context cache, plain form: one CTA
// per (sequence, KV head, 16 query rows) walks the keys 32 at a time with a
// running maximum and sum in fp32.
#include <cuda_fp16.h>
#include <math.h>

#include "tt_q8.h"
#include "tt_ptx.cuh"

namespace tt {

namespace {

constexpr int kRows = 16, kKeys = 32, kThreads = 128;

__device__ __forceinline__ float code_value(int type, uint8_t b) {
  if (type == TT_Q8_INT8) return (float)(int8_t)b;
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)b));
  return __half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu)));
}

__global__ void __launch_bounds__(kThreads) attn_q8_kernel(const AttnQ8Args a, int type) {
  griddep_launch();
  griddep_wait();
  __shared__ float sq[kRows][129], sk[kKeys][129], sv[kKeys][129], sp[kRows][kKeys + 1];
  const int nrt = (a.S * a.G + kRows - 1) / kRows;
  const int pair = blockIdx.x / nrt, rt = blockIdx.x - pair * nrt;
  const int b = pair / a.Hkv, g = pair - b * a.Hkv;
  int L = a.ctx_len[b];
  if (L < 0 || L > a.L_cap) {
    if (threadIdx.x == 0) atomicCAS(a.err, 0, (int)TT_ERR_INVALID_ARG);
    L = min(max(L, 0), a.L_cap);
  }
  const int dh = a.dh, nrows = a.S * a.G;
  for (int i = threadIdx.x; i < kRows * dh; i += kThreads) {
    const int r = rt * kRows + i / dh, e = i % dh;
    const int s = r / a.G, h = g * a.G + r % a.G;
    sq[i / dh][e] =
        r < nrows ? bf16_value(a.q[((long long)(b * a.S + s) * a.Hq + h) * dh + e]) : 0.f;
  }
  // thread = (row, every 8th column): 8 threads share a row
  const int row = threadIdx.x >> 3, c8 = threadIdx.x & 7;
  float o[16], m = -INFINITY, l = 0.f;
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  const long long crow = (long long)(b * a.Hkv + g) * a.L_cap;
  for (int k0 = 0; k0 < a.S + L; k0 += kKeys) {
    __syncthreads();
    for (int i = threadIdx.x; i < kKeys * dh; i += kThreads) {
      const int j = k0 + i / dh, e = i % dh;
      float kv = 0.f, vv = 0.f;
      if (j < a.S) {
        const long long at = ((long long)(b * a.S + j) * a.Hkv + g) * dh + e;
        kv = bf16_value(a.k_blk[at]);
        vv = bf16_value(a.v_blk[at]);
      } else if (j < a.S + L) {
        const int p = j - a.S;
        const long long at = (crow + p) * dh + e;
        const long long sb = (long long)(b * a.Hkv + g) * a.n_blocks + p / a.block;
        kv = code_value(type, a.k_ctx[at]) * a.k_scale[sb];
        vv = code_value(type, a.v_ctx[at]) * a.v_scale[sb];
      }
      sk[i / dh][e] = kv;
      sv[i / dh][e] = vv;
    }
    __syncthreads();
    for (int j = c8; j < kKeys; j += 8) {
      float s = -INFINITY;
      if (k0 + j < a.S + L) {
        s = 0.f;
        for (int e = 0; e < dh; ++e) s = fmaf(sq[row][e], sk[j][e], s);
        s *= a.scale_log2;
      }
      sp[row][j] = s;
    }
    __syncwarp();
    float mn = m;
    for (int j = 0; j < kKeys; ++j) mn = fmaxf(mn, sp[row][j]);
    const float alpha = ex2(m - mn);
    m = mn;
    l *= alpha;
    for (int i = 0; i < 16; ++i) o[i] *= alpha;
    for (int j = 0; j < kKeys; ++j) {
      const float p = ex2(sp[row][j] - m);
      l += p;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i * 8 < dh) o[i] = fmaf(p, sv[j][i * 8 + c8], o[i]);
    }
  }
  const int r = rt * kRows + row;
  if (r >= nrows) return;
  const int s = r / a.G, h = g * a.G + r % a.G;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i * 8 < dh)
      a.out[((long long)(b * a.S + s) * a.Hq + h) * dh + i * 8 + c8] = bf16_bits(o[i] / l);
}

}  // namespace

cudaError_t launch_attn_q8(const AttnQ8Args& a, int type, cudaStream_t st) {
  const int nrt = (a.S * a.G + kRows - 1) / kRows;
  return launch_k(attn_q8_kernel, dim3(a.B * a.Hkv * nrt), dim3(kThreads), 0, st, a, type);
}

}  // namespace tt
