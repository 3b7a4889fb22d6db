// kv_attention.cu -- causal attention of new tokens over the paged 8-bit
// cache:  o = softmax(scale q K^T) V  with K = s_K[page, head] * code and V
// likewise; row i of a request with n new and m cached tokens (the new ones
// included) sees the cached positions 0 .. m - n + i.
#include "kernels.h"
#include "ptx.cuh"

namespace bsk {

constexpr int kAttnThreads = 128;

__device__ __forceinline__ float e4m3_val(uint32_t c) { return e4m3_to_f32(c); }

// One CTA per (row, query head): a thread scores one token of a chunk of 128,
// then owns one output element.
template <int D>
__global__ void __launch_bounds__(kAttnThreads) kv_attention_kernel(const __grid_constant__ KvAttentionParams p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float qs[D], ps[kAttnThreads], red[kAttnThreads / 32];
  const int row = blockIdx.x, hq = blockIdx.y, tid = threadIdx.x;
  const int h = hq / (p.Hq / p.Hkv);
  // the request of this row: cu_q ascends
  int lo = 0, hi = p.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_q[mid + 1] > row) hi = mid; else lo = mid + 1;
  }
  if (lo == p.B) return;  // rows past the last request are not written
  const int n = p.cu_q[lo + 1] - p.cu_q[lo];
  const int len = min(p.kv_lens[lo], p.max_pages << p.page_shift) - n + (row - p.cu_q[lo]) + 1;
  if (tid < D)
    qs[tid] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[row * p.q_tok_stride + hq * p.q_head_stride + tid]);
  __syncthreads();
  const int page_mask = (1 << p.page_shift) - 1;
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int t0 = 0; t0 < len; t0 += kAttnThreads) {
    const int t = t0 + tid;
    float s = -INFINITY;
    const int id = t < len ? p.table[lo * p.ld_table + (t >> p.page_shift)] : -1;
    if (t < len && (unsigned)id >= (unsigned)p.num_pages) record_status(p.status, kStatusOffsets, 50);
    if ((unsigned)id < (unsigned)p.num_pages) {
      const long long blk = (long long)id * p.Hkv + h;
      const uint8_t* k = p.k_codes + ((blk << p.page_shift) + (t & page_mask)) * D;
      s = 0.0f;
      for (int d = 0; d < D; ++d) s += qs[d] * e4m3_val(k[d]);
      s *= p.k_scales[blk] * p.scale_log2;
    }
    float mx = s;
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, d));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, mx);
    const float c = mn > -INFINITY ? exp2f(m - mn) : 1.0f, e = mn > -INFINITY ? exp2f(s - mn) : 0.0f;
    ps[tid] = e;
    float sum = e;
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    l = l * c + (red[0] + red[1]) + (red[2] + red[3]);
    o *= c;
    m = mn;
    if (tid < D) {
      const int cnt = min(kAttnThreads, len - t0);
      for (int i = 0; i < cnt; ++i) {
        const int vid = p.table[lo * p.ld_table + ((t0 + i) >> p.page_shift)];
        if ((unsigned)vid >= (unsigned)p.num_pages) continue;
        const long long blk = (long long)vid * p.Hkv + h;
        o += ps[i] * p.v_scales[blk] * e4m3_val(p.v_codes[((blk << p.page_shift) + ((t0 + i) & page_mask)) * D + tid]);
      }
    }
    __syncthreads();
  }
  if (tid < D)
    static_cast<__nv_bfloat16*>(p.out)[row * p.out_tok_stride + hq * p.out_head_stride + tid] =
        __float2bfloat16(l > 0.0f ? o / l : 0.0f);
  if (tid == 0 && p.lse)
    p.lse[(long long)row * p.Hq + hq] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

cudaError_t launch_kv_attention(const KvAttentionLaunch& L, cudaStream_t stream) {
  const KvAttentionParams& p = L.p;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.T, (unsigned)p.Hq, 1);
  cfg.blockDim = dim3(kAttnThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return p.D == 64 ? cudaLaunchKernelEx(&cfg, kv_attention_kernel<64>, p)
                   : cudaLaunchKernelEx(&cfg, kv_attention_kernel<128>, p);
}

}  // namespace bsk
