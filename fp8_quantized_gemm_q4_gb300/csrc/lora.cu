// lora.cu -- low-rank adapters of many requests beside a projection that they share:
//   out = y + s_a (x A_a^T) B_a^T,  a = the adapter of the row's request.
// One CTA for a row, in fp32.
#include "decode.h"
#include "decode.cuh"

namespace bsk {
namespace {

template <bool kBf16>
__global__ void __launch_bounds__(256) lora_kernel(const __grid_constant__ LoraParams p) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ float t[];
  __shared__ int found;
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) found = -2;
  __syncthreads();
  for (int b = threadIdx.x; b < p.B; b += 256) {
    const int lo = p.cu[b], hi = p.cu[b + 1];
    if (row == 0 && (lo < 0 || hi < lo || hi > p.T || p.which[b] >= p.adapters)) record_status(p.status, kStatusOffsets, 57);
    if (lo >= 0 && lo <= row && row < hi) found = p.which[b] >= p.adapters ? -1 : max(p.which[b], -1);
  }
  __syncthreads();
  const int id = found;
  if (id == -2) return;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + row * p.ldx;
  if (id >= 0)
    for (int i = warp; i < p.r; i += 8) {
      const __nv_bfloat16* a = static_cast<const __nv_bfloat16*>(p.a) + ((long long)id * p.r + i) * p.K;
      float sum = 0.0f;
      for (int k = lane; k < p.K; k += 32) sum = fmaf(__bfloat162float(x[k]), __bfloat162float(a[k]), sum);
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
      if (lane == 0) t[i] = sum * (p.scales ? p.scales[id] : 1.0f);
    }
  __syncthreads();
  for (int n = threadIdx.x; n < p.N; n += 256) {
    float sum = 0.0f;
    if (id >= 0) {
      const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(p.b) + ((long long)id * p.N + n) * p.r;
      for (int i = 0; i < p.r; ++i) sum = fmaf(t[i], __bfloat162float(b[i]), sum);
    }
    if constexpr (kBf16)
      static_cast<__nv_bfloat16*>(p.out)[row * p.ldo + n] =
          __float2bfloat16(__bfloat162float(static_cast<const __nv_bfloat16*>(p.y)[row * p.ldy + n]) + sum);
    else
      static_cast<float*>(p.out)[row * p.ldo + n] = static_cast<const float*>(p.y)[row * p.ldy + n] + sum;
  }
}

}  // namespace

size_t lora_workspace_bytes(int, int, int, int, int, int) { return 16; }

cudaError_t launch_lora(const LoraParams& p, int, cudaStream_t stream) {
  return p.bf16 ? launch_kernel(lora_kernel<true>, (unsigned)p.T, 256, p.r * sizeof(float), stream, 1, p)
                : launch_kernel(lora_kernel<false>, (unsigned)p.T, 256, p.r * sizeof(float), stream, 1, p);
}

}  // namespace bsk
