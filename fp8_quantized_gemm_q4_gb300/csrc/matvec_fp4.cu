// matvec_fp4.cu -- a few bf16 rows times FP4 weights:
//   y[m, n] = alpha * ts * sum_k x[m, k] * e2m1[n, k] * sf[n, k / 16] + bias[n]
// with the codes and MMA-layout group scales that q4_quantize writes and the
// activations left in bf16.
#include "kernels.h"
#include "ptx.cuh"

namespace bsk {

constexpr int kMvWarps = 4;
constexpr int kMvMaxM = 16;

// One warp per weight row; a lane takes every 32nd group of 16.
__global__ void __launch_bounds__(kMvWarps * 32) fp4_matvec_kernel(const __grid_constant__ Fp4MatvecParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, n = blockIdx.x * kMvWarps + (threadIdx.x >> 5);
  if (n >= p.N) return;
  float acc[kMvMaxM] = {};
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x);
  for (int g = lane; g < p.K / 16; g += 32) {
    const uint2 w = *reinterpret_cast<const uint2*>(p.codes + (long long)n * (p.K / 2) + g * 8);
    const long long at = ((long long)(n / 128) * (p.K / 64) + g / 4) * 512 + (n % 32) * 16 + (n % 128) / 32 * 4 + g % 4;
    const float s = e4m3_to_f32(p.sf[at]);
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t h2 = e2m1x2_to_f16x2(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xff);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      v[2 * i] = f.x * s, v[2 * i + 1] = f.y * s;
    }
#pragma unroll
    for (int m = 0; m < kMvMaxM; ++m)
      if (m < p.M)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[m] = fmaf(__bfloat162float(x[m * p.ldx + g * 16 + i]), v[i], acc[m]);
  }
  const float a = p.alpha * (p.tensor_scale ? *p.tensor_scale : 1.0f);
  const float bias = p.bias ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[n]) : 0.0f;
#pragma unroll
  for (int m = 0; m < kMvMaxM; ++m) {
    float t = acc[m];
    for (int d = 16; d; d >>= 1) t += __shfl_xor_sync(kFullMask, t, d);
    if (lane == 0 && m < p.M) {
      const float y = fmaf(a, t, bias);
      if (p.out_bf16)
        static_cast<__nv_bfloat16*>(p.out)[m * p.ldo + n] = __float2bfloat16(y);
      else
        static_cast<float*>(p.out)[m * p.ldo + n] = y;
    }
  }
}

cudaError_t launch_fp4_matvec(const Fp4MatvecParams& p, int sms, cudaStream_t stream) {
  (void)sms;
  return launch_kernel(fp4_matvec_kernel, (unsigned)((p.N + kMvWarps - 1) / kMvWarps), kMvWarps * 32, 0, stream, 1, p);
}

}  // namespace bsk
