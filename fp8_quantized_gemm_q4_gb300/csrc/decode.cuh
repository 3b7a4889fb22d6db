// decode.cuh -- device helpers of the decode-step kernels beside ptx.cuh's.
#pragma once
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace bsk {

// Device status word code (mirrors bs_status in bsgemm.h), beside those of ptx.cuh.
constexpr int kStatusPages = 7;

// The two e4m3 codes of a 16-bit word as fp16 (exact), low code in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
// Four bytes of e4m3 as two f16x2
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

}  // namespace bsk
