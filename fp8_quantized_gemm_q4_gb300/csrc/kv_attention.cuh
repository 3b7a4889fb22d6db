// kv_attention.cuh -- what the two attention kernels over the 8-bit cache share.
#pragma once
#include "decode.cuh"
#include "decode.h"

namespace bsk {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The power of two that brings a row with this largest element to [2^14, 2^15)
__device__ __forceinline__ int fp16_up(float amax) {
  const int ex = max((int)(__float_as_uint(amax) >> 23) - 127, -112);
  return amax > 0.0f ? 14 - min(ex, 127) : 0;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 0x80 in every byte of w that is a NaN code (0x7f or 0xff)
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// w with the codes marked by n at 0
__device__ __forceinline__ uint32_t without(uint32_t w, uint32_t n) { return w & ~((n >> 7) * 0xffu); }

// natural log of the softmax sum 2^m l
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;  // NaN sums stay NaN
}

// A request's rows: the first, how many, and how many of them the call has (row < T).
// Offsets that do not ascend from 0 give none, and work never goes past T.
struct Rows {
  int row0, n, in;
  bool bad;  // offsets that break the contract
};
__device__ __forceinline__ Rows rows_of(const KvAttentionParams& p, int b) {
  const int r0 = p.cu_q[b], r1 = p.cu_q[b + 1];
  const int n = r0 < 0 || r1 <= r0 ? 0 : r1 - r0;
  return {r0, n, n ? max(0, min(n, p.T - r0)) : 0, r0 < 0 || r1 < r0 || r1 > p.T};
}

// Cached tokens of a request, as far as its table row can name them; a length beyond
// that, or a negative one, is the status's to tell.
__device__ __forceinline__ int cached(const KvAttentionParams& p, int b) {
  return min(max(p.kv_lens[b], 0), p.max_pages << p.page_shift);
}
__device__ __forceinline__ bool length_bad(const KvAttentionParams& p, int b) {
  return (unsigned)p.kv_lens[b] > (unsigned)(p.max_pages << p.page_shift);
}
}  // namespace bsk
