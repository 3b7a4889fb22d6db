// kv_attention.cuh -- what the two attention kernels over the paged cache share.
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
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// 0x80 in every byte of w that is a NaN code (0x7f or 0xff)
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// w with the codes marked by n at 0
__device__ __forceinline__ uint32_t without(uint32_t w, uint32_t n) { return w & ~((n >> 7) * 0xffu); }

// a / b for a >= 0 and b > 0: 64-bit division only where it takes one
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

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

// Rows of all heads times tokens of a request in the sum that decides whether the few-rows kernel
// takes the whole call.  Whatever passes the bound counts as just above it: offsets that break
// the contract may claim any number of rows, and 32 bits hold a CTA's sum.
__device__ __forceinline__ int whole_part(const KvAttentionParams& p, const Rows& r, int len) {
  return (int)min((long long)min(r.n, p.T) * p.Hq * max(len, 128), (long long)p.whole_most + 1);
}
// The most rows per KV head of a request that the few-rows kernel takes, from that sum over the
// CTA's requests: a thread's are b0 .. b1 - 1, the first as read already.  parts: a place a warp, free
// again after another barrier.
template <int kThreads>
__device__ __forceinline__ int most_few_rows(const KvAttentionParams& p, int b0, int b1, const Rows& first, int len, int* parts, int G) {
  const int over = p.whole_most + 1;
  int sum = b0 < b1 ? whole_part(p, first, len) : 0;
  for (int b = b0 + 1; b < b1; ++b) sum = min(sum + whole_part(p, rows_of(p, b), cached(p, b)), over);
  sum = __reduce_add_sync(kFullMask, sum);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = min(sum, over);
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) all += parts[w];
  return all <= p.whole_most ? max(p.few_rows, p.T * G) : p.few_rows;
}

// Arrival of a piece: how many came before it.  Called by one thread between two
// barriers of those that wrote it and will read the others': the barrier before makes
// their stores part of what this releases, the one after makes what this acquires theirs
// (a fence by every thread instead took 1 us more of 10 and of 75 us calls).
__device__ __forceinline__ int arrive_piece(int* counter) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old;
}
}  // namespace bsk
