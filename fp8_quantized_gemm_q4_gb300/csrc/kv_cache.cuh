// kv_cache.cuh -- what the kernels that write the 8-bit cache share: a page's scale
// and the check of a slot.
#pragma once
#include "decode.cuh"

namespace bsk {

// log2 of the scale for this amax (>= 0)
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // amax = 1.m * 2^x; 448 = 1.75 * 2^8, so the smallest e with
  // amax <= 1.75 * 2^(e + 8) is x - 8, or x - 7 where 1.m > 1.75
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -32), 64);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The new scale of a run, and where it grows the page's earlier codes rounded
// again to it, by the threads 0 .. kThreads - 1 (a warp, or several).  Returns the
// scale; old is the page's (used if off > 0).
template <int D, int kThreads = 32>
__device__ __forceinline__ float page_scale(uint8_t* codes, int off, float amax, float old, int thread) {
  const float s = exp2_int(scale_exp(amax));
  if (off == 0) return s;
  if (s <= old) return old;
  const float ratio = old / s;
  for (int x = thread; x < off * (D / 8); x += kThreads) {
    uint2* at = reinterpret_cast<uint2*>(codes) + x;
    const uint2 w = *at;
    const uint32_t in[2] = {w.x, w.y};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h2 = e4m3x2_to_f16x2((uint16_t)(in[i >> 1] >> (16 * (i & 1))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      h[i] = f32x2_to_e4m3x2(f.x * ratio, f.y * ratio);
    }
    *at = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  }
  return s;
}

template <typename Params>
__device__ __forceinline__ bool slot_ok(const Params& p, int slot) {
  if (slot < 0) return false;
  if ((slot >> p.page_shift) < p.num_pages) return true;
  record_status(p.status, kStatusOffsets, 45);
  return false;
}

}  // namespace bsk
