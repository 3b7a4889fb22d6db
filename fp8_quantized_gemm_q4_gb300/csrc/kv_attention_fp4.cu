// kv_attention_fp4.cu -- causal attention of new tokens over the paged 4-bit cache.
// One warp for a row and query head, in fp32.
#include "kv_attention.cuh"

namespace bsk {
namespace {

template <int D>
__global__ void __launch_bounds__(128) kv_attention_fp4_kernel(const __grid_constant__ KvAttentionParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, head = blockIdx.x % p.Hq;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += 128) {
      const Rows r = rows_of(p, b);
      if ((long long)r.n * (p.Hq / p.Hkv) > p.most_rows || r.bad || length_bad(p, b)) record_status(p.status, kStatusOffsets, 53);
    }
  const int row = blockIdx.x / p.Hq * 4 + (threadIdx.x >> 5);
  if (row >= p.T) return;
  constexpr int kE = D / 32;  // elements of a lane
  const int h = head / (p.Hq / p.Hkv);
  for (int b = 0; b < p.B; ++b) {
    const Rows r = rows_of(p, b);
    if (r.in <= 0 || row < r.row0 || row >= r.row0 + r.in) continue;
    const int len = cached(p, b), seen = max(0, min(len, len - r.n + (row - r.row0) + 1));
    float q[kE], o[kE] = {}, m = -INFINITY, l = 0.0f;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q) + row * p.q_tok_stride + head * p.q_head_stride;
    for (int i = 0; i < kE; ++i) q[i] = __bfloat162float(qp[kE * lane + i]) * p.scale_log2;
    for (int t = 0; t < seen; ++t) {
      const int id = p.table[b * p.ld_table + (t >> p.page_shift)];
      if ((unsigned)id >= (unsigned)p.num_pages) {
        record_status(p.status, kStatusOffsets, 50);
        continue;
      }
      const long long at = (((long long)id * p.Hkv + h) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
      float k[kE], v[kE];
      auto get = [&](const uint8_t* codes, const void* scales, float(&x)[kE]) {
        uint32_t w = 0, f[4];
        for (int i = 0; i < kE / 2; ++i) w |= (uint32_t)codes[at * (D / 2) + lane * (kE / 2) + i] << (8 * i);
        e2m1x8_to_f16(w, f);
        const float s = e4m3_to_f32(static_cast<const uint8_t*>(scales)[at * (D / 16) + lane * kE / 16]);
        for (int i = 0; i < kE; ++i) {
          const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&f[i / 2]));
          x[i] = (i & 1 ? e.y : e.x) * s;
        }
      };
      get(p.k_codes, p.k_scales, k);
      get(p.v_codes, p.v_scales, v);
      float u = 0.0f;
      for (int i = 0; i < kE; ++i) u = fmaf(q[i], k[i], u);
      for (int d = 16; d; d >>= 1) u += __shfl_xor_sync(kFullMask, u, d);
      const float top = fmaxf(m, u), f = m == -INFINITY ? 0.0f : ex2(m - top), e = ex2(u - top);
      m = top;
      l = l * f + e;
      for (int i = 0; i < kE; ++i) o[i] = o[i] * f + e * v[i];
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.out_tok_stride + head * p.out_head_stride;
    for (int i = 0; i < kE; ++i) out[kE * lane + i] = __float2bfloat16(o[i] * inv);
    if (lane == 0 && p.lse) p.lse[(long long)row * p.Hq + head] = lse_of(m, l);
  }
}

}  // namespace

cudaError_t launch_kv_attention_fp4(const KvAttentionLaunch& L, cudaStream_t stream) {
  const KvAttentionParams& p = L.p;
  const unsigned grid = (unsigned)((p.T + 3) / 4 * p.Hq);
  return p.D == 64 ? launch_kernel(kv_attention_fp4_kernel<64>, grid, 128, 0, stream, 1, p)
                   : launch_kernel(kv_attention_fp4_kernel<128>, grid, 128, 0, stream, 1, p);
}

}  // namespace bsk
