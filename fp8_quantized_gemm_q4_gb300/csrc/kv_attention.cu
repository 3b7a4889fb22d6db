// kv_attention.cu -- causal attention of new tokens over the paged 8-bit or 4-bit
// cache.  Of 8 bits:  o = softmax(scale q K^T) V  with K = s_K[page, head] * code and V
// likewise; row i of a request with n new and m cached tokens (the new ones
// included) sees the cached positions 0 .. m - n + i.
//
// e4m3 codes are exact in fp16, so both products run on fp16 operands with fp32
// accumulation and no code is rounded.  q goes to fp16 by a power of two per
// row (largest element in [2^14, 2^15): exact within 2^-29 of it).  With
// u_t = scale log2(e) s_K q.k_t + log2 s_V(page of t) and m a running reference
// at most 8 below max u, the weights w_t = 2^(u_t - m) carry the V scales:
//   sum_t w_t code_t = 2^-m sum_t 2^(score) v_t,    l = sum_t w_t / s_V = 2^-m sum_t 2^(score)
// so pages with scales far apart meet in one accumulator, every w_t <= 2^8
// fits fp16 (rounded to 11 bits, the only rounding below fp32), and o, lse
// follow from (m, l, sum).  m moves, and the accumulators are rescaled, only
// when max u passes m + 8.
//
// 4-bit cache: a value is an E2M1 code times the e4m3 scale of its 16 elements of a
// token, 1 + 3 significant bits from 2^-10 to 2688: exact in fp16, as K and V are.  So
// u_t = scale log2(e) q.k_t, w_t = 2^(u_t - m), and o, lse = sum w_t v_t / sum w_t, m + log2.
#include "kv_attention.cuh"

namespace bsk {

namespace {

template <bool kFp4>
constexpr int kTileOf = kFp4 ? 128 : 64;  // cached tokens per stage

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Shared memory of a tile as TMA writes it: rows of 128 bytes (one token of kBytes,
// or two or four: rows of 64 bytes came in at half the rate), their 16-byte chunks
// exchanged by the 128-byte swizzle.
template <int kBytes>
__device__ __forceinline__ int code_at(int tok, int chunk) {
  if constexpr (kBytes == 128) return tok * 128 + ((chunk ^ (tok & 7)) << 4);
  if constexpr (kBytes == 64) return (tok >> 1) * 128 + (((((tok & 1) << 2) | chunk) ^ ((tok >> 1) & 7)) << 4);
  return (tok >> 2) * 128 + (((((tok & 3) << 1) | chunk) ^ ((tok >> 2) & 7)) << 4);
}
// Which of 8 tokens stands at place n of the MMA's token axis: any order does,
// as long as scores, masks and V rows agree.  For D = 128 places 2 i, 2 i + 1
// are four tokens apart, so that the 16-byte loads of K meet no bank twice.
template <int D>
__device__ __forceinline__ int token_of(int n) {
  return D == 128 ? (n >> 1) | ((n & 1) << 2) : n;
}

__device__ __forceinline__ void store_floats(float4* at, float x, float y, float z, float w) { *at = make_float4(x, y, z, w); }
__device__ __forceinline__ void store_floats(float2* at, float x, float y, float, float) { *at = make_float2(x, y); }
__device__ __forceinline__ void add_floats(const float4* at, float& x, float& y, float& z, float& w) {
  const float4 v = *at;
  x += v.x, y += v.y, z += v.z, w += v.w;
}
__device__ __forceinline__ void add_floats(const float2* at, float& x, float& y, float&, float&) {
  const float2 v = *at;
  x += v.x, y += v.y;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// NaN codes among the first cnt of 16 tokens of V that some row does not see: a
// weight of 0 would spread them, so they become 0 in shared memory.  The lane's
// accumulators whose row does see one are returned: bit 4 a + 2 i + e for column
// 16 a + 2 g + i and the row that sees `seen[e]` of the 16.  Called by a whole
// warp; out of line, for calls that meet none.
template <int D>
__device__ __noinline__ uint32_t take_nan(uint8_t* vt, int cnt, int seen0, int seen1, int lane) {
  uint32_t hit = 0;
  for (int tok = 0; tok < cnt; ++tok)
#pragma unroll 1
    for (int a = 0; a < D / 16; ++a)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if ((vt[code_at<D>(tok, a) + 2 * (lane >> 2) + i] & 0x7f) == 0x7f)
          hit |= (tok < seen0 ? 1u : 0u) << (4 * a + 2 * i) | (tok < seen1 ? 2u : 0u) << (4 * a + 2 * i);
  __syncwarp();
  for (int x = lane; x < cnt * (D / 4); x += 32) {
    uint32_t* w = reinterpret_cast<uint32_t*>(vt + code_at<D>(x / (D / 4), x % (D / 4) / 4)) + x % 4;
    *w = without(*w, nan_codes(*w));
  }
  __syncwarp();
  return hit;
}

// The same of a 4-bit cache, where a NaN scale stands for a NaN in its 16 columns:
// `scales` are those of V.  Bit e is returned if row e's columns of this lane, which are of
// one group, have met one.
template <int D>
__device__ __noinline__ uint32_t take_nan_scales(uint8_t* scales, int cnt, int seen0, int seen1, int lane) {
  uint32_t hit = 0;
  for (int tok = 0; tok < cnt; ++tok)
    if ((scales[tok * (D / 16) + (lane >> 2) * D / 128] & 0x7f) == 0x7f) hit |= (tok < seen0 ? 1u : 0u) | (tok < seen1 ? 2u : 0u);
  __syncwarp();
  for (int x = lane; x < cnt * (D / 16); x += 32)
    if ((scales[x] & 0x7f) == 0x7f) scales[x] = 0;
  __syncwarp();
  return hit;
}

// One step of the online softmax over 16 tokens for 8 rows.  u[e]: logit of
// row 2 c + e % 2 for token place g + 8 (e / 2).  Returns the weights as the B
// fragment (places on k) of the product with V.
template <int NA>
__device__ __forceinline__ void softmax_step(float (&u)[4], float inv_sv, float (&m)[2], float (&l)[2],
                                             float (&o)[NA][4], uint32_t (&pb)[2]) {
  float mx[2] = {fmaxf(u[0], u[2]), fmaxf(u[1], u[3])};
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) {
    mx[0] = fmaxf(mx[0], __shfl_xor_sync(kFullMask, mx[0], d));
    mx[1] = fmaxf(mx[1], __shfl_xor_sync(kFullMask, mx[1], d));
  }
  if (__any_sync(kFullMask, mx[0] > m[0] + 8.0f || mx[1] > m[1] + 8.0f)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool up = mx[h] > m[h] + 8.0f;
      const float f = up ? ex2(m[h] - mx[h]) : 1.0f;
      m[h] = up ? mx[h] : m[h];
      l[h] *= f;
#pragma unroll
      for (int a = 0; a < NA; ++a) o[a][h] *= f, o[a][2 + h] *= f;
    }
  }
  const float r0 = m[0] == -INFINITY ? 0.0f : m[0], r1 = m[1] == -INFINITY ? 0.0f : m[1];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float a = ex2(u[2 * t] - r0), b = ex2(u[2 * t + 1] - r1);
    l[0] = fmaf(a, inv_sv, l[0]);
    l[1] = fmaf(b, inv_sv, l[1]);
    pb[t] = movmatrix_trans(pack_f16x2(a, b));
  }
}

// Which of 16 tokens of a 4-bit tile stands at place n of the MMA's token axis: an order in
// which neither the loads of K (a token a lane, 8 lanes' at once) nor those of V (four tokens a
// lane) meet a bank twice.
template <int D>
__device__ __forceinline__ constexpr int fp4_token(int n) {
  return D == 128 ? 4 * ((n & 7) >> 1) + (n & 1) + 2 * (n >> 3) : n ^ ((n >> 2) & 1);
}

// Places in shared memory of what a lane reads of the 32 tokens of a 4-bit tile that its
// warp takes, from the stage's codes and the scales of those tokens on; h: 16 of them.
template <int D>
struct Fp4At {
  // of the second 16 tokens of D = 128: 1024 bytes on, with the same exchange of pieces
  static constexpr int kHalves = D == 128 ? 1 : 2;
  uint32_t k_[kHalves][2], v_[kHalves][4], ks, vs_[2];
  __device__ __forceinline__ Fp4At(int warp, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int tok = warp * 32 + 16 * h;
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // D / 4 columns of the tokens at places g and g + 8
        const int t = tok + fp4_token<D>(8 * i + g);
        k_[h][i] = D == 128 ? code_at<64>(t, c) : code_at<32>(t, c >> 1) + 8 * (c & 1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // D / 8 columns of those at places 2 c, 2 c + 1, 2 c + 8, 2 c + 9
        const int t = tok + fp4_token<D>(2 * c + (i & 1) + 8 * (i >> 1));
        v_[h][i] = kTileOf<true> * (D / 2) + (D == 128 ? code_at<64>(t, g >> 1) + 8 * (g & 1) : code_at<32>(t, g >> 2) + 4 * (g & 3));
      }
    }
    ks = fp4_token<D>(g) * (D / 16) + (D == 128 ? 2 : 1) * c;
#pragma unroll
    for (int i = 0; i < 2; ++i) vs_[i] = (kTileOf<true> + fp4_token<D>(2 * c + i)) * (D / 16) + g * D / 128;
  }
  __device__ __forceinline__ uint32_t k(int h, int i) const { return D == 128 ? k_[0][i] + 1024 * h : k_[h % kHalves][i]; }
  __device__ __forceinline__ uint32_t v(int h, int i) const { return D == 128 ? v_[0][i] + 1024 * h : v_[h % kHalves][i]; }
  // scales of the same tokens; places eight apart are two tokens apart, or eight
  static constexpr int kEight = fp4_token<D>(8) * (D / 16);
  __device__ __forceinline__ uint32_t k_scale(int h, int i) const { return ks + 16 * h * (D / 16) + kEight * i; }
  __device__ __forceinline__ uint32_t v_scale(int h, int i) const { return vs_[i & 1] + 16 * h * (D / 16) + kEight * (i >> 1); }
};
// mma_f16 that the compiler may move among the loads and conversions
__device__ __forceinline__ void mma_f16_free(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
constexpr int kAllThere = 16 | 16 << 8;
constexpr float kNone = -3.0e38f;  // reference of a row that has seen no token

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Loads from shared memory that stay behind the stores before them
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return (uint16_t)v;
}
__device__ __forceinline__ uint16_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// 32 tokens of a 4-bit tile for 8 rows: scores, a step of the online softmax (as
// softmax_step, with the distance from the reference, score * qscale - m, in place of the
// logit, and the rows' maxima looked for only where some distance passes 8), and the
// product with V.  codes, scales: the stage's in shared memory; vs the same of V; cnt:
// there: tokens that are there, of the first 16 in the low byte, of the others above it.
template <int D>
__device__ __forceinline__ void fp4_tile(uint32_t codes, uint32_t scales, uint8_t* vs, int there, int tok0,
                                         int all_seen, const int (&seen)[2], const float (&qscale)[2],
                                         uint32_t q, float (&m)[2], float (&l)[2], float (&o)[D / 16][4],
                                         const Fp4At<D>& at, int lane) {
  const bool edge = there != kAllThere || tok0 + 32 > all_seen;
  const int cnt[2] = {there & 0xff, there >> 8};
  if (edge) {
    // a NaN scale of V behind the last token, or where some row does not look
    uint32_t any = 0;
#pragma unroll
    for (int x = lane; x < D / 2; x += 32) {
      uint32_t* w = reinterpret_cast<uint32_t*>(vs) + x;
      const int tok = 4 * x / (D / 16);
      if ((tok & 15) >= (tok < 16 ? cnt[0] : cnt[1])) *w = 0;
      any |= nan_codes(*w);
    }
    __syncwarp();
    if (__any_sync(kFullMask, any)) {
      const uint32_t hit = take_nan_scales<D>(vs, 32, seen[0] - tok0, seen[1] - tok0, lane);
#pragma unroll
      for (int a = 0; a < D / 16; ++a)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (hit >> (x & 1) & 1) o[a][x] = __int_as_float(0x7fffffff);
    }
    __syncwarp();
  }
  float s[2][4] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[2][D / 32], f[2];  // [i]: columns of the token at place 8 i + g, their one or two scales
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t at_scale = scales + at.k_scale(h, i);
      if constexpr (D == 128) {
        const uint4 a = lds128(codes + at.k(h, i));
        w[i][0] = a.x, w[i][1] = a.y, w[i][2] = a.z, w[i][3] = a.w;
        f[i] = e4m3x2_to_f16x2(lds16(at_scale));
      } else {
        const uint2 a = lds64(codes + at.k(h, i));
        w[i][0] = a.x, w[i][1] = a.y;
        f[i] = e4m3x2_to_f16x2(lds8(at_scale));
      }
    }
#pragma unroll
    for (int y = 0; y < D / 32; ++y) {
      const uint4 b = lds128(q + y * 512);
      const uint32_t fa = __byte_perm(f[0], 0, y < 2 ? 0x1010 : 0x3232), fb = __byte_perm(f[1], 0, y < 2 ? 0x1010 : 0x3232);
      uint32_t ka[4], kb[4];
      e2m1x8_to_f16(w[0][y], ka);
      e2m1x8_to_f16(w[1][y], kb);
      const uint32_t lo[4] = {hmul2(ka[0], fa), hmul2(kb[0], fb), hmul2(ka[1], fa), hmul2(kb[1], fb)};
      const uint32_t hi[4] = {hmul2(ka[2], fa), hmul2(kb[2], fb), hmul2(ka[3], fa), hmul2(kb[3], fb)};
      mma_f16_free(s[h], lo, b.x, b.y);
      mma_f16_free(s[h], hi, b.z, b.w);
    }
  }
  if (edge) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = fp4_token<D>(lane >> 2) + fp4_token<D>(8) * (e >> 1);
        if (tok >= cnt[h] || tok0 + 16 * h + tok >= seen[e & 1]) s[h][e] = -INFINITY;
      }
  }
  float z[2][4];
  auto distances = [&] {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[h][e] = fmaf(s[h][e], qscale[e & 1], -m[e & 1]);
  };
  distances();
  const float far = max3(max3(z[0][0], z[0][1], z[0][2]), max3(z[0][3], z[1][0], z[1][1]), fmaxf(z[1][2], z[1][3]));
  if (__any_sync(kFullMask, far > 8.0f)) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float mx = fmaxf(fmaxf(s[0][e], s[0][2 + e]), fmaxf(s[1][e], s[1][2 + e])) * qscale[e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, d));
      const bool up = mx > m[e] + 8.0f;
      const float f = up ? ex2(m[e] - mx) : 1.0f;
      m[e] = up ? mx : m[e];
      l[e] *= f;
#pragma unroll
      for (int a = 0; a < D / 16; ++a) o[a][e] *= f, o[a][2 + e] *= f;
    }
    distances();
  }
  uint32_t pb[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float a = ex2(z[h][2 * t]), b = ex2(z[h][2 * t + 1]);
      l[0] += a, l[1] += b;
      pb[h][t] = movmatrix_trans(pack_f16x2(a, b));
    }
  // A lane has D / 8 columns, of one group, of four tokens: a byte of two columns of a token
  // and that of its neighbour exchange a column, and each byte's conversion gives a column of two tokens.
  // Tile 4 w + b has the columns D / 8 g + 8 w + 2 b (g on its first rows) and + 1.
  constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t sv[2], v[4][D / 64];
#pragma unroll
    for (int t = 0; t < 2; ++t)
      sv[t] = e4m3x2_to_f16x2((uint16_t)__byte_perm(lds8(scales + at.v_scale(h, 2 * t)), lds8(scales + at.v_scale(h, 2 * t + 1)), 0x0040));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (D == 128) {
        const uint2 a = lds64(codes + at.v(h, i));
        v[i][0] = a.x, v[i][1] = a.y;
      } else {
        v[i][0] = lds32(codes + at.v(h, i));
      }
    }
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
      uint32_t even[2][4], odd[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t x = v[2 * t][w], y = v[2 * t + 1][w];
        e2m1x8_to_f16((x & kLow) | ((y << 4) & ~kLow), even[t]);
        e2m1x8_to_f16(((x >> 4) & kLow) | (y & ~kLow), odd[t]);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t va[4] = {hmul2(even[0][b], sv[0]), hmul2(odd[0][b], sv[0]), hmul2(even[1][b], sv[1]), hmul2(odd[1][b], sv[1])};
        mma_f16_free(o[4 * w + b], va, pb[h][0], pb[h][1]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Requests with at most few_rows rows per KV head (decode, drafts): bound by the
// cache stream.  Work is a list of (request, head, 8 rows) units of 64-token
// tiles (4 bits: 128), cut into contiguous shares of equal cost, whatever the lengths.  Three CTAs an
// SM take one each: a producer warp keeps 64 KB of codes in flight with TMA copies
// page by page, four consumer warps take 16 tokens of a tile each (4 bits: 32), and while one
// CTA joins the warps' results of a unit, the other two stream (one CTA with 12
// consumer warps lost 25 of 134 us to that).  Both products run transposed,
// tokens and then head columns on the MMA's M and the rows on its N = 8:
// S^T = K Q^T, O^T = V^T P^T; a group of 4 or 8 query heads fills N, where it would
// leave half of M = 16 empty.  More than 8 rows are units of their own beside the
// first, whose tiles they find in L2.
// 64 requests of 500 to 16000 tokens, 32 heads over 8, D = 128 (604 MB): 105 us, 0.85
// of HBM.  63 drafted tokens of 16 requests, 16 heads, D = 64, 16-token pages (60 MB):
// 24 us, bound by what a unit costs beside its tiles (q, the join of the warps, its
// piece); one token over 1000: 9.5 us, a chain of dependent reads.  Three CTAs an SM
// leave 128 registers a thread, and 20 to 24 bytes of it are spilled.
// Of 4 bits, which halve the stream, the same calls take 73 us (340 MB, 0.69 of HBM; with 16000
// tokens each 216, 0.81), 21 us (34 MB) and 9 us: about 14 us that no stream fills (shares,
// lists and the first tiles, the joins) and then 0.86 of HBM.  A cached element costs what it does
// with 8 bits and the product with its scale: 335 instructions a warp and 16 tokens, 0.55 of the
// issue slots and 0.54 of the pipe that converts and exchanges bytes.  So 32 tokens a step, whose
// chains of products run side by side, maxima looked for only where a score passes its
// reference by 8, q as fragments in shared memory (with each 107, 83 and 77 us in one
// setting), and V as four tokens a lane, whose columns share a scale (75.5, then 74.5; two tokens
// by ldmatrix before).  The three CTAs of an SM end their equal shares one after the other, after
// 57, 66 and 72 us, and what goes on has the stream for itself.  Measured beside it: smaller
// shares for CTAs that take the place of those that end first 84 to 86 (a start costs more
// than the waiting), shares by place in the grid and four CTAs of 96 registers
// no gain; units of 16 rows, whose K and V are converted once, by two CTAs an SM: 64 requests of
// 16 rows 82, not 98, but one such request 28, not 18, and 64 of 8 rows beside one of 12 77, not 57.
// ---------------------------------------------------------------------------
constexpr int kItems = 32;         // units listed at a time
constexpr int kMinTiles = 2;       // least cost worth a CTA of its own
// What a unit costs beside its tiles (q, the join of the warps, a piece), in tiles.
// us with 0 / 2 / 4 / 10: 64 decode requests 107.6 / 106.1 / 105.5 / 106, drafts over 16
// heads 24.8 / 23.3 / 22.9 / 23.9, 64 requests of 30 to 14000 tokens 20.6 / 17.4 / 16.6 / 16.7.  Of 4 bits,
// tiles twice as long, with 0 / 1 / 2 / 4: 64 decode requests 80 / 77 / 75 / 77, drafts 23.1 / 22.7 /
// 21.9 / 23.0, 300 requests of 200 to 2000 tokens 90 / 81 / 77 / 81
template <bool kFp4>
constexpr int kUnitTilesOf = kFp4 ? 2 : 4;
constexpr int kCounters = 1024;    // arrival counters at the head of the workspace
constexpr int kFewWarps = 4;       // consumers; one more warp produces
constexpr int kFewThreads = kFewWarps * 32 + 32;
constexpr int kFewCtas = 3;        // an SM

template <int D, bool kFp4>
struct FewSmem {
  static constexpr int kTile = kTileOf<kFp4>;
  static constexpr int kStages = kFp4 ? 384 / D : 512 / D;  // 64 KB of codes, or 54 KB of them and scales
  static constexpr int kRow = kFp4 ? D / 2 : D;             // bytes of a token's codes
  static constexpr int kStageBytes = 2 * kTile * kRow;
  alignas(1024) uint8_t kv[kStages][kStageBytes];  // K rows, then V rows
  alignas(16) uint8_t scale[kFp4 ? kStages : 1][2][kFp4 ? kTile * D / 16 : 16];  // of K and V, 4 bits
  uint4 q[kFp4 ? D / 32 : 1][kFp4 ? 32 : 1];  // of 4 bits: the unit's q as B fragments (in registers otherwise)
  float red[kFewWarps / 2][8 * D];
  float2 ml[kFewWarps][8];
  float4 group[kFp4 ? 1 : kStages][4];  // per 16 tokens: K scale, log2 of V scale, 1 / V scale, valid tokens (int)
  int there[kFp4 ? kStages : 1][kFewWarps];  // of 4 bits: valid tokens of a warp's first 16, and 256 times those of the others
  // units of this share: request, KV head, first of the 8 rows, cached tokens;
  // first row, rows (true), rows within T; the share's tile at which the unit
  // would begin, its end tile within the share (0: no unit)
  int4 item[kItems];
  int4 rows[kItems];
  int begin[kItems], end[kItems];
  uint64_t full[kStages], empty[kStages];
  int2 scan[kFewThreads / 32];
  int parts[kFewThreads / 32];
  int few;  // of 4 bits: most rows per KV head of a request that this kernel takes
  long long first_unit;      // of this share, counted over requests with tiles
  long long bound[2];        // its first tile in the list, the next share's
  int abort_flag, last;
};

// Tiles of each unit of a request in this kernel's list: none without rows or
// with more than `few` per KV head, else one at least (rows that see nothing
// are written too).  Which kernel serves a request follows from its own rows, the call's
// and (4 bits) their tokens, so that its result depends neither on the bound that the call
// gives nor on the width of its table.
template <int kTile>
__device__ __forceinline__ int few_tiles(int few, int n, int len, int G) {
  return n <= 0 || (long long)n * G > few ? 0 : max(1, (len + kTile - 1) / kTile);
}

// A piece of a unit that is cut between CTAs: partial sums [8][D], then (m, l) of
// the 8 rows.  A CTA has at most two: of the unit that begins before its share
// (0) and of one that begins in it (1).
template <int D>
__device__ __forceinline__ long long piece_at(int cta, int first_cta) {
  return ((long long)cta * 2 + (cta == first_cta)) * (8 * (D + 2));
}
// Place of column d of a row in a reduction buffer: 16-column windows and their
// halves exchanged by row, so that the fragments' stores meet no bank twice.
// For 4 bits, whose fragments store four of D / 8 columns at a time, pieces of 4 by row.
template <int D, bool kFp4>
__device__ __forceinline__ int red_at(int r, int d) {
  if constexpr (kFp4) return r * D + (d ^ (D == 128 ? ((r >> 1) & 3) << 2 : ((r >> 1) & 1) << 2 | ((r >> 2) & 1) << 4));
  return r * D + ((((d >> 4) ^ ((r >> 1) & 1)) << 4) | ((d & 15) ^ (((r >> 2) & 1) << 3)));
}

template <int D, bool kFp4>
__global__ void __launch_bounds__(kFewThreads, kFewCtas)
    kv_attention_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ KvAttentionParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = FewSmem<D, kFp4>;
  constexpr int kRow = Smem::kRow, kTile = Smem::kTile, kUnitTiles = kUnitTilesOf<kFp4>;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kStages = Smem::kStages, kWarps = kFewWarps, kThreads = kFewThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.Hkv;
  const WaitGuard wg{&sm.abort_flag, p.status, p.wait_ns};
  auto consumer_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); };
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], kFp4 ? 1 + kTile / 16 : 1);  // 4 bits: and a lane's scales of 16 tokens each
      mbar_init(&sm.empty[s], kFewWarps);
    }
    fence_barrier_init();
    sm.abort_flag = 0;
  }
  griddep_wait();
  griddep_launch_dependents();

  // Each thread takes `per` requests in a row: their tiles and row tiles, summed
  // over the block, place its units in the list.
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  Rows own = {};  // of the last of them: all there is while B <= threads
  int len_own = 0;
  int few = p.few_rows;
  if (kFp4 && b0 < b1) own = rows_of(p, b0), len_own = cached(p, b0);
  if (kFp4 && p.whole_most) few = most_few_rows<kThreads>(p, b0, b1, own, len_own, sm.parts, G);
  if (kFp4 && tid == 0) sm.few = few;
  int2 mine = make_int2(0, 0);
  for (int b = b0; b < b1; ++b) {
    if (!kFp4 || b > b0) own = rows_of(p, b), len_own = cached(p, b);
    const int nt = few_tiles<kTile>(few, own.n, len_own, G), rt = nt ? (own.n * G + 7) / 8 : 0;
    mine.x += nt * rt;
    mine.y += rt;
    // one CTA tells: the check in all of them cost a call of prompts, whose other kernel
    // waits for this one to end, 11 of 276 us
    if (blockIdx.x == 0 && ((long long)own.n * G > p.most_rows || own.bad || length_bad(p, b)))
      record_status(p.status, kStatusOffsets, 53);
  }
  int2 incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(kFullMask, incl.x, d), y = __shfl_up_sync(kFullMask, incl.y, d);
    if (lane >= d) incl.x += x, incl.y += y;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  int2 before = make_int2(incl.x - mine.x, incl.y - mine.y), sum = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 v = sm.scan[w];
    if (w < warp) before.x += v.x, before.y += v.y;
    sum.x += v.x, sum.y += v.y;
  }
  // Shares are equal in cost: a unit costs kUnitTiles beside its tiles.  Tile i of
  // the unit that is the u-th of the list and has x tiles before it stands at
  // x + u kUnitTiles + kUnitTiles + i on the axis of costs.
  const long long total = (long long)sum.x * p.Hkv, cost = total + (long long)sum.y * p.Hkv * kUnitTiles;
  const int shares = (int)min((long long)gridDim.x, (cost + kMinTiles - 1) / kMinTiles);
  if ((int)blockIdx.x >= shares) return;
  const long long own_at = (long long)before.x * p.Hkv;
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {  // the share's first tile and the next one's
    const long long c = quotient(cost * (blockIdx.x + e), shares);
    long long at = own_at, units = (long long)before.y * p.Hkv;
    const long long from = at + units * kUnitTiles;
    if (c < from || c >= from + (long long)mine.x * p.Hkv + (long long)mine.y * p.Hkv * kUnitTiles) continue;
    for (int b = b0; b < b1; ++b) {
      int n = own.n, len = len_own;
      if (per > 1) n = rows_of(p, b).n, len = cached(p, b);
      const int nt = few_tiles<kTile>(kFp4 ? sm.few : p.few_rows, n, len, G);
      if (!nt) continue;
      const int u = p.Hkv * ((n * G + 7) / 8);
      const long long off = c - (at + units * kUnitTiles);
      if (off < (long long)(nt + kUnitTiles) * u) {
        const long long i = quotient(off, nt + kUnitTiles);
        if (e == 0) sm.first_unit = units + i;
        sm.bound[e] = at + i * nt + max(0ll, off - i * (nt + kUnitTiles) - kUnitTiles);
        break;
      }
      at += (long long)nt * u;
      units += u;
    }
  }
  __syncthreads();
  const long long t_first = sm.bound[0];
  // of this share; none if it is all beside the tiles
  const int tiles = (int)(((int)blockIdx.x + 1 < shares ? sm.bound[1] : total) - t_first);

  bool dead = false;  // producer: a wait gave up, nothing more is copied
  uint32_t issued = 0;
  int k_done = 0;     // tiles of the share in earlier lists
  int tile = 0;                  // consumer: the share's tile that comes next
  uint32_t stage = 0, phase = 0;  // and where it lies
  for (long long base = sm.first_unit; k_done < tiles; base += kItems) {
    // list units base .. base + kItems - 1 and their tiles within the share
    if (k_done) __syncthreads();  // the list before has been used
    if (tid < kItems) sm.end[tid] = 0;
    __syncthreads();
    {
      long long at = own_at, units = (long long)before.y * p.Hkv;
      for (int b = b0; b < b1 && units < base + kItems && at < t_first + tiles; ++b) {
        int row0 = own.row0, n = own.n, len = len_own;
        if (per > 1) {
          const Rows r = rows_of(p, b);
          row0 = r.row0, n = r.n, len = cached(p, b);
        }
        const int nt = few_tiles<kTile>(kFp4 ? sm.few : p.few_rows, n, len, G);
        if (!nt) continue;
        const int rt = (n * G + 7) / 8, u = p.Hkv * rt;
        for (int h = (int)max(0ll, base - units); h < u && units + h < base + kItems; ++h) {
          const long long p0 = at + (long long)h * nt - t_first;
          if (p0 >= tiles) break;
          const int i = (int)(units + h - base);
          sm.item[i] = make_int4(b, h / rt, h % rt * 8, len);
          sm.rows[i] = make_int4(row0, n, max(0, min(n, p.T - row0)), nt);
          sm.begin[i] = (int)p0;
          sm.end[i] = (int)min((long long)tiles, p0 + nt);
        }
        at += (long long)nt * u;
        units += u;
      }
    }
    __syncthreads();
    const int k_end = sm.end[kItems - 1] ? sm.end[kItems - 1] : tiles;  // where this list ends in the share

    if (warp == kWarps) {
      // ---- producer: lane kGroups k + j prepares group j (16 tokens) of the k-th of
      // kRound tiles, then each tile's copies go out as its stage frees.  Page
      // ids are read two rounds ahead and scales one, so that neither
      // latency stands between two rounds.
      constexpr int kGroups = kTile / 16, kRound = 32 / kGroups;
      struct Group {
        int id, tok, h, cnt;
        float ks, vs;
      };
      const int box = min(kTile, 1 << p.page_shift);  // tokens of a copy
      const int k = lane / kGroups, j = lane % kGroups;
      int at_item = 0;  // this lane's unit: its tiles ascend
      auto find = [&](int k0) {
        Group x = {-1, 0, 0, 0, 0.0f, 1.0f};
        if (k0 + k < k_end) {
          while (sm.end[at_item] <= k0 + k) ++at_item;
          const int4 im = sm.item[at_item];
          x.tok = (k0 + k - sm.begin[at_item]) * kTile + 16 * j;
          x.h = im.y;
          x.cnt = max(0, min(16, im.w - x.tok));
          if (x.cnt > 0) x.id = p.table[im.x * p.ld_table + (x.tok >> p.page_shift)];
        }
        return x;
      };
      auto scales = [&](Group& x) {
        if (x.cnt <= 0) return;
        if ((unsigned)x.id >= (unsigned)p.num_pages) {
          record_status(p.status, kStatusOffsets, 50);
          x.cnt = 0;
          return;
        }
        if constexpr (!kFp4) {
          x.ks = static_cast<const float*>(p.k_scales)[(long long)x.id * p.Hkv + x.h];
          x.vs = static_cast<const float*>(p.v_scales)[(long long)x.id * p.Hkv + x.h];
        }
      };
      Group now = find(k_done), next = find(k_done + kRound);
      scales(now);
      uint32_t s = k_done % kStages, ph = (k_done / kStages) & 1;
      for (int k0 = k_done; k0 < k_end; k0 += kRound) {
        scales(next);
        const Group later = find(k0 + 2 * kRound);
        const bool copies = now.cnt > 0 && (16 * j) % box == 0;
        const unsigned copy_mask = __ballot_sync(kFullMask, copies);
        const long long token = (((long long)now.id * p.Hkv + now.h) << p.page_shift) + (now.tok & ((1 << p.page_shift) - 1));
        const int row = (int)(token * kRow / 128);
        const int rounds = min(kRound, k_end - k0);
        const int both = max(now.cnt, 0) | max(__shfl_down_sync(kFullMask, now.cnt, 1), 0) << 8;  // on even lanes
        float log_vs = 0.0f, inv_vs = 0.0f;
        for (int i = 0; i < rounds; ++i) {
          const bool ok = mbar_wait(&sm.empty[s], ph ^ 1, wg, 51);
          dead |= __any_sync(kFullMask, !ok) != 0;
          if (!dead) {
            if (k == i && copies) {
              tma_load_2d(&sm.kv[s][16 * j * kRow], &tm_k, &sm.full[s], 0, row);
              tma_load_2d(&sm.kv[s][(kTile + 16 * j) * kRow], &tm_v, &sm.full[s], 0, row);
            }
            // scales: pieces of 16 bytes that do not pass through the TMA unit, whose requests
            // bound calls on 16-token pages (drafts over 16 heads: 23 us, not 26; 64 requests, D = 64:
            // 62, not 78)
            if (kFp4 && k == i) {
              if (now.cnt > 0) {
                const uint8_t* ks = static_cast<const uint8_t*>(p.k_scales) + token * (D / 16);
                const uint8_t* vs = static_cast<const uint8_t*>(p.v_scales) + token * (D / 16);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                  cp_async16(smem_u32(&sm.scale[s][0][j * D + 16 * x]), ks + 16 * x);
                  cp_async16(smem_u32(&sm.scale[s][1][j * D + 16 * x]), vs + 16 * x);
                }
              }
              asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sm.full[s])) : "memory");
            }
            if (!kFp4 && i == 0) log_vs = log2f(now.vs), inv_vs = 1.0f / now.vs;  // the scales may still be on their way
            if constexpr (kFp4) {
              if (k == i && !(j & 1)) sm.there[s][j >> 1] = both;
            } else {
              if (k == i) sm.group[s][j] = make_float4(now.ks, log_vs, inv_vs, __int_as_float(now.cnt));
            }
            __syncwarp();
            const int n = __popc((copy_mask >> (kGroups * i)) & ((1u << kGroups) - 1));
            if (lane == kGroups * i) mbar_arrive_expect_tx(&sm.full[s], (uint32_t)(n * box * kRow * 2));
            issued = k0 + i + 1;
          }
          if (++s == kStages) s = 0, ph ^= 1;
        }
        now = next;
        next = later;
      }
    } else {
      // ---- consumers: warp w takes tokens 16 w .. + 15 of every tile (of 4 bits 32 w .. + 31)
      const int g = lane >> 2, c = lane & 3;
      constexpr int kQ = D / 64;  // 64-wide parts of a row
      const Fp4At<D> at(warp, lane);
      for (int im = 0; im < kItems; ++im) {
        const int end = sm.end[im];
        if (!end) break;
        const int4 item = sm.item[im], rows = sm.rows[im];
        const int h = item.y, r0 = item.z, len = item.w;  // the unit's rows are r0 .. r0 + 7
        const int row0 = rows.x, n = rows.y, R = min(8, rows.z * G - r0);
        // q row g as a B fragment, fp16 by a power of two
        uint32_t qb[4 * kQ][2];
        float qscale[2];
        int seen[2];
        {
          const int r = r0 + g;
          const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (row0 + r / G) * p.q_tok_stride +
                                   (h * G + r % G) * p.q_head_stride + (kFp4 ? D / 4 : 16) * c;
          uint32_t w[8 * kQ];
#pragma unroll
          for (int x = 0; x < 2 * kQ; ++x) {
            const uint4 v = g < R ? *reinterpret_cast<const uint4*>(q + (kFp4 ? 8 * x : 64 * (x >> 1) + 8 * (x & 1)))
                                  : make_uint4(0, 0, 0, 0);
            w[4 * x] = v.x, w[4 * x + 1] = v.y, w[4 * x + 2] = v.z, w[4 * x + 3] = v.w;
          }
          // the next unit's q on its way to L1 meanwhile
          if (im + 1 < kItems && sm.end[im + 1]) {
            const int4 ni = sm.item[im + 1], nr = sm.rows[im + 1];
            const int rn = ni.z + g;
            if (rn < nr.z * G && c < kQ) {
              const __nv_bfloat16* qn = static_cast<const __nv_bfloat16*>(p.q) + (nr.x + rn / G) * p.q_tok_stride +
                                        (ni.y * G + rn % G) * p.q_head_stride + 64 * c;
              asm volatile("prefetch.global.L1 [%0];" ::"l"(qn));
            }
          }
          float amax = 0.0f;
#pragma unroll
          for (int x = 0; x < 8 * kQ; ++x)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[x] << 16)), fabsf(__uint_as_float(w[x] & 0xffff0000u))));
          amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
          const int up = fp16_up(amax);
          const float mul = exp2i(up);
#pragma unroll
          for (int x = 0; x < 4 * kQ; ++x)  // k step x: columns 64 (x / 4) + 16 c + 4 (x % 4) .. + 3, or (4 bits) D / 4 c + 4 x .. + 3
#pragma unroll
            for (int y = 0; y < 2; ++y)
              qb[x][y] = pack_f16x2(__uint_as_float(w[2 * x + y] << 16) * mul,
                                    __uint_as_float(w[2 * x + y] & 0xffff0000u) * mul);
          // the four warps write the same; none is at the unit after while another reads this one's
          if constexpr (kFp4) {
#pragma unroll
            for (int x = 0; x < D / 32; ++x) sm.q[x][lane] = make_uint4(qb[2 * x][0], qb[2 * x][1], qb[2 * x + 1][0], qb[2 * x + 1][1]);
            __syncwarp();
          }
          const float undo = exp2i(-up) * p.scale_log2;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qscale[e] = __shfl_sync(kFullMask, undo, 4 * (2 * c + e));
            seen[e] = 2 * c + e < R ? len - n + (r0 + 2 * c + e) / G + 1 : 0;
          }
        }
        const int all_seen = len - n + r0 / G + 1;  // tokens that every row sees
        float o[D / 16][4] = {};
        float m[2], l[2] = {0.0f, 0.0f};  // reference and sum of weights of the two rows
        m[0] = m[1] = kFp4 ? kNone : -INFINITY;

        const int begin = sm.begin[im];
        for (; tile < end; ++tile) {
          mbar_wait(&sm.full[stage], phase, wg, 52);
          const float4 sc = kFp4 ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : sm.group[stage][warp];
          // after a wait that gave up, whatever lies here
          const int cnt = kFp4 ? sm.there[stage][warp] & 0x1f1f : min(__float_as_int(sc.w), 16);
          if (cnt <= 0) {
          } else if constexpr (kFp4) {
            fp4_tile<D>(smem_u32(sm.kv[stage]), smem_u32(sm.scale[stage]) + warp * 2 * D, &sm.scale[stage][1][warp * 2 * D], cnt,
                        (tile - begin) * kTile + warp * 32, all_seen, seen, qscale, smem_u32(&sm.q[0][lane]), m, l, o, at, lane);
          } else {
            uint8_t* kt = &sm.kv[stage][warp * 16 * D];
            uint8_t* vt = kt + kTile * D;
            if (cnt < 16) {  // codes behind the last token may stand for NaN
              for (int x = cnt * (D / 16) + lane; x < D; x += 32)
                *reinterpret_cast<uint4*>(vt + code_at<D>(x / (D / 16), x % (D / 16))) = make_uint4(0, 0, 0, 0);
              __syncwarp();
            }
            const int tok0 = (tile - begin) * kTile + warp * 16;
            if (tok0 + cnt > all_seen) {
              uint32_t any = 0;
              for (int x = lane; x < cnt * (D / 16); x += 32) {
                const uint4 w = *reinterpret_cast<const uint4*>(vt + code_at<D>(x / (D / 16), x % (D / 16)));
                any |= nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w);
              }
              if (__any_sync(kFullMask, any)) {
                const uint32_t hit = take_nan<D>(vt, cnt, seen[0] - tok0, seen[1] - tok0, lane);
#pragma unroll
                for (int a = 0; a < D / 16; ++a)
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    if (hit >> (4 * a + x) & 1) o[a][x] = __int_as_float(0x7fffffff);
                __syncwarp();
              }
            }
            float u[4] = {}, u2[4] = {};  // two chains of products
            {
              const int tok = token_of<D>(g);
#pragma unroll
              for (int part = 0; part < kQ; ++part) {
                const uint4 a = *reinterpret_cast<const uint4*>(kt + code_at<D>(tok, 4 * part + c));
                const uint4 b = *reinterpret_cast<const uint4*>(kt + code_at<D>(8 + tok, 4 * part + c));
                const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const uint32_t ka[4] = {e4m3x2_to_f16x2((uint16_t)wa[x]), e4m3x2_to_f16x2((uint16_t)wb[x]),
                                          e4m3x2_to_f16x2((uint16_t)(wa[x] >> 16)), e4m3x2_to_f16x2((uint16_t)(wb[x] >> 16))};
                  mma_f16(x & 1 ? u2 : u, ka, qb[4 * part + x][0], qb[4 * part + x][1]);
                }
              }
            }
            const float f[2] = {qscale[0] * sc.x, qscale[1] * sc.x};
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = fmaf(u[e] + u2[e], f[e & 1], sc.y);
            if (cnt < 16 || tok0 + 16 > all_seen) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tok = 8 * (e >> 1) + token_of<D>(g);
                if (tok >= cnt || tok0 + tok >= seen[e & 1]) u[e] = -INFINITY;
              }
            }
            uint32_t pb[2];
            softmax_step<D / 16>(u, sc.z, m, l, o, pb);
#pragma unroll
            for (int a = 0; a < D / 32; ++a) {
              // lanes 8 i .. + 7 give the rows of matrix i: tokens 8 (i % 2) .. + 7 at 16-byte chunk 2 a + i / 2
              uint32_t v[4];
              const int tok = 8 * ((lane >> 3) & 1) + token_of<D>(lane & 7);
              ldmatrix_x4_trans(v, smem_u32(vt + code_at<D>(tok, 2 * a + (lane >> 4))));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                // a pair of codes (columns 2 g, 2 g + 1) of two tokens each: to pairs of tokens
                const uint32_t w0 = __byte_perm(v[2 * x], 0, 0x3120), w1 = __byte_perm(v[2 * x + 1], 0, 0x3120);
                const uint32_t va[4] = {e4m3x2_to_f16x2((uint16_t)w0), e4m3x2_to_f16x2((uint16_t)(w0 >> 16)),
                                        e4m3x2_to_f16x2((uint16_t)w1), e4m3x2_to_f16x2((uint16_t)(w1 >> 16))};
                mma_f16(o[2 * a + x], va, pb[0], pb[1]);
              }
            }
            if (cnt < 16 || tok0 + cnt > all_seen) fence_proxy_async_smem();  // the zeros, before the next copy into this stage
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.empty[stage]);
          if (++stage == kStages) stage = 0, phase ^= 1;
        }

        if constexpr (kFp4) {
#pragma unroll
          for (int e = 0; e < 2; ++e) m[e] = m[e] == kNone ? -INFINITY : m[e];
        }
        // ---- the warps' (m, l, o) to one: o[a] holds columns 16 a + 2 g and + 1
        // (e / 2) of rows 2 c and + 1 (e % 2); of 4 bits, columns D / 8 g + 2 a and + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(kFullMask, l[e], d);
          if (g == 0) sm.ml[warp][2 * c + e] = make_float2(m[e], l[e]);
        }
        consumer_sync();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.ml[w][2 * c + e].x);
          const float f = ex2(m[e] - (M == -INFINITY ? 0.0f : M));
#pragma unroll
          for (int a = 0; a < D / 16; ++a) o[a][e] *= f, o[a][2 + e] *= f;
        }
        float* buf = sm.red[warp % (kWarps / 2)];
        // the lane's columns, by as many as lie side by side
        auto each = [&](auto&& f) {
          if constexpr (kFp4) {
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float* at = buf + red_at<D, true>(2 * c + e, D / 8 * g + 4 * x);
                f(reinterpret_cast<float4*>(at), o[2 * x][e], o[2 * x][2 + e], o[2 * x + 1][e], o[2 * x + 1][2 + e]);
              }
          } else {
            float none = 0.0f;
#pragma unroll
            for (int a = 0; a < D / 16; ++a)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                f(reinterpret_cast<float2*>(buf + red_at<D, false>(2 * c + e, 16 * a + 2 * g)), o[a][e], o[a][2 + e], none, none);
          }
        };
        auto put = [&] { each([](auto* at, float x, float y, float z, float w) { store_floats(at, x, y, z, w); }); };
        if (warp >= kWarps / 2) put();
        consumer_sync();
        if (warp < kWarps / 2) {
          each([](const auto* at, float& x, float& y, float& z, float& w) { add_floats(at, x, y, z, w); });
          put();
        }
        consumer_sync();
        const int nt = rows.w;
        const bool starts = begin >= 0, alone = starts && end == begin + nt;
        // a unit cut between CTAs: this piece goes to the workspace, the last
        // CTA to finish one joins the pieces in order
        float* slot = p.work + ((long long)blockIdx.x * 2 + starts) * (8 * (D + 2));
        for (int x = tid * 4; x < R * D; x += kWarps * 128) {
          const int r = x / D, d = x % D;
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kWarps / 2; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.red[w][red_at<D, kFp4>(r, d)]);
            y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
          }
          float M = -INFINITY, L = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.ml[w][r].x);
          const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) L += sm.ml[w][r].y * ex2(sm.ml[w][r].x - ref);
          if (alone) {
            const float inv = L > 0.0f ? 1.0f / L : 0.0f;
            const long long tr = row0 + (r0 + r) / G;
            const int hq = h * G + (r0 + r) % G;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + tr * p.out_tok_stride + hq * p.out_head_stride + d;
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
            if (d == 0 && p.lse) p.lse[tr * p.Hq + hq] = lse_of(M, L);
          } else {
            *reinterpret_cast<float4*>(slot + x) = y;
            if (d == 0) *reinterpret_cast<float2*>(slot + 8 * D + 2 * r) = make_float2(M, L);
          }
        }
        if (alone) {
          consumer_sync();  // ml and red have been read
          continue;
        }
        // the shares that hold the unit's first and last tile
        const long long first = t_first + begin + (base + im + 1) * kUnitTiles;  // on the axis of costs
        const int c0 = (int)quotient((first + 1) * shares - 1, cost), c1 = (int)quotient((first + nt) * shares - 1, cost);
        consumer_sync();
        if (tid == 0) {
          sm.last = arrive_piece(p.counters + c0) == c1 - c0;
          if (sm.last) p.counters[c0] = 0;
        }
        consumer_sync();
        if (sm.last) {
          for (int r = warp; r < R; r += kWarps) {
            // the first pieces are on their way while the maximum over all is found (drafts over 16
            // heads 21.1 us, not 21.6)
            constexpr int kAhead = 4;
            float2 first_ml[kAhead];
            float first_o[kAhead][D / 32];
#pragma unroll
            for (int y = 0; y < kAhead; ++y) {
              const float* from = p.work + piece_at<D>(min(c0 + y, c1), c0);
              first_ml[y] = __ldcg(reinterpret_cast<const float2*>(from + 8 * D + 2 * r));
#pragma unroll
              for (int d = 0; d < D / 32; ++d) first_o[y][d] = __ldcg(from + r * D + 32 * d + lane);
            }
            float mx = -INFINITY;
            for (int x = c0 + lane; x <= c1; x += 32) mx = fmaxf(mx, __ldcg(p.work + piece_at<D>(x, c0) + 8 * D + 2 * r));
#pragma unroll
            for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, d));
            const float ref = mx == -INFINITY ? 0.0f : mx;
            float acc[D / 32] = {}, sum_l = 0.0f;
#pragma unroll
            for (int y = 0; y < kAhead; ++y) {
              if (c0 + y > c1) break;
              const float f = ex2(first_ml[y].x - ref);
              sum_l += first_ml[y].y * f;
#pragma unroll
              for (int d = 0; d < D / 32; ++d) acc[d] += f * first_o[y][d];
            }
#pragma unroll 4
            for (int x = c0 + kAhead; x <= c1; ++x) {
              const float* from = p.work + piece_at<D>(x, c0);
              const float2 e = __ldcg(reinterpret_cast<const float2*>(from + 8 * D + 2 * r));
              const float f = ex2(e.x - ref);
              sum_l += e.y * f;
#pragma unroll
              for (int d = 0; d < D / 32; ++d) acc[d] += f * __ldcg(from + r * D + 32 * d + lane);
            }
            const float inv = sum_l > 0.0f ? 1.0f / sum_l : 0.0f;
            const long long tr = row0 + (r0 + r) / G;
            const int hq = h * G + (r0 + r) % G;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + tr * p.out_tok_stride + hq * p.out_head_stride + lane;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) dst[32 * d] = __float2bfloat16(acc[d] * inv);
            if (lane == 0 && p.lse) p.lse[tr * p.Hq + hq] = lse_of(mx, sum_l);
          }
        }
      }
    }
    k_done = k_end;
  }
  // after a wait that gave up, the producer's or a consumer's: copies in flight
  // land before the CTA's memory goes
  __syncthreads();
  if (warp == kWarps && *wg.abort_flag)
    for (uint32_t k = issued > kStages ? issued - kStages : 0; k < issued; ++k)
      mbar_drain(&sm.full[k % kStages], (k / kStages) & 1, 100000000ull);
}

template <int D, bool kFp4>
cudaError_t launch_few(const KvAttentionLaunch& L, cudaStream_t stream) {
  constexpr int kSmem = (int)sizeof(FewSmem<D, kFp4>) + 1024;
  static_assert(kFewCtas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
  return launch_kernel_smem(kv_attention_few_kernel<D, kFp4>, (unsigned)L.few_grid, kFewThreads, kSmem, stream, L.tm_k, L.tm_v,
                            L.p);
}

}  // namespace

int kv_attention_few_grid(int sms) { return kFewCtas * sms < kCounters ? kFewCtas * sms : kCounters; }
size_t kv_attention_piece_bytes(int D) { return (size_t)2 * 8 * (D + 2) * sizeof(float); }
int kv_attention_box(int page_size, bool fp4) { return min(page_size, fp4 ? kTileOf<true> : kTileOf<false>); }

cudaError_t launch_kv_attention(const KvAttentionLaunch& L, cudaStream_t stream) {
  const KvAttentionParams& p = L.p;
  const int G = p.Hq / p.Hkv;
  if (G <= p.few_rows) {
    cudaError_t e = p.fp4 ? (p.D == 64 ? launch_few<64, true>(L, stream) : launch_few<128, true>(L, stream))
                          : (p.D == 64 ? launch_few<64, false>(L, stream) : launch_few<128, false>(L, stream));
    if (e != cudaSuccess) return e;
  }
  if (L.few_only) return cudaSuccess;
  return launch_kv_attention_rows(L, stream);
}

}  // namespace bsk
