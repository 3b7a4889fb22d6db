// matvec_fp4.cu -- a few bf16 rows times FP4 weights:
//   y[m, n] = alpha * ts * sum_k x[m, k] * e2m1[n, k] * sf[n, k / 16] + bias[n]
// with the codes and MMA-layout group scales that q4_quantize writes and the
// activations left in bf16.
//
// Bound by the weight stream (9/16 byte a weight).  A weight times its group
// scale has at most 6 significant bits and lies in [2^-10, 2688], so it is
// exact in fp16; x is brought to fp16 by a power of two per (row, phase of K)
// that puts the largest element in [2^14, 2^15): exact for every
// element within 2^-29 of it, and 2^-40 of it is the error of the others.
// The products go through mma.sync m16n8k16 with the 16 weight rows on its M
// and 8 (or 2 x 8) x rows on its N, accumulated in fp32.
//
// Work: one CTA per SM walks a contiguous share of the 16-row weight tiles, two
// at a time; its 16 warps split K, 2 chunks of 128 each (K <= 4096 in one phase,
// longer K in several).  A warp keeps its slice of x as MMA fragments in
// registers for all its tiles, so x is read once per CTA and never passes
// shared memory.  Every lane copies the 48 bytes a chunk that it will itself
// use (16 bytes of codes of two rows, 16 of scales) with cp.async into a ring of
// its own: three tiles (147 KB an SM) in flight without registers or barriers.
// The warps' partial tiles are added in warp order through shared memory.
#include "kernels.h"
#include "ptx.cuh"

namespace bsk {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kCh = 2;                     // chunks of 128 K per warp and phase
constexpr int kPhaseChunks = kWarps * kCh;
constexpr int kStages = 3;                 // tiles in flight
constexpr int kUnit = kThreads * 16;       // a 16-byte unit of every lane
constexpr int kStageBytes = kCh * 3 * kUnit;
constexpr int kPart = 16 * 16;             // floats of a warp's partial tile
constexpr int kTurn = 2 * kWarps * kPart;  // two tiles' partials
constexpr int kBlockTiles = 15;            // tiles whose sums are kept between phases
constexpr int kAmaxBytes = 2 * 16 * 4;     // per x row, of this phase and the next
constexpr int kSmem = kStages * kStageBytes + 2 * kTurn * 4 + kAmaxBytes;
constexpr int kSmemPhases = kSmem + kBlockTiles * kPart * 4;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four bytes of E2M1 pairs as f16x2
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Tile t: 16 rows 128 (t / 8) + 4 (t % 8) + (i % 4) + 32 (i / 4), i = 0 .. 15,
// whose scales of a 64-wide K chunk are 64 consecutive bytes.  Lane 4 g + c
// holds rows i = g and g + 8 and, of each chunk of 128, the 32 columns from
// 32 c on; MMA step s takes columns 32 c + 4 s .. + 3 of each lane, the same
// for codes and x, so neither is shuffled.  Rows from N on repeat row N - 1 and
// are not written; where K ends in half a chunk, the lanes past it repeat the
// half's codes and scales against x fragments of zero.
//
// A partial tile is [row][pair of x rows], 8 bytes a pair, pairs 0-3 and 4-7
// exchanged in rows 2, 3, 6, 7, ..: neither the fragments' stores nor the sums'
// loads meet a bank twice.
template <int NT>  // tiles of 8 x rows
__global__ void __launch_bounds__(kThreads, 1) fp4_matvec_kernel(const __grid_constant__ Fp4MatvecParams p, int tiles) {
  extern __shared__ __align__(16) uint8_t smem[];
  float2* parts = reinterpret_cast<float2*>(smem + kStages * kStageBytes);
  int* amaxes = reinterpret_cast<int*>(smem + kStages * kStageBytes + 2 * kTurn * 4);  // [2][16] fp32 bits
  float2* sums = reinterpret_cast<float2*>(smem + kSmem);  // [kBlockTiles][16][8], several phases only
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem) + tid * 16;
  const int t_first = (int)((long long)tiles * blockIdx.x / gridDim.x);
  const int t_last = (int)((long long)tiles * (blockIdx.x + 1) / gridDim.x);
  const int chunks = (p.K + 127) / 128, phases = (chunks + kPhaseChunks - 1) / kPhaseChunks;
  const int blocks = phases == 1 ? 1 : (t_last - t_first + kBlockTiles - 1) / kBlockTiles;
  const long long row_bytes = p.K / 2;
  int turn = 0;     // which half of parts
  int amax_at = 0;  // which half of amaxes
  if (tid < 32) amaxes[tid] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  for (int blk = 0; blk < blocks; ++blk) {
    const int t0 = t_first + (int)((long long)(t_last - t_first) * blk / blocks);
    const int t1 = t_first + (int)((long long)(t_last - t_first) * (blk + 1) / blocks);
    for (int ph = 0; ph < phases; ++ph) {
      // the phase's chunks, in warp order, as even as they go
      const int in_phase = min(chunks - ph * kPhaseChunks, kPhaseChunks);
      const int ch0 = ph * kPhaseChunks + in_phase * warp / kWarps;
      const int n_ch = ph * kPhaseChunks + in_phase * (warp + 1) / kWarps - ch0;
      // the chunk that is half a chunk: its upper lanes read 32 columns back
      const int half = p.K % 128 && ch0 + n_ch == chunks && c >= 2 ? n_ch - 1 : kCh;

      // where the next tile to be copied lies for this lane; N's last block of
      // 128 rows, if it is not whole, is addressed anew for each tile
      const int whole = p.N / 128 * 8;
      const uint8_t *lo, *hi, *sf;
      auto locate = [&](int t) {
        const int r0 = 128 * (t >> 3) + 4 * (t & 7) + (g & 3) + 32 * (g >> 2);
        lo = p.codes + min(r0, p.N - 1) * row_bytes + (long long)ch0 * 64 + c * 16;
        hi = p.codes + min(r0 + 64, p.N - 1) * row_bytes + (long long)ch0 * 64 + c * 16;
        sf = p.sf + ((long long)(t >> 3) * (p.K / 64) + 2 * ch0 + (c >> 1)) * 512 + (4 * (t & 7) + (g & 3)) * 16;
      };
      auto issue = [&](int t, int stage) {
        if (t < t1) {
          const uint32_t dst = ring + stage * kStageBytes;
#pragma unroll
          for (int i = 0; i < kCh; ++i) {
            if (i >= n_ch) break;
            const int back = i == half ? 32 : 0;
            cp_async16(dst + (3 * i) * kUnit, lo + (i * 64 - back));
            cp_async16(dst + (3 * i + 1) * kUnit, hi + (i * 64 - back));
            cp_async16(dst + (3 * i + 2) * kUnit, sf + (i * 1024 - 16 * back));
          }
          if (t + 1 >= whole) {
            locate(t + 1);
          } else {
            const bool next = (t & 7) == 7;
            const long long step = (next ? 128 - 28 : 4) * row_bytes;
            lo += step;
            hi += step;
            sf += next ? (long long)(p.K / 64) * 512 - 7 * 64 : 64;
          }
        }
        cp_async_commit();
      };
      locate(t0);
#pragma unroll
      for (int s = 0; s < kStages; ++s) issue(t0 + s, s);

      // this warp's slice of x as B fragments, brought to fp16 by a power of
      // two that all warps share
      uint32_t xb[kCh][NT][16];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int m = 8 * j + g;
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + m * p.ldx + c * 32;
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          const bool in = m < p.M && i < n_ch && (ch0 + i) * 128 + c * 32 < p.K;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 v = in ? reinterpret_cast<const uint4*>(x + (ch0 + i) * 128)[q] : make_uint4(0, 0, 0, 0);
            xb[i][j][4 * q] = v.x, xb[i][j][4 * q + 1] = v.y, xb[i][j][4 * q + 2] = v.z, xb[i][j][4 * q + 3] = v.w;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kCh; ++i)
#pragma unroll
          for (int q = 0; q < 16; ++q)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(xb[i][j][q] << 16)),
                                     fabsf(__uint_as_float(xb[i][j][q] & 0xffff0000u))));
        amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
        if (c == 0 && amax > 0.0f) atomicMax(&amaxes[amax_at + 8 * j + g], __float_as_int(amax));
      }
      __syncthreads();
      if (tid < 16) amaxes[(amax_at ^ 16) + tid] = 0;  // read last before this phase's first barrier
      // up = 14 - floor(log2 amax), at most 126
      auto up_of = [&](int m) {
        const int bits = amaxes[amax_at + m];
        return bits ? 14 - min(max((bits >> 23) - 127, -112), 127) : 0;
      };
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float mul = __uint_as_float((uint32_t)(up_of(8 * j + g) + 127) << 23);
#pragma unroll
        for (int i = 0; i < kCh; ++i)
#pragma unroll
          for (int q = 0; q < 16; ++q)
            xb[i][j][q] = pack_f16x2(__uint_as_float(xb[i][j][q] << 16) * mul,
                                     __uint_as_float(xb[i][j][q] & 0xffff0000u) * mul);
      }

      int stage = 0;
      for (int t = t0; t < t1; ++t) {
        cp_async_wait<kStages - 1>();  // this lane's copies for tile t have landed
        float acc[NT][4] = {};
        const uint32_t src0 = ring + stage * kStageBytes;
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
          if (i >= n_ch) break;
          const uint32_t src = src0 + 3 * i * kUnit;
          const uint4 cl4 = lds128(src), ch4 = lds128(src + kUnit), sc = lds128(src + 2 * kUnit);
          // scale words: row quarters g / 4 and g / 4 + 2, bytes 2 (c % 2) and + 1
          const uint32_t pick = (c & 1) ? 0x7632 : 0x5410;
          const uint32_t w = __byte_perm((g >> 2) ? sc.y : sc.x, (g >> 2) ? sc.w : sc.z, pick);
          const uint32_t sl = e4m3x2_to_f16x2((uint16_t)w), sh = e4m3x2_to_f16x2((uint16_t)(w >> 16));
          const uint32_t cl[4] = {cl4.x, cl4.y, cl4.z, cl4.w}, ch[4] = {ch4.x, ch4.y, ch4.z, ch4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t s0 = __byte_perm(sl, 0, q < 2 ? 0x1010 : 0x3232);
            const uint32_t s1 = __byte_perm(sh, 0, q < 2 ? 0x1010 : 0x3232);
            uint32_t l[4], h[4];
            e2m1x8_to_f16(cl[q], l);
            e2m1x8_to_f16(ch[q], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) l[e] = hmul2(l[e], s0), h[e] = hmul2(h[e], s1);
#pragma unroll
            for (int e = 0; e < 4; e += 2)
#pragma unroll
              for (int j = 0; j < NT; ++j)
                mma_f16(acc[j], l[e], h[e], l[e + 1], h[e + 1], xb[i][j][4 * q + e], xb[i][j][4 * q + e + 1]);
          }
        }
        issue(t + kStages, stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        const int which = (t - t0) & 1;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          // pair 4 j + c, with the rows' exchange
          float2* at = parts + (turn * kTurn + (which * kWarps + warp) * kPart) / 2 + g * 8 + ((4 * j + c) ^ ((g & 2) << 1));
          at[0] = make_float2(acc[j][0], acc[j][1]);
          at[64] = make_float2(acc[j][2], acc[j][3]);
        }
        if (which == 0 && t + 1 < t1) continue;
        __syncthreads();  // both tiles' partials are there, and the other half of parts has been read
        const int tile = tid >> 7, i = (tid >> 3) & 15, pair = tid & 7, tt = t - which + tile;
        if (tile <= which && 2 * pair < p.M) {
          const float2* all = parts + (turn * kTurn + tile * kWarps * kPart) / 2 + i * 8 + (pair ^ ((i & 2) << 1));
          float2 y = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 v = all[w * kPart / 2];
            y.x += v.x, y.y += v.y;
          }
          y.x *= __uint_as_float((uint32_t)(127 - up_of(2 * pair)) << 23);
          y.y *= __uint_as_float((uint32_t)(127 - up_of(2 * pair + 1)) << 23);
          float2* kept = sums + (tt - t0) * (kPart / 2) + i * 8 + pair;
          if (ph > 0) y.x += kept->x, y.y += kept->y;
          const int n = 128 * (tt >> 3) + 4 * (tt & 7) + (i & 3) + 32 * (i >> 2);
          if (ph + 1 < phases) {
            *kept = y;
          } else if (n < p.N) {
            const float a = p.alpha * (p.tensor_scale ? *p.tensor_scale : 1.0f);
            const float bias = p.bias ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[n]) : 0.0f;
            y.x = fmaf(a, y.x, bias), y.y = fmaf(a, y.y, bias);
            const long long at = 2 * pair * p.ldo + n;
            if (p.out_bf16) {
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
              o[0] = __float2bfloat16(y.x);
              if (2 * pair + 1 < p.M) o[p.ldo] = __float2bfloat16(y.y);
            } else {
              float* o = static_cast<float*>(p.out) + at;
              o[0] = y.x;
              if (2 * pair + 1 < p.M) o[p.ldo] = y.y;
            }
          }
        }
        turn ^= 1;
      }
      cp_async_wait<0>();
      amax_at ^= 16;
    }
  }
}

template <int NT>
cudaError_t launch(const Fp4MatvecParams& p, int sms, cudaStream_t stream) {
  static const cudaError_t attr =
      cudaFuncSetAttribute(fp4_matvec_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPhases);
  if (attr != cudaSuccess) return attr;
  const int tiles = (p.N + 127) / 128 * 8;
  const bool phases = p.K > kPhaseChunks * 128;
  return launch_kernel(fp4_matvec_kernel<NT>, (unsigned)(tiles < sms ? tiles : sms), kThreads,
                       phases ? kSmemPhases : kSmem, stream, 1, p, tiles);
}

}  // namespace

cudaError_t launch_fp4_matvec(const Fp4MatvecParams& p, int sms, cudaStream_t stream) {
  return p.M <= 8 ? launch<1>(p, sms, stream) : launch<2>(p, sms, stream);
}

}  // namespace bsk
