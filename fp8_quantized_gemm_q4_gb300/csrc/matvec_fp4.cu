// matvec_fp4.cu -- a few bf16 rows times FP4 weights:
//   y[m, n] = alpha * ts * sum_k x[m, k] * e2m1[n, k] * sf[n, k / 16] + bias[n]
// with the codes and MMA-layout group scales that q4_quantize writes and the
// activations left in bf16.
//
// Bound by the weight stream (9/16 byte a weight).  A weight times its group
// scale has at most 6 significant bits and lies in [2^-10, 2688], so it is
// exact in fp16; x is brought to fp16 by a power of two per row that puts the
// largest element in [2^14, 2^15): exact for every element within 2^-29 of it,
// and 2^-39 of it bounds the error of the others.  The products go through mma.sync
// m16n8k16 with 16 weight rows on its M and 8 (or 2 x 8) x rows on its N,
// accumulated in fp32.  With so few rows tcgen05 has nothing to gain: its
// M = 128 tile takes the same 64 clocks per 16 of K for 16 columns as for 128,
// 35 us for N = 40960, K = 7168 against 16 us here (built and measured: 96 us
// with the widening warps beside it).
//
// One CTA per SM has a contiguous share of the 16-row weight tiles.  Every lane
// copies the 48 bytes of a tile's chunk (128 of K) that it will itself use (16
// bytes of codes of two rows, 16 of scales) with cp.async into a ring of its
// own, so 100 to 170 KB an SM are in flight without registers or barriers.  Two
// ways to share a CTA's tiles and K among its 16 warps:
//
//   few tiles: all warps split K, the tiles are the only loop; x stays in
//   registers, the warps' partial tiles are added in warp order through shared
//   memory.  Up to K = 4096.
//
//   many tiles: K is the outer loop, 4 x 4 warps share tiles and K and keep the
//   sums of up to five tiles each in registers until the end; x passes through
//   shared memory once.
//
// The second pays a pass over x for its largest elements and the join at the
// end, and needs tiles for its warps; the first pays the join for every tile.
// us, few / many (16-row tiles per SM in brackets):
//   M = 1,  N = 7168,  K = 4096 (3)   7.4 /  9.4   M = 16, 4096 x 1024 (1.7)    6.3 /  6.2
//   M = 4,  N = 10000, K = 4096 (4)  10.2 / 12.6   M = 16, 7168 x 4096 (3)     11.8 / 12.8
//   M = 8,  N = 20000, K = 4096 (8)  16.0 / 15.5   M = 16, 28672 x 4096 (12)   26.1 / 22.8
//   M = 8,  N = 40960, K = 7168 (17)   53 / 35     M = 16, 40960 x 7168 (17)     73 / 48
// So: many from 8 tiles per SM on, and for K above 4096.  At 16 rows neither HBM
// (0.48), the issue slots (0.47) nor the tensor pipe (0.33) is full: four warps a
// scheduler wait for their own chains from ring to product.  Registers are at their
// limit of 128; 144 bytes a thread are spilled in the first kernel at 9 to 16 rows, 36
// in the second.
#include "decode.cuh"
#include "decode.h"

namespace bsk {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kCh = 2;                     // chunks of 128 K per warp
constexpr int kMostChunks = kWarps * kCh;   // K <= 4096
constexpr int kStages = 3;                 // tiles in flight
constexpr int kUnit = kThreads * 16;       // a 16-byte unit of every lane
constexpr int kStageBytes = kCh * 3 * kUnit;
constexpr int kPart = 16 * 16;             // floats of a warp's partial tile
constexpr int kTurn = 2 * kWarps * kPart;  // two tiles' partials
constexpr int kSmem = kStages * kStageBytes + 2 * kTurn * 4 + 16 * 4;

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
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Row i = 0 .. 15 of tile t, whose scales of 64 of K are 64 consecutive bytes
__device__ __forceinline__ int tile_row(int t, int i) { return 128 * (t >> 3) + 4 * (t & 7) + (i & 3) + 32 * (i >> 2); }

// up, the power of two for x: 14 - floor(log2 amax) of the fp32 exponent given, at most 126
__device__ __forceinline__ int up_of_exponent(int e) { return 14 - min(max(e - 127, -112), 127); }

// A tile's chunk: lane 4 g + c holds rows g and g + 8 of the tile and the 32
// columns from 32 c on (codes lo and hi), and the scales of rows g % 4 + 4 x of
// 64 columns; MMA step s takes columns 32 c + 4 s .. + 3 of each lane, the same for
// codes and x, so neither is shuffled.
template <int NT>
__device__ __forceinline__ void multiply(uint4 lo, uint4 hi, uint4 sf, int g, int c, const uint32_t (&xb)[NT][16],
                                         float (&acc)[NT][4]) {
  // scale words: row quarters g / 4 and g / 4 + 2, bytes 2 (c % 2) and + 1
  const uint32_t pick = (c & 1) ? 0x7632 : 0x5410;
  const uint32_t w = __byte_perm((g >> 2) ? sf.y : sf.x, (g >> 2) ? sf.w : sf.z, pick);
  const uint32_t sl = e4m3x2_to_f16x2((uint16_t)w), sh = e4m3x2_to_f16x2((uint16_t)(w >> 16));
  const uint32_t cl[4] = {lo.x, lo.y, lo.z, lo.w}, ch[4] = {hi.x, hi.y, hi.z, hi.w};
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
        mma_f16(acc[j], l[e], h[e], l[e + 1], h[e + 1], xb[j][4 * q + e], xb[j][4 * q + e + 1]);
  }
}

// Few tiles.  Rows from N on repeat row N - 1 and are not written; where K ends in
// half a chunk, the lanes past it repeat the half's codes and scales against x
// fragments of zero.
//
// A partial tile is [row][pair of x rows], 8 bytes a pair, pairs 0-3 and 4-7
// exchanged in rows 2, 3, 6, 7, ..: neither the fragments' stores nor the sums'
// loads meet a bank twice.
template <int NT>  // tiles of 8 x rows
__global__ void __launch_bounds__(kThreads, 1) fp4_matvec_few_kernel(const __grid_constant__ Fp4MatvecParams p, int tiles) {
  extern __shared__ __align__(16) uint8_t smem[];
  float2* parts = reinterpret_cast<float2*>(smem + kStages * kStageBytes);
  int* amaxes = reinterpret_cast<int*>(smem + kStages * kStageBytes + 2 * kTurn * 4);  // [16] fp32 bits
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem) + tid * 16;
  const int t0 = (int)((long long)tiles * blockIdx.x / gridDim.x);
  const int t1 = (int)((long long)tiles * (blockIdx.x + 1) / gridDim.x);
  const int chunks = (p.K + 127) / 128;
  const long long row_bytes = p.K / 2;
  int turn = 0;  // which half of parts
  if (tid < 16) amaxes[tid] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  // chunks in warp order, as even as they go
  const int ch0 = chunks * warp / kWarps, n_ch = chunks * (warp + 1) / kWarps - ch0;
  // the chunk that is half a chunk: its upper lanes read 32 columns back
  const int half = p.K % 128 && ch0 + n_ch == chunks && c >= 2 ? n_ch - 1 : kCh;

  // where the next tile to be copied lies for this lane; N's last block of
  // 128 rows, if it is not whole, is addressed anew for each tile
  const int whole = p.N / 128 * 8;
  const uint8_t *lo, *hi, *sf;
  auto locate = [&](int t) {
    const int r0 = tile_row(t, g);
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
    if (c == 0 && amax > 0.0f) atomicMax(&amaxes[8 * j + g], __float_as_int(amax));
  }
  __syncthreads();
  auto up_of = [&](int m) { return amaxes[m] ? up_of_exponent(amaxes[m] >> 23) : 0; };
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
      multiply(lds128(src), lds128(src + kUnit), lds128(src + 2 * kUnit), g, c, xb[i], acc);
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
      const int n = 128 * (tt >> 3) + 4 * (tt & 7) + (i & 3) + 32 * (i >> 2);
      if (n < p.N) {
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
}

// Many tiles.  Warp (rg, kp) of 4 x 4 takes every fourth tile and every fourth
// chunk of K; a share of more than 20 tiles is walked in blocks.
constexpr int kRg = 4, kKp = 4;            // row groups, parts of K
constexpr int kOwn = 5;                    // tiles of a warp
constexpr int kRingBytes = 3 * 32 * 16;    // a tile's chunk
constexpr int kXRow = 256;                 // a row's chunk of x in fp16

constexpr int many_slots(int nt) { return nt == 1 ? 7 : 5; }  // chunks in flight a warp: whole steps of its tiles

template <int NT>
struct ManySmem {
  uint8_t ring[kWarps][many_slots(NT)][kRingBytes];
  uint8_t x[kKp][2][8 * NT * kXRow];
  int amax[16];
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) fp4_matvec_many_kernel(const __grid_constant__ Fp4MatvecParams p, int tiles) {
  extern __shared__ __align__(16) uint8_t smem[];
  ManySmem<NT>& sm = *reinterpret_cast<ManySmem<NT>*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int rg = warp >> 2, kp = warp & 3;  // the warps of an SM quarter differ in rg: its share is even
  const int t_first = (int)((long long)tiles * blockIdx.x / gridDim.x);
  const int t_last = (int)((long long)tiles * (blockIdx.x + 1) / gridDim.x);
  const int blocks = (t_last - t_first + kRg * kOwn - 1) / (kRg * kOwn);
  const int chunks = (p.K + 127) / 128, steps = (chunks - kp + kKp - 1) / kKp;
  const long long row_bytes = p.K / 2;
  const uint32_t ring = smem_u32(sm.ring[warp]) + lane * 16;
  if (tid < 16) sm.amax[tid] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  for (int blk = 0; blk < blocks; ++blk) {
    const int t0 = t_first + (int)((long long)(t_last - t_first) * blk / blocks);
    const int t1 = t_first + (int)((long long)(t_last - t_first) * (blk + 1) / blocks);
    const int nt = t1 - t0, mine = (nt - rg + kRg - 1) / kRg;
    // Where this lane's bytes of a chunk lie: rows from N on repeat row N - 1 and
    // are not written; where K ends in half a chunk the lanes past it read the
    // half's, against x of zero.
    const int n0 = 128 * (t0 >> 3);
    const uint8_t* code_at = p.codes + n0 * row_bytes + kp * 64 + c * 16;
    const uint8_t* sf_at = p.sf + (long long)(t0 >> 3) * (p.K / 64) * 512 + (2 * kp + (c >> 1)) * 512 + (g & 3) * 16;
    const uint32_t sf_block = (uint32_t)(p.K / 64) * 512u;  // scales of 128 rows
    const uint32_t far = 64u * (uint32_t)row_bytes, last = (uint32_t)min(p.N - 1 - n0, 1023) * (uint32_t)row_bytes;
    uint32_t lo[kOwn], sf[2];
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      lo[i] = (uint32_t)(min(tile_row(t0 + rg + kRg * i, g), p.N - 1) - n0) * (uint32_t)row_bytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + rg + kRg * i;
      sf[i] = (uint32_t)((t >> 3) - (t0 >> 3)) * sf_block + (t & 7) * 64;
    }
    const bool half = (p.K & 127) && c >= 2 && (steps - 1) * kKp + kp == chunks - 1;
    int copied = 0;  // steps whose copies have been issued
    const uint32_t depth = many_slots(NT) / max(mine, 1), ring_end = ring + depth * mine * kRingBytes;
    auto copy = [&](int i, uint32_t dst) {
      if (copied < steps) {
        cp_async16(dst, code_at + lo[i]);
        cp_async16(dst + 512, code_at + min(lo[i] + far, last));
        cp_async16(dst + 1024, sf_at + (sf[i & 1] + (i >> 1) * sf_block));
      }
      cp_async_commit();
    };
    auto next_step = [&]() {
      ++copied;
      code_at += kKp * 64;
      sf_at += kKp * 1024;
      if (half && copied == steps - 1) code_at -= 32, sf_at -= 512;
    };
    if (half && steps == 1) code_at -= 32, sf_at -= 512;
    uint32_t slot = ring;
#pragma unroll 1
    for (uint32_t d = 0; d < depth; ++d) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (i < mine) copy(i, slot), slot += kRingBytes;
      next_step();
    }
    slot = ring;

    if (blk == 0) {
      const int each = p.M <= 1 ? 16 : p.M <= 2 ? 8 : p.M <= 4 ? 4 : p.M <= 8 ? 2 : 1;  // warps a row
      const int m = warp / each;
      if (m < p.M) {
        const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + m * p.ldx);
        __nv_bfloat162 top = __float2bfloat162_rn(0.0f);
#pragma unroll 8
        for (int i = warp % each * 32 + lane; i < p.K / 8; i += 32 * each) {
          const uint4 v = x[i];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
        }
        const uint32_t bits = *reinterpret_cast<const uint32_t*>(&top);
        const int amax = (int)__reduce_max_sync(kFullMask, max(bits & 0xffffu, bits >> 16));
        if (lane == 0) atomicMax(&sm.amax[m], amax);
      }
      __syncthreads();
    }
    auto up_of = [&](int m) { return sm.amax[m] ? up_of_exponent(sm.amax[m] >> 7) : 0; };
    // x passes to fp16 in shared memory, 8 columns of NT rows a thread of the part
    const int xt = rg * 32 + lane, v = xt & 15;
    uint4 xv[NT];
    float mul[NT];
    auto load_x = [&](int s) {
      const int col = (s * kKp + kp) * 128 + v * 8;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int m = 8 * j + (xt >> 4);
        xv[j] = m < p.M && col < p.K && s < steps
                    ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.x) + m * p.ldx + col)
                    : make_uint4(0, 0, 0, 0);
      }
    };
    auto store_x = [&](int s) {
      // chunks of 16 bytes exchanged so that neither these nor the fragments' loads meet a bank twice
      const int m = xt >> 4, q = (v & 3) ^ (2 * (m & 1) + (v >> 3));
      const uint32_t at = smem_u32(sm.x[kp][s & 1]) + m * kXRow + ((v & 12) + q) * 16;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint32_t in[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = pack_f16x2(__uint_as_float(in[e] << 16) * mul[j], __uint_as_float(in[e] & 0xffff0000u) * mul[j]);
        st_shared_v4(at + j * 8 * kXRow, h[0], h[1], h[2], h[3]);
      }
    };
    load_x(0);
#pragma unroll
    for (int j = 0; j < NT; ++j) mul[j] = __uint_as_float((uint32_t)(up_of(8 * j + (xt >> 4)) + 127) << 23);
    store_x(0);
    load_x(1);

    float acc[kOwn][NT][4] = {};
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      asm volatile("bar.sync %0, 128;" ::"r"(kp + 1) : "memory");  // x(s) is there, x(s - 1) has been read
      store_x(s + 1);
      load_x(s + 2);
      uint32_t xb[NT][16];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 f = lds128(smem_u32(sm.x[kp][s & 1]) + (8 * j + g) * kXRow + (4 * c + (q ^ (2 * (g & 1) + (c >> 1)))) * 16);
          xb[j][4 * q] = f.x, xb[j][4 * q + 1] = f.y, xb[j][4 * q + 2] = f.z, xb[j][4 * q + 3] = f.w;
        }
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (i >= mine) break;
        // this lane's copies have landed: all but those of the tiles since
        if (mine == 5)
          cp_async_wait<4>();
        else if (mine <= 3 && NT == 1)
          cp_async_wait<5>();
        else if (mine == 3 && NT == 2)
          cp_async_wait<2>();
        else
          cp_async_wait<3>();
        multiply(lds128(slot), lds128(slot + 512), lds128(slot + 1024), g, c, xb, acc[i]);
        copy(i, slot);
        slot += kRingBytes;
      }
      if (slot == ring_end) slot = ring;
      next_step();
    }
    cp_async_wait<0>();
    __syncthreads();  // the ring is free

    // parts[kp][pair of x rows][weight row]: weight rows in an order whose
    // neighbours are neighbours in the output, pairs 32 bytes apart in the banks
    float2* parts = reinterpret_cast<float2*>(sm.ring);
    const int stride = 16 * nt + 4;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      if (i >= mine) break;
      const int row = ((g >> 2) * nt + rg + kRg * i) * 4 + (g & 3);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float2* at = parts + (kp * 4 * NT + 4 * j + c) * stride + row;
        at[0] = make_float2(acc[i][j][0], acc[i][j][1]);
        at[8 * nt] = make_float2(acc[i][j][2], acc[i][j][3]);
      }
    }
    __syncthreads();
    const float a = p.alpha * (p.tensor_scale ? *p.tensor_scale : 1.0f);
    for (int o = tid; o < 16 * nt * ((p.M + 1) / 2); o += kThreads) {
      const int pair = o / (16 * nt), row = o % (16 * nt), i2 = row / (4 * nt), t = t0 + row % (4 * nt) / 4;
      const int n = 128 * (t >> 3) + 4 * (t & 7) + (row & 3) + 32 * i2;
      float2 y = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kKp; ++k) {
        const float2 q = parts[(k * 4 * NT + pair) * stride + row];
        y.x += q.x, y.y += q.y;
      }
      if (n >= p.N) continue;
      const float bias = p.bias ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[n]) : 0.0f;
      y.x = fmaf(a, y.x * __uint_as_float((uint32_t)(127 - up_of(2 * pair)) << 23), bias);
      y.y = fmaf(a, y.y * __uint_as_float((uint32_t)(127 - up_of(2 * pair + 1)) << 23), bias);
      const long long at = 2 * pair * p.ldo + n;
      if (p.out_bf16) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + at;
        out[0] = __float2bfloat16(y.x);
        if (2 * pair + 1 < p.M) out[p.ldo] = __float2bfloat16(y.y);
      } else {
        float* out = static_cast<float*>(p.out) + at;
        out[0] = y.x;
        if (2 * pair + 1 < p.M) out[p.ldo] = y.y;
      }
    }
    __syncthreads();  // parts have been read
  }
}

template <int NT>
cudaError_t launch_many(const Fp4MatvecParams& p, int sms, cudaStream_t stream) {
  constexpr int kBytes = (int)sizeof(ManySmem<NT>);
  static_assert(kBytes <= 227 * 1024 && kKp * 4 * NT * (16 * kRg * kOwn + 4) * 8 <= (int)sizeof(ManySmem<NT>::ring), "shared memory");
  const int tiles = (p.N + 127) / 128 * 8;
  return launch_kernel_smem(fp4_matvec_many_kernel<NT>, (unsigned)(tiles < sms ? tiles : sms), kThreads, kBytes, stream, p,
                            tiles);
}

template <int NT>
cudaError_t launch_few(const Fp4MatvecParams& p, int sms, cudaStream_t stream) {
  const int tiles = (p.N + 127) / 128 * 8;
  return launch_kernel_smem(fp4_matvec_few_kernel<NT>, (unsigned)(tiles < sms ? tiles : sms), kThreads, kSmem, stream, p, tiles);
}

}  // namespace

cudaError_t launch_fp4_matvec(const Fp4MatvecParams& p, int sms, cudaStream_t stream) {
  if (p.K > kMostChunks * 128 || (p.N + 127) / 128 >= sms) return p.M <= 8 ? launch_many<1>(p, sms, stream) : launch_many<2>(p, sms, stream);
  return p.M <= 8 ? launch_few<1>(p, sms, stream) : launch_few<2>(p, sms, stream);
}

}  // namespace bsk
