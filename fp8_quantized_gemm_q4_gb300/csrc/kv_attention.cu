// kv_attention.cu -- causal attention of new tokens over the paged 8-bit
// cache:  o = softmax(scale q K^T) V  with K = s_K[page, head] * code and V
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
#include "kernels.h"
#include "ptx.cuh"

namespace bsk {

namespace {

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
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// natural log of the softmax sum 2^m l
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Shared memory of a tile as TMA writes it: rows of D bytes, 16-byte chunks
// exchanged by the 128-byte (D = 128) or 64-byte (D = 64) swizzle.
template <int D>
__device__ __forceinline__ int code_at(int tok, int chunk) {
  return D == 128 ? tok * 128 + ((chunk ^ (tok & 7)) << 4) : tok * 64 + ((chunk ^ ((tok >> 1) & 3)) << 4);
}
// Which of 8 tokens stands at place n of the MMA's token axis: any order does,
// as long as scores, masks and V rows agree.  For D = 128 places 2 i, 2 i + 1
// are four tokens apart, so that the 16-byte loads of K meet no bank twice.
template <int D>
__device__ __forceinline__ int token_of(int n) {
  return D == 128 ? (n >> 1) | ((n & 1) << 2) : n;
}

// One step of the online softmax over 16 tokens.  u[t][e]: logit of token
// place 8 t + 2 c + e % 2 for row g + 8 (e / 2); returns the weights as the A
// fragment of the product with V.
template <int NA>
__device__ __forceinline__ void softmax_step(float (&u)[2][4], float inv_sv, float (&m)[2], float (&l)[2],
                                             float (&o)[NA][2][4], uint32_t (&pa)[4]) {
  float mx[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    mx[h] = fmaxf(fmaxf(u[0][2 * h], u[0][2 * h + 1]), fmaxf(u[1][2 * h], u[1][2 * h + 1]));
    mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFullMask, mx[h], 1));
    mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFullMask, mx[h], 2));
  }
  if (__any_sync(kFullMask, mx[0] > m[0] + 8.0f || mx[1] > m[1] + 8.0f)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool up = mx[h] > m[h] + 8.0f;
      const float f = up ? ex2(m[h] - mx[h]) : 1.0f;
      m[h] = up ? mx[h] : m[h];
      l[h] *= f;
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) o[a][e][2 * h] *= f, o[a][e][2 * h + 1] *= f;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float ref = m[h] == -INFINITY ? 0.0f : m[h];
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float a = ex2(u[t][2 * h] - ref), b = ex2(u[t][2 * h + 1] - ref);
      sum += a + b;
      pa[2 * t + h] = pack_f16x2(a, b);
    }
    l[h] = fmaf(sum, inv_sv, l[h]);
  }
}

// ---------------------------------------------------------------------------
// Requests with at most 16 rows per KV head (decode, drafts).
// ---------------------------------------------------------------------------
constexpr int kTile = 64;          // cached tokens per stage
constexpr int kRows = 16;          // rows (token i, head of the group g): r = i * G + g
constexpr int kItems = 64;         // (request, KV head) pairs listed at a time
constexpr int kMinTiles = 2;       // least tiles worth a CTA of its own
constexpr int kFewThreads = 160;   // 4 consumer warps, 1 producer warp
constexpr int kCounters = 1024;    // arrival counters at the head of the workspace

template <int D>
struct FewSmem {
  static constexpr int kStages = 640 / D;  // 80 KB of codes
  static constexpr int kStageBytes = 2 * kTile * D;
  alignas(1024) uint8_t kv[kStages][kStageBytes];  // K rows, then V rows
  float red[2][kRows][D];
  float2 ml[4][kRows];
  float4 group[kStages][4];  // per 16 tokens: K scale, log2 of V scale, 1 / V scale, valid tokens (int)
  int4 item[kItems];         // request, KV head, first tile, end tile
  long long item_at[kItems]; // the pair's first tile in the list of all
  int tile_sum[kItems + 1];  // tiles of this CTA before each item
  uint64_t full[kStages], empty[kStages];
  int scan[8];
  long long start[4];
  int abort_flag, last;
};

// Cached tokens of a request, as far as its table row can name them.
__device__ __forceinline__ int cached(const KvAttentionParams& p, int b) {
  return min(max(p.kv_lens[b], 0), p.max_pages << p.page_shift);
}
// Tiles of a request in this kernel's list: none without rows or with more
// than 16 per KV head, else one at least (rows that see nothing are written too).
__device__ __forceinline__ int few_tiles(const KvAttentionParams& p, int b, int G) {
  const long long n = p.cu_q[b + 1] - p.cu_q[b];
  if (n <= 0 || n * G > kRows) return 0;
  return max(1, (cached(p, b) + kTile - 1) / kTile);
}

// A piece of a pair that is cut between CTAs: partial sums [16][D], then
// (m, l) of the 16 rows.  A CTA has at most two: of the pair that begins before
// its share (0) and of one that begins in it (1).
template <int D>
__device__ __forceinline__ long long piece_at(int cta, int first_cta) {
  return ((long long)cta * 2 + (cta == first_cta)) * (kRows * (D + 2));
}

template <int D>
__global__ void __launch_bounds__(kFewThreads, 2) kv_attention_few_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                          const __grid_constant__ CUtensorMap tm_v,
                                                                          const __grid_constant__ KvAttentionParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = FewSmem<D>;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kStages = Smem::kStages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.Hkv;
  const WaitGuard wg{&sm.abort_flag, p.status, p.wait_ns};
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 4);
    }
    fence_barrier_init();
    sm.abort_flag = 0;
  }
  griddep_wait();
  griddep_launch_dependents();

  // All tiles of all (request, head) pairs form one list, cut into equal
  // contiguous shares.  Each thread sums the tiles of its own requests; the one
  // whose requests hold the share's first tile finds the pair.
  const int per = (p.B + kFewThreads - 1) / kFewThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += few_tiles(p, b, G);
    if (p.only_few && (long long)(p.cu_q[b + 1] - p.cu_q[b]) * G > kRows) record_status(p.status, kStatusOffsets, 53);
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(kFullMask, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  int before = incl - mine, sum = 0;
#pragma unroll
  for (int w = 0; w < kFewThreads / 32; ++w) {
    if (w < warp) before += sm.scan[w];
    sum += sm.scan[w];
  }
  const long long total = (long long)sum * p.Hkv;
  const int shares = (int)min((long long)gridDim.x, (total + kMinTiles - 1) / kMinTiles);
  if ((int)blockIdx.x >= shares) return;
  const long long t_first = total * blockIdx.x / shares, t_last = total * (blockIdx.x + 1) / shares;
  {
    long long at = (long long)before * p.Hkv;
    if (t_first >= at && t_first < at + (long long)mine * p.Hkv) {
      for (int b = b0; b < b1; ++b) {
        const int nt = few_tiles(p, b, G);
        if (nt && t_first < at + (long long)nt * p.Hkv) {
          const int h = (int)((t_first - at) / nt);
          sm.start[0] = b;
          sm.start[1] = h;
          sm.start[2] = at + (long long)h * nt;  // the pair's first tile
          break;
        }
        at += (long long)nt * p.Hkv;
      }
    }
  }
  __syncthreads();
  long long pair = sm.start[0] * p.Hkv + sm.start[1], pair_at = sm.start[2];

  uint32_t it = 0;  // stages used so far: the same count in every role
  bool dead = false;  // producer: a wait gave up, nothing more is copied
  uint32_t issued = 0;
  while (pair_at < t_last) {
    // list the next pairs of this share
    __syncthreads();
    if (warp == 0) {
      long long at = pair_at;
      int tiles_before = 0;
      for (int k0 = 0; k0 < kItems; k0 += 32) {
        const long long q = pair + k0 + lane;
        const int b = (int)(q / p.Hkv);
        const int nt = b < p.B ? few_tiles(p, b, G) : 0;
        int inc = nt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(kFullMask, inc, d);
          if (lane >= d) inc += v;
        }
        const long long p0 = at + inc - nt;
        const int lo = (int)max(0ll, min((long long)nt, t_first - p0)), hi = (int)max(0ll, min((long long)nt, t_last - p0));
        sm.item[k0 + lane] = make_int4(b, (int)(q % p.Hkv), lo, hi);
        sm.item_at[k0 + lane] = p0;
        int cnt = hi > lo ? hi - lo : 0, ci = cnt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(kFullMask, ci, d);
          if (lane >= d) ci += v;
        }
        sm.tile_sum[k0 + lane] = tiles_before + ci - cnt;
        tiles_before += __shfl_sync(kFullMask, ci, 31);
        at += __shfl_sync(kFullMask, inc, 31);
      }
      if (lane == 0) {
        sm.tile_sum[kItems] = tiles_before;
        sm.start[3] = at;
      }
    }
    __syncthreads();
    const int tiles = sm.tile_sum[kItems];

    if (warp == 4) {
      // ---- producer: lane 4 k + j prepares group j (16 tokens) of the k-th of
      // the next eight tiles, then each tile's copies go out as its stage frees
      const int box = min(kTile, 1 << p.page_shift);  // rows of a copy
      for (int k0 = 0; k0 < tiles; k0 += 8) {
        const int k = k0 + (lane >> 2), j = lane & 3;
        int id = -1, cnt = 0, tok = 0, h = 0;
        float ks = 0.0f, vs = 1.0f;
        if (k < tiles) {
          int lo = 0, hi = kItems;  // the item with tile_sum[lo] <= k < tile_sum[lo + 1]
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.tile_sum[mid] <= k) lo = mid; else hi = mid;
          }
          const int4 im = sm.item[lo];
          const int len = cached(p, im.x);
          tok = (im.z + k - sm.tile_sum[lo]) * kTile + 16 * j;
          h = im.y;
          cnt = max(0, min(16, len - tok));
          if (cnt > 0) {
            id = p.table[im.x * p.ld_table + (tok >> p.page_shift)];
            if ((unsigned)id >= (unsigned)p.num_pages) {
              record_status(p.status, kStatusOffsets, 50);
              id = -1;
              cnt = 0;
            } else {
              ks = p.k_scales[(long long)id * p.Hkv + h];
              vs = p.v_scales[(long long)id * p.Hkv + h];
            }
          }
        }
        const bool copies = cnt > 0 && (16 * j) % box == 0;
        const unsigned copy_mask = __ballot_sync(kFullMask, copies);
        const int row = (int)((((long long)id * p.Hkv + h) << p.page_shift) + (tok & ((1 << p.page_shift) - 1)));
        const float lvs = log2f(vs), ivs = 1.0f / vs;
        for (int i = 0; i < 8 && k0 + i < tiles; ++i) {
          const uint32_t s = it % kStages, phase = (it / kStages) & 1;
          const bool ok = mbar_wait(&sm.empty[s], phase ^ 1, wg, 51);
          dead |= __any_sync(kFullMask, !ok) != 0;
          if (dead) {
            ++it;
            continue;
          }
          if ((lane >> 2) == i) sm.group[s][j] = make_float4(ks, lvs, ivs, __int_as_float(cnt));
          __syncwarp();
          const int n = __popc((copy_mask >> (4 * i)) & 15u);
          if (lane == 4 * i) mbar_arrive_expect_tx(&sm.full[s], (uint32_t)(n * box * D * 2));
          if ((lane >> 2) == i && copies) {
            tma_load_2d(&sm.kv[s][16 * j * D], &tm_k, &sm.full[s], 0, row);
            tma_load_2d(&sm.kv[s][(kTile + 16 * j) * D], &tm_v, &sm.full[s], 0, row);
          }
          issued = ++it;
        }
      }
    } else {
      // ---- consumers: warp w takes tokens 16 w .. + 15 of every tile
      const int g = lane >> 2, c = lane & 3;
      constexpr int kQ = D / 64;  // 64-wide parts of a row
      for (int im = 0; im < kItems; ++im) {
        const int4 item = sm.item[im];
        if (item.z >= item.w) continue;
        const int b = item.x, h = item.y;
        const int row0 = p.cu_q[b], n = p.cu_q[b + 1] - row0, R = min(n, p.T - row0) * G;
        const int len = cached(p, b);
        // q rows g and g + 8 as A fragments, fp16 by a power of two per row
        uint32_t qa[4 * kQ][4];
        float qscale[2];
        int seen[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = g + 8 * half;
          const bool in = r < R;
          const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (row0 + r / G) * p.q_tok_stride +
                                   (h * G + r % G) * p.q_head_stride + 16 * c;
          uint4 raw[2 * kQ];
#pragma unroll
          for (int x = 0; x < 2 * kQ; ++x)
            raw[x] = in ? *reinterpret_cast<const uint4*>(q + 64 * (x >> 1) + 8 * (x & 1)) : make_uint4(0, 0, 0, 0);
          const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
          float amax = 0.0f;
#pragma unroll
          for (int x = 0; x < 8 * kQ; ++x)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[x] << 16)), fabsf(__uint_as_float(w[x] & 0xffff0000u))));
          amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
          const int up = fp16_up(amax);
          const float mul = exp2i(up);
          qscale[half] = exp2i(-up) * p.scale_log2;
          seen[half] = in ? len - n + r / G + 1 : 0;
#pragma unroll
          for (int x = 0; x < 4 * kQ; ++x)  // k step x: columns 64 (x / 4) + 16 c + 4 (x % 4) .. + 3
#pragma unroll
            for (int y = 0; y < 2; ++y)
              qa[x][half + 2 * y] = pack_f16x2(__uint_as_float(w[2 * x + y] << 16) * mul,
                                               __uint_as_float(w[2 * x + y] & 0xffff0000u) * mul);
        }
        const int all_seen = len - n + 1;  // tokens that every row sees
        float o[D / 16][2][4] = {};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        for (int t = item.z; t < item.w; ++t, ++it) {
          const uint32_t s = it % kStages, phase = (it / kStages) & 1;
          mbar_wait(&sm.full[s], phase, wg, 52);
          const float4 sc = sm.group[s][warp];
          const int cnt = __float_as_int(sc.w);
          if (cnt > 0) {
            uint8_t* kt = &sm.kv[s][warp * 16 * D];
            uint8_t* vt = &sm.kv[s][(kTile + warp * 16) * D];
            if (cnt < 16) {  // codes behind the last token may stand for NaN
              for (int x = cnt * (D / 16) + lane; x < D; x += 32) reinterpret_cast<uint4*>(vt)[x] = make_uint4(0, 0, 0, 0);
              __syncwarp();
            }
            float u[2][4] = {};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int tok = 8 * half + token_of<D>(g);
#pragma unroll
              for (int part = 0; part < kQ; ++part) {
                const uint4 v = *reinterpret_cast<const uint4*>(kt + code_at<D>(tok, 4 * part + c));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  mma_f16(u[half], qa[4 * part + x], e4m3x2_to_f16x2((uint16_t)w[x]), e4m3x2_to_f16x2((uint16_t)(w[x] >> 16)));
              }
            }
            const float f0 = qscale[0] * sc.x, f1 = qscale[1] * sc.x;
            const int tok0 = t * kTile + warp * 16;
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int e = 0; e < 4; ++e) u[half][e] = fmaf(u[half][e], e < 2 ? f0 : f1, sc.y);
            if (cnt < 16 || tok0 + 16 > all_seen) {
#pragma unroll
              for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int tok = 8 * half + token_of<D>(2 * c + (e & 1));
                  if (tok >= cnt || tok0 + tok >= seen[e >> 1]) u[half][e] = -INFINITY;
                }
            }
            uint32_t pa[4];
            softmax_step<D / 16>(u, sc.z, m, l, o, pa);
#pragma unroll
            for (int a = 0; a < D / 32; ++a) {
              // lanes 8 i .. + 7 give the rows of matrix i: tokens 8 (i % 2) .. + 7 at 16-byte chunk 2 a + i / 2
              uint32_t v[4];
              const int tok = 8 * ((lane >> 3) & 1) + token_of<D>(lane & 7);
              ldmatrix_x4_trans(v, smem_u32(vt + code_at<D>(tok, 2 * a + (lane >> 4))));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t w0 = __byte_perm(v[2 * x], 0, 0x3120), w1 = __byte_perm(v[2 * x + 1], 0, 0x3120);
                mma_f16(o[2 * a + x][0], pa, e4m3x2_to_f16x2((uint16_t)w0), e4m3x2_to_f16x2((uint16_t)w1));
                mma_f16(o[2 * a + x][1], pa, e4m3x2_to_f16x2((uint16_t)(w0 >> 16)), e4m3x2_to_f16x2((uint16_t)(w1 >> 16)));
              }
            }
            if (cnt < 16) fence_proxy_async_smem();  // the zeros, before the next copy into this stage
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.empty[s]);
        }

        // ---- the four warps' (m, l, o) to one
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          l[half] += __shfl_xor_sync(kFullMask, l[half], 1);
          l[half] += __shfl_xor_sync(kFullMask, l[half], 2);
          if (c == 0) sm.ml[warp][g + 8 * half] = make_float2(m[half], l[half]);
        }
        consumer_sync();
        float M[2], L[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float2 x[4];
          M[half] = -INFINITY;
          L[half] = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) x[w] = sm.ml[w][g + 8 * half], M[half] = fmaxf(M[half], x[w].x);
          const float ref = M[half] == -INFINITY ? 0.0f : M[half];
#pragma unroll
          for (int w = 0; w < 4; ++w) L[half] += x[w].y * ex2(x[w].x - ref);
          const float f = ex2(m[half] - ref);
#pragma unroll
          for (int a = 0; a < D / 16; ++a)
#pragma unroll
            for (int e = 0; e < 2; ++e) o[a][e][2 * half] *= f, o[a][e][2 * half + 1] *= f;
        }
        // element (row, 16 a + 4 c + 2 x + e) is o[a][e][2 half + x]: four in a row
        auto put = [&](int buf, int a) {
#pragma unroll
          for (int half = 0; half < 2; ++half)
            *reinterpret_cast<float4*>(&sm.red[buf][g + 8 * half][16 * (a ^ (g & 1)) + 4 * c]) =
                make_float4(o[a][0][2 * half], o[a][1][2 * half], o[a][0][2 * half + 1], o[a][1][2 * half + 1]);
        };
        auto add = [&](int buf, int a) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.red[buf][g + 8 * half][16 * (a ^ (g & 1)) + 4 * c]);
            o[a][0][2 * half] += v.x, o[a][1][2 * half] += v.y, o[a][0][2 * half + 1] += v.z, o[a][1][2 * half + 1] += v.w;
          }
        };
        if (warp >= 2)
#pragma unroll
          for (int a = 0; a < D / 16; ++a) put(warp - 2, a);
        consumer_sync();
        if (warp < 2)
#pragma unroll
          for (int a = 0; a < D / 16; ++a) add(warp, a);
        consumer_sync();
        // warp 0 keeps the first half of the columns, warp 1 the second
        if (warp == 0)
#pragma unroll
          for (int a = D / 32; a < D / 16; ++a) put(0, a);
        if (warp == 1)
#pragma unroll
          for (int a = 0; a < D / 32; ++a) put(1, a);
        consumer_sync();
        if (warp == 0)
#pragma unroll
          for (int a = 0; a < D / 32; ++a) add(1, a);
        if (warp == 1)
#pragma unroll
          for (int a = D / 32; a < D / 16; ++a) add(0, a);

        const int nt = max(1, (len + kTile - 1) / kTile);
        if (item.z == 0 && item.w == nt) {
          if (warp < 2) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int r = g + 8 * half;
              if (r >= R) continue;
              const float inv = L[half] > 0.0f ? 1.0f / L[half] : 0.0f;
              const long long tr = row0 + r / G;
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + tr * p.out_tok_stride +
                                   (h * G + r % G) * p.out_head_stride + 4 * c;
#pragma unroll
              for (int a = 0; a < D / 16; ++a)
                if (a / (D / 32) == warp)
                  *reinterpret_cast<uint2*>(dst + 16 * a) =
                      make_uint2(pack_bf16x2(o[a][0][2 * half] * inv, o[a][1][2 * half] * inv),
                                 pack_bf16x2(o[a][0][2 * half + 1] * inv, o[a][1][2 * half + 1] * inv));
              if (warp == 0 && c == 0 && p.lse) p.lse[tr * p.Hq + h * G + r % G] = lse_of(M[half], L[half]);
            }
          }
          continue;
        }
        // ---- a pair cut between CTAs: this piece goes to the workspace, the
        // last CTA to finish one joins the pieces in order
        float* slot = p.work + ((long long)blockIdx.x * 2 + (item.z == 0 ? 1 : 0)) * (kRows * (D + 2));
        if (warp < 2) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = g + 8 * half;
            if (r >= R) continue;
#pragma unroll
            for (int a = 0; a < D / 16; ++a)
              if (a / (D / 32) == warp)
                *reinterpret_cast<float4*>(slot + r * D + 16 * a + 4 * c) =
                    make_float4(o[a][0][2 * half], o[a][1][2 * half], o[a][0][2 * half + 1], o[a][1][2 * half + 1]);
            if (warp == 0 && c == 0) *reinterpret_cast<float2*>(slot + kRows * D + 2 * r) = make_float2(M[half], L[half]);
          }
          __threadfence();
        }
        // the shares that hold the pair's first and last tile
        const long long first = sm.item_at[im];
        const int c0 = (int)(((first + 1) * shares - 1) / total), c1 = (int)(((first + nt) * shares - 1) / total);
        consumer_sync();
        if (tid == 0) {
          const int old = atomicAdd(p.counters + c0, 1);
          __threadfence();
          sm.last = old == c1 - c0;
          if (sm.last) p.counters[c0] = 0;
        }
        consumer_sync();
        if (sm.last) {
          for (int r = warp; r < R; r += 4) {
            float mx = -INFINITY;
            for (int x = c0 + lane; x <= c1; x += 32) mx = fmaxf(mx, __ldcg(p.work + piece_at<D>(x, c0) + kRows * D + 2 * r));
#pragma unroll
            for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, d));
            const float ref = mx == -INFINITY ? 0.0f : mx;
            float acc[D / 32] = {}, sum_l = 0.0f;
#pragma unroll 4
            for (int x = c0; x <= c1; ++x) {
              const float* from = p.work + piece_at<D>(x, c0);
              const float2 e = __ldcg(reinterpret_cast<const float2*>(from + kRows * D + 2 * r));
              const float f = ex2(e.x - ref);
              sum_l += e.y * f;
#pragma unroll
              for (int d = 0; d < D / 32; ++d) acc[d] += f * __ldcg(from + r * D + 32 * d + lane);
            }
            const float inv = sum_l > 0.0f ? 1.0f / sum_l : 0.0f;
            const long long tr = row0 + r / G;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + tr * p.out_tok_stride +
                                 (h * G + r % G) * p.out_head_stride + lane;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) dst[32 * d] = __float2bfloat16(acc[d] * inv);
            if (lane == 0 && p.lse) p.lse[tr * p.Hq + h * G + r % G] = lse_of(mx, sum_l);
          }
        }
      }
    }
    pair += kItems;
    pair_at = sm.start[3];
  }
  // after a wait that gave up: copies in flight land before the CTA's memory goes
  if (warp == 4 && dead)
    for (uint32_t k = issued > kStages ? issued - kStages : 0; k < issued; ++k)
      mbar_drain(&sm.full[k % kStages], (k / kStages) & 1, 100000000ull);
}

// ---------------------------------------------------------------------------
// Requests with more rows.
// ---------------------------------------------------------------------------
constexpr int kAttnThreads = 128;
__device__ __forceinline__ float e4m3_val(uint32_t c) { return e4m3_to_f32(c); }

// One CTA per (row, query head): a thread scores one token of a chunk of 128,
// then owns one output element.
template <int D>
__global__ void __launch_bounds__(kAttnThreads) kv_attention_kernel(const __grid_constant__ KvAttentionParams p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float qs[D], ps[kAttnThreads], red[kAttnThreads / 32];
  const int row = blockIdx.x, hq = blockIdx.y, tid = threadIdx.x;
  const int h = hq / (p.Hq / p.Hkv);
  // the request of this row: cu_q ascends
  int lo = 0, hi = p.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_q[mid + 1] > row) hi = mid; else lo = mid + 1;
  }
  if (lo == p.B) return;  // rows past the last request are not written
  const int n = p.cu_q[lo + 1] - p.cu_q[lo];
  if ((long long)n * (p.Hq / p.Hkv) <= kRows) return;
  const int len = min(p.kv_lens[lo], p.max_pages << p.page_shift) - n + (row - p.cu_q[lo]) + 1;
  if (tid < D)
    qs[tid] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[row * p.q_tok_stride + hq * p.q_head_stride + tid]);
  __syncthreads();
  const int page_mask = (1 << p.page_shift) - 1;
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int t0 = 0; t0 < len; t0 += kAttnThreads) {
    const int t = t0 + tid;
    float s = -INFINITY;
    const int id = t < len ? p.table[lo * p.ld_table + (t >> p.page_shift)] : -1;
    if (t < len && (unsigned)id >= (unsigned)p.num_pages) record_status(p.status, kStatusOffsets, 50);
    if ((unsigned)id < (unsigned)p.num_pages) {
      const long long blk = (long long)id * p.Hkv + h;
      const uint8_t* k = p.k_codes + ((blk << p.page_shift) + (t & page_mask)) * D;
      s = 0.0f;
      for (int d = 0; d < D; ++d) s += qs[d] * e4m3_val(k[d]);
      s *= p.k_scales[blk] * p.scale_log2;
    }
    float mx = s;
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, d));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, mx);
    const float c = mn > -INFINITY ? exp2f(m - mn) : 1.0f, e = mn > -INFINITY ? exp2f(s - mn) : 0.0f;
    ps[tid] = e;
    float sum = e;
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    l = l * c + (red[0] + red[1]) + (red[2] + red[3]);
    o *= c;
    m = mn;
    if (tid < D) {
      const int cnt = min(kAttnThreads, len - t0);
      for (int i = 0; i < cnt; ++i) {
        const int vid = p.table[lo * p.ld_table + ((t0 + i) >> p.page_shift)];
        if ((unsigned)vid >= (unsigned)p.num_pages) continue;
        const long long blk = (long long)vid * p.Hkv + h;
        o += ps[i] * p.v_scales[blk] * e4m3_val(p.v_codes[((blk << p.page_shift) + ((t0 + i) & page_mask)) * D + tid]);
      }
    }
    __syncthreads();
  }
  if (tid < D)
    static_cast<__nv_bfloat16*>(p.out)[row * p.out_tok_stride + hq * p.out_head_stride + tid] =
        __float2bfloat16(l > 0.0f ? o / l : 0.0f);
  if (tid == 0 && p.lse)
    p.lse[(long long)row * p.Hq + hq] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

template <int D>
cudaError_t launch_few(const KvAttentionLaunch& L, cudaStream_t stream) {
  constexpr int kSmem = (int)sizeof(FewSmem<D>) + 1024;
  static const cudaError_t attr =
      cudaFuncSetAttribute(kv_attention_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (attr != cudaSuccess) return attr;
  return launch_kernel(kv_attention_few_kernel<D>, (unsigned)L.few_grid, kFewThreads, kSmem, stream, 1, L.tm_k, L.tm_v,
                       L.p);
}

}  // namespace

int kv_attention_few_grid(int sms) { return min(2 * sms, kCounters); }
size_t kv_attention_piece_bytes(int D) { return (size_t)2 * kRows * (D + 2) * sizeof(float); }
int kv_attention_box(int page_size) { return min(page_size, kTile); }
int kv_attention_few_rows() { return kRows; }

cudaError_t launch_kv_attention(const KvAttentionLaunch& L, cudaStream_t stream) {
  const KvAttentionParams& p = L.p;
  cudaError_t e = p.D == 64 ? launch_few<64>(L, stream) : launch_few<128>(L, stream);
  if (e != cudaSuccess || p.only_few) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.T, (unsigned)p.Hq, 1);
  cfg.blockDim = dim3(kAttnThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return p.D == 64 ? cudaLaunchKernelEx(&cfg, kv_attention_kernel<64>, p)
                   : cudaLaunchKernelEx(&cfg, kv_attention_kernel<128>, p);
}

}  // namespace bsk
