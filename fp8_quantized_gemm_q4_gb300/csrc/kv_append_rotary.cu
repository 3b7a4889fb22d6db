// kv_append_rotary.cu -- new keys and values into the paged cache (8 or 4 bits) and
// queries to bf16, with the position rotation applied on the way:
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin
// for the pairs (i, i + R/2) of the first R elements of a head, or (2i, 2i + 1).
// Products and sums are rounded to fp32 one by one (no fused multiply-add), so what a
// code is rounded from follows from the definition alone.
//
// A lane has 16 elements of a row: the two vectors of 8 whose elements meet in pairs
// (vectors j and j + R/16 of the halves; 2j and 2j + 1 otherwise), so that no element
// is read twice or passed between lanes, and 8 cosines and 8 sines, which it keeps in
// registers while it goes through several heads of its token.
//
// 4-bit cache: scale e4m3(amax / 6) and codes E2M1(x / scale) for 16 elements of a
// token, as q4_quantize has them; rows are independent of each other.  8-bit cache: as
// kv_append, a run of rows that lie in one page shares a scale.
//
// Bound by the stream of rows, angles and codes.  16384 rows, 32 + 16 heads of 128, bf16:
// 8 bits 77 us (372 MB, 0.71 of HBM; the queries alone 0.9, keys and values 41 us of them, at 64 rows a CTA a
// chain of reads, maxima and codes), 4 bits 63 us (355 MB, 0.83), the cached rows read back
// 19 us (88 MB, most of them in L2).  A third of the warps' time is waiting for rows, the rest issue (0.5
// of the slots); 46 % of the SM's warps at 64 registers.  64 rows: 2.7 and 4.7 us, of which a
// launch that does nothing is about 2.
#include "decode.h"
#include "kv_cache.cuh"

namespace bsk {
namespace {

// Heads of a token that a warp goes through: angles and places are worked out once for
// them.  Two, all of whose elements are on their way at once, in a call that does not fill
// the SMs with warps of eight (us, 2 / 8 heads, 32 + 16 heads, 4-bit cache with the rows
// read back: 64 rows 4.6 / 8.3, 512 rows 8.0 / 9.4, 2047 rows 18 / 18).
constexpr int kFewHeads = 2, kHeads = 8;

template <int D>
constexpr int kLanes = D / 16;  // lanes of a row
template <int D>
constexpr int kRows = 32 / kLanes<D>;  // rows of a warp's pass
constexpr int kShort = 8;              // rows of a run that is a single warp's

// A lane's two vectors of 8 elements of a row
struct Pair {
  int a, b;
};
__device__ __forceinline__ Pair vectors(const KvRotaryParams& p, int j) {
  const int n = p.rot >> 4;
  return !p.interleaved && j < n ? Pair{j, j + n} : Pair{2 * j, 2 * j + 1};
}

// A lane's sixteen elements of a row, as they lie in memory
template <bool kBf16>
struct Raw {
  uint4 w[kBf16 ? 2 : 4];
  __device__ __forceinline__ void load(const void* x, long long at, const Pair& v) {
    constexpr int kEach = kBf16 ? 1 : 2;
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + at * (kBf16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < kEach; ++i) w[i] = from[v.a * kEach + i], w[kEach + i] = from[v.b * kEach + i];
  }
  __device__ __forceinline__ void values(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < (kBf16 ? 2 : 4); ++i) {
      const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if constexpr (kBf16)
          v[8 * i + 2 * x] = __uint_as_float(in[x] << 16), v[8 * i + 2 * x + 1] = __uint_as_float(in[x] & 0xffff0000u);
        else
          v[4 * i + x] = __uint_as_float(in[x]);
      }
    }
  }
};

// The angles of a lane's eight pairs
struct Turn {
  float c[8], s[8];
  bool on;
  // of the row at this position (positions[row], read beside what else the row needs)
  __device__ __forceinline__ void load(const KvRotaryParams& p, int at, int j) {
    on = j < p.rot >> 4;
    if (!on) return;
    if ((unsigned)at >= (unsigned)p.max_positions) {
      record_status(p.status, kStatusOffsets, 47);
      at = min(max(at, 0), p.max_positions - 1);
    }
    const float4* t = reinterpret_cast<const float4*>(p.angles + (long long)at * p.rot + 8 * j);
    const float4* u = reinterpret_cast<const float4*>(p.angles + (long long)at * p.rot + p.rot / 2 + 8 * j);
    const float4 c0 = t[0], c1 = t[1], s0 = u[0], s1 = u[1];
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
  }
  __device__ __forceinline__ void apply(float (&v)[16], bool interleaved) const {
    if (!on) return;
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) pair(v[2 * i], v[2 * i + 1], c[i], s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) pair(v[i], v[8 + i], c[i], s[i]);
    }
  }
  static __device__ __forceinline__ void pair(float& x, float& y, float c, float s) {
    const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = u;
  }
};

__device__ __forceinline__ uint4 to_bf16(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Largest finite magnitude of eight elements, as bits; above infinity's where one is NaN
__device__ __forceinline__ uint32_t amax8(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
    m = max(m, u == 0x7f800000u ? 0u : u);
  }
  return m;
}
// Scale code of a group
__device__ __forceinline__ uint32_t scale4(uint32_t amax) {
  return amax > 0x7f800000u ? 0x7fu : f32_to_e4m3(quot_rn(__uint_as_float(amax), 6.0f, __frcp_rn(6.0f)));
}
// E2M1 codes of eight elements; what passes 6 scales (an infinity too) is held at 6
__device__ __forceinline__ uint32_t codes4(const float* v, uint32_t scale) {
  if (scale == 0 || scale == 0x7f) return 0;
  const float s = e4m3_to_f32(scale), r = __frcp_rn(s), most = 8.0f * s;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quot_rn(fminf(fmaxf(v[i], -most), most), s, r);
  return f32x8_to_e2m1x8(q);
}

// Rows of a warp's pass: queries to bf16, or keys and values to 4 bits; up to kHeads
// heads from `head` on, of kind 0 (q), 1 (k), 2 (v).  Everything that does not depend on
// something read is asked for first: the heads' elements, slots, positions.
template <bool kBf16, int D, bool kQ>
__device__ __forceinline__ void flat_heads(const KvRotaryParams& p, int first, int kind, int head, int lane) {
  constexpr int kBatch = kBf16 ? 2 : 1;  // heads on their way
  const int j = lane % kLanes<D>, row = min(first + lane / kLanes<D>, p.T - 1);
  const Pair at = vectors(p, j);
  const int heads = min(p.heads, (kQ ? p.Hq : p.Hkv) - head), which = kQ ? 0 : kind - 1;
  const void* x = kQ ? p.q : p.x[which];
  const long long step = kQ ? p.q_head_stride : p.head_stride[which];
  const long long from = row * (kQ ? p.q_tok_stride : p.tok_stride[which]) + head * step;
  Raw<kBf16> raw[kBatch] = {};
  const int slot_here = p.slots[row], position = kind < 2 && p.rot ? p.positions[row] : 0;
#pragma unroll
  for (int h = 0; h < kBatch; ++h)
    if (h < heads) raw[h].load(x, from + h * step, at);
  const int slot = first + lane / kLanes<D> < p.T ? slot_here : -1;
  const bool ok = slot_ok(p, slot);
  Turn turn = {};
  if (ok && kind < 2) turn.load(p, position, j);
  // who has the vector beside a, and the one beside b, in their groups of 16
  const int n = p.interleaved ? 0 : p.rot >> 4;
  auto owner = [&](int vec) { return vec < n ? vec : vec < 2 * n ? vec - n : vec >> 1; };
  auto second = [&](int vec) { return vec < n ? false : vec < 2 * n ? true : (vec & 1) != 0; };
  const int base = lane - j, oa = base + owner(at.a ^ 1), ob = base + owner(at.b ^ 1);
  const bool sa = second(at.a ^ 1), sb = second(at.b ^ 1);
  const long long line = ((((long long)(slot >> p.page_shift) * p.Hkv + head) << p.page_shift) + (slot & ((1 << p.page_shift) - 1)));
#pragma unroll 1
  for (int h0 = 0; h0 < heads; h0 += kBatch) {
#pragma unroll
    for (int h = 0; h < kBatch; ++h) {
      if (h0 + h >= heads) break;
      float v[16];
      raw[h].values(v);
      if (h0 + h + kBatch < heads) raw[h].load(x, from + (h0 + h + kBatch) * step, at);
      turn.apply(v, p.interleaved);
      if constexpr (kQ) {
        if (!ok) continue;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.q_out) + row * p.qo_tok_stride + (head + h0 + h) * p.qo_head_stride;
        *reinterpret_cast<uint4*>(out + 8 * at.a) = to_bf16(v);
        *reinterpret_cast<uint4*>(out + 8 * at.b) = to_bf16(v + 8);
      } else {
        const uint32_t ma = amax8(v), mb = amax8(v + 8);
        const uint32_t a0 = __shfl_sync(kFullMask, ma, oa), a1 = __shfl_sync(kFullMask, mb, oa);
        const uint32_t b0 = __shfl_sync(kFullMask, ma, ob), b1 = __shfl_sync(kFullMask, mb, ob);
        if (!ok) continue;
        const uint32_t fa = scale4(max(ma, sa ? a1 : a0)), fb = scale4(max(mb, sb ? b1 : b0));
        const long long to = line + ((long long)(h0 + h) << p.page_shift);
        uint32_t* codes = reinterpret_cast<uint32_t*>(p.codes[which]) + to * (D / 8);
        uint8_t* scales = static_cast<uint8_t*>(p.scales[which]) + to * (D / 16);
        codes[at.a] = codes4(v, fa);
        codes[at.b] = codes4(v + 8, fb);
        if (!(at.a & 1)) scales[at.a / 2] = (uint8_t)fa;
        if (!(at.b & 1)) scales[at.b / 2] = (uint8_t)fb;
      }
    }
  }
}

// A run of n rows from row `row` on into page `id` at place off, one head of the keys
// (which = 0) or values, by a warp (n <= kShort) or by the kWarps warps of the CTA, whose
// rows up to two passes stay in registers between the maximum and the codes and the rest
// is read again.
template <bool kBf16, int D, int kWarps>
__device__ __forceinline__ void append_run(const KvRotaryParams& p, int which, int h, int row, int n, int id, int off,
                                           int thread) {
  constexpr int kPass = kRows<D> * kWarps, kKeep = kWarps == 1 ? kShort / kPass : 2;
  constexpr bool kRest = kWarps > 1;
  const int lane = thread & 31, j = lane % kLanes<D>, r0 = thread / kLanes<D>;
  const Pair at = vectors(p, j);
  const long long page = (long long)id * p.Hkv + h;
  float* scale = static_cast<float*>(p.scales[which]) + page;
  uint8_t* codes = p.codes[which] + (page << p.page_shift) * D;
  const float old = off > 0 ? *scale : 0.0f;
  auto get = [&](int r, float(&v)[16]) {
    Raw<kBf16> raw;
    const int position = which == 0 && p.rot ? p.positions[row + r] : 0;
    raw.load(p.x[which], (long long)(row + r) * p.tok_stride[which] + h * p.head_stride[which], at);
    Turn turn = {};  // what is not set would be carried from run to run, and spilled
    if (which == 0) turn.load(p, position, j);
    raw.values(v);
    turn.apply(v, p.interleaved);
  };
  // running maximum of the finite magnitudes: bits one step of the exponent up keep
  // their order as signed integers, and the non-finite ones turn negative
  constexpr uint32_t kUp = 0x00800000u;
  int top = kUp;
  auto amax = [&](const float(&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, (int)((__float_as_uint(v[i]) & 0x7fffffffu) + kUp));
  };
  float kept[kKeep][16] = {};
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (r0 + i * kPass < n) get(r0 + i * kPass, kept[i]);
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (r0 + i * kPass < n) amax(kept[i]);
#pragma unroll 1
  for (int r = r0 + kKeep * kPass; kRest && r < n; r += kPass) {
    float v[16];
    get(r, v);
    amax(v);
  }
  top = __reduce_max_sync(kFullMask, top);
  if constexpr (kWarps > 1) {
    __shared__ int tops[kWarps];
    __syncthreads();  // those of the run before have been read
    if (lane == 0) tops[thread >> 5] = top;
    __syncthreads();  // and the page's scale by all
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, tops[w]);
  }
  const float s = page_scale<D, 32 * kWarps>(codes, off, __uint_as_float((uint32_t)top - kUp), old, thread);
  const float inv = 1.0f / s;
  auto put = [&](int r, const float(&v)[16]) {
    uint2* out = reinterpret_cast<uint2*>(codes + (long long)(off + r) * D);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = f32x2_to_e4m3x2(v[8 * x + 2 * i] * inv, v[8 * x + 2 * i + 1] * inv);
      out[x ? at.b : at.a] = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (r0 + i * kPass < n) put(r0 + i * kPass, kept[i]);
#pragma unroll 1
  for (int r = r0 + kKeep * kPass; kRest && r < n; r += kPass) {
    float v[16];
    get(r, v);
    put(r, v);
  }
  __syncwarp();  // the old scale has been read by all
  if (thread == 0) *scale = s;
}

constexpr int kThreads = 128, kRunThreads = 256;
constexpr int kWindow = 64;  // rows whose long runs a CTA takes
// Rows whose short runs a warp takes, one after the other: 1, from 512 rows 4, from 4096 rows
// 16 (us, 1 / 4 / 16: 64 single tokens 2.6 / 5.9 / 19, 512 of them 7.0 / 7.8 / 21, 1500 18 / 15 / 28,
// 4096 54 / 45 / 51; prompts of 1024 rows 7.8 / 6.2 / 6.2, 4096 rows 34 / 27 / 25, 16384 rows
// 121 / 91 / 83).  How the rows fall into pages is known on the device only.
constexpr long long kManyWarps = 2432;  // 16 an SM

// The runs of more than kShort rows that begin in the kWindow rows from `first` on, by a
// warp, in any order; returns how many.
__device__ __forceinline__ int list_runs(const KvRotaryParams& p, int first, int lane, int4* runs) {
  constexpr int kWords = 6;  // 32 rows each, from first on: as far as a run can go
  const int page = 1 << p.page_shift;
  int slot[kWords];
  unsigned inside[kWords + 1];  // rows that carry on the run of the row before
  int last = first ? p.slots[first - 1] : -1;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const int r = first + 32 * w + lane;
    slot[w] = r < p.T ? p.slots[r] : -1;
  }
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    int before = __shfl_up_sync(kFullMask, slot[w], 1);
    if (lane == 0) before = last;
    last = __shfl_sync(kFullMask, slot[w], 31);
    inside[w] = __ballot_sync(kFullMask, (slot[w] & (page - 1)) > 0 && slot[w] == before + 1 && before >= 0);
  }
  inside[kWords] = 0;
  int count = 0;
#pragma unroll
  for (int e = 0; e < kWindow / 32; ++e) {
    const int at = 32 * e + lane;
    int n = 1;
    bool on = slot[e] >= 0 && !(inside[e] >> lane & 1);
#pragma unroll
    for (int w = e; w < kWords; ++w) {  // the rows behind, a word from at + 1 on
      const unsigned bits = lane == 31 ? inside[w + 1] : __funnelshift_r(inside[w], inside[w + 1], lane + 1);
      if (on) n += bits == kFullMask ? 32 : __ffs(~bits) - 1;
      on &= bits == kFullMask;
    }
    const int off = slot[e] & (page - 1);
    const bool here = n > kShort && slot_ok(p, slot[e]);
    const unsigned all = __ballot_sync(kFullMask, here);
    if (here) runs[count + __popc(all & ((1u << lane) - 1))] = make_int4(first + at, min(n, page - off), slot[e] >> p.page_shift, off);
    count += __popc(all);
  }
  return count;
}

template <bool kBf16, int D, bool kFp4>
__global__ void __launch_bounds__(kFp4 ? kThreads : kRunThreads, kFp4 ? 7 : 4)
    kv_append_rotary_kernel(const __grid_constant__ KvRotaryParams p, unsigned long_blocks, unsigned short_blocks) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kWarps = (kFp4 ? kThreads : kRunThreads) / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!kFp4 && blockIdx.x < long_blocks) {
    const unsigned block = blockIdx.x / (2 * p.Hkv), head = blockIdx.x % (2 * p.Hkv);
    __shared__ int4 runs[kWindow / kShort];  // first row, rows, page, place in it
    __shared__ int count;
    if (warp == 0) {
      const int n = list_runs(p, (int)block * kWindow, lane, runs);
      if (lane == 0) count = n;
    }
    __syncthreads();
    const int n = count;
#pragma unroll 1
    for (int i = 0; i < n; ++i)
      append_run<kBf16, D, kWarps>(p, head / p.Hkv, head % p.Hkv, runs[i].x, runs[i].y, runs[i].z, runs[i].w, threadIdx.x);
    return;
  }
  if (!kFp4 && blockIdx.x < long_blocks + short_blocks) {
    // lane i has the slot of row first - 1 + i
    const unsigned task = (blockIdx.x - long_blocks) * kWarps + warp, head = task % (2 * p.Hkv);
    const int first = (int)(task / (2 * p.Hkv)) * p.rows_each, page = 1 << p.page_shift, near = first - 1 + lane;
    const int slot = near >= 0 && near < p.T ? p.slots[near] : -1;
    int before = __shfl_up_sync(kFullMask, slot, 1);
    if (lane == 0) before = -1;
    const unsigned inside = __ballot_sync(kFullMask, (slot & (page - 1)) > 0 && slot == before + 1 && before >= 0);
    unsigned todo = __ballot_sync(kFullMask, slot >= 0) & ~inside & (2u << p.rows_each) - 2;
#pragma unroll 1
    for (; todo; todo &= todo - 1) {
      const int i = __ffs(todo) - 1, mine = __shfl_sync(kFullMask, slot, i), n = __ffs(~(inside >> (i + 1)));
      if (n <= kShort && slot_ok(p, mine))
        append_run<kBf16, D, 1>(p, head / p.Hkv, head % p.Hkv, first - 1 + i, n, mine >> p.page_shift, mine & (page - 1), lane);
    }
    return;
  }
  const int cq = (p.Hq + p.heads - 1) / p.heads, ck = kFp4 ? (p.Hkv + p.heads - 1) / p.heads : 0, parts = cq + 2 * ck;
  const long long task = (long long)(blockIdx.x - long_blocks - short_blocks) * kWarps + warp;
  const long long group = task / parts;
  const int part = (int)(task % parts);
  if (group * kRows<D> >= p.T) return;
  const int kind = part < cq ? 0 : part < cq + ck ? 1 : 2;
  const int chunk = kind == 0 ? part : part - cq - (kind - 1) * ck;
  if (!kFp4 || kind == 0)
    flat_heads<kBf16, D, true>(p, (int)(group * kRows<D>), 0, chunk * p.heads, lane);
  else
    flat_heads<kBf16, D, false>(p, (int)(group * kRows<D>), kind, chunk * p.heads, lane);
}

template <bool kBf16, int D, bool kFp4>
cudaError_t launch(const KvRotaryParams& p, cudaStream_t stream) {
  constexpr int threads = kFp4 ? kThreads : kRunThreads, warps = threads / 32;
  KvRotaryParams q = p;
  q.rows_each = p.T < 512 ? 1 : p.T < 4096 ? 4 : 16;
  const long long longs = kFp4 ? 0 : ((long long)p.T + kWindow - 1) / kWindow * 2 * p.Hkv;
  const long long shorts = kFp4 ? 0 : (((long long)p.T + q.rows_each - 1) / q.rows_each * 2 * p.Hkv + warps - 1) / warps;
  const long long groups = (p.T + kRows<D> - 1) / kRows<D>;
  auto flat = [&](int heads) {
    return groups * ((p.Hq + heads - 1) / heads + (kFp4 ? (p.Hkv + heads - 1) / heads * 2 : 0));
  };
  q.heads = flat(kHeads) < kManyWarps ? kFewHeads : kHeads;
  return launch_kernel(kv_append_rotary_kernel<kBf16, D, kFp4>, (unsigned)(longs + shorts + (flat(q.heads) + warps - 1) / warps), threads, 0, stream, 1, q, (unsigned)longs,
                       (unsigned)shorts);
}
template <bool kBf16, int D>
cudaError_t launch_fmt(const KvRotaryParams& p, cudaStream_t stream) {
  return p.fp4 ? launch<kBf16, D, true>(p, stream) : launch<kBf16, D, false>(p, stream);
}

// ---------------------------------------------------------------------------
// kv_gather: rows of the cache as bf16.  A lane has 16 elements of a row and head.
// ---------------------------------------------------------------------------
template <int D, bool kIsFp4>
__global__ void __launch_bounds__(256) kv_gather_kernel(const __grid_constant__ KvGatherParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
  const int j = (int)(at % (D / 16));
  const long long line = at / (D / 16);  // (row, k or v, head)
  const int h = (int)(line % p.Hkv), which = (int)(line / p.Hkv % 2);
  const long long row = line / (2 * p.Hkv);
  if (row >= p.T) return;
  const int slot = p.slots[row];
  if (!slot_ok(p, slot)) return;
  const long long page = (long long)(slot >> p.page_shift) * p.Hkv + h;
  const long long token = (page << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
  float v[16];
  if constexpr (kIsFp4) {
    const uint2 w = *reinterpret_cast<const uint2*>(p.codes[which] + token * (D / 2) + 8 * j);
    const float s = e4m3_to_f32(static_cast<const uint8_t*>(p.scales[which])[token * (D / 16) + j]);
    const uint32_t in[2] = {w.x, w.y};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t f[4];
      e2m1x8_to_f16(in[x], f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        v[8 * x + 2 * i] = e.x * s, v[8 * x + 2 * i + 1] = e.y * s;
      }
    }
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(p.codes[which] + token * D + 16 * j);
    const float s = static_cast<const float*>(p.scales[which])[page];
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t f = e4m3x2_to_f16x2((uint16_t)(in[x] >> (16 * i)));
        const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&f));
        v[4 * x + 2 * i] = e.x * s, v[4 * x + 2 * i + 1] = e.y * s;
      }
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out[which]) + row * p.out_tok_stride[which] + h * p.out_head_stride[which] + 16 * j;
  reinterpret_cast<uint4*>(out)[0] = to_bf16(v);
  reinterpret_cast<uint4*>(out)[1] = to_bf16(v + 8);
}

}  // namespace

cudaError_t launch_kv_append_rotary(const KvRotaryParams& p, cudaStream_t stream) {
  if (p.x_bf16) return p.D == 64 ? launch_fmt<true, 64>(p, stream) : launch_fmt<true, 128>(p, stream);
  return p.D == 64 ? launch_fmt<false, 64>(p, stream) : launch_fmt<false, 128>(p, stream);
}

cudaError_t launch_kv_gather(const KvGatherParams& p, cudaStream_t stream) {
  const long long lanes = (long long)p.T * 2 * p.Hkv * (p.D / 16);
  const unsigned grid = (unsigned)((lanes + 255) / 256);
  if (p.fp4)
    return p.D == 64 ? launch_kernel(kv_gather_kernel<64, true>, grid, 256, 0, stream, 1, p)
                     : launch_kernel(kv_gather_kernel<128, true>, grid, 256, 0, stream, 1, p);
  return p.D == 64 ? launch_kernel(kv_gather_kernel<64, false>, grid, 256, 0, stream, 1, p)
                   : launch_kernel(kv_gather_kernel<128, false>, grid, 256, 0, stream, 1, p);
}

}  // namespace bsk
