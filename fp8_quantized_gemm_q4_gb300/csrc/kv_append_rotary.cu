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
#include "decode.h"
#include "kv_cache.cuh"

namespace bsk {
namespace {

constexpr int kFp8 = 0, kFp8Wide = 1, kFp4 = 2;
constexpr int kHeads = 4;  // heads of a token that a warp goes through

template <int D>
constexpr int kLanes = D / 16;  // lanes of a row
template <int D>
constexpr int kRows = 32 / kLanes<D>;  // rows of a warp's pass

// A lane's two vectors of 8 elements of a row
struct Pair {
  int a, b;
};
__device__ __forceinline__ Pair vectors(const KvRotaryParams& p, int j) {
  const int n = p.rot >> 4;
  return !p.interleaved && j < n ? Pair{j, j + n} : Pair{2 * j, 2 * j + 1};
}

// Eight elements as floats
template <bool kBf16>
__device__ __forceinline__ void load8(const void* x, long long at, float* v) {
  const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + at * (kBf16 ? 2 : 4));
  if constexpr (kBf16) {
    const uint4 w = *from;
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(in[i] << 16), v[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
  } else {
    const uint4 w = from[0], z = from[1];
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
    v[4] = __uint_as_float(z.x), v[5] = __uint_as_float(z.y), v[6] = __uint_as_float(z.z), v[7] = __uint_as_float(z.w);
  }
}

// The angles of a lane's eight pairs
struct Turn {
  float c[8], s[8];
  bool on;
  __device__ __forceinline__ void load(const KvRotaryParams& p, int row, int j) {
    on = j < p.rot >> 4;
    if (!on) return;
    int at = p.positions[row];
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
// heads from `head` on, of kind 0 (q), 1 (k), 2 (v).
template <bool kBf16, int D>
__device__ __forceinline__ void flat_heads(const KvRotaryParams& p, int first, int kind, int head, int lane) {
  const int j = lane % kLanes<D>, row = first + lane / kLanes<D>;
  const int slot = row < p.T ? p.slots[row] : -1;
  const bool ok = slot_ok(p, slot);
  Turn turn;
  turn.on = false;
  if (ok && kind < 2) turn.load(p, row, j);
  const Pair at = vectors(p, j);
  const int heads = min(kHeads, (kind ? p.Hkv : p.Hq) - head);
  const void* x = kind ? p.x[kind - 1] : p.q;
  const long long step = kind ? p.head_stride[kind - 1] : p.q_head_stride;
  const long long from = row * (kind ? p.tok_stride[kind - 1] : p.q_tok_stride) + head * step;
  float v[kHeads][16];
#pragma unroll
  for (int h = 0; h < kHeads; ++h)
    if (ok && h < heads) {
      load8<kBf16>(x, from + h * step + 8 * at.a, v[h]);
      load8<kBf16>(x, from + h * step + 8 * at.b, v[h] + 8);
    }
  if (kind == 0) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.q_out) + row * p.qo_tok_stride + head * p.qo_head_stride;
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (ok && h < heads) {
        turn.apply(v[h], p.interleaved);
        *reinterpret_cast<uint4*>(out + h * p.qo_head_stride + 8 * at.a) = to_bf16(v[h]);
        *reinterpret_cast<uint4*>(out + h * p.qo_head_stride + 8 * at.b) = to_bf16(v[h] + 8);
      }
    return;
  }
  // who has the vector beside a, and the one beside b, in their groups of 16
  const int n = p.interleaved ? 0 : p.rot >> 4;
  auto owner = [&](int vec) { return vec < n ? vec : vec < 2 * n ? vec - n : vec >> 1; };
  auto second = [&](int vec) { return vec < n ? false : vec < 2 * n ? true : (vec & 1) != 0; };
  const int base = lane - j, oa = base + owner(at.a ^ 1), ob = base + owner(at.b ^ 1);
  const bool sa = second(at.a ^ 1), sb = second(at.b ^ 1);
  const long long line = ((((long long)(slot >> p.page_shift) * p.Hkv + head) << p.page_shift) + (slot & ((1 << p.page_shift) - 1)));
  uint32_t* codes = reinterpret_cast<uint32_t*>(p.codes[kind - 1]);
  uint8_t* scales = static_cast<uint8_t*>(p.scales[kind - 1]);
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (h >= heads) break;
    uint32_t ma = 0, mb = 0;
    if (ok) {
      turn.apply(v[h], p.interleaved);
      ma = amax8(v[h]), mb = amax8(v[h] + 8);
    }
    const uint32_t a0 = __shfl_sync(kFullMask, ma, oa), a1 = __shfl_sync(kFullMask, mb, oa);
    const uint32_t b0 = __shfl_sync(kFullMask, ma, ob), b1 = __shfl_sync(kFullMask, mb, ob);
    if (!ok) continue;
    const uint32_t fa = scale4(max(ma, sa ? a1 : a0)), fb = scale4(max(mb, sb ? b1 : b0));
    const long long to = line + ((long long)h << p.page_shift);
    codes[to * (D / 8) + at.a] = codes4(v[h], fa);
    codes[to * (D / 8) + at.b] = codes4(v[h] + 8, fb);
    if (!(at.a & 1)) scales[to * (D / 16) + at.a / 2] = (uint8_t)fa;
    if (!(at.b & 1)) scales[to * (D / 16) + at.b / 2] = (uint8_t)fb;
  }
}

// A run of n rows from row `row` on into page `id` at place off, one head of the keys
// (which = 0) or values, by kWarps warps (1, or all of the CTA); its rows up to kKeep
// passes stay in registers between the maximum and the codes, the rest is read again.
template <bool kBf16, int D, int kWarps, int kKeep>
__device__ __forceinline__ void append_run(const KvRotaryParams& p, int which, int h, int row, int n, int id, int off,
                                           int thread) {
  constexpr int kPass = kRows<D> * kWarps;
  const int lane = thread & 31, j = lane % kLanes<D>, r0 = thread / kLanes<D>;
  const Pair at = vectors(p, j);
  const long long page = (long long)id * p.Hkv + h;
  float* scale = static_cast<float*>(p.scales[which]) + page;
  uint8_t* codes = p.codes[which] + (page << p.page_shift) * D;
  const float old = off > 0 ? *scale : 0.0f;
  auto get = [&](int r, float(&v)[16]) {
    Turn turn;
    turn.on = false;
    if (which == 0) turn.load(p, row + r, j);
    const long long from = (long long)(row + r) * p.tok_stride[which] + h * p.head_stride[which];
    load8<kBf16>(p.x[which], from + 8 * at.a, v);
    load8<kBf16>(p.x[which], from + 8 * at.b, v + 8);
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
  float kept[kKeep][16];
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (r0 + i * kPass < n) get(r0 + i * kPass, kept[i]);
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (r0 + i * kPass < n) amax(kept[i]);
  for (int r = r0 + kKeep * kPass; r < n; r += kPass) {
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
  for (int r = r0 + kKeep * kPass; r < n; r += kPass) {
    float v[16];
    get(r, v);
    put(r, v);
  }
  __syncwarp();  // the old scale has been read by all
  if (thread == 0) *scale = s;
}

// Row `row` as the head of a run: its slot and the rows that go with it, or 0.  A warp.
__device__ __forceinline__ int run_at(const KvRotaryParams& p, int row, int lane, int& slot) {
  const int page = 1 << p.page_shift;
  // lane i has the slot of row - 1 + i
  const int near = row - 1 + lane;
  const int mine = near >= 0 && near < p.T ? p.slots[near] : -1;
  slot = __shfl_sync(kFullMask, mine, 1);
  const int before = __shfl_sync(kFullMask, mine, 0), off = slot & (page - 1);
  if (slot < 0 || (off > 0 && before == slot - 1) || !slot_ok(p, slot)) return 0;
  const unsigned run = __ballot_sync(kFullMask, lane == 0 || (lane - 1 < page - off && mine == slot + lane - 1));
  int n = run == kFullMask ? 31 : __ffs(~run) - 2;
  if (n == 31)
    while (n < page - off && row + n < p.T && p.slots[row + n] == slot + n) ++n;
  return n;
}

constexpr int kThreads = 128, kWideThreads = 256;
constexpr int kWindow = 64;  // rows whose runs a CTA of the wide form takes
constexpr int kWideRows = 2048;

template <bool kBf16, int D, int kFmt>
__global__ void __launch_bounds__(kFmt == kFp8Wide ? kWideThreads : kThreads)
    kv_append_rotary_kernel(const __grid_constant__ KvRotaryParams p, unsigned run_blocks) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kWarps = (kFmt == kFp8Wide ? kWideThreads : kThreads) / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (kFmt != kFp4 && blockIdx.x < run_blocks) {
    const unsigned block = blockIdx.x / (2 * p.Hkv), head = blockIdx.x % (2 * p.Hkv);
    const int which = head / p.Hkv, h = head % p.Hkv, page = 1 << p.page_shift;
    if constexpr (kFmt == kFp8) {
      // a warp per row that begins a run
      const int row = block * kWarps + warp;
      if (row >= p.T) return;
      int slot;
      const int n = run_at(p, row, lane, slot);
      if (n) append_run<kBf16, D, 1, 2>(p, which, h, row, n, slot >> p.page_shift, slot & (page - 1), lane);
    } else {
      // the runs that begin in a window of rows: short ones a warp each, others the CTA
      constexpr int kWords = 6, kShort = 2 * kRows<D>;  // 32 rows a word, from first - 1 on
      const int first = (int)block * kWindow;
      int slot[kWords];
      unsigned inside[kWords + 1];  // rows that carry on the run of the row before
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const int r = first - 1 + 32 * w + lane;
        slot[w] = r >= 0 && r < p.T ? p.slots[r] : -1;
      }
      uint64_t begins = 0;
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        int before = __shfl_up_sync(kFullMask, slot[w], 1);
        const int last = w ? __shfl_sync(kFullMask, slot[w ? w - 1 : 0], 31) : -1;
        if (lane == 0) before = last;
        inside[w] = __ballot_sync(kFullMask, (slot[w] & (page - 1)) > 0 && slot[w] == before + 1 && before >= 0);
        const unsigned begin = __ballot_sync(kFullMask, slot[w] >= 0) & ~inside[w];
        // bit i: row first + i
        if (w == 0) begins = begin >> 1;
        if (w == 1) begins |= (uint64_t)begin << 31;
        if (w == 2) begins |= (uint64_t)(begin & 1) << 63;
      }
      inside[kWords] = 0;
      int turn = 0;
      for (uint64_t todo = begins; todo; todo &= todo - 1) {
        const int i = __ffsll((long long)todo);  // its place from first - 1 on
        const int mine = __shfl_sync(kFullMask, i < 32 ? slot[0] : i < 64 ? slot[1] : slot[2], i & 31);
        if (!slot_ok(p, mine)) continue;
        int n = 1;
        bool on = true;
        const int whole = (i + 1) >> 5, rest = (i + 1) & 31;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          if (w < whole) continue;
          const unsigned bits = __funnelshift_r(inside[w], inside[w + 1], rest);
          if (on) n += bits == kFullMask ? 32 : __ffs(~bits) - 1;
          on &= bits == kFullMask;
        }
        n = min(n, page - (mine & (page - 1)));
        if (n <= kShort) {
          if (turn++ % kWarps == warp)
            append_run<kBf16, D, 1, 2>(p, which, h, first - 1 + i, n, mine >> p.page_shift, mine & (page - 1), lane);
        } else {
          append_run<kBf16, D, kWarps, 2>(p, which, h, first - 1 + i, n, mine >> p.page_shift, mine & (page - 1), threadIdx.x);
        }
      }
    }
    return;
  }
  const int cq = (p.Hq + kHeads - 1) / kHeads, ck = kFmt == kFp4 ? (p.Hkv + kHeads - 1) / kHeads : 0, parts = cq + 2 * ck;
  const long long task = (long long)(blockIdx.x - run_blocks) * kWarps + warp;
  const long long group = task / parts;
  const int part = (int)(task % parts);
  if (group * kRows<D> >= p.T) return;
  const int kind = part < cq ? 0 : part < cq + ck ? 1 : 2;
  const int chunk = kind == 0 ? part : part - cq - (kind - 1) * ck;
  flat_heads<kBf16, D>(p, (int)(group * kRows<D>), kind, chunk * kHeads, lane);
}

template <bool kBf16, int D, int kFmt>
cudaError_t launch(const KvRotaryParams& p, cudaStream_t stream) {
  constexpr int threads = kFmt == kFp8Wide ? kWideThreads : kThreads, warps = threads / 32;
  const long long rows = kFmt == kFp8Wide ? kWindow : warps;
  const long long runs = kFmt == kFp4 ? 0 : (p.T + rows - 1) / rows * 2 * p.Hkv;
  const long long parts = (p.Hq + kHeads - 1) / kHeads + (kFmt == kFp4 ? (p.Hkv + kHeads - 1) / kHeads * 2 : 0);
  const long long flat = ((p.T + kRows<D> - 1) / kRows<D> * parts + warps - 1) / warps;
  return launch_kernel(kv_append_rotary_kernel<kBf16, D, kFmt>, (unsigned)(runs + flat), threads, 0, stream, 1, p,
                       (unsigned)runs);
}
template <bool kBf16, int D>
cudaError_t launch_fmt(const KvRotaryParams& p, cudaStream_t stream) {
  if (p.fp4) return launch<kBf16, D, kFp4>(p, stream);
  return p.T >= kWideRows ? launch<kBf16, D, kFp8Wide>(p, stream) : launch<kBf16, D, kFp8>(p, stream);
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
