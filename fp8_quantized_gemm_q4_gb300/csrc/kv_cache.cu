// kv_cache.cu -- the pages of the 8-bit KV cache: block tables and slots from
// request lengths (kv_plan), pages given back (kv_release), and new keys and
// values quantized into their slots (kv_append).
//
// Pages hold 2^page_shift tokens.  Codes are e4m3 [page][KV head][token][D],
// one fp32 power-of-two scale per (page, KV head).
#include <limits.h>

#include "decode.h"
#include "kv_cache.cuh"

namespace bsk {

// ---------------------------------------------------------------------------
// kv_plan: with before = ceil(seq / page), after = ceil((seq + new) / page),
// need = after - before and end = inclusive sum of need over the requests,
// request b takes the entries n_free - 1 - (end_b - need_b) - j, j < need_b, of
// the free list; it fits if need_b == 0 or end_b <= n_free.  Every CTA scans
// all lengths (a few kB from L2) and then handles its own rows of the slot
// map and its own share of the taken pages, so one launch does and nothing
// waits on another CTA: slots read the table only below `before`, the table is
// written only from `before` on.  Its bytes are nothing (1024 requests and 20000
// rows: 0.2 MB): 4.2 us for 64 requests, 5.3 us for 1024, of which a launch with
// dependent reads takes about 2 (kv_append's) and the rest goes to the scan of two
// 64-bit sums by 1024 threads and its barriers.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

// First index with v[i] > x, in the ascending v[0, n).
__device__ __forceinline__ int upper_bound(const int* v, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Block-wide inclusive scan of (a, b); the sums over the block are returned
// in ta, tb.  All threads of the block call it.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& ta, long long& tb) {
  __shared__ long long wa[32], wb[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long va = __shfl_up_sync(kFullMask, a, d), vb = __shfl_up_sync(kFullMask, b, d);
    if (lane >= d) a += va, b += vb;
  }
  __syncthreads();  // the sums of an earlier call have been read
  if (lane == 31) wa[warp] = a, wb[warp] = b;
  __syncthreads();
  long long sa = lane < warps ? wa[lane] : 0, sb = lane < warps ? wb[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long va = __shfl_up_sync(kFullMask, sa, d), vb = __shfl_up_sync(kFullMask, sb, d);
    if (lane >= d) sa += va, sb += vb;
  }
  ta = __shfl_sync(kFullMask, sa, 31);
  tb = __shfl_sync(kFullMask, sb, 31);
  const long long pa = __shfl_sync(kFullMask, sa, warp ? warp - 1 : 0);
  const long long pb = __shfl_sync(kFullMask, sb, warp ? warp - 1 : 0);
  if (warp) a += pa, b += pb;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const __grid_constant__ KvPlanParams p) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ int sm[];
  int* cu = sm;                // [B + 1] rows before each request
  int* ends = cu + p.B + 1;    // [B]
  int* seqs = ends + p.B;      // [B], -1: lengths that break the contract
  const int tid = threadIdx.x, page = 1 << p.page_shift;
  const int n_free = min(max(*p.n_free, 0), p.capacity);
  long long new_sum = 0, need_sum = 0;
  if (tid == 0) cu[0] = 0;
  for (int base = 0; base < p.B; base += kPlanThreads) {
    const int b = base + tid;
    long long added = 0, need = 0;
    if (b < p.B) {
      int seq = p.seq_lens[b];
      added = max(p.new_lens[b], 0);
      const long long last = (long long)seq + added;
      if (seq < 0 || p.new_lens[b] < 0 || last > ((long long)p.max_pages << p.page_shift)) seq = -1;
      if (seq >= 0) need = ((last + page - 1) >> p.page_shift) - (((long long)seq + page - 1) >> p.page_shift);
      seqs[b] = seq;
    }
    long long new_block, need_block;
    block_scan2(added, need, new_block, need_block);
    if (b < p.B) {
      cu[b + 1] = (int)min(new_sum + added, (long long)INT_MAX);
      ends[b] = (int)min(need_sum + need, (long long)INT_MAX);
    }
    new_sum += new_block;
    need_sum += need_block;
  }
  __syncthreads();
  const int total = p.B ? ends[p.B - 1] : 0;
  const int rows = cu[p.B];

  if (blockIdx.x == 0) {
    for (int b = tid; b <= p.B; b += kPlanThreads) p.cu_new[b] = cu[b];
    for (int b = tid; b < p.B; b += kPlanThreads) {
      const bool fits = ends[b] <= n_free || ends[b] == (b ? ends[b - 1] : 0);
      const int seq = seqs[b];
      p.kv_lens[b] = seq >= 0 && fits ? seq + cu[b + 1] - cu[b] : 0;
      if (seq < 0) record_status(p.status, kStatusOffsets, 40);
      if (!fits) record_status(p.status, kStatusPages, 41);
    }
    if (tid == 0) {
      const int u = upper_bound(ends, p.B, n_free);
      *p.n_free_out = n_free - (u ? ends[u - 1] : 0);
      if (new_sum > p.T) record_status(p.status, kStatusOffsets, 42);
    }
  }

  const long long first = (long long)blockIdx.x * kPlanThreads + tid, step = (long long)gridDim.x * kPlanThreads;
  for (long long r = first; r < p.T; r += step) {
    int slot = -1;
    if (r < rows) {
      const int b = upper_bound(cu + 1, p.B, (int)r);
      const int seq = seqs[b], end0 = b ? ends[b - 1] : 0;
      if (seq >= 0 && (ends[b] <= n_free || ends[b] == end0)) {
        const int pos = seq + ((int)r - cu[b]);
        const int j = pos >> p.page_shift, before = (int)(((long long)seq + page - 1) >> p.page_shift);
        const long long id = j < before ? p.table[b * p.ld_table + j] : p.free_pages[n_free - 1 - end0 - (j - before)];
        const long long at = (id << p.page_shift) + (pos & (page - 1));
        if (id >= 0 && at <= INT_MAX) slot = (int)at;
      }
    }
    p.slots[r] = slot;
  }
  for (long long e = first; e < min(total, n_free); e += step) {
    const int b = upper_bound(ends, p.B, (int)e);
    if (ends[b] > n_free) break;  // ends ascend: the later ones do not fit either
    const int end0 = b ? ends[b - 1] : 0;
    const int before = (int)(((long long)seqs[b] + page - 1) >> p.page_shift);
    p.table[b * p.ld_table + before + ((int)e - end0)] = p.free_pages[n_free - 1 - (int)e];
  }
}

cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)(3 * p.B + 1) * sizeof(int);
  const long long ctas = ((long long)p.T + kPlanThreads - 1) / kPlanThreads;
  const unsigned grid = (unsigned)(ctas < 1 ? 1 : ctas > 148 ? 148 : ctas);
  return smem <= 48000 ? launch_kernel(kv_plan_kernel, grid, kPlanThreads, smem, stream, 1, p)
                       : launch_kernel_smem(kv_plan_kernel, grid, kPlanThreads, smem, stream, p);
}

// ---------------------------------------------------------------------------
// kv_release: the pages of finished requests go back on the end of the free
// list, in request order; their table entries become -1.  Entries that are
// negative already are left out, so that a page is never handed out twice.  One CTA:
// 3.2 us for 400 pages of 4 requests, 62 us for 61000 of 1024.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) kv_release_kernel(const __grid_constant__ KvReleaseParams p) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ int ends[];  // [B]
  const int tid = threadIdx.x, page = 1 << p.page_shift;
  const int n_free = min(max(*p.n_free, 0), p.capacity);
  long long sum = 0;
  for (int base = 0; base < p.B; base += kPlanThreads) {
    const int b = base + tid;
    long long n = 0, unused = 0, block, unused_block;
    if (b < p.B && p.done[b]) {
      n = ((long long)p.lens[b] + page - 1) >> p.page_shift;
      if (n < 0 || n > p.max_pages) {
        record_status(p.status, kStatusOffsets, 43);
        n = 0;
      }
    }
    block_scan2(n, unused, block, unused_block);
    if (b < p.B) ends[b] = (int)min(sum + n, (long long)INT_MAX);
    sum += block;
  }
  __syncthreads();
  const int entries = (int)min(sum, (long long)INT_MAX);
  int at = n_free;  // where the next page goes
  constexpr int kEach = 4;  // entries a thread has on their way
  for (int base = 0; base < entries; base += kEach * kPlanThreads) {
    int* entry[kEach];
    int id[kEach];
    bool missing = false;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = base + i * kPlanThreads + tid;
      id[i] = -1;
      if (e >= entries) continue;
      const int b = upper_bound(ends, p.B, e);
      entry[i] = p.table + b * p.ld_table + (e - (b ? ends[b - 1] : 0));
      id[i] = *entry[i];
      missing |= id[i] < 0;
    }
    // a page given back before, or a length that the table does not have
    if (missing) record_status(p.status, kStatusOffsets, 46);
    const bool gaps = __syncthreads_or(missing);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      long long rank = tid, unused = 0, here = min(entries - base - i * kPlanThreads, kPlanThreads), unused_here;
      if (here <= 0) break;
      if (gaps) {
        rank = id[i] >= 0;
        block_scan2(rank, unused, here, unused_here);
        --rank;
      }
      if (id[i] >= 0 && at + rank < p.capacity) {
        p.free_pages[at + rank] = id[i];
        *entry[i] = -1;
      }
      if (at + here > p.capacity && tid == 0) record_status(p.status, kStatusPages, 44);
      at = (int)min(at + here, (long long)p.capacity);
    }
  }
  if (tid == 0) *p.n_free = at;
}

cudaError_t launch_kv_release(const KvReleaseParams& p, cudaStream_t stream) {
  return launch_kernel(kv_release_kernel, 1, kPlanThreads, (size_t)p.B * sizeof(int), stream, 1, p);
}

// ---------------------------------------------------------------------------
// kv_positions: the place of every new token in its request, a row a thread, from the
// requests' row offsets in shared memory.  64 rows: 2.0 us, a launch and two dependent reads.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) kv_positions_kernel(const int* seq_lens, const int* cu_new, int B, int T, int* positions) {
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ int ends[];
  for (int b = threadIdx.x; b < B; b += 256) ends[b] = cu_new[b + 1];
  __syncthreads();
  const unsigned r = blockIdx.x * 256 + threadIdx.x;
  if (r >= (unsigned)T) return;
  const int b = upper_bound(ends, B, (int)r);
  positions[r] = b < B ? seq_lens[b] + ((int)r - cu_new[b]) : 0;
}

cudaError_t launch_kv_positions(const int* seq_lens, const int* cu_new, int B, int T, int* positions, cudaStream_t stream) {
  return launch_kernel(kv_positions_kernel, (unsigned)(((long long)T + 255) / 256), 256, (size_t)B * sizeof(int), stream, 1, seq_lens,
                       cu_new, B, T, positions);
}

// ---------------------------------------------------------------------------
// kv_append.  The rows of a call that lie in one page follow one another with
// ascending slots (a run).  A run's scale is the smallest power of two s, in
// [2^-32, 2^64], with amax <= 448 s; a run that does not begin its page takes
// the larger of that and the page's scale, and where the scale grows the
// page's earlier codes are rounded again to it.  Powers of two: a quotient by
// one is exact, and re-rounding changes only codes that fall among e4m3's
// subnormals.  What a lane reads stays in its registers between the maximum and the
// codes: with a warp a row, a run's first 8 rows of D = 128 (16 of 64), with a warp for
// 16 rows, 64 of bf16 (128) or 32 of fp32 (64); a longer run's rest is read
// again.  64 tokens of 8 heads: 2.1 us (launch and three dependent reads); 16384
// tokens, 100 MB: 22.9 us, 0.65 of HBM, bound by latency: with 168 registers a thread
// 10 warps an SM hide it, whose issue slots are 39 % busy (24 bytes a thread are
// spilled at D = 128, 76 in fp32).
// ---------------------------------------------------------------------------
constexpr int kAppendWarps = 4;
constexpr int kAppendThreads = kAppendWarps * 32;
// Rows from which a warp takes 16 rows instead of one, and the runs among them one
// after the other.  us, one row / 16 rows a warp (8 heads, D = 128, bf16):
//   prompts on 64-token pages, 16384 rows   80 / 22   1900 rows  14.5 / 8   512 rows  8.7 / 8
//   single tokens               4000 rows   19 / 44   2048 rows    11 / 29    64 rows  2.2 / 15
// How the rows fall into pages is known on the device only; calls of thousands of
// rows hold prompts, calls of hundreds are decode steps.
constexpr int kAppendWideRows = 2048, kWideRows = 16, kShort = 4;

// Eight elements of a row, as they lie in memory
template <bool kBf16>
struct Eight {
  uint32_t w[kBf16 ? 4 : 8];
  __device__ __forceinline__ void load(const void* x, long long at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + at * (kBf16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (kBf16 ? 1 : 2); ++i) {
      const uint4 v = p[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (kBf16) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    return __uint_as_float(w[i]);
  }
  // Running maximum of the finite magnitudes' bits, bf16 in pairs.  (One infinity's
  // scale would take all that the page holds to 0.)  Bits one step of the exponent
  // up keep their order as signed integers, and the non-finite ones turn negative.
  static constexpr uint32_t kUp = kBf16 ? 0x00800080u : 0x00800000u;
  __device__ __forceinline__ void amax(uint32_t& m) const {
#pragma unroll
    for (int i = 0; i < (kBf16 ? 4 : 8); ++i) {
      if constexpr (kBf16)
        m = __vmaxs2(m, (w[i] & 0x7fff7fffu) + kUp);
      else
        m = max((int)m, (int)((w[i] & 0x7fffffffu) + kUp));
    }
  }
  // of a warp's lanes, as fp32
  static __device__ __forceinline__ float amax_of(uint32_t m) {
    if constexpr (kBf16) m = max((int)(m << 16), (int)(m & 0xffff0000u));
    return __uint_as_float((uint32_t)__reduce_max_sync(kFullMask, (int)m) - 0x00800000u);
  }
  __device__ __forceinline__ uint2 codes(float inv) const {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __fmul2_rn(make_float2(value(2 * i), value(2 * i + 1)), make_float2(inv, inv));
      h[i] = f32x2_to_e4m3x2(v.x, v.y);
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  }
};

// A run of n rows from row `row` on, into page `id` at place off, by a warp.  What
// a lane reads stays in its registers, up to kKeep times 8 elements; a longer
// run's rest is read again.
template <bool kBf16, int D, int kKeep>
__device__ __forceinline__ void append_run(const KvAppendParams& p, int which, int h, int row, int n, int id, int off,
                                           int lane) {
  constexpr int kVecs = D / 8, kPass = 32 / kVecs;  // lanes a row, rows a pass
  const long long page = (long long)id * p.Hkv + h;
  const long long step = p.tok_stride[which] * kPass;
  const int r0 = lane / kVecs, col = lane % kVecs;
  long long at = (row + r0) * p.tok_stride[which] + h * p.head_stride[which] + col * 8;
  const long long again = at + kKeep * step;
  float* scale = p.scales[which] + page;
  uint8_t* codes = p.codes[which] + (page << p.page_shift) * D;
  const float old = off > 0 ? *scale : 0.0f;
  Eight<kBf16> kept[kKeep], more;
  uint32_t top = Eight<kBf16>::kUp;
#pragma unroll
  for (int i = 0; i < kKeep; ++i, at += step)
    if (r0 + i * kPass < n) kept[i].load(p.x[which], at);
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (r0 + i * kPass < n) kept[i].amax(top);
  for (int i = kKeep; r0 + i * kPass < n; ++i, at += step) {
    more.load(p.x[which], at);
    more.amax(top);
  }
  __syncwarp();
  const float s = page_scale<D>(codes, off, Eight<kBf16>::amax_of(top), old, lane);
  const float inv = 1.0f / s;
  uint2* out = reinterpret_cast<uint2*>(codes) + (off + r0) * kVecs + col;
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (r0 + i * kPass < n) out[i * 32] = kept[i].codes(inv);
  at = again;
  for (int i = kKeep; r0 + i * kPass < n; ++i, at += step) {
    more.load(p.x[which], at);
    out[i * 32] = more.codes(inv);
  }
  __syncwarp();  // the old scale has been read by all
  if (lane == 0) *scale = s;
}

// A warp per row that begins a run.
template <bool kBf16, int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const unsigned block = blockIdx.x / (2 * p.Hkv), head = blockIdx.x % (2 * p.Hkv);
  const int row = block * kAppendWarps + (threadIdx.x >> 5);
  if (row >= p.T) return;
  const int page = 1 << p.page_shift;
  // lane i has the slot of row - 1 + i: whether the row begins a run, and its length
  const int near = row - 1 + lane;
  const int mine = near >= 0 && near < p.T ? p.slots[near] : -1;
  const int slot = __shfl_sync(kFullMask, mine, 1), before = __shfl_sync(kFullMask, mine, 0);
  const int off = slot & (page - 1);
  if (slot < 0 || (off > 0 && before == slot - 1)) return;
  if (!slot_ok(p, slot)) return;
  const unsigned run = __ballot_sync(kFullMask, lane == 0 || (lane - 1 < page - off && mine == slot + lane - 1));
  int n = run == kFullMask ? 31 : __ffs(~run) - 2;
  if (n == 31)
    while (n < page - off && row + n < p.T && p.slots[row + n] == slot + n) ++n;
  append_run<kBf16, D, 4>(p, head / p.Hkv, head % p.Hkv, row, n, slot >> p.page_shift, off, lane);
}

// A warp for the runs that begin in 16 rows; the CTA's four warps take four heads
// of the same rows.
template <bool kBf16, int D>
__global__ void __launch_bounds__(kAppendThreads, 3) kv_append_wide_kernel(const __grid_constant__ KvAppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kWords = 5;  // 32 rows each, from first - 1 on: as far as a run can go
  const int lane = threadIdx.x & 31, heads = 2 * p.Hkv, groups = (heads + kAppendWarps - 1) / kAppendWarps;
  const int first = (int)(blockIdx.x / groups) * kWideRows;
  const int head = (int)(blockIdx.x % groups) * kAppendWarps + (threadIdx.x >> 5);
  if (head >= heads) return;
  const int page = 1 << p.page_shift;
  int slot[kWords];
  unsigned inside[kWords + 1];  // rows that carry on the run of the row before
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const int r = first - 1 + 32 * j + lane;
    slot[j] = r >= 0 && r < p.T ? p.slots[r] : -1;
  }
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    int before = __shfl_up_sync(kFullMask, slot[j], 1);
    const int last = j ? __shfl_sync(kFullMask, slot[j ? j - 1 : 0], 31) : -1;
    if (lane == 0) before = last;
    inside[j] = __ballot_sync(kFullMask, (slot[j] & (page - 1)) > 0 && slot[j] == before + 1 && before >= 0);
  }
  inside[kWords] = 0;
  const unsigned begins = __ballot_sync(kFullMask, slot[0] >= 0) & ~inside[0] & ((1u << (kWideRows + 1)) - 2);
  for (unsigned todo = begins; todo; todo &= todo - 1) {
    const int i = __ffs(todo) - 1, mine = __shfl_sync(kFullMask, slot[0], i);
    if (!slot_ok(p, mine)) continue;
    int n = 1;
    bool on = true;
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const unsigned w = __funnelshift_r(inside[j], inside[j + 1], i + 1);
      if (on) n += w == kFullMask ? 32 : __ffs(~w) - 1;
      on &= w == kFullMask;
    }
    // a short run passes through little code, a page's worth stays in registers
    if (n <= kShort)
      append_run<kBf16, D, kShort / (256 / D)>(p, head / p.Hkv, head % p.Hkv, first - 1 + i, n, mine >> p.page_shift,
                                               mine & (page - 1), lane);
    else
      append_run<kBf16, D, kBf16 ? 32 : 16>(p, head / p.Hkv, head % p.Hkv, first - 1 + i, n, mine >> p.page_shift,
                                            mine & (page - 1), lane);
  }
}

template <bool kBf16, int D>
static cudaError_t launch_append(const KvAppendParams& p, cudaStream_t stream) {
  const bool wide = p.T >= kAppendWideRows;
  const int rows = wide ? kWideRows : kAppendWarps, heads = wide ? (2 * p.Hkv + kAppendWarps - 1) / kAppendWarps : 2 * p.Hkv;
  cudaLaunchConfig_t cfg = {};
  // the heads of the same rows side by side: together they read whole rows
  cfg.gridDim = dim3((unsigned)(((long long)p.T + rows - 1) / rows * heads), 1, 1);
  cfg.blockDim = dim3(kAppendThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, kv_append_wide_kernel<kBf16, D>, p)
              : cudaLaunchKernelEx(&cfg, kv_append_kernel<kBf16, D>, p);
}

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream) {
  if (p.x_bf16) return p.D == 64 ? launch_append<true, 64>(p, stream) : launch_append<true, 128>(p, stream);
  return p.D == 64 ? launch_append<false, 64>(p, stream) : launch_append<false, 128>(p, stream);
}

}  // namespace bsk
