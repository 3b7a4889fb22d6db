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
#include "kv_attention.cuh"

namespace bsk {

namespace {

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
// Shared memory of a tile as TMA writes it: rows of 128 bytes (one token, or two
// for D = 64: rows of 64 bytes came in at half the rate), their 16-byte chunks
// exchanged by the 128-byte swizzle.
template <int D>
__device__ __forceinline__ int code_at(int tok, int chunk) {
  return D == 128 ? tok * 128 + ((chunk ^ (tok & 7)) << 4)
                  : (tok >> 1) * 128 + (((((tok & 1) << 2) | chunk) ^ ((tok >> 1) & 7)) << 4);
}
// Which of 8 tokens stands at place n of the MMA's token axis: any order does,
// as long as scores, masks and V rows agree.  For D = 128 places 2 i, 2 i + 1
// are four tokens apart, so that the 16-byte loads of K meet no bank twice.
template <int D>
__device__ __forceinline__ int token_of(int n) {
  return D == 128 ? (n >> 1) | ((n & 1) << 2) : n;
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

// ---------------------------------------------------------------------------
// Requests with at most few_rows rows per KV head (decode, drafts): bound by the
// cache stream.  Work is a list of (request, head, 8 rows) units of 64-token
// tiles, cut into contiguous shares of equal cost, whatever the lengths.  Three CTAs an
// SM take one each: a producer warp keeps 64 KB of codes in flight with TMA copies
// page by page, four consumer warps take 16 tokens of a tile each, and while one
// CTA joins the warps' results of a unit, the other two stream (one CTA with 12
// consumer warps lost 25 of 134 us to that).  Both products run transposed,
// tokens and then head columns on the MMA's M and the rows on its N = 8:
// S^T = K Q^T, O^T = V^T P^T; a group of 4 or 8 query heads fills N, where it would
// leave half of M = 16 empty.  More than 8 rows are units of their own beside the
// first, whose tiles they find in L2.
// 64 requests of 500 to 16000 tokens, 32 heads over 8, D = 128 (604 MB): 105 us, 0.85
// of HBM.  63 drafted tokens of 16 requests, 16 heads, D = 64, 16-token pages (60 MB):
// 24 us, bound by what a unit costs beside its tiles (q, the join of the warps, its
// piece); one token over 1000: 10 us, a chain of dependent reads.  Three CTAs an SM
// leave 128 registers a thread, of which 16 to 20 bytes are spilled.
// ---------------------------------------------------------------------------
constexpr int kTile = 64;          // cached tokens per stage
constexpr int kItems = 32;         // units listed at a time
constexpr int kMinTiles = 2;       // least cost worth a CTA of its own
// What a unit costs beside its tiles (q, the join of the warps, a piece), in tiles.
// us with 0 / 2 / 4 / 10: 64 decode requests 107.6 / 106.1 / 105.5 / 106, drafts over 16
// heads 24.8 / 23.3 / 22.9 / 23.9, 64 requests of 30 to 14000 tokens 20.6 / 17.4 / 16.6 / 16.7
constexpr int kUnitTiles = 4;
constexpr int kCounters = 1024;    // arrival counters at the head of the workspace
constexpr int kFewWarps = 4;       // consumers; one more warp produces
constexpr int kFewThreads = kFewWarps * 32 + 32;
constexpr int kFewCtas = 3;        // an SM

template <int D>
struct FewSmem {
  static constexpr int kStages = 512 / D;  // 64 KB of codes
  static constexpr int kStageBytes = 2 * kTile * D;
  alignas(1024) uint8_t kv[kStages][kStageBytes];  // K rows, then V rows
  float red[kFewWarps / 2][8 * D];
  float2 ml[kFewWarps][8];
  float4 group[kStages][4];  // per 16 tokens: K scale, log2 of V scale, 1 / V scale, valid tokens (int)
  // units of this share: request, KV head, first of the 8 rows, cached tokens;
  // first row, rows (true), rows within T; the share's tile at which the unit
  // would begin, its end tile within the share (0: no unit)
  int4 item[kItems];
  int4 rows[kItems];
  int begin[kItems], end[kItems];
  uint64_t full[kStages], empty[kStages];
  int2 scan[kFewThreads / 32];
  long long first_unit;      // of this share, counted over requests with tiles
  long long bound[2];        // its first tile in the list, the next share's
  int abort_flag, last;
};

// Tiles of each unit of a request in this kernel's list: none without rows or
// with more than few_rows per KV head, else one at least (rows that see nothing
// are written too).  Which kernel serves a request follows from its own rows and
// the call's, so that its result does not depend on the bound that the call gives.
__device__ __forceinline__ int few_tiles(const KvAttentionParams& p, int n, int len, int G) {
  return n <= 0 || (long long)n * G > p.few_rows ? 0 : max(1, (len + kTile - 1) / kTile);
}

// a / b for a >= 0 and b > 0: 64-bit division only where it takes one
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
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
template <int D>
__device__ __forceinline__ int red_at(int r, int d) {
  return r * D + ((((d >> 4) ^ ((r >> 1) & 1)) << 4) | ((d & 15) ^ (((r >> 2) & 1) << 3)));
}

template <int D>
__global__ void __launch_bounds__(kFewThreads, kFewCtas)
    kv_attention_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ KvAttentionParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = FewSmem<D>;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kStages = Smem::kStages, kWarps = kFewWarps, kThreads = kFewThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.Hkv;
  const WaitGuard wg{&sm.abort_flag, p.status, p.wait_ns};
  auto consumer_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); };
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
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
  int row0_own = 0, n_own = 0, len_own = 0;  // of the last of them: all there is while B <= threads
  int2 mine = make_int2(0, 0);
  for (int b = b0; b < b1; ++b) {
    const Rows own = rows_of(p, b);
    row0_own = own.row0, n_own = own.n;
    len_own = cached(p, b);
    const int nt = few_tiles(p, n_own, len_own, G), rt = nt ? (n_own * G + 7) / 8 : 0;
    mine.x += nt * rt;
    mine.y += rt;
    // one CTA tells: the check in all of them cost a call of prompts, whose other kernel
    // waits for this one to end, 11 of 276 us
    if (blockIdx.x == 0 && ((long long)n_own * G > p.most_rows || own.bad || length_bad(p, b)))
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
      int n = n_own, len = len_own;
      if (per > 1) n = rows_of(p, b).n, len = cached(p, b);
      const int nt = few_tiles(p, n, len, G);
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
        int row0 = row0_own, n = n_own, len = len_own;
        if (per > 1) {
          const Rows r = rows_of(p, b);
          row0 = r.row0, n = r.n, len = cached(p, b);
        }
        const int nt = few_tiles(p, n, len, G);
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
      // ---- producer: lane 4 k + j prepares group j (16 tokens) of the k-th of
      // eight tiles, then each tile's copies go out as its stage frees.  Page
      // ids are read two rounds of eight ahead and scales one, so that neither
      // latency stands between two rounds.
      struct Group {
        int id, tok, h, cnt;
        float ks, vs;
      };
      const int box = min(kTile, 1 << p.page_shift);  // tokens of a copy
      const int k = lane >> 2, j = lane & 3;
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
        x.ks = p.k_scales[(long long)x.id * p.Hkv + x.h];
        x.vs = p.v_scales[(long long)x.id * p.Hkv + x.h];
      };
      Group now = find(k_done), next = find(k_done + 8);
      scales(now);
      uint32_t s = k_done % kStages, ph = (k_done / kStages) & 1;
      for (int k0 = k_done; k0 < k_end; k0 += 8) {
        scales(next);
        const Group later = find(k0 + 16);
        const bool copies = now.cnt > 0 && (16 * j) % box == 0;
        const unsigned copy_mask = __ballot_sync(kFullMask, copies);
        const long long token = (((long long)now.id * p.Hkv + now.h) << p.page_shift) + (now.tok & ((1 << p.page_shift) - 1));
        const int row = (int)(token * D / 128);
        const int rounds = min(8, k_end - k0);
        float log_vs = 0.0f, inv_vs = 0.0f;
        for (int i = 0; i < rounds; ++i) {
          const bool ok = mbar_wait(&sm.empty[s], ph ^ 1, wg, 51);
          dead |= __any_sync(kFullMask, !ok) != 0;
          if (!dead) {
            if (k == i && copies) {
              tma_load_2d(&sm.kv[s][16 * j * D], &tm_k, &sm.full[s], 0, row);
              tma_load_2d(&sm.kv[s][(kTile + 16 * j) * D], &tm_v, &sm.full[s], 0, row);
            }
            if (i == 0) log_vs = log2f(now.vs), inv_vs = 1.0f / now.vs;  // the scales may still be on their way
            if (k == i) sm.group[s][j] = make_float4(now.ks, log_vs, inv_vs, __int_as_float(now.cnt));
            __syncwarp();
            const int n = __popc((copy_mask >> (4 * i)) & 15u);
            if (lane == 4 * i) mbar_arrive_expect_tx(&sm.full[s], (uint32_t)(n * box * D * 2));
            issued = k0 + i + 1;
          }
          if (++s == kStages) s = 0, ph ^= 1;
        }
        now = next;
        next = later;
      }
    } else {
      // ---- consumers: warp w takes tokens 16 w .. + 15 of every tile
      const int g = lane >> 2, c = lane & 3;
      constexpr int kQ = D / 64;  // 64-wide parts of a row
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
                                   (h * G + r % G) * p.q_head_stride + 16 * c;
          uint32_t w[8 * kQ];
#pragma unroll
          for (int x = 0; x < 2 * kQ; ++x) {
            const uint4 v = g < R ? *reinterpret_cast<const uint4*>(q + 64 * (x >> 1) + 8 * (x & 1)) : make_uint4(0, 0, 0, 0);
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
          for (int x = 0; x < 4 * kQ; ++x)  // k step x: columns 64 (x / 4) + 16 c + 4 (x % 4) .. + 3
#pragma unroll
            for (int y = 0; y < 2; ++y)
              qb[x][y] = pack_f16x2(__uint_as_float(w[2 * x + y] << 16) * mul,
                                    __uint_as_float(w[2 * x + y] & 0xffff0000u) * mul);
          const float undo = exp2i(-up) * p.scale_log2;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qscale[e] = __shfl_sync(kFullMask, undo, 4 * (2 * c + e));
            seen[e] = 2 * c + e < R ? len - n + (r0 + 2 * c + e) / G + 1 : 0;
          }
        }
        const int all_seen = len - n + r0 / G + 1;  // tokens that every row sees
        float o[D / 16][4] = {};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        const int begin = sm.begin[im];
        for (; tile < end; ++tile) {
          mbar_wait(&sm.full[stage], phase, wg, 52);
          const float4 sc = sm.group[stage][warp];
          const int cnt = min(__float_as_int(sc.w), 16);  // after a wait that gave up, whatever lies here
          if (cnt > 0) {
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

        // ---- the warps' (m, l, o) to one: o[a] holds columns 16 a + 2 g and + 1
        // (e / 2) of rows 2 c and + 1 (e % 2)
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
        auto put = [&] {
#pragma unroll
          for (int a = 0; a < D / 16; ++a)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<float2*>(buf + red_at<D>(2 * c + e, 16 * a + 2 * g)) = make_float2(o[a][e], o[a][2 + e]);
        };
        if (warp >= kWarps / 2) put();
        consumer_sync();
        if (warp < kWarps / 2) {
#pragma unroll
          for (int a = 0; a < D / 16; ++a)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 add = *reinterpret_cast<const float2*>(buf + red_at<D>(2 * c + e, 16 * a + 2 * g));
              o[a][e] += add.x, o[a][2 + e] += add.y;
            }
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
            const float4 v = *reinterpret_cast<const float4*>(&sm.red[w][red_at<D>(r, d)]);
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
        __threadfence();
        // the shares that hold the unit's first and last tile
        const long long first = t_first + begin + (base + im + 1) * kUnitTiles;  // on the axis of costs
        const int c0 = (int)quotient((first + 1) * shares - 1, cost), c1 = (int)quotient((first + nt) * shares - 1, cost);
        consumer_sync();
        if (tid == 0) {
          const int old = atomicAdd(p.counters + c0, 1);
          __threadfence();
          sm.last = old == c1 - c0;
          if (sm.last) p.counters[c0] = 0;
        }
        consumer_sync();
        if (sm.last) {
          for (int r = warp; r < R; r += kWarps) {
            float mx = -INFINITY;
            for (int x = c0 + lane; x <= c1; x += 32) mx = fmaxf(mx, __ldcg(p.work + piece_at<D>(x, c0) + 8 * D + 2 * r));
#pragma unroll
            for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, d));
            const float ref = mx == -INFINITY ? 0.0f : mx;
            float acc[D / 32] = {}, sum_l = 0.0f;
#pragma unroll 4
            for (int x = c0; x <= c1; ++x) {
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

template <int D>
cudaError_t launch_few(const KvAttentionLaunch& L, cudaStream_t stream) {
  constexpr int kSmem = (int)sizeof(FewSmem<D>) + 1024;
  return launch_kernel_smem(kv_attention_few_kernel<D>, (unsigned)L.few_grid, kFewThreads, kSmem, stream, L.tm_k, L.tm_v,
                            L.p);
}

}  // namespace

int kv_attention_few_grid(int sms) { return kFewCtas * sms < kCounters ? kFewCtas * sms : kCounters; }
size_t kv_attention_piece_bytes(int D) { return (size_t)2 * 8 * (D + 2) * sizeof(float); }
int kv_attention_box(int page_size) { return min(page_size, kTile); }

cudaError_t launch_kv_attention(const KvAttentionLaunch& L, cudaStream_t stream) {
  const KvAttentionParams& p = L.p;
  const int G = p.Hq / p.Hkv;
  if (G <= p.few_rows) {
    cudaError_t e = p.D == 64 ? launch_few<64>(L, stream) : launch_few<128>(L, stream);
    if (e != cudaSuccess) return e;
  }
  if (p.most_rows <= p.few_rows) return cudaSuccess;
  return launch_kv_attention_rows(L, stream);
}

}  // namespace bsk
