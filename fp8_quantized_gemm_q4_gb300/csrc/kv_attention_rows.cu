// kv_attention_rows.cu -- attention over the paged 8-bit cache for requests with
// many rows (prompts, chunks): the mathematics is kv_attention.cu's, on tcgen05.
//
// A unit is 128 rows (row r = i * G + g: token i, head g of a KV head's group)
// against its cached tokens in tiles of 128.  The codes are exact in fp16 but not
// an operand type that fp16 may be multiplied with, so every tile is widened on
// the way: warps read the codes from L2, convert them and write K and V to shared
// memory as fp16 in the tensor core's 128-byte swizzled layout, both as rows of
// tokens (K-major for S = Q K^T, MN-major for O = P V).  q and
// the softmax weights are A operands in tensor memory and cost no shared
// memory traffic.  Per tile and SM: 1024 clocks of MMA, 512 of writing and 512 of
// the MMAs' reading 64 KB, 500 of exponentials, so the pieces balance where each
// runs beside the others:
//   warps 0-15   softmax, four threads per row, each a quarter of the columns: S
//                from tensor memory once, weights back into S's place, the running
//                (m, l), rare rescaling of O
//   warps 16-19  K codes -> fp16        warps 20-23  V codes -> fp16
//   warp 24      MMA issue: S(j + 1) = Q K^T goes ahead of O += P(j) V
//   warp 25      the next units, page ids and scales of the next tiles
// What bounds it: the softmax of a tile, whose steps follow one another (S, the
// maximum, the vote on the reference, the exponentials, the store) and whose
// warps have 1540 issue slots of about 2800 clocks a tile with the converters.  832
// threads leave 72 registers each, 20 bytes of which are spilled.
// B = 2, 2048 rows x 32 heads over 4000 to 8000 tokens, D = 128: 265 us (840 TFLOP/s); the
// same with D = 64, half the MMAs: 225.  With two threads per row 303, with one 2.5 times the MMAs' time.  Also built and
// measured: two groups of warps on alternate tiles, each with an O of its own and
// Q in shared memory (303 us: both operands of Q K^T from shared memory take all of
// its bandwidth), with one O and a reference settled in turn (324 us: P in S's place
// holds the next scores back), and with columns of its own for P (443 us: there
// is room for one P only).
// The tiles of all units form one list that is cut into equal shares, one CTA
// each; units cut between CTAs are joined by the last CTA to finish a piece.
#include "kv_attention.cuh"

namespace bsk {
namespace {

constexpr int kM = 128;           // rows of a unit
constexpr int kN = 128;           // cached tokens of a tile
constexpr int kGroups = kN / 16;  // groups of 16 tokens: each lies in one page
constexpr int kSoft = 16, kMma = kSoft + 8;  // softmax warps, the MMA warp
constexpr int kThreads = (kMma + 2) * 32;
constexpr int kOwn = kN / 4;      // columns of S a softmax thread has
// Least tiles worth a CTA of its own: a unit's pieces are joined by one CTA, which
// takes about 0.7 us a piece (of 64 rows x 4 heads over 6000 tokens: 58 us with 2
// tiles a CTA, 32 with 4, 30 with 6, 34 with 12; over 2000 tokens 25, 25, 27, 37).
constexpr int kMinTiles = 4;
constexpr int kPageSlots = 8;     // tiles whose pages are known ahead
constexpr int kUnitSlots = 4;     // units known ahead
constexpr int kCounters = 1024;   // arrival counters at the head of the workspace
constexpr int kTmemCols = 512;
// Tensor memory columns: S twice (the weights of 32 tokens go into the first half of
// the 32 columns that their scores had), O, Q
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384;

// A unit as the roles read it; t0 == t1: the share is done
struct UnitInfo {
  int t0, t1, nt, len;     // its tiles within the share, all its tiles, cached tokens
  int b;                   // request
  int h, rt, row0, n;      // KV head, row tile; the request's first row and rows
  long long at;            // its first tile's place in the list
};

template <int D>
struct RowsSmem {
  alignas(1024) uint8_t k[2][kN * D * 2];  // [D / 64][token][64 columns]
  alignas(1024) uint8_t v[2][kN * D * 2];  // the same of V
  float4 page[kPageSlots][kGroups];        // first row of codes (int, -1: none), K scale, log2 of V scale, 1 / V scale
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2];
  uint64_t page_full[kPageSlots], page_empty[kPageSlots], o_done, unit_done, q_full, drain;
  UnitInfo unit[kUnitSlots];
  uint64_t unit_full[kUnitSlots], unit_empty[kUnitSlots];
  float swap[4][kM];                       // between the four threads of a row
  // of the unit of that number modulo 8, if NaN codes of V were taken out where not every row
  // sees them: the number + 1, request, KV head, the first token of such tiles
  int4 nan_unit[8];
  long long scan[kThreads / 32];
  long long start_at;
  int start[3];
  // tiles in the list and CTAs that share them, for the joins: in registers through
  // the tiles they cost the softmax its room there (287 us, not 265, for the prompts above)
  long long total;
  int shares;
  uint32_t tmem;
  int abort_flag, last;
};

// fp16 x fp16 -> fp32; A K-major, B K-major or (mn) MN-major
__device__ __forceinline__ uint32_t idesc_f16(int M, int N, bool mn) {
  return (1u << 4) | (static_cast<uint32_t>(mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] B[smem]^T
__device__ __forceinline__ void mma_ts_f16(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A unit and where its tiles lie in the list
struct Unit {
  int b, h, rt;              // request, KV head, row tile
  int row0, n, len, rts;     // the request's first row, rows, cached tokens, row tiles
  int nt;                    // tiles
  long long at;              // the first one's place in the list
};
__device__ __forceinline__ bool takes(const KvAttentionParams& p, const Rows& r, int G) {
  return r.in > 0 && (long long)r.n * G > p.few_rows;
}
__device__ __forceinline__ int row_tiles(const Rows& r, int G) { return (int)(((long long)r.in * G + kM - 1) / kM); }
// Tiles that the unit's last row sees (one at least)
__device__ __forceinline__ int unit_tiles(int n, int len, int G, int rt) {
  const int last = (int)min((long long)n - 1, ((long long)rt * kM + kM - 1) / G);
  return max(1, (len - n + last + 1 + kN - 1) / kN);
}
__device__ __forceinline__ void load_request(const KvAttentionParams& p, int G, Unit& u) {
  const Rows r = rows_of(p, u.b);
  u.row0 = r.row0;
  u.n = r.n;
  u.len = cached(p, u.b);
  u.rts = row_tiles(r, G);
}
__device__ __forceinline__ void next_unit(const KvAttentionParams& p, int G, Unit& u) {
  u.at += u.nt;
  if (++u.rt == u.rts) {
    u.rt = 0;
    if (++u.h == p.Hkv) {
      u.h = 0;
      while (++u.b < p.B)
        if (takes(p, rows_of(p, u.b), G)) break;
      if (u.b >= p.B) return;  // the list ends here, and so does the last share
      load_request(p, G, u);
    }
  }
  u.nt = unit_tiles(u.n, u.len, G, u.rt);
}
template <int D>
__device__ __forceinline__ long long piece_at(int cta, int first_cta) {
  return ((long long)cta * 2 + (cta == first_cta)) * (kM * (D + 2));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// NaN into the columns part * D / 4 .. of a row whose tokens from .. to - 1 hold NaN
// codes of V there, in the output (dst) or the unit's piece.  Out of line, for units
// that meet none.
template <int D>
__device__ __noinline__ void put_nan(const KvAttentionParams& p, int b, int h, int part, int from, int to,
                                     __nv_bfloat16* dst, float* piece) {
  for (int x = from; x < to; ++x) {
    const int id = p.table[b * p.ld_table + (x >> p.page_shift)];
    if ((unsigned)id >= (unsigned)p.num_pages) continue;
    const uint8_t* code =
        p.v_codes + ((((long long)id * p.Hkv + h) << p.page_shift) + (x & ((1 << p.page_shift) - 1))) * D;
    for (int d = part * (D / 4); d < (part + 1) * (D / 4); ++d)
      if ((code[d] & 0x7f) == 0x7f) {
        if (dst)
          dst[d] = __ushort_as_bfloat16(0x7fff);
        else
          piece[(d & ~3) * kM + (d & 3)] = __int_as_float(0x7fffffff);
      }
  }
}

// all softmax warps: barrier 1; the four with the same 32 rows: barriers 2 to 5
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoft * 32) : "memory"); }
__device__ __forceinline__ void rows_sync(int rows) { asm volatile("bar.sync %0, 128;" ::"r"(2 + rows) : "memory"); }
__device__ __forceinline__ bool any_of(int bar, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(bar), "r"(threads), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool softmax_any(bool x) { return any_of(1, kSoft * 32, x); }
__device__ __forceinline__ bool rows_any(int rows, bool x) { return any_of(2 + rows, 128, x); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_rows_kernel(const __grid_constant__ KvAttentionParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = RowsSmem<D>;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.Hkv;
  const WaitGuard wg{&sm.abort_flag, p.status, p.wait_ns};
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.k_full[s], 4);
      mbar_init(&sm.v_full[s], 4);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_empty[s], 1);
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], kSoft);
    }
    for (int s = 0; s < kPageSlots; ++s) {
      mbar_init(&sm.page_full[s], 1);
      mbar_init(&sm.page_empty[s], kSoft + 8);
    }
    for (int s = 0; s < kUnitSlots; ++s) {
      mbar_init(&sm.unit_full[s], 1);
      mbar_init(&sm.unit_empty[s], kSoft + 8 + 1);
    }
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.unit_done, 1);
    mbar_init(&sm.q_full, kSoft);
    mbar_init(&sm.drain, 1);
    fence_barrier_init();
    sm.abort_flag = 0;
  }
  if (tid < 8) sm.nan_unit[tid] = make_int4(0, 0, 0, 0);
  // whoever goes on after a wait that gave up finds no page here, or an old one
  if (tid < kPageSlots * kGroups) sm.page[tid / kGroups][tid % kGroups].x = __int_as_float(-1);
  if (warp == kMma) {
    tmem_alloc(&sm.tmem, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  griddep_launch_dependents();

  // Each thread sums the tiles of `per` requests in a row; the one whose
  // requests hold the share's first tile finds its unit.
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  auto request_tiles = [&](int b) {  // of one KV head
    const Rows r = rows_of(p, b);
    if (!takes(p, r, G)) return 0ll;
    const int len = cached(p, b), rts = row_tiles(r, G);
    long long x = 0;
    for (int rt = 0; rt < rts; ++rt) x += unit_tiles(r.n, len, G, rt);
    return x;
  };
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += request_tiles(b);
    const Rows r = rows_of(p, b);
    if ((long long)r.n * G > p.most_rows) record_status(p.status, kStatusOffsets, 53);
    if (r.bad || length_bad(p, b)) record_status(p.status, kStatusOffsets, 54);
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(kFullMask, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  tc_fence_after();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm.scan[w];
    total += sm.scan[w];
  }
  total *= p.Hkv;
  before *= p.Hkv;
  const int shares = (int)min((long long)gridDim.x, (total + kMinTiles - 1) / kMinTiles);
  if (tid == 0) sm.total = total, sm.shares = shares;
  const bool works = (int)blockIdx.x < shares;
  const long long t_first = works ? total * blockIdx.x / shares : 0;
  const long long t_last = works ? total * (blockIdx.x + 1) / shares : 0;
  if (works && t_first >= before && t_first < before + mine * p.Hkv) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const long long x = request_tiles(b);
      if (x && t_first < at + x * p.Hkv) {
        const int h = (int)((t_first - at) / x);
        at += h * x;
        const int n = rows_of(p, b).n, len = cached(p, b);
        int rt = 0;
        for (;; ++rt) {
          const int nt = unit_tiles(n, len, G, rt);
          if (t_first < at + nt) break;
          at += nt;
        }
        sm.start[0] = b;
        sm.start[1] = h;
        sm.start[2] = rt;
        sm.start_at = at;
        break;
      }
      at += x * p.Hkv;
    }
  }
  __syncthreads();
  const uint32_t tmem = sm.tmem;

  uint32_t c = 0;  // tiles of the share so far: ring places and phases follow from it in every role
  uint32_t k = 0;  // units so far, likewise
  // the next unit, for a whole warp; false after a wait that gave up
  auto unit_open = [&](const UnitInfo*& u) {
    const bool ok = mbar_wait(&sm.unit_full[k % kUnitSlots], (k / kUnitSlots) & 1, wg, 74);
    u = &sm.unit[k % kUnitSlots];
    return __all_sync(kFullMask, ok) != 0;
  };
  auto unit_close = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.unit_empty[k % kUnitSlots]);
    ++k;
  };

  if (warp < kSoft) {
    // ------------------------------------------------------------ softmax: four threads per row
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // quarter of the columns, of the rows, row of the unit
    const int part = warp >> 2, rows = warp & 3, r128 = tid & (kM - 1);
    struct Row {
      int i, hq;     // token, query head
      bool in;
      float qscale;
    };
    // q to tensor memory, fp16 by a power of two; the scores of the unit before are done
    auto load_q = [&](const UnitInfo& u) {
      Row w;
      const long long r = (long long)u.rt * kM + r128;
      w.i = (int)(r / G), w.hq = u.h * G + (int)(r % G);
      w.in = r < (long long)u.n * G && u.row0 + w.i < p.T;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (u.row0 + (long long)w.i) * p.q_tok_stride +
                               w.hq * p.q_head_stride + part * (D / 4);
      uint4 v[D / 32];
#pragma unroll
      for (int x = 0; x < D / 32; ++x) v[x] = w.in ? __ldg(reinterpret_cast<const uint4*>(q) + x) : make_uint4(0, 0, 0, 0);
      float amax = 0.0f;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint32_t y[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
        for (int z = 0; z < 4; ++z)
          amax = max3(amax, fabsf(__uint_as_float(y[z] << 16)), fabsf(__uint_as_float(y[z] & 0xffff0000u)));
      }
      rows_sync(rows);  // what was in swap has been read
      sm.swap[part][r128] = amax;
      rows_sync(rows);
      const int up = fp16_up(fmaxf(fmaxf(sm.swap[0][r128], sm.swap[1][r128]), fmaxf(sm.swap[2][r128], sm.swap[3][r128])));
      const float mul = exp2i(up);
      w.qscale = exp2i(-up) * p.scale_log2;
#pragma unroll
      for (int x = 0; x < D / 32; x += 2) {
        const uint32_t y[8] = {v[x].x, v[x].y, v[x].z, v[x].w, v[x + 1].x, v[x + 1].y, v[x + 1].z, v[x + 1].w};
        uint32_t h[8];
#pragma unroll
        for (int z = 0; z < 8; ++z)
          h[z] = pack_f16x2(__uint_as_float(y[z] << 16) * mul, __uint_as_float(y[z] & 0xffff0000u) * mul);
        tmem_st8(lanes + kColQ + part * (D / 8) + 4 * x, h);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);
      return w;
    };
    Row row = {};
    const UnitInfo* u;
    // the softmax warps go on or end together, whichever of them gave up
    bool dead = softmax_any(!unit_open(u));
    if (!dead && u->t0 < u->t1) row = load_q(*u);
    while (!dead && u->t0 < u->t1) {
      const int t0 = u->t0, t1 = u->t1;
      const bool in = row.in;
      const float qscale = row.qscale;
      const int seen = in ? max(0, u->len - u->n + row.i + 1) : 0;
      float m = -INFINITY, l = 0.0f;  // the row's reference; the sum of this thread's weights
      for (int t = t0; t < t1; ++t, ++c) {
        const uint32_t sb = c & 1, slot = c % kPageSlots;
        mbar_wait(&sm.s_full[sb], (c >> 1) & 1, wg, 61);
        mbar_wait(&sm.page_full[slot], (c / kPageSlots) & 1, wg, 60);
        tc_fence_after();
        const uint32_t s_at = lanes + kColS + sb * kN + part * kOwn;
        const int limit = seen - t * kN - part * kOwn;  // of its columns, those that this row sees
        const float4* page = &sm.page[slot][part * (kGroups / 4)];
        uint32_t raw[kOwn];
        tmem_ld32(s_at, raw);
        tmem_ld_wait();
        if (limit < kOwn) {
#pragma unroll
          for (int y = 0; y < kOwn; ++y)
            if (y >= limit) raw[y] = __float_as_uint(-INFINITY);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int h = 0; h < kOwn / 16; ++h) {
          const float4 pg = page[h];
          float g = __uint_as_float(raw[16 * h]);
#pragma unroll
          for (int y = 1; y < 15; y += 2)
            g = max3(g, __uint_as_float(raw[16 * h + y]), __uint_as_float(raw[16 * h + y + 1]));
          g = fmaxf(g, __uint_as_float(raw[16 * h + 15]));
          mx = fmaxf(mx, fmaf(g, qscale * pg.y, pg.z));
        }
        if (rows_any(rows, mx > m + 8.0f)) {
          sm.swap[part][r128] = mx;
          rows_sync(rows);
          mx = fmaxf(fmaxf(sm.swap[0][r128], sm.swap[1][r128]), fmaxf(sm.swap[2][r128], sm.swap[3][r128]));
          const bool up = mx > m + 8.0f;
          const float f = up ? ex2(m - mx) : 1.0f;
          m = up ? mx : m;
          l *= f;
          if (t > t0) {
            // the product of the tile before; those further back were done before
            // these scores, so the phase's parity says which one it is
            mbar_wait(&sm.o_done, (c - 1) & 1, wg, 62);
            tc_fence_after();
#pragma unroll 1
            for (int x = part * (D / 4); x < (part + 1) * (D / 4); x += 8) {
              uint32_t o[8];
              tmem_ld8(lanes + kColO + x, o);
              tmem_ld_wait();
#pragma unroll
              for (int y = 0; y < 8; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st8(lanes + kColO + x, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int h = 0; h < kOwn / 16; ++h) {
          const float4 pg = page[h];
          // a scale is positive, or 0 with pg.z = -infinity: masked scores must not meet the 0
          const float f1 = fmaxf(qscale * pg.y, 1e-37f), o1 = pg.z - ref;
          const float2 f = make_float2(f1, f1), off = make_float2(o1, o1);
          float2 sum = make_float2(0.0f, 0.0f);
          uint32_t w[8];
#pragma unroll
          for (int y = 0; y < 16; y += 2) {
            const float2 z = __ffma2_rn(make_float2(__uint_as_float(raw[16 * h + y]), __uint_as_float(raw[16 * h + y + 1])), f, off);
            const float2 e = make_float2(ex2(z.x), ex2(z.y));
            sum = __fadd2_rn(sum, e);
            w[y / 2] = pack_f16x2(e.x, e.y);
          }
          tmem_st8(s_at + 8 * h, w);
          l = fmaf(sum.x + sum.y, pg.w, l);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.p_full[sb]);
          mbar_arrive(&sm.page_empty[slot]);
        }
      }
      // ---- the unit's rows.  Its scores are done: the next unit's q goes first,
      // so that the next scores run beside what follows.
      const Row was = row;
      const uint32_t unit = k;
      const int row0 = u->row0, nt = u->nt;
      const long long at = u->at;
      unit_close();
      dead = softmax_any(!unit_open(u));
      if (!dead && u->t0 < u->t1) row = load_q(*u);
      mbar_wait(&sm.unit_done, unit & 1, wg, 64);
      tc_fence_after();
      rows_sync(rows);  // swap has been read
      sm.swap[part][r128] = l;
      rows_sync(rows);
      l = (sm.swap[0][r128] + sm.swap[1][r128]) + (sm.swap[2][r128] + sm.swap[3][r128]);
      const bool alone = t0 == 0 && t1 == nt;
      const float inv = !alone ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
      const long long tr = row0 + (long long)was.i, lse_at = tr * p.Hq + was.hq;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + tr * p.out_tok_stride + was.hq * p.out_head_stride;
      float* slot = p.work + ((long long)blockIdx.x * 2 + (t0 == 0)) * (kM * (D + 2));
#pragma unroll 1
      for (int x = part * (D / 4); x < (part + 1) * (D / 4); x += 16) {
        uint32_t o[16];
        tmem_ld16(lanes + kColO + x, o);
        tmem_ld_wait();
#pragma unroll
        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * inv);
        if (in && alone) {
#pragma unroll
          for (int y = 0; y < 16; y += 8) {
            uint32_t w[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) w[z] = pack_bf16x2(__uint_as_float(o[y + 2 * z]), __uint_as_float(o[y + 2 * z + 1]));
            *reinterpret_cast<uint4*>(dst + x + y) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (in) {
#pragma unroll
          for (int y = 0; y < 16; y += 4)
            *reinterpret_cast<uint4*>(slot + (x + y) * kM + r128 * 4) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
        }
        __syncwarp();
      }
      tc_fence_before();
      if (sm.nan_unit[unit & 7].x == (int)unit + 1) {
        const int4 bad = sm.nan_unit[unit & 7];
        if (in) put_nan<D>(p, bad.y, bad.z, part, max(bad.w, t0 * kN), min(seen, t1 * kN), alone ? dst : nullptr, slot + r128 * 4);
        __syncwarp();
      }
      if (alone) {
        if (in && part == 0 && p.lse) p.lse[lse_at] = lse_of(m, l);
      } else {
        if (in && part == 0) *reinterpret_cast<float2*>(slot + kM * D + 2 * r128) = make_float2(m, l);
        __threadfence();
        const long long all = sm.total;
        const int c0 = (int)(((at + 1) * sm.shares - 1) / all), c1 = (int)(((at + nt) * sm.shares - 1) / all);
        softmax_sync();
        if (tid == 0) {
          const int old = atomicAdd(p.counters + c0, 1);
          __threadfence();
          sm.last = old == c1 - c0;
          if (sm.last) p.counters[c0] = 0;
        }
        softmax_sync();
        if (sm.last && in) {
          float mx = -INFINITY, sum = 0.0f;
          for (int x = c0; x <= c1; ++x) mx = fmaxf(mx, __ldcg(p.work + piece_at<D>(x, c0) + kM * D + 2 * r128));
          const float ref = mx == -INFINITY ? 0.0f : mx;
          for (int x = c0; x <= c1; ++x) {
            const float2 e = __ldcg(reinterpret_cast<const float2*>(p.work + piece_at<D>(x, c0) + kM * D + 2 * r128));
            sum += e.y * ex2(e.x - ref);
          }
          const float by = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll 1
          for (int d = part * (D / 4); d < (part + 1) * (D / 4); d += 8) {
            float acc[8] = {};
#pragma unroll 4
            for (int x = c0; x <= c1; ++x) {
              const float* from = p.work + piece_at<D>(x, c0);
              const float4 v = __ldcg(reinterpret_cast<const float4*>(from + d * kM + r128 * 4));
              const float4 w = __ldcg(reinterpret_cast<const float4*>(from + (d + 4) * kM + r128 * 4));
              const float f = ex2(__ldcg(from + kM * D + 2 * r128) - ref);
              acc[0] += f * v.x, acc[1] += f * v.y, acc[2] += f * v.z, acc[3] += f * v.w;
              acc[4] += f * w.x, acc[5] += f * w.y, acc[6] += f * w.z, acc[7] += f * w.w;
            }
            *reinterpret_cast<uint4*>(dst + d) = make_uint4(pack_bf16x2(acc[0] * by, acc[1] * by), pack_bf16x2(acc[2] * by, acc[3] * by),
                                                            pack_bf16x2(acc[4] * by, acc[5] * by), pack_bf16x2(acc[6] * by, acc[7] * by));
          }
          if (part == 0 && p.lse) p.lse[lse_at] = lse_of(mx, sum);
        }
        __syncwarp();
      }
    }
    if (dead && tid == 0 && works) {
      // a wait gave up: the pieces that were not written count as arrived, so
      // that the counters are zero again for the next call
      Unit w = {};
      w.b = sm.start[0], w.h = sm.start[1], w.rt = sm.start[2], w.at = sm.start_at;
      load_request(p, G, w);
      w.nt = unit_tiles(w.n, w.len, G, w.rt);
      for (uint32_t x = 0; w.at < t_last; ++x, next_unit(p, G, w)) {
        if (x < k || (w.at >= t_first && w.at + w.nt <= t_last)) continue;
        const int c0 = (int)(((w.at + 1) * sm.shares - 1) / sm.total), c1 = (int)(((w.at + w.nt) * sm.shares - 1) / sm.total);
        if (atomicAdd(p.counters + c0, 1) == c1 - c0) p.counters[c0] = 0;
      }
    }
  } else if (warp < kSoft + 8) {
    // ------------------------------------------------------------ K (four warps) and V (four warps) codes -> fp16
    // Lane: 16 codes of a token (and the token's place among its warp's), such
    // that eight lanes in a row store to eight different chunks.  The codes of
    // a tile are read while those of the tile before are converted.
    constexpr int kSteps = kN * D / (128 * 16);           // 16-byte loads per thread
    constexpr int kStepTokens = kN / kSteps;
    const bool is_v = warp >= kSoft + 4;
    const int w = warp & 3, q = lane & 3;
    const int panel = D == 128 ? (lane >> 3) & 1 : 0;
    const int tok = D == 128 ? w * 4 + (lane >> 4) * 2 + ((lane >> 2) & 1) : w * 8 + (lane >> 2);
    const uint8_t* codes = (is_v ? p.v_codes : p.k_codes) + (tok & 15) * D + 64 * panel + 16 * q;
    const uint32_t base = smem_u32(is_v ? sm.v[0] : sm.k[0]) + panel * (kN * 128) + tok * 128;
    const uint32_t at0 = base + (((2 * q) ^ (tok & 7)) << 4), at1 = base + (((2 * q + 1) ^ (tok & 7)) << 4);
    uint64_t* full = is_v ? sm.v_full : sm.k_full;
    uint64_t* empty = is_v ? sm.v_empty : sm.k_empty;
    for (;;) {
      const UnitInfo* u;
      if (!unit_open(u)) break;
      const int t0 = u->t0, t1 = u->t1, len = u->len;
      if (t0 == t1) break;
      // from this token on, some row of the unit does not see V: a NaN code there
      // would reach that row with a weight of 0.  Tiles with such tokens go without
      // theirs, and the rows that see one get the NaN at the end.
      const int hidden = max(0, len - u->n + (int)((long long)u->rt * kM / G) + 1);
      const int4 bad = make_int4((int)k + 1, u->b, u->h, hidden / kN * kN);
      unit_close();
      uint4 raw[kSteps];
      auto load = [&](uint4& r, int s, int left, const float4* page) {
        const int x = s * kStepTokens + tok, first = __float_as_int(page[x >> 4].x);
        r = make_uint4(0, 0, 0, 0);
        if (first >= 0 && x < left) r = __ldg(reinterpret_cast<const uint4*>(codes + (long long)first * D));
      };
      auto page_open = [&](uint32_t c) {
        mbar_wait(&sm.page_full[c % kPageSlots], (c / kPageSlots) & 1, wg, 65);
        return sm.page[c % kPageSlots];
      };
      auto page_close = [&](uint32_t c) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.page_empty[c % kPageSlots]);
      };
      const float4* page = page_open(c);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) load(raw[s], s, len - t0 * kN, page);
      page_close(c);
      for (int t = t0; t < t1; ++t, ++c) {
        const bool more = t + 1 < t1;
        if (more) page = page_open(c + 1);
        const uint32_t b = c & 1, to = b * (kN * D * 2);
        if (is_v && (t + 1) * kN > hidden) {
          uint32_t any = 0;
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            const uint4 n = make_uint4(nan_codes(raw[s].x), nan_codes(raw[s].y), nan_codes(raw[s].z), nan_codes(raw[s].w));
            any |= n.x | n.y | n.z | n.w;
            raw[s] = make_uint4(without(raw[s].x, n.x), without(raw[s].y, n.y), without(raw[s].z, n.z), without(raw[s].w, n.w));
          }
          if (any) sm.nan_unit[(bad.x - 1) & 7] = bad;
        }
        mbar_wait(&empty[b], ((c >> 1) & 1) ^ 1, wg, 66);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const uint32_t in[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
          uint32_t h[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            e4m3x4_to_f16(in[y], h[2 * y], h[2 * y + 1]);
          }
          st_shared_v4(at0 + to + s * (kStepTokens * 128), h[0], h[1], h[2], h[3]);
          st_shared_v4(at1 + to + s * (kStepTokens * 128), h[4], h[5], h[6], h[7]);
          if (more) load(raw[s], s, len - (t + 1) * kN, page);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[b]);
        if (more) page_close(c + 1);
      }
    }
  } else if (warp == kMma) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t kPanel = kN * 128;  // 64 columns of a tile
    const uint32_t idesc_s = idesc_f16(kM, kN, false), idesc_o = idesc_f16(kM, D, true);
    bool ok = true;
    auto scores = [&](uint32_t c) {  // S(c) = Q K(c)^T
      const uint32_t b = c & 1;
      ok = ok && mbar_wait_warp(&sm.k_full[b], (c >> 1) & 1, wg, 69);
      if (!ok) return;
      tc_fence_after();
      const uint64_t dk = smem_desc(smem_u32(sm.k[b]), 16, 1024, kLayoutSw128);
      if (elect_one()) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          mma_ts_f16(tmem + kColS + b * kN, tmem + kColQ + 8 * x, dk + (x / 4) * (kPanel >> 4) + 2 * (x % 4), idesc_s, x > 0);
        tc_commit(&sm.k_empty[b]);
        tc_commit(&sm.s_full[b]);
      }
      __syncwarp();
    };
    for (;;) {
      const UnitInfo* u;
      ok = unit_open(u) && ok;
      if (!ok) break;
      const int t0 = warp_bcast(u->t0), t1 = warp_bcast(u->t1);
      if (t0 == t1) break;
      ok = ok && mbar_wait_warp(&sm.q_full, k & 1, wg, 70);
      tc_fence_after();
      scores(c);
      for (int t = t0; t < t1; ++t, ++c) {
        // S(c + 1) goes where P(c - 1) was: its product has been issued before
        if (t + 1 < t1) scores(c + 1);
        const uint32_t b = c & 1;
        ok = ok && mbar_wait_warp(&sm.v_full[b], (c >> 1) & 1, wg, 71);
        ok = ok && mbar_wait_warp(&sm.p_full[b], (c >> 1) & 1, wg, 72);
        if (!ok) continue;
        tc_fence_after();
        // 64 columns a panel, 8 tokens 1024 bytes
        const uint64_t dv = smem_desc(smem_u32(sm.v[b]), kPanel, 1024, kLayoutSw128);
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < kN / 16; ++x)
            mma_ts_f16(tmem + kColO, tmem + kColS + b * kN + (x / 2) * kOwn + 8 * (x % 2), dv + x * (16 * 128 >> 4), idesc_o,
                       t > t0 || x > 0);
          tc_commit(&sm.v_empty[b]);
          tc_commit(&sm.o_done);
          if (t + 1 == t1) tc_commit(&sm.unit_done);
        }
        __syncwarp();
      }
      unit_close();
    }
    if (elect_one()) {
      tc_commit(&sm.drain);
      mbar_drain(&sm.drain, 0, 1000000000ull);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ units; page ids and scales, four tiles at a time
    Unit u = {};
    if (works) {
      u.b = sm.start[0];
      u.h = sm.start[1];
      u.rt = sm.start[2];
      u.at = sm.start_at;
      load_request(p, G, u);
      u.nt = unit_tiles(u.n, u.len, G, u.rt);
    }
    auto announce = [&](int t0, int t1) {
      const uint32_t slot = k % kUnitSlots;
      // a unit is never replaced before every role is done with it
      const bool ok = mbar_wait(&sm.unit_empty[slot], ((k / kUnitSlots) & 1) ^ 1, wg, 75);
      if (!__all_sync(kFullMask, ok)) return false;
      if (lane == 0) {
        sm.unit[slot] = UnitInfo{t0, t1, u.nt, u.len, u.b, u.h, u.rt, u.row0, u.n, u.at};
        mbar_arrive(&sm.unit_full[slot]);
      }
      __syncwarp();
      ++k;
      return true;
    };
    bool ok = true;
    while (works && u.at < t_last) {
      const int t0 = (int)max(0ll, t_first - u.at), t1 = (int)min((long long)u.nt, t_last - u.at);
      ok = announce(t0, t1);
      if (!ok) break;
      for (int t = t0; t < t1; t += 4) {
        const int j = lane & 7, tt = t + (lane >> 3), token = tt * kN + 16 * j;
        int first = -1;
        float ks = 0.0f, log_vs = -INFINITY, inv_vs = 0.0f;
        if (tt < t1 && token < u.len) {
          const int id = p.table[u.b * p.ld_table + (token >> p.page_shift)];
          if ((unsigned)id >= (unsigned)p.num_pages) {
            record_status(p.status, kStatusOffsets, 50);
          } else {
            first = (int)((((long long)id * p.Hkv + u.h) << p.page_shift) + (token & ((1 << p.page_shift) - 1)));
            ks = p.k_scales[(long long)id * p.Hkv + u.h];
            const float vs = p.v_scales[(long long)id * p.Hkv + u.h];
            log_vs = log2f(vs);
            inv_vs = 1.0f / vs;
          }
        }
        for (int x = 0; x < 4 && t + x < t1; ++x, ++c) {
          const uint32_t slot = c % kPageSlots;
          mbar_wait(&sm.page_empty[slot], ((c / kPageSlots) & 1) ^ 1, wg, 73);
          if (lane >> 3 == x) sm.page[slot][j] = make_float4(__int_as_float(first), ks, log_vs, inv_vs);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.page_full[slot]);
        }
      }
      next_unit(p, G, u);
    }
    if (ok) announce(0, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch(const KvAttentionLaunch& L, cudaStream_t stream) {
  // all of an SM's shared memory: one CTA an SM, as tensor memory has it
  constexpr int kSmem = 227 * 1024;
  static_assert(sizeof(RowsSmem<D>) + 1024 <= kSmem, "shared memory");
  return launch_kernel_smem(kv_attention_rows_kernel<D>, (unsigned)L.rows_grid, kThreads, kSmem, stream, L.p);
}

}  // namespace

int kv_attention_rows_grid(int sms) { return sms < kCounters ? sms : kCounters; }
size_t kv_attention_rows_piece_bytes(int D) { return (size_t)2 * kM * (D + 2) * sizeof(float); }

cudaError_t launch_kv_attention_rows(const KvAttentionLaunch& L, cudaStream_t stream) {
  return L.p.D == 64 ? launch<64>(L, stream) : launch<128>(L, stream);
}

}  // namespace bsk
