// lora.cu -- low-rank adapters of many requests beside a projection that they share:
//   out = y + s_a (x A_a^T) B_a^T,  a = the adapter of the row's request.
//
// A tile is up to 8 or 64 rows of one request, and a cluster of CTAs takes it: the CTAs
// share K, and their partial products t = x A^T (mma.sync, rows on M, ranks on N) meet in
// distributed shared memory, where every CTA adds them in the same order; then the CTAs share N.  t stays fp32 and enters the second product scaled and
// split into two bf16 (within 2^-16 of it), or three where out is fp32 (within 2^-28);
// products with the bf16 B are exact, sums fp32.
#include "decode.h"
#include "decode.cuh"

namespace bsk {
namespace {

constexpr int kThreads = 256, kWarps = 8;

__device__ __forceinline__ void mma_bf16_16x8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ uint4 load16(const void* p, bool in) {
  return in ? *static_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
}

// A request's rows within the call (none if they are not this launch's to take), its adapter,
// and whether its numbers break the contract
struct Rows {
  int row0, n, id;
  bool bad;
};
__device__ __forceinline__ Rows rows_of(const LoraParams& p, int b) {
  const int r0 = p.cu[b], r1 = p.cu[b + 1], w = p.which[b], n = r0 < 0 || r1 <= r0 ? 0 : max(0, min(r1, p.T) - r0);
  return {r0, n < p.least || n > p.most ? 0 : n, w >= p.adapters ? -1 : w,
          r0 < 0 || r1 < r0 || r1 > p.T || w >= p.adapters};
}

// The cluster's tile: requests in order, their rows in tiles of kRows.
struct Tile {
  int row0, rows, id;  // first row, rows, adapter (-1: none)
  bool there;
};
template <int kRows>
__device__ __forceinline__ Tile find_tile(const LoraParams& p, int tile, long long* scan, int4* found) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.B + kThreads - 1) / kThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  if (tid == 0) *found = make_int4(0, 0, -1, 0);
  long long mine = 0;  // offsets that break the contract may claim rows twice
  Rows r;              // of the last of them: all there is while B <= kThreads
  for (int b = b0; b < b1; ++b) {
    r = rows_of(p, b);
    if (r.bad && blockIdx.x == 0) record_status(p.status, kStatusOffsets, 57);
    mine += (r.n + kRows - 1) / kRows;
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(kFullMask, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) before += w < warp ? scan[w] : 0;
  if (tile >= before && tile < before + mine) {
    for (int b = b0; b < b1; ++b) {
      if (per > 1) r = rows_of(p, b);
      const int n = (r.n + kRows - 1) / kRows;
      const long long i = tile - before;
      if (i < n) {
        const int at = (int)i * kRows;
        *found = make_int4(r.row0 + at, min(kRows, r.n - at), r.id, 1);
        break;
      }
      before += n;
    }
  }
  __syncthreads();
  return {found->x, found->y, found->z, found->w != 0};
}

// Rows without an adapter: y to out, columns n0 .. n1 - 1
__device__ __forceinline__ void copy_rows(const LoraParams& p, const Tile& t, int n0, int n1) {
  if (p.out == p.y || n1 <= n0) return;
  const int es = p.bf16 ? 2 : 4, vecs = (n1 - n0) * es / 16;
  for (int x = threadIdx.x; x < t.rows * vecs; x += kThreads) {
    const long long row = t.row0 + x / vecs;
    const char* from = static_cast<const char*>(p.y) + (row * p.ldy + n0) * es;
    reinterpret_cast<uint4*>(static_cast<char*>(p.out) + (row * p.ldo + n0) * es)[x % vecs] = reinterpret_cast<const uint4*>(from)[x % vecs];
  }
}

// Terms that t is split into for outputs of this type, and their bits.  All but the last are
// cut, not rounded, so that every term has t's sign and none is infinite where t is not;
// a remainder of 0 becomes 2^-30 of t.  So the terms' products with an infinite element of B
// are infinities of one sign, as t's own, and those of an infinite t never meet inf - inf
// (down to |t| = 2^-96, below which that remainder underflows).
template <bool kBf16>
constexpr int kTerms = kBf16 ? 2 : 3;
template <int kTerm>
__device__ __forceinline__ void split(float t, uint32_t (&term)[kTerm]) {
  const uint32_t head = t == t ? __float_as_uint(t) & 0xffff0000u : 0x7fff0000u;
  const float least = __uint_as_float(head) * 0x1p-30f;
  term[0] = head >> 16;
#pragma unroll
  for (int i = 1; i < kTerm; ++i) {
    t -= __uint_as_float(term[i - 1] << 16);
    t = fabsf(t) > 0.0f ? t : least;  // of an infinite t the difference is NaN
    term[i] = i + 1 < kTerm ? __float_as_uint(t) >> 16 : pack_bf16x2(t, 0.0f) & 0xffffu;
  }
}
// Those of four values, two in a word
template <int kTerm>
__device__ __forceinline__ void split4(const float4& v, uint2 (&w)[kTerm]) {
  uint32_t a[kTerm], b[kTerm], c[kTerm], d[kTerm];
  split(v.x, a), split(v.y, b), split(v.z, c), split(v.w, d);
#pragma unroll
  for (int i = 0; i < kTerm; ++i) w[i] = make_uint2(a[i] | b[i] << 16, c[i] | d[i] << 16);
}

// t of the cluster: the CTAs' sums (kVecs float4 at `sums` in each) added in order of rank,
// scaled, as its terms at t, kVecs times 8 bytes each
template <int kVecs, int kTerm>
__device__ __forceinline__ void gather_t(const LoraParams& p, int id, int size, const float* sums, void* t) {
  const float scale = p.scales ? p.scales[id] : 1.0f;
  const uint32_t mine = smem_u32(sums);
  for (int x = threadIdx.x; x < kVecs; x += kThreads) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int r = 0; r < size; ++r) {
      const float4 e = ld_cluster(mapa_shared(mine + 16 * x, r));
      v.x += e.x, v.y += e.y, v.z += e.z, v.w += e.w;
    }
    v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
    uint2 w[kTerm];
    split4(v, w);
#pragma unroll
    for (int i = 0; i < kTerm; ++i) static_cast<uint2*>(t)[i * kVecs + x] = w[i];
  }
}

// Eight columns of a row of y: read, and written with the products added (accumulators e
// and e + 1 of the four tiles of a chunk)
template <bool kBf16>
struct Eight {
  static constexpr int kSize = kBf16 ? 2 : 4;
  uint4 v[kBf16 ? 1 : 2];
  __device__ __forceinline__ void load(const LoraParams& p, long long row, int n, bool in) {
    const char* from = static_cast<const char*>(p.y) + (row * p.ldy + n) * kSize;
#pragma unroll
    for (int i = 0; i < kSize / 2; ++i) v[i] = load16(from + 16 * i, in);
  }
  __device__ __forceinline__ void put(const LoraParams& p, long long row, int n, bool in, const float (&acc)[4][4], int e) const {
    if (!in) return;
    char* to = static_cast<char*>(p.out) + (row * p.ldo + n) * kSize;
    if constexpr (kBf16) {
      const uint32_t o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16x2(__uint_as_float(o[i] << 16) + acc[i][e], __uint_as_float(o[i] & 0xffff0000u) + acc[i][e + 1]);
      *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        reinterpret_cast<float4*>(to)[i] =
            make_float4(__uint_as_float(v[i].x) + acc[2 * i][e], __uint_as_float(v[i].y) + acc[2 * i][e + 1],
                        __uint_as_float(v[i].z) + acc[2 * i + 1][e], __uint_as_float(v[i].w) + acc[2 * i + 1][e + 1]);
    }
  }
};

// ---------------------------------------------------------------------------
// Few rows a request: tiles of 8 rows.  Operands come as 16 consecutive bytes of a row a
// lane: a lane's k are 8 c .. + 7 of every 32, the same for both operands, and its columns
// 8 c .. + 7 of 32, so that neither weights nor outputs pass through shared memory.  What
// the second product reads of B and y does not depend on t and is on its way before t is
// there.
// ---------------------------------------------------------------------------
constexpr int kFewRows = 8;

template <int kRank, int kTerm>
struct FewSmem {
  float part[kWarps][kFewRows][kRank];      // of the warps; [0]: of the CTA
  __nv_bfloat16 t[kTerm][kFewRows][kRank];  // the terms of the scaled t
  long long scan[kWarps];
  int4 tile;
};

template <int kRank, bool kBf16>
__global__ void __launch_bounds__(kThreads, kRank > 64 ? 1 : kRank > 32 ? 2 : 4) lora_few_kernel(const __grid_constant__ LoraParams p) {
  constexpr int kTerm = kTerms<kBf16>;
  __shared__ __align__(16) FewSmem<kRank, kTerm> sm;
  constexpr int kNT = kRank / 8, kKB = kRank / 32;  // tiles of 8 ranks, blocks of 32
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int size = (int)cluster_size(), rank = (int)cluster_ctarank();
  griddep_wait();
  griddep_launch_dependents();
  const Tile tile = find_tile<kFewRows>(p, (int)(blockIdx.x / size), sm.scan, &sm.tile);
  if (!tile.there) return;  // all CTAs of the cluster alike
  const int chunks = (p.N + 31) / 32;  // of 32 columns, shared by the CTAs
  const int c0 = (int)((long long)chunks * rank / size), c1 = (int)((long long)chunks * (rank + 1) / size);
  if (tile.id < 0) {
    copy_rows(p, tile, c0 * 32, min(p.N, c1 * 32));
    return;
  }
  const bool row_in = g < tile.rows;
  {
    // ---- t = x A^T: the warps share the CTA's part of K
    float acc[kNT][4] = {};
    const int blocks = (p.K + 31) / 32, parts = size * kWarps, part = rank * kWarps + warp;
    const int k0 = (int)((long long)blocks * part / parts), k1 = (int)((long long)blocks * (part + 1) / parts);
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + (tile.row0 + (long long)g) * p.ldx;
    const __nv_bfloat16* a = static_cast<const __nv_bfloat16*>(p.a) + (long long)tile.id * p.r * p.K;
#pragma unroll 2
    for (int k = k0; k < k1; ++k) {
      const int at = 32 * k + 8 * c;
      const bool in = at < p.K;
      const uint4 xa = load16(x + at, in && row_in);
      uint4 w[kNT];
#pragma unroll
      for (int n = 0; n < kNT; ++n) w[n] = load16(a + (long long)(8 * n + g) * p.K + at, in && 8 * n < p.r);
      const uint32_t f0[4] = {xa.x, 0, xa.y, 0}, f1[4] = {xa.z, 0, xa.w, 0};
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        if (8 * n >= p.r) break;
        mma_bf16_16x8(acc[n], f0, w[n].x, w[n].y);
        mma_bf16_16x8(acc[n], f1, w[n].z, w[n].w);
      }
    }
#pragma unroll
    for (int n = 0; n < kNT; ++n) *reinterpret_cast<float2*>(&sm.part[warp][g][8 * n + 2 * c]) = make_float2(acc[n][0], acc[n][1]);
  }
  __syncthreads();
  constexpr int kVecs = kFewRows * kRank / 4;  // of t
  for (int x = tid; x < kVecs; x += kThreads) {
    float4* at = reinterpret_cast<float4*>(&sm.part[0][0][0]) + x;
    float4 v = *at;
#pragma unroll
    for (int s = 1; s < kWarps; ++s) {
      const float4 w = at[s * kVecs];
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    *at = v;
  }
  __syncwarp();
  cluster_arrive();

  // ---- out = y + t B^T: a warp has every eighth chunk of columns.  Tile i of a chunk has
  // the columns 8 (n / 2) + 2 i + n % 2, n = 0 .. 7.
  const __nv_bfloat16* bw = static_cast<const __nv_bfloat16*>(p.b) + (long long)tile.id * p.N * p.r;
  const long long row = tile.row0 + (long long)g;
  uint4 w[4][kKB];
  Eight<kBf16> y;
  auto load = [&](int chunk) {
    y.load(p, row, 32 * chunk + 8 * c, row_in && chunk < c1 && 32 * chunk + 8 * c < p.N);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 32 * chunk + 8 * (g >> 1) + 2 * i + (g & 1);
#pragma unroll
      for (int k = 0; k < kKB; ++k)
        w[i][k] = load16(bw + (long long)n * p.r + 32 * k + 8 * c, chunk < c1 && n < p.N && 32 * k + 8 * c < p.r);
    }
  };
  int chunk = c0 + warp;
  load(chunk);
  __syncwarp();
  cluster_wait();
  gather_t<kVecs, kTerm>(p, tile.id, size, &sm.part[0][0][0], sm.t);
  __syncthreads();
  cluster_arrive();  // this CTA has read the others' sums
  uint4 t[kTerm][kKB];
#pragma unroll
  for (int h = 0; h < kTerm; ++h)
#pragma unroll
    for (int k = 0; k < kKB; ++k) t[h][k] = *reinterpret_cast<const uint4*>(&sm.t[h][g][32 * k + 8 * c]);
#pragma unroll 1
  for (; chunk < c1; chunk += kWarps) {
    float acc[4][4] = {};
#pragma unroll
    for (int h = kTerm - 1; h >= 0; --h)
#pragma unroll
      for (int k = 0; k < kKB; ++k) {
        const uint32_t f0[4] = {t[h][k].x, 0, t[h][k].y, 0}, f1[4] = {t[h][k].z, 0, t[h][k].w, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mma_bf16_16x8(acc[i], f0, w[i][k].x, w[i][k].y);
          mma_bf16_16x8(acc[i], f1, w[i][k].z, w[i][k].w);
        }
      }
    const Eight<kBf16> old = y;
    load(chunk + kWarps);
    old.put(p, row, 32 * chunk + 8 * c, row_in && 32 * chunk + 8 * c < p.N, acc, 0);
  }
  __syncwarp();
  cluster_wait();  // until the others have read this CTA's sums
}

// ---------------------------------------------------------------------------
// Many rows a request: tiles of 64 rows.  x and A, then B and y, come through a ring of
// shared memory with cp.async, so that the four warps that need a slice of weights read it
// from L2 once.  Warps: a block of 16 rows and half the ranks, then half the columns of a
// chunk.  Of t each CTA adds its share and hands it to all.
// 8190 rows of rank 64, K = 7168, N = 4096: 72 us (240 MB, 0.49 of HBM; 151 with the few rows' operands
// straight from L2, 133 with y not through the ring and one CTA adding all of t); 20000 rows of rank
// 32: 99 us, 0.73.  A CTA's 27 us there with clusters of eight: 1 to find its tile, 11 x A^T, 5 waiting
// for the cluster and exchanging, 9 t B^T; each part waits for its first slices, which three CTAs an SM
// cover in part, and then for shared memory (its data pipe 0.63 of the active cycles, the tensor pipe
// 0.35).  Tiles of 128 rows, which halve the reads of A and B and leave room for two CTAs: 71 us there, 106
// for 124 at 16384 rows, but 32 for 27 at 2048 rows and 64 for 40 over 64 requests; not kept.
// ---------------------------------------------------------------------------
constexpr int kManyRows = 64, kSlice = 64;  // rows of a tile; K, or columns, of a stage

// Shared memory: four stages of x and A, or in their place three of B and y, the last of
// which holds the CTA's sums until it is needed, and t's terms.
template <int kRank, bool kBf16>
struct ManySmem {
  static constexpr int kStages1 = 4, kStages2 = 3;
  static constexpr int kStage1 = (kManyRows + kRank) * kSlice * 2;
  static constexpr int kB = kSlice * kRank * 2, kPieces = kBf16 ? 2 : 4;  // bytes of B; 16-byte pieces of y a thread
  static constexpr int kStage2 = kB + kPieces * kThreads * 16;
  static constexpr int kT = kManyRows * kRank * 2, kSums = 2 * kT;        // bytes of a term of t, of the sums
  static constexpr int kSumsAt = (kStages2 - 1) * kStage2;
  static constexpr int kTAt = kSumsAt + (kSums > kStage2 ? kSums : kStage2);
  static constexpr int kEnd = kTAt + kTerms<kBf16> * kT;
  static constexpr int kBytes = kEnd > kStages1 * kStage1 ? kEnd : kStages1 * kStage1;
};

// Place of the 16-byte piece `chunk` of a row of x or A, of a column of B or of a row of t
// (kBytes each), pieces exchanged so that the eight rows, or columns, of a matrix that
// ldmatrix reads meet all banks
__device__ __forceinline__ uint32_t piece_at(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }
template <int kBytes>
__device__ __forceinline__ uint32_t column_at(int col, int chunk) {
  const int x = (col >> 3) & 3;
  return col * kBytes + ((chunk ^ (kBytes == 64 ? x : 2 * x + (col & 1))) << 4);
}
template <int kBytes>
__device__ __forceinline__ uint32_t t_at(int row, int chunk) {
  return row * kBytes + ((chunk ^ (kBytes == 64 ? (row >> 1) & 3 : row & 7)) << 4);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

// CTAs of an SM
constexpr int many_resident(int rank, bool bf16) { return rank > 64 ? 1 : rank > 32 && !bf16 ? 2 : 3; }

template <int kRank, bool kBf16>
__global__ void __launch_bounds__(kThreads, many_resident(kRank, kBf16)) lora_many_kernel(const __grid_constant__ LoraParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ long long scan[kWarps];
  __shared__ int4 found;
  using S = ManySmem<kRank, kBf16>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int size = (int)cluster_size(), rank = (int)cluster_ctarank();
  griddep_wait();
  griddep_launch_dependents();
  const Tile tile = find_tile<kManyRows>(p, (int)(blockIdx.x / size), scan, &found);
  if (!tile.there) return;  // all CTAs of the cluster alike
  const int chunks = (p.N + kSlice - 1) / kSlice;  // of columns, shared by the CTAs
  const int c0 = (int)((long long)chunks * rank / size), c1 = (int)((long long)chunks * (rank + 1) / size);
  if (tile.id < 0) {
    copy_rows(p, tile, c0 * kSlice, min(p.N, c1 * kSlice));
    return;
  }
  const int block = warp & 3, half = warp >> 2;
  const bool works = 16 * block < tile.rows;
  const uint32_t smem = smem_u32(smem_raw);

  // ---- t = x A^T
  constexpr int kNT = kRank / 16;  // tiles of 8 ranks of a warp
  {
    const int slices = (p.K + kSlice - 1) / kSlice;
    const int k0 = (int)((long long)slices * rank / size), k1 = (int)((long long)slices * (rank + 1) / size);
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + (long long)tile.row0 * p.ldx;
    const __nv_bfloat16* a = static_cast<const __nv_bfloat16*>(p.a) + (long long)tile.id * p.r * p.K;
    auto issue = [&](int k) {
      if (k < k1) {
        const uint32_t to = smem + (k - k0) % S::kStages1 * S::kStage1;
#pragma unroll
        for (int i = 0; i < kManyRows * 8 / kThreads; ++i) {
          const int v = i * kThreads + tid, row = v >> 3, piece = v & 7, at = kSlice * k + 8 * piece;
          const bool in = row < tile.rows && at < p.K;
          cp_async16(to + piece_at(row, piece), in ? x + row * p.ldx + at : x, in);
        }
#pragma unroll
        for (int i = 0; i < kRank * 8 / kThreads; ++i) {
          const int v = i * kThreads + tid, row = v >> 3, piece = v & 7, at = kSlice * k + 8 * piece;
          const bool in = row < p.r && at < p.K;
          cp_async16(to + kManyRows * 128 + piece_at(row, piece), in ? a + (long long)row * p.K + at : a, in);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    float acc[kNT][4] = {};
#pragma unroll
    for (int s = 0; s < S::kStages1 - 1; ++s) issue(k0 + s);
#pragma unroll 1
    for (int k = k0; k < k1; ++k) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages1 - 2) : "memory");
      __syncthreads();  // everybody's part of the stage is there, and the stage before has been read
      issue(k + S::kStages1 - 1);
      if (!works) continue;
      const uint32_t xs = smem + (k - k0) % S::kStages1 * S::kStage1, as = xs + kManyRows * 128;
#pragma unroll
      for (int j = 0; j < kSlice / 16; ++j) {
        uint32_t f[4];
        ldmatrix_x4(f, xs + piece_at(16 * block + (lane & 15), 2 * j + (lane >> 4)));
#pragma unroll
        for (int n = 0; n < kNT; n += 2) {
          uint32_t w[4];  // two tiles of 8 ranks
          ldmatrix_x4(w, as + piece_at(8 * (half * kNT + n) + (lane & 7) + 8 * (lane >> 4), 2 * j + ((lane >> 3) & 1)));
          mma_bf16_16x8(acc[n], f, w[0], w[1]);
          mma_bf16_16x8(acc[n + 1], f, w[2], w[3]);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // the ring has been read
    float* sums = reinterpret_cast<float*>(smem_raw + S::kSumsAt);
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      float* at = sums + (16 * block + g) * kRank + 8 * (half * kNT + n) + 2 * c;
      *reinterpret_cast<float2*>(at) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(at + 8 * kRank) = make_float2(acc[n][2], acc[n][3]);
    }
  }
  __syncwarp();
  cluster_arrive();

  // ---- out = y + t B^T.  Tile i of 32 columns has 8 (n / 2) + 2 i + n % 2, n = 0 .. 7, so that a
  // lane ends with eight columns in a row.
  constexpr int kRow = kRank * 2;  // bytes of a column of B, of a row of t
  const __nv_bfloat16* bw = static_cast<const __nv_bfloat16*>(p.b) + (long long)tile.id * p.N * p.r;
  const int ra = 16 * block + g, rb = ra + 8;
  const long long to_a = tile.row0 + (long long)ra, to_b = tile.row0 + (long long)rb;
  auto issue = [&](int k) {
    if (k < c1) {
      const uint32_t to = smem + (k - c0) % S::kStages2 * S::kStage2;
#pragma unroll
      for (int i = 0; i < kSlice * (kRank / 8) / kThreads; ++i) {
        const int v = i * kThreads + tid, col = v / (kRank / 8), piece = v % (kRank / 8), n = kSlice * k + col;
        const bool in = n < p.N && 8 * piece < p.r;
        cp_async16(to + column_at<kRow>(col, piece), in ? bw + (long long)n * p.r + 8 * piece : bw, in);
      }
      // y: what this thread will add to
      const int n = kSlice * k + 32 * half + 8 * c;
#pragma unroll
      for (int i = 0; i < S::kPieces; ++i) {
        const bool second = i >= S::kPieces / 2, in = n < p.N && (second ? rb : ra) < tile.rows;
        const char* from = static_cast<const char*>(p.y) + ((second ? to_b : to_a) * p.ldy + n) * (kBf16 ? 2 : 4) + 16 * (i % (S::kPieces / 2));
        cp_async16(to + S::kB + (i * kThreads + tid) * 16, in ? from : p.y, in);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < S::kStages2 - 1; ++s) issue(c0 + s);
  __syncwarp();
  cluster_wait();
  {
    // this CTA's share of t: the sums of all CTAs in order of rank, scaled, its terms to all
    constexpr int kVecs = kManyRows * kRank / 4;
    const float scale = p.scales ? p.scales[tile.id] : 1.0f;
    for (int x = kVecs * rank / size + tid; x < kVecs * (rank + 1) / size; x += kThreads) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
      for (int r = 0; r < size; ++r) {
        const float4 e = ld_cluster(mapa_shared(smem + S::kSumsAt + 16 * x, r));
        v.x += e.x, v.y += e.y, v.z += e.z, v.w += e.w;
      }
      v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
      const int row = x / (kRank / 4), half_piece = x % (kRank / 4);
      // ranks that there are not: an infinite x times their zeros in A is NaN
      if (4 * half_piece >= p.r) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      uint2 w[kTerms<kBf16>];
      split4(v, w);
      const uint32_t to = smem + S::kTAt + t_at<kRow>(row, half_piece >> 1) + 8 * (half_piece & 1);
#pragma unroll
      for (int i = 0; i < kTerms<kBf16>; ++i) {
#pragma unroll 8
        for (int r = 0; r < size; ++r) st_cluster(mapa_shared(to, r) + i * S::kT, w[i].x, w[i].y);
      }
    }
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
#pragma unroll 1
  for (int k = c0; k < c1; ++k) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages2 - 2) : "memory");
    __syncthreads();
    issue(k + S::kStages2 - 1);
    if (!works) continue;
    const uint32_t bs = smem + (k - c0) % S::kStages2 * S::kStage2;
    float acc[4][4] = {};
#pragma unroll
    for (int j = 0; j < kRank / 16; ++j) {
      uint32_t t[kTerms<kBf16>][4];
#pragma unroll
      for (int h = 0; h < kTerms<kBf16>; ++h)
        ldmatrix_x4(t[h], smem + S::kTAt + h * S::kT + t_at<kRow>(16 * block + (lane & 15), 2 * j + (lane >> 4)));
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        // lanes 0 .. 7: column n = lane of tile i, 16 .. 23: of tile i + 1; 8 .. 15 and 24 .. 31 the next 8 ranks
        const int n = lane & 7, col = 32 * half + 8 * (n >> 1) + 2 * (i + (lane >> 4)) + (n & 1);
        uint32_t w[4];
        ldmatrix_x4(w, bs + column_at<kRow>(col, 2 * j + ((lane >> 3) & 1)));
#pragma unroll
        for (int h = kTerms<kBf16> - 1; h >= 0; --h) {
          mma_bf16_16x8(acc[i], t[h], w[0], w[1]);
          mma_bf16_16x8(acc[i + 1], t[h], w[2], w[3]);
        }
      }
    }
    const int n = kSlice * k + 32 * half + 8 * c;
    const uint32_t ys = bs + S::kB + tid * 16;
    Eight<kBf16> y;
#pragma unroll
    for (int i = 0; i < S::kPieces / 2; ++i) y.v[i] = lds128(ys + i * kThreads * 16);
    y.put(p, to_a, n, n < p.N && ra < tile.rows, acc, 0);
#pragma unroll
    for (int i = 0; i < S::kPieces / 2; ++i) y.v[i] = lds128(ys + (S::kPieces / 2 + i) * kThreads * 16);
    y.put(p, to_b, n, n < p.N && rb < tile.rows, acc, 2);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int kRank, bool kBf16>
cudaError_t launch(const LoraParams& p, bool many, int cluster, long long tiles, cudaStream_t stream) {
  const unsigned grid = (unsigned)(tiles * cluster);
  if (!many) return launch_kernel(lora_few_kernel<kRank, kBf16>, grid, kThreads, 0, stream, cluster, p);
  constexpr int kSmem = ManySmem<kRank, kBf16>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(lora_many_kernel<kRank, kBf16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(lora_many_kernel<kRank, kBf16>, grid, kThreads, kSmem, stream, cluster, p);
}
template <bool kBf16>
cudaError_t launch_rank(const LoraParams& p, bool many, int cluster, long long tiles, cudaStream_t stream) {
  if (p.r <= 32) return launch<32, kBf16>(p, many, cluster, tiles, stream);
  return p.r <= 64 ? launch<64, kBf16>(p, many, cluster, tiles, stream) : launch<128, kBf16>(p, many, cluster, tiles, stream);
}

// Which tiles a request gets follows from its own rows, in two launches; T and B, which also count
// padding and requests without rows, say only whether one launch would do.  Tiles of 8 rows alone
// do up to kFewEach rows a request, and where all of them stand on the GPU at once in clusters of
// two; tiles of 64 alone where they are mostly full ones whatever the requests' lengths; what is
// between may hold prompts beside single tokens (us, 8 rows / 64 rows / both, K = 4096, N = 6144: rank 16, 4096
// rows of one request and 255 single ones 75 / 86 / 58, and 127 single ones 72 / 82 / 49, the one of 256 requests alone
// 47 / 62 / 37; rank 64 131 / 116 / 89, 128 / 111 / 71, 92 / 82 / 46; but 64 requests of 32 rows 27 / 24 / 29 and
// 40 / 28 / 31, for a launch without tiles takes 2 to 10).
constexpr int kTall = 32;  // rows from which a request's tiles have 64
constexpr long long kManyEach = 64, kFewEach = 8;
constexpr long long few_places(int r, int sms) { return (long long)sms * (r <= 32 ? 4 : r <= 64 ? 2 : 1); }

// Tiles of 8 rows for requests of up to `most`; at most `tiles` of them, of which `expected` to expect
cudaError_t launch_few(LoraParams p, int most, long long tiles, long long expected, int sms, cudaStream_t stream) {
  // Eight CTAs a tile, fewer where not all would be on the GPU at once, for each has its own
  // start and exchange (us with 8 / 4 / 2 / 1, K = 4096, N = 6144: rank 16, 1 request 6.3 / 8.6 / 12 / 19, 64
  // requests 10.4 / 10.3 / 12.6 / 19, 256 requests 36 / 26 / 25 / 28; rank 64, 256 requests 81 / 62 / 53 / 49).
  int cluster = 8;
  while (cluster > 1 && expected * cluster > few_places(p.r, sms)) cluster /= 2;
  p.least = 1, p.most = most;
  return p.bf16 ? launch_rank<true>(p, false, cluster, tiles, stream) : launch_rank<false>(p, false, cluster, tiles, stream);
}

// Tiles of 64 rows for requests of `least` rows and more, `requests` of them at most
cudaError_t launch_many(LoraParams p, int least, long long requests, int sms, cudaStream_t stream) {
  // The size whose CTAs take the fewest rounds on the GPU for their shares of a tile, the
  // smaller of equals: a round that is not full costs as much as one that is.  Clusters do
  // not fill the last twentieth (us with 8 / 6 / 4 / 3 / 2, K = N = 4096 but where given: rank 16, bf16,
  // 3584 rows 31 / 26 / 33 / 32 / 34, 4800 rows 37 / 38 / 34 / 42 / 36, 8192 rows, N = 6144, 66 / 62 / 79 / 57 / 77,
  // 9600 rows 56 / 60 / 62 / 67 / 60; rank 64, 8190 rows, K = 7168, 77 / 74 / 77 / 72 / 99; rank 128, 4096 rows
  // 94 / 76 / 65 / 83 / 59, 1200 rows 38 / 26 / 33 / 42 / 58; fp32, rank 16, 3000 rows 37 / 49 / 46 / 60 / 51).
  // Where other requests are the other launch's, the rounds of as few tiles as there may be count as well.
  const long long full = p.T / kManyRows, expected = full + (requests + 1) / 2;
  const long long at_once = (long long)sms * many_resident(p.r <= 32 ? 32 : p.r <= 64 ? 64 : 128, p.bf16) * 19 / 20;
  const auto rounds = [&](int size) {
    return (expected * size + at_once - 1) / at_once + (least > 1 ? ((full + 1) * size + at_once - 1) / at_once : 0);
  };
  int cluster = 8;
  for (const int size : {6, 4, 3, 2})
    if (rounds(size) * cluster <= rounds(cluster) * size) cluster = size;
  p.least = least, p.most = p.T;
  return p.bf16 ? launch_rank<true>(p, true, cluster, full + requests, stream)
                : launch_rank<false>(p, true, cluster, full + requests, stream);
}

}  // namespace

cudaError_t launch_lora(const LoraParams& p, int sms, cudaStream_t stream) {
  // every request may end in a tile that is not full, half of them do
  const long long requests = p.B < p.T ? p.B : p.T, few = p.T / kFewRows;
  const long long expected = p.T <= kFewRows * requests ? requests : few + requests / 2;
  if (p.T >= kManyEach * p.B) return launch_many(p, 1, requests, sms, stream);
  if (p.T <= kFewEach * p.B || 2 * expected <= few_places(p.r, sms))
    return launch_few(p, p.T, few + requests, expected, sms, stream);
  // (calls of less than kTall rows all fit, so neither grid is empty)
  constexpr int kEach = (kTall - 1 + kFewRows - 1) / kFewRows;  // most tiles of a request that is not tall
  const cudaError_t e = launch_few(p, kTall - 1, few < (kEach - 1) * requests ? few + requests : kEach * requests, requests, sms, stream);
  if (e != cudaSuccess) return e;
  return launch_many(p, kTall, requests < p.T / kTall ? requests : p.T / kTall, sms, stream);
}

}  // namespace bsk
