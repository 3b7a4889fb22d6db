// lora.cu -- low-rank adapters of many requests beside a projection that they share:
//   out = y + s_a (x A_a^T) B_a^T,  a = the adapter of the row's request.
//
// A tile is up to 16 or 64 rows of one request, and a cluster of CTAs takes it in one
// launch: the CTAs share K, each warp brings a slice of x and of A to registers and
// multiplies (mma.sync, 16 rows on M, ranks on N); the partial products t = x A^T meet in
// distributed shared memory, where every CTA adds them in the same order; then the CTAs
// share N.  t stays fp32 and enters the second product scaled and split into two bf16
// (hi + lo, within 2^-17 of it; products with the bf16 B are exact, sums fp32).
// Operands come as 16 consecutive bytes of a row a lane: a lane's k are 8 c .. + 7 of
// every 32, the same for both operands, and its columns 8 c .. + 7 of 32, so that neither
// weights nor outputs pass through shared memory.  What the second product reads of B and y
// does not depend on t and is on its way before t is there.
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

// A request's rows within the call, and whether its numbers keep the contract
struct Rows {
  int row0, n;
  bool bad;
};
__device__ __forceinline__ Rows rows_of(const LoraParams& p, int b) {
  const int r0 = p.cu[b], r1 = p.cu[b + 1];
  return {r0, r0 < 0 || r1 <= r0 ? 0 : max(0, min(r1, p.T) - r0), r0 < 0 || r1 < r0 || r1 > p.T || p.which[b] >= p.adapters};
}

// kBlocks: blocks of 16 rows of a tile (1 or 4); kRank: the ranks that there is room for
template <int kBlocks, int kRank>
struct Smem {
  static constexpr int kRows = 16 * kBlocks;
  static constexpr int kSplit = kWarps / kBlocks;  // warps that share a block's K
  float part[kSplit][kRows][kRank];  // of the warps; [0]: of the CTA
  __nv_bfloat16 t[2][kRows][kRank];  // hi, lo of the scaled t
  long long scan[kWarps];
  int4 tile;                         // first row, rows, adapter, whether there is one
};

template <int kBlocks, int kRank>
__global__ void __launch_bounds__(kThreads, kRank > 64 ? 1 : 2) lora_kernel(const __grid_constant__ LoraParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  using S = Smem<kBlocks, kRank>;
  S& sm = *reinterpret_cast<S*>(smem_raw);
  constexpr int kNT = kRank / 8, kKB = kRank / 32;  // tiles of 8 ranks, blocks of 32
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int size = (int)cluster_size(), rank = (int)cluster_ctarank();
  const int tile = (int)(blockIdx.x / size);
  griddep_wait();
  griddep_launch_dependents();

  // ---- the cluster's tile: requests in order, their rows in tiles of kRows
  if (tid == 0) sm.tile = make_int4(0, 0, -1, 0);
  {
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;  // offsets that break the contract may claim rows twice
    for (int b = b0; b < b1; ++b) {
      const Rows r = rows_of(p, b);
      if (r.bad && blockIdx.x == 0) record_status(p.status, kStatusOffsets, 57);
      mine += (r.n + S::kRows - 1) / S::kRows;
    }
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long v = __shfl_up_sync(kFullMask, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) before += w < warp ? sm.scan[w] : 0;
    if (tile >= before && tile < before + mine) {
      for (int b = b0; b < b1; ++b) {
        const Rows r = rows_of(p, b);
        const int n = (r.n + S::kRows - 1) / S::kRows;
        const long long i = tile - before;
        if (i < n) {
          const int w = p.which[b];
          const int at = (int)i * S::kRows;
          sm.tile = make_int4(r.row0 + at, min(S::kRows, r.n - at), w >= p.adapters ? -1 : w, 1);
          break;
        }
        before += n;
      }
    }
    __syncthreads();
  }
  const int row0 = sm.tile.x, rows = sm.tile.y, id = sm.tile.z;
  if (!sm.tile.w) return;  // all CTAs of the cluster alike

  const int es = p.bf16 ? 2 : 4;
  const int chunks = (p.N + 31) / 32;  // of 32 columns, shared by the CTAs
  const int c0 = (int)((long long)chunks * rank / size), c1 = (int)((long long)chunks * (rank + 1) / size);
  if (id < 0) {
    if (p.out == p.y) return;
    const int n0 = c0 * 32, n1 = min(p.N, c1 * 32), vecs = (n1 - n0) * es / 16;
    for (int x = tid; x < rows * vecs; x += kThreads) {
      const long long row = row0 + x / vecs;
      const int at = x % vecs;
      const char* from = static_cast<const char*>(p.y) + (row * p.ldy + n0) * es;
      reinterpret_cast<uint4*>(static_cast<char*>(p.out) + (row * p.ldo + n0) * es)[at] = reinterpret_cast<const uint4*>(from)[at];
    }
    return;
  }

  // ---- t = x A^T: a warp has a block of 16 rows and a share of K
  const int block = warp % kBlocks, split = warp / kBlocks;
  const bool works = 16 * block < rows;
  const int ra = 16 * block + g, rb = ra + 8;  // this lane's rows of the tile
  {
    float acc[kNT][4] = {};
    const int blocks = (p.K + 31) / 32, parts = size * S::kSplit, part = rank * S::kSplit + split;
    const int k0 = (int)((long long)blocks * part / parts), k1 = (int)((long long)blocks * (part + 1) / parts);
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + (long long)row0 * p.ldx;
    const __nv_bfloat16* a = static_cast<const __nv_bfloat16*>(p.a) + (long long)id * p.r * p.K;
    if (works) {
#pragma unroll 2
      for (int k = k0; k < k1; ++k) {
        const int at = 32 * k + 8 * c;
        const bool in = at < p.K;
        const uint4 xa = load16(x + ra * p.ldx + at, in && ra < rows), xb = load16(x + rb * p.ldx + at, in && rb < rows);
        uint4 w[kNT];
#pragma unroll
        for (int n = 0; n < kNT; ++n) w[n] = load16(a + (long long)(8 * n + g) * p.K + at, in && 8 * n < p.r);
        const uint32_t f0[4] = {xa.x, xb.x, xa.y, xb.y}, f1[4] = {xa.z, xb.z, xa.w, xb.w};
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          if (8 * n >= p.r) break;
          mma_bf16_16x8(acc[n], f0, w[n].x, w[n].y);
          mma_bf16_16x8(acc[n], f1, w[n].z, w[n].w);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      *reinterpret_cast<float2*>(&sm.part[split][ra][8 * n + 2 * c]) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(&sm.part[split][rb][8 * n + 2 * c]) = make_float2(acc[n][2], acc[n][3]);
    }
  }
  __syncthreads();
  constexpr int kVecs = S::kRows * kRank / 4;  // of t
  for (int x = tid; x < kVecs; x += kThreads) {
    float4* at = reinterpret_cast<float4*>(&sm.part[0][0][0]) + x;
    float4 v = *at;
#pragma unroll
    for (int s = 1; s < S::kSplit; ++s) {
      const float4 w = at[s * kVecs];
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    *at = v;
  }
  __syncwarp();
  cluster_arrive();

  // ---- out = y + t B^T: a warp has a block of 16 rows and every kSplit-th chunk of columns.
  // Tile i of a chunk has the columns 8 (n / 2) + 2 i + n % 2, n = 0 .. 7.
  const __nv_bfloat16* bw = static_cast<const __nv_bfloat16*>(p.b) + (long long)id * p.N * p.r;
  uint4 w[4][kKB];
  auto load_b = [&](int chunk) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 32 * chunk + 8 * (g >> 1) + 2 * i + (g & 1);
#pragma unroll
      for (int k = 0; k < kKB; ++k)
        w[i][k] = load16(bw + (long long)n * p.r + 32 * k + 8 * c, chunk < c1 && n < p.N && 32 * k + 8 * c < p.r);
    }
  };
  int chunk = works ? c0 + split : c1;
  load_b(chunk);
  __syncwarp();
  cluster_wait();
  {
    const float scale = p.scales ? p.scales[id] : 1.0f;
    const uint32_t mine = smem_u32(&sm.part[0][0][0]);
    for (int x = tid; x < kVecs; x += kThreads) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
      for (int r = 0; r < size; ++r) {
        const float4 e = ld_cluster(mapa_shared(mine + 16 * x, r));
        v.x += e.x, v.y += e.y, v.z += e.z, v.w += e.w;
      }
      v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
      const uint32_t h0 = pack_bf16x2(v.x, v.y), h1 = pack_bf16x2(v.z, v.w);
      const uint32_t l0 = pack_bf16x2(v.x - __uint_as_float(h0 << 16), v.y - __uint_as_float(h0 & 0xffff0000u));
      const uint32_t l1 = pack_bf16x2(v.z - __uint_as_float(h1 << 16), v.w - __uint_as_float(h1 & 0xffff0000u));
      reinterpret_cast<uint2*>(&sm.t[0][0][0])[x] = make_uint2(h0, h1);
      reinterpret_cast<uint2*>(&sm.t[1][0][0])[x] = make_uint2(l0, l1);
    }
  }
  __syncthreads();
  cluster_arrive();  // this CTA has read the others' sums
  if (works) {
    uint4 ta[2][kKB], tb[2][kKB];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < kKB; ++k) {
        ta[h][k] = *reinterpret_cast<const uint4*>(&sm.t[h][ra][32 * k + 8 * c]);
        tb[h][k] = *reinterpret_cast<const uint4*>(&sm.t[h][rb][32 * k + 8 * c]);
      }
    const char* y = static_cast<const char*>(p.y);
    char* out = static_cast<char*>(p.out);
#pragma unroll 1
    for (; chunk < c1; chunk += S::kSplit) {
      const int n = 32 * chunk + 8 * c;
      const bool ina = n < p.N && ra < rows, inb = n < p.N && rb < rows;
      uint4 ya[2], yb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ya[i] = load16(y + ((row0 + ra) * p.ldy + n) * es + 16 * i, ina && (i == 0 || !p.bf16));
        yb[i] = load16(y + ((row0 + rb) * p.ldy + n) * es + 16 * i, inb && (i == 0 || !p.bf16));
      }
      float acc[4][4] = {};
#pragma unroll
      for (int h = 1; h >= 0; --h)
#pragma unroll
        for (int k = 0; k < kKB; ++k) {
          const uint32_t f0[4] = {ta[h][k].x, tb[h][k].x, ta[h][k].y, tb[h][k].y};
          const uint32_t f1[4] = {ta[h][k].z, tb[h][k].z, ta[h][k].w, tb[h][k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_bf16_16x8(acc[i], f0, w[i][k].x, w[i][k].y);
            mma_bf16_16x8(acc[i], f1, w[i][k].z, w[i][k].w);
          }
        }
      load_b(chunk + S::kSplit);
      auto put = [&](const uint4(&old)[2], long long row, int e, bool in) {
        if (!in) return;
        char* to = out + (row * p.ldo + n) * es;
        if (p.bf16) {
          const uint32_t o[4] = {old[0].x, old[0].y, old[0].z, old[0].w};
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = pack_bf16x2(__uint_as_float(o[i] << 16) + acc[i][e], __uint_as_float(o[i] & 0xffff0000u) + acc[i][e + 1]);
          *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            reinterpret_cast<float4*>(to)[i] =
                make_float4(__uint_as_float(old[i].x) + acc[2 * i][e], __uint_as_float(old[i].y) + acc[2 * i][e + 1],
                            __uint_as_float(old[i].z) + acc[2 * i + 1][e], __uint_as_float(old[i].w) + acc[2 * i + 1][e + 1]);
        }
      };
      put(ya, row0 + ra, 0, ina);
      put(yb, row0 + rb, 2, inb);
    }
  }
  __syncwarp();
  cluster_wait();  // until the others have read this CTA's sums
}

template <int kBlocks, int kRank>
cudaError_t launch(const LoraParams& p, int cluster, long long tiles, cudaStream_t stream) {
  constexpr int kSmem = (int)sizeof(Smem<kBlocks, kRank>);
  const cudaError_t e = cudaFuncSetAttribute(lora_kernel<kBlocks, kRank>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(lora_kernel<kBlocks, kRank>, (unsigned)(tiles * cluster), kThreads, kSmem, stream, cluster, p);
}
template <int kBlocks>
cudaError_t launch_rank(const LoraParams& p, int cluster, long long tiles, cudaStream_t stream) {
  if (p.r <= 32) return launch<kBlocks, 32>(p, cluster, tiles, stream);
  return p.r <= 64 ? launch<kBlocks, 64>(p, cluster, tiles, stream) : launch<kBlocks, 128>(p, cluster, tiles, stream);
}

}  // namespace

cudaError_t launch_lora(const LoraParams& p, int sms, cudaStream_t stream) {
  const bool many = p.T >= 32ll * p.B;
  // every request may end in a tile that is not full
  const int rows = many ? 64 : 16;
  const long long tiles = p.T / rows + (p.B < p.T ? p.B : p.T);
  const int cluster = 8;
  return many ? launch_rank<4>(p, cluster, tiles, stream) : launch_rank<1>(p, cluster, tiles, stream);
}

}  // namespace bsk
