// decode.h -- the decode-step operators' part of the interface between the C-ABI
// layer (api.cu) and their kernels.
#pragma once
#include "kernels.h"

namespace bsk {

// launch_kernel for a kernel that needs more dynamic shared memory than 48 KB: the
// limit belongs to the function in one context, so it is set with each launch.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel_smem(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                               Args&&... args) {
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, grid, block, smem, stream, 1, std::forward<Args>(args)...);
}

// Paged 8-bit cache (kv_cache.cu)
constexpr int kKvPlanMaxB = 8192;
struct KvPlanParams {
  const int* seq_lens;    // [B] tokens cached so far
  const int* new_lens;    // [B] tokens of this step
  int B;
  int* table;             // [B, ld_table] page ids
  long long ld_table;
  int max_pages;          // usable entries of a table row
  const int* free_pages;  // [capacity]
  const int* n_free;      // device scalar
  int capacity;
  int page_shift;         // log2(page_size)
  int T;                  // entries of slots
  int* cu_new;            // [B + 1]
  int* kv_lens;           // [B]
  int* slots;             // [T]
  int* n_free_out;
  int* status;
};
cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t stream);
struct KvReleaseParams {
  const int* lens;        // [B]
  const int* done;        // [B]: nonzero = give the pages back
  int B;
  int* table;
  long long ld_table;
  int max_pages;
  int* free_pages;
  int* n_free;
  int capacity;
  int page_shift;
  int* status;
};
cudaError_t launch_kv_release(const KvReleaseParams& p, cudaStream_t stream);
cudaError_t launch_kv_positions(const int* seq_lens, const int* cu_new, int B, int T, int* positions, cudaStream_t stream);
struct KvAppendParams {
  const void* x[2];       // keys, values
  long long tok_stride[2], head_stride[2];  // elements
  uint8_t* codes[2];      // [pages, Hkv, page, D]
  float* scales[2];       // [pages, Hkv]
  const int* slots;       // [T]
  int T, Hkv, D;
  int num_pages, page_shift;
  int x_bf16;
  int* status;
};
cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream);

// New keys, values and queries with the rotation on the way (kv_append_rotary.cu)
struct KvRotaryParams {
  const void* q;          // [T, Hq, D]
  long long q_tok_stride, q_head_stride;  // elements
  void* q_out;            // bf16 [T, Hq, D]
  long long qo_tok_stride, qo_head_stride;
  const void* x[2];       // keys, values
  long long tok_stride[2], head_stride[2];
  const int* slots;       // [T]
  const int* positions;   // [T]
  const float* angles;    // [max_positions, rot]: cosines, then sines
  int max_positions, rot, interleaved;
  uint8_t* codes[2];      // [pages, Hkv, page, D] e4m3, or [.., D / 2] E2M1 pairs
  void* scales[2];        // fp32 [pages, Hkv], or e4m3 [pages, Hkv, page, D / 16]
  int fp4;
  int T, Hq, Hkv, D;
  int num_pages, page_shift;
  int x_bf16;             // type of q, k and v
  int heads, rows_each;   // the launch's choice: heads that a warp goes through, rows whose short runs it takes
  int* status;
};
cudaError_t launch_kv_append_rotary(const KvRotaryParams& p, cudaStream_t stream);
struct KvGatherParams {
  const uint8_t* codes[2];
  const void* scales[2];
  int fp4;
  const int* slots;       // [T]
  void* out[2];           // bf16 [T, Hkv, D]
  long long out_tok_stride[2], out_head_stride[2];
  int T, Hkv, D;
  int num_pages, page_shift;
  int* status;
};
cudaError_t launch_kv_gather(const KvGatherParams& p, cudaStream_t stream);

// Attention over the paged cache (kv_attention.cu)
// Most rows (new tokens x heads of a group) per KV head of a request for the
// few-rows kernel; kv_attention_rows.cu takes the others.  A call whose rows do not
// fill the GPU with units of 8 lets the few-rows kernel read a request's cache
// several times, from L2 (us, few / many rows: one request, 8 heads of 8, 8000
// tokens, 32 rows per KV head 22 / 43, 64 rows 27 / 45, 128 rows 40 / 59; 8 requests, 4
// heads, 2000 tokens, 32 rows 20 / 26, 64 rows 28 / 27, and where requests of both kinds
// meet, one kernel instead of two, 16 / 38); a larger one does not (64 requests, 8
// heads, 3000 tokens, 16 rows 131 / 166, 32 rows 247 / 158, 64 rows 477 / 163).  Over 4 bits: one
// request 32 rows 20 / 39, 128 rows 38 / 57; 8 requests, 64 rows 28 / 24; 64 requests, 16 rows 98 / 144,
// 32 rows 182 / 139 (D = 64: 16 rows 63 / 133, 32 rows 113 / 127).
constexpr int few_rows(long long T, int Hq) { return T * Hq <= 2048 ? 128 : 16; }
// Over 4 bits the few-rows kernel also takes whole calls of few rows times tokens: a request's rows
// (of all heads) times its cached tokens, 128 (a tile) at least, summed over the requests, are at
// most 2^23 over one or two KV heads, which leave the many-rows kernel short of units, 15 2^18 over
// more; else as above (us, few / many rows, one
// request: 512 tokens x 8 heads over 512 cached 20 / 31, over 1024 27 / 34, over 2048 40 / 38; 128 x 32
// heads, 8 of KV, over 512 20 / 19, over 2048 40 / 27; three requests, 75 x 3 heads, 1 of KV, over 2700
// 18 / 45, 50 x 24 heads, 8 of KV, over 1000 18 / 25; 8 requests of 16 x 32 heads over 1000 26 / 23).
// Both kernels form that sum from the lengths, so they agree, and the width of the table changes
// no result; a call whose T rows pass it with 128 tokens each is not asked.  Where the table has
// room for more, the many-rows kernel starts only to find nothing, which takes 6 us (one request, 32
// heads, 8 of KV, 64 tokens, nothing cached: 7 and 13, by the many-rows kernel 31; 128 tokens, 600 cached 20
// and 26, 29; four requests of 64 tokens, 400 cached 26 and 32, 29).
constexpr int whole_most(int Hkv) { return Hkv <= 2 ? 1 << 23 : 15 << 18; }
struct KvAttentionParams {
  const void* q;          // bf16 [T, Hq, D]
  long long q_tok_stride, q_head_stride;
  void* out;              // bf16 [T, Hq, D]
  long long out_tok_stride, out_head_stride;
  float* lse;             // [T, Hq] or null
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const void* k_scales;   // fp32 [pages, Hkv]; 4-bit cache: e4m3 [pages, Hkv, page, D / 16]
  const void* v_scales;
  const int* table;       // [B, ld_table]
  long long ld_table;
  int max_pages;
  const int* cu_q;        // [B + 1]
  const int* kv_lens;     // [B]
  int B, T, Hq, Hkv, D;
  int num_pages, page_shift;
  int fp4;                // the cache holds 4 bits
  float scale_log2;       // softmax scale * log2(e)
  int most_rows;          // bound of the rows per KV head of a request (at most 2^30)
  int few_rows;           // few_rows(T, Hq)
  int whole_most;         // 4 bits: the few-rows kernel takes all of a call of no more rows times tokens; 0: do not ask
  float* work;            // pieces of (request, head) pairs cut between CTAs
  int* counters;          // arrivals of those pieces (zero between calls)
  int* status;
  unsigned long long wait_ns;
};
struct KvAttentionLaunch {
  KvAttentionParams p;
  CUtensorMap tm_k, tm_v; // codes as rows of 128 bytes, box kv_attention_box tokens
  int few_grid, rows_grid;
  bool few_only;          // no request is the many-rows kernel's
};
int kv_attention_few_grid(int sms);
size_t kv_attention_piece_bytes(int D);  // per CTA of the few-rows grid
int kv_attention_box(int page_size, bool fp4);
// requests with more than few_rows rows per KV head (kv_attention_rows.cu)
int kv_attention_rows_grid(int sms);
size_t kv_attention_rows_piece_bytes(int D);
cudaError_t launch_kv_attention_rows(const KvAttentionLaunch& L, cudaStream_t stream);
cudaError_t launch_kv_attention(const KvAttentionLaunch& L, cudaStream_t stream);

// Few bf16 rows times FP4 weights (matvec_fp4.cu)
struct Fp4MatvecParams {
  const void* x;          // bf16 [M, ldx]
  long long ldx;
  const uint8_t* codes;   // [N, K/2]
  const uint8_t* sf;      // MMA layout for [N, K]
  int M, N, K;
  float alpha;
  const float* tensor_scale;  // device fp32 or null
  const void* bias;       // bf16 [N] or null
  void* out;
  int out_bf16;
  long long ldo;
};
cudaError_t launch_fp4_matvec(const Fp4MatvecParams& p, int sms, cudaStream_t stream);

// Low-rank adapters of many requests (lora.cu)
struct LoraParams {
  const void* x;          // bf16 [T, ldx]
  long long ldx;
  const void* a;          // bf16 [adapters, r, K]
  const void* b;          // bf16 [adapters, N, r]
  const float* scales;    // [adapters] or null
  const int* cu;          // [B + 1]
  const int* which;       // [B]
  const void* y;          // [T, ldy]
  long long ldy;
  void* out;              // [T, ldo]
  long long ldo;
  int bf16;               // type of y and out
  int T, B, K, N, r, adapters;
  int least, most;        // rows of the requests that a launch takes; the launch's choice
  int* status;
};
cudaError_t launch_lora(const LoraParams& p, int sms, cudaStream_t stream);

}  // namespace bsk
