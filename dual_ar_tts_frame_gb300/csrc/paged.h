// Paged key/value operators (include/dualar_paged.h): arguments shared by the
// entry points (paged_api.cu) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace dualar {

constexpr int kPageTokens = 64;
constexpr int kMaxPlanSeqs = 8192;      // requests of a call
constexpr int kMaxTableWidth = 1 << 20;  // pages per request
constexpr int kAttnSms = 152;            // multiprocessors that the attention kernels use at most (GB300's; workspaces fit them)

struct KvView {
  unsigned char* data;
  int64_t page_stride;   // bytes
  int32_t n_pages, n_kv_head, head_dim, bits;
};

// Bytes of one (page, key or value, head) block.
__host__ __device__ inline int kv_block_bytes(int head_dim, int bits) {
  return bits == 16 ? kPageTokens * head_dim * 2 : kPageTokens * head_dim / 2 + kPageTokens * 2;
}

struct PlanArgs {
  const int32_t *kv_len, *n_new;
  int32_t n_seq;
  int32_t* page_refs;
  int32_t n_pages;
  int32_t* table;
  int32_t width, max_rows;
  int32_t *row_start, *pos, *slot, *new_len, *status;
};
cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t st);

struct NormRopeArgs {
  const void* qkv;
  int64_t ld;            // elements
  int32_t rows, n_head;
  KvView kv;
  const int32_t *pos, *slot;
  const uint16_t *q_norm, *k_norm;
  float eps;
  const uint16_t *cos, *sin;
  int32_t n_pos;
  void* q_out;
  int64_t ldq;
  uint32_t* err;
};
cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, bool bf16, cudaStream_t st);

cudaError_t launch_kv_read(const KvView& kv, const int32_t* slot, int n, float* k, float* v, uint32_t* err,
                           cudaStream_t st);

struct AttnArgs {
  const void* q;
  int64_t ldq;           // elements
  int32_t rows, n_head;
  KvView kv;
  const int32_t* table;
  int32_t width;
  const int32_t* table_row;   // row of the table of each request; null: its own number
  const int32_t* row_start;
  const int32_t* kv_len;
  int32_t n_seq, window, sinks;
  float scale;
  void* out;
  int64_t ldo;
  float* ws;
  uint32_t* err;
  int32_t no_waiting;    // tests: the waits inside the kernel for many rows run out at once
};
// The workspace begins with a header per CTA: of its unfinished last unit, for the
// join, and (kHeadLost) whether a wait of the CTA ran out.  Then the pieces.
constexpr int kHeadInts = 8, kHeadLost = 6;
// Few rows per request (paged_decode.cu), then the join of units that fell on
// several CTAs.
cudaError_t launch_attn_decode(const AttnArgs& a, bool bf16, int n_sm, cudaStream_t st);
int64_t decode_workspace_floats(int bits, int head_dim);
// The join: of the pieces that grid CTAs left in the workspace, for units of
// `tile` rows (8; 256 for bf16 and 128 for fp32 activations).
cudaError_t launch_attn_join(const AttnArgs& a, bool bf16, int tile, int grid, cudaStream_t st);
// Many rows per request (paged_prompt.cu), then the join.
cudaError_t launch_attn_prompt(const AttnArgs& a, bool bf16, int n_sm, cudaStream_t st);
int64_t prompt_workspace_floats(bool f32, int head_dim);

// The decoder's rows as a step: n_seq + 1 row starts and, per request, its length
// with its new positions and its row of the page table (requests: every row its
// own, or one for all rows); per row its position and cache slot (-1: inactive).
struct DevPtrs;
struct StepBuffers {
  int32_t *row_start, *kv_len, *table_row;   // [kMaxRows + 1], [kMaxRows], [kMaxRows]
  int32_t *pos, *slot;                       // [kMaxRows]
};
cudaError_t launch_decoder_step(const DevPtrs& d, int nrows, bool one_sequence, const StepBuffers& b, cudaStream_t st);

cudaError_t launch_paged_attention(const AttnArgs& a, bool bf16, int n_sm, cudaStream_t st);
int64_t paged_attention_workspace(bool bf16, int bits, int rows, int n_head, int n_kv_head, int head_dim, int n_seq);

}  // namespace dualar
