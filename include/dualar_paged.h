/* dualar_paged.h -- the paged key/value cache as operators on the caller's own
 * device buffers (libdualar.so).
 *
 * The decoder of dualar.h owns its cache and its page tables.  These calls give
 * the same cache to a caller that runs its own step, one layer at a time:
 *
 *   dualar_kv_plan          once per step: pages for the new tokens, page tables,
 *                           slot map and row positions, from request lengths
 *   dualar_qk_norm_rope     per layer: QK-norm, rotation, append to the cache
 *   dualar_paged_attention  per layer: the step's rows against the cache, causal,
 *                           with an optional sliding window and first tokens
 *                           ("sinks") that stay visible
 *   dualar_kv_read          cached vectors as values
 *
 * A step's rows are the new tokens of all its requests, request by request:
 * request s has rows row_start[s] .. row_start[s+1] - 1, which are its last
 * row_start[s+1] - row_start[s] positions.  Any mix of single tokens and prompts
 * goes in one call.
 *
 * Conventions (as in dualar.h):
 *   - Return value: DUALAR_OK or a negative DUALAR_ERR_* code; nothing aborts.
 *     dualar_paged_error returns the calling thread's last message.
 *   - All pointers are device memory unless said otherwise.  Work is queued on
 *     cuda_stream (a cudaStream_t, NULL = legacy default stream) and is
 *     asynchronous; the stream's device must be current.  The calls allocate
 *     nothing, keep nothing, never synchronise, and can be captured into a graph.
 *   - Values that only the device knows (lengths, pages, slots) are checked
 *     there: an access outside its buffer is skipped and, where dev_error is not
 *     NULL, a bit is OR-ed into *dev_error (DUALAR_PAGED_ERR_*).  The caller
 *     zeroes and reads that word.
 *   - Calls are thread-safe; two calls whose GPU work overlaps need their own
 *     workspaces and outputs.  So do two calls that two threads make at once on
 *     one stream: dualar_paged_attention queues two kernels, and the other
 *     call's may come between them.
 *
 * Pages follow the decoder's layout.  [P2] of dualar.h ("The slow AR is
 * Qwen3-4B", "Streaming: whose numbers") gives QK-norm and the bf16 rotation
 * tables; the window, the sinks and the 4-bit cache are this library's own.
 */
#ifndef DUALAR_PAGED_H
#define DUALAR_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "dualar.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { DUALAR_PAGE_TOKENS = 64 };

/* Types of activations (queries, outputs, qkv rows). */
enum { DUALAR_F32 = 0, DUALAR_BF16 = 1 };

/* Bits of *dev_error. */
enum {
  DUALAR_PAGED_ERR_WAIT = 1 << 0,  /* a wait inside a kernel ran out (see dualar_paged_attention) */
  DUALAR_PAGED_ERR_INDEX = 1 << 2, /* a row, slot, position or length out of range */
  DUALAR_PAGED_ERR_PAGE = 1 << 3   /* a page-table entry out of range */
};

/* One layer of a paged cache.  A page holds, for this layer,
 *   bits 16: bf16 [2][n_kv_head][64][head_dim], keys then values (the decoder's
 *            layout: a pool of several layers is [page][layer][...]);
 *   bits 4:  [2][n_kv_head] blocks of 32 head_dim + 128 bytes: the codes of 64
 *            tokens, head_dim / 2 bytes each (element 2i in the low nibble of
 *            byte i, 2i + 1 in the high one, stored as q + 8), then the 64
 *            bf16 scales (>= 0).  An element stands for q * scale of its token.
 * A token's slot is page * 64 + (position % 64). */
typedef struct dualar_kv {
  void* data;          /* page 0 of this layer; 16-byte aligned */
  int64_t page_stride; /* bytes from a page to the next; a multiple of 16 */
  int32_t n_pages;     /* 1 .. 2^25 - 1 */
  int32_t n_kv_head;
  int32_t head_dim;    /* 64 or 128 */
  int32_t bits;        /* 16 or 4 */
} dualar_kv;

/* Bytes of one layer of one page; -1 for a shape outside the limits above. */
int64_t dualar_kv_page_bytes(int32_t n_kv_head, int32_t head_dim, int32_t bits);

/* Plans a step on the GPU.  Request s holds kv_len[s] tokens and gets n_new[s]
 * (>= 0) more; its pages 0 .. ceil(kv_len / 64) - 1 are in its row of the table.
 * The pages it lacks are taken from those with page_refs == 0, lowest first, in
 * request order (the rule of dualar_prefill), their page_refs set to 1 and their
 * numbers written into the table.  Outputs:
 *   row_start [n_seq + 1]  first row of each request, then the number of rows
 *   pos       [max_rows]   position of each row in its request
 *   slot      [max_rows]   its cache slot
 *   new_len   [n_seq]      kv_len + n_new
 *   status    [3]          0, rows, pages taken
 * Rows behind the last get pos 0 and slot -1, which the other calls skip, so a
 * step can be captured at a fixed max_rows.
 * A step that cannot be planned changes neither table nor page_refs and plans
 * no row (row_start all 0, every slot -1, new_len = kv_len): status[0] is then 3
 * (a negative length; rows and pages are 0) or else the highest that holds of 1
 * (more pages needed than are free), 2 (a request needs more than table_width
 * pages), 4 (more than max_rows rows) and 5 (the table's entry of a partly filled
 * page that gets tokens is outside [0, n_pages)), followed by the rows and pages
 * that the step would need (at most 2^31 - 1).
 * A page is released by lowering its page_refs (a shared prefix counts its
 * holders).  n_seq <= 8192, max_rows <= 2^24, table_width <= 2^20.  Outputs may
 * not overlap inputs, but new_len may be kv_len. */
int dualar_kv_plan(const int32_t* kv_len, const int32_t* n_new, int32_t n_seq, int32_t* page_refs,
                   int32_t n_pages, int32_t* table, int32_t table_width, int32_t max_rows,
                   int32_t* row_start, int32_t* pos, int32_t* slot, int32_t* new_len, int32_t* status,
                   void* cuda_stream);

/* QK-norm, rotation and append of `rows` rows (<= 2^24).
 *   qkv: act [rows][ld], of each row n_head query heads, then n_kv_head key and
 *        n_kv_head value heads (kv->head_dim each); 16-byte aligned rows
 *   q_norm, k_norm: bf16 [head_dim] RMSNorm gains over each head, or both NULL
 *   cos, sin: bf16 [n_pos][head_dim / 2]; pairs (2i, 2i + 1) rotate by the angle
 *        of row pos[r]; 4-byte aligned
 *   q_out: act [rows][ldq]: normed and rotated queries; may be the q part of qkv
 * Key and value of row r go to slot[r] (negative: nowhere); two rows of a call
 * have different slots.  bits 16: rounded to bf16.  bits 4: the
 * rule of dualar_quantize_w4a16 on each head's vector x: scale s = bf16(max|x| / 7),
 * code rint(x / s) clamped to [-8, 7] (0 when s = 0), both of exact arithmetic
 * (decided in 64 bits next to a border), so they depend on no order of sums.
 * A vector with an infinity or a NaN gets a NaN scale and reads back as NaN.
 * A row whose pos is outside [0, n_pos) is skipped (nothing written). */
int dualar_qk_norm_rope(const void* qkv, int32_t act, int64_t ld, int32_t rows, int32_t n_head,
                        const dualar_kv* kv, const int32_t* pos, const int32_t* slot,
                        const void* q_norm, const void* k_norm, float eps, const void* cos,
                        const void* sin, int32_t n_pos, void* q_out, int64_t ldq,
                        uint32_t* dev_error, void* cuda_stream);

/* Keys and values of n slots as fp32 [n][n_kv_head][head_dim]; zeros where the
 * slot is negative.  k, v: 16-byte aligned. */
int dualar_kv_read(const dualar_kv* kv, const int32_t* slot, int32_t n, float* k, float* v,
                   uint32_t* dev_error, void* cuda_stream);

/* Workspace bytes of a dualar_paged_attention call with these sizes; -1 for
 * sizes outside its limits. */
int64_t dualar_paged_attention_workspace(int32_t act, int32_t rows, int32_t n_head, const dualar_kv* kv,
                                         int32_t n_seq);

/* Attention of a step's rows over the cache.  Row r of request s (row_start) has
 * position p = kv_len[s] - (row_start[s+1] - r), with kv_len the tokens in the
 * cache, the new ones among them.  It sees the positions j <= p with
 * j > p - window or j < sinks (window 0: all j <= p) and gets
 *   out = sum_j softmax_j(scale * q . k_j) v_j
 * per query head (head h reads key/value head h / (n_head / n_kv_head)); zeros
 * where it sees nothing (p < 0, or only pages out of range).
 *   q, out: act [rows][ld], n_head heads of head_dim; 16-byte aligned rows
 *   table:  [n_seq][table_width] page numbers; entries that no row sees are not
 *           read as pages (a page that left the window may be reused)
 * Rows before row_start[0] and behind row_start[n_seq] are left as they were.
 * What cached positions that no row of the call sees hold (infinities, NaN) has no
 * effect; a non-finite value that one row of a request sees may reach its other
 * rows of the call.
 * Sums and softmax statistics are fp32.  fp32 activations: queries and weights
 * keep 22 significant bits at least.  bf16: queries are taken as they are, weights
 * keep 16 bits at least.
 * The result depends on the arguments and the device alone, not on timing; but
 * for waits inside the kernels, which end after 2 s (a device taken from the call
 * meanwhile): every row of the call is then NaN and *dev_error has
 * DUALAR_PAGED_ERR_WAIT.
 * One of two kernels serves the whole call, chosen by rows / n_seq: few rows per
 * request, or many (padding counts).  Where a long prompt comes beside many single
 * tokens, two calls can take a fraction of the time: one for the requests of single
 * tokens, which come first (their rows and n_seq), one for the others (row_start,
 * kv_len and table from their first request on, the same q, out and rows).
 * n_head / n_kv_head <= 32, rows <= 2^24, table_width <= 2^20, n_seq <= 8192;
 * workspace: dualar_paged_attention_workspace bytes, 16-byte aligned, any
 * contents. */
int dualar_paged_attention(const void* q, int32_t act, int64_t ldq, int32_t rows, int32_t n_head,
                           const dualar_kv* kv, const int32_t* table, int32_t table_width,
                           const int32_t* row_start, const int32_t* kv_len, int32_t n_seq,
                           int32_t window, int32_t sinks, float scale, void* out, int64_t ldo,
                           void* workspace, int64_t workspace_bytes, uint32_t* dev_error,
                           void* cuda_stream);

/* Copies the calling thread's last error message of these calls (NUL-terminated,
 * truncated to len). */
int dualar_paged_error(char* buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* DUALAR_PAGED_H */
