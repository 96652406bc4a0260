// Entry points of the paged key/value operators (include/dualar_paged.h):
// argument checks, then one launch each.
#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "dualar_paged.h"
#include "paged.h"

namespace dualar {
namespace {

thread_local char g_paged_error[256];

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_paged_error, sizeof(g_paged_error), fmt, ap);
  va_end(ap);
  return code;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The cache view, or an error.
int check_kv(const dualar_kv* kv, KvView* v) {
  if (!kv) return fail(DUALAR_ERR_INVALID_ARG, "kv is NULL");
  const int64_t pb = dualar_kv_page_bytes(kv->n_kv_head, kv->head_dim, kv->bits);
  if (pb < 0)
    return fail(DUALAR_ERR_INVALID_ARG, "kv: %d heads of %d in %d bits (head_dim 64 or 128, bits 16 or 4)",
                kv->n_kv_head, kv->head_dim, kv->bits);
  if (kv->n_pages < 1 || kv->n_pages >= (1 << 25))
    return fail(DUALAR_ERR_INVALID_ARG, "kv: %d pages outside [1, 2^25)", kv->n_pages);
  if (!kv->data || !aligned(kv->data, 16)) return fail(DUALAR_ERR_INVALID_ARG, "kv: data is NULL or not 16-byte aligned");
  if (kv->page_stride < pb || kv->page_stride % 16)
    return fail(DUALAR_ERR_INVALID_ARG, "kv: page_stride %lld below %lld or not a multiple of 16",
                static_cast<long long>(kv->page_stride), static_cast<long long>(pb));
  *v = KvView{static_cast<unsigned char*>(kv->data), kv->page_stride, kv->n_pages, kv->n_kv_head, kv->head_dim, kv->bits};
  return DUALAR_OK;
}

// Row stride (elements) and base of an activation matrix.
int check_rows(const char* what, const void* p, int act, int64_t ld, int64_t width) {
  const int64_t es = act == DUALAR_F32 ? 4 : 2;
  if (!p || !aligned(p, 16) || ld < width || (ld * es) % 16)
    return fail(DUALAR_ERR_INVALID_ARG, "%s: NULL, rows not 16-byte aligned, or row stride %lld below %lld", what,
                static_cast<long long>(ld), static_cast<long long>(width));
  return DUALAR_OK;
}

int done(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return DUALAR_OK;
  return fail(DUALAR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Multiprocessors of the current device (asked once per device).
int sm_count(int* n) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64 && (*n = known[dev].load(std::memory_order_relaxed)) > 0) return DUALAR_OK;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*n, std::memory_order_relaxed);
  return done("device query", e);
}

}  // namespace
}  // namespace dualar

using namespace dualar;

extern "C" {

int dualar_paged_error(char* buf, size_t len) {
  if (!buf || len == 0) return DUALAR_ERR_INVALID_ARG;
  snprintf(buf, len, "%s", g_paged_error);
  return DUALAR_OK;
}

int64_t dualar_kv_page_bytes(int32_t n_kv_head, int32_t head_dim, int32_t bits) {
  if (n_kv_head < 1 || n_kv_head > 1024 || (head_dim != 64 && head_dim != 128) || (bits != 16 && bits != 4)) return -1;
  return int64_t(2) * n_kv_head * kv_block_bytes(head_dim, bits);
}

int dualar_kv_plan(const int32_t* kv_len, const int32_t* n_new, int32_t n_seq, int32_t* page_refs, int32_t n_pages,
                   int32_t* table, int32_t table_width, int32_t max_rows, int32_t* row_start, int32_t* pos,
                   int32_t* slot, int32_t* new_len, int32_t* status, void* cuda_stream) {
  if (n_seq < 0 || n_seq > kMaxPlanSeqs)
    return fail(DUALAR_ERR_INVALID_ARG, "kv_plan: %d requests outside [0, %d]", n_seq, kMaxPlanSeqs);
  if (n_pages < 0 || n_pages >= (1 << 25) || table_width < 0 || table_width > kMaxTableWidth)
    return fail(DUALAR_ERR_INVALID_ARG, "kv_plan: %d pages, table width %d", n_pages, table_width);
  if (max_rows < 0 || max_rows > (1 << 24))
    return fail(DUALAR_ERR_INVALID_ARG, "kv_plan: max_rows %d outside [0, 2^24]", max_rows);
  if (!row_start || !status || (n_seq > 0 && (!kv_len || !n_new || !new_len)) || (n_pages > 0 && !page_refs) ||
      (n_seq > 0 && table_width > 0 && !table) || (max_rows > 0 && (!pos || !slot)))
    return fail(DUALAR_ERR_INVALID_ARG, "kv_plan: a pointer is NULL");
  const PlanArgs a{kv_len, n_new, n_seq, page_refs, n_pages, table, table_width, max_rows, row_start, pos, slot,
                   new_len, status};
  return done("kv_plan", launch_kv_plan(a, static_cast<cudaStream_t>(cuda_stream)));
}

int dualar_qk_norm_rope(const void* qkv, int32_t act, int64_t ld, int32_t rows, int32_t n_head, const dualar_kv* kv,
                        const int32_t* pos, const int32_t* slot, const void* q_norm, const void* k_norm, float eps,
                        const void* cos, const void* sin, int32_t n_pos, void* q_out, int64_t ldq,
                        uint32_t* dev_error, void* cuda_stream) {
  NormRopeArgs a{};
  if (const int rc = check_kv(kv, &a.kv)) return rc;
  if (act != DUALAR_F32 && act != DUALAR_BF16) return fail(DUALAR_ERR_INVALID_ARG, "qk_norm_rope: type %d", act);
  if (rows < 0 || rows > (1 << 24) || n_head < 1 || n_head > 4096 || n_pos < 1)
    return fail(DUALAR_ERR_INVALID_ARG, "qk_norm_rope: %d rows, %d heads, %d positions", rows, n_head, n_pos);
  if (rows == 0) return DUALAR_OK;
  const int64_t hd = kv->head_dim;
  if (const int rc = check_rows("qk_norm_rope: qkv", qkv, act, ld, (n_head + 2 * int64_t(kv->n_kv_head)) * hd)) return rc;
  if (const int rc = check_rows("qk_norm_rope: q_out", q_out, act, ldq, n_head * hd)) return rc;
  if (!pos || !slot || !cos || !sin || !aligned(cos, 4) || !aligned(sin, 4))
    return fail(DUALAR_ERR_INVALID_ARG, "qk_norm_rope: pos, slot, cos or sin is NULL or unaligned");
  if (!q_norm != !k_norm || !aligned(q_norm, 4) || !aligned(k_norm, 4))
    return fail(DUALAR_ERR_INVALID_ARG, "qk_norm_rope: q_norm and k_norm go together, 4-byte aligned");
  if (q_norm && !(eps > 0.f)) return fail(DUALAR_ERR_INVALID_ARG, "qk_norm_rope: eps must be positive");
  a.qkv = qkv;
  a.ld = ld;
  a.rows = rows;
  a.n_head = n_head;
  a.pos = pos;
  a.slot = slot;
  a.q_norm = static_cast<const uint16_t*>(q_norm);
  a.k_norm = static_cast<const uint16_t*>(k_norm);
  a.eps = eps;
  a.cos = static_cast<const uint16_t*>(cos);
  a.sin = static_cast<const uint16_t*>(sin);
  a.n_pos = n_pos;
  a.q_out = q_out;
  a.ldq = ldq;
  a.err = dev_error;
  return done("qk_norm_rope", launch_qk_norm_rope(a, act == DUALAR_BF16, static_cast<cudaStream_t>(cuda_stream)));
}

int dualar_kv_read(const dualar_kv* kv, const int32_t* slot, int32_t n, float* k, float* v, uint32_t* dev_error,
                   void* cuda_stream) {
  KvView view;
  if (const int rc = check_kv(kv, &view)) return rc;
  if (n < 0) return fail(DUALAR_ERR_INVALID_ARG, "kv_read: %d slots", n);
  if (n == 0) return DUALAR_OK;
  if (!slot || !k || !v || !aligned(k, 16) || !aligned(v, 16))
    return fail(DUALAR_ERR_INVALID_ARG, "kv_read: slot, k or v is NULL or unaligned");
  return done("kv_read", launch_kv_read(view, slot, n, k, v, dev_error, static_cast<cudaStream_t>(cuda_stream)));
}

int64_t dualar_paged_attention_workspace(int32_t act, int32_t rows, int32_t n_head, const dualar_kv* kv,
                                         int32_t n_seq) {
  if (!kv || dualar_kv_page_bytes(kv->n_kv_head, kv->head_dim, kv->bits) < 0 || rows < 0 || rows > (1 << 24) || n_seq < 0 || n_head < 1 ||
      n_seq > kMaxPlanSeqs || (act != DUALAR_F32 && act != DUALAR_BF16) || n_head % kv->n_kv_head ||
      n_head / kv->n_kv_head > 32)
    return -1;
  return paged_attention_workspace(act == DUALAR_BF16, kv->bits, rows, n_head, kv->n_kv_head, kv->head_dim, n_seq);
}

int dualar_paged_attention(const void* q, int32_t act, int64_t ldq, int32_t rows, int32_t n_head, const dualar_kv* kv,
                           const int32_t* table, int32_t table_width, const int32_t* row_start, const int32_t* kv_len,
                           int32_t n_seq, int32_t window, int32_t sinks, float scale, void* out, int64_t ldo,
                           void* workspace, int64_t workspace_bytes, uint32_t* dev_error, void* cuda_stream) {
  AttnArgs a{};
  if (const int rc = check_kv(kv, &a.kv)) return rc;
  if (act != DUALAR_F32 && act != DUALAR_BF16) return fail(DUALAR_ERR_INVALID_ARG, "paged_attention: type %d", act);
  if (rows < 0 || rows > (1 << 24) || n_seq < 0 || n_seq > kMaxPlanSeqs)
    return fail(DUALAR_ERR_INVALID_ARG, "paged_attention: %d rows (at most 2^24), %d requests (at most %d)", rows, n_seq,
                kMaxPlanSeqs);
  if (n_head < 1 || n_head % kv->n_kv_head || n_head / kv->n_kv_head > 32)
    return fail(DUALAR_ERR_INVALID_ARG, "paged_attention: %d query heads on %d key/value heads", n_head, kv->n_kv_head);
  if (table_width < 0 || table_width > kMaxTableWidth)
    return fail(DUALAR_ERR_INVALID_ARG, "paged_attention: table width %d outside [0, 2^20]", table_width);
  if (window < 0 || sinks < 0 || !(scale > 0.f) || scale > 3e38f)
    return fail(DUALAR_ERR_INVALID_ARG, "paged_attention: window %d, sinks %d, scale %g", window, sinks, scale);
  if (rows == 0 || n_seq == 0) return DUALAR_OK;
  const int64_t width = int64_t(n_head) * kv->head_dim;
  if (const int rc = check_rows("paged_attention: q", q, act, ldq, width)) return rc;
  if (const int rc = check_rows("paged_attention: out", out, act, ldo, width)) return rc;
  if ((table_width > 0 && !table) || !row_start || !kv_len)
    return fail(DUALAR_ERR_INVALID_ARG, "paged_attention: table, row_start or kv_len is NULL");
  const int64_t need = dualar_paged_attention_workspace(act, rows, n_head, kv, n_seq);
  if (workspace_bytes < need || (need > 0 && (!workspace || !aligned(workspace, 16))))
    return fail(DUALAR_ERR_INVALID_ARG, "paged_attention: workspace of %lld bytes, %lld needed (16-byte aligned)",
                static_cast<long long>(workspace_bytes), static_cast<long long>(need));
  a.q = q;
  a.ldq = ldq;
  a.rows = rows;
  a.n_head = n_head;
  a.table = table;
  a.width = table_width;
  a.row_start = row_start;
  a.kv_len = kv_len;
  a.n_seq = n_seq;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  a.out = out;
  a.ldo = ldo;
  a.ws = static_cast<float*>(workspace);
  a.err = dev_error;
  int n_sm = 0;
  if (const int rc = sm_count(&n_sm)) return rc;
  return done("paged_attention",
              launch_paged_attention(a, act == DUALAR_BF16, n_sm, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
