// Entry points of the generation operators: argument checks of the paged
// append and attention, of their 4-bit forms, of the page selection and its
// attention, and of the token sampling.
#include <math.h>
#include <stdio.h>

#include "cb_common.cuh"
#include "cb_internal.h"

using namespace cb;

namespace {

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
size_t bytes_of(cb_dtype d) { return d == CB_BF16 ? 2 : 4; }
cb_status bad(const char *msg) { return record_error(CB_ERR_INVALID_ARG, msg); }
cb_status cuda(cudaError_t e) {
  return e == cudaSuccess ? CB_OK : record_error(CB_ERR_CUDA, cudaGetErrorString(e));
}

// A row tensor: base and leading dimension give 16-byte aligned rows of
// `cols` elements.
bool rows_ok(const void *p, int64_t ld, int64_t cols, size_t eb) {
  return p && aligned(p, 16) && ld >= cols && ld * (int64_t)eb % 16 == 0;
}

// The sequences and their table.
cb_status check_table(int n_seq, int n_pages, int page_size, const int32_t *block_table, int64_t ld_table,
                      int max_pages, const int32_t *row_offsets, const int32_t *kv_lens) {
  if (n_seq < 0 || n_seq > CB_MAX_SEQS) return bad("n_seq must be in [0, CB_MAX_SEQS]");
  if (n_pages <= 0) return bad("n_pages must be > 0");
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)))
    return record_error(CB_ERR_UNSUPPORTED, "page_size must be a power of two from 8 to 1024");
  if (max_pages < 0 || ld_table < max_pages) return bad("ld_table must be >= max_pages >= 0");
  if (n_seq > 0 && (!row_offsets || !kv_lens || (max_pages > 0 && !block_table)))
    return bad("NULL block_table, row_offsets or kv_lens");
  if (!aligned(row_offsets, 4) || !aligned(kv_lens, 4) || !aligned(block_table, 4))
    return bad("misaligned block_table, row_offsets or kv_lens");
  return CB_OK;
}

// Which pools a call reads.
enum Pools { kNone, kKeys, kBoth };

// The cache's geometry for rows of `cols` elements.
cb_status check_paged(const cb_paged_kv *kv, int64_t cols, cb_dtype dtype, Pools pools = kBoth) {
  if (!kv) return bad("kv is NULL");
  if (dtype != CB_F32 && dtype != CB_BF16) return bad("bad dtype");
  const int64_t eb = (int64_t)bytes_of(dtype);
  if (const cb_status s = check_table(kv->n_seq, kv->n_pages, kv->page_size, kv->block_table, kv->ld_table,
                                      kv->max_pages, kv->row_offsets, kv->kv_lens))
    return s;
  if ((pools != kNone && !rows_ok(kv->k_pages, kv->ld, cols, eb)) ||
      (pools == kBoth && !rows_ok(kv->v_pages, kv->ld, cols, eb)) ||
      (pools != kNone && (kv->page_stride < (kv->page_size - 1) * kv->ld + cols || kv->page_stride * eb % 16)))
    return bad("pages: NULL, misaligned, or strides below a row or a page");
  return CB_OK;
}

// The 4-bit cache's geometry.
cb_status check_paged4(const cb_paged4_kv *kv, int n_kv_heads, int head_dim, cb_dtype dtype) {
  if (!kv) return bad("kv is NULL");
  if (dtype != CB_F32 && dtype != CB_BF16) return bad("bad dtype");
  if (const cb_status s = check_table(kv->n_seq, kv->n_pages, kv->page_size, kv->block_table, kv->ld_table,
                                      kv->max_pages, kv->row_offsets, kv->kv_lens))
    return s;
  if ((head_dim != 64 && head_dim != 128) || n_kv_heads <= 0 || n_kv_heads > 4096)
    return bad("n_kv_heads must be in [1, 4096], head_dim 64 or 128");
  if (!kv->pages || !aligned(kv->pages, 16) || kv->page_stride % 16 ||
      kv->page_stride < (int64_t)cb_paged4_page_bytes(kv->page_size, n_kv_heads, head_dim))
    return bad("pages: NULL, misaligned, or a stride below a page");
  if (kv->k_exp < -64 || kv->k_exp > 64 || kv->v_exp < -64 || kv->v_exp > 64)
    return bad("k_exp and v_exp must be in [-64, 64]");
  return CB_OK;
}

cb_status status_word(int **st) {
  *st = device_status_ptr();
  return *st ? CB_OK : record_error(CB_ERR_CUDA, "cannot resolve the device status word");
}

}  // namespace

// The rows of an append, behind the geometry's checks; `cache_eb`: bytes that cache_layer_stride
// counts in.  *done: there is nothing to append.
static cb_status check_rows(const cb_paged_rows &r, int n_seq, cb_dtype dtype, int64_t cache_eb, bool *done) {
  const int64_t cols = (int64_t)r.n_kv_heads * r.head_dim;
  if (r.n_rows < 0 || r.n_layers < 0 || r.n_layers > 65535)
    return bad("n_rows < 0 or n_layers outside [0, 65535]");
  if ((*done = r.n_rows == 0 || r.n_layers == 0 || n_seq == 0)) return CB_OK;
  const size_t eb = bytes_of(dtype);
  if (!rows_ok(r.k, r.ld_k, cols, eb) || !rows_ok(r.v, r.ld_v, cols, eb))
    return bad("k / v: NULL, misaligned, or a leading dimension below a row");
  if (r.n_layers > 1 && r.cache_layer_stride == 0) return bad("layers need a cache of their own each");
  if (r.n_layers > 1 && (r.k_layer_stride * (int64_t)eb % 16 || r.v_layer_stride * (int64_t)eb % 16 ||
                         r.cache_layer_stride * cache_eb % 16))
    return bad("layer strides must be multiples of 16 bytes");
  if (r.rope_table && (!aligned(r.rope_table, 16) || r.max_positions <= 0))
    return bad("rope_table misaligned or max_positions <= 0");
  if (r.q || r.q_out) {
    if (!r.rope_table || r.n_layers != 1) return bad("q is rotated: it needs rope_table and one layer");
    if (r.n_q_heads <= 0 || r.n_q_heads > 4096) return bad("n_q_heads must be in [1, 4096]");
    const int64_t qc = (int64_t)r.n_q_heads * r.head_dim;
    if (!rows_ok(r.q, r.ld_q, qc, eb) || !rows_ok(r.q_out, r.ld_q_out, qc, eb))
      return bad("q / q_out: NULL, misaligned, or a leading dimension below a row");
  }
  return CB_OK;
}

extern "C" cb_status cb_paged_append(const cb_paged_kv *kv, const cb_paged_rows *rows, cb_dtype dtype,
                                     cb_stream stream) {
  if (!rows) return bad("rows is NULL");
  const cb_paged_rows &r = *rows;
  if (r.n_kv_heads <= 0 || r.head_dim <= 0 || r.head_dim % 16 || r.head_dim > 1024 || r.n_kv_heads > 4096)
    return bad("n_kv_heads must be in [1, 4096], head_dim a multiple of 16 up to 1024");
  const int64_t cols = (int64_t)r.n_kv_heads * r.head_dim;
  if (const cb_status s = check_paged(kv, cols, dtype)) return s;
  bool done;
  if (const cb_status s = check_rows(r, kv->n_seq, dtype, (int64_t)bytes_of(dtype), &done)) return s;
  if (done) return CB_OK;
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  return cuda(launch_paged_append(*kv, r, dtype, st, stream));
}

extern "C" size_t cb_paged4_page_bytes(int page_size, int n_kv_heads, int head_dim) {
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) || n_kv_heads <= 0 || n_kv_heads > 4096 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return (size_t)n_kv_heads * page_size * (head_dim + head_dim / 8);
}

extern "C" cb_status cb_paged4_append(const cb_paged4_kv *kv, const cb_paged_rows *rows, cb_dtype dtype,
                                      cb_stream stream) {
  if (!rows) return bad("rows is NULL");
  const cb_paged_rows &r = *rows;
  if (const cb_status s = check_paged4(kv, r.n_kv_heads, r.head_dim, dtype)) return s;
  bool done;
  if (const cb_status s = check_rows(r, kv->n_seq, dtype, 1, &done)) return s;
  if (done) return CB_OK;
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  return cuda(launch_paged4_append(*kv, r, dtype, st, stream));
}

extern "C" cb_status cb_paged4_gather(const cb_paged4_kv *kv, const cb_paged_rows_out *rows, cb_dtype dtype,
                                      cb_stream stream) {
  if (!rows) return bad("rows is NULL");
  const cb_paged_rows_out &r = *rows;
  if (const cb_status s = check_paged4(kv, r.n_kv_heads, r.head_dim, dtype)) return s;
  cb_paged_rows as = {};
  as.k = r.k; as.v = r.v; as.ld_k = r.ld_k; as.ld_v = r.ld_v;
  as.k_layer_stride = r.k_layer_stride; as.v_layer_stride = r.v_layer_stride;
  as.cache_layer_stride = r.cache_layer_stride;
  as.n_rows = r.n_rows; as.n_layers = r.n_layers; as.n_kv_heads = r.n_kv_heads; as.head_dim = r.head_dim;
  bool done;
  if (const cb_status s = check_rows(as, kv->n_seq, dtype, 1, &done)) return s;
  if (done) return CB_OK;
  if (r.n_layers > 1 && (r.k_layer_stride == 0 || r.v_layer_stride == 0)) return bad("layers need rows of their own each");
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  return cuda(launch_paged4_gather(*kv, r, dtype, st, stream));
}

static bool paged_heads_ok(int Hq, int Hkv, int hd) {
  return Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && Hq / Hkv <= 128 && Hkv <= 4096 && (hd == 64 || hd == 128);
}

// Sizes of a call that has something to do.
static bool paged_sizes_ok(int n_rows, int n_seq, int max_kv_len, int Hq, int Hkv, int hd, cb_dtype dtype) {
  return n_rows > 0 && n_seq > 0 && n_seq <= CB_MAX_SEQS && max_kv_len >= 0 && paged_heads_ok(Hq, Hkv, hd) &&
         (dtype == CB_F32 || dtype == CB_BF16);
}

extern "C" size_t cb_paged_attention_workspace_size(int n_rows, int n_seq, int max_kv_len,
                                                    int n_q_heads, int n_kv_heads, int head_dim,
                                                    cb_dtype dtype) {
  if (!paged_sizes_ok(n_rows, n_seq, max_kv_len, n_q_heads, n_kv_heads, head_dim, dtype)) return 256;
  const size_t n = paged_attention_ws_bytes(n_rows, n_seq, max_kv_len, n_q_heads, n_kv_heads, head_dim, dtype);
  return n > 256 ? n : 256;
}

extern "C" cb_status cb_debug_paged_plan(int n_rows, int n_seq, int max_kv_len, int n_q_heads, int n_kv_heads,
                                         int head_dim, cb_dtype dtype, int64_t plan[7]) {
  if (!plan || max_kv_len > CB_MAX_KV_LEN ||
      !paged_sizes_ok(n_rows, n_seq, max_kv_len, n_q_heads, n_kv_heads, head_dim, dtype))
    return bad("plan is NULL, or sizes that cb_paged_attention refuses");
  paged_attention_plan(n_rows, n_seq, max_kv_len, n_q_heads, n_kv_heads, head_dim, dtype, plan);
  return CB_OK;
}

// The rows of an attention call, behind the geometry's checks.  *done: there are none.
static cb_status check_query(const cb_paged_query &a, int n_seq, cb_dtype dtype, bool *done) {
  if (a.n_rows < 0 || a.max_kv_len < 0) return bad("n_rows < 0 or max_kv_len < 0");
  if (a.max_kv_len > CB_MAX_KV_LEN) return record_error(CB_ERR_UNSUPPORTED, "max_kv_len > CB_MAX_KV_LEN");
  // (the kernels work with scale * log2(e))
  if (!(a.scale >= 0.f) || isinf(2.f * a.scale)) return bad("scale must be >= 0 and below 2^127");
  if ((*done = a.n_rows == 0 || n_seq == 0)) return CB_OK;
  const size_t eb = bytes_of(dtype);
  const int64_t cols = (int64_t)a.n_q_heads * a.head_dim;
  if (!rows_ok(a.q, a.ld_q, cols, eb) || !rows_ok(a.out, a.ld_out, cols, eb))
    return bad("q / out: NULL, misaligned, or a leading dimension below a row");
  return CB_OK;
}

static cb_status check_ws(const void *ws, size_t bytes, size_t need, const char *what) {
  if (need == 0 || (ws && bytes >= need && aligned(ws, 16))) return CB_OK;
  char msg[96];
  snprintf(msg, sizeof msg, "%s workspace too small or misaligned (%zu < %zu)", what, bytes, need);
  return record_error(CB_ERR_WORKSPACE, msg);
}

extern "C" cb_status cb_paged_attention(const cb_paged_kv *kv, const cb_paged_query *query, cb_dtype dtype,
                                        cb_stream stream) {
  if (!query) return bad("query is NULL");
  const cb_paged_query &a = *query;
  if (!paged_heads_ok(a.n_q_heads, a.n_kv_heads, a.head_dim))
    return bad("n_q_heads must be 1 to 128 times n_kv_heads, head_dim 64 or 128");
  if (const cb_status s = check_paged(kv, (int64_t)a.n_kv_heads * a.head_dim, dtype)) return s;
  bool done;
  if (const cb_status s = check_query(a, kv->n_seq, dtype, &done)) return s;
  if (done) return CB_OK;
  if (const cb_status s = check_ws(a.ws, a.ws_bytes,
                                   paged_attention_ws_bytes(a.n_rows, kv->n_seq, a.max_kv_len, a.n_q_heads,
                                                            a.n_kv_heads, a.head_dim, dtype),
                                   "paged attention"))
    return s;
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  const cudaError_t e = launch_paged_attention(*kv, a, dtype, st, stream);
  if (e == cudaErrorInvalidConfiguration)
    return record_error(CB_ERR_UNSUPPORTED, "more query tiles than one launch takes: split the call");
  return cuda(e);
}

extern "C" size_t cb_paged4_attention_workspace_size(int n_rows, int n_seq, int max_kv_len, int n_q_heads,
                                                     int n_kv_heads, int head_dim, cb_dtype dtype) {
  if (!paged_sizes_ok(n_rows, n_seq, max_kv_len, n_q_heads, n_kv_heads, head_dim, dtype)) return 256;
  const size_t n = paged4_attention_ws_bytes(n_rows, n_seq, max_kv_len, n_q_heads, n_kv_heads, head_dim, dtype);
  return n > 256 ? n : 256;
}

extern "C" cb_status cb_debug_paged4_plan(int n_rows, int n_seq, int max_kv_len, int n_q_heads, int n_kv_heads,
                                          int head_dim, cb_dtype dtype, int64_t plan[6]) {
  if (!plan || max_kv_len > CB_MAX_KV_LEN ||
      !paged_sizes_ok(n_rows, n_seq, max_kv_len, n_q_heads, n_kv_heads, head_dim, dtype))
    return bad("plan is NULL, or sizes that cb_paged4_attention refuses");
  paged4_attention_plan(n_rows, n_seq, max_kv_len, n_q_heads, n_kv_heads, head_dim, dtype, plan);
  return CB_OK;
}

extern "C" cb_status cb_paged4_attention(const cb_paged4_kv *kv, const cb_paged_query *query, cb_dtype dtype,
                                         cb_stream stream) {
  if (!query) return bad("query is NULL");
  const cb_paged_query &a = *query;
  if (!paged_heads_ok(a.n_q_heads, a.n_kv_heads, a.head_dim))
    return bad("n_q_heads must be 1 to 128 times n_kv_heads, head_dim 64 or 128");
  if (const cb_status s = check_paged4(kv, a.n_kv_heads, a.head_dim, dtype)) return s;
  bool done;
  if (const cb_status s = check_query(a, kv->n_seq, dtype, &done)) return s;
  if (done) return CB_OK;
  if (const cb_status s = check_ws(a.ws, a.ws_bytes,
                                   paged4_attention_ws_bytes(a.n_rows, kv->n_seq, a.max_kv_len, a.n_q_heads,
                                                             a.n_kv_heads, a.head_dim, dtype),
                                   "4-bit attention"))
    return s;
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  const cudaError_t e = launch_paged4_attention(*kv, a, dtype, st, stream);
  if (e == cudaErrorInvalidConfiguration)
    return record_error(CB_ERR_UNSUPPORTED, "more query tiles than one launch takes: split the call");
  return cuda(e);
}

// The bounds' layout.
static cb_status check_bounds(const cb_page_bounds &b, size_t eb) {
  const int64_t cols = (int64_t)b.n_kv_heads * b.head_dim;
  if (b.n_rows < 0) return bad("n_rows < 0");
  if (!rows_ok(b.bounds, b.ld, cols, eb) || b.page_stride < b.ld + cols || b.page_stride * (int64_t)eb % 16)
    return bad("bounds: NULL, misaligned, or strides below a row or a page's two");
  return CB_OK;
}

extern "C" cb_status cb_paged_bounds(const cb_paged_kv *kv, const cb_page_bounds *bounds, cb_dtype dtype,
                                     cb_stream stream) {
  if (!bounds) return bad("bounds is NULL");
  const cb_page_bounds &b = *bounds;
  if (b.n_kv_heads <= 0 || b.head_dim <= 0 || b.head_dim % 16 || b.head_dim > 1024 || b.n_kv_heads > 4096)
    return bad("n_kv_heads must be in [1, 4096], head_dim a multiple of 16 up to 1024");
  if (const cb_status s = check_paged(kv, (int64_t)b.n_kv_heads * b.head_dim, dtype, kKeys)) return s;
  const size_t eb = bytes_of(dtype);
  if (b.n_layers < 0 || b.n_layers > 65535) return bad("n_layers outside [0, 65535]");
  if (const cb_status s = check_bounds(b, eb)) return s;
  if (b.n_layers > 1 && (b.bounds_layer_stride == 0 || b.cache_layer_stride == 0))
    return bad("layers need a cache and bounds of their own each");
  if (b.n_layers > 1 && (b.bounds_layer_stride * (int64_t)eb % 16 || b.cache_layer_stride * (int64_t)eb % 16))
    return bad("layer strides must be multiples of 16 bytes");
  if (b.n_rows == 0 || b.n_layers == 0 || kv->n_seq == 0) return CB_OK;
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  return cuda(launch_paged_bounds(*kv, b, dtype, st, stream));
}

extern "C" size_t cb_paged_select_workspace_size(int n_rows, int max_kv_len, int page_size, int n_kv_heads) {
  if (n_rows <= 0 || max_kv_len <= 0 || page_size <= 0 || n_kv_heads <= 0) return 256;
  const size_t n = paged_select_ws_bytes(n_rows, max_kv_len, page_size, n_kv_heads);
  return n > 256 ? n : 256;
}

extern "C" cb_status cb_paged_select(const cb_paged_kv *kv, const cb_page_bounds *bounds, const cb_page_select *select,
                                     cb_dtype dtype, cb_stream stream) {
  if (!bounds || !select) return bad("bounds or select is NULL");
  const cb_page_bounds &b = *bounds;
  const cb_page_select &a = *select;
  if (!paged_heads_ok(a.n_q_heads, b.n_kv_heads, b.head_dim))
    return bad("n_q_heads must be 1 to 128 times n_kv_heads, head_dim 64 or 128");
  if (const cb_status s = check_paged(kv, (int64_t)b.n_kv_heads * b.head_dim, dtype, kNone)) return s;
  if (a.max_kv_len < 0) return bad("max_kv_len < 0");
  if (a.max_kv_len > CB_MAX_KV_LEN) return record_error(CB_ERR_UNSUPPORTED, "max_kv_len > CB_MAX_KV_LEN");
  if (a.n_picks < 1 || a.n_picks > CB_MAX_PICKS) return bad("n_picks must be in [1, CB_MAX_PICKS]");
  if (a.n_first < 0 || a.n_last < 0 || (int64_t)a.n_first + a.n_last > a.n_picks)
    return bad("n_first and n_last must be >= 0 and together at most n_picks");
  const size_t eb = bytes_of(dtype);
  if (const cb_status s = check_bounds(b, eb)) return s;
  if (b.n_rows == 0 || kv->n_seq == 0) return CB_OK;
  if (!rows_ok(a.q, a.ld_q, (int64_t)a.n_q_heads * b.head_dim, eb))
    return bad("q: NULL, misaligned, or a leading dimension below a row");
  if (!a.picks || !aligned(a.picks, 4)) return bad("picks: NULL or misaligned");
  if (const cb_status s = check_ws(a.ws, a.ws_bytes,
                                   paged_select_ws_bytes(b.n_rows, a.max_kv_len, kv->page_size, b.n_kv_heads),
                                   "page selection"))
    return s;
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  const cudaError_t e = launch_paged_select(*kv, b, a, dtype, st, stream);
  if (e == cudaErrorInvalidConfiguration)
    return record_error(CB_ERR_UNSUPPORTED, "more pages than one launch takes: split the call");
  return cuda(e);
}

extern "C" size_t cb_paged_attention_picked_workspace_size(int n_rows, int n_picks, int page_size, int n_q_heads,
                                                           int n_kv_heads, int head_dim, cb_dtype dtype) {
  if (n_rows <= 0 || !paged_heads_ok(n_q_heads, n_kv_heads, head_dim)) return 256;
  const size_t n = paged_picked_ws_bytes(n_rows, n_picks, page_size, n_q_heads, n_kv_heads, head_dim, dtype);
  return n > 256 ? n : 256;
}

extern "C" cb_status cb_paged_attention_picked(const cb_paged_kv *kv, const cb_paged_query *query, const int32_t *picks,
                                               int n_picks, cb_dtype dtype, cb_stream stream) {
  if (!query) return bad("query is NULL");
  cb_paged_query a = *query;
  a.max_kv_len = 0;
  if (!paged_heads_ok(a.n_q_heads, a.n_kv_heads, a.head_dim))
    return bad("n_q_heads must be 1 to 128 times n_kv_heads, head_dim 64 or 128");
  if (const cb_status s = check_paged(kv, (int64_t)a.n_kv_heads * a.head_dim, dtype)) return s;
  if (n_picks < 1 || n_picks > CB_MAX_PICKS) return bad("n_picks must be in [1, CB_MAX_PICKS]");
  bool done;
  if (const cb_status s = check_query(a, kv->n_seq, dtype, &done)) return s;
  if (done) return CB_OK;
  if (!picks || !aligned(picks, 4)) return bad("picks: NULL or misaligned");
  if (const cb_status s = check_ws(a.ws, a.ws_bytes,
                                   paged_picked_ws_bytes(a.n_rows, n_picks, kv->page_size, a.n_q_heads, a.n_kv_heads,
                                                         a.head_dim, dtype),
                                   "picked attention"))
    return s;
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  return cuda(launch_paged_picked(*kv, a, picks, n_picks, dtype, st, stream));
}

extern "C" cb_status cb_debug_picked_plan(int n_rows, int n_picks, int page_size, int n_q_heads, int n_kv_heads,
                                          int head_dim, cb_dtype dtype, int64_t plan[3]) {
  if (!plan || n_rows <= 0 || n_picks < 1 || n_picks > CB_MAX_PICKS || page_size < 8 || page_size > 1024 ||
      (page_size & (page_size - 1)) || !paged_heads_ok(n_q_heads, n_kv_heads, head_dim) ||
      (dtype != CB_F32 && dtype != CB_BF16))
    return bad("plan is NULL, or sizes that cb_paged_attention_picked refuses");
  paged_picked_plan(n_rows, n_picks, page_size, n_q_heads, n_kv_heads, head_dim, dtype, plan);
  return CB_OK;
}

extern "C" cb_status cb_sample_tokens(const void *logits, int64_t ld_logits, int n_rows, int vocab,
                                      cb_dtype dtype, const float *u, const float *temperature,
                                      const int32_t *top_k, const float *top_p, const float *min_p,
                                      int32_t *tokens, cb_stream stream) {
  if (dtype != CB_F32 && dtype != CB_BF16) return bad("bad dtype");
  if (n_rows < 0 || n_rows > (1 << 20)) return bad("n_rows must be in [0, 2^20]");
  if (vocab <= 0 || ld_logits < vocab) return bad("vocab must be > 0 and ld_logits >= vocab");
  if (vocab > CB_MAX_SAMPLE_VOCAB) return record_error(CB_ERR_UNSUPPORTED, "vocab > CB_MAX_SAMPLE_VOCAB");
  if (n_rows == 0) return CB_OK;
  if (!logits || !u || !tokens) return bad("NULL logits, u or tokens");
  if (!aligned(logits, bytes_of(dtype)) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
      !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4))
    return bad("misaligned pointer");
  return cuda(launch_sample(logits, ld_logits, n_rows, vocab, dtype, u, temperature, top_k, top_p, min_p, tokens,
                            stream));
}
