// Entry points of the generation operators: argument checks of the paged
// append, the paged attention and the token sampling.
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

// The cache's geometry for rows of `cols` elements.
cb_status check_paged(const cb_paged_kv *kv, int64_t cols, cb_dtype dtype) {
  if (!kv) return bad("kv is NULL");
  if (dtype != CB_F32 && dtype != CB_BF16) return bad("bad dtype");
  const int64_t eb = (int64_t)bytes_of(dtype);
  if (kv->n_seq < 0 || kv->n_seq > CB_MAX_SEQS) return bad("n_seq must be in [0, CB_MAX_SEQS]");
  if (kv->n_pages <= 0) return bad("n_pages must be > 0");
  if (kv->page_size < 8 || kv->page_size > 1024 || (kv->page_size & (kv->page_size - 1)))
    return record_error(CB_ERR_UNSUPPORTED, "page_size must be a power of two from 8 to 1024");
  if (!rows_ok(kv->k_pages, kv->ld, cols, eb) || !rows_ok(kv->v_pages, kv->ld, cols, eb) ||
      kv->page_stride < (kv->page_size - 1) * kv->ld + cols || kv->page_stride * eb % 16)
    return bad("pages: NULL, misaligned, or strides below a row or a page");
  if (kv->max_pages < 0 || kv->ld_table < kv->max_pages) return bad("ld_table must be >= max_pages >= 0");
  if (kv->n_seq > 0 && (!kv->row_offsets || !kv->kv_lens || (kv->max_pages > 0 && !kv->block_table)))
    return bad("NULL block_table, row_offsets or kv_lens");
  if (!aligned(kv->row_offsets, 4) || !aligned(kv->kv_lens, 4) || !aligned(kv->block_table, 4))
    return bad("misaligned block_table, row_offsets or kv_lens");
  return CB_OK;
}

cb_status status_word(int **st) {
  *st = device_status_ptr();
  return *st ? CB_OK : record_error(CB_ERR_CUDA, "cannot resolve the device status word");
}

}  // namespace

extern "C" cb_status cb_paged_append(const cb_paged_kv *kv, const cb_paged_rows *rows, cb_dtype dtype,
                                     cb_stream stream) {
  if (!rows) return bad("rows is NULL");
  const cb_paged_rows &r = *rows;
  if (r.n_kv_heads <= 0 || r.head_dim <= 0 || r.head_dim % 16 || r.head_dim > 1024 || r.n_kv_heads > 4096)
    return bad("n_kv_heads must be in [1, 4096], head_dim a multiple of 16 up to 1024");
  const int64_t cols = (int64_t)r.n_kv_heads * r.head_dim;
  if (const cb_status s = check_paged(kv, cols, dtype)) return s;
  if (r.n_rows < 0 || r.n_layers < 0 || r.n_layers > 65535)
    return bad("n_rows < 0 or n_layers outside [0, 65535]");
  if (r.n_rows == 0 || r.n_layers == 0 || kv->n_seq == 0) return CB_OK;
  const size_t eb = bytes_of(dtype);
  if (!rows_ok(r.k, r.ld_k, cols, eb) || !rows_ok(r.v, r.ld_v, cols, eb))
    return bad("k / v: NULL, misaligned, or a leading dimension below a row");
  if (r.n_layers > 1 && r.cache_layer_stride == 0) return bad("layers need a cache of their own each");
  if (r.n_layers > 1 && (r.k_layer_stride * (int64_t)eb % 16 || r.v_layer_stride * (int64_t)eb % 16 ||
                         r.cache_layer_stride * (int64_t)eb % 16))
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
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  return cuda(launch_paged_append(*kv, r, dtype, st, stream));
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

extern "C" cb_status cb_paged_attention(const cb_paged_kv *kv, const cb_paged_query *query, cb_dtype dtype,
                                        cb_stream stream) {
  if (!query) return bad("query is NULL");
  const cb_paged_query &a = *query;
  if (!paged_heads_ok(a.n_q_heads, a.n_kv_heads, a.head_dim))
    return bad("n_q_heads must be 1 to 128 times n_kv_heads, head_dim 64 or 128");
  if (const cb_status s = check_paged(kv, (int64_t)a.n_kv_heads * a.head_dim, dtype)) return s;
  if (a.n_rows < 0 || a.max_kv_len < 0) return bad("n_rows < 0 or max_kv_len < 0");
  if (a.max_kv_len > CB_MAX_KV_LEN) return record_error(CB_ERR_UNSUPPORTED, "max_kv_len > CB_MAX_KV_LEN");
  // (the kernels work with scale * log2(e))
  if (!(a.scale >= 0.f) || isinf(2.f * a.scale)) return bad("scale must be >= 0 and below 2^127");
  if (a.n_rows == 0 || kv->n_seq == 0) return CB_OK;
  const size_t eb = bytes_of(dtype);
  const int64_t cols = (int64_t)a.n_q_heads * a.head_dim;
  if (!rows_ok(a.q, a.ld_q, cols, eb) || !rows_ok(a.out, a.ld_out, cols, eb))
    return bad("q / out: NULL, misaligned, or a leading dimension below a row");
  const size_t need = paged_attention_ws_bytes(a.n_rows, kv->n_seq, a.max_kv_len, a.n_q_heads, a.n_kv_heads,
                                               a.head_dim, dtype);
  if (need > 0 && (!a.ws || a.ws_bytes < need || !aligned(a.ws, 16))) {
    char msg[96];
    snprintf(msg, sizeof msg, "paged attention workspace too small or misaligned (%zu < %zu)", a.ws_bytes, need);
    return record_error(CB_ERR_WORKSPACE, msg);
  }
  int *st;
  if (const cb_status s = status_word(&st)) return s;
  const cudaError_t e = launch_paged_attention(*kv, a, dtype, st, stream);
  if (e == cudaErrorInvalidConfiguration)
    return record_error(CB_ERR_UNSUPPORTED, "more query tiles than one launch takes: split the call");
  return cuda(e);
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
