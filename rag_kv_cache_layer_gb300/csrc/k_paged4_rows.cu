// Rows into and out of a paged cache of 4-bit floats.
//
// Append: row r of sequence s has position p (see paged_append_kernel) and goes to
// slot p % page_size of its page.  With a RoPE table the key is rotated as there and
// rounded to the rows' type, then quantised: the 4-bit cache holds what a cache of
// the rows' type would hold, in 16 steps.  Which code a value gets changes at
// borders, so the rotation and the quotient x / scale are rounded exactly, by pairs
// of floats (q4::turned, q4::divide_odd): a key's codes do not depend on how a
// compiler contracts its products.
// Gather: the same rows back, code * scale * 2^exp.
//
// Both are streams: rows are read once and written once, 4.5 bits a value on the
// cache's side.  A thread has 16 values (a scale's group, or the two groups that a
// rotation mixes), whose codes are one 8-byte store; eight neighbours make a head's
// line.  The rows' places come as in paged_append_kernel: three dependent rounds of
// loads in a call of any size.
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"
#include "cb_q4.cuh"

namespace cb {

struct Rows4Params {
  PagedKV kv;                           // k_pages: the pool; page_stride in bytes
  const void *k, *v, *q;
  void *k_out, *v_out, *q_out;          // gather: rows; append: q_out
  int64_t ld_k, ld_v, ld_q, ld_qo;      // elements between rows
  int64_t k_layer_stride, v_layer_stride;
  int64_t cache_stride;                 // bytes between layers of the pool
  int n_rows, max_pos, hd;
  int k_units, v_units, q_units;        // threads' shares of a row
  int rows_per_block;
  float k_mul, v_mul;                   // 2^-exp (append), 2^exp (gather)
  const float2 *rope;                   // nullptr: keys are taken as they are
};

constexpr int kR4Threads = 256;
constexpr int kR4Rows = 32;             // rows a block may own at most, a warp's lanes

template <typename T> __device__ __forceinline__ void load_group(const T *p, float (&x)[16]) {
  constexpr int VEC = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16; i += VEC) {
    const uint4 raw = ldg16(p + i);
    const T *e = reinterpret_cast<const T *>(&raw);
#pragma unroll
    for (int k = 0; k < VEC; ++k) x[i + k] = to_f(e[k]);
  }
}
template <typename T> __device__ __forceinline__ void store_group(T *p, const float (&x)[16]) {
  constexpr int VEC = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16; i += VEC) {
    float y[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) y[k] = x[i + k];
    store16<T>(p + i, y);
  }
}

// The places of the block's rows: page (-1: none) and position of each.
struct Places4 {
  int off[CB_MAX_SEQS + 1], len[CB_MAX_SEQS];
  int pos[kR4Rows], page[kR4Rows], bad;
};
__device__ __forceinline__ void find_places(const Rows4Params &P, int row0, int rows, bool rotate, Places4 &s,
                                            int *status) {
  const int S = P.kv.n_seq;
  for (int i = threadIdx.x; i <= S; i += kR4Threads) {
    s.off[i] = __ldg(P.kv.row_offsets + i);
    if (i < S) s.len[i] = __ldg(P.kv.kv_lens + i);
  }
  if (threadIdx.x == 0) s.bad = 0;
  __syncthreads();
  const int shift = __ffs(P.kv.page_size) - 1;
  auto place = [&](int x, int n, int i) {
    int pos = -1, page = -1;
    if (i >= 0 && i < n) {
      const int64_t p = (int64_t)s.len[x] - n + i;
      if (p >= 0) {
        page = paged_page(P.kv, x, (int)(p >> shift), status);
        if (rotate && p >= P.max_pos) {
          report(status, CB_ERR_DEVICE_INDEX);
          page = -1;
        }
        pos = (int)p;
      }
    }
    s.pos[threadIdx.x] = pos;
    s.page[threadIdx.x] = page;
  };
  paged_find_rows<kR4Threads, kR4Rows>(S, P.n_rows, row0, rows, s.off, &s.bad, status, place);
}

template <typename T, bool ROT>
__global__ void __launch_bounds__(kR4Threads)
paged4_append_kernel(const __grid_constant__ Rows4Params P, int *status) {
  __shared__ Places4 s_at;
  grid_dep_wait();
  grid_dep_launch();
  const int row0 = blockIdx.x * P.rows_per_block;
  const int rows = min(P.rows_per_block, P.n_rows - row0);
  find_places(P, row0, rows, ROT, s_at, status);
  const int layer = blockIdx.y, hd = P.hd, groups = hd / 16, page = P.kv.page_size;
  uint8_t *pool = reinterpret_cast<uint8_t *>(P.kv.k_pages) + layer * P.cache_stride;
  const T *kn = reinterpret_cast<const T *>(P.k) + layer * P.k_layer_stride;
  const T *vn = reinterpret_cast<const T *>(P.v) + layer * P.v_layer_stride;
  const int per_row = P.k_units + P.v_units + P.q_units;
  for (int t = threadIdx.x; t < rows * per_row; t += kR4Threads) {
    const int lr = t / per_row;
    int u = t - lr * per_row;
    if (s_at.page[lr] < 0) continue;
    const int64_t r = row0 + lr;
    const int slot = s_at.pos[lr] & (page - 1);
    uint8_t *at = pool + s_at.page[lr] * P.kv.page_stride;
    // codes and scale of group e of head h
    auto put = [&](float (&x)[16], int h, int e, bool v, float mul) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= mul;
      uint2 codes;
      const uint32_t scale = q4::quantise<T>(x, codes);
      uint8_t *head = at + (int64_t)h * q4::head_bytes(page, hd);
      *reinterpret_cast<uint2 *>(head + q4::codes_at(page, hd, v) + slot * (hd / 2) + e * 8) = codes;
      head[q4::scales_at(page, hd, v) + slot * groups + e] = (uint8_t)scale;
    };
    if (u < P.v_units) {
      float x[16];
      load_group(vn + r * P.ld_v + u * 16, x);
      put(x, u / groups, u % groups, true, P.v_mul);
      continue;
    }
    u -= P.v_units;
    if constexpr (!ROT) {
      float x[16];
      load_group(kn + r * P.ld_k + u * 16, x);
      put(x, u / groups, u % groups, false, P.k_mul);
    } else {
      const bool is_q = u >= P.k_units;
      if (is_q) u -= P.k_units;
      const int per_head = groups / 2, h = u / per_head, e = u % per_head, half = hd / 2;
      const T *src = (is_q ? reinterpret_cast<const T *>(P.q) + r * P.ld_q : kn + r * P.ld_k) + h * hd + e * 16;
      float x1[16], x2[16];
      load_group(src, x1);
      load_group(src + half, x2);
      const float4 *cs = reinterpret_cast<const float4 *>(P.rope + (int64_t)s_at.pos[lr] * half + e * 16);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float4 w = __ldg(cs + i / 2);
        const float a0 = x1[i], b0 = x2[i], a1 = x1[i + 1], b1 = x2[i + 1];
        x1[i] = q4::turned<T>(a0, w.x, b0, w.y);
        x2[i] = q4::turned<T>(b0, w.x, -a0, w.y);
        x1[i + 1] = q4::turned<T>(a1, w.z, b1, w.w);
        x2[i + 1] = q4::turned<T>(b1, w.z, -a1, w.w);
      }
      if (is_q) {
        T *dst = reinterpret_cast<T *>(P.q_out) + r * P.ld_qo + h * hd + e * 16;
        store_group(dst, x1);
        store_group(dst + half, x2);
      } else {
        put(x1, h, e, false, P.k_mul);
        put(x2, h, e + per_head, false, P.k_mul);
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kR4Threads)
paged4_gather_kernel(const __grid_constant__ Rows4Params P, int *status) {
  __shared__ Places4 s_at;
  grid_dep_wait();
  grid_dep_launch();
  const int row0 = blockIdx.x * P.rows_per_block;
  const int rows = min(P.rows_per_block, P.n_rows - row0);
  find_places(P, row0, rows, false, s_at, status);
  const int layer = blockIdx.y, hd = P.hd, groups = hd / 16, page = P.kv.page_size;
  const uint8_t *pool = reinterpret_cast<const uint8_t *>(P.kv.k_pages) + layer * P.cache_stride;
  T *ko = reinterpret_cast<T *>(P.k_out) + layer * P.k_layer_stride;
  T *vo = reinterpret_cast<T *>(P.v_out) + layer * P.v_layer_stride;
  const int per_row = 2 * P.k_units;
  for (int t = threadIdx.x; t < rows * per_row; t += kR4Threads) {
    const int lr = t / per_row;
    int u = t - lr * per_row;
    if (s_at.page[lr] < 0) continue;
    const bool v = u >= P.k_units;
    if (v) u -= P.k_units;
    const int h = u / groups, e = u % groups, slot = s_at.pos[lr] & (page - 1);
    const uint8_t *head = pool + s_at.page[lr] * P.kv.page_stride + (int64_t)h * q4::head_bytes(page, hd);
    const uint2 codes = __ldg(reinterpret_cast<const uint2 *>(head + q4::codes_at(page, hd, v) + slot * (hd / 2) + e * 8));
    const uint32_t s = q4::both(q4::decode_scales(__ldg(head + q4::scales_at(page, hd, v) + slot * groups + e)), false);
    const float mul = v ? P.v_mul : P.k_mul;
    float x[16];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t h2[4];
      q4::decode8(w ? codes.y : codes.x, h2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t p = q4::mul2(h2[i], s);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p));
        x[w * 8 + 2 * i] = f.x * mul;
        x[w * 8 + 2 * i + 1] = f.y * mul;
      }
    }
    const int64_t r = row0 + lr;
    store_group((v ? vo + r * P.ld_v : ko + r * P.ld_k) + u * 16, x);
  }
}

PagedKV paged4_plain_kv(const cb_paged4_kv &kv) {
  PagedKV p = {};
  p.k_pages = p.v_pages = kv.pages;
  p.page_stride = kv.page_stride;
  p.n_pages = kv.n_pages;
  p.page_size = kv.page_size;
  p.block_table = kv.block_table;
  p.ld_table = kv.ld_table;
  p.max_pages = kv.max_pages;
  p.row_offsets = kv.row_offsets;
  p.kv_lens = kv.kv_lens;
  p.n_seq = kv.n_seq;
  return p;
}

static dim3 plan_rows(Rows4Params &P, int n_layers) {
  const int per_row = P.k_units + P.v_units + P.q_units;
  P.rows_per_block = max(1, min(kR4Rows, 4 * kR4Threads / per_row));
  return dim3((P.n_rows + P.rows_per_block - 1) / P.rows_per_block, n_layers);
}

cudaError_t launch_paged4_append(const cb_paged4_kv &kv, const cb_paged_rows &r, cb_dtype dt, int *status,
                                 cudaStream_t s) {
  Rows4Params P = {};
  P.kv = paged4_plain_kv(kv);
  P.k = r.k; P.v = r.v; P.q = r.q; P.q_out = r.q_out;
  P.ld_k = r.ld_k; P.ld_v = r.ld_v; P.ld_q = r.ld_q; P.ld_qo = r.ld_q_out;
  P.k_layer_stride = r.k_layer_stride;
  P.v_layer_stride = r.v_layer_stride;
  P.cache_stride = r.cache_layer_stride;
  P.n_rows = r.n_rows;
  P.max_pos = r.max_positions;
  P.hd = r.head_dim;
  P.rope = reinterpret_cast<const float2 *>(r.rope_table);
  P.v_units = r.n_kv_heads * r.head_dim / 16;
  P.k_units = P.rope ? P.v_units / 2 : P.v_units;
  P.q_units = r.q ? r.n_q_heads * r.head_dim / 32 : 0;
  P.k_mul = ldexpf(1.f, -kv.k_exp);
  P.v_mul = ldexpf(1.f, -kv.v_exp);
  const dim3 grid = plan_rows(P, r.n_layers);
  cudaError_t e;
  if (dt == CB_BF16)
    e = P.rope ? launch_pdl(paged4_append_kernel<bf16, true>, grid, dim3(kR4Threads), 0, s, P, status)
               : launch_pdl(paged4_append_kernel<bf16, false>, grid, dim3(kR4Threads), 0, s, P, status);
  else
    e = P.rope ? launch_pdl(paged4_append_kernel<float, true>, grid, dim3(kR4Threads), 0, s, P, status)
               : launch_pdl(paged4_append_kernel<float, false>, grid, dim3(kR4Threads), 0, s, P, status);
  return e == cudaSuccess ? launched(1) : e;
}

cudaError_t launch_paged4_gather(const cb_paged4_kv &kv, const cb_paged_rows_out &r, cb_dtype dt, int *status,
                                 cudaStream_t s) {
  Rows4Params P = {};
  P.kv = paged4_plain_kv(kv);
  P.k_out = r.k; P.v_out = r.v;
  P.ld_k = r.ld_k; P.ld_v = r.ld_v;
  P.k_layer_stride = r.k_layer_stride;
  P.v_layer_stride = r.v_layer_stride;
  P.cache_stride = r.cache_layer_stride;
  P.n_rows = r.n_rows;
  P.hd = r.head_dim;
  P.k_units = P.v_units = r.n_kv_heads * r.head_dim / 16;
  P.k_mul = ldexpf(1.f, kv.k_exp);
  P.v_mul = ldexpf(1.f, kv.v_exp);
  const dim3 grid = plan_rows(P, r.n_layers);
  const cudaError_t e = dt == CB_BF16
      ? launch_pdl(paged4_gather_kernel<bf16>, grid, dim3(kR4Threads), 0, s, P, status)
      : launch_pdl(paged4_gather_kernel<float>, grid, dim3(kR4Threads), 0, s, P, status);
  return e == cudaSuccess ? launched(1) : e;
}

}  // namespace cb
