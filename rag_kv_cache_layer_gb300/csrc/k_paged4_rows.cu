// Rows into and out of a paged cache of 4-bit floats.
//
// Append: row r of sequence s has position p (see paged_append_kernel) and goes to
// slot p % page_size of its page.  With a RoPE table the key is rotated as there and
// rounded to the rows' type, then quantised: the 4-bit cache holds what a cache of
// the rows' type would hold, in 16 steps.  Which code a value gets changes at
// borders, so the rotation and the quotient x / scale are rounded exactly, by pairs
// of floats (q4::turned, q4::turned_near, q4::divide_odd): a key's codes do not depend on how a
// compiler contracts its products.
// Gather: the same rows back, code * scale * 2^exp.
//
// Both are streams: rows are read once and written once, 4.5 bits a value on the
// cache's side.  Appending, a thread has 16 values (a scale's group, or the two groups that a
// rotation mixes), whose codes are one 8-byte store; eight neighbours make a head's
// line; a thread keeps its group of a row, so that its addresses are made once, and goes down
// the rows with four of them under way (32 layers of 3136 rows stored and read back 168 us;
// two under way 172 appending, 183 reading, one 179 appending).  The rows' places come as
// in paged_append_kernel: three dependent rounds of loads in a call of any size.
//
// Measured, 8 heads of 128: those 32 layers are appended in 82 us (6.4 TB/s of 527 MB) and
// gathered in 80 (6.6 TB/s), bound by memory; one rotated row each of 96 sequences and its
// way back take 7.3 us in a graph, launches and the three rounds; 8 ragged prompts of up to 1490
// rows, 32/8 heads, rotated, 56 us (floor 26), bound by the rotation's pairs, fp32 85 (50).
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"
#include "cb_paged_attn.cuh"
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
  paged::Divisor by_row;                // units of a row
  int width;                            // threads side by side on a row, a power of two (all but rotated rows)
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

// The places of the block's rows.
struct Places4 {
  int off[CB_MAX_SEQS + 1], len[CB_MAX_SEQS];
  int pos[kR4Rows], bad;
  // byte offsets of the row's slot among its page's first codes (-1: no place) and first
  // scales in the pool, and of its key and value rows, so that a unit's addresses take no
  // 64-bit products
  int64_t codes[kR4Rows], scales[kR4Rows], k[kR4Rows], v[kR4Rows];
};
template <typename T>
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
    const int slot = pos & (P.kv.page_size - 1);
    s.pos[threadIdx.x] = pos;
    s.codes[threadIdx.x] = page < 0 ? -1 : page * P.kv.page_stride + slot * (P.hd / 2);
    s.scales[threadIdx.x] = page * P.kv.page_stride + slot * (P.hd / 16);
    s.k[threadIdx.x] = (row0 + (int64_t)threadIdx.x) * P.ld_k * (int)sizeof(T);
    s.v[threadIdx.x] = (row0 + (int64_t)threadIdx.x) * P.ld_v * (int)sizeof(T);
  };
  paged_find_rows<kR4Threads, kR4Rows>(S, P.n_rows, row0, rows, s.off, &s.bad, status, place);
}

template <typename T, int HD, bool ROT>
__global__ void __launch_bounds__(kR4Threads)
paged4_append_kernel(const __grid_constant__ Rows4Params P, int *status) {
  __shared__ Places4 s_at;
  constexpr int kGroups = HD / 16;
  grid_dep_wait();
  grid_dep_launch();
  const int row0 = blockIdx.x * P.rows_per_block;
  const int rows = min(P.rows_per_block, P.n_rows - row0);
  find_places<T>(P, row0, rows, ROT, s_at, status);
  const int layer = blockIdx.y, page = P.kv.page_size, head_bytes = q4::head_bytes(page, HD);
  uint8_t *pool = reinterpret_cast<uint8_t *>(P.kv.k_pages) + layer * P.cache_stride;
  const uint8_t *kn = reinterpret_cast<const uint8_t *>(reinterpret_cast<const T *>(P.k) + layer * P.k_layer_stride);
  const uint8_t *vn = reinterpret_cast<const uint8_t *>(reinterpret_cast<const T *>(P.v) + layer * P.v_layer_stride);
  // codes and scale of group e of head h of a row
  auto put = [&](float (&x)[16], int64_t codes_of, int64_t scales_of, int h, int e, bool v, float mul) {
    if (mul != 1.f) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= mul;
    }
    uint2 codes;
    const uint32_t scale = q4::quantise<T>(x, codes);
    *reinterpret_cast<uint2 *>(pool + codes_of + (h * head_bytes + q4::codes_at(page, HD, v) + e * 8)) = codes;
    pool[scales_of + (h * head_bytes + q4::scales_at(page, HD, v) + e)] = (uint8_t)scale;
  };
  if constexpr (!ROT) {
    // a thread keeps its group and goes down the rows, kAhead of them under way
    constexpr int kAhead = sizeof(T) == 2 ? 4 : 1, kLoads = sizeof(T);
    const int per_row = P.v_units + P.k_units, step = kR4Threads / P.width;
    for (int t = threadIdx.x & (P.width - 1); t < per_row; t += P.width) {
      const bool v = t < P.v_units;
      const int u = v ? t : t - P.v_units, h = u / kGroups, e = u % kGroups;
      const uint8_t *src = (v ? vn : kn) + u * (16 * (int)sizeof(T));
      const int64_t *row_at = v ? s_at.v : s_at.k;
      const float mul = v ? P.v_mul : P.k_mul;
      for (int lr = threadIdx.x / P.width; lr < rows; lr += kAhead * step) {
        uint4 raw[kAhead][kLoads];
        int64_t at[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int l = lr + i * step;
          at[i] = l < rows ? s_at.codes[l] : -1;
          if (at[i] >= 0) {
#pragma unroll
            for (int c = 0; c < kLoads; ++c) raw[i][c] = ldg16(src + row_at[l] + c * 16);
          }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (at[i] < 0) continue;
          float x[16];
          const T *y = reinterpret_cast<const T *>(raw[i]);
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = to_f(y[k]);
          put(x, at[i], s_at.scales[lr + i * step], h, e, v, mul);
        }
      }
    }
  } else {
    const int per_row = P.k_units + P.v_units + P.q_units;
    for (int t = threadIdx.x; t < rows * per_row; t += kR4Threads) {
      const int lr = P.by_row.div(t);
      int u = t - lr * per_row;
      const int64_t at = s_at.codes[lr];
      if (at < 0) continue;
      if (u < P.v_units) {
        float x[16];
        load_group(reinterpret_cast<const T *>(vn + s_at.v[lr]) + u * 16, x);
        put(x, at, s_at.scales[lr], u / kGroups, u % kGroups, true, P.v_mul);
        continue;
      }
      u -= P.v_units;
      const bool is_q = u >= P.k_units;
      if (is_q) u -= P.k_units;
      constexpr int kPairs = kGroups / 2, kHalf = HD / 2;
      const int h = u / kPairs, e = u % kPairs;
      const int64_t r = row0 + lr;
      const T *src = (is_q ? reinterpret_cast<const T *>(P.q) + r * P.ld_q : reinterpret_cast<const T *>(kn + s_at.k[lr])) +
                     h * HD + e * 16;
      float x1[16], x2[16];
      load_group(src, x1);
      load_group(src + kHalf, x2);
      const float2 *const rope = P.rope + (int64_t)s_at.pos[lr] * kHalf + e * 16;
      const float4 *cs = reinterpret_cast<const float4 *>(rope);
      uint32_t near = 0;                        // values that turned_near is to have
      auto turn = [&](float x, float a, float y, float b, int bit) -> float {
        bool n = false;
        const float r = q4::turned<T>(x, a, y, b, n);
        if (sizeof(T) == 4 && n) near |= 1u << bit;
        return r;
      };
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float4 w = __ldg(cs + i / 2);
        const float a0 = x1[i], b0 = x2[i], a1 = x1[i + 1], b1 = x2[i + 1];
        x1[i] = turn(a0, w.x, b0, w.y, i);
        x2[i] = turn(b0, w.x, -a0, w.y, 16 + i);
        x1[i + 1] = turn(a1, w.z, b1, w.w, i + 1);
        x2[i + 1] = turn(b1, w.z, -a1, w.w, 16 + i + 1);
      }
      if constexpr (sizeof(T) == 4) {
        while (near) {                          // (one value in 2^18, of few bits more)
          const int at_bit = __ffs(near) - 1, i = at_bit & 15;
          near &= near - 1;
          const float a = src[i], b = src[kHalf + i];
          const float2 w = __ldg(rope + i);
          const float y = at_bit < 16 ? q4::turned_near(a, w.x, b, w.y) : q4::turned_near(b, w.x, -a, w.y);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            x1[k] = k == at_bit ? y : x1[k];
            x2[k] = k + 16 == at_bit ? y : x2[k];
          }
        }
      }
      if (is_q) {
        T *dst = reinterpret_cast<T *>(P.q_out) + r * P.ld_qo + h * HD + e * 16;
        store_group(dst, x1);
        store_group(dst + kHalf, x2);
      } else {
        put(x1, at, s_at.scales[lr], h, e, false, P.k_mul);
        put(x2, at, s_at.scales[lr], h, e + kPairs, false, P.k_mul);
      }
    }
  }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kR4Threads)
paged4_gather_kernel(const __grid_constant__ Rows4Params P, int *status) {
  __shared__ Places4 s_at;
  grid_dep_wait();
  grid_dep_launch();
  const int row0 = blockIdx.x * P.rows_per_block;
  const int rows = min(P.rows_per_block, P.n_rows - row0);
  find_places<T>(P, row0, rows, false, s_at, status);
  const int page = P.kv.page_size, head_bytes = q4::head_bytes(page, HD);
  const bool v = blockIdx.z != 0;         // a block reads keys or values
  const uint8_t *pool = reinterpret_cast<const uint8_t *>(P.kv.k_pages) + blockIdx.y * P.cache_stride;
  const uint8_t *codes_of = pool + q4::codes_at(page, HD, v), *scales_of = pool + q4::scales_at(page, HD, v);
  uint8_t *out = v ? reinterpret_cast<uint8_t *>(reinterpret_cast<T *>(P.v_out) + blockIdx.y * P.v_layer_stride)
                   : reinterpret_cast<uint8_t *>(reinterpret_cast<T *>(P.k_out) + blockIdx.y * P.k_layer_stride);
  const int64_t *row_at = v ? s_at.v : s_at.k;
  const float mul = v ? P.v_mul : P.k_mul;
  // a unit is 8 values (4 bytes of codes), so that neighbours write neighbouring 16 bytes; a
  // thread keeps its unit of a row and goes down the rows, kUnits of them under way
  constexpr int kUnits = 4, kHead = HD / 8;     // rows of a thread; units of a head
  const int step = kR4Threads / P.width;
  for (int u = threadIdx.x & (P.width - 1); u < P.k_units; u += P.width) {
  const int h = u / kHead, e = u % kHead;
  const uint8_t *codes_at = codes_of + (h * head_bytes + e * 4), *scales_at = scales_of + (h * head_bytes + e / 2);
  uint8_t *to_unit = out + u * (8 * (int)sizeof(T));
  for (int lr = threadIdx.x / P.width; lr < rows; lr += kUnits * step) {
    uint32_t codes[kUnits], scale[kUnits];
    uint8_t *dst[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int l = lr + k * step;
      const int64_t at = l < rows ? s_at.codes[l] : -1;
      dst[k] = nullptr;
      if (at >= 0) {
        codes[k] = __ldg(reinterpret_cast<const uint32_t *>(codes_at + at));
        scale[k] = __ldg(scales_at + s_at.scales[l]);
        dst[k] = to_unit + row_at[l];
      }
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      if (!dst[k]) continue;
      const uint32_t s = q4::both(q4::decode_scales(scale[k]), false);
      uint32_t h2[4];
      q4::decode8(codes[k], h2);
      float2 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t p = q4::mul2(h2[e], s);
        x[e] = __half22float2(*reinterpret_cast<const __half2 *>(&p));
      }
      if (mul != 1.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = make_float2(x[e].x * mul, x[e].y * mul);
      }
      if constexpr (sizeof(T) == 4) {
        float4 *to = reinterpret_cast<float4 *>(dst[k]);
        to[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        to[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
      } else {
        uint4 y;
        __nv_bfloat162 *to = reinterpret_cast<__nv_bfloat162 *>(&y);
#pragma unroll
        for (int e = 0; e < 4; ++e) to[e] = __floats2bfloat162_rn(x[e].x, x[e].y);
        *reinterpret_cast<uint4 *>(dst[k]) = y;
      }
    }
  }
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

// As many rows a block as leave every SM its eight blocks once: a block's three rounds of
// lookups are paid for a row where rows are few, and for 32 where they are many (32 layers
// of 3136 rows: 168 us; with at most 16 rows 173, with 8 196).
static dim3 plan_rows(Rows4Params &P, int n_layers) {
  P.rows_per_block = (int)max((int64_t)1, min((int64_t)kR4Rows, (int64_t)P.n_rows * n_layers / (8 * device_sm_count())));
  const int units = P.k_units + P.v_units + P.q_units;
  P.by_row = paged::Divisor(units);
  P.width = 1;
  while (P.width < units && P.width < kR4Threads) P.width *= 2;
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
  const bool rot = P.rope != nullptr;
  auto go = [&](auto *kernel) { return launch_pdl(kernel, grid, dim3(kR4Threads), 0, s, P, status); };
  cudaError_t e;
  if (dt == CB_BF16 && P.hd == 128)
    e = rot ? go(paged4_append_kernel<bf16, 128, true>) : go(paged4_append_kernel<bf16, 128, false>);
  else if (dt == CB_BF16)
    e = rot ? go(paged4_append_kernel<bf16, 64, true>) : go(paged4_append_kernel<bf16, 64, false>);
  else if (P.hd == 128)
    e = rot ? go(paged4_append_kernel<float, 128, true>) : go(paged4_append_kernel<float, 128, false>);
  else
    e = rot ? go(paged4_append_kernel<float, 64, true>) : go(paged4_append_kernel<float, 64, false>);
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
  P.k_units = r.n_kv_heads * r.head_dim / 8;
  P.k_mul = ldexpf(1.f, kv.k_exp);
  P.v_mul = ldexpf(1.f, kv.v_exp);
  dim3 grid = plan_rows(P, r.n_layers);
  grid.z = 2;                             // keys, values
  auto go = [&](auto *kernel) { return launch_pdl(kernel, grid, dim3(kR4Threads), 0, s, P, status); };
  cudaError_t e;
  if (dt == CB_BF16) e = P.hd == 128 ? go(paged4_gather_kernel<bf16, 128>) : go(paged4_gather_kernel<bf16, 64>);
  else e = P.hd == 128 ? go(paged4_gather_kernel<float, 128>) : go(paged4_gather_kernel<float, 64>);
  return e == cudaSuccess ? launched(1) : e;
}

}  // namespace cb
