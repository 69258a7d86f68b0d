// Appends new keys and values to a paged cache and rotates keys and queries
// to their positions on the way.
//
// Row r of sequence s (its i-th of n new rows) has position
// p = kv_lens[s] - n + i; its key and value go to slot p % page_size of page
// block_table[s][p / page_size].  With a RoPE table the key (and the query)
// is rotated by p * theta_e in rotate-half pairs (e, e + hd/2), in fp32:
//   y_e = x_e cos - x_{e+hd/2} sin,  y_{e+hd/2} = x_{e+hd/2} cos + x_e sin,
// rounded once to the cache's type; values are copied.
//
// A pure stream: every byte of K, V (and Q) is read once and written once.
// A block owns a few rows of one layer.  It reads all offsets and lengths in
// one coalesced round, finds its rows' sequences in shared memory, reads their
// page entries, and then streams the rows: three dependent rounds of loads in
// a call of any size, not a search in global memory per row.
//
// Measured: 32 layers of 3136 rows of 1024 (822 MB read and written) 130 us, 6.3 TB/s;
// one row with its query 3.0 us, 128 rows 4.3, where the three rounds count.
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"

namespace cb {

struct AppendParams {
  PagedKV kv;
  const void *k, *v, *q;
  void *q_out;
  int64_t ld_k, ld_v, ld_q, ld_qo;      // elements between rows
  int64_t new_stride_k, new_stride_v;   // elements between layers of k / v
  int64_t cache_stride;                 // elements between layers of the pools
  int n_rows, max_pos, half;            // half: head_dim / 2
  int k_units, v_units, q_units;        // 16-byte units (pair units when rotated) per row
  int rows_per_block;
  const float2 *rope;                   // nullptr: keys are copied
};

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 32;         // rows a block may own at most, a warp's lanes

template <typename T, bool ROT>
__global__ void __launch_bounds__(kAppendThreads)
paged_append_kernel(const __grid_constant__ AppendParams P, int *status) {
  constexpr int VEC = 16 / sizeof(T);
  __shared__ int s_off[CB_MAX_SEQS + 1];
  __shared__ int s_len[CB_MAX_SEQS];
  __shared__ int s_pos[kAppendRows];
  __shared__ int64_t s_dst[kAppendRows];     // element offset of the row's slot, -1: not stored
  __shared__ int s_bad;                      // some sequence's offsets do not ascend inside the rows
  grid_dep_wait();
  grid_dep_launch();
  const int S = P.kv.n_seq;
  const int row0 = blockIdx.x * P.rows_per_block;
  const int rows = min(P.rows_per_block, P.n_rows - row0);
  for (int i = threadIdx.x; i <= S; i += kAppendThreads) {
    s_off[i] = __ldg(P.kv.row_offsets + i);
    if (i < S) s_len[i] = __ldg(P.kv.kv_lens + i);
  }
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  // The row is row i of sequence x, which has n rows; none where i is not in [0, n).
  const int shift = __ffs(P.kv.page_size) - 1;
  auto place = [&](int x, int n, int i) {
    int pos = -1;
    int64_t dst = -1;
    if (i >= 0 && i < n) {
      const int64_t p = (int64_t)s_len[x] - n + i;
      if (p >= 0) {
        const int page = paged_page(P.kv, x, (int)(p >> shift), status);
        if (ROT && p >= P.max_pos) {
          report(status, CB_ERR_DEVICE_INDEX);
        } else if (page >= 0) {
          pos = (int)p;
          dst = (int64_t)page * P.kv.page_stride + (p & (P.kv.page_size - 1)) * P.kv.ld;
        }
      }
    }
    s_pos[threadIdx.x] = pos;
    s_dst[threadIdx.x] = dst;
  };
  paged_find_rows<kAppendThreads, kAppendRows>(S, P.n_rows, row0, rows, s_off, &s_bad, status, place);
  const int layer = blockIdx.y;
  const T *kn = reinterpret_cast<const T *>(P.k) + layer * P.new_stride_k;
  const T *vn = reinterpret_cast<const T *>(P.v) + layer * P.new_stride_v;
  T *kp = reinterpret_cast<T *>(P.kv.k_pages) + layer * P.cache_stride;
  T *vp = reinterpret_cast<T *>(P.kv.v_pages) + layer * P.cache_stride;
  const int per_row = P.k_units + P.v_units + P.q_units;
  const int total = rows * per_row;
  for (int t = threadIdx.x; t < total; t += kAppendThreads) {
    const int lr = t / per_row;
    int u = t - lr * per_row;
    const int64_t dst = s_dst[lr];
    if (dst < 0) continue;
    const int64_t r = row0 + lr;
    if (u < P.v_units) {
      stg16(vp + dst + u * VEC, ldg16(vn + r * P.ld_v + u * VEC));
      continue;
    }
    u -= P.v_units;
    const bool is_q = u >= P.k_units;
    if (is_q) u -= P.k_units;
    const T *src = is_q ? reinterpret_cast<const T *>(P.q) + r * P.ld_q : kn + r * P.ld_k;
    T *out = is_q ? reinterpret_cast<T *>(P.q_out) + r * P.ld_qo : kp + dst;
    if (!ROT) {
      stg16(out + u * VEC, ldg16(src + u * VEC));
      continue;
    }
    const int per_head = P.half / VEC;
    const int e0 = (u % per_head) * VEC;
    const int c1 = (u / per_head) * 2 * P.half + e0, c2 = c1 + P.half;
    float x1[VEC], x2[VEC], o1[VEC], o2[VEC];
    load16<T>(src + c1, x1);
    load16<T>(src + c2, x2);
    const float4 *cs = reinterpret_cast<const float4 *>(P.rope + (int64_t)s_pos[lr] * P.half + e0);
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      const float4 w = __ldg(cs + i / 2);
      o1[i] = x1[i] * w.x - x2[i] * w.y;
      o2[i] = x2[i] * w.x + x1[i] * w.y;
      o1[i + 1] = x1[i + 1] * w.z - x2[i + 1] * w.w;
      o2[i + 1] = x2[i + 1] * w.z + x1[i + 1] * w.w;
    }
    store16<T>(out + c1, o1);
    store16<T>(out + c2, o2);
  }
}

cudaError_t launch_paged_append(const PagedKV &kv, const cb_paged_rows &r, cb_dtype dt, int *status,
                                cudaStream_t s) {
  AppendParams P;
  P.kv = kv;
  P.k = r.k; P.v = r.v; P.q = r.q; P.q_out = r.q_out;
  P.ld_k = r.ld_k; P.ld_v = r.ld_v; P.ld_q = r.ld_q; P.ld_qo = r.ld_q_out;
  P.new_stride_k = r.k_layer_stride; P.new_stride_v = r.v_layer_stride;
  P.cache_stride = r.cache_layer_stride;
  P.n_rows = r.n_rows;
  P.max_pos = r.max_positions;
  P.half = r.head_dim / 2;
  P.rope = reinterpret_cast<const float2 *>(r.rope_table);
  const float2 *rope = P.rope;
  const int vec = dt == CB_BF16 ? 8 : 4;
  P.v_units = r.n_kv_heads * r.head_dim / vec;
  P.k_units = rope ? P.v_units / 2 : P.v_units;
  P.q_units = r.q ? r.n_q_heads * r.head_dim / vec / 2 : 0;
  const int per_row = P.v_units + P.k_units + P.q_units;
  P.rows_per_block = max(1, min(kAppendRows, 4 * kAppendThreads / per_row));
  const dim3 grid((r.n_rows + P.rows_per_block - 1) / P.rows_per_block, r.n_layers);
  cudaError_t e;
  if (dt == CB_BF16)
    e = rope ? launch_pdl(paged_append_kernel<bf16, true>, grid, dim3(kAppendThreads), 0, s, P, status)
             : launch_pdl(paged_append_kernel<bf16, false>, grid, dim3(kAppendThreads), 0, s, P, status);
  else
    e = rope ? launch_pdl(paged_append_kernel<float, true>, grid, dim3(kAppendThreads), 0, s, P, status)
             : launch_pdl(paged_append_kernel<float, false>, grid, dim3(kAppendThreads), 0, s, P, status);
  if (e != cudaSuccess) return e;
  return launched(1);
}

}  // namespace cb
