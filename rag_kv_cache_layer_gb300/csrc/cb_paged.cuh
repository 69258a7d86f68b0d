// Paged-cache addressing shared by the append and the paged attention
// kernels: the cache's geometry, and the search that maps a block to its
// query tile from the row offsets on the device.
#pragma once

#include "cb_common.cuh"
#include "cb_internal.h"

namespace cb {

// Sequences of one block's tile search: with NT threads per block (a template
// parameter below), each looks at CB_MAX_SEQS / NT consecutive sequences at most.
static_assert(CB_MAX_SEQS == 1024, "the searches below cover 1024 sequences");

// Physical page of logical page `j` of sequence s; -1 when the table names a
// page outside the pool (recorded) or j lies outside the table's row.
__device__ __forceinline__ int paged_page(const PagedKV &kv, int s, int j, int *status) {
  if (j < 0 || j >= kv.max_pages) {
    report(status, CB_ERR_DEVICE_INDEX);
    return -1;
  }
  const int p = __ldg(kv.block_table + (int64_t)s * kv.ld_table + j);
  if (p < 0 || p >= kv.n_pages) {
    report(status, CB_ERR_DEVICE_INDEX);
    return -1;
  }
  return p;
}

// One tile of query rows: sequence s, its rows [row0, row0 + n) of q / out,
// its cached length kv (new rows included) and the tile's index in it.
// Row l of a sequence's kv head is query l / G, head l % G of the group
// (l < n * G), so tiles carry no unused rows whatever G is.
struct PagedTile {
  int s, t, row0, n, kv;
};

// Rows of sequence i, 0 (and an error recorded) for offsets that do not
// ascend inside [0, n_rows].
__device__ __forceinline__ int paged_rows(const PagedKV &kv, int i, int n_rows, int *status) {
  const int a = __ldg(kv.row_offsets + i), b = __ldg(kv.row_offsets + i + 1);
  if (a < 0 || b < a || b > n_rows) {
    report(status, CB_ERR_DEVICE_INDEX);
    return 0;
  }
  return b - a;
}

// Finds the tile-th tile of R rows over the sequences with more than rows_lo
// rows (queries x G); a sequence's last tile, which sees the most keys, comes
// first.  Every thread of the
// block calls it (NT threads, NT a multiple of 32); on return `out` (shared
// memory) holds the tile, out->s = -1 when there are fewer tiles or the
// sequence's length does not fit the table or max_kv (recorded; its rows are
// left unwritten).  One round of loads and one block scan whatever n_seq is.
template <int NT>
__device__ __forceinline__ void paged_find_tile(const PagedKV &kv, int n_rows, int G, int R,
                                                int max_kv, int tile, PagedTile *out,
                                                int *warp_sums, int *status, int rows_lo = 0) {
  constexpr int kPer = (CB_MAX_SEQS + NT - 1) / NT;
  const int per = (kv.n_seq + NT - 1) / NT;
  const int i0 = threadIdx.x * per;
  int cnt[kPer], len[kPer], row0[kPer], rows_of[kPer];
  int sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    cnt[k] = 0;
    if (k < per && i0 + k < kv.n_seq) {
      len[k] = __ldg(kv.kv_lens + i0 + k);
      row0[k] = __ldg(kv.row_offsets + i0 + k);
      rows_of[k] = paged_rows(kv, i0 + k, n_rows, status);
      const int64_t rows = (int64_t)rows_of[k] * G;
      cnt[k] = rows > rows_lo ? (int)((rows + R - 1) / R) : 0;
    }
    sum += cnt[k];
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[w] = incl;
  if (threadIdx.x == 0) out->s = -1;
  __syncthreads();
  int first = incl - sum;
  for (int x = 0; x < w; ++x) first += warp_sums[x];
  if (tile >= first && tile < first + sum) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (tile >= first && tile < first + cnt[k]) {
        if (len[k] < 0 || len[k] > max_kv || len[k] > (int64_t)kv.max_pages * kv.page_size)
          report(status, CB_ERR_DEVICE_INDEX);
        else
          *out = PagedTile{i0 + k, cnt[k] - 1 - (tile - first), row0[k], rows_of[k], len[k]};
      }
      first += cnt[k];
    }
  }
  __syncthreads();
}

// Calls place(x, n, i) in the first `rows` threads of the block, once or, where the
// offsets are wrong, twice: thread t's row row0 + t is the i-th of the n rows of
// sequence x (of none where i is not in [0, n)).  s_off: the call's offsets in
// shared memory, *s_bad 0; every thread of the block calls it after a barrier, and
// another one ends it.
template <int NT, int ROWS, typename F>
__device__ __forceinline__ void paged_find_rows(int S, int n_rows, int row0, int rows, const int *s_off, int *s_bad,
                                                int *status, const F &place) {
  // The first warp looks up the rows, the others look at every sequence: one
  // whose offsets do not ascend may hold no row that a search ends in.
  const int r = row0 + threadIdx.x;
  if ((int)threadIdx.x < rows) {
    // the last sequence that starts at or before r
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_off[mid] <= r) lo = mid; else hi = mid - 1;
    }
    place(lo, s_off[lo + 1] - s_off[lo], r - s_off[lo]);
  }
  for (int x = (int)threadIdx.x - ROWS; x < S; x += NT - ROWS)
    if (x >= 0 && (s_off[x] < 0 || s_off[x + 1] < s_off[x] || s_off[x + 1] > n_rows)) *s_bad = 1;
  __syncthreads();
  if (*s_bad) {
    // Once more: of the sequences whose offsets ascend from all before them,
    // the one that holds r; rows of the others belong to none.
    if (threadIdx.x == 0) report(status, CB_ERR_DEVICE_INDEX);
    if ((int)threadIdx.x < rows) {
      int seq = 0, n = 0, i = 0;
      for (int x = 0, top = 0; x < S; ++x) {
        const int a = s_off[x], b = s_off[x + 1];
        if (a >= top && a <= r && r < b && b <= n_rows) {
          seq = x;
          n = b - a;
          i = r - a;
        }
        top = max(top, max(a, b));
      }
      place(seq, n, i);
    }
    __syncthreads();
  }
}

}  // namespace cb
