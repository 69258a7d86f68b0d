// Bounds of the keys of every page, and the selection of pages by them.
//
// Bounds.  min and max over a page's slots, dimension by dimension, from the keys
// themselves: a page that received rows is read once more (it is in the L2 cache
// after the append), and nothing has to be cleared or carried from call to call.
// The first of a sequence's new rows in a page brings it up to date.
//
// Selection.  A page's score for q, the largest dot product that its bounds allow,
//   max over the group's heads h of sum_d max(q_d min_d, q_d max_d)
//     = max_h (q_h^+ . max + q_h^- . min),   q^+ = max(q, 0), q^- = min(q, 0),
// is computed in fp32 first, off by at most
//   eps = 2^-15 max_h |q_h|_1 max |bounds|
// (256 products of one sum, each rounded, summed in fp32: 2 * 256 * 2^-24).  With t
// the fp32 score in the place of the last one that fits, pages above t + 2 eps are in,
// pages below t - 2 eps are not, and the few between are scored again in fp64, where
// the products are exact, and ranked (ties: the lower page): the picks are those of
// the exact scores.
//
// A generated token reads two bounds for a page in place of its keys: the scores are
// a stream over the bounds.
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"

namespace cb {
namespace pages {

// Sequence of row r and the row's position in it: every thread of a block of NT calls
// it with the same r.  s = -1: outside every range, or the sequence's offsets are wrong
// (recorded).  One round of loads whatever n_seq is.
struct RowPlace { int s, pos, kv; };
template <int NT>
__device__ __forceinline__ RowPlace find_row(const PagedKV &kv, int n_rows, int r, RowPlace *shared, int *status) {
  __syncthreads();
  if (threadIdx.x == 0) shared->s = 0x7fffffff;
  __syncthreads();
  for (int i = threadIdx.x; i < kv.n_seq; i += NT) {
    const int a = __ldg(kv.row_offsets + i), b = __ldg(kv.row_offsets + i + 1);
    if (a < 0 || b < a || b > n_rows) report(status, CB_ERR_DEVICE_INDEX);
    else if (a <= r && r < b) atomicMin(&shared->s, i);
  }
  __syncthreads();
  RowPlace p = {shared->s, -1, 0};
  if (p.s == 0x7fffffff) return {-1, -1, 0};
  const int b = __ldg(kv.row_offsets + p.s + 1);
  p.kv = __ldg(kv.kv_lens + p.s);
  const int64_t pos = (int64_t)p.kv - b + r;
  p.pos = pos < 0 ? -1 : (int)pos;
  return p;
}

// ---------------------------------------------------------------- bounds --
constexpr int kBThreads = 256, kBCols = 32, kBRows = 32;

struct BoundsParams {
  PagedKV kv;
  void *bounds;
  int64_t page_stride, ld, layer_stride, cache_stride;
  int n_rows, rows_per_block, cols;     // cols: 16-byte columns of a row
};

template <typename T>
__global__ void __launch_bounds__(kBThreads)
paged_bounds_kernel(const __grid_constant__ BoundsParams P, int *status) {
  constexpr int VEC = 16 / sizeof(T), kSlots = kBThreads / kBCols;
  __shared__ int s_off[CB_MAX_SEQS + 1];
  __shared__ int s_page[kBRows], s_n[kBRows], s_bad;   // page (-1: none) and covered slots of an owning row
  __shared__ float s_lo[kSlots][kBCols][VEC + 1], s_hi[kSlots][kBCols][VEC + 1];
  grid_dep_wait();
  grid_dep_launch();
  const int S = P.kv.n_seq, row0 = blockIdx.x * P.rows_per_block;
  const int rows = min(P.rows_per_block, P.n_rows - row0);
  for (int i = threadIdx.x; i <= S; i += kBThreads) s_off[i] = __ldg(P.kv.row_offsets + i);
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  const int page = P.kv.page_size, shift = __ffs(page) - 1;
  auto place = [&](int x, int n, int i) {
    int pg = -1, slots = 0;
    if (i >= 0 && i < n) {
      const int kv = __ldg(P.kv.kv_lens + x);
      const int64_t p = (int64_t)kv - n + i;
      // the sequence's first new row in this page
      if (p >= 0 && (i == 0 || p == 0 || (p & (page - 1)) == 0)) {
        pg = paged_page(P.kv, x, (int)(p >> shift), status);
        slots = (int)min((int64_t)page, kv - (p >> shift << shift));
      }
    }
    s_page[threadIdx.x] = pg;
    s_n[threadIdx.x] = slots;
  };
  paged_find_rows<kBThreads, kBRows>(S, P.n_rows, row0, rows, s_off, &s_bad, status, place);
  const T *keys = reinterpret_cast<const T *>(P.kv.k_pages) + blockIdx.z * P.cache_stride;
  T *bounds = reinterpret_cast<T *>(P.bounds) + blockIdx.z * P.layer_stride;
  const int c = threadIdx.x % kBCols, g = threadIdx.x / kBCols, col = blockIdx.y * kBCols + c;
  for (int r = 0; r < rows; ++r) {
    if (s_page[r] < 0) continue;
    const int n = s_n[r];
    float lo[VEC], hi[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      lo[i] = INFINITY;
      hi[i] = -INFINITY;
    }
    if (col < P.cols) {
      const T *src = keys + s_page[r] * P.kv.page_stride + col * VEC;
#pragma unroll 4
      for (int t = g; t < n; t += kSlots) {
        float x[VEC];
        load16<T>(src + t * P.kv.ld, x);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          lo[i] = fminf(lo[i], x[i]);
          hi[i] = fmaxf(hi[i], x[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      s_lo[g][c][i] = lo[i];
      s_hi[g][c][i] = hi[i];
    }
    __syncthreads();
    if (g < 2 && col < P.cols) {
      float y[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        y[i] = g ? s_hi[0][c][i] : s_lo[0][c][i];
#pragma unroll
        for (int k = 1; k < kSlots; ++k) y[i] = g ? fmaxf(y[i], s_hi[k][c][i]) : fminf(y[i], s_lo[k][c][i]);
      }
      store16<T>(bounds + s_page[r] * P.page_stride + g * P.ld + col * VEC, y);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- scores --
struct SelectParams {
  PagedKV kv;
  const void *bounds, *q;
  int64_t page_stride, ld, ld_q;        // elements
  int32_t *picks;
  float2 *approx;                       // [rows][Hkv][max_pages]: fp32 score, largest |bound|
  double *exact;                        // the same shape: exact scores of the pages at the border, one after another
  int *list;                            // the same shape: those pages
  int n_rows, G, Hkv, hd, max_kv;
  int held, parts;                      // pages of max_kv; blocks that score them
  int n_picks, n_first, n_last;
};

constexpr int kSThreads = 256, kSPages = 64;   // pages of a block

// The pages of a row: 0 at a negative position, -1 where the row has no sequence or its
// length is wrong (recorded).
__device__ __forceinline__ int pages_of(const SelectParams &P, const RowPlace &at, int *status) {
  if (at.s < 0) return -1;
  if (at.kv < 0 || at.kv > P.max_kv || at.kv > (int64_t)P.kv.max_pages * P.kv.page_size) {
    report(status, CB_ERR_DEVICE_INDEX);
    return -1;
  }
  return at.pos < 0 ? 0 : at.pos / P.kv.page_size + 1;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kSThreads)
paged_score_kernel(const __grid_constant__ SelectParams P, int *status) {
  constexpr int PER = HD / 32;
  __shared__ RowPlace s_row;
  grid_dep_wait();
  grid_dep_launch();
  const int part = blockIdx.x % P.parts, g = blockIdx.x / P.parts % P.Hkv, r = blockIdx.x / P.parts / P.Hkv;
  const RowPlace at = find_row<kSThreads>(P.kv, P.n_rows, r, &s_row, status);
  const int pages = pages_of(P, at, status);
  if (pages <= P.n_picks) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2 *out = P.approx + ((int64_t)r * P.Hkv + g) * P.held;
  const T *q = reinterpret_cast<const T *>(P.q) + r * P.ld_q + (int64_t)g * P.G * HD + lane * PER;
  const int end = min(pages - P.n_last, (part + 1) * kSPages);
  for (int j = part * kSPages + warp; j < end; j += kSThreads / 32) {
    if (j < P.n_first) continue;
    const int page = paged_page(P.kv, at.s, j, status);
    if (page < 0) {
      if (lane == 0) out[j] = make_float2(-INFINITY, 0.f);
      continue;
    }
    const T *b = reinterpret_cast<const T *>(P.bounds) + page * P.page_stride + g * HD + lane * PER;
    float lo[PER], hi[PER], top = 0.f, best = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      lo[i] = to_f(b[i]);
      hi[i] = to_f(b[P.ld + i]);
      top = fmaxf(top, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
    }
    for (int h = 0; h < P.G; ++h) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float x = to_f(q[h * HD + i]);
        sum = fmaf(x, x > 0.f ? hi[i] : lo[i], sum);
      }
      best = fmaxf(best, warp_sum(sum));
    }
    top = warp_max(top);
    if (lane == 0) out[j] = make_float2(best, top);
  }
}

// ---------------------------------------------------------------- choice --
constexpr int kCThreads = 512;

// A float's order as an unsigned number.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

// Sum of v over the block's threads before this one, and the whole.
__device__ __forceinline__ int block_scan(int v, int *s_warp, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = incl - v;
  total = 0;
#pragma unroll
  for (int w = 0; w < kCThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  return before;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kCThreads)
paged_choose_kernel(const __grid_constant__ SelectParams P, int *status) {
  __shared__ RowPlace s_row;
  __shared__ int s_hist[256], s_warp[kCThreads / 32], s_bin, s_rest, s_count;
  __shared__ float s_f[kCThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int g = blockIdx.x % P.Hkv, r = blockIdx.x / P.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RowPlace at = find_row<kCThreads>(P.kv, P.n_rows, r, &s_row, nullptr);
  const int pages = pages_of(P, at, nullptr);
  int32_t *out = P.picks + ((int64_t)r * P.Hkv + g) * P.n_picks;
  if (pages < 0) return;
  if (pages <= P.n_picks) {
    for (int i = tid; i < P.n_picks; i += kCThreads) out[i] = i < pages ? i : -1;
    return;
  }
  const int64_t base = ((int64_t)r * P.Hkv + g) * P.held;
  float2 *a = P.approx + base;
  double *exact = P.exact + base;
  int *list = P.list + base;
  const int lo = P.n_first, hi = pages - P.n_last;          // scored pages
  const int want = P.n_picks - P.n_first - P.n_last;        // of them are picked, fewer than there are
  float t = INFINITY, eps = 0.f;
  if (want > 0) {
    // eps: |q|_1 of the heads, the largest bound
    const T *q = reinterpret_cast<const T *>(P.q) + r * P.ld_q + (int64_t)g * P.G * HD;
    float norm = 0.f, top = 0.f;
    for (int h = warp; h < P.G; h += kCThreads / 32) {
      float s = 0.f;
      for (int i = lane; i < HD; i += 32) s += fabsf(to_f(q[h * HD + i]));
      norm = fmaxf(norm, warp_sum(s));
    }
    for (int j = lo + tid; j < hi; j += kCThreads) top = fmaxf(top, a[j].y);
    auto block_max = [&](float v) {
      v = warp_max(v);
      __syncthreads();
      if (lane == 0) s_f[warp] = v;
      __syncthreads();
      float x = s_f[0];
      for (int w = 1; w < kCThreads / 32; ++w) x = fmaxf(x, s_f[w]);
      return x;
    };
    norm = block_max(norm);
    top = block_max(top);
    eps = 0x1p-15f * norm * top;
    // the want-th largest fp32 score, eight bits at a time
    uint32_t prefix = 0;
    int rest = want;
    for (int sh = 24; sh >= 0; sh -= 8) {
      for (int i = tid; i < 256; i += kCThreads) s_hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kCThreads) {
        const uint32_t u = ordered(a[j].x);
        if (sh == 24 || u >> (sh + 8) == prefix >> (sh + 8)) atomicAdd(&s_hist[u >> sh & 255], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // lane: bins 255 - 8 lane .. 248 - 8 lane, from the largest down
        int n = 0;
        for (int i = 0; i < 8; ++i) n += s_hist[255 - 8 * lane - i];
        int incl = n;
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        int above = incl - n;
        if (above < rest && incl >= rest) {
          int b = 255 - 8 * lane;
          while (above + s_hist[b] < rest) above += s_hist[b--];
          s_bin = b;
          s_rest = rest - above;
        }
      }
      __syncthreads();
      prefix |= (uint32_t)s_bin << sh;
      rest = s_rest;
      __syncthreads();
    }
    t = unordered(prefix);
  }
  // how many are in for certain; exact scores of those at the border
  const float sure = t + 2.f * eps, none = t - 2.f * eps;
  if (tid == 0) s_count = 0;
  __syncthreads();
  int in = 0, total;
  for (int j0 = lo + warp * 32; j0 < hi && want > 0; j0 += kCThreads) {
    const float x = j0 + lane < hi ? a[j0 + lane].x : -INFINITY;
    if (j0 + lane < hi) in += x > sure;
    unsigned border = __ballot_sync(0xffffffffu, j0 + lane < hi && !(x > sure) && x >= none);
    while (border) {
      const int j = j0 + __ffs(border) - 1;
      border &= border - 1;
      const int page = paged_page(P.kv, at.s, j, nullptr);
      double best = -INFINITY;
      if (page >= 0) {
        const T *b = reinterpret_cast<const T *>(P.bounds) + page * P.page_stride + g * HD;
        const T *q = reinterpret_cast<const T *>(P.q) + r * P.ld_q + (int64_t)g * P.G * HD;
        for (int h = 0; h < P.G; ++h) {
          double sum = 0.0;
#pragma unroll
          for (int i = lane; i < HD; i += 32) {
            const float y = to_f(q[h * HD + i]);
            sum += (double)y * (double)to_f(y > 0.f ? b[P.ld + i] : b[i]);
          }
          best = fmax(best, warp_sum_d(sum));
        }
      }
      if (lane == 0) {
        const int c = atomicAdd(&s_count, 1);
        exact[c] = best;
        list[c] = j;
      }
    }
  }
  block_scan(in, s_warp, total);
  const int need = want - total;                            // of the pages at the border
  __syncthreads();
  // their ranks: -1 in place of the bound of a page that is picked, -2 of one that is not
  for (int c = tid; c < s_count; c += kCThreads) {
    const double e = exact[c];
    const int j = list[c];
    int better = 0;
    for (int k = 0; k < s_count && better < need; ++k) {
      const double f = exact[k];
      better += f > e || (f == e && list[k] < j);
    }
    a[j].y = better < need ? -1.f : -2.f;
  }
  __syncthreads();
  int written = 0;
  for (int j0 = 0; j0 < pages; j0 += kCThreads) {
    const int j = j0 + tid;
    bool pick = j < pages && (j < lo || j >= hi);
    if (j >= lo && j < hi && want > 0) {
      const float2 x = a[j];
      pick = x.y < 0.f ? x.y == -1.f : x.x > sure;
    }
    int n;
    const int before = block_scan(pick, s_warp, n);
    if (pick) out[written + before] = j;
    written += n;
  }
}

}  // namespace pages

cudaError_t launch_paged_bounds(const PagedKV &kv, const cb_page_bounds &b, cb_dtype dt, int *status, cudaStream_t s) {
  using namespace pages;
  BoundsParams P;
  P.kv = kv;
  P.bounds = b.bounds;
  P.page_stride = b.page_stride;
  P.ld = b.ld;
  P.layer_stride = b.bounds_layer_stride;
  P.cache_stride = b.cache_layer_stride;
  P.n_rows = b.n_rows;
  P.cols = b.n_kv_heads * b.head_dim / (dt == CB_BF16 ? 8 : 4);
  P.rows_per_block = max(1, min(kBRows, b.n_rows / (4 * device_sm_count())));
  const dim3 grid((b.n_rows + P.rows_per_block - 1) / P.rows_per_block, (P.cols + kBCols - 1) / kBCols, b.n_layers);
  const cudaError_t e = dt == CB_BF16 ? launch_pdl(paged_bounds_kernel<bf16>, grid, dim3(kBThreads), 0, s, P, status)
                                      : launch_pdl(paged_bounds_kernel<float>, grid, dim3(kBThreads), 0, s, P, status);
  return e == cudaSuccess ? launched(1) : e;
}

static int64_t held_pages(int max_kv, int page_size) { return ((int64_t)max_kv + page_size - 1) / page_size; }

size_t paged_select_ws_bytes(int n_rows, int max_kv, int page_size, int Hkv) {
  return (size_t)n_rows * Hkv * held_pages(max_kv, page_size) * (sizeof(float2) + sizeof(double) + sizeof(int));
}

template <typename T, int HD>
static cudaError_t run_select(const pages::SelectParams &P, int *status, cudaStream_t s) {
  using namespace pages;
  int n = 0;
  if (P.held > P.n_picks) {
    const cudaError_t e = launch_pdl(paged_score_kernel<T, HD>, dim3(P.parts * P.Hkv * P.n_rows), dim3(kSThreads), 0, s, P, status);
    if (e != cudaSuccess) return e;
    ++n;
  }
  const cudaError_t e = launch_pdl(paged_choose_kernel<T, HD>, dim3(P.Hkv * P.n_rows), dim3(kCThreads), 0, s, P, status);
  return e == cudaSuccess ? launched(n + 1) : e;
}

cudaError_t launch_paged_select(const PagedKV &kv, const cb_page_bounds &b, const cb_page_select &a, cb_dtype dt,
                                int *status, cudaStream_t s) {
  pages::SelectParams P;
  P.kv = kv;
  P.bounds = b.bounds;
  P.q = a.q;
  P.page_stride = b.page_stride;
  P.ld = b.ld;
  P.ld_q = a.ld_q;
  P.picks = a.picks;
  P.n_rows = b.n_rows;
  P.G = a.n_q_heads / b.n_kv_heads;
  P.Hkv = b.n_kv_heads;
  P.hd = b.head_dim;
  P.max_kv = a.max_kv_len;
  P.held = (int)held_pages(a.max_kv_len, kv.page_size);
  P.n_picks = a.n_picks;
  P.n_first = a.n_first;
  P.n_last = a.n_last;
  P.approx = reinterpret_cast<float2 *>(a.ws);
  const size_t all = (size_t)b.n_rows * P.Hkv * P.held;
  P.exact = reinterpret_cast<double *>(P.approx + all);
  P.list = reinterpret_cast<int *>(P.exact + all);
  P.parts = (P.held + pages::kSPages - 1) / pages::kSPages;
  if ((int64_t)P.parts * P.Hkv * b.n_rows > 0x7fffffffLL || (int64_t)P.Hkv * b.n_rows > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  if (dt == CB_BF16) return P.hd == 128 ? run_select<bf16, 128>(P, status, s) : run_select<bf16, 64>(P, status, s);
  return P.hd == 128 ? run_select<float, 128>(P, status, s) : run_select<float, 64>(P, status, s);
}

}  // namespace cb
