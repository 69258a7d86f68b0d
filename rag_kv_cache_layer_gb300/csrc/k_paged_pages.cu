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
// (256 products of one sum, each rounded, summed in fp32 with truncated sums: 2 * 256 *
// 2^-24).  The fp32 score in the place of the last one that fits lies in some range
// [from, to]; pages above to + 2 eps are in, pages below from - 2 eps are not, and the
// few between are scored again with exact products in pairs of floats (2^-44 of the
// terms; an fp64 sum costs twenty times as much here) and ranked (ties: the lower
// page): the picks are those of the exact scores.  How many there are follows the data, since
// the bound takes the largest |bound| of any page: see kRanked for many.
//
// A generated token reads two bounds for a page in place of its keys: the scores are
// a stream over the bounds.
//
// Measured, bf16, 32/8 heads of 128, the three launches after one another: 64 requests of up
// to 65,536 keys in pages of 32 47 us (158 MB of bounds), two of 131,072 keys in pages of 16
// 31 us (66 MB; 24 where they stay in L2).  Of the first about 33 are the scores (4.8 TB/s, with 6 us of launch, line
// and first loads in them), 7 the choice, a block of dependent steps for each row and
// head, and 4.5 the bounds.
#include "cb_common.cuh"
#include "cb_internal.h"
#include <type_traits>

#include "cb_paged.cuh"
#include "cb_paged_attn.cuh"
#include "cb_paged_few.cuh"

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
  __shared__ int s_off[CB_MAX_SEQS + 1], s_len[CB_MAX_SEQS];
  __shared__ int s_page[kBRows], s_n[kBRows], s_bad;   // page (-1: none) and covered slots of an owning row
  __shared__ float s_lo[kSlots][kBCols][VEC + 1], s_hi[kSlots][kBCols][VEC + 1];
  grid_dep_wait();
  grid_dep_launch();
  const int S = P.kv.n_seq, row0 = blockIdx.x * P.rows_per_block;
  const int rows = min(P.rows_per_block, P.n_rows - row0);
  for (int i = threadIdx.x; i <= S; i += kBThreads) {
    s_off[i] = __ldg(P.kv.row_offsets + i);
    if (i < S) s_len[i] = __ldg(P.kv.kv_lens + i);
  }
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  const int page = P.kv.page_size, shift = __ffs(page) - 1;
  auto place = [&](int x, int n, int i) {
    int pg = -1, slots = 0;
    if (i >= 0 && i < n) {
      const int kv = s_len[x];
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
  float2 *exact;                        // the same shape: exact scores of the pages at the border, one after another
  int *list;                            // the same shape: those pages
  int n_rows, G, Hkv, hd, max_kv;
  int held, parts;                      // pages of max_kv; blocks that score them
  int n_picks, n_first, n_last;
  paged::Divisor by_heads;              // Hkv
  bool scored;                          // the launch before the choice is the scores'
};

constexpr int kSThreads = 256;
constexpr int kSPages = kSThreads / 32 * 8;   // fp32: pages of a block

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

// v[0..7], each over the warp's lanes: lane l has that of v[l / 4] (nine shuffles in place of
// forty).
template <typename F> __device__ __forceinline__ float reduce8(float (&v)[8], int lane, F &&op) {
#pragma unroll
  for (int n = 4; n > 0; n >>= 1) {
    const bool up = lane & (4 * n);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + n], 4 * n);
      v[i] = op(up ? v[i + n] : v[i], other);
    }
  }
  float r = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
  return op(r, __shfl_xor_sync(0xffffffffu, r, 1));
}

// fp32: a warp's eight pages at once, a lane HD / 32 dimensions of them; the selection of 64
// pages for 64 requests of 30,000 keys in pages of 32, 32/8 heads of 128, takes 136 to 141 us (a
// page and head at a time 219), bf16 56.
template <int HD>
__global__ void __launch_bounds__(kSThreads)
paged_score_kernel(const __grid_constant__ SelectParams P, int *status) {
  constexpr int PER = HD / 32;
  typedef typename std::conditional<PER == 4, float4, float2>::type Vec;
  __shared__ RowPlace s_row;
  grid_dep_wait();
  grid_dep_launch();
  const int part = blockIdx.x % P.parts, g = blockIdx.x / P.parts % P.Hkv, r = blockIdx.x / P.parts / P.Hkv;
  const RowPlace at = find_row<kSThreads>(P.kv, P.n_rows, r, &s_row, status);
  const int pages = pages_of(P, at, status);
  if (pages <= P.n_picks) return;
  const int lane = threadIdx.x & 31, j0 = part * kSPages + (threadIdx.x >> 5) * 8;
  const int end = pages - P.n_last;
  int page = -1;
  if (lane < 8 && j0 + lane >= P.n_first && j0 + lane < end) page = paged_page(P.kv, at.s, j0 + lane, status);
  const float *bounds = reinterpret_cast<const float *>(P.bounds) + g * HD + lane * PER;
  float lo[8][PER], hi[8][PER], v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = __shfl_sync(0xffffffffu, page, i);
    Vec a = {}, b = {};
    if (p >= 0) {
      a = __ldg(reinterpret_cast<const Vec *>(bounds + p * P.page_stride));
      b = __ldg(reinterpret_cast<const Vec *>(bounds + p * P.page_stride + P.ld));
    }
    v[i] = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      lo[i][k] = reinterpret_cast<const float *>(&a)[k];
      hi[i][k] = reinterpret_cast<const float *>(&b)[k];
      v[i] = fmaxf(v[i], fmaxf(fabsf(lo[i][k]), fabsf(hi[i][k])));
    }
  }
  const float top = reduce8(v, lane, [](float a, float b) { return fmaxf(a, b); });
  const float *q = reinterpret_cast<const float *>(P.q) + r * P.ld_q + (int64_t)g * P.G * HD + lane * PER;
  float best = -INFINITY;
  for (int h = 0; h < P.G; ++h) {
    const Vec x = __ldg(reinterpret_cast<const Vec *>(q + (int64_t)h * HD));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const float y = reinterpret_cast<const float *>(&x)[k];
      const bool up = y > 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(y, up ? hi[i][k] : lo[i][k], v[i]);
    }
    best = fmaxf(best, reduce8(v, lane, [](float a, float b) { return a + b; }));
  }
  const int j = j0 + lane / 4;
  const bool there = __shfl_sync(0xffffffffu, page, lane / 4) >= 0;
  if (lane % 4 == 0 && j >= P.n_first && j < end)
    P.approx[((int64_t)r * P.Hkv + g) * P.held + j] = there ? make_float2(best, top) : make_float2(-INFINITY, 0.f);
}

// bf16: a warp takes 16 pages and one kv head at a time, 8 q heads per instruction: the
// bounds are the 16-row side of mma.m16n8k16, (q^+, q^-) the 8-column side; each warp
// keeps two tiles of bounds on their way by cp.async.  All rows' tiles of 16
// pages form one line that the grid shares in equal parts (long and short requests in
// one batch keep every SM busy); neighbouring warps take neighbouring heads of the same
// pages, whose bounds lie side by side.
constexpr int kTStages = 3;              // of each warp: 192 KB of bounds in a block (64 requests 47.7 us; two stages 48.1)

// The line: tiles of a sequence, each of its rows as many as its last one.
struct ScoreLine {
  int64_t begin[CB_MAX_SEQS + 1];       // first tile of each sequence
  int tiles[CB_MAX_SEQS];               // tiles of one of its rows
  int row0[CB_MAX_SEQS + 1], kv[CB_MAX_SEQS];
};

// (the bound of 384 threads leaves registers for a block of the choice beside this one's)
template <int HD>
__global__ void __launch_bounds__(384, 1)
paged_score_tc_kernel(const __grid_constant__ SelectParams P, int *status) {
  constexpr int kBytes = HD * 2, kStage = 16 * 2 * kBytes;   // of a bound; 16 pages' minima and maxima
  constexpr int PER = (CB_MAX_SEQS + kSThreads - 1) / kSThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ScoreLine line;
  __shared__ int64_t s_sums[kSThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, q4 = lane & 3;
  const int S = P.kv.n_seq, page_size = P.kv.page_size, shift = __ffs(page_size) - 1;
  {
    const int per = (S + kSThreads - 1) / kSThreads, i0 = threadIdx.x * per;
    int64_t n[PER], sum = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      n[k] = 0;
      const int i = i0 + k;
      if (k < per && i < S) {
        const int rows = paged_rows(P.kv, i, P.n_rows, status), kv = __ldg(P.kv.kv_lens + i);
        int tiles = 0;
        if (rows > 0) {
          if (kv < 0 || kv > P.max_kv || kv > (int64_t)P.kv.max_pages * page_size) {
            report(status, CB_ERR_DEVICE_INDEX);
          } else {
            const int pages = kv > 0 ? ((kv - 1) >> shift) + 1 : 0;
            if (pages > P.n_picks) tiles = (pages - P.n_first - P.n_last + 15) / 16;
          }
        }
        line.tiles[i] = tiles;
        line.row0[i] = __ldg(P.kv.row_offsets + i);
        line.kv[i] = kv;
        n[k] = (int64_t)rows * tiles;
        sum += n[k];
      }
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_sums[warp] = incl;
    __syncthreads();
    int64_t first = incl - sum;
    for (int w = 0; w < warp; ++w) first += s_sums[w];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (k < per && i0 + k < S) line.begin[i0 + k] = first;
      first += n[k];
    }
    if (threadIdx.x == kSThreads - 1) {
      line.begin[S] = first;
      line.row0[S] = __ldg(P.kv.row_offsets + S);
    }
    __syncthreads();
  }
  const int64_t units = line.begin[S] * P.Hkv;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  const uint32_t ring = smem_u32(smem) + warp * kTStages * kStage;
  // A unit's tile: row r, head g, pages j .. j + count - 1 (0: nothing), and in lanes 0..15
  // their places in the pool (-1: none).  What the table says is looked at only when the
  // tile is loaded: until then the entries are on their way.
  struct Tile { int r, g, j, count, page; };
  int s = -1, row0 = 0, n = 0, kv = 0;
  auto describe = [&](int64_t u) -> Tile {
    Tile t = {0, 0, 0, 0, -1};
    if (u >= u1) return t;
    int64_t tile;
    if (units >> 31 == 0) {             // (a 64-bit division is several times slower)
      tile = P.by_heads.div((int)u);
      t.g = (int)u - (int)tile * P.Hkv;
    } else {
      tile = u / P.Hkv;
      t.g = (int)(u - tile * P.Hkv);
    }
    if (s < 0 || line.begin[s + 1] <= tile) {
      int lo = max(s, 0), hi = S - 1;   // the last sequence that begins at or before the tile
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (line.begin[mid] <= tile) lo = mid; else hi = mid - 1;
      }
      s = lo;
      row0 = line.row0[s];
      n = line.row0[s + 1] - row0;
      kv = line.kv[s];
    }
    const int64_t local = tile - line.begin[s];
    const int per = line.tiles[s], i = n == 1 ? 0 : (int)(local / per);
    const int pos = kv - n + i, pages = pos < 0 ? 0 : (pos >> shift) + 1;
    t.r = row0 + i;
    t.j = P.n_first + (int)(local - (int64_t)i * per) * 16;
    // 0: the row has fewer pages than the sequence's last, or takes all
    t.count = pages > P.n_picks ? max(0, min(16, pages - P.n_last - t.j)) : 0;
    if (lane < t.count) t.page = __ldg(P.kv.block_table + (int64_t)s * P.kv.ld_table + t.j + lane);
    return t;
  };
  // Its bounds to a stage: a warp copies a page's two at once.  16-byte columns are swizzled
  // by the page so that ldmatrix meets all banks.
  auto load = [&](Tile &t, int st) {
    if (lane < t.count && (t.page < 0 || t.page >= P.kv.n_pages)) {
      report(status, CB_ERR_DEVICE_INDEX);
      t.page = -1;
    }
    constexpr int kCols = kBytes / 16, kPages = 16 / kCols;      // pages of one copy (1 or 2)
    const int x = lane / (2 * kCols), half = lane / kCols & 1, col = lane % kCols;
    const bf16 *src = reinterpret_cast<const bf16 *>(P.bounds) + half * P.ld + t.g * HD + col * 8;
    uint32_t dst = ring + st * kStage + half * kBytes;
    if (__all_sync(0xffffffffu, t.page >= 0 || lane >= 16)) {
#pragma unroll
      for (int i = 0; i < 16 / kPages; ++i) {
        const int p = i * kPages + x, page = __shfl_sync(0xffffffffu, t.page, p);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + p * 2 * kBytes + ((col ^ (p & 7)) << 4)),
                     "l"(src + page * P.page_stride) : "memory");
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16 / kPages; ++i) {
        const int p = i * kPages + x, page = __shfl_sync(0xffffffffu, t.page, p);
        paged::copy16(dst + p * 2 * kBytes + ((col ^ (p & 7)) << 4), src + (page < 0 ? 0 : page * P.page_stride), page >= 0);
      }
    }
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
  // Tiles in flight, the first of them to be scored next; places are looked up one tile
  // ahead of the bounds.  The first kTStages rounds only fill the line: code that stands
  // here once is fetched once (64 requests 47.6 us; with a prologue of its own 48.1).
  Tile wait[kTStages];
#pragma unroll
  for (int i = 0; i < kTStages; ++i) wait[i].count = 0;
  constexpr int kStep = kSThreads / 32;
  uint32_t up[HD / 8], down[HD / 8];
  int q_row = -1, q_head = -1, q_first = -1;
  int st = 0, fill = kTStages - 1;
#pragma unroll 1
  for (int64_t u = u0 + warp - kTStages * kStep; u < u1; u += kStep) {
    const Tile t = wait[0];
    asm volatile("cp.async.wait_group %0;" ::"n"(kTStages - 2) : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i + 1 < kTStages; ++i) wait[i] = wait[i + 1];
    if (wait[kTStages - 2].count) load(wait[kTStages - 2], fill);
    commit();
    wait[kTStages - 1] = describe(u + kTStages * kStep);
    const uint32_t stage = ring + st * kStage;
    st = st + 1 == kTStages ? 0 : st + 1;
    fill = fill + 1 == kTStages ? 0 : fill + 1;
    if (!t.count) continue;
    const int g = t.g, r = t.r, j = t.j, j1 = t.j + t.count;
    const bf16 *q = reinterpret_cast<const bf16 *>(P.q) + r * P.ld_q + (int64_t)g * P.G * HD + q4 * 2;
    // ldmatrix: lanes 0..7 the first eight pages' eight dimensions, 8..15 the other pages',
    // 16..31 the next dimensions
    const int page = lane & 15;
    const uint32_t rows = stage + page * 2 * kBytes;
    float best[2] = {-INFINITY, -INFINITY};
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 least[2] = {zero, zero}, most[2] = {zero, zero};     // of pages gid and gid + 8
    for (int h0 = 0; h0 < P.G; h0 += 8) {
      // q^+ and q^- of this lane's head: kept while the row and the heads stay
      if (r != q_row || g != q_head || h0 != q_first) {
        q_row = r;
        q_head = g;
        q_first = h0;
#pragma unroll
        for (int k = 0; k < HD / 8; ++k) {
          uint32_t x = 0;
          if (h0 + gid < P.G) x = __ldg(reinterpret_cast<const uint32_t *>(q + (int64_t)(h0 + gid) * HD + k * 8));
          const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162 *>(&x);
          const __nv_bfloat162 p = __hmax2(v, zero), m = __hmin2(v, zero);
          up[k] = *reinterpret_cast<const uint32_t *>(&p);
          down[k] = *reinterpret_cast<const uint32_t *>(&m);
        }
      }
      float c[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        uint32_t lo[4], hi[4];
        const uint32_t at = rows + (((2 * k + (lane >> 4)) ^ (page & 7)) << 4);
        paged::ldsm_x4(at, lo);
        paged::ldsm_x4(at + kBytes, hi);
        paged::mma16816(c, hi, up[2 * k], up[2 * k + 1]);
        paged::mma16816(d, lo, down[2 * k], down[2 * k + 1]);
        if (h0 == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            least[e & 1] = __hmin2(least[e & 1], *reinterpret_cast<const __nv_bfloat162 *>(&lo[e]));
            most[e & 1] = __hmax2(most[e & 1], *reinterpret_cast<const __nv_bfloat162 *>(&hi[e]));
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (h0 + 2 * q4 + (e & 1) < P.G) best[e >> 1] = fmaxf(best[e >> 1], c[e] + d[e]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // the largest |bound|: of the maxima, or of the minima's opposites
      float top = fmaxf(fmaxf(__low2float(most[h]), __high2float(most[h])), -fminf(__low2float(least[h]), __high2float(least[h])));
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        best[h] = fmaxf(best[h], __shfl_xor_sync(0xffffffffu, best[h], o));
      }
      const int jj = j + gid + 8 * h;
      const bool there = __shfl_sync(0xffffffffu, t.page, gid + 8 * h) >= 0;
      if (q4 == 0 && jj < j1)
        P.approx[((int64_t)r * P.Hkv + g) * P.held + jj] = there ? make_float2(best[h], top) : make_float2(-INFINITY, 0.f);
    }
  }
}

// ---------------------------------------------------------------- choice --
// The largest v of the warp (redux.sync of floats: one instruction in place of ten).
__device__ __forceinline__ float warp_top(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Sum of v over the block's NT threads before this one, and the whole.
template <int NT> __device__ __forceinline__ int block_scan(int v, int *s_warp, int &total) {
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
  const int sum = lane < NT / 32 ? s_warp[lane] : 0;
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  total = __shfl_sync(0xffffffffu, upto, 31);
  const int before = __shfl_sync(0xffffffffu, upto - sum, warp) + incl - v;
  return before;
}

constexpr int kBins = 2048, kHeld = 8;  // bins of a histogram; scores a thread keeps in registers
constexpr int kFew = 32;                // candidates that need no narrower bins
constexpr int kPairs = 8;               // pages, and heads, scored exactly at a time
// Candidates that are ranked against each other; the border among more is found digit by digit
// (two requests of 131,072 keys with one page of large bounds 85 us, with 1024 for 256 200).
constexpr int kRanked = 256;

// Sums in pairs of floats: (hi, lo) + x, with the sum's rounding kept in lo.
__device__ __forceinline__ void add_exact(float &hi, float &lo, float x) {
  const float s = hi + x, t = s - hi;
  lo += (hi - (s - t)) + (x - t);
  hi = s;
}
// x y as a pair (__fmul_rn: the rounded product, whatever it is added to).
__device__ __forceinline__ void add_product(float &hi, float &lo, float x, float y) {
  const float p = __fmul_rn(x, y);
  lo += fmaf(x, y, -p);
  add_exact(hi, lo, p);
}

// A float's bits in its order (0 and -0 are one).
__device__ __forceinline__ unsigned ordered(float x) {
  const unsigned b = __float_as_uint(x + 0.f);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}

// kCThreads: 256 for up to 2048 pages, all in registers, 1024 for more (512 rows and heads of
// up to 2048 pages: 48 us with 256, 64 with 1024; 16 of 8192 pages: 31 with 1024, 49 with 256).
template <typename T, int HD, int kCThreads>
__global__ void __launch_bounds__(kCThreads, 1024 / kCThreads)
paged_choose_kernel(const __grid_constant__ SelectParams P, int *status) {
  constexpr int NW = kCThreads / 32;
  __shared__ RowPlace s_row;
  __shared__ int s_hist[kBins + kBins / 32], s_warp[NW], s_bin, s_in, s_count, s_sure;
  __shared__ float s_f[4][NW];
  __shared__ unsigned s_mask[kCThreads];
  __shared__ float2 s_pair[kPairs * kPairs];
  static_assert(kCThreads <= kBins, "the masks' places reuse the bins");
  if (!P.scored) grid_dep_wait();
  const int g = blockIdx.x % P.Hkv, r = blockIdx.x / P.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (the scores' kernel records what is wrong, where it runs)
  int *const record = P.scored ? nullptr : status;
  const RowPlace at = find_row<kCThreads>(P.kv, P.n_rows, r, &s_row, record);
  const int pages = pages_of(P, at, record);
  int32_t *out = P.picks + ((int64_t)r * P.Hkv + g) * P.n_picks;
  const int want = P.n_picks - P.n_first - P.n_last;        // of the scored pages are picked, fewer than there are
  const T *q = reinterpret_cast<const T *>(P.q) + r * P.ld_q + (int64_t)g * P.G * HD;
  float norm = 0.f;                                         // |q|_1 of this warp's heads
  if (pages > P.n_picks && want > 0)
    for (int h = warp; h < P.G; h += NW) {
      float s = 0.f;
#pragma unroll
      for (int i = lane; i < HD; i += 32) s += fabsf(to_f(q[h * HD + i]));
      norm = fmaxf(norm, warp_sum(s));
    }
  // what was read so far was there before the scores' kernel began, which waited for it
  if (P.scored) grid_dep_wait();
  grid_dep_launch();
  if (pages < 0) return;
  if (pages <= P.n_picks) {
    for (int i = tid; i < P.n_picks; i += kCThreads) out[i] = i < pages ? i : -1;
    return;
  }
  const int64_t base = ((int64_t)r * P.Hkv + g) * P.held;
  float2 *a = P.approx + base;
  float2 *exact = P.exact + base;
  int *list = P.list + base;
  const int lo = P.n_first, hi = pages - P.n_last;          // scored pages
  float sure = INFINITY, none = INFINITY;                   // above: in; below: out; between: scored exactly
  bool flat = false;                                        // those between all have the same score
  // scores lo + tid + i * kCThreads, the first kHeld of them in registers
  float held[kHeld];
  auto each = [&](auto &&f) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (lo + tid + i * kCThreads < hi) f(lo + tid + i * kCThreads, held[i]);
    for (int j = lo + tid + kHeld * kCThreads; j < hi; j += kCThreads) f(j, a[j].x > -INFINITY ? a[j].x : -INFINITY);
  };
  if (want > 0) {
    float v[4] = {-INFINITY, -INFINITY, 0.f, norm};          // largest score, largest negative, |bound|, |q|_1
    int finite = 0, in_pool;
    auto take = [&](float2 x) {
      if (x.x > -INFINITY) {                                // (a page outside the pool has -inf)
        v[1] = fmaxf(v[1], -x.x);
        ++finite;
      }
      v[0] = fmaxf(v[0], x.x);
      v[2] = fmaxf(v[2], x.y);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int j = lo + tid + i * kCThreads;
      const float2 x = j < hi ? a[j] : make_float2(-INFINITY, 0.f);
      held[i] = x.x > -INFINITY ? x.x : -INFINITY;          // (a NaN counts as a page outside the pool)
      take(x);
    }
    for (int j = lo + tid + kHeld * kCThreads; j < hi; j += kCThreads) take(a[j]);
    finite = __reduce_add_sync(0xffffffffu, finite);
    if (lane == 0) s_warp[warp] = finite;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = warp_top(v[k]);
      if (lane == 0) s_f[k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = warp_top(lane < NW ? s_f[k][lane] : v[k]);
    const float eps = 0x1p-15f * v[3] * v[2];
    in_pool = __reduce_add_sync(0xffffffffu, lane < NW ? s_warp[lane] : 0);
    // zeros (a slot of a batch without a request, say), or the pages outside the pool
    flat = v[3] == 0.f || v[2] == 0.f || in_pool < want;
    // [from, to] holds the score in the last place that fits: bins over it, the one with
    // that place in turn, until few scores (or nothing to tell apart) are left
    float from = -v[1], to = v[0];
    int above = 0;                                          // scores above `to`
    for (int round = 0; round < 8 && in_pool >= want; ++round) {
      for (int i = tid; i < kBins + kBins / 32; i += kCThreads) s_hist[i] = 0;
      __syncthreads();
      const float width = to - from, inv = kBins / width;
      if (!(width > 2.f * eps) || !(inv < INFINITY)) break;
      auto place = [](int b) { return b + (b >> 5); };       // so that a scan's threads meet all banks
      auto bin = [&](float x) { return min(kBins - 1, (int)((x - from) * inv)); };
      each([&](int, float x) {
        if (x >= from && x <= to) atomicAdd(&s_hist[place(bin(x))], 1);
      });
      __syncthreads();
      // thread t: bins from the largest down, kBins / kCThreads of them
      constexpr int PER = kBins / kCThreads;
      int n[PER], sum = 0, all;
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += n[i] = s_hist[place(kBins - 1 - tid * PER - i)];
      int before = above + block_scan<kCThreads>(sum, s_warp, all);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (before < want && before + n[i] >= want) {
          s_bin = kBins - 1 - tid * PER - i;
          s_in = n[i];
        }
        before += n[i];
      }
      __syncthreads();
      // the bin's scores lie between its edges; a rounding of the edges moves them by
      // less than 2^-20 of the range, which the margins cover
      const float b0 = from + s_bin * (width / kBins), b1 = from + (s_bin + 1) * (width / kBins), slack = 0x1p-20f * (fabsf(from) + fabsf(to));
      const bool few = s_in <= kFew;
      to = fminf(to, b1 + slack);
      from = fmaxf(from, b0 - slack);
      __syncthreads();
      if (few || !(to - from < width)) break;
      // (with the slack the range may hold scores of the neighbouring bins: count anew)
      int over = 0;
      each([&](int, float x) { over += x > to; });
      block_scan<kCThreads>(over, s_warp, above);
      __syncthreads();
    }
    // (all pages of the pool, and some outside, where those do not suffice)
    sure = in_pool >= want ? to + 2.f * eps : -3.402823466e38f;
    none = in_pool >= want ? from - 2.f * eps : -INFINITY;
  }
  // how many are in for certain (where registers hold all scores, as masks of 32 pages
  // each); the list of those between
  const bool masks = hi - lo <= kHeld * kCThreads;
  if (tid == 0) s_count = s_sure = 0;
  __syncthreads();
  if (want > 0) {
    int in = 0;
    if (masks) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int j = lo + tid + i * kCThreads;
        const bool sure_in = j < hi && held[i] > sure;
        const unsigned mask = __ballot_sync(0xffffffffu, sure_in);
        if (lane == 0) s_mask[i * NW + warp] = mask;
        in += __popc(mask);
        if (j < hi && !sure_in && held[i] >= none) list[atomicAdd(&s_count, 1)] = j;
      }
      if (lane == 0) atomicAdd(&s_sure, in);
    } else {
      each([&](int j, float x) {
        if (x > sure) ++in;
        else if (x >= none) list[atomicAdd(&s_count, 1)] = j;
      });
      atomicAdd(&s_sure, in);
    }
  } else if (masks) {
    for (int i = tid; i < kHeld * NW; i += kCThreads) s_mask[i] = 0;
  }
  __syncthreads();
  const int need = want - s_sure;                           // of the pages between
  // the exact score of page j: the largest of the heads h0, h0 + step, ..
  auto exact_score = [&](int j, int h0, int step) -> float2 {
    const int page = paged_page(P.kv, at.s, j, nullptr);
    float2 best = make_float2(-INFINITY, 0.f);
    if (page < 0) return best;
    const T *b = reinterpret_cast<const T *>(P.bounds) + page * P.page_stride + g * HD;
    for (int h = h0; h < P.G; h += step) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = lane; i < HD; i += 32) {
        const float y = to_f(q[h * HD + i]);
        add_product(sum.x, sum.y, y, to_f(y > 0.f ? b[P.ld + i] : b[i]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, sum.x, o), y = __shfl_xor_sync(0xffffffffu, sum.y, o);
        // (both lanes of a pair add the same two numbers in the same order)
        float hi = lane & o ? x : sum.x, lo = sum.y + y;
        add_exact(hi, lo, lane & o ? sum.x : x);
        sum = make_float2(hi, lo);
      }
      const float hi = sum.x + sum.y, lo = fabsf(hi) < INFINITY ? sum.y - (hi - sum.x) : 0.f;   // one pair for one sum
      if (hi > best.x || (hi == best.x && lo > best.y)) best = make_float2(hi, lo);
    }
    return best;
  };
  const bool many = s_count > kRanked && s_count > need && need > 0;
  if (many && !flat) {
    for (int c = warp; c < s_count; c += NW) {
      const float2 best = exact_score(list[c], 0, 1);
      if (lane == 0) exact[c] = best;
    }
    __syncthreads();
  } else if (s_count > need && !flat) {
    // a warp takes a page and, of up to eight heads, one; the largest of a page's heads
    // afterwards
    const int heads = min(P.G, kPairs);
    for (int c0 = 0; c0 < s_count; c0 += kPairs) {
      const int pairs = min(kPairs, s_count - c0) * heads;
      for (int k = warp; k < pairs; k += NW) {
        const float2 best = exact_score(list[c0 + k / heads], k % heads, heads);
        if (lane == 0) s_pair[k] = best;
      }
      __syncthreads();
      if (tid < kPairs && c0 + tid < s_count) {
        float2 best = s_pair[tid * heads];
        for (int h = 1; h < heads; ++h) {
          const float2 x = s_pair[tid * heads + h];
          if (x.x > best.x || (x.x == best.x && x.y > best.y)) best = x;
        }
        exact[c0 + tid] = best;
      }
      __syncthreads();
    }
  }
  // Many of them: the need-th's (score, rest, lower page) from the highest digit down, so that
  // their number counts once a digit and not squared: one row of 131,072 keys in pages of 8 with
  // 1024 picks and 8 heads of 128, all bounds equal, 1.7 ms (ranked against each other 8.9), q zero
  // 61 us (8700); 64 requests of 65,536 keys, 64 picks, all q zero, 96 us (1790), one page of 2048
  // with bounds of 1000 221 us (245), without it 85.
  unsigned last0 = 0, last1 = 0, last2 = 0;
  auto word = [&](int c, int w) { return w == 2 ? ~(unsigned)list[c] : flat ? 0u : ordered(w ? exact[c].y : exact[c].x); };
  if (many) {
    int left = need;                                        // of those that share the digits so far
    for (int pass = flat ? 8 : 0; pass < 12; ++pass) {
      const int w = pass / 4, shift = 24 - 8 * (pass % 4);
      const unsigned upto = w == 0 ? last0 : w == 1 ? last1 : last2;
      for (int i = tid; i < 256; i += kCThreads) s_hist[i] = 0;
      __syncthreads();
      for (int c0 = 0; c0 < s_count; c0 += kCThreads) {
        const int c = c0 + tid;
        unsigned digit = 256;                               // (of none)
        if (c < s_count && (w < 1 || word(c, 0) == last0) && (w < 2 || word(c, 1) == last1)) {
          const unsigned x = word(c, w);
          if ((x ^ upto) >> shift <= 255) digit = x >> shift & 255;
        }
        // (equal digits of a warp are one addition)
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        if (digit < 256 && lane == __ffs(same) - 1) atomicAdd(&s_hist[digit], __popc(same));
      }
      __syncthreads();
      const int n = tid < 256 ? s_hist[255 - tid] : 0;
      int all;
      const int before = block_scan<kCThreads>(n, s_warp, all);
      if (before < left && before + n >= left) {
        s_bin = 255 - tid;
        s_in = before;
        s_sure = before + n;
      }
      __syncthreads();
      const unsigned with = upto | (unsigned)s_bin << shift;
      if (w == 0) last0 = with;
      else if (w == 1) last1 = with;
      else last2 = with;
      const bool whole = s_sure == left;                    // all that share these digits are in
      left -= s_in;
      if (whole) break;
    }
  }
  // their ranks: -1 in place of the bound of a page that is picked, -2 of one that is not
  for (int c = tid; c < s_count; c += kCThreads) {
    const int j = list[c];
    bool pick;
    if (many) {
      const unsigned x = word(c, 0), y = word(c, 1);
      pick = x != last0 ? x > last0 : y != last1 ? y > last1 : word(c, 2) >= last2;
    } else {
      int better = 0;
      if (s_count > need) {
        const float2 e = flat ? make_float2(0.f, 0.f) : exact[c];
        for (int k = 0; k < s_count && better < need; ++k) {
          const float2 f = flat ? e : exact[k];
          better += f.x > e.x || (f.x == e.x && (f.y > e.y || (f.y == e.y && list[k] < j)));
        }
      }
      pick = better < need;
    }
    if (!masks) a[j].y = pick ? -1.f : -2.f;
    else if (pick) atomicOr(&s_mask[(j - lo) >> 5], 1u << ((j - lo) & 31));
  }
  __syncthreads();
  if (masks) {
    // ascending: the first pages, those of the masks, the last pages
    const int words = kHeld * NW;
    int n;
    const int before = block_scan<kCThreads>(tid < words ? __popc(s_mask[tid]) : 0, s_warp, n);
    s_hist[tid] = P.n_first + before;
    __syncthreads();
    for (int k = warp; k < words; k += NW) {
      const unsigned mask = s_mask[k];
      const int at = s_hist[k] + __popc(mask & ((1u << lane) - 1));
      if (mask >> lane & 1 && at < P.n_picks - P.n_last) out[at] = lo + k * 32 + lane;
    }
    // (scores that are not finite may leave places, or be too many)
    for (int i = P.n_first + n + tid; i < P.n_picks - P.n_last; i += kCThreads) out[i] = -1;
    for (int i = tid; i < P.n_first; i += kCThreads) out[i] = i;
    for (int i = tid; i < P.n_last; i += kCThreads) out[P.n_picks - P.n_last + i] = hi + i;
    return;
  }
  // ascending: a mask for every 32 pages, one scan over the masks of 32 kCThreads pages
  int written = 0;
  for (int j0 = 0; j0 < pages; j0 += 32 * kCThreads) {
    const int groups = min(kCThreads, (pages - j0 + 31) / 32);
    for (int k = warp; k < groups; k += NW) {
      const int j = j0 + k * 32 + lane;
      bool pick = j < pages && (j < lo || j >= hi);
      if (j >= lo && j < hi && want > 0) {
        const float2 x = a[j];
        pick = x.y < 0.f ? x.y == -1.f : x.x > sure;
      }
      const unsigned mask = __ballot_sync(0xffffffffu, pick);
      if (lane == 0) s_mask[k] = mask;
    }
    __syncthreads();
    int n;
    const int before = block_scan<kCThreads>(tid < groups ? __popc(s_mask[tid]) : 0, s_warp, n);
    s_hist[tid] = written + before;
    __syncthreads();
    for (int k = warp; k < groups; k += NW) {
      const unsigned mask = s_mask[k];
      const int at = s_hist[k] + __popc(mask & ((1u << lane) - 1));
      if (mask >> lane & 1 && at < P.n_picks) out[at] = j0 + k * 32 + lane;
    }
    written += n;
    __syncthreads();
  }
  for (int i = written + tid; i < P.n_picks; i += kCThreads) out[i] = -1;
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
  return (size_t)n_rows * Hkv * held_pages(max_kv, page_size) * (sizeof(float2) + sizeof(float2) + sizeof(int));
}

template <typename T, int HD>
static cudaError_t run_select(const pages::SelectParams &P, int *status, cudaStream_t s) {
  using namespace pages;
  int n = 0;
  if (P.scored) {
    cudaError_t e;
    if constexpr (std::is_same<T, bf16>::value) {
      constexpr int kSmem = kSThreads / 32 * kTStages * 16 * 2 * HD * 2;
      static PerDeviceOnce attr;
      e = attr.run([](int) {
        return cudaFuncSetAttribute(paged_score_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      });
      if (e == cudaSuccess)
        e = launch_pdl(paged_score_tc_kernel<HD>, dim3(device_sm_count()), dim3(kSThreads), kSmem, s, P, status);
    } else {
      e = launch_pdl(paged_score_kernel<HD>, dim3(P.parts * P.Hkv * P.n_rows), dim3(kSThreads), 0, s, P, status);
    }
    if (e != cudaSuccess) return e;
    ++n;
  }
  const dim3 grid(P.Hkv * P.n_rows);
  const cudaError_t e = P.held <= 256 * kHeld
      ? launch_pdl(paged_choose_kernel<T, HD, 256>, grid, dim3(256), 0, s, P, status)
      : launch_pdl(paged_choose_kernel<T, HD, 1024>, grid, dim3(1024), 0, s, P, status);
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
  P.by_heads = paged::Divisor(P.Hkv);
  P.scored = P.held > P.n_picks;
  P.approx = reinterpret_cast<float2 *>(a.ws);
  const size_t all = (size_t)b.n_rows * P.Hkv * P.held;
  P.exact = P.approx + all;
  P.list = reinterpret_cast<int *>(P.exact + all);
  P.parts = (P.held + pages::kSPages - 1) / pages::kSPages;
  if ((int64_t)P.parts * P.Hkv * b.n_rows > 0x7fffffffLL || (int64_t)P.Hkv * b.n_rows > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  if (dt == CB_BF16) return P.hd == 128 ? run_select<bf16, 128>(P, status, s) : run_select<bf16, 64>(P, status, s);
  return P.hd == 128 ? run_select<float, 128>(P, status, s) : run_select<float, 64>(P, status, s);
}

}  // namespace cb
