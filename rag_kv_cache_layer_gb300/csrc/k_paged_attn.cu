// Causal attention of every sequence's new rows over its paged cache on the
// CUDA cores, and the merge of split key ranges.
//
// A tile is R rows of one sequence and kv head (cb_paged.cuh), its keys the
// positions up to its last query.  For row l at position p:
//   o = sum_{j <= p} softmax_j(scale q . k_j) v_j
// computed 64 keys at a time with a running maximum m and sum l (log2
// domain): P = 2^(s - m), O = O 2^(m_old - m) + P V, all fp32.  A row with
// p < 0 sees no key and gets zeros.  Keys past the cached length are read as
// zeros whatever the pages hold, so nothing unwritten in a page reaches O.
//
// 256 threads: 16 row groups x 16 columns.  Each thread scores R / 16 rows x
// 4 keys and accumulates R / 16 rows x HD / 16 output columns.
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"
#include "cb_paged_attn.cuh"

namespace cb {
namespace paged {

constexpr int kSimtThreads = 256;
constexpr int kBN = 64;                   // keys per block

template <int R, int HD>
constexpr size_t simt_smem() {
  return sizeof(float) * ((size_t)(R + kBN) * (HD + 4) + (size_t)kBN * HD + (size_t)R * kBN);
}

template <int R, int HD>
__global__ void __launch_bounds__(kSimtThreads)
paged_simt_kernel(const __grid_constant__ AttnParams P, int *status) {
  typedef float T;
  constexpr int TM = R / 16, TD = HD / 64, VEC = 16 / sizeof(T), LD = HD + 4;
  extern __shared__ __align__(16) float sm[];
  float *sq = sm, *sk = sq + R * LD, *sv = sk + kBN * LD, *sp = sv + kBN * HD;
  __shared__ PagedTile s_tile;
  __shared__ int s_sums[kSimtThreads / 32];
  __shared__ int64_t s_off[kBN];          // element offset of each key's slot, -1: zeros
  grid_dep_wait();
  grid_dep_launch();
  const int split = blockIdx.x % P.n_split, g = blockIdx.x / P.n_split % P.Hkv;
  const int tile = blockIdx.x / P.n_split / P.Hkv;
  paged_find_tile<kSimtThreads>(P.kv, P.n_rows, P.G, R, P.max_kv, tile, &s_tile, s_sums, status);
  const PagedTile tl = s_tile;
  if (tl.s < 0) return;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int l0 = tl.t * R, rows = min(R, tl.n * P.G - l0);
  const int base = tl.kv - tl.n;          // position of the sequence's first new row
  const int last = base + (l0 + rows - 1) / P.G;
  const int nb = last < 0 ? 0 : last / kBN + 1;
  const int jb = (int)((int64_t)nb * split / P.n_split);
  const int je = (int)((int64_t)nb * (split + 1) / P.n_split);

  const T *q = reinterpret_cast<const T *>(P.q);
  for (int i = tid; i < R * (HD / VEC); i += kSimtThreads) {
    const int l = i / (HD / VEC), c = i % (HD / VEC) * VEC;
    float x[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = 0.f;
    if (l < rows) {
      const int qi = (l0 + l) / P.G, h = (l0 + l) % P.G;
      load16<T>(q + (int64_t)(tl.row0 + qi) * P.ld_q + (int64_t)(g * P.G + h) * HD + c, x);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) sq[l * LD + c + e] = x[e] * P.scale_log2;
  }
  float m[TM], l[TM], o[TM][TD * 4];
  int pos[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    pos[i] = base + (l0 + ty + 16 * i) / P.G;
#pragma unroll
    for (int d = 0; d < TD * 4; ++d) o[i][d] = 0.f;
  }
  const T *kp = reinterpret_cast<const T *>(P.kv.k_pages) + (int64_t)g * HD;
  const T *vp = reinterpret_cast<const T *>(P.kv.v_pages) + (int64_t)g * HD;
  for (int j = jb; j < je; ++j) {
    const int key0 = j * kBN;
    __syncthreads();                      // the last block's K, V and P are used up
    if (tid < kBN) {
      const int key = key0 + tid;
      int64_t off = -1;
      if (key < tl.kv) {
        const int page = paged_page(P.kv, tl.s, key / P.kv.page_size, status);
        if (page >= 0)
          off = (int64_t)page * P.kv.page_stride + (int64_t)(key % P.kv.page_size) * P.kv.ld;
      }
      s_off[tid] = off;
    }
    __syncthreads();
    for (int i = tid; i < kBN * (HD / VEC); i += kSimtThreads) {
      const int r = i / (HD / VEC), c = i % (HD / VEC) * VEC;
      float a[VEC], b[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) a[e] = b[e] = 0.f;
      if (s_off[r] >= 0) {
        load16<T>(kp + s_off[r] + c, a);
        load16<T>(vp + s_off[r] + c, b);
      }
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        *reinterpret_cast<float4 *>(sk + r * LD + c + e) = make_float4(a[e], a[e + 1], a[e + 2], a[e + 3]);
        *reinterpret_cast<float4 *>(sv + r * HD + c + e) = make_float4(b[e], b[e + 1], b[e + 2], b[e + 3]);
      }
    }
    __syncthreads();
    float x[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i][k] = 0.f;
#pragma unroll 4
    for (int d = 0; d < HD; d += 4) {
      float4 a[TM], b[4];
#pragma unroll
      for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const float4 *>(sq + (ty + 16 * i) * LD + d);
#pragma unroll
      for (int k = 0; k < 4; ++k) b[k] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * k) * LD + d);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[i][k] = fmaf(a[i].x, b[k].x, x[i][k]);
          x[i][k] = fmaf(a[i].y, b[k].y, x[i][k]);
          x[i][k] = fmaf(a[i].z, b[k].z, x[i][k]);
          x[i][k] = fmaf(a[i].w, b[k].w, x[i][k]);
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (key0 + tx + 16 * k > pos[i]) x[i][k] = -INFINITY;
        mx = fmaxf(mx, x[i][k]);
      }
#pragma unroll
      for (int s = 8; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      const float mn = fmaxf(m[i], mx);
      // no visible key yet: nothing to scale, every probability is zero
      const float corr = mn == -INFINITY ? 1.f : exp2f(m[i] - mn);
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float p = x[i][k] == -INFINITY ? 0.f : exp2f(x[i][k] - mn);
        sum += p;
        sp[(ty + 16 * i) * kBN + tx + 16 * k] = p;
      }
#pragma unroll
      for (int s = 8; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
      m[i] = mn;
      l[i] = l[i] * corr + sum;
#pragma unroll
      for (int d = 0; d < TD * 4; ++d) o[i][d] *= corr;
    }
    __syncwarp();                         // a row's 16 threads are one half-warp
#pragma unroll 4
    for (int k = 0; k < kBN; ++k) {
      float4 b[TD];
#pragma unroll
      for (int d = 0; d < TD; ++d) b[d] = *reinterpret_cast<const float4 *>(sv + k * HD + d * 64 + tx * 4);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const float p = sp[(ty + 16 * i) * kBN + k];
#pragma unroll
        for (int d = 0; d < TD; ++d) {
          o[i][4 * d] = fmaf(p, b[d].x, o[i][4 * d]);
          o[i][4 * d + 1] = fmaf(p, b[d].y, o[i][4 * d + 1]);
          o[i][4 * d + 2] = fmaf(p, b[d].z, o[i][4 * d + 2]);
          o[i][4 * d + 3] = fmaf(p, b[d].w, o[i][4 * d + 3]);
        }
      }
    }
  }
  const int64_t slot = ((int64_t)(tile * P.Hkv + g) * P.n_split + split) * R;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = ty + 16 * i;
    if (r >= rows) continue;
    if (P.n_split > 1) {
#pragma unroll
      for (int d = 0; d < TD; ++d)
        *reinterpret_cast<float4 *>(P.part_o + (slot + r) * HD + d * 64 + tx * 4) =
            make_float4(o[i][4 * d], o[i][4 * d + 1], o[i][4 * d + 2], o[i][4 * d + 3]);
      if (tx == 0) P.part_ml[slot + r] = make_float2(m[i], l[i]);
      continue;
    }
    const int qi = (l0 + r) / P.G, h = (l0 + r) % P.G;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    T *dst = reinterpret_cast<T *>(P.out) + (int64_t)(tl.row0 + qi) * P.ld_out +
             (int64_t)(g * P.G + h) * HD;
#pragma unroll
    for (int d = 0; d < TD; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[d * 64 + tx * 4 + e] = from_f<T>(o[i][4 * d + e] * inv);
  }
}

// Merges the partials of a tile's key ranges: with M = max m_c,
// O = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c, in split order.  A block
// takes eight rows of a tile, a warp a row, each lane HD / 32 columns: the
// merge is a latency of three dependent reads, so it runs as wide as it can.
constexpr int kMergeThreads = 256, kMergeRows = kMergeThreads / 32;
template <int HD>
__global__ void __launch_bounds__(kMergeThreads)
paged_merge_kernel(const __grid_constant__ AttnParams P, int R) {
  constexpr int PER = HD / 32;
  __shared__ PagedTile s_tile;
  __shared__ int s_sums[kMergeThreads / 32];
  const int slices = R / kMergeRows, slice = blockIdx.x % slices;
  const int g = blockIdx.x / slices % P.Hkv, tile = blockIdx.x / slices / P.Hkv;
  paged_find_tile<kMergeThreads>(P.kv, P.n_rows, P.G, R, P.max_kv, tile, &s_tile, s_sums, nullptr);
  grid_dep_wait();                        // the tile's metadata was there before the partials' kernel began
  grid_dep_launch();
  const PagedTile tl = s_tile;
  if (tl.s < 0) return;
  const int lane = threadIdx.x & 31, r = slice * kMergeRows + (threadIdx.x >> 5);
  const int l0 = tl.t * R, rows = min(R, tl.n * P.G - l0);
  if (r >= rows) return;
  const int64_t row0 = (int64_t)(tile * P.Hkv + g) * P.n_split * R + r;
  // lane c holds part c's (m, l); parts beyond 32 are met in further rounds
  float M = -INFINITY;
  for (int c = lane; c < P.n_split; c += 32) M = fmaxf(M, P.part_ml[row0 + (int64_t)c * R].x);
  M = warp_max(M);
  float l = 0.f, o[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
  for (int c0 = 0; c0 < P.n_split; c0 += 32) {
    float w = 0.f;
    if (c0 + lane < P.n_split) {
      const float2 ml = P.part_ml[row0 + (int64_t)(c0 + lane) * R];
      w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);      // no visible key in this range
      l += w * ml.y;
    }
    const int n = min(32, P.n_split - c0);
#pragma unroll 8
    for (int c = 0; c < n; ++c) {
      const float wc = __shfl_sync(0xffffffffu, w, c);
      if (wc == 0.f) continue;                            // its row may not have been written
      const float *src = P.part_o + (row0 + (int64_t)(c0 + c) * R) * HD + lane * PER;
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] = fmaf(wc, src[e], o[e]);
    }
  }
  l = warp_sum(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float *dst = reinterpret_cast<float *>(P.out) + (int64_t)(tl.row0 + (l0 + r) / P.G) * P.ld_out +
               (int64_t)(g * P.G + (l0 + r) % P.G) * HD + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; ++e) dst[e] = o[e] * inv;
}

// Tiles of R rows that n_rows rows over S sequences can make at most.
static int64_t tile_bound(int64_t n_rows, int S, int G, int R) {
  const int64_t a = (n_rows * G + (int64_t)S * (R - 1)) / R;
  const int64_t b = n_rows * ((G + R - 1) / R);
  return a < b ? a : b;
}

// How a call runs.
struct Plan {
  int few_R;                              // bf16, few rows: rows per tile, 0: none
  int R;                                  // chunk (128, 256) or fp32 tiles (16, 64): rows, 0: none
  int few_hi, rows_lo;                    // which sequences each takes
  int64_t tiles;                          // R-row tiles at most
  int n_split;                            // parts of their key ranges
  int64_t few_partials, partials;         // partial rows in the workspace (reused)
};

// Rows per unit and parts of the key ranges of the chunk kernel: the cheapest
// by a model of its time, in microseconds, measured on four chunks of 2048
// rows over 8192 keys, 512 rows over 4000 and 64 over 3200.  A part of 256
// rows (one CTA per SM) costs 7.5 and each of its 64-key blocks 0.93, one of
// 128 rows 5 and 1.04 (two CTAs on the SM) or 0.85 (alone on it); parts run in waves of CTA slots, and partials (written
// and read once, about 8 MB per microsecond) and their merge come on top.
// Large work takes 256 rows unsplit; a few tiles over many keys are split
// until the SMs are full; and where the last of few waves would be nearly
// empty, splitting evens it out (192 units of 30,000 keys, head_dim 64: 780
// unsplit, 476 in three parts each).
static void plan_chunk(Plan &p, int64_t n_rows, int S, int max_kv, int G, int Hkv, int hd) {
  const int sms = device_sm_count(), nb = (max_kv + 63) / 64 > 0 ? (max_kv + 63) / 64 : 1;
  double best = 1e300;
  for (int R = 128; R <= 256; R += 128) {
    const int64_t tiles = tile_bound(n_rows, S, G, R), units = tiles * Hkv;
    for (int n = 1; n <= 32 && (n == 1 || 2 * n <= nb); ++n) {
      const bool alone = R == 256 || units * n <= sms;
      const int64_t slots = alone ? sms : 2LL * sms;
      const double block = R == 256 ? 0.93 : alone ? 0.85 : 1.04;
      double t = (double)((units * n + slots - 1) / slots) * ((double)nb / n * block + (R == 256 ? 7.5 : 5.0));
      if (n > 1) t += 5.0 + (double)units * n * R * hd * 8 / 8e6;
      if (t < best) {
        best = t;
        p.R = R;
        p.tiles = tiles;
        p.n_split = n;
      }
    }
  }
}

// bf16: sequences of up to 64 rows (queries x G) go through the few-rows
// kernel, longer ones through the chunk kernel.  Both are launched when the
// sizes leave it open; a call whose rows do not exceed its sequences is taken
// for one generated token each and runs the few-rows kernel alone (which
// takes any number of rows), a single sequence runs the one its rows call
// for.  The few-rows tile is 16, 32 or 64 rows by the average sequence.
// fp32: 16-row tiles where a sequence brings few rows (the wider tile would
// mostly multiply zeros), else 64; key ranges are split while the tiles alone
// leave SMs idle, in parts of at least 128 keys.
static Plan plan(int64_t n_rows, int S, int max_kv, int G, int Hkv, int hd, cb_dtype dt) {
  Plan p = {};
  const int64_t all = n_rows * G, per_seq = (all + S - 1) / S;
  p.few_hi = 0x7fffffff;
  p.n_split = 1;
  if (dt == CB_BF16) {
    const bool few = all <= 64 || n_rows <= S;
    if (few || S > 1) p.few_R = per_seq <= 16 || per_seq > 64 ? 16 : per_seq <= 32 ? 32 : 64;
    p.few_partials = p.few_R ? 2LL * decode_grid() * p.few_R : 0;
    if (few) return p;
    if (S > 1) p.few_hi = p.rows_lo = 64;
    plan_chunk(p, n_rows, S, max_kv, G, Hkv, hd);
  } else {
    p.R = per_seq <= 16 ? 16 : 64;
    p.tiles = tile_bound(n_rows, S, G, p.R);
    const int64_t units = p.tiles * Hkv > 0 ? p.tiles * Hkv : 1;
    const int64_t want = 4LL * device_sm_count() / units, most = (max_kv + 127) / 128;
    const int64_t n = want < most ? want : most;
    p.n_split = n < 1 ? 1 : n > 64 ? 64 : (int)n;
  }
  p.partials = p.n_split == 1 ? 0 : p.tiles * Hkv * p.n_split * p.R;
  return p;
}

static size_t plan_bytes(const Plan &p, int hd) {
  const size_t row = hd * sizeof(float) + sizeof(float2);
  const size_t few = (size_t)p.few_partials * row + (p.few_R ? decode_grid() * sizeof(Join) : 0);
  const size_t rest = (size_t)p.partials * row;
  return few > rest ? few : rest;
}

template <int R, int HD>
static cudaError_t run_simt(const AttnParams &P, const Plan &p, int *status, cudaStream_t s) {
  static PerDeviceOnce attr;
  cudaError_t e = attr.run([](int) {
    return cudaFuncSetAttribute(paged_simt_kernel<R, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)simt_smem<R, HD>());
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_simt_kernel<R, HD>, dim3((unsigned)(p.tiles * P.Hkv * P.n_split)),
                 dim3(kSimtThreads), simt_smem<R, HD>(), s, P, status);
  return e == cudaSuccess ? launched(1) : e;
}

// The partials of a launch reuse the workspace of the launch before it: each
// waits for its predecessor's end, and a merge has read them by then.
template <int HD>
static cudaError_t run_all(AttnParams P, const Plan &p, cb_dtype dt, void *ws, int *status, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  auto bind = [&](int64_t partials) {
    P.part_o = reinterpret_cast<float *>(ws);
    P.part_ml = reinterpret_cast<float2 *>(P.part_o + (size_t)partials * HD);
    P.joins = reinterpret_cast<Join *>(P.part_ml + partials);
  };
  if (p.few_R) {
    bind(p.few_partials);
    e = launch_decode(P, p.few_R, HD, status, s);
    if (e != cudaSuccess) return e;
  }
  if (!p.R) return e;
  bind(p.partials);
  if (dt == CB_BF16) return launch_chunk(P, p.R, p.tiles, HD, status, s);
  e = p.R == 16 ? run_simt<16, HD>(P, p, status, s) : run_simt<64, HD>(P, p, status, s);
  if (e != cudaSuccess || p.n_split == 1) return e;
  const dim3 grid((unsigned)(p.tiles * P.Hkv * (p.R / kMergeRows)));
  e = launch_pdl(paged_merge_kernel<HD>, grid, dim3(kMergeThreads), 0, s, P, p.R);
  return e == cudaSuccess ? launched(1) : e;
}

}  // namespace paged

size_t paged_attention_ws_bytes(int n_rows, int n_seq, int max_kv, int Hq, int Hkv, int hd, cb_dtype dt) {
  using namespace paged;
  if (n_rows <= 0 || n_seq <= 0) return 0;
  return plan_bytes(plan(n_rows, n_seq, max_kv, Hq / Hkv, Hkv, hd, dt), hd);
}

cudaError_t launch_paged_attention(const PagedKV &kv, const void *q, int64_t ld_q, int n_rows, int max_kv,
                                   int Hq, int Hkv, int hd, float scale, void *out, int64_t ld_out,
                                   cb_dtype dt, void *ws, int *status, cudaStream_t s) {
  using namespace paged;
  if (n_rows == 0 || kv.n_seq == 0) return cudaSuccess;
  const Plan p = plan(n_rows, kv.n_seq, max_kv, Hq / Hkv, Hkv, hd, dt);
  if (p.tiles * Hkv * p.n_split > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  AttnParams P;
  P.kv = kv;
  P.q = q;
  P.out = out;
  P.ld_q = ld_q;
  P.ld_out = ld_out;
  P.n_rows = n_rows;
  P.G = Hq / Hkv;
  P.Hkv = Hkv;
  P.max_kv = max_kv;
  P.n_split = p.n_split;
  P.few_hi = p.few_hi;
  P.rows_lo = p.rows_lo;
  P.scale_log2 = scale * 1.4426950408889634f;
  return hd == 128 ? run_all<128>(P, p, dt, ws, status, s) : run_all<64>(P, p, dt, ws, status, s);
}

}  // namespace cb
