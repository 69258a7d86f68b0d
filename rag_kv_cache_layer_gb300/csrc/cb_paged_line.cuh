// The line of units that the few-rows attention kernels cut into equal parts, and
// the kernel that joins the pieces of an item that more than one part holds.
#pragma once

#include <type_traits>

#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"
#include "cb_paged_attn.cuh"
#include "cb_paged_few.cuh"
#include "cb_tc.cuh"

namespace cb {
namespace paged {

constexpr int kDecThreads = 128;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// 2^x, relative error about 2^-22, far below the rounding of P to bf16.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// ------------------------------------------------------------------ plan --
// The line of units.  A sequence's tiles are taken in pairs, one from its end
// and one from its start: a late tile sees many keys, an early one few, and
// the two together about the same in every pair, C units at most.  Pair q of a
// group of heads is C units: the late tile's blocks, then the early one's (the
// few units behind its last block are empty); behind the pairs comes an odd
// middle tile.  Counted one by one at the sequence's length, early tiles leave
// half of the parts idle (2000 rows from nothing in fp32, 4/2 heads of 64: 108
// us, 68 so; 201 rows over 1501 keys, where tiles differ little, 27.8 and 28.8).
struct Line {
  int64_t begin[CB_MAX_SEQS];     // first unit of each sequence
  int blocks[CB_MAX_SEQS];        // units per pair (C), or of the only tile; 0: nothing to do
  int64_t total;                  // units
  int parts;                      // blocks of the grid that take part
};

// Part c is [c total / parts, (c + 1) total / parts), each rounded down.  The
// products fit 32 bits in all but the longest calls, and 64-bit division is
// several times slower.
__device__ __forceinline__ int64_t part_begin(const Line &L, int c) {
  const int64_t x = L.total * c;
  return x >> 32 == 0 ? (uint32_t)x / (uint32_t)L.parts : x / L.parts;
}
__device__ __forceinline__ int part_of(const Line &L, int64_t u) {
  const int64_t x = (u + 1) * L.parts - 1;
  return x >> 32 == 0 ? (int)((uint32_t)x / (uint32_t)L.total) : (int)(x / L.total);
}
// a / b and a % b, in 32 bits where a fits (64-bit division is several times
// slower and on every piece's path).
__device__ __forceinline__ void divide(int64_t a, int b, int &quot, int &rem) {
  if (a >> 32 == 0) {
    quot = (int)((uint32_t)a / (uint32_t)b);
    rem = (int)((uint32_t)a % (uint32_t)b);
  } else {
    quot = (int)(a / b);
    rem = (int)(a % b);
  }
}

// Key blocks that row l of a sequence's tile sees, at least one (rows without
// keys get their zeros).
__device__ __forceinline__ int blocks_seen(const AttnParams &P, int base, int l, int BN) {
  const int seen = base + P.by_G.div(l) + 1;
  return seen > 0 ? (seen - 1) / BN + 1 : 1;
}

// Every thread of the block calls it; one round of loads, one block scan.
// pad: empty units behind each tile's blocks, for what a tile costs beyond them.
__device__ __forceinline__ void make_line(const AttnParams &P, int R, int BN, int grid, Line &L, int64_t *warp_sums,
                                          int *status, int pad = 0) {
  constexpr int NT = kDecThreads;
  const int per = (P.kv.n_seq + NT - 1) / NT, i0 = threadIdx.x * per, i1 = min(i0 + per, P.kv.n_seq);
  int64_t sum = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    const int n = paged_rows(P.kv, i, P.n_rows, status), len = __ldg(P.kv.kv_lens + i);
    int pair = 0, units = 0;                            // per group of heads
    const int tiles = (int)(((int64_t)n * P.G + R - 1) / R);
    if (n > 0 && (int64_t)n * P.G <= P.few_hi) {
      if (len < 0 || len > P.max_kv || len > (int64_t)P.kv.max_pages * P.kv.page_size)
        report(status, CB_ERR_DEVICE_INDEX);
      else if (tiles == 1)
        units = pair = blocks_seen(P, len - n, n * P.G - 1, BN) + pad;
      else {
        // each of a pair's two counts is within one of a linear function of
        // the tile, and those add up to the same in every pair
        pair = blocks_seen(P, len - n, R - 1, BN) + blocks_seen(P, len - n, tiles * R - 1, BN) + 2 + 2 * pad;
        units = tiles & 1 ? blocks_seen(P, len - n, (tiles / 2 + 1) * R - 1, BN) + pad : 0;
      }
    }
    L.blocks[i] = pair;
    L.begin[i] = sum;
    sum += ((int64_t)(tiles / 2) * pair + units) * P.by_quads.d;
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  int64_t first = incl - sum;
  for (int x = 0; x < w; ++x) first += warp_sums[x];
#pragma unroll 1
  for (int i = i0; i < i1; ++i) L.begin[i] += first;
  first += sum;
  if (threadIdx.x == NT - 1) {
    L.total = first;
    // a part has at least one unit, or one for each group that shares its head
    const int64_t most = P.hc > 1 ? first : (first + 3) / 4;
    L.parts = (int)(most < grid ? most : grid);
    // One sequence's pairs, where they are fewer than the parts, take the same
    // number of parts each, so that no part has two pieces of single tiles, which
    // costs it a second prologue and join (one row, 28/4 heads of 128: 10.0 us over
    // 1000 keys, 8.4 so; where no part had two anyway, the arithmetic costs 0.2 us).
    if (P.kv.n_seq == 1 && L.parts > 0) {
      int items, none;
      divide(first, L.blocks[0], items, none);
      if (items < L.parts) L.parts -= L.parts % items;
    }
  }
  __syncthreads();
}

// The sequence that holds unit u.
__device__ __forceinline__ int seq_of(const Line &L, int n_seq, int64_t u) {
  int lo = 0, hi = n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.begin[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;                      // the last one that begins at or before u
}

// Joins the pieces of the item whose first piece part blockIdx.x holds, four
// rows per block (blockIdx.y).  The weights are made once in shared memory, so the partial
// rows' loads depend on nothing: warp w takes every eighth piece, a lane HD /
// 32 columns, and the warps' sums meet in shared memory.
constexpr int kJoinThreads = 256, kJoinRows = 4;
template <typename T, int HD>
__global__ void __launch_bounds__(kJoinThreads)
decode_merge_kernel(const __grid_constant__ AttnParams P, int R) {
  constexpr int PER = HD / 32, NW = kJoinThreads / 32;
  extern __shared__ float2 s_ml[];              // [pieces][kJoinRows]: (m, l), then the weight in x
  __shared__ float s_o[NW][kJoinRows][HD];
  __shared__ float s_inv[kJoinRows];
  grid_dep_wait();
  grid_dep_launch();
  const Join J = P.joins[blockIdx.x];
  // rows r0 .. r0 + 3 of one of the item's heads
  const int hs = blockIdx.y * kJoinRows / R, r0 = blockIdx.y * kJoinRows % R;
  if (r0 >= J.rows) return;
  const int first = blockIdx.x, count = J.last - first + 1;
  // a later part's first slot; this part's first or second
  auto slot = [&](int c) { return ((2 * (int64_t)(first + c) + (c == 0 ? J.second : 0)) * P.hc + hs) * R; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < count * kJoinRows; i += kJoinThreads) {
    const int c = i / kJoinRows, r = r0 + i % kJoinRows;
    s_ml[i] = r < J.rows ? P.part_ml[slot(c) + r] : make_float2(-INFINITY, 0.f);
  }
  __syncthreads();
  if (warp < kJoinRows) {
    float M = -INFINITY, l = 0.f;
    for (int c = lane; c < count; c += 32) M = fmaxf(M, s_ml[c * kJoinRows + warp].x);
    M = warp_max(M);
    for (int c = lane; c < count; c += 32) {
      const float2 ml = s_ml[c * kJoinRows + warp];
      const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);   // no visible key in this piece
      s_ml[c * kJoinRows + warp].x = w;
      l += w * ml.y;
    }
    l = warp_sum(l);
    if (lane == 0) s_inv[warp] = l == 0.f ? 0.f : 1.f / l;
  }
  __syncthreads();
  float o[kJoinRows][PER];
#pragma unroll
  for (int k = 0; k < kJoinRows; ++k)
#pragma unroll
    for (int e = 0; e < PER; ++e) o[k][e] = 0.f;
#pragma unroll 4
  for (int c = warp; c < count; c += NW) {
    const float *src = P.part_o + (slot(c) + r0) * HD + lane * PER;
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
      const float w = s_ml[c * kJoinRows + k].x;
      if (r0 + k < J.rows) {
        float v[PER];
        if constexpr (PER == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(src + k * HD);
        else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(src + k * HD);
#pragma unroll
        for (int e = 0; e < PER; ++e) o[k][e] = fmaf(w, v[e], o[k][e]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kJoinRows; ++k)
#pragma unroll
    for (int e = 0; e < PER; ++e) s_o[warp][k][lane * PER + e] = o[k][e];
  __syncthreads();
  for (int i = threadIdx.x; i < kJoinRows * HD / 2; i += kJoinThreads) {
    const int k = i / (HD / 2), c = i % (HD / 2) * 2, l = J.l0 + r0 + k;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      a += s_o[w][k][c];
      b += s_o[w][k][c + 1];
    }
    if (r0 + k >= J.rows) continue;
    const int qi = P.by_G.div(l);
    T *dst = reinterpret_cast<T *>(P.out) + (int64_t)(J.row0 + qi) * P.ld_out +
             (int64_t)((J.g + hs) * P.G + l - qi * P.G) * HD + c;
    if constexpr (std::is_same<T, float>::value)
      *reinterpret_cast<float2 *>(dst) = make_float2(a * s_inv[k], b * s_inv[k]);
    else
      *reinterpret_cast<uint32_t *>(dst) = pack_bf16(a * s_inv[k], b * s_inv[k]);
  }
}

// Joins the parts (unnormalised O in `part` [rows][HD], (m, l) in `ml`, in shared memory) of
// the `ranks` blocks of a cluster, a power of two up to 16: block `rank` writes a share of
// the rows' columns, four at a time, by write(row, column, O, l).  A lane has one block's
// part of them, and neighbouring lanes add up in the order of a tree.  Every thread of the
// cluster's blocks (of NTH) calls it.
template <int NTH, int HD, typename F>
__device__ __forceinline__ void cluster_join(const float *part, const float2 *ml, int rows, int rank, int ranks,
                                             const F &write) {
  tcx::cluster_sync();
  const int all = rows * (HD / 4), per = (all + ranks - 1) / ranks, groups = NTH / ranks;
  const int from = threadIdx.x & (ranks - 1), k0 = threadIdx.x / ranks;
  for (int k = 0; k < per; k += groups) {
    const int i = rank * per + k + k0;
    const bool valid = k + k0 < per && i < all;
    const int r = valid ? i / (HD / 4) : 0, c = valid ? i % (HD / 4) * 4 : 0;
    float2 x;
    float4 a;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y)
                 : "r"(tcx::map_to_rank(smem_u32(ml + r), from)) : "memory");
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w)
                 : "r"(tcx::map_to_rank(smem_u32(part + r * HD + c), from)) : "memory");
    float M = x.x;
    for (int o = 1; o < ranks; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float w = x.x == -INFINITY ? 0.f : ex2(x.x - M);
    float L = w * x.y;
    a = make_float4(w * a.x, w * a.y, w * a.z, w * a.w);
    for (int o = 1; o < ranks; o <<= 1) {
      L += __shfl_xor_sync(0xffffffffu, L, o);
      a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
      a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
      a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
      a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
    }
    if (valid && from == 0) write(r, c, a, L);
  }
  tcx::cluster_sync();                          // no block leaves while its parts are read
}

}  // namespace paged
}  // namespace cb
