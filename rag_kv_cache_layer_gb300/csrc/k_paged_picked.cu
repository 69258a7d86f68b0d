// Attention over picked pages: every row and kv head has a list of its own.
//
// An item is 16 q heads (a tile of the group) of one row and kv head; its keys are
// its list's pages one after the other, in blocks of BN.  All items count as many
// blocks as the longest list can have, and that line of units is cut into equal parts
// for the grid's blocks (two per SM); an item inside a part is written out, one that
// crosses parts leaves its pieces for decode_merge_kernel (cb_paged_line.cuh).  Few items
// take a cluster each, blocks of eight warps, and join in its shared memory (one row over
// 128 pages of 16: 9.0 us, on the line 12.1).  Nothing is loaded behind a list's last page
// (27 requests with 35 pages of 32 each and room for 128: 34 us, 87 with zeros for the rest).
//
// A block first turns its part of the list into pages of the pool and the number of
// slots that the row sees in each (two dependent rounds of loads for all of them, not
// two on every key block's path); from then on the keys stream as in
// paged_decode_kernel: four warps with a cp.async ring each take the key blocks in
// turn and hold the 16 rows' maximum, sum and O in registers.  The products and the fp32
// steps are those of that kernel, but P meets the values as two halves of bf16 (16 bits in
// place of 8): a group of up to 8 heads leaves the instruction's other 8 rows for the second
// half, at no cost (one half 95.1 us, two 92.7; in products of their own 100.5, as larger
// groups have them).  Bound by the picked pages' bytes: 64 requests with 64 pages of 32
// each, 32/8 heads of 128, take 93 us, 5.8 TB/s of 538 MB in slices of 256 bytes.
#include <type_traits>

#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"
#include "cb_paged_attn.cuh"
#include "cb_paged_few.cuh"
#include "cb_paged_line.cuh"
#include "cb_tc.cuh"

namespace cb {
namespace picked {

using namespace paged;

struct Params : AttnParams {
  const int32_t *picks;
  int n_picks, blocks, tiles;           // list length; units per item; 16-row tiles of a group
  int64_t units;
  int parts;
};

constexpr int kBlocksPerSm = 2;

// CL: an item's keys in one cluster, eight warps a block.
template <bool CL> struct Form {
  static constexpr int kWarps = CL ? 8 : 4, kThreads = 32 * kWarps, kPerSm = CL ? 1 : kBlocksPerSm;
};

__device__ __forceinline__ int64_t begin_of(const Params &P, int c) { return P.units * c / P.parts; }
__device__ __forceinline__ int part_of(const Params &P, int64_t u) { return (int)(((u + 1) * P.parts - 1) / P.units); }

// HALF (bf16, groups of up to 8 heads): rows 8 to 15 of the instruction's 16, which have no head,
// take what P's rounding to bf16 leaves of rows 0 to 7.
template <typename T, int HD, bool CL, bool HALF>
__global__ void __launch_bounds__(Form<CL>::kThreads, Form<CL>::kPerSm)
paged_picked_kernel(const __grid_constant__ Params P, int *status) {
  constexpr int NW = Form<CL>::kWarps, NTH = Form<CL>::kThreads;
  typedef DecCfg<T, HD, 1> C;
  constexpr bool F32 = std::is_same<T, float>::value;
  constexpr int R = 16, ND = HD / 8, KS = F32 ? HD / 8 : HD / 16, BN = C::kBN, NS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int s_page[CB_MAX_PICKS], s_vis[CB_MAX_PICKS];   // page of the pool, slots that the row sees
  __shared__ float2 s_ml[NW * R];
  __shared__ int s_seq, s_last;                 // s_last: picks up to the last one with a slot that the row sees
  // CL: the block's joined rows, read by the cluster's others
  __shared__ __align__(16) float s_part[CL ? R * HD : 4];
  __shared__ float2 s_pml[CL ? R : 1];
  grid_dep_wait();
  grid_dep_launch();
  // CL: block `rank` of an item's cluster; the line's units are not used
  const int ranks = CL ? tcx::cluster_size() : 1, rank = CL ? (int)(blockIdx.x % ranks) : 0;
  const int64_t u0 = CL ? 0 : begin_of(P, blockIdx.x), u1 = CL ? 1 : begin_of(P, blockIdx.x + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, q4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * NS * C::kStage;
  const int page_size = P.kv.page_size, shift = __ffs(page_size) - 1;
  const T *kp = reinterpret_cast<const T *>(P.kv.k_pages), *vp = reinterpret_cast<const T *>(P.kv.v_pages);
  constexpr int kVec = 16 / sizeof(T), kCols = HD / kVec, kRows = 32 / kCols;
  const int crow = lane / kCols, ccol = lane % kCols;
  const int krow = lane & 7, kcol = lane >> 3, vrow = lane & 15, vcol = lane >> 4;
  const float sl2 = P.scale_log2;
  if (!CL && threadIdx.x == 0) P.joins[blockIdx.x].rows = 0;

  int at_r = -1, s = 0;                         // row at_r: its sequence (0x7fffffff: none), position
  int64_t pos = 0;
  if (threadIdx.x == 0) s_last = 0;
  for (int64_t u = u0; u < u1;) {
    const int64_t item = CL ? blockIdx.x / ranks : u / P.blocks;
    int jb = CL ? 0 : (int)(u - item * P.blocks), je = CL ? P.blocks : (int)min((int64_t)P.blocks, jb + (u1 - u));
    const bool whole = CL || je - jb == P.blocks, first = u == u0;
    const int tile = (int)(item % P.tiles), g = (int)(item / P.tiles % P.Hkv), r = (int)(item / P.tiles / P.Hkv);
    const int l0 = tile * R, rows = min(R, P.G - l0);
    u = CL ? u1 : u + (je - jb);
    // the row's sequence and position (kept for the row's next head); the part's picks,
    // while the sequence is found
    const bool fresh = r != at_r;
    if (fresh) {
      if (threadIdx.x == 0) s_seq = 0x7fffffff;
      __syncthreads();
      for (int i = threadIdx.x; i < P.kv.n_seq; i += NTH) {
        const int a = __ldg(P.kv.row_offsets + i), b = __ldg(P.kv.row_offsets + i + 1);
        if (a < 0 || b < a || b > P.n_rows) report(status, CB_ERR_DEVICE_INDEX);
        else if (a <= r && r < b) atomicMin(&s_seq, i);
      }
    }
    const int p0 = jb * BN >> shift, p1 = min(P.n_picks, (je * BN + page_size - 1) >> shift);
    const int32_t *list = P.picks + ((int64_t)r * P.Hkv + g) * P.n_picks;
    for (int i = p0 + threadIdx.x; i < p1; i += NTH) s_page[i] = __ldg(list + i);
    if (fresh) {
      __syncthreads();
      at_r = r;
      s = s_seq;
      if (s != 0x7fffffff) {
        const int kv = __ldg(P.kv.kv_lens + s);
        pos = (int64_t)kv - __ldg(P.kv.row_offsets + s + 1) + r;
        if (kv < 0 || kv > (int64_t)P.kv.max_pages * page_size) {
          report(status, CB_ERR_DEVICE_INDEX);
          s = 0x7fffffff;
        }
      }
    }
    if (s == 0x7fffffff) {                      // a row of no sequence is left alone
      __syncthreads();
      continue;
    }
    const int32_t *table = P.kv.block_table + (int64_t)s * P.kv.ld_table;
    int last = 0;
    for (int i = p0 + threadIdx.x; i < p1; i += NTH) {
      const int j = s_page[i];
      int page = -1, vis = 0;
      if (j < -1 || j >= P.kv.max_pages) {
        report(status, CB_ERR_DEVICE_INDEX);
      } else if (j >= 0) {
        const int64_t left = pos - ((int64_t)j << shift) + 1;
        if (left > 0) {
          page = __ldg(table + j);
          vis = (int)min((int64_t)page_size, left);
          if (page < 0 || page >= P.kv.n_pages) {
            report(status, CB_ERR_DEVICE_INDEX);
            page = -1;
            vis = 0;
          }
        }
      }
      s_page[i] = page;
      s_vis[i] = vis;
      if (vis > 0) last = i + 1;
    }
    if (last > 0) atomicMax(&s_last, last);
    if (!CL && threadIdx.x == 0 && u == u1 && jb == 0 && !whole)     // the last piece: the one that goes on in the next part
      P.joins[blockIdx.x] = Join{r, l0, rows, g, part_of(P, (item + 1) * P.blocks - 1), first ? 0 : 1};
    __syncthreads();
    // nothing is streamed behind the list's last page (short contexts leave lists half
    // empty); a cluster shares what is in front of it
    const int full = (int)min((int64_t)je, (((int64_t)s_last << shift) + BN - 1) / BN);
    if constexpr (CL) {
      jb = (int)((int64_t)full * rank / ranks);
      je = (int)((int64_t)full * (rank + 1) / ranks);
    }
    const int end = CL ? je : max(full, jb);

    const int64_t lane_off = g * HD + ccol * kVec;
    // slots that the row sees of key block j * BN + x's page, from that key on (<= 0: none)
    auto load = [&](int j, int st) {
      const uint32_t dst = ring + st * C::kStage;
#pragma unroll
      for (int i = 0; i < BN / kRows; ++i) {
        const int x = i * kRows + crow, key = j * BN + x, pick = key >> shift, slot = key & (page_size - 1);
        const bool there = pick < P.n_picks && slot < s_vis[pick];
        const int64_t from = there ? s_page[pick] * P.kv.page_stride + slot * P.kv.ld + lane_off : 0;
        const uint32_t d = dst + x * C::kRow, sw = F32 ? ((x >> 1) & 3) << 1 : x & 7;
        copy16(d + ((ccol ^ (x & 7)) << 4), kp + from, there);
        copy16(d + C::kTile + ((ccol ^ sw) << 4), vp + from, there);
      }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i) {
      const int j = jb + warp + NW * i;
      if (j < end) load(j, i);
      commit();
    }
    uint32_t qf[KS][4];                         // bf16 pairs, or fp32 values
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int x = gid + 8 * h;
      const T *src = reinterpret_cast<const T *>(P.q) + (int64_t)r * P.ld_q + (int64_t)(g * P.G + l0 + x) * HD +
                     (F32 ? q4 : q4 * 2);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          qf[k][h + 2 * c] =
              x < rows ? *reinterpret_cast<const uint32_t *>(src + (F32 ? k * 8 + c * 4 : k * 16 + c * 8)) : 0u;
    }
    float o[ND][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    int st = 0, fill = NS - 1;
    for (int j = jb + warp; j < end; j += NW) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
      __syncwarp();                             // landed for every lane; the stage before is used up
      if (j + NW * (NS - 1) < end) load(j + NW * (NS - 1), fill);
      commit();
      fill = fill + 1 == NS ? 0 : fill + 1;
      const uint32_t ks = ring + st * C::kStage, vs = ks + C::kTile;
      st = st + 1 == NS ? 0 : st + 1;
      float x[BN / 8][4];
#pragma unroll
      for (int t = 0; t < BN / 8; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[t][k] = 0.f;
      const uint32_t krows = ks + krow * C::kRow;
      if constexpr (F32) {
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2) {
          uint32_t b[BN / 8][4];
#pragma unroll
          for (int t = 0; t < BN / 8; ++t) ldsm_x4(krows + t * 8 * C::kRow + (((k2 * 4 + kcol) ^ krow) << 4), b[t]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) halves(__uint_as_float(qf[2 * k2 + c][e]), ah[e], al[e]);
#pragma unroll
            for (int t = 0; t < BN / 8; ++t)
              step_f32(x[t], ah, al, __uint_as_float(b[t][2 * c]), __uint_as_float(b[t][2 * c + 1]));
          }
        }
      } else {
#pragma unroll
        for (int t = 0; t < BN / 8; ++t)
#pragma unroll
          for (int k2 = 0; k2 < KS / 2; ++k2) {
            uint32_t b[4];
            ldsm_x4(krows + t * 8 * C::kRow + (((k2 * 4 + kcol) ^ krow) << 4), b);
            mma16816(x[t], qf[2 * k2], b[0], b[1]);
            mma16816(x[t], qf[2 * k2 + 1], b[2], b[3]);
          }
      }
      float mx = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int t = 0; t < BN / 8; ++t) {
        // eight keys lie in one page (page_size >= 8)
        const int key = j * BN + t * 8, pick = key >> shift;
        const int vis = pick < P.n_picks ? s_vis[pick] - (key & (page_size - 1)) : 0;
#pragma unroll
        for (int k = 0; k < (HALF ? 2 : 4); ++k) x[t][k] = q4 * 2 + (k & 1) < vis ? x[t][k] * sl2 : -INFINITY;
        mx = fmaxf(mx, fmaxf(x[t][0], x[t][1]));
        if constexpr (!HALF) mx1 = fmaxf(mx1, fmaxf(x[t][2], x[t][3]));
      }
      float mxs[2] = {mx, mx1}, corr[2];
      bool moved = false;
#pragma unroll
      for (int h = 0; h < (HALF ? 1 : 2); ++h) {
        mxs[h] = fmaxf(mxs[h], __shfl_xor_sync(0xffffffffu, mxs[h], 1));
        mxs[h] = fmaxf(mxs[h], __shfl_xor_sync(0xffffffffu, mxs[h], 2));
        const float mn = fmaxf(m[h], mxs[h]);
        corr[h] = mn == m[h] ? 1.f : ex2(m[h] - mn);          // also where both are -inf
        moved |= mn != m[h];
        m[h] = mn;
        l[h] *= corr[h];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[d][k] *= corr[HALF ? 0 : k >> 1];
      }
#pragma unroll
      for (int t = 0; t < BN / 8; ++t)
#pragma unroll
        for (int k = 0; k < (HALF ? 2 : 4); ++k) {
          const float p = x[t][k] == -INFINITY ? 0.f : ex2(x[t][k] - m[k >> 1]);
          x[t][k] = p;
          l[k >> 1] += p;
        }
      if constexpr (F32) {
        // a step takes the keys of a tile in the order 0 2 4 6 1 3 5 7, in which the
        // scores' registers already are its operand
#pragma unroll
        for (int t = 0; t < BN / 8; ++t) {
          uint32_t ah[4], al[4];
          halves(x[t][0], ah[0], al[0]);
          halves(x[t][2], ah[1], al[1]);
          halves(x[t][1], ah[2], al[2]);
          halves(x[t][3], ah[3], al[3]);
          const uint32_t row = vs + (t * 8 + 2 * q4) * C::kRow;
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const uint32_t at = row + (((d * 2 + (gid >> 2)) ^ (q4 << 1)) << 4) + (gid & 3) * 4;
            float b0, b1;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(b0) : "r"(at) : "memory");
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(b1) : "r"(at + C::kRow) : "memory");
            step_f32(o[d], ah, al, b0, b1);
          }
        }
      } else {
#pragma unroll
        for (int k2 = 0; k2 < BN / 16; ++k2) {
          // rows gid and gid + 8 of the keys 0..7, then of 8..15; P as two halves of bf16, so that it
          // keeps 16 bits
          uint32_t a[4], rest[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (HALF && (i & 1)) continue;
            const float p0 = x[2 * k2 + (i >> 1)][2 * (i & 1)], p1 = x[2 * k2 + (i >> 1)][2 * (i & 1) + 1];
            a[i] = pack_bf16(p0, p1);
            rest[i] = pack_bf16(p0 - __uint_as_float(a[i] << 16), p1 - __uint_as_float(a[i] & 0xffff0000u));
            if (HALF) a[i + 1] = rest[i];
          }
          const uint32_t row = vs + (k2 * 16 + vrow) * C::kRow;
#pragma unroll
          for (int d2 = 0; d2 < ND / 2; ++d2) {
            uint32_t b[4];
            ldsm_x4_t(row + (((d2 * 2 + vcol) ^ (vrow & 7)) << 4), b);
            if constexpr (!HALF) {
              mma16816(o[2 * d2], rest, b[0], b[1]);
              mma16816(o[2 * d2 + 1], rest, b[2], b[3]);
            }
            mma16816(o[2 * d2], a, b[0], b[1]);
            mma16816(o[2 * d2 + 1], a, b[2], b[3]);
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (q4 == 0) s_ml[warp * R + gid + 8 * h] = make_float2(m[h], l[h]);
    }
    __syncthreads();                            // the rings are used up
    if (threadIdx.x == 0) s_last = 0;           // (for the next piece)
    constexpr int LD = HD + 4;
    static_assert(R * LD * 4 <= NS * C::kStage, "the warps' O fit the rings");
    float *so = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int h = 0; h < (HALF ? 1 : 2); ++h)
        *reinterpret_cast<float2 *>(so + (warp * R + gid + 8 * h) * LD + d * 8 + q4 * 2) =
            HALF ? make_float2(o[d][0] + o[d][2], o[d][1] + o[d][3]) : make_float2(o[d][2 * h], o[d][2 * h + 1]);
    __syncthreads();
    const int64_t slot = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * R;
    auto write = [&](int x, int c, float4 a, float L) {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      T *dst = reinterpret_cast<T *>(P.out) + (int64_t)r * P.ld_out + (int64_t)(g * P.G + l0 + x) * HD + c;
      if constexpr (F32)
        *reinterpret_cast<float4 *>(dst) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
      else
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
    };
    for (int i = threadIdx.x; i < rows * (HD / 4); i += NTH) {
      const int x = i / (HD / 4), c = i % (HD / 4) * 4;
      float M = -INFINITY, L = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < NW; ++k) M = fmaxf(M, s_ml[k * R + x].x);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float2 ml = s_ml[k * R + x];
        const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
        const float4 v = *reinterpret_cast<const float4 *>(so + (k * R + x) * LD + c);
        L += w * ml.y;
        a.x += w * v.x; a.y += w * v.y; a.z += w * v.z; a.w += w * v.w;
      }
      if constexpr (CL) {
        *reinterpret_cast<float4 *>(s_part + x * HD + c) = a;
        if (c == 0) s_pml[x] = make_float2(M, L);
      } else if (!whole) {
        *reinterpret_cast<float4 *>(P.part_o + (slot + x) * HD + c) = a;
        if (c == 0) P.part_ml[slot + x] = make_float2(M, L);
      } else {
        write(x, c, a, L);
      }
    }
    if constexpr (CL) cluster_join<NTH, HD>(s_part, s_pml, rows, rank, ranks, write);
    __syncthreads();                            // before the next piece fills the rings and the list
  }
}

static int full_grid() { return kBlocksPerSm * device_sm_count(); }

static size_t partials() { return 2ull * full_grid() * 16; }

// Few items over few keys: each item's keys go to one cluster of up to 8 blocks, which
// joins in its shared memory.  0: the line.
template <typename T, int HD, bool HALF> static cudaError_t set_attributes() {
  const cudaError_t e = cudaFuncSetAttribute(paged_picked_kernel<T, HD, false, HALF>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, DecCfg<T, HD, 1>::kSmem);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(paged_picked_kernel<T, HD, true, HALF>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * DecCfg<T, HD, 1>::kSmem);
}
template <typename T, int HD, bool HALF> static int cluster_of(int64_t items, int64_t blocks) {
  static ClusterRoom room;
  return plan_cluster(items, blocks, device_sm_count(), 1, full_grid(), 8,
                      room.of(paged_picked_kernel<T, HD, true, HALF>, Form<true>::kThreads, 2 * DecCfg<T, HD, 1>::kSmem,
                              set_attributes<T, HD, HALF>));
}
// f(kernel's type, head_dim, HALF) as values of types, for a call's dtype, head_dim and group.
template <typename F> static auto with_form(cb_dtype dt, int hd, int G, F &&f) {
  typedef std::integral_constant<int, 64> D64;
  typedef std::integral_constant<int, 128> D128;
  if (dt == CB_F32) return hd == 128 ? f(0.f, D128{}, std::false_type{}) : f(0.f, D64{}, std::false_type{});
  if (G <= 8) return hd == 128 ? f(bf16{}, D128{}, std::true_type{}) : f(bf16{}, D64{}, std::true_type{});
  return hd == 128 ? f(bf16{}, D128{}, std::false_type{}) : f(bf16{}, D64{}, std::false_type{});
}

// Key blocks of an item.
static int64_t key_blocks(int n_picks, int page_size, int hd, cb_dtype dt) {
  const int bn = dt == CB_BF16 ? (hd == 128 ? DecCfg<bf16, 128, 1>::kBN : DecCfg<bf16, 64, 1>::kBN)
                               : (hd == 128 ? DecCfg<float, 128, 1>::kBN : DecCfg<float, 64, 1>::kBN);
  return ((int64_t)n_picks * page_size + bn - 1) / bn;
}

template <typename T, int HD, bool HALF>
static cudaError_t run(Params &P, int page_size, int *status, cudaStream_t s) {
  typedef DecCfg<T, HD, 1> C;
  static PerDeviceOnce attr;
  cudaError_t e = attr.run([](int) { return set_attributes<T, HD, HALF>(); });
  if (e != cudaSuccess) return e;
  P.blocks = (int)key_blocks(P.n_picks, page_size, HD, std::is_same<T, float>::value ? CB_F32 : CB_BF16);
  const int64_t items = (int64_t)P.n_rows * P.Hkv * P.tiles;
  P.units = items * P.blocks;
  if (const int c = cluster_of<T, HD, HALF>(items, P.blocks)) {
    e = launch_clusters(paged_picked_kernel<T, HD, true, HALF>, dim3((unsigned)(items * c)), dim3(Form<true>::kThreads), c,
                        2 * C::kSmem, s, P, status);
    return e == cudaSuccess ? launched(1) : e;
  }
  // a part has a block for each warp; few items take the same number of parts each
  const int64_t most = (P.units + 3) / 4;
  P.parts = (int)(most < full_grid() ? most : full_grid());
  if (items < P.parts) P.parts -= (int)(P.parts % items);
  e = launch_pdl(paged_picked_kernel<T, HD, false, HALF>, dim3(P.parts), dim3(kDecThreads), C::kSmem, s, P, status);
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_merge_kernel<T, HD>, dim3(P.parts, 16 / kJoinRows), dim3(kJoinThreads),
                 P.parts * kJoinRows * sizeof(float2), s, static_cast<const AttnParams &>(P), 16);
  return e == cudaSuccess ? launched(2) : e;
}

}  // namespace picked

size_t paged_picked_ws_bytes(int n_rows, int, int, int, int, int hd, cb_dtype) {
  using namespace picked;
  if (n_rows <= 0) return 0;
  return partials() * (hd * sizeof(float) + sizeof(float2)) + full_grid() * sizeof(Join);
}

void paged_picked_plan(int n_rows, int n_picks, int page_size, int Hq, int Hkv, int hd, cb_dtype dt, int64_t out[3]) {
  const int64_t items = (int64_t)n_rows * Hkv * ((Hq / Hkv + 15) / 16), blocks = picked::key_blocks(n_picks, page_size, hd, dt);
  out[0] = picked::with_form(dt, hd, Hq / Hkv, [&](auto t, auto d, auto half) {
    return picked::cluster_of<decltype(t), decltype(d)::value, decltype(half)::value>(items, blocks);
  });
  out[1] = items;
  out[2] = blocks;
}

cudaError_t launch_paged_picked(const PagedKV &kv, const cb_paged_query &a, const int32_t *picks, int n_picks,
                                cb_dtype dt, int *status, cudaStream_t s) {
  using namespace picked;
  Params P;
  P.kv = kv;
  P.q = a.q;
  P.out = a.out;
  P.ld_q = a.ld_q;
  P.ld_out = a.ld_out;
  P.n_rows = a.n_rows;
  P.G = a.n_q_heads / a.n_kv_heads;
  P.Hkv = a.n_kv_heads;
  P.max_kv = 0;
  P.n_split = 1;
  P.few_hi = P.rows_lo = 0;
  P.hc = 1;
  P.by_G = Divisor(P.G);
  P.by_quads = Divisor(a.n_kv_heads);
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.picks = picks;
  P.n_picks = n_picks;
  P.tiles = (P.G + 15) / 16;
  P.part_o = reinterpret_cast<float *>(a.ws);
  P.part_ml = reinterpret_cast<float2 *>(P.part_o + partials() * a.head_dim);
  P.joins = reinterpret_cast<Join *>(P.part_ml + partials());
  return with_form(dt, a.head_dim, P.G, [&](auto t, auto d, auto half) {
    return run<decltype(t), decltype(d)::value, decltype(half)::value>(P, kv.page_size, status, s);
  });
}

}  // namespace cb
