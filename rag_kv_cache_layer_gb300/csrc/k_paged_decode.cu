// Paged attention of a few rows per sequence (generated tokens, short drafts)
// in bf16, and of any rows in fp32: keys and values stream through shared
// memory once, and the group's q heads share them.
//
// Work.  A tile is R = 16 WM rows of one sequence and kv head (an item); its
// keys come in blocks of BN.  All blocks of all items form one line of units,
// which is cut into equal parts, one per block of the grid (two per SM): a
// long sequence is shared by many blocks, short ones are taken whole, and the
// lengths decide that on the device, so lengths of any mix keep every SM busy
// until the end.  An item inside one part is written out directly; one that
// crosses parts leaves its pieces' (O, m, l) in the workspace, at most two per
// block, and decode_merge_kernel joins them; the block with an item's first
// piece also leaves the join's record, so the joining kernel searches nothing.
//
// A block's four warps form WK = 4 / WM groups of WM warps.  With many items
// (hc = WK, decode_heads) an item is WK neighbouring heads, one per group, all
// groups walking the same keys: their slices of a cache row lie side by side
// and are read together, which the memory's pages like (64 ragged requests:
// 142 us with a head per item, 123 so), and the groups' states need no join.
// Else (hc = 1) an item is one head, and key block i goes to group i mod WK.
// A group fills a ring of its own by 16-byte cp.async, kStages - 1 blocks ahead
// (2 for 16-row tiles, 5 for 32, 11 or 5 for 64), with zeros for keys past the
// cached length (so nothing unwritten in a page reaches the products), and meets
// nobody else inside the loop.  TMA is not used here: a page's slice of one head is a box of 8 to 64
// rows of 256 bytes, and a box costs about 140 ns of one SM's copy unit
// whatever its height, which held the same loop to 12 - 27 GB/s per block.
//
// Each warp holds 16 rows, with the running maximum, sum and O in registers
// (base-2 exponentials, fp32).  bf16: S = Q K^T and O += P V by mma.m16n8k16 on
// fragments from ldmatrix; P rounds to bf16 as the second product's operand.
// The legacy tensor instruction is the right one there: the work is bound by
// the pages' bytes, 45 bytes per nanosecond and SM, and a 128-row tcgen05 tile
// with 4 rows in use would not read them faster.
// fp32: the same products by mma.m16n8k8 on TF32 halves, x = hi + lo with hi
// the nearest TF32 value and lo = x - hi: hi hi + hi lo + lo hi drops 2^-22 of
// a product, as much as an fp32 rounding or two.  The tensor core truncates
// its sums, so every step of eight goes into a fresh accumulator that is added
// in fp32 (one chain over 128 dimensions and thousands of keys would drift by
// 1e-5 and more).  That is 2 to 5 times the CUDA cores' rate and keeps their
// error.
//
// Measured (32/8 heads of 128): 64 ragged requests of 200 to 16,384 keys 122 to
// 125 us, 6.0 TB/s; two of 120 to 131 thousand 162 to 166 us, 6.3 TB/s: memory.  One
// row over 3137 keys 10.8 us: a block's 12,000 cycles of mostly dependent instructions
// and the join.  fp32: 37 TFLOP/s on many rows (4.2 TB/s on single ones), bound
// by instructions, about 25 for each step's three products.
#include <type_traits>

#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"
#include "cb_paged_attn.cuh"
#include "cb_paged_few.cuh"
#include "cb_paged_line.cuh"

namespace cb {
namespace paged {

constexpr int kDecBlocksPerSm = 2;

// Meets the WM warps of group `wk` (named barrier 1 + wk).
template <int WM> __device__ __forceinline__ void group_sync(int wk) {
  if (WM == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + wk), "r"(32 * WM) : "memory");
}

// HEADS: an item is WK heads, one per group (P.hc = WK); else one head.
template <typename T, int HD, int WM, bool HEADS>
__global__ void __launch_bounds__(kDecThreads, kDecBlocksPerSm)
paged_decode_kernel(const __grid_constant__ AttnParams P, int *status) {
  typedef DecCfg<T, HD, WM> C;
  constexpr bool F32 = std::is_same<T, float>::value;
  // KS: k-steps of Q K^T (16 dims in bf16, 8 in fp32)
  constexpr int R = 16 * WM, WK = 4 / WM, ND = HD / 8, KS = F32 ? HD / 8 : HD / 16, BN = C::kBN, NS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Line line;
  __shared__ int64_t s_sums[kDecThreads / 32];
  __shared__ float2 s_ml[4 * 16];               // (m, l) of each warp's rows
  grid_dep_wait();
  grid_dep_launch();
  make_line(P, R, BN, gridDim.x, line, s_sums, status);
  Join *const join = P.joins + blockIdx.x;
  if ((int)blockIdx.x >= line.parts) {
    if (threadIdx.x == 0) join->rows = 0;
    return;
  }
  const int64_t u0 = part_begin(line, blockIdx.x), u1 = part_begin(line, blockIdx.x + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp % WM, wk = warp / WM, gid = lane >> 2, q4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + wk * NS * C::kStage;
  // heads per item; this group's head among them, its first key block, its step
  constexpr int hc = HEADS ? WK : 1, step = HEADS ? 1 : WK;
  const int sub = HEADS ? wk : 0, first_block = HEADS ? 0 : wk;
  const int shift = __ffs(P.kv.page_size) - 1;
  const T *kp = reinterpret_cast<const T *>(P.kv.k_pages), *vp = reinterpret_cast<const T *>(P.kv.v_pages);
  // rows and column that this lane copies: row i * kRows + crow of a stage
  constexpr int kVec = 16 / sizeof(T), kCols = HD / kVec, kRows = 32 / kCols;
  const int crow = lane / kCols, ccol = lane % kCols;
  // ldmatrix row of this lane: K tiles as 8 keys x 4 8-dim columns, V tiles as
  // 16 keys x 2 8-dim columns
  const int krow = lane & 7, kcol = lane >> 3, vrow = lane & 15, vcol = lane >> 4;
  const float sl2 = P.scale_log2;

  int s = seq_of(line, P.kv.n_seq, u0);
  for (int64_t u = u0; u < u1;) {
    // this piece: a tile of sequence s for a group of heads (an item), its blocks [jb, je)
    while (line.blocks[s] == 0 || (s + 1 < P.kv.n_seq && line.begin[s + 1] <= u)) ++s;
    const int row0 = __ldg(P.kv.row_offsets + s), n = __ldg(P.kv.row_offsets + s + 1) - row0;
    const int kv = __ldg(P.kv.kv_lens + s), base = kv - n, all = n * P.G, tiles = (all - 1) / R + 1;
    int64_t local = u - line.begin[s];
    int nbs = line.blocks[s], ph, jb, l0 = 0;    // the item's units; its pair and heads, its unit, its first row
    const int64_t pairs = (int64_t)(tiles / 2) * P.by_quads.d * nbs;
    if (local >= pairs) {                       // the only tile, or an odd middle one
      if (tiles > 1) {
        l0 = tiles / 2 * R;
        nbs = blocks_seen(P, base, l0 + R - 1, BN);
      }
      divide(local - pairs, nbs, ph, jb);
    } else {
      divide(local, nbs, ph, jb);
      const int q = P.by_quads.div(ph), late = blocks_seen(P, base, min((tiles - q) * R, all) - 1, BN);
      ph -= q * (int)P.by_quads.d;
      if (jb < late) {
        nbs = late;
        l0 = (tiles - 1 - q) * R;
      } else {
        nbs -= late;
        jb -= late;
        l0 = q * R;
      }
    }
    const int g0 = ph * hc, g = g0 + sub, rows = min(R, all - l0);
    const int take = (int)min((int64_t)(nbs - jb), u1 - u);
    const bool whole = jb == 0 && take == nbs, first = u == u0;
    const int64_t item_end = u - jb + nbs;
    u += take;
    const int seen = base + P.by_G.div(l0 + rows - 1) + 1;    // keys the tile's last row sees
    const int je = min(jb + take, seen > 0 ? (seen - 1) / BN + 1 : 0);
    const int32_t *table = P.kv.block_table + (int64_t)s * P.kv.ld_table;
    if (threadIdx.x == 0 && u == u1)            // the last piece: the one that may go on in the next part
      *join = Join{row0, l0, jb == 0 && item_end > u1 ? rows : 0, g0, part_of(line, item_end - 1), first ? 0 : 1};

    auto fetch = [&](int j) -> int {            // page of key j * BN + lane
      const int key = j * BN + lane;
      return j < je && lane < BN && key < kv ? __ldg(table + (key >> shift)) : -1;
    };
    const int64_t lane_off = g * HD + ccol * kVec, down = (int64_t)(WM * kRows) * P.kv.ld;
    auto load = [&](int j, int st, int page) {
      const uint32_t dst = ring + st * C::kStage;
      if (page >= 0 && page >= P.kv.n_pages) {
        report(status, CB_ERR_DEVICE_INDEX);
        page = -1;
      } else if (page < 0 && j < je && lane < BN && j * BN + lane < kv) {
        report(status, CB_ERR_DEVICE_INDEX);
      }
      // eight rows lie in one page (page_size >= 8): one lookup, then a stride
      int pg = 0;
      int64_t off = 0;
#pragma unroll
      for (int i = 0; i < BN / kRows / WM; ++i) {
        const int r = (i * WM + wm) * kRows + crow;
        pg = __shfl_sync(0xffffffffu, page, r);
        if (i * WM * kRows % 8 == 0) {
          const int slot = (j * BN + r) & (P.kv.page_size - 1);
          off = (int64_t)pg * P.kv.page_stride + (int64_t)slot * P.kv.ld + lane_off;
        } else {
          off += down;
        }
        const int64_t from = pg < 0 ? 0 : off;
        // 16-byte columns are swizzled so that the fragments' reads meet all
        // banks: by the row, or (V in fp32) by the pair of rows
        const uint32_t d = dst + r * C::kRow, x = F32 ? ((r >> 1) & 3) << 1 : r & 7;
        copy16(d + ((ccol ^ (r & 7)) << 4), kp + from, pg >= 0);
        copy16(d + C::kTile + ((ccol ^ x) << 4), vp + from, pg >= 0);
      }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    // the table is read kAhead blocks further ahead than the pages: the first
    // stages' entries one after the other would cost a memory latency each
    constexpr int kAhead = 3;
    int ahead[kAhead], from = jb + first_block;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ahead[i] = fetch(from + i * step);
    auto next_page = [&]() -> int {
      const int page = ahead[0];
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) ahead[i] = ahead[i + 1];
      ahead[kAhead - 1] = fetch(from + kAhead * step);
      from += step;
      return page;
    };
    int pos[2];
    uint32_t qf[KS][4];                         // bf16 pairs, or fp32 values
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = wm * 16 + gid + 8 * h;
      const bool valid = r < rows;
      const int qi = P.by_G.div(l0 + r);
      pos[h] = valid ? base + qi : -1;
      const T *src = reinterpret_cast<const T *>(P.q) + (int64_t)(row0 + qi) * P.ld_q +
                     (int64_t)(g * P.G + l0 + r - qi * P.G) * HD + (F32 ? q4 : q4 * 2);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          qf[k][h + 2 * c] =
              valid ? *reinterpret_cast<const uint32_t *>(src + (F32 ? k * 8 + c * 4 : k * 16 + c * 8)) : 0u;
    }
    float o[ND][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;

#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i) {
      const int j = from, page = next_page();
      if (j < je) load(j, i, page);
      commit();
    }
    int st = 0, fill = NS - 1;
    for (int j = jb + first_block; j < je; j += step) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
      group_sync<WM>(wk);                       // landed for every warp; the stage before is used up
      {
        const int jn = from, page = next_page();
        if (jn < je) load(jn, fill, page);
        commit();
        fill = fill + 1 == NS ? 0 : fill + 1;
      }
      const uint32_t ks = ring + st * C::kStage, vs = ks + C::kTile;
      st = st + 1 == NS ? 0 : st + 1;
      float x[BN / 8][4];
#pragma unroll
      for (int t = 0; t < BN / 8; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[t][k] = 0.f;
      const uint32_t krows = ks + krow * C::kRow;
      // 64 bytes of 8 keys: two k-steps
      if constexpr (F32) {
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2) {
          uint32_t b[BN / 8][4];
#pragma unroll
          for (int t = 0; t < BN / 8; ++t)
            ldsm_x4(krows + t * 8 * C::kRow + (((k2 * 4 + kcol) ^ krow) << 4), b[t]);
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
      const int key0 = j * BN;
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int t = 0; t < BN / 8; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = key0 + t * 8 + q4 * 2 + (k & 1);
          x[t][k] = key <= pos[k >> 1] ? x[t][k] * sl2 : -INFINITY;
          mx[k >> 1] = fmaxf(mx[k >> 1], x[t][k]);
        }
      bool moved = false;
      float corr[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        const float mn = fmaxf(m[h], mx[h]);
        corr[h] = mn == m[h] ? 1.f : ex2(m[h] - mn);        // also where both are -inf
        moved |= mn != m[h];
        m[h] = mn;
        l[h] *= corr[h];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[d][k] *= corr[k >> 1];
      }
#pragma unroll
      for (int t = 0; t < BN / 8; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = x[t][k] == -INFINITY ? 0.f : ex2(x[t][k] - m[k >> 1]);
          x[t][k] = p;
          l[k >> 1] += p;
        }
      if constexpr (F32) {
        // The product's step takes the keys of a tile in the order 0 2 4 6 1 3
        // 5 7, in which the scores' registers already are its operand.
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
            // dims d * 8 + gid of keys 2 q4 and 2 q4 + 1
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
          const uint32_t a[4] = {pack_bf16(x[2 * k2][0], x[2 * k2][1]), pack_bf16(x[2 * k2][2], x[2 * k2][3]),
                                 pack_bf16(x[2 * k2 + 1][0], x[2 * k2 + 1][1]),
                                 pack_bf16(x[2 * k2 + 1][2], x[2 * k2 + 1][3])};
          const uint32_t row = vs + (k2 * 16 + vrow) * C::kRow;
#pragma unroll
          for (int d2 = 0; d2 < ND / 2; ++d2) {
            uint32_t b[4];
            ldsm_x4_t(row + (((d2 * 2 + vcol) ^ (vrow & 7)) << 4), b);
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
      if (q4 == 0) s_ml[warp * 16 + gid + 8 * h] = make_float2(m[h], l[h]);
    }
    __syncthreads();                            // the rings are used up
    // Every warp leaves its O in rows of HD + 4 floats (a quad's four rows
    // fall into different banks), then the groups' states join.
    constexpr int LD = HD + 4;
    static_assert(4 * 16 * LD * 4 <= C::kSmem, "the warps' O fit the rings");
    float *so = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2 *>(so + (warp * 16 + gid + 8 * h) * LD + d * 8 + q4 * 2) =
            make_float2(o[d][2 * h], o[d][2 * h + 1]);
    __syncthreads();
    const int64_t slot = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * R * hc;
    const int per_head = rows * (HD / 4);
    for (int i = threadIdx.x; i < hc * per_head; i += kDecThreads) {
      const int hs = HEADS ? i / per_head : 0, e = i - hs * per_head;
      const int r = e / (HD / 4), c = e % (HD / 4) * 4;
      float M = -INFINITY, L = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      // the states of the head's groups: all, or its own
#pragma unroll
      for (int k = 0; k < WK / hc; ++k) M = fmaxf(M, s_ml[((hs + k) * WM + r / 16) * 16 + r % 16].x);
#pragma unroll
      for (int k = 0; k < WK / hc; ++k) {
        const int row = ((hs + k) * WM + r / 16) * 16 + r % 16;
        const float2 ml = s_ml[row];
        const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
        const float4 v = *reinterpret_cast<const float4 *>(so + row * LD + c);
        L += w * ml.y;
        a.x += w * v.x; a.y += w * v.y; a.z += w * v.z; a.w += w * v.w;
      }
      if (!whole) {
        const int64_t at = slot + hs * R + r;
        *reinterpret_cast<float4 *>(P.part_o + at * HD + c) = a;
        if (c == 0) P.part_ml[at] = make_float2(M, L);
      } else {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int qi = P.by_G.div(l0 + r);
        T *dst = reinterpret_cast<T *>(P.out) + (int64_t)(row0 + qi) * P.ld_out +
                 (int64_t)((g0 + hs) * P.G + l0 + r - qi * P.G) * HD + c;
        if constexpr (F32)
          *reinterpret_cast<float4 *>(dst) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        else
          *reinterpret_cast<uint2 *>(dst) =
              make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
      }
    }
    __syncthreads();                            // before the next piece fills the rings
  }
}

int decode_grid() { return kDecBlocksPerSm * device_sm_count(); }
// Heads per item: as many as the block has groups where that leaves at least
// one item for every eight parts, else one (an item in many pieces is joined
// slowly: one row over 3137 keys takes 20.8 us with four heads per item, 10.9 with
// one; 64 ragged sequences 123 and 142).
int decode_heads(int R, int64_t tiles, int Hkv) {
  const int groups = 64 / R;
  return Hkv % groups == 0 && 8 * tiles * (Hkv / groups) >= decode_grid() ? groups : 1;
}

template <typename T, int HD, int WM, bool HEADS>
static cudaError_t run(const AttnParams &P, int *status, cudaStream_t s) {
  typedef DecCfg<T, HD, WM> C;
  static PerDeviceOnce attr;
  cudaError_t e = attr.run([](int) {
    return cudaFuncSetAttribute(paged_decode_kernel<T, HD, WM, HEADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::kSmem);
  });
  if (e != cudaSuccess) return e;
  const int grid = decode_grid();               // 32 bytes of weights for each: within the default limit
  e = launch_pdl(paged_decode_kernel<T, HD, WM, HEADS>, dim3(grid), dim3(kDecThreads), C::kSmem, s, P, status);
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_merge_kernel<T, HD>, dim3(grid, 16 * WM * P.hc / kJoinRows), dim3(kJoinThreads),
                 grid * kJoinRows * sizeof(float2), s, P, 16 * WM);
  return e == cudaSuccess ? launched(2) : e;
}

template <typename T, int HD>
static cudaError_t run_rows(const AttnParams &P, int R, int *status, cudaStream_t s) {
  if (R == 64) return run<T, HD, 4, false>(P, status, s);
  if (R == 32) return P.hc > 1 ? run<T, HD, 2, true>(P, status, s) : run<T, HD, 2, false>(P, status, s);
  return P.hc > 1 ? run<T, HD, 1, true>(P, status, s) : run<T, HD, 1, false>(P, status, s);
}

cudaError_t launch_decode(const AttnParams &P, int R, int hd, cb_dtype dt, int *status, cudaStream_t s) {
  if (dt == CB_BF16) return hd == 128 ? run_rows<bf16, 128>(P, R, status, s) : run_rows<bf16, 64>(P, R, status, s);
  return hd == 128 ? run_rows<float, 128>(P, R, status, s) : run_rows<float, 64>(P, R, status, s);
}

}  // namespace paged
}  // namespace cb
