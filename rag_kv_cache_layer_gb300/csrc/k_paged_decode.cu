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

namespace cb {
namespace paged {

constexpr int kDecThreads = 128;
constexpr int kDecBlocksPerSm = 2;

template <typename T, int HD, int WM> struct DecCfg {
  // keys per stage: 8 KB of K and V together; fp32 tiles of 64 rows take at least 16
  // keys, since a block of 8 costs them as much in its meeting and its softmax as in
  // products (256 rows over 8192 keys, 32/8 heads of 128: 1089 us, 918 so; 16 keys
  // are enough at head_dim 64: 27.8 us for ragged chunks, 28.6 with 32)
  static constexpr int kMul = sizeof(T) == 4 && WM == 4 && HD == 128 ? 2 : 1;
  static constexpr int kBN = kMul * 4096 / (int)sizeof(T) / HD;
  static constexpr int kRow = HD * (int)sizeof(T);
  static constexpr int kTile = kBN * kRow;
  static constexpr int kStage = 2 * kTile;      // K then V
  static constexpr int kStages = 3 * WM / kMul; // of each group: 96 KB per block
  static constexpr int kSmem = (4 / WM) * kStages * kStage;
};

__device__ __forceinline__ void ldsm_x4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo, hi the nearest TF32 value (10 bits after the point; ties away
// from zero).
__device__ __forceinline__ void halves(float x, uint32_t &hi, uint32_t &lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// c += A B of one m16n8k8 step in fp32: three TF32 products in a fresh
// accumulator.
__device__ __forceinline__ void step_f32(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], float b0,
                                         float b1) {
  uint32_t h0, l0, h1, l1;
  halves(b0, h0, l0);
  halves(b1, h1, l1);
  float t[4] = {0.f, 0.f, 0.f, 0.f};
  mma1688(t, al, h0, h1);
  mma1688(t, ah, l0, l1);
  mma1688(t, ah, h0, h1);
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] += t[i];
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// 16 bytes to shared memory, or 16 zero bytes when `there` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// 2^x, relative error about 2^-22, far below the rounding of P to bf16.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Meets the WM warps of group `wk` (named barrier 1 + wk).
template <int WM> __device__ __forceinline__ void group_sync(int wk) {
  if (WM == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + wk), "r"(32 * WM) : "memory");
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
__device__ __forceinline__ void make_line(const AttnParams &P, int R, int BN, int grid, Line &L, int64_t *warp_sums,
                                          int *status) {
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
        units = pair = blocks_seen(P, len - n, n * P.G - 1, BN);
      else {
        // each of a pair's two counts is within one of a linear function of
        // the tile, and those add up to the same in every pair
        pair = blocks_seen(P, len - n, R - 1, BN) + blocks_seen(P, len - n, tiles * R - 1, BN) + 2;
        units = tiles & 1 ? blocks_seen(P, len - n, (tiles / 2 + 1) * R - 1, BN) : 0;
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
