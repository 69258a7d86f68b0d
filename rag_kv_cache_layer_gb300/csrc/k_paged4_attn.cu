// Attention over a paged cache of 4-bit floats, few rows per sequence.
//
// Work is cut as in the few-rows kernel of the 16-bit cache (cb_paged_line.cuh): a
// tile is R = 8 NT rows of one sequence and kv head, its keys come in blocks of 32,
// all blocks of all tiles form one line that the grid's blocks share in equal parts,
// and decode_merge_kernel joins tiles that several parts hold.  The block's four
// warps take a tile's key blocks in turn, each with a cp.async ring of its own.  A call
// of few tiles over few keys gives each tile to a cluster instead, blocks of eight
// warps, which join in its shared memory: one launch (see plan_cluster).
//
// Mathematics.  A code times its scale is exact in fp16 (cb_q4.cuh), so keys and
// values meet the tensor cores as fp16 without a rounding.  q is put into fp16 after
// a power of two per row that brings its largest magnitude to [2^13, 2^14): a bf16 q
// is then exact down to 2^-27 of that magnitude and off by at most 2^-38 of it
// below.  P = 2^(x - m + 8), m a reference that the scores x exceed by 7 at most (so that
// most blocks leave it and O as they are), rounds to fp16 (2^-11 of itself, 2^-33 of the
// reference's weight at the bottom: the results' error is that of their own rounding, 0.0017
// with P in fp16 and in fp32, and a second half of P would be products on the pipes that bound
// this kernel); both powers of two leave with the softmax scale and
// the division by the sum.  fp32 rows take q and P as two fp16 halves (hi, lo with
// 2^-22 and less dropped) and every step of 16 in a fresh accumulator that is added
// in fp32, since the tensor core truncates its sums.
//
// Both products put the cache on the 16-row side of mma.m16n8k16 and the query rows
// on the 8-column side: S^T = K Q^T, O^T = V^T P^T.  A group of up to 8 heads then
// fills the instruction, and a lane's operand is made of neighbouring dimensions of
// one key (K: 32, one 16-byte load and two scales) or of 16 dimensions of four keys
// (V: four 8-byte loads), so that codes go from shared memory to fp16 pairs by one
// conversion and one product with the scale for two values; V's pairs are two keys'
// codes of one dimension, put into a byte by a shift and a select first.  S^T comes
// out as P^T's operand up to a transposition of 8x8 blocks (movmatrix).
//
// Measured, 32/8 heads of 128: 64 ragged requests of up to 16,384 keys 50.1 us (4.3 TB/s
// of 216 MB), two of 131 k keys 60 (4.9 TB/s), one row over 3137 keys 9.0, from a graph.
// Bound by instructions, not by the cache's bytes: a block of 32 keys costs a warp about
// 590, of which 250 go to the ALU pipe at half a warp a cycle (the codes' conversions,
// the maximum, the masks), 220 to the FMA pipes, 30 to the tensor cores (26% busy); a
// scheduler issues in 0.60 of its cycles with its four warps and waits mostly for the
// results of the warp's own instructions.  A piece of a tile costs about 6000 cycles beside
// (places 1000, pages and q 2000, join and output 2000), the cut of the line 4000.  The
// 16-bit cache's kernel is bound by bytes (128 us for the same requests).
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"
#include "cb_paged_attn.cuh"
#include "cb_paged_line.cuh"
#include "cb_q4.cuh"
#include "cb_tc.cuh"

namespace cb {
namespace paged4 {

using namespace paged;

typedef AttnParams Params;

constexpr int kBN = 32;                 // keys per block
// Blocks that a tile's own cost (its q, the joins) counts as when the line is cut: 64 ragged
// requests 51 us, without 73, with 24 55; two of 131 k keys 61.6 and 63.4.
constexpr int kPad = 12;
constexpr float kPShift = 8.f;          // log2 of P at the reference
// log2 of what a score may exceed it by: P stays below 2^15 (64 ragged requests 51.0 us; 52.4
// with a reference that follows every rise)
constexpr float kRise = 7.f;
// A row whose reference (log2) is larger than this is scaled down to it: fp32 tells such scores
// apart by 0.5 at best, and x sl + shift would be off by more than P has room for (the same
// branch that moves the reference looks: the batch above 50.1 us with and without, one row over
// 3137 keys 8.7 without and 8.85 with).
constexpr float kBig = 0x1p22f;

// CL: a tile's keys in one cluster, eight warps a block.
template <int HD, int NT, bool F32, bool CL> struct Cfg {
  static constexpr int kRows = 8 * NT, kWarps = CL ? 8 : 4, kThreads = 32 * kWarps;
  static constexpr int kPerSm = CL ? (NT == 1 && !F32 ? 2 : 1) : NT == 4 || F32 ? 2 : NT == 2 ? 3 : 4;
  static constexpr int kStages = CL ? (NT == 1 ? 2 : NT == 2 ? 3 : 4) : NT == 4 || F32 ? 4 : NT == 2 ? 3 : 2;
  static constexpr int kCodes = kBN * HD / 2, kScales = kBN * HD / 16;
  static constexpr int kOffV = kCodes, kOffKs = 2 * kCodes, kOffVs = kOffKs + kScales;
  static constexpr int kStage = kOffVs + kScales;
  static constexpr int kSmem = kWarps * kStages * kStage;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from c = 0
__device__ __forceinline__ void mma_f16_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// hi: the halves of (x, y) nearest in fp16; the result: what they leave.
__device__ __forceinline__ uint32_t pack_rest(float x, float y, uint32_t hi) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  return pack_f16(x - h.x, y - h.y);
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// W words from shared memory.
template <int W> __device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[W]) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  else
    w[0] = lds32(a);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void copy_all(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// `bytes` bytes to shared memory and zeros up to 16.
__device__ __forceinline__ void copy_part(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

struct None {};

template <typename T, int HD, int NT, bool CL>
__global__ void __launch_bounds__((Cfg<HD, NT, std::is_same<T, float>::value, CL>::kThreads),
                                  (Cfg<HD, NT, std::is_same<T, float>::value, CL>::kPerSm))
paged4_few_kernel(const __grid_constant__ Params P, int *status) {
  constexpr bool F32 = std::is_same<T, float>::value;
  typedef Cfg<HD, NT, F32, CL> C;
  constexpr int NW = C::kWarps;
  constexpr int R = C::kRows, NS = C::kStages, KS = HD / 16, MT = HD / 16;
  // words of codes that a lane takes of a key (K: HD / 4 dimensions; V: HD / 8)
  constexpr int KW = HD / 32, VW = HD / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ typename std::conditional<CL, None, Line>::type s_line;
  __shared__ int64_t s_sums[NW];
  __shared__ float2 s_ml[NW * R];               // (m, l) of each warp's rows
  __shared__ float s_sl[NW * R];                // their log2 scales, where sl is scaled down
  __shared__ PagedTile s_tile;
  // CL: the block's joined rows, read by the cluster's others
  __shared__ __align__(16) float s_part[CL ? R * HD : 4];
  __shared__ float2 s_pml[CL ? R : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, q4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * NS * C::kStage;
  const int page_size = P.kv.page_size, shift = __ffs(page_size) - 1;
  const uint8_t *const pool = reinterpret_cast<const uint8_t *>(P.kv.k_pages);
  grid_dep_wait();
  grid_dep_launch();
  int64_t u0 = 0, u1 = 1;
  int s = 0, rank = 0, ranks = 1;
  int at_s = -1, row0 = 0, n = 0, kv = 0;       // of sequence at_s: first row, rows, length
  if constexpr (CL) {
    ranks = tcx::cluster_size();
    rank = blockIdx.x % ranks;
    paged_find_tile<C::kThreads>(P.kv, P.n_rows, P.G, R, P.max_kv, (int)P.by_quads.div(blockIdx.x / ranks), &s_tile,
                                 reinterpret_cast<int *>(s_sums), status);
    if (s_tile.s < 0) return;                   // (as in the cluster's other blocks)
  } else {
    make_line(P, R, kBN, gridDim.x, s_line, s_sums, status, P.pad);
    Join *const join = P.joins + blockIdx.x;
    if (threadIdx.x == 0) join->rows = 0;
    if ((int)blockIdx.x >= s_line.parts) return;
    u0 = part_begin(s_line, blockIdx.x);
    u1 = part_begin(s_line, blockIdx.x + 1);
    s = seq_of(s_line, P.kv.n_seq, u0);
  }
  for (int64_t u = u0; u < u1;) {
    // this piece: rows [l0, l0 + rows) of sequence s and kv head g, key blocks [jb, je)
    int base, g, l0 = 0, rows, jb, je, seen;
    bool whole = true, first = true;
    if constexpr (CL) {
      const PagedTile t = s_tile;
      u = u1;
      s = t.s;
      row0 = t.row0;
      kv = t.kv;
      base = kv - t.n;
      const int item = blockIdx.x / ranks;
      g = item - P.by_quads.div(item) * (int)P.by_quads.d;
      l0 = t.t * R;
      rows = min(R, t.n * P.G - l0);
      seen = base + P.by_G.div(l0 + rows - 1) + 1;            // keys the tile's last row sees
      const int nb = seen > 0 ? (seen - 1) / kBN + 1 : 0;
      jb = (int)((int64_t)nb * rank / ranks);
      je = (int)((int64_t)nb * (rank + 1) / ranks);
    } else {
      // (as in paged_decode_kernel)
      const Line &line = s_line;
      while (line.blocks[s] == 0 || (s + 1 < P.kv.n_seq && line.begin[s + 1] <= u)) ++s;
      if (s != at_s) {                          // (most often the next head of the same sequence)
        at_s = s;
        row0 = __ldg(P.kv.row_offsets + s);
        n = __ldg(P.kv.row_offsets + s + 1) - row0;
        kv = __ldg(P.kv.kv_lens + s);
      }
      base = kv - n;
      const int all = n * P.G, tiles = (all - 1) / R + 1;
      int64_t local = u - line.begin[s];
      int nbs = line.blocks[s];
      const int64_t pairs = (int64_t)(tiles / 2) * P.by_quads.d * nbs;
      if (local >= pairs) {                     // the only tile, or an odd middle one
        if (tiles > 1) {
          l0 = tiles / 2 * R;
          nbs = blocks_seen(P, base, l0 + R - 1, kBN) + P.pad;
        }
        divide(local - pairs, nbs, g, jb);
      } else {
        divide(local, nbs, g, jb);
        const int q = P.by_quads.div(g), late = blocks_seen(P, base, min((tiles - q) * R, all) - 1, kBN) + P.pad;
        g -= q * (int)P.by_quads.d;
        if (jb < late) {
          nbs = late;
          l0 = (tiles - 1 - q) * R;
        } else {
          nbs -= late;
          jb -= late;
          l0 = q * R;
        }
      }
      rows = min(R, all - l0);
      const int take = (int)min((int64_t)(nbs - jb), u1 - u);
      const int real = blocks_seen(P, base, l0 + rows - 1, kBN);   // of the tile's units, the others are padding
      const int64_t item_end = u - jb + real;
      whole = jb == 0 && item_end <= u1;
      first = u == u0;
      u += take;
      if (jb >= real) continue;                 // nothing but padding
      seen = base + P.by_G.div(l0 + rows - 1) + 1;
      je = min(jb + take, seen > 0 ? real : 0);
      if (threadIdx.x == 0 && jb == 0 && item_end > u1)   // goes on in the next part (no more pieces here)
        P.joins[blockIdx.x] = Join{row0, l0, rows, g, part_of(line, item_end - 1), first ? 0 : 1};
    }
    const int sure = base + P.by_G.div(l0);                   // every row sees the keys up to this one
    // q, on its way while the pages are looked up: column gid of tile nt is row nt * 8 + gid;
    // k-step k takes dimensions HD / 4 * q4 + 4 k .. + 3 of it
    constexpr int VEC = 16 / sizeof(T);
    uint4 raw[NT][HD / 4 / VEC];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + gid, qi = P.by_G.div(l0 + r);
      const T *src = reinterpret_cast<const T *>(P.q) + (int64_t)(row0 + qi) * P.ld_q +
                     (int64_t)(g * P.G + l0 + r - qi * P.G) * HD + q4 * (HD / 4);
#pragma unroll
      for (int i = 0; i < HD / 4 / VEC; ++i) raw[nt][i] = r < rows ? ldg16(src + i * VEC) : make_uint4(0, 0, 0, 0);
    }
    const int32_t *table = P.kv.block_table + (int64_t)s * P.kv.ld_table;

    const uint8_t *const head = pool + (int64_t)g * P.head_bytes;
    // places of this lane's 16 bytes of a stage's values and scales; a 16-byte column of
    // the values is swizzled by the key's bit 1 (see below)
    const uint32_t vdst = C::kOffV + (HD == 128 ? (lane & ~3) * 16 + ((lane & 3) ^ ((lane >> 2) & 2)) * 16 : lane * 16);
    constexpr int kHalf = C::kScales / 16;      // lanes that copy the keys' scales
    const uint8_t *const codes = head + lane * 16, *const scales = head +
        (lane < kHalf ? q4::scales_at(page_size, HD, false) + lane * 16
                      : q4::scales_at(page_size, HD, true) + (lane - kHalf) * 16);
    const int to_v = q4::codes_at(page_size, HD, true);
    // A block has 1, 2 or 4 pages (page_size >= 32, 16, 8), 2^es.  The warp reads the table
    // for 32 >> es of its blocks at once: lane i has page i mod 2^es of the (i >> es)-th,
    // -1 where there is no key or no page of the pool.
    const bool one_page = page_size >= kBN && P.kv.page_stride >> 32 == 0;
    const uint32_t stride32 = (uint32_t)P.kv.page_stride;
    const int es = shift >= 5 ? 0 : 5 - shift, batch = 32 >> es;
    int from = jb + warp, ahead = from, left_in = batch, pages, next_pages;    // from: the next block to load
    auto fetch = [&]() -> int {
      const int key = (ahead + (lane >> es) * NW) * kBN + (lane & ((1 << es) - 1)) * (kBN >> es);
      const bool there = ahead + (lane >> es) * NW < je && key < kv;
      ahead += batch * NW;
      int page = there ? __ldg(table + (key >> shift)) : -1;
      if (there && (page < 0 || page >= P.kv.n_pages)) {
        report(status, CB_ERR_DEVICE_INDEX);
        page = -1;
      }
      return page;
    };
    pages = fetch();
    next_pages = -1;                            // (a batch outlasts the prologue)
    // Loads block `from`, the batch's (batch - left_in)-th, to the stage at dst, and goes on to
    // the next.
    auto load = [&](uint32_t dst) {
      const int j = from, at = (batch - left_in) << es;       // lane of the block's first page
      const int key0 = j * kBN, left = kv - key0;             // keys from key0 on
      from += NW;
      // A whole block inside one page: everything lies at fixed distances.
      const int pg0 = __shfl_sync(0xffffffffu, pages, at);
      const int these = pages;
      if (--left_in == 0) {
        pages = next_pages;
        left_in = batch;
        next_pages = fetch();
      }
      if (one_page && left >= kBN && pg0 >= 0) {
        const int slot = key0 & (page_size - 1);
        const uint64_t off = (uint64_t)(uint32_t)pg0 * stride32;
        const uint8_t *src = codes + off + slot * (HD / 2), *vsrc = src + to_v;
#pragma unroll
        for (int i = 0; i < C::kCodes / 512; ++i) {
          copy_all(dst + lane * 16 + i * 512, src + i * 512);
          copy_all(dst + vdst + i * 512, vsrc + i * 512);
        }
        if (HD == 128 || lane < 16) copy_all(dst + C::kOffKs + lane * 16, scales + off + slot * (HD / 16));
        return;
      }
      const int page = __shfl_sync(0xffffffffu, these, at + (lane >> (5 - es)));   // of key key0 + lane
      // Codes: a warp copies 512 bytes at once, 1024 / HD keys: a group of eight
      // keys lies in one page (page_size >= 8).  The values' 16-byte columns are
      // swizzled by the key (bit 1) so that the fragments' loads meet all banks.
      constexpr int kCols = HD / 32, kKeys = 32 / kCols;
      const int crow = lane / kCols, ccol = lane % kCols;
#pragma unroll
      for (int i = 0; i < kBN / kKeys; ++i) {
        const int r = i * kKeys + crow, pg = __shfl_sync(0xffffffffu, page, kKeys == 8 ? i * 8 : r);
        const int slot = (key0 + r) & (page_size - 1);
        const bool there = pg >= 0 && r < left;
        const uint8_t *src = head + (there ? pg * P.kv.page_stride + slot * (HD / 2) + ccol * 16 : 0);
        const uint32_t d = dst + r * (HD / 2);
        copy16(d + ccol * 16, src, there);
        const int vcol = HD == 128 ? ccol ^ (r & 2) : ccol;
        copy16(d + C::kOffV + vcol * 16, src + (there ? q4::codes_at(page_size, HD, true) : 0), there);
      }
      // Scales: 16 bytes are 256 / HD keys'; lanes 0..15 the keys', 16..31 the values'.
      constexpr int kPer = 256 / HD, kChunks = kBN / kPer;    // keys a chunk; chunks
      const int c = lane & 15, r = min(c, kChunks - 1) * kPer, pg = __shfl_sync(0xffffffffu, page, r);
      if (c < kChunks) {
        const bool v = lane >= 16;
        const int slot = (key0 + r) & (page_size - 1);
        const int bytes = pg < 0 ? 0 : max(0, min(16, (left - r) * (HD / 16)));
        copy_part(dst + (v ? C::kOffVs : C::kOffKs) + c * 16,
                  head + (bytes ? pg * P.kv.page_stride + q4::scales_at(page_size, HD, v) + slot * (HD / 16) : 0), bytes);
      }
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i) {
      if (from < je) load(ring + i * C::kStage);
      commit();
    }
    next_pages = fetch();
    uint32_t qh[NT][KS][2], ql[F32 ? NT : 1][F32 ? KS : 1][2];
    float sl[NT][2];                            // log2 scale of this lane's two score columns
    int pos[NT][2];                             // their positions, -1: no row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[HD / 4];
      const T *e = reinterpret_cast<const T *>(raw[nt]);
#pragma unroll
      for (int i = 0; i < HD / 4; ++i) x[i] = to_f(e[i]);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 4; ++i) top = fmaxf(top, fabsf(x[i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int up = q4::exponent_up(top);
      const float f1 = ldexpf(1.f, up / 2), f2 = ldexpf(1.f, up - up / 2);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float y0 = x[4 * k + 2 * c] * f1 * f2, y1 = x[4 * k + 2 * c + 1] * f1 * f2;
          qh[nt][k][c] = pack_f16(y0, y1);
          if constexpr (F32) ql[nt][k][c] = pack_rest(y0, y1, qh[nt][k][c]);
        }
      // scores of this lane are of rows nt * 8 + 2 q4 and + 1, whose q lanes 8 q4 and 8 q4 + 4 have
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rc = nt * 8 + 2 * q4 + e;
        sl[nt][e] = q4::scale_down(P.scale_log2, P.scale_exp, __shfl_sync(0xffffffffu, up, 8 * q4 + 4 * e));
        pos[nt][e] = rc < rows ? base + P.by_G.div(l0 + rc) : -1;
      }
    }
    // P = 2^(x sl + shift), x the products: shift = kPShift - m sl of the reference m (before the
    // first one large, so that any product sets it)
    float o[MT][NT][4], m[NT][2], l[NT][2], shift[NT][2];
    bool scaled = false;                        // sl is less for some row (kBig)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
        shift[nt][e] = 0x1.fffffep127f;
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[t][nt][k] = 0.f;
    }
    // Rows 2 a and 2 a + 1 of a score tile's eight keys are keys a and 4 + (a ^ 1): the keys
    // whose values a lane needs then are q4 and 4 + (q4 ^ 1) of each eight, and both the
    // keys' loads (neighbouring rows) and the values' (a lane's four keys) meet all banks.
    const int krow = gid & 1 ? 4 + ((gid >> 1) ^ 1) : gid >> 1;
    const int vkey[2] = {q4, 4 + (q4 ^ 1)};
    int st = 0, fill = NS - 1;
    for (int j = jb + warp; j < je; j += NW) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
      __syncwarp();                             // landed for every lane; the stage before is used up
      if (from < je) load(ring + fill * C::kStage);
      commit();
      fill = fill + 1 == NS ? 0 : fill + 1;
      const uint32_t stage = ring + st * C::kStage;
      st = st + 1 == NS ? 0 : st + 1;
      float x[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t w[2][KW], sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = mt * 16 + 8 * h + krow;
          lds_words<KW>(stage + key * (HD / 2) + q4 * (HD / 8), w[h]);
          const uint32_t at = stage + C::kOffKs + key * (HD / 16) + q4 * (HD / 64);
          sc[h] = q4::decode_scales(HD == 128 ? lds16(at) : lds8(at));
        }
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            q4::decode8(w[h][i], a[h]);
            const uint32_t scale = q4::both(sc[h], i >= 2);
#pragma unroll
            for (int b = 0; b < 4; ++b) a[h][b] = q4::mul2(a[h][b], scale);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t f[4] = {a[0][2 * c], a[1][2 * c], a[0][2 * c + 1], a[1][2 * c + 1]};
            const int k = 2 * i + c;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (F32) {
                float t[4];
                mma_f16_new(t, f, ql[nt][k][0], ql[nt][k][1]);
                mma_f16(t, f, qh[nt][k][0], qh[nt][k][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[mt][nt][e] = k == 0 ? t[e] : x[mt][nt][e] + t[e];
              } else if (k == 0) {
                mma_f16_new(x[mt][nt], f, qh[nt][k][0], qh[nt][k][1]);
              } else {
                mma_f16(x[mt][nt], f, qh[nt][k][0], qh[nt][k][1]);
              }
            }
          }
        }
      }
      const int key0 = j * kBN;
      float mx[NT][2];
      // no masking where every row sees the block (columns without a row do not matter)
      const bool clear = key0 + kBN - 1 <= sure;
      if (!clear) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key0 + mt * 16 + (k >> 1) * 8 + krow > pos[nt][k & 1]) x[mt][nt][k] = -INFINITY;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          mx[nt][e] = fmaxf(max3(x[0][nt][e], x[0][nt][2 + e], x[1][nt][e]), x[1][nt][2 + e]);
      // The reference m stays until P of some lane would exceed its own by more than 2^kRise:
      // most blocks need no exchange between lanes (the scale is positive: the largest
      // score is the largest product).
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) over |= fmaf(mx[nt][e], sl[nt][e], shift[nt][e]) > kPShift + kRise;
      if (__any_sync(0xffffffffu, over)) {
        bool far = scaled;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], d));
            const float mn = fmaxf(m[nt][e], mx[nt][e]);
            const float corr = mn == m[nt][e] ? 1.f : ex2((m[nt][e] - mn) * sl[nt][e]);    // also where both are -inf
            m[nt][e] = mn;
            if (mn != -INFINITY) {
              const float score = mn * sl[nt][e];
              shift[nt][e] = kPShift - score;
              far |= fabsf(score) > kBig;
            }
            l[nt][e] *= corr;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              o[t][nt][e] *= corr;
              o[t][nt][2 + e] *= corr;
            }
          }
        if (__any_sync(0xffffffffu, far)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float &whole = s_sl[warp * R + nt * 8 + 2 * q4 + e];   // (a lane reads what it wrote)
              if (!scaled) whole = sl[nt][e];
              sl[nt][e] = whole;
              if (m[nt][e] != -INFINITY) {
                if (fabsf(m[nt][e] * whole) > kBig) sl[nt][e] = __fdividef(kBig, fabsf(m[nt][e]));
                shift[nt][e] = kPShift - m[nt][e] * sl[nt][e];
              }
            }
          scaled = true;
        }
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t ph[NT][2], pl[F32 ? NT : 1][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              p[e] = ex2(fmaf(x[mt][nt][2 * h + e], sl[nt][e], shift[nt][e]));   // 0 where masked
              l[nt][e] += p[e];
            }
            const uint32_t hi = pack_f16(p[0], p[1]);
            ph[nt][h] = transposed(hi);
            if constexpr (F32) pl[nt][h] = transposed(pack_rest(p[0], p[1], hi));
          }
        // values of the lane's four keys; pairs (i = 0, 1) and (2, 3)
        uint32_t w[4][VW], sc[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = mt * 16 + 8 * (i >> 1) + vkey[i & 1];
          const int col = HD == 128 ? ((gid >> 1) ^ (key & 2)) * 16 + (gid & 1) * 8 : gid * 4;
          lds_words<VW>(stage + C::kOffV + key * (HD / 2) + col, w[i]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = stage + C::kOffVs + (mt * 16 + 8 * h) * (HD / 16) + gid * HD / 128;
          sc[h] = q4::decode_scales(__byte_perm(lds8(at + vkey[0] * (HD / 16)), lds8(at + vkey[1] * (HD / 16)), 0x0040));
        }
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          uint32_t even[2][4], odd[2][4];       // pairs of keys, of dimensions 2 t and 2 t + 1
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a = w[2 * h][i], b = w[2 * h + 1][i];
            q4::decode8((a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u), even[h]);
            q4::decode8(((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u), odd[h]);
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t f[4] = {q4::mul2(even[0][t], sc[0]), q4::mul2(odd[0][t], sc[0]),
                                   q4::mul2(even[1][t], sc[1]), q4::mul2(odd[1][t], sc[1])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float (&acc)[4] = o[i * 4 + t][nt];
              if constexpr (F32) {
                float c[4];
                mma_f16_new(c, f, pl[nt][0], pl[nt][1]);
                mma_f16(c, f, ph[nt][0], ph[nt][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] += c[e];
              } else {
                mma_f16(acc, f, ph[nt][0], ph[nt][1]);
              }
            }
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
        if (gid == 0) s_ml[warp * R + nt * 8 + 2 * q4 + e] =
              make_float2(m[nt][e] * (scaled ? s_sl[warp * R + nt * 8 + 2 * q4 + e] : sl[nt][e]), l[nt][e]);
      }
    __syncthreads();                            // the rings are used up
    // Every warp leaves its O in rows of HD + 4 floats, then the four states join.
    constexpr int LD = HD + 4;
    static_assert(NW * R * LD * 4 <= C::kSmem, "the warps' O fit the rings");
    float *so = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2 *>(so + (warp * R + nt * 8 + 2 * q4 + e) * LD + gid * (HD / 8) + 2 * t) =
              make_float2(o[t][nt][e], o[t][nt][2 + e]);
    __syncthreads();
    const int64_t slot = (2 * (int64_t)blockIdx.x + (first ? 0 : 1)) * R;
    // an output's four columns, divided by the sum
    auto write = [&](int r, int c, float4 a, float L) {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const int qi = P.by_G.div(l0 + r);
      T *dst = reinterpret_cast<T *>(P.out) + (int64_t)(row0 + qi) * P.ld_out +
               (int64_t)(g * P.G + l0 + r - qi * P.G) * HD + c;
      if constexpr (F32)
        *reinterpret_cast<float4 *>(dst) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
      else
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
    };
    for (int i = threadIdx.x; i < rows * (HD / 4); i += C::kThreads) {
      const int r = i / (HD / 4), c = i % (HD / 4) * 4;
      float M = -INFINITY, L = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < NW; ++k) M = fmaxf(M, s_ml[k * R + r].x);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float2 ml = s_ml[k * R + r];
        const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
        const float4 v = *reinterpret_cast<const float4 *>(so + (k * R + r) * LD + c);
        L += w * ml.y;
        a.x += w * v.x; a.y += w * v.y; a.z += w * v.z; a.w += w * v.w;
      }
      a.x *= P.v_mul; a.y *= P.v_mul; a.z *= P.v_mul; a.w *= P.v_mul;
      if constexpr (CL) {
        *reinterpret_cast<float4 *>(s_part + r * HD + c) = a;
        if (c == 0) s_pml[r] = make_float2(M, L);
      } else if (!whole) {
        *reinterpret_cast<float4 *>(P.part_o + (slot + r) * HD + c) = a;
        if (c == 0) P.part_ml[slot + r] = make_float2(M, L);
      } else {
        write(r, c, a, L);
      }
    }
    if constexpr (CL) cluster_join<C::kThreads, HD>(s_part, s_pml, rows, rank, ranks, write);
    __syncthreads();                            // before the next piece fills the rings
  }
}

// ------------------------------------------------------------------ plan --
struct Plan {
  int nt, grid;                         // few-rows kernel: score columns / 8 per tile (0: not launched), blocks
  int cluster;                          // blocks of a tile's cluster, 0: the line
  int few_hi, rows_lo;                  // which sequences each kernel takes
  ChunkPlan chunk;                      // R 0: not launched
};

// bf16: sequences of up to few_rows rows (queries x G) go through the few-rows kernel,
// longer ones through the chunk kernel, which is made for 128 rows; fp32 runs the
// few-rows kernel alone.  At head_dim 128, 64 x 32 rows over 4096 keys take 177 us so and 266
// by the chunk kernel, 48 rows 365 (in tiles of 32) and 271; at 64, where the chunk kernel's
// softmax has half the products to hide behind, 16 x 36 or 64 rows over 8192 keys take 84
// and 87 against 106 and 98 (one sequence of 64 rows over 4096 keys 15 against 17.5).
static int few_rows(int hd) { return hd == 64 ? 64 : 32; }

// Attributes of a form of the kernel.
template <typename T, int HD, int NT, bool CL> static cudaError_t set_attributes() {
  typedef Cfg<HD, NT, std::is_same<T, float>::value, CL> C;
  const cudaError_t e =
      cudaFuncSetAttribute(paged4_few_kernel<T, HD, NT, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  return e != cudaSuccess || !CL
      ? e : cudaFuncSetAttribute(paged4_few_kernel<T, HD, NT, CL>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

template <typename T, int HD, int NT> static const int *cluster_room_of() {
  typedef Cfg<HD, NT, std::is_same<T, float>::value, true> C;
  static ClusterRoom room;
  return room.of(paged4_few_kernel<T, HD, NT, true>, C::kThreads, C::kSmem, set_attributes<T, HD, NT, true>);
}
static const int *cluster_room_of(int nt, int hd, cb_dtype dt) {
  if (dt == CB_F32) {
    if (nt == 1) return hd == 128 ? cluster_room_of<float, 128, 1>() : cluster_room_of<float, 64, 1>();
    return hd == 128 ? cluster_room_of<float, 128, 2>() : cluster_room_of<float, 64, 2>();
  }
  if (nt == 1) return hd == 128 ? cluster_room_of<bf16, 128, 1>() : cluster_room_of<bf16, 64, 1>();
  if (nt == 2) return hd == 128 ? cluster_room_of<bf16, 128, 2>() : cluster_room_of<bf16, 64, 2>();
  return hd == 128 ? cluster_room_of<bf16, 128, 4>() : cluster_room_of<bf16, 64, 4>();
}

static Plan plan(int64_t n_rows, int S, int max_kv, int G, int Hkv, int hd, cb_dtype dt) {
  Plan p = {};
  const int64_t all = n_rows * G, per_seq = (all + S - 1) / S;
  const bool few = dt == CB_F32 || all <= few_rows(hd) || n_rows <= S;
  p.few_hi = 0x7fffffff;
  // Tiles of 32 rows read the keys less often and leave two blocks an SM: bf16, 64 sequences
  // of 32 rows over 4096 keys 188 us, 177 with tiles of 16; at head_dim 64, 48 rows 169 and
  // 163, 64 rows 173 and 207 (on the line; in a cluster 64 rows over 4096 keys take 15.4 with
  // tiles of 32 and 9.9 with 16: the rule does not look).  In fp32 they do not fit the registers (256 rows over 8192 keys
  // 387 us, 266 with tiles of 16).
  if (few || S > 1)
    p.nt = per_seq <= 8 ? 1 : per_seq <= 48 || dt == CB_F32 ? 2 : few || per_seq <= few_rows(hd) ? 4 : 1;
  p.grid = device_sm_count() * (p.nt == 4 || dt == CB_F32 ? 2 : p.nt == 2 ? 3 : 4);
  if (few) {
    // few tiles over few keys: each tile's keys go to one cluster of up to 16 blocks, which
    // joins in its shared memory: one launch in place of two (counted is one tile for
    // every sequence at least; clusters of tiles that there are not leave at once)
    const int64_t full = (all + 8 * p.nt - 1) / (8 * p.nt), seqs = S < n_rows ? S : n_rows;
    p.cluster = plan_cluster((full > seqs ? full : seqs) * Hkv, max_kv > 0 ? (max_kv + kBN - 1) / kBN : 1,
                             device_sm_count(), p.nt == 1 && dt == CB_BF16 ? 2 : 1, p.grid, 16, cluster_room_of(p.nt, hd, dt));
    return p;
  }
  if (S > 1) p.few_hi = p.rows_lo = few_rows(hd);
  p.chunk = plan_chunk(n_rows, S, max_kv, G, Hkv, hd);
  return p;
}
static int64_t few_partials(const Plan &p) { return p.nt && !p.cluster ? 2LL * p.grid * 8 * p.nt : 0; }
static int64_t chunk_partials(const Plan &p, int Hkv) {
  return p.chunk.R && p.chunk.n_split > 1 ? p.chunk.units * Hkv * p.chunk.n_split * p.chunk.R : 0;
}
static size_t plan_bytes(const Plan &p, int Hkv, int hd) {
  const size_t row = hd * sizeof(float) + sizeof(float2);
  const size_t few = (size_t)few_partials(p) * row + (p.nt && !p.cluster ? p.grid * sizeof(Join) : 0);
  const size_t chunk = (size_t)chunk_partials(p, Hkv) * row;
  return few > chunk ? few : chunk;
}

template <typename T, int HD, int NT, bool CL>
static cudaError_t run(const Params &P, const Plan &p, int *status, cudaStream_t s) {
  typedef Cfg<HD, NT, std::is_same<T, float>::value, CL> C;
  static PerDeviceOnce attr;
  cudaError_t e = attr.run([](int) { return set_attributes<T, HD, NT, CL>(); });
  if (e != cudaSuccess) return e;
  if constexpr (CL) {
    const int64_t blocks = tile_bound(P.n_rows, P.kv.n_seq, P.G, C::kRows) * P.Hkv * p.cluster;
    e = launch_clusters(paged4_few_kernel<T, HD, NT, CL>, dim3((unsigned)blocks), dim3(C::kThreads), p.cluster, C::kSmem, s,
                        P, status);
    return e == cudaSuccess ? launched(1) : e;
  } else {
    e = launch_pdl(paged4_few_kernel<T, HD, NT, CL>, dim3(p.grid), dim3(kDecThreads), C::kSmem, s, P, status);
    if (e != cudaSuccess) return e;
    e = launch_pdl(decode_merge_kernel<T, HD>, dim3(p.grid, C::kRows / kJoinRows), dim3(kJoinThreads),
                   p.grid * kJoinRows * sizeof(float2), s, P, C::kRows);
    return e == cudaSuccess ? launched(2) : e;
  }
}

template <typename T, int HD, int NT>
static cudaError_t run_form(const Params &P, const Plan &p, int *status, cudaStream_t s) {
  return p.cluster ? run<T, HD, NT, true>(P, p, status, s) : run<T, HD, NT, false>(P, p, status, s);
}
template <typename T, int HD>
static cudaError_t run_rows(const Params &P, const Plan &p, int *status, cudaStream_t s) {
  if constexpr (std::is_same<T, bf16>::value)
    if (p.nt == 4) return run_form<T, HD, 4>(P, p, status, s);
  return p.nt == 1 ? run_form<T, HD, 1>(P, p, status, s) : run_form<T, HD, 2>(P, p, status, s);
}

}  // namespace paged4

size_t paged4_attention_ws_bytes(int n_rows, int n_seq, int max_kv, int Hq, int Hkv, int hd, cb_dtype dt) {
  if (n_rows <= 0 || n_seq <= 0) return 0;
  return paged4::plan_bytes(paged4::plan(n_rows, n_seq, max_kv, Hq / Hkv, Hkv, hd, dt), Hkv, hd);
}

void paged4_attention_plan(int n_rows, int n_seq, int max_kv, int Hq, int Hkv, int hd, cb_dtype dt, int64_t out[6]) {
  const paged4::Plan p = paged4::plan(n_rows, n_seq, max_kv, Hq / Hkv, Hkv, hd, dt);
  const int64_t v[6] = {8 * p.nt, p.cluster, p.grid, p.chunk.R, p.chunk.n_split, p.nt ? p.few_hi : 0};
  for (int i = 0; i < 6; ++i) out[i] = v[i];
}

cudaError_t launch_paged4_attention(const cb_paged4_kv &kv, const cb_paged_query &a, cb_dtype dt, int *status,
                                    cudaStream_t s) {
  using namespace paged4;
  const int G = a.n_q_heads / a.n_kv_heads;
  const Plan p = plan(a.n_rows, kv.n_seq, a.max_kv_len, G, a.n_kv_heads, a.head_dim, dt);
  if (p.chunk.units * a.n_kv_heads * p.chunk.n_split > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  Params P;
  P.kv = paged4_plain_kv(kv);
  P.q = a.q;
  P.out = a.out;
  P.ld_q = a.ld_q;
  P.ld_out = a.ld_out;
  P.n_rows = a.n_rows;
  P.G = G;
  P.Hkv = a.n_kv_heads;
  P.max_kv = a.max_kv_len;
  P.pad = kPad;
  P.n_split = p.chunk.n_split;
  P.few_hi = p.few_hi;
  P.rows_lo = p.rows_lo;
  P.hc = 1;
  P.by_G = Divisor(G);
  P.by_quads = Divisor(a.n_kv_heads);
  P.scale_log2 = frexpf(a.scale, &P.scale_exp) * 1.4426950408889634f;
  P.scale_exp += kv.k_exp;
  P.head_bytes = q4::head_bytes(kv.page_size, a.head_dim);
  P.v_mul = ldexpf(1.f, kv.v_exp);
  // the partials of a launch reuse the workspace of the one before it: each waits for its
  // predecessor's end
  auto bind = [&](int64_t partials) {
    P.part_o = reinterpret_cast<float *>(a.ws);
    P.part_ml = reinterpret_cast<float2 *>(P.part_o + partials * a.head_dim);
    P.joins = reinterpret_cast<Join *>(P.part_ml + partials);
  };
  if (p.nt) {
    bind(few_partials(p));
    cudaError_t e;
    if (dt == CB_BF16)
      e = a.head_dim == 128 ? run_rows<bf16, 128>(P, p, status, s) : run_rows<bf16, 64>(P, p, status, s);
    else
      e = a.head_dim == 128 ? run_rows<float, 128>(P, p, status, s) : run_rows<float, 64>(P, p, status, s);
    if (e != cudaSuccess) return e;
  }
  if (!p.chunk.R) return cudaSuccess;
  bind(chunk_partials(p, a.n_kv_heads));
  return launch_chunk(P, p.chunk.R, p.chunk.units, a.head_dim, status, s, true);
}

}  // namespace cb
