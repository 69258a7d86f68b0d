// bf16 paged attention of many rows per sequence on the tensor cores
// (tcgen05): chunks of a prompt over what the cache holds.
//
// Work unit: NT tiles of 128 rows of one sequence and kv head (row l is query
// l / G, head l % G of the group, so any group size fills the tiles) and,
// where the units alone do not fill the SMs, a part of their key range.  Units
// of a sequence are taken last first: they see the most keys.
//
// NT = 2, one CTA per SM: two tiles share every K and V block, so a block is
// fetched once for 256 rows and four stages fit; a unit of up to 128 rows runs
// its first tile alone.  NT = 1: two CTAs per SM with two stages each, for calls
// whose units of 256 rows would leave SMs empty or tiles without rows.  The cost
// model in plan_chunk picks NT for a call.
//
// Roles: producer warps fill the 64-key K and V stages; one MMA warp per tile
// owns 256 TMEM columns and issues tcgen05.mma: S_j = Q K_j^T into columns
// 0..63 and O += P_j V_j into columns 128.., P_j read from TMEM (columns 64..95
// or 96..127 by the parity of j); four warps per tile load Q, then do the
// online softmax, one row per thread, in the log2 domain and store P_j as
// packed bf16.  S_{j+1} is issued as soon as the softmax has taken S_j into
// registers, so it is computed while the softmax works, and P V of block j
// while the softmax is at block j + 1; with P in columns of its own neither
// product waits for the other.  (With P_j over S_j and two S slots instead,
// S_{j+1} had to wait for P_{j-1} V_{j-1}, and a block took 2100 cycles.)  The
// row's reference maximum m only moves when a block raises it by more than
// 2^kChRescale: then O (after P_{j-1} V_{j-1} has landed) and l are scaled by
// 2^(m_old - m_new); O / l does not depend on m.
//
// Keys and values come by 16-byte cp.async to their swizzled places, each
// eight rows of one page together, with zeros for keys past the cached length
// (an unwritten slot may hold NaN, and 0 * NaN would reach O).  A TMA box
// would be a page's rows: at 16 slots a page sixteen boxes per block, about
// 90 ns each, twice what the block's arithmetic takes.
//
// Parts of a split key range leave (O, m, l) in fp32 for chunk_merge_kernel.
// All waits are bounded.
//
// Measured: four chunks of 2048 rows over 8192 keys, 32/8 heads of 128: 760 to 785
// us on several GPUs, 1225 to 1266 TFLOP/s.  A 64-key block of 256 rows takes 1668 cycles: the tensor pipe's
// two S (about 500 each; N = 64 reads Q again for every 64 keys) and two P V (256)
// are 1512 of them, the softmax alone takes 1500.  S of 128 keys would halve its
// cost, but two tiles of 128 score and 128 output columns leave P no place of its
// own, and with P over S the chain through P V is longer than what it saves (804 us
// where this form took 762).
#include <type_traits>

#include "cb_attn_tc.cuh"
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged.cuh"
#include "cb_paged_attn.cuh"

namespace cb {
namespace paged {

using namespace attn;

constexpr int kChBN = 64;                 // keys per block
constexpr float kChRescale = 8.f;         // log2 of the largest p between rescales
constexpr int kChTmem = 256, kChP = 64, kChO = 128;   // columns per tile: S from 0, P_0, P_1 (32 each), O

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}

template <int HD, int NT> struct ChCfg {
  static constexpr int kRows = 128 * NT, kPerSm = NT == 1 ? 2 : 1;
  static constexpr int kStages = NT == 1 ? 2 : 4, kProd = NT;   // producer warps each for K and V
  // warps: K producers, V producers, MMA, (idle), softmax from a multiple of 4
  static constexpr int kMma = 2 * kProd, kSoft = (kMma + NT + 3) / 4 * 4, kThreads = 32 * (kSoft + 4 * NT);
  static constexpr int kAtom = 128 * 128;            // [128 rows x 64 dims], 128-byte swizzle
  static constexpr int kAtomKV = kChBN * 128;        // [64 keys x 64 dims]
  static constexpr int kQ = kAtom * (HD / 64), kKV = kAtomKV * (HD / 64);
  static constexpr int kOffK = NT * kQ, kOffV = kOffK + kStages * kKV, kOffBar = kOffV + kStages * kKV;
  static constexpr int kSmem = kOffBar + 512 + 1024;
};

// Fills one K or V stage: 64 keys of one head.  Lane = (row of 32 / cols,
// 16-byte column); eight consecutive keys share a page (page_size >= 8), so a
// group of eight rows is one page lookup and steps of a constant stride.
// ALL: every key exists and every page is valid.
template <int HD, bool ALL>
__device__ __forceinline__ void chunk_load(uint32_t dst, const bf16 *pool, const PagedKV &kv, int key0, int n_keys,
                                           int page_lo, int page_hi, int lane) {
  constexpr int kCols = HD / 8, kRows = 32 / kCols;
  const int crow = lane / kCols, col = lane % kCols;
  const int64_t step = (int64_t)kRows * kv.ld;
  pool += (int64_t)crow * kv.ld + col * 8;
  uint32_t at[8 / kRows];
#pragma unroll
  for (int i = 0; i < 8 / kRows; ++i) {
    const int r = i * kRows + crow;
    at[i] = dst + (col >> 3) * (kChBN * 128) + r * 128 + (((col ^ r) & 7) << 4);
  }
#pragma unroll
  for (int g8 = 0; g8 < kChBN / 8; ++g8) {
    const int page = __shfl_sync(0xffffffffu, g8 < 4 ? page_lo : page_hi, (g8 & 3) * 8);
    const int slot = (key0 + g8 * 8) & (kv.page_size - 1);
    const bf16 *src = pool + (ALL || page >= 0 ? (int64_t)page * kv.page_stride + (int64_t)slot * kv.ld : 0);
#pragma unroll
    for (int i = 0; i < 8 / kRows; ++i) {
      if (ALL) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at[i] + g8 * 1024), "l"(src) : "memory");
      } else {
        // a row past the cached length, or of a bad page: zeros, nothing read
        const bool there = page >= 0 && g8 * 8 + i * kRows + crow < n_keys;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at[i] + g8 * 1024),
                     "l"(there ? src : pool), "r"(there ? 16 : 0)
                     : "memory");
      }
      src += step;
    }
  }
}

template <int HD, int NT>
__global__ void __launch_bounds__(ChCfg<HD, NT>::kThreads, ChCfg<HD, NT>::kPerSm)
paged_chunk_kernel(const __grid_constant__ AttnParams P, int *status) {
  typedef ChCfg<HD, NT> C;
  constexpr int NS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
  uint64_t *k_full = bar;                      // [NS] K_j landed
  uint64_t *k_empty = k_full + NS;             // [NS] every tile's S_j = Q K_j^T done with K_j
  uint64_t *v_full = k_empty + NS;             // [NS] V_j landed
  uint64_t *v_empty = v_full + NS;             // [NS] every tile's P_j V_j done with V_j
  uint64_t *q_full = v_empty + NS;             // [NT]
  uint64_t *s_full = q_full + NT;              // [NT] S_j in TMEM
  uint64_t *s_read = s_full + NT;              // [NT] S_j in the softmax's registers
  uint64_t *p_full = s_read + NT;              // [NT][2] P_j in its columns (and O rescaled)
  uint64_t *pv_done = p_full + 2 * NT;         // [NT][2] O += P_j V_j has landed
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(pv_done + 2 * NT);
  volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert(8 * (4 * NS + 7 * NT) + 8 <= 512, "barriers fit");
  __shared__ PagedTile s_tile;
  __shared__ int s_sums[C::kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  const int split = blockIdx.x % P.n_split, g = blockIdx.x / P.n_split % P.Hkv;
  const int tile = blockIdx.x / P.n_split / P.Hkv;
  paged_find_tile<C::kThreads>(P.kv, P.n_rows, P.G, C::kRows, P.max_kv, tile, &s_tile, s_sums, status, P.rows_lo);
  const PagedTile tl = s_tile;
  if (tl.s < 0) return;
  const int l0 = tl.t * C::kRows, rows = min(C::kRows, tl.n * P.G - l0);
  const int active = NT == 1 || rows <= 128 ? 1 : 2;           // tiles with rows
  const int base = tl.kv - tl.n;
  const int last = base + P.by_G.div(l0 + rows - 1);
  const int nb_tile = last < 0 ? 0 : last / kChBN + 1;
  const int jb = (int)((int64_t)nb_tile * split / P.n_split);
  const int nb = (int)((int64_t)nb_tile * (split + 1) / P.n_split) - jb;
  const int64_t slot0 = ((int64_t)(tile * P.Hkv + g) * P.n_split + split) * C::kRows;
  if (nb == 0) {
    // no key of this part is seen: an empty partial, or rows of zeros
    if ((int)threadIdx.x < rows) {
      if (P.n_split > 1) {
        P.part_ml[slot0 + threadIdx.x] = make_float2(-INFINITY, 0.f);
      } else {
        const int l = l0 + threadIdx.x, qi = P.by_G.div(l);
        uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<bf16 *>(P.out) +
                                               (int64_t)(tl.row0 + qi) * P.ld_out +
                                               (int64_t)(g * P.G + l - qi * P.G) * HD);
        for (int c = 0; c < HD / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&k_full[i]), 32);
      mbar_init(smem_u32(&k_empty[i]), active);
      mbar_init(smem_u32(&v_full[i]), 32);
      mbar_init(smem_u32(&v_empty[i]), active);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(smem_u32(&q_full[i]), 128);
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_read[i]), 128);
    }
    for (int i = 0; i < 2 * NT; ++i) {
      mbar_init(smem_u32(&p_full[i]), 128);
      mbar_init(smem_u32(&pv_done[i]), 1);
    }
    *fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::kMma) tcx::tmem_alloc(smem_u32(tmem_slot), NT * kChTmem);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_launch();                           // after the allocation (see cb_common.cuh)
  auto proxy_fence = [] { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); };

  if (warp < 2 * C::kProd) {
    // ------------------------------------------- producers (K, then V warps)
    const bool is_v = warp >= C::kProd;
    const int first = warp % C::kProd;           // this warp's blocks: first, first + kProd, ..
    uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
    const bf16 *pool = reinterpret_cast<const bf16 *>(is_v ? P.kv.v_pages : P.kv.k_pages) + (int64_t)g * HD;
    const uint32_t dst = smem_u32(smem + (is_v ? C::kOffV : C::kOffK));
    const int32_t *table = P.kv.block_table + (int64_t)tl.s * P.kv.ld_table;
    const int shift = __ffs(P.kv.page_size) - 1;
    auto fetch = [&](int key) -> int {           // the page of a key, -1: none
      return key < tl.kv ? __ldg(table + (key >> shift)) : -1;
    };
    auto checked = [&](int page, int key) -> int {
      if (page >= 0 && page < P.kv.n_pages) return page;
      if (key < tl.kv) report(status, CB_ERR_DEVICE_INDEX);
      return -1;
    };
    int lo = fetch((jb + first) * kChBN + lane), hi = fetch((jb + first) * kChBN + 32 + lane);
    // Two loads are in flight: a block is handed over (its bytes fenced for
    // the tensor core) after the warp's next one has been issued, or at once
    // where the next one's stage is still in use.
    int open = -1;                               // block issued but not handed over
    auto hand_over = [&] {
      proxy_fence();
      arrive(smem_u32(&full[open % NS]));
      open = -1;
    };
    for (int j = first; j < nb; j += C::kProd) {
      const int sl = j % NS, key0 = (jb + j) * kChBN;
      const uint32_t eb = smem_u32(&empty[sl]), ph = ((j / NS) & 1) ^ 1;
      if (open >= 0 && !__all_sync(0xffffffffu, mbar_test(eb, ph))) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        hand_over();
      }
      const bool ok = mbar_wait_bounded(eb, ph, kWaitLimitNs, status);
      if (__any_sync(0xffffffffu, !ok || *fail)) {
        *fail = 1;
        break;
      }
      lo = checked(lo, key0 + lane);
      hi = checked(hi, key0 + 32 + lane);
      if (__all_sync(0xffffffffu, lo >= 0 && hi >= 0))
        chunk_load<HD, true>(dst + sl * C::kKV, pool, P.kv, key0, kChBN, lo, hi, lane);
      else
        chunk_load<HD, false>(dst + sl * C::kKV, pool, P.kv, key0, tl.kv - key0, lo, hi, lane);
      asm volatile("cp.async.commit_group;" ::: "memory");
      lo = fetch(key0 + C::kProd * kChBN + lane);
      hi = fetch(key0 + C::kProd * kChBN + 32 + lane);
      if (open >= 0) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        hand_over();
      }
      open = j;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (open >= 0) hand_over();
  } else if (warp >= C::kMma && warp < C::kMma + active) {
    // ----------------------------------------------------- MMA, one per tile
    const int t = warp - C::kMma;
    const uint32_t idS = idesc(false, kChBN), idPV = idesc(true, HD);
    const uint32_t q_addr = smem_u32(smem + t * C::kQ), tm = tmem + t * kChTmem;
    uint64_t *const sf = s_full + t, *const sr = s_read + t, *const pf = p_full + 2 * t, *const pd = pv_done + 2 * t;
    auto wait_all = [&](uint64_t *b, uint32_t ph) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(b), ph, kWaitLimitNs, status));
    };
    bool ok = wait_all(q_full + t, 0);
    auto issue_s = [&](int j) -> bool {
      const int st = j % NS;
      if (!wait_all(&k_full[st], (j / NS) & 1)) return false;
      if (j >= 1 && !wait_all(sr, (j & 1) ^ 1)) return false;   // S_{j-1} has been read
      fence_after();
      if (tcx::elect_one()) {
        const uint32_t k_addr = smem_u32(smem + C::kOffK + st * C::kKV);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t qo = (k >> 2) * C::kAtom + (k & 3) * 32;
          const uint32_t ko = (k >> 2) * C::kAtomKV + (k & 3) * 32;
          mma(tm, desc_kmajor(q_addr + qo), desc_kmajor(k_addr + ko), idS, k > 0);
        }
        commit(smem_u32(sf));
        commit(smem_u32(&k_empty[st]));
      }
      __syncwarp();
      return true;
    };
    if (ok) ok = issue_s(0);
    for (int j = 0; j < nb && ok; ++j) {
      if (__any_sync(0xffffffffu, *fail != 0)) break;
      const int sl = j & 1, st = j % NS;
      if (j + 1 < nb && !issue_s(j + 1)) { ok = false; break; }
      if (!wait_all(&pf[sl], (j >> 1) & 1) || !wait_all(&v_full[st], (j / NS) & 1)) {
        ok = false;
        break;
      }
      fence_after();
      if (tcx::elect_one()) {
        const uint32_t v_addr = smem_u32(smem + C::kOffV + st * C::kKV);
#pragma unroll
        for (int k = 0; k < kChBN / 16; ++k)
          mma_ts(tm + kChO, tm + kChP + sl * 32 + k * 8, desc_mnmajor(v_addr + k * 16 * 128, C::kAtomKV), idPV,
                 (j > 0 || k > 0) ? 1u : 0u);
        commit(smem_u32(&pd[sl]));
        commit(smem_u32(&v_empty[st]));
      }
      __syncwarp();
    }
    if (!ok && lane == 0) *fail = 1;
  } else if (warp >= C::kSoft && warp < C::kSoft + 4 * active) {
    // ------------------------------------------------------ Q, then softmax
    const int t = (warp - C::kSoft) / 4;
    uint64_t *const sf = s_full + t, *const sr = s_read + t, *const pf = p_full + 2 * t, *const pd = pv_done + 2 * t;
    {
      // a thread loads its row: all its loads are in flight at once, and eight
      // neighbouring rows fall into different banks
      const int r = threadIdx.x - 32 * C::kSoft, l = l0 + r, qi = P.by_G.div(l);
      const bf16 *q = reinterpret_cast<const bf16 *>(P.q) + (int64_t)(tl.row0 + qi) * P.ld_q +
                      (int64_t)(g * P.G + l - qi * P.G) * HD;
      uint4 v[HD / 8];
#pragma unroll
      for (int c = 0; c < HD / 8; ++c)
        v[c] = r < rows ? *reinterpret_cast<const uint4 *>(q + c * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < HD / 8; ++c)
        *reinterpret_cast<uint4 *>(smem + t * C::kQ + (c >> 3) * C::kAtom + (r & 127) * 128 +
                                   (((c ^ r) & 7) << 4)) = v[c];
      proxy_fence();
      arrive(smem_u32(q_full + t));
    }
    const int quad = warp & 3;
    const int row = t * 128 + quad * 32 + lane;  // row of the unit
    const bool valid = row < rows;
    const int p = valid ? base + P.by_G.div(l0 + row) : -1;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tm = tmem + t * kChTmem + lane_off, obase = tm + kChO;
    float m = -INFINITY, l = 0.f;                // reference max (log2 domain), sum
    const float sl2 = P.scale_log2;
    bool failed = false;
    auto pv_landed = [&](int j) -> bool {
      const bool bad = !mbar_wait_bounded(smem_u32(&pd[j & 1]), (j >> 1) & 1, kWaitLimitNs, status);
      if (__any_sync(0xffffffffu, bad)) return false;
      fence_after();
      return true;
    };
    for (int j = 0; j < nb; ++j) {
      const int sl = j & 1;
      // (a failure elsewhere is met here as a wait that runs out: polling the
      // flag would put another shared-memory read on every block's path)
      const bool bad = !mbar_wait_bounded(smem_u32(sf), j & 1, kWaitLimitNs, status);
      if (__any_sync(0xffffffffu, bad)) { failed = true; break; }
      fence_after();
      const int key0 = (jb + j) * kChBN;
      const int n_vis = p - key0 + 1;            // keys of the block this row sees; >= 64: no masking
      float x[kChBN];
      ld32_nw(tm, x);
      ld32_nw(tm + 32, x + 32);
      wait_ld();
      fence_before();
      arrive(smem_u32(sr));
      float mx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) mx[i] = -INFINITY;
      if (n_vis >= kChBN) {
#pragma unroll
        for (int i = 0; i < kChBN; i += 8) {
          mx[0] = max3(mx[0], x[i], x[i + 1]);
          mx[1] = max3(mx[1], x[i + 2], x[i + 3]);
          mx[2] = max3(mx[2], x[i + 4], x[i + 5]);
          mx[3] = max3(mx[3], x[i + 6], x[i + 7]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kChBN; ++i)
          if (i < n_vis) mx[i & 3] = fmaxf(mx[i & 3], x[i]);
      }
      const float mloc = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
      // move the reference only for a large rise; the first visible key
      // always sets it (m = -inf before)
      const bool move = mloc > m + kChRescale;
      const bool rescale = move && m != -INFINITY;   // O and l hold earlier blocks
      if (__any_sync(0xffffffffu, rescale) && j > 0) {
        // O must hold P_{j-1} V_{j-1} first; rows that keep m scale by 1
        if (!pv_landed(j - 1)) { failed = true; break; }
        const float corr = rescale ? fast_exp2(m - mloc) : 1.f;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float y[32];
          ld32(obase + c, y);
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] *= corr;
          st32(obase + c, y);
        }
        l *= corr;
      }
      if (move) m = mloc;
      // P_j for keys c..c+31 -> columns c/2 .. c/2+15; the scale-and-shift and
      // the sums run on packed pairs.  The columns held P_{j-2}: S_j was
      // issued after P_{j-2} V_{j-2} and its commit covers what came before,
      // so that product is done.
      const unsigned long long s2 = pack2(sl2, sl2), nm2 = pack2(-m, -m);
      unsigned long long ls2[2] = {0ull, 0ull};
      auto exps = [&](auto masked) {
#pragma unroll
        for (int c = 0; c < kChBN; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const unsigned long long a = fma2(pack2(x[c + i], x[c + i + 1]), s2, nm2);
            float p0 = fast_exp2(lo2(a));
            float p1 = fast_exp2(hi2(a));
            if (decltype(masked)::value) {
              p0 = c + i < n_vis ? p0 : 0.f;
              p1 = c + i + 1 < n_vis ? p1 : 0.f;
            }
            ls2[(i >> 1) & 1] = add2(ls2[(i >> 1) & 1], pack2(p0, p1));
            __nv_bfloat162 v2 = __floats2bfloat162_rn(p0, p1);
            pk[i / 2] = *reinterpret_cast<uint32_t *>(&v2);
          }
          st16(tm + kChP + sl * 32 + c / 2, pk);
        }
      };
      // most blocks lie wholly before every row of the warp: no selects there
      if (__all_sync(0xffffffffu, n_vis >= kChBN)) exps(std::false_type{});
      else exps(std::true_type{});
      wait_st();
      l += (lo2(ls2[0]) + hi2(ls2[0])) + (lo2(ls2[1]) + hi2(ls2[1]));
      fence_before();
      arrive(smem_u32(&pf[sl]));
    }
    // the whole key range is in O once the last P V has landed
    if (!failed && !pv_landed(nb - 1)) failed = true;
    if (failed) *fail = 1;
    const bool ok = !failed && !*fail;
    if (__any_sync(0xffffffffu, ok)) {
      const int lr = l0 + row, qi = P.by_G.div(lr);
      const float inv = l == 0.f ? 0.f : 1.f / l;    // no visible key: zeros
      bf16 *out = reinterpret_cast<bf16 *>(P.out) + (int64_t)(tl.row0 + qi) * P.ld_out +
                  (int64_t)(g * P.G + lr - qi * P.G) * HD;
      // partials lie four columns of all the unit's rows together, which a warp with
      // a row per lane writes (and the merge reads) in whole lines
      float4 *part = reinterpret_cast<float4 *>(P.part_o + slot0 * HD) + row;
#pragma unroll 1
      for (int c = 0; c < HD; c += 32) {
        float o[32];
        ld32(obase + c, o);
        if (!(valid && ok)) continue;
        if (P.n_split > 1) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            part[(c + i) / 4 * C::kRows] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          continue;
        }
#pragma unroll
        for (int c8 = 0; c8 < 32; c8 += 8) {
          uint4 pk;
          __nv_bfloat162 *e = reinterpret_cast<__nv_bfloat162 *>(&pk);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            e[i] = __floats2bfloat162_rn(o[c8 + 2 * i] * inv, o[c8 + 2 * i + 1] * inv);
          *reinterpret_cast<uint4 *>(out + c + c8) = pk;
        }
      }
      if (valid && ok && P.n_split > 1) P.part_ml[slot0 + row] = make_float2(m, l);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == C::kMma) {
    fence_after();
    tcx::tmem_dealloc(tmem, NT * kChTmem);
  }
}

// Merges the parts of a unit: with M = max m_c, O = sum_c 2^(m_c - M) O_c /
// sum_c 2^(m_c - M) l_c, in part order.  A block takes 32 rows (one per lane)
// and 32 columns (four per warp).  The unit is found before the parts are
// waited for: what it reads was there before the chunk kernel began.
constexpr int kChMergeThreads = 256;
template <int HD, int NT>
__global__ void __launch_bounds__(kChMergeThreads)
chunk_merge_kernel(const __grid_constant__ AttnParams P) {
  constexpr int kChRows = ChCfg<HD, NT>::kRows, kQuads = kChRows / 32, kColBlocks = HD / 32;
  __shared__ PagedTile s_tile;
  __shared__ int s_sums[kChMergeThreads / 32];
  __shared__ __align__(16) bf16 s_out[32][40];
  const int sub = blockIdx.x % (kQuads * kColBlocks), quad = sub / kColBlocks, cb = sub % kColBlocks;
  const int g = blockIdx.x / (kQuads * kColBlocks) % P.Hkv, tile = blockIdx.x / (kQuads * kColBlocks) / P.Hkv;
  paged_find_tile<kChMergeThreads>(P.kv, P.n_rows, P.G, kChRows, P.max_kv, tile, &s_tile, s_sums, nullptr, P.rows_lo);
  grid_dep_wait();
  grid_dep_launch();
  const PagedTile tl = s_tile;
  const int l0 = tl.t * kChRows + quad * 32;
  if (tl.s < 0 || l0 >= tl.n * P.G) return;
  const int rows = min(32, tl.n * P.G - l0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t slot0 = (int64_t)(tile * P.Hkv + g) * P.n_split * kChRows;
  const float2 *ml = P.part_ml + slot0 + quad * 32 + lane;
  const float4 *po = reinterpret_cast<const float4 *>(P.part_o + slot0 * HD) + (cb * 8 + warp) * kChRows + quad * 32 + lane;
  float M = -INFINITY, l = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < rows) {
#pragma unroll 8
    for (int c = 0; c < P.n_split; ++c) M = fmaxf(M, ml[c * kChRows].x);
#pragma unroll 4
    for (int c = 0; c < P.n_split; ++c) {
      const float2 x = ml[c * kChRows];
      if (x.x == -INFINITY) continue;            // no visible key in this part; its O is not written
      const float w = fast_exp2(x.x - M);
      const float4 v = po[(int64_t)c * kChRows * HD / 4];
      l = fmaf(w, x.y, l);
      a.x = fmaf(w, v.x, a.x);
      a.y = fmaf(w, v.y, a.y);
      a.z = fmaf(w, v.z, a.z);
      a.w = fmaf(w, v.w, a.w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat162 *so = reinterpret_cast<__nv_bfloat162 *>(&s_out[lane][warp * 4]);
  so[0] = __floats2bfloat162_rn(a.x * inv, a.y * inv);
  so[1] = __floats2bfloat162_rn(a.z * inv, a.w * inv);
  __syncthreads();
  // 64 bytes of each row, four lanes a row
  const int r = threadIdx.x / 4, c8 = threadIdx.x % 4 * 8;
  if (r < rows) {
    const int lr = l0 + r, qi = P.by_G.div(lr);
    *reinterpret_cast<uint4 *>(reinterpret_cast<bf16 *>(P.out) + (int64_t)(tl.row0 + qi) * P.ld_out +
                               (int64_t)(g * P.G + lr - qi * P.G) * HD + cb * 32 + c8) =
        *reinterpret_cast<const uint4 *>(&s_out[r][c8]);
  }
}

template <int HD, int NT>
static cudaError_t run(const AttnParams &P, int64_t tiles, int *status, cudaStream_t s) {
  typedef ChCfg<HD, NT> C;
  static PerDeviceOnce attr;
  cudaError_t e = attr.run([](int) {
    return cudaFuncSetAttribute(paged_chunk_kernel<HD, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_chunk_kernel<HD, NT>, dim3((unsigned)(tiles * P.Hkv * P.n_split)), dim3(C::kThreads), C::kSmem,
                 s, P, status);
  if (e != cudaSuccess) return e;
  if (P.n_split == 1) return launched(1);
  e = launch_pdl(chunk_merge_kernel<HD, NT>, dim3((unsigned)(tiles * P.Hkv * (C::kRows / 32) * (HD / 32))),
                 dim3(kChMergeThreads), 0, s, P);
  return e == cudaSuccess ? launched(2) : e;
}

cudaError_t launch_chunk(const AttnParams &P, int R, int64_t tiles, int hd, int *status, cudaStream_t s) {
  if (hd == 128) return R == 128 ? run<128, 1>(P, tiles, status, s) : run<128, 2>(P, tiles, status, s);
  return R == 128 ? run<64, 1>(P, tiles, status, s) : run<64, 2>(P, tiles, status, s);
}

}  // namespace paged
}  // namespace cb
