// Token sampling from logits with temperature, top-k, top-p and min-p, from
// given uniform numbers.
//
// For a row x with maximum X and temperature t, w_i = exp((x_i - X) / t).
// The kept set is a prefix of the order "larger x first, then lower index":
// the top_k first of it, of those the shortest prefix that carries top_p of
// their weight, of those the tokens with w >= min_p.  The token is the lowest
// index i at which the kept weights up to i, in vocabulary order, exceed
// u times their total.
//
// A token must not depend on the order of a sum, and a border is met to the
// last bit only if both sides agree on the weights, so weights are 64-bit
// fixed point numbers, w * 2^S rounded, with exp evaluated to about 2^-38:
// every sum is then exact and the same whatever its order, and a token can
// differ from the real-number definition only where u falls within about
// 2^-36 of a border.  Sums of float weights would err by 2^-24, which over
// 10^5 borders is a wrong token in every hundredth row.
//
// One cluster of C blocks holds a row in shared memory, C slices of it, so
// the logits are read once from device memory.  The two selections share one
// histogram over equal steps of x, from the maximum down to where weights
// vanish.  Under top_k it counts tokens only: top_p is then of the kept
// tokens' weight, and they are few (when that was brought in, one row of 128,256
// with top_k 50 and top_p went from 26 us to 14.5; it takes 11.7 now).  The step at which the count
// reaches top_k, or the weight top_p, is found from its sums, and only the
// tokens that matter there are gathered, in vocabulary order:
//   small  all tokens down to that step (at most kCand): the cluster's first
//          block orders them and finishes the row alone.  The steps order them
//          but for the few inside one, which are compared with each other
//          (1000 tokens: 17 us in all; sorted, which crowded steps still are, 21);
//   large  the step's own tokens: the exact cut goes back to the cluster,
//          whose blocks then draw from everything above it;
//   wide   more tokens in one step than kCand (long ties): a radix selection
//          over the keys finds the cut instead.
//
// What it measures: one row of 128,256 in bf16 4.2 us when greedy, 11 to 17 us
// with top_k 5 to 1000 and top_p; 96 rows of 151,936 in fp32 with mixed
// settings 76 to 88 us, by the settings drawn.  One row is a chain of a dozen dependent phases of 0.3 to 2 us
// (load, maximum, histogram, its sums over the cluster, search, gather, order,
// draw), with a cluster barrier between most; many rows are bound by the
// arithmetic, about 90 instructions per token where weights are exact.
#include <math.h>

#include <type_traits>

#include "cb_attn_tc.cuh"
#include "cb_common.cuh"
#include "cb_internal.h"

namespace cb {
namespace smp {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;                 // steps of the histogram
constexpr int kCand = 2048;                 // tokens the first block takes
constexpr int kCrowd = 64;                  // tokens of a step that are compared one by one
constexpr int kMaxCluster = 8;
typedef unsigned long long u64;
using attn::add2;
using attn::fma2;
using attn::hi2;
using attn::lo2;
using attn::pack2;

// 2^(j / 128) * 2^62 for j = 0 .. 127, rounded.
__device__ const u64 kExp2Table[128] = {
    0x4000000000000000ull, 0x4058f6a7ecccd5b6ull, 0x40b268f9de0183baull, 0x410c57a1b9fe12f6ull,
    0x4166c34c5615d0ecull, 0x41c1aca777db771bull, 0x421d1461d66f2023ull, 0x4278fb2b1bce0d15ull,
    0x42d561b3e6243d8aull, 0x433248adc91fdd02ull, 0x438fb0cb4f468808ull, 0x43ed9abffb4c6bc9ull,
    0x444c0740496d4294ull, 0x44aaf701b0c72feeull, 0x450a6abaa4b77ecdull, 0x456a632296394492ull,
    0x45cae0f1f545eb73ull, 0x462be4e23237a6efull, 0x468d6fadbf2dd4f3ull, 0x46ef821011734e6bull,
    0x47521cc5a2e6a9e0ull, 0x47b5408bf36472e2ull, 0x4818ee218a3358eeull, 0x487d2645f7725895ull,
    0x48e1e9b9d588e19bull, 0x4947393eca98fcd6ull, 0x49ad159789f37496ull, 0x4a137f87d58e025bull,
    0x4a7a77d47f7b84b1ull, 0x4ae1ff436b663ff7ull, 0x4b4a169b900c2d00ull, 0x4bb2bea4f8bd5847ull,
    0x4c1bf828c6dc54b8ull, 0x4c85c3f13360c4d5ull, 0x4cf022c9905bfd32ull, 0x4d5b157e4a7fc325ull,
    0x4dc69cdceaa72a9cull, 0x4e32b9b417619617ull, 0x4e9f6cd3967fdba8ull, 0x4f0cb70c4ea39210ull,
    0x4f7a993048d088d7ull, 0x4fe91412b2006e83ull, 0x50582887dcb8a7e1ull, 0x50c7d76542a25b72ull,
    0x513821818624b40cull, 0x51a907b474015dc9ull, 0x521a8ad704f3404full, 0x528cabc35f4f799dull,
    0x52ff6b54d8a89c75ull, 0x5372ca67f774358full, 0x53e6c9da74b29ab5ull, 0x545b6a8b3d990704ull,
    0x54d0ad5a753e077cull, 0x5546932976483b15ull, 0x55bd1cdad49f699cull, 0x56344b525f1ff495ull,
    0x56ac1f752150a563ull, 0x57249a29651adc07ull, 0x579dbc56b48521baull, 0x581786e5db7022c2ull,
    0x5891fac0e95612c8ull, 0x590d18d3330c7f1eull, 0x5988e20954889245ull, 0x5a05575132a5cc20ull,
    0x5a827999fcef3242ull, 0x5b0049d42f6afbb6ull, 0x5b7ec8f19468bbc9ull, 0x5bfdf7e546520f3eull,
    0x5c7dd7a3b17dcf75ull, 0x5cfe69229605cef5ull, 0x5d7fad59099f22feull, 0x5e01a53f7974fd86ull,
    0x5e8451cfac061b5full, 0x5f07b404c304c9f1ull, 0x5f8bccdb3d398841ull, 0x60109d50f86846d8ull,
    0x6096266533384a2bull, 0x611c69188f1eb339ull, 0x61a3666d124bb204ull, 0x622b1f66299a6599ull,
    0x62b39508aa836d6full, 0x633cc85ad5122fbdull, 0x63c6ba6455dcd8aeull, 0x64516c2e47ff1623ull,
    0x64dcdec3371793d1ull, 0x6569132f21483ba7ull, 0x65f60a7f79393e2eull, 0x6683c5c3281ee6e9ull,
    0x6712460a8fc24072ull, 0x67a18c678c8c8c61ull, 0x683199ed779592caull, 0x68c26fb128b4cd63ull,
    0x69540ec8f895722dull, 0x69e6784cc2cd61bdull, 0x6a79ad55e7f6fd10ull, 0x6b0daeff4fcde703ull,
    0x6ba27e656b4eb57aull, 0x6c381ca636d99642ull, 0x6cce8ae13c57ebdbull, 0x6d65ca379564e639ull,
    0x6dfddbcbed791babull, 0x6e96c0c284192610ull, 0x6f307a412f074892ull, 0x6fcb096f5c782210ull,
    0x70666f76154a7089ull, 0x7102ad7fff41e9b4ull, 0x719fc4b95f452d29ull, 0x723db6501b9ed447ull,
    0x72dc8373be41a454ull, 0x737c2d55770fe711ull, 0x741cb5281e25ee34ull, 0x74be1c203627c62bull,
    0x75606373ee921c97ull, 0x76038c5b260e5eeeull, 0x76a7980f6cca15c2ull, 0x774c87cc06d1812eull,
    0x77f25ccdee6d7ae6ull, 0x78991853d684a285ull, 0x7940bb9e2cffd89dull, 0x79e947ef1d320d2dull,
    0x7a92be8a92436616ull, 0x7b3d20b6399fc237ull, 0x7be86fb985689ddcull, 0x7c94acddaeea5d3aull,
    0x7d41d96db915019dull, 0x7deff6b672f84e24ull, 0x7e9f06067a4360baull, 0x7f4f08ae3dc7c426ull,
};

struct Params {
  const void *logits;
  int64_t ld;
  int vocab, slice;                   // slice: tokens of a block, a multiple of 8
  int shift;                          // S: weights are held as w * 2^S
  const float *u, *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int32_t *tokens;
};

// ------------------------------------------------------------- weights --
// Scale of one row: the maximum and log2(e) / temperature as hi + lo.
struct Scale {
  float top, ch, cl;
  int shift;
};

// w * 2^S of two logits, on packed pairs of floats.  (x - X) log2(e) / t is
// formed as an unevaluated sum ph + pl of two floats: two-sum gives the
// subtraction's error, fma the product's.  Adding and taking away a large
// constant rounds ph to a multiple of 1/128, whose integer part becomes a
// shift and whose rest picks a table entry; e = ph - that (|e| <= 2^-8) and
// pl enter 2^(e + pl) - 1 = e ln 2 + pl ln 2 + (e + pl)^2 (c2 + e (c3 + e c4)),
// the first product again as two floats.  The large part on a grid of 2^-30
// and the rest on one of 2^-38 are read off as integers the same way, and one
// 32 x 32 bit product scales the table entry.  Relative error about 2^-38.
__device__ __forceinline__ void weight2(float x0, float x1, const Scale &c, const u64 *table, u64 &w0, u64 &w1) {
  typedef unsigned long long P2;
  constexpr float kM1 = 98304.f;                    // 1.5 * 2^16: steps of 2^-7
  constexpr float kM2 = 0x1.8p-7f, kM3 = 0x1.8p-15f; // steps of 2^-30 (|.| < 2^-8) and 2^-38 (< 2^-16)
  constexpr float kLn2h = 0x1.62e430p-1f, kLn2l = -1.9046543e-9f;   // ln 2
  constexpr float kC2 = 2.402265070e-1f, kC3 = 5.550410866e-2f, kC4 = 9.618129108e-3f;   // ln2^k / k!
  auto both = [](float v) { return pack2(v, v); };
  const P2 neg = both(-1.f), X = pack2(x0, x1), T = both(-c.top), ch = both(c.ch);
  const P2 D = add2(X, T), B = fma2(X, neg, D);
  const P2 DL = add2(fma2(fma2(B, neg, D), neg, X), fma2(B, neg, T));
  const P2 PH = fma2(D, ch, both(0.f));
  P2 PL = fma2(D, ch, fma2(D, both(-c.ch), both(0.f)));
  PL = fma2(DL, ch, fma2(D, both(c.cl), PL));
  const P2 R = add2(PH, both(kM1)), E = fma2(add2(R, both(-kM1)), neg, PH), EP = add2(E, PL);
  const P2 YH = fma2(E, both(kLn2h), both(0.f));
  P2 YL = fma2(E, both(kLn2h), fma2(E, both(-kLn2h), both(0.f)));
  YL = fma2(PL, both(kLn2h), fma2(E, both(kLn2l), YL));
  YL = fma2(fma2(EP, EP, both(0.f)), fma2(EP, fma2(EP, both(kC4), both(kC3)), both(kC2)), YL);
  const P2 R2 = add2(YH, both(kM2)), SM = add2(fma2(add2(R2, both(-kM2)), neg, YH), YL), R3 = add2(SM, both(kM3));
  auto fixed = [&](float ph, float r, float r2, float r3) -> u64 {
    const int k = __float_as_int(r) - __float_as_int(kM1);
    const int q = ((__float_as_int(r2) - __float_as_int(kM2)) << 8) + (__float_as_int(r3) - __float_as_int(kM3));
    const u64 t = table[k & 127];
    const u64 w62 = t + (u64)(((long long)(int)(uint32_t)(t >> 32) * q) >> 6);
    const int sh = min(62 - c.shift - (k >> 7), 64);
    // below half a unit, or -inf (whose integers are meaningless)
    return ph > -(float)(c.shift + 2) ? ((w62 >> (sh - 1)) + 1) >> 1 : 0ull;
  };
  w0 = fixed(lo2(PH), lo2(R), lo2(R2), lo2(R3));
  w1 = fixed(hi2(PH), hi2(R), hi2(R2), hi2(R3));
  if (c.top == INFINITY) {                          // tokens at +inf share the draw
    w0 = x0 == c.top ? 1ull << c.shift : 0ull;
    w1 = x1 == c.top ? 1ull << c.shift : 0ull;
  }
}
__device__ __forceinline__ u64 weight(float x, const Scale &c, const u64 *table) {
  u64 w, none;
  weight2(x, -INFINITY, c, table, w, none);
  return w;
}

// floor(a * f) for f in [0, 1], a < 2^63; `inexact`: the product has a
// fraction.
__device__ __forceinline__ u64 scaled(u64 a, float f, bool *inexact) {
  const uint32_t b = __float_as_uint(f);
  const int ex = (int)(b >> 23);
  const u64 m = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int sh = ex ? 150 - ex : 149;                  // f = m * 2^-sh, sh >= 23
  const u64 lo = a * m, hi = __umul64hi(a, m);
  *inexact = false;
  if (sh >= 64) {
    const int s2 = sh - 64;
    *inexact = lo != 0 || (s2 < 64 ? (hi & ((1ull << s2) - 1)) != 0 : hi != 0);
    return s2 < 64 ? hi >> s2 : 0ull;
  }
  *inexact = (lo & ((1ull << sh) - 1)) != 0;
  return (lo >> sh) | (hi << (64 - sh));
}

// --------------------------------------------------------------- layout --
struct Shared {
  union {
    struct {
      uint32_t cnt[kBins], m0[kBins], m1[kBins], m2[kBins];   // this block's histogram
    };
    u64 cand[kCand];        // gathered tokens, sorted
  };
  u64 rmass[kBins];         // the bins this block reduces over the cluster
  uint32_t rcnt[kBins];
  u64 table[128];
  u64 warp[kWarps];         // a pass's sum per warp
  u64 sum[3];               // this block's sums: weights to cut, ties, kept weights
  u64 best;                 // this block's largest (key, ~index)
  float least;              // and its smallest logit above -inf
  u64 left, total;          // a search's answer
  int bin, count;
  u64 cut;                  // the cut: key << 32 | last index kept with that key
  float ch, cl;             // log2(e) / temperature
};

// Order-preserving integer of a float, and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
// NaN counts as -inf, -0 as 0: equal values have equal keys.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : x + 0.f; }

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  tcx::cluster_sync();
}
// The same shared variable in block `rank` of the cluster.  What it reads was
// written before the last cluster barrier, so several reads may be in flight.
__device__ __forceinline__ u64 remote(const u64 *p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(tcx::map_to_rank(smem_u32(p), rank)));
  return v;
}
__device__ __forceinline__ uint32_t remote(const uint32_t *p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tcx::map_to_rank(smem_u32(p), rank)));
  return v;
}
__device__ __forceinline__ float remote(const float *p, uint32_t rank) {
  return __uint_as_float(remote(reinterpret_cast<const uint32_t *>(p), rank));
}
// Sum of the same variable over the cluster's C blocks.
__device__ __forceinline__ u64 remote_sum(const uint32_t *p, int C) {
  uint32_t v[kMaxCluster];
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) v[c] = c < C ? remote(p, c) : 0u;
  u64 s = 0;
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) s += v[c];
  return s;
}
__device__ __forceinline__ void remote_store(u64 *p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tcx::map_to_rank(smem_u32(p), rank)), "l"(v)
               : "memory");
}
// Exclusive prefix sum of v over the block, the block's sum in *total.
__device__ __forceinline__ u64 block_scan(Shared &sh, u64 v, u64 *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();
  if (lane == 31) sh.warp[warp] = incl;
  __syncthreads();
  // every warp scans the warps' sums
  u64 w = lane < kWarps ? sh.warp[lane] : 0ull;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += t;
  }
  *total = __shfl_sync(0xffffffffu, w, kWarps - 1);
  const u64 before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp ? before : 0ull) + incl - v;
}

// Adds a weight to bin b of this block's histogram, in three 16-bit parts:
// their sums over a slice of at most 2^16 tokens stay below 2^32.
__device__ __forceinline__ void add_weight(Shared &sh, int b, u64 m) {
  atomicAdd(&sh.m0[b], (uint32_t)m & 0xffffu);
  const uint32_t hi = (uint32_t)(m >> 16) & 0xffffu, top = (uint32_t)(m >> 32);
  if (hi) atomicAdd(&sh.m1[b], hi);
  if (top) atomicAdd(&sh.m2[b], top);
}
// A bin's weight over the cluster.
__device__ __forceinline__ u64 remote_weight(const Shared &sh, int b, int C) {
  const u64 p0 = remote_sum(&sh.m0[b], C), p1 = remote_sum(&sh.m1[b], C), p2 = remote_sum(&sh.m2[b], C);
  return p0 + (p1 << 16) + (p2 << 32);
}

// The consecutive range of a block's n tokens that warp w owns: whole rounds of
// 16 bytes per lane.
__device__ __forceinline__ int warp_begin(int n, int w) {
  return min(n, w * (((n + kWarps - 1) / kWarps + 255) / 256 * 256));
}

// A pass weighs its tokens in pairs: f(xa, a, xb, b, wa, wb) gives the weights
// of tokens a and b of the slice; a token past its end has index -1 and x
// -inf and must get 0.

// This block's sum of a pass over its tokens, left in sh.sum[slot] and, per
// warp, in sh.warp; then meets the cluster.  Returns the sums of the blocks
// before this one, and of all in *total.
template <typename T, typename F>
__device__ __forceinline__ u64 cluster_sum(Shared &sh, int slot, const T *x, int n, int rank, int C, F f,
                                           u64 *total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = warp_begin(n, warp + 1);
  u64 s = 0;
#pragma unroll 2
  for (int i = warp_begin(n, warp) + lane; i < e; i += 64) {
    const bool two = i + 32 < e;
    u64 wa, wb;
    f(to_f(x[i]), i, two ? to_f(x[i + 32]) : -INFINITY, two ? i + 32 : -1, wa, wb);
    s += wa + wb;
  }
  s = warp_sum64(s);
  __syncthreads();
  if (lane == 0) sh.warp[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const u64 t = warp_sum64(lane < kWarps ? sh.warp[lane] : 0ull);
    if (lane == 0) sh.sum[slot] = t;
  }
  cluster_barrier();
  u64 v[kMaxCluster], before = 0, all = 0;
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) v[c] = c < C ? remote(&sh.sum[slot], c) : 0ull;
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) {
    if (c < rank) before += v[c];
    all += v[c];
  }
  *total = all;
  return before;
}

// After cluster_sum of the same pass: the token at which the running sum over
// the cluster, `before` at this block's first token, first exceeds `target`
// is passed to found(i) by one thread of the block that holds it.  The block
// scans the range of the warp that holds the token with all its threads.
template <typename T, typename F, typename G>
__device__ __forceinline__ void ordered_find(Shared &sh, int slot, const T *x, int n, u64 before, u64 target, F f,
                                             G found) {
  if (target < before || target >= before + sh.sum[slot]) return;   // the same in the whole block
  int w = 0;
  while (target >= before + sh.warp[w]) before += sh.warp[w++];
  const int b = warp_begin(n, w), e = warp_begin(n, w + 1);
  const int per = (e - b + kThreads - 1) / kThreads;
  static_assert((CB_MAX_SAMPLE_VOCAB / kMaxCluster / kWarps + 255) / 256 * 256 <= 4 * kThreads, "four tokens each");
  const int i0 = b + (int)threadIdx.x * per, i1 = min(e, i0 + per);
  u64 v[4], s = 0, total;
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const int i = i0 + k;
    v[k] = v[k + 1] = 0;
    if (i < i1) f(to_f(x[i]), i, i + 1 < i1 ? to_f(x[i + 1]) : -INFINITY, i + 1 < i1 ? i + 1 : -1, v[k], v[k + 1]);
    s += v[k] + v[k + 1];
  }
  u64 acc = before + block_scan(sh, s, &total);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (acc <= target && target < acc + v[k]) found(i0 + k);
    acc += v[k];
  }
}

// Sorts a[0 .. n) ascending (n a power of two, bitonic); the block's threads
// all call.  Exchanges over at most 32 places stay inside the 64 tokens of one
// warp, so only the wider ones meet the block.
__device__ __forceinline__ void sort_block(u64 *a, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      if (j >= 64) __syncthreads();
      for (int t = threadIdx.x; t < n / 2; t += kThreads) {
        const int i = ((t & ~(j - 1)) << 1) | (t & (j - 1)), l = i + j;
        const u64 x = a[i], y = a[l];
        if ((x > y) == ((i & k) == 0)) {
          a[i] = y;
          a[l] = x;
        }
      }
      if (j >= 64) __syncthreads();
      else __syncwarp();
    }
  __syncthreads();
}
// Sorts the first n gathered tokens (padded to a power of two).
__device__ __forceinline__ void sort_cand(Shared &sh, int n) {
  int m = 2;
  while (m < n) m <<= 1;
  for (int i = n + threadIdx.x; i < m; i += kThreads) sh.cand[i] = ~0ull;
  __syncthreads();
  sort_block(sh.cand, m);
}
// A gathered token: ascending order is larger x first, then lower index.
__device__ __forceinline__ u64 pack(uint32_t key, uint32_t index) { return ((u64)~key << 32) | index; }
__device__ __forceinline__ uint32_t packed_key(u64 v) { return ~(uint32_t)(v >> 32); }

// Radix selection over the cluster's tokens, largest key first: the key at
// which the running count (MASS false) or weight (MASS true) first reaches
// `need` (>= 1 and at most the total), and in *left what of `need` falls to
// the tokens with that key.  Tokens with a key above `above` take part, and
// an extra weight at extra_key (the part of a tie that takes part).
template <typename T, bool MASS>
__device__ __forceinline__ uint32_t radix_select(Shared &sh, const T *x, int n, int rank, int C, u64 need,
                                                 const Scale &sc, int64_t above, uint32_t extra_key,
                                                 u64 extra_mass, u64 *left) {
  constexpr int kDigit = 8, nb = 1 << kDigit;
  static_assert(nb <= kThreads && nb <= kBins, "a bin per thread");
  const int per = nb / C;
  uint32_t prefix = 0;
  for (int lo = 32 - kDigit; lo >= 0; lo -= kDigit) {
    const int hi = lo + kDigit;
    for (int i = threadIdx.x; i < nb; i += kThreads) sh.cnt[i] = sh.m0[i] = sh.m1[i] = sh.m2[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float v = to_f(x[i]);
      const uint32_t k = key_of(v);
      if ((hi < 32 && (k >> hi) != prefix) || (int64_t)k <= above) continue;
      const uint32_t b = (k >> lo) & (nb - 1);
      if (MASS) {
        const u64 m = weight(v, sc, sh.table);
        if (m) add_weight(sh, b, m);
      } else {
        atomicAdd(&sh.cnt[b], 1u);
      }
    }
    cluster_barrier();
    for (int b = rank * per + threadIdx.x; b < (rank + 1) * per; b += kThreads) {
      u64 s = MASS ? remote_weight(sh, b, C) : remote_sum(&sh.cnt[b], C);
      if (MASS && extra_mass && (hi == 32 || (extra_key >> hi) == prefix) &&
          ((extra_key >> lo) & (nb - 1)) == (uint32_t)b)
        s += extra_mass;
      sh.rmass[b] = s;
    }
    cluster_barrier();
    // every block scans all bins, largest first
    const int b = nb - 1 - (int)threadIdx.x;
    const u64 v = b >= 0 ? remote(&sh.rmass[b], b / per) : 0ull;
    u64 total;
    const u64 acc = block_scan(sh, v, &total);
    if (acc < need && need <= acc + v) {
      sh.bin = b;
      sh.left = need - acc;
    }
    __syncthreads();
    prefix = (prefix << kDigit) | (uint32_t)sh.bin;
    need = sh.left;
    __syncthreads();
  }
  *left = need;
  return prefix;
}

// Loads the block's slice, cleaned, and finds its largest logit (lowest
// index first) and its smallest above -inf.
template <typename T>
__device__ __forceinline__ void load_slice(Shared &sh, T *x, const T *src, int n, int lo) {
  constexpr int VEC = 16 / sizeof(T);
  float mx = -INFINITY, mn = INFINITY;
  int at = 0x7fffffff;
  auto see = [&](float v, int i) {
    if (v > mx) {                       // indices ascend within a thread
      mx = v;
      at = i;
    }
    if (v > -INFINITY) mn = fminf(mn, v);
  };
  const int nv = ((uintptr_t)src & 15) == 0 ? n / VEC : 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < nv; i += kThreads) {
    uint4 raw = ldg16(src + i * VEC);
    T *e = reinterpret_cast<T *>(&raw);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float v = clean(to_f(e[k]));
      e[k] = from_f<T>(v);
      see(v, i * VEC + k);
    }
    *reinterpret_cast<uint4 *>(x + i * VEC) = raw;
  }
#pragma unroll 4
  for (int i = nv * VEC + threadIdx.x; i < n; i += kThreads) {
    const float v = clean(to_f(src[i]));
    x[i] = from_f<T>(v);
    see(v, i);
  }
  u64 best = at == 0x7fffffff ? 0ull : ((u64)key_of(mx) << 32) | (uint32_t)~(uint32_t)(lo + at);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const u64 t = __shfl_xor_sync(0xffffffffu, best, o);
    best = t > best ? t : best;
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *wmin = reinterpret_cast<float *>(sh.rmass);
  if (lane == 0) {
    sh.warp[warp] = best;
    wmin[warp] = mn;
  }
  __syncthreads();
  if (warp == 0) {
    best = sh.warp[lane % kWarps];
    mn = wmin[lane % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) {
      const u64 t = __shfl_xor_sync(0xffffffffu, best, o);
      best = t > best ? t : best;
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    }
    if (lane == 0) {
      sh.best = best;
      sh.least = mn;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared &sh = *reinterpret_cast<Shared *>(raw);
  T *x = reinterpret_cast<T *>(raw + (sizeof(Shared) + 15) / 16 * 16);
  const int rank = (int)tcx::cluster_rank();
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int C = (int)csize, row = blockIdx.x / C;
  const int lo = min(P.vocab, rank * P.slice), n = min(P.vocab, lo + P.slice) - lo;
  if (threadIdx.x < 128) sh.table[threadIdx.x] = kExp2Table[threadIdx.x];
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.cnt[i] = sh.m0[i] = sh.m1[i] = sh.m2[i] = 0;
  grid_dep_wait();
  grid_dep_launch();
  const float temp = P.temperature ? P.temperature[row] : 1.f;
  const int k = P.top_k ? P.top_k[row] : 0;
  const float p = P.top_p ? P.top_p[row] : 1.f;
  const float mp = P.min_p ? P.min_p[row] : 0.f;
  const float u = P.u[row];
  if (threadIdx.x == kThreads - 1) {
    // log2(e) / t as two floats, by one thread: double precision is scarce
    // (a temperature below 1e-30 acts as 1e-30)
    const double c = 1.4426950408889634 / (double)fmaxf(temp, 1e-30f);
    sh.ch = (float)c;
    sh.cl = (float)(c - (double)sh.ch);
  }
  load_slice(sh, x, reinterpret_cast<const T *>(P.logits) + (int64_t)row * P.ld + lo, n, lo);
  cluster_barrier();
  u64 best = 0, bests[kMaxCluster];
  float low = INFINITY, lows[kMaxCluster];
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) {
    bests[c] = c < C ? remote(&sh.best, c) : 0ull;
    lows[c] = c < C ? remote(&sh.least, c) : INFINITY;
  }
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) {
    best = bests[c] > best ? bests[c] : best;
    low = fminf(low, lows[c]);
  }
  const bool empty = best == 0;                       // every logit is -inf or NaN
  if (empty || !(temp > 0.f) || k == 1 || p <= 0.f) {
    if (rank == 0 && threadIdx.x == 0) P.tokens[row] = empty ? -1 : (int)~(uint32_t)best;
    cluster_barrier();                                // its shared memory has been read
    return;
  }
  Scale sc;
  sc.top = value_of((uint32_t)(best >> 32));
  sc.shift = P.shift;
  sc.ch = sh.ch;
  sc.cl = sh.cl;
  bool use_k = k > 0 && k < P.vocab;
  const bool use_p = p < 1.f;
  u64 least = 1;                                      // min_p of the largest weight
  if (mp > 0.f) {
    bool more = false;
    least = mp >= 1.f ? 1ull << P.shift : scaled(1ull << P.shift, mp, &more);
    least += more;
  }
  bool cut = false, wide = false;
  uint32_t cut_key = 0;
  int last = P.vocab;                                 // largest index kept at cut_key
  if (use_k || use_p) {
    // steps of x from the maximum down to where weights vanish (tokens beyond
    // are in none: no cut can matter there)
    const float range = fminf(sc.top - low, (float)(P.shift + 3) / sc.ch);
    const float scale = ((float)kBins - 1.f) / fmaxf(range * 1.0001f, 1e-35f);
    // monotone in v: the nearest step (not contracted, so that every pass finds the same)
    auto bin_of = [&](float v) -> int {
      const float t = __fmul_rn(sc.top - v, scale);
      return t < (float)kBins - 1.f ? __float_as_int(t + 12582912.f) - 0x4b400000 : kBins;
    };
    wide = sc.top == INFINITY;                        // no distance to measure by
    if (!wide) {
      // Counts per step, and weights where top_p is taken of the whole row;
      // under top_k its tokens' weights are enough, and they are few.
      constexpr int VEC = 16 / sizeof(T);
      const int per = kBins / C;
      auto histogram = [&](bool counts, bool weights) {
        for (int i = threadIdx.x * VEC; i < n; i += kThreads * VEC) {
          float v[VEC];
          load16<T>(x + i, v);
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const float xa = i + e < n ? v[e] : -INFINITY, xb = i + e + 1 < n ? v[e + 1] : -INFINITY;
            const int ba = bin_of(xa), bb = bin_of(xb);
            if (counts) {
              if (ba < kBins) atomicAdd(&sh.cnt[ba], 1u);
              if (bb < kBins) atomicAdd(&sh.cnt[bb], 1u);
            }
            if (weights) {
              u64 wa, wb;
              weight2(xa, xb, sc, sh.table, wa, wb);
              if (wa) add_weight(sh, ba, wa);
              if (wb) add_weight(sh, bb, wb);
            }
          }
        }
        cluster_barrier();
        for (int b = rank * per + threadIdx.x; b < (rank + 1) * per; b += kThreads) {
          if (counts) sh.rcnt[b] = (uint32_t)remote_sum(&sh.cnt[b], C);
          if (weights) sh.rmass[b] = remote_weight(sh, b, C);
        }
        cluster_barrier();
      };
      if (use_k) histogram(true, false);
      else histogram(true, true);
      // every block scans all bins, two per thread, from the maximum down
      static_assert(kBins == 2 * kThreads, "two bins per thread");
      const int b = threadIdx.x * 2;
      const uint32_t q0 = remote(&sh.rcnt[b], b / per), q1 = remote(&sh.rcnt[b + 1], b / per);
      u64 count, total = 0, w0 = 0, w1 = 0, wacc = 0;
      const u64 qacc = block_scan(sh, (u64)q0 + q1, &count);
      if (use_k && (u64)k > count) {                  // only vanished weights fall to it
        use_k = false;
        if (use_p) histogram(false, true);
      }
      if (use_p && !use_k) {
        w0 = remote(&sh.rmass[b], b / per);
        w1 = remote(&sh.rmass[b + 1], b / per);
        wacc = block_scan(sh, w0 + w1, &total);
      }
      // the step that reaches top_k, or else top_p
      bool more;
      u64 need = (u64)k;
      if (!use_k && use_p) {
        need = scaled(total, p, &more);
        need += more;
        need = need ? need : 1;
      }
      if (use_k || use_p) {
        const u64 a = use_k ? qacc : wacc, v0 = use_k ? q0 : w0, v1 = use_k ? q1 : w1;
        if (a < need && need <= a + v0 + v1) {
          const int second = need > a + v0;
          sh.bin = b + second;
          sh.left = need - a - (second ? v0 : 0);     // still needed inside the step
          sh.count = (int)(qacc + q0 + (second ? q1 : 0));   // tokens down to and with it
          sh.total = total;
        }
        __syncthreads();
        const int step = sh.bin, in_step = (int)remote(&sh.rcnt[step], step / per), down = sh.count;
        const bool small = down <= kCand;
        // a step of its own serves one selection: large top_k with top_p goes wide
        wide = !small && (in_step > kCand || (use_k && use_p));
        if (!wide) {
          // Every warp marks and counts its tokens (its range is consecutive),
          // then stores them at their places: the list comes in vocabulary order.
          const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
          const int wb = warp_begin(n, warp), we = warp_begin(n, warp + 1);
          static_assert((CB_MAX_SAMPLE_VOCAB / kMaxCluster / kWarps + 255) / 256 * 256 <= 32 * 64, "64 tokens a lane");
          u64 marks = 0;                              // VEC bits per 16 bytes of tokens
          // a bin is its distance rounded to even: as borders of the distance,
          // below < distance <= upto
          auto border = [&](int b) -> float {
            const float h = (float)b + 0.5f;
            return fminf(b & 1 ? nextafterf(h, 0.f) : h, nextafterf((float)kBins - 1.f, 0.f));
          };
          const float upto = border(step), below = small || step == 0 ? -1.f : border(step - 1);
#pragma unroll 2
          for (int i0 = wb, at = 0; i0 < we; i0 += 32 * VEC, at += VEC) {
            const int i = i0 + lane * VEC;
            if (i < we) {
              float v[VEC];
              load16<T>(x + i, v);                     // past we: another warp's, or past n, unmarked below
              uint32_t m = 0;
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                const float t = __fmul_rn(sc.top - v[e], scale);
                m |= (uint32_t)(t > below && t <= upto) << e;
              }
              if (we - i < VEC) m &= (1u << (we - i)) - 1;
              marks |= (u64)m << at;
            }
          }
          const uint32_t mine = __reduce_add_sync(0xffffffffu, (uint32_t)__popcll(marks));
          if (lane == 0) sh.warp[warp] = mine;
          __syncthreads();
          if (warp == 0) {
            const uint32_t t = __reduce_add_sync(0xffffffffu, lane < kWarps ? (uint32_t)sh.warp[lane] : 0u);
            if (lane == 0) sh.sum[0] = t;
          }
          cluster_barrier();
          uint32_t place = 0;                         // tokens of the blocks and warps before this one
          if (lane < rank) place = (uint32_t)remote(&sh.sum[0], lane);
          if (lane < warp) place += (uint32_t)sh.warp[lane];
          place = __reduce_add_sync(0xffffffffu, place);
          if (mine)
            for (int i0 = wb; i0 < we; i0 += 32 * VEC, marks >>= VEC) {
              uint32_t m = (uint32_t)marks & ((1u << VEC) - 1);
              if (!__any_sync(0xffffffffu, m)) continue;
              uint32_t before = 0, all = 0;
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                const uint32_t lanes = __ballot_sync(0xffffffffu, m >> e & 1);
                before += __popc(lanes & ((1u << lane) - 1));
                all += __popc(lanes);
              }
              for (uint32_t at = place + before; m; m &= m - 1) {
                const int i = i0 + lane * VEC + __ffs(m) - 1;
                remote_store(&sh.cand[at++], 0, pack(key_of(to_f(x[i])), lo + i));
              }
              place += all;
            }
          cluster_barrier();
          if (rank == 0) {
            const int nc = small ? down : in_step;
            const u64 in_left = sh.left, all = sh.total;
            // weights of list entries 4t .. 4t + 3 (thread t), 0 past `n` and
            // after `cut` in sorted order
            auto weigh4 = [&](const u64 *list, int n, u64 cut, u64 (&w)[4]) {
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const int i = threadIdx.x * 4 + e;
                w[e] = w[e + 1] = 0;
                if (i >= n) continue;
                const u64 a = list[i], b = i + 1 < n ? list[i + 1] : ~0ull;
                weight2(value_of(packed_key(a)), i + 1 < n ? value_of(packed_key(b)) : -INFINITY, sc, sh.table, w[e],
                        w[e + 1]);
                if (a > cut) w[e] = 0;
                if (b > cut) w[e + 1] = 0;
              }
            };
            // a copy in vocabulary order stays in the slice's place, which the
            // first block no longer needs if it finishes the row
            u64 *listed = reinterpret_cast<u64 *>(x);
            if (small && !__syncthreads_or((b <= step && q0 > kCrowd) || (b < step && q1 > kCrowd))) {
              // The steps order the tokens already: each goes to its step's
              // segment (the counts' prefix sums), and its place is found
              // among the few there.
              uint32_t *const next = sh.rcnt;          // read by the other blocks before the last barriers
              next[b] = (uint32_t)qacc;
              next[b + 1] = (uint32_t)(qacc + q0);
              __syncthreads();
              // E tokens per thread, which keeps their weights and places
              auto finish = [&](auto per_thread) {
                constexpr int E = decltype(per_thread)::value;
                const int t = threadIdx.x * E, nk = use_k ? min(k, nc) : nc;
                u64 v[E], w[E];
                int order[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                  v[e] = t + e < nc ? sh.cand[t + e] : ~0ull;
                  order[e] = t + e < nc ? bin_of(value_of(packed_key(v[e]))) : 0;
                  if (t + e < nc) listed[atomicAdd(&next[order[e]], 1u)] = v[e];
                }
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                  const bool two = e + 1 < E && t + e + 1 < nc;
                  u64 second;
                  weight2(t + e < nc ? value_of(packed_key(v[e])) : -INFINITY,
                          two ? value_of(packed_key(v[(e + 1) % E])) : -INFINITY, sc, sh.table, w[e], second);
                  if (e + 1 < E) w[(e + 1) % E] = second;
                }
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) {
                  if (t + e >= nc) continue;
                  const int end = next[order[e]], begin = order[e] ? next[order[e] - 1] : 0;
                  order[e] = begin;
                  for (int i = begin; i < end; ++i) order[e] += listed[i] < v[e];
                }
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e)
                  if (t + e < nc) listed[order[e]] = order[e] < nk ? w[e] : 0ull;   // weights in order now
                __syncthreads();
                u64 s = 0, sum, sorted[E];
#pragma unroll
                for (int e = 0; e < E; ++e) s += sorted[e] = t + e < nc ? listed[t + e] : 0ull;
                u64 acc = block_scan(sh, s, &sum), need_p = ~0ull;
                if (use_p) {
                  need_p = scaled(use_k ? sum : all, p, &more);
                  need_p += more;
                  need_p = need_p ? need_p : 1;
                }
                // kept: what lies before it is short of need_p, and w >= least
                int kept = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                  kept += __syncthreads_count(sorted[e] >= least && acc < need_p);
                  acc += sorted[e];
                }
                s = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) s += w[e] = t + e < nc && order[e] < kept ? w[e] : 0ull;
                acc = block_scan(sh, s, &sum);
                const u64 target = u >= 1.f ? sum - 1 : u > 0.f ? scaled(sum, u, &more) : 0ull;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                  if (acc <= target && target < acc + w[e]) P.tokens[row] = (int)(uint32_t)v[e];
                  acc += w[e];
                }
              };
              if (nc <= kThreads) finish(std::integral_constant<int, 1>());
              else finish(std::integral_constant<int, kCand / kThreads>());
              return;
            }
            if (small)
              for (int i = threadIdx.x; i < nc; i += kThreads) listed[i] = sh.cand[i];
            sort_cand(sh, nc);
            // thread t holds sorted tokens 4t .. 4t + 3 and their weights
            u64 w[4], s = 0, sum;
            weigh4(sh.cand, small || use_p ? nc : 0, ~0ull, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) s += w[e];
            if (!small) {
              // the cut: the in_left-th token of the step, or the one whose
              // weight completes in_left
              const u64 acc0 = block_scan(sh, s, &sum);
              u64 acc = acc0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i = threadIdx.x * 4 + e;
                const bool hit = use_k ? (u64)i + 1 == in_left && i < nc : acc < in_left && in_left <= acc + w[e];
                if (hit) {
                  const u64 v = sh.cand[i];
                  const u64 c64 = ((u64)packed_key(v) << 32) | (uint32_t)v;
                  for (int c = 0; c < C; ++c) remote_store(&sh.cut, c, c64);
                }
                acc += w[e];
              }
            } else {
              // the kept prefix: top_k of the tokens, top_p of their weight, min_p
              const int nk = use_k ? k : nc;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((int)threadIdx.x * 4 + e >= nk) {
                  s -= w[e];
                  w[e] = 0;
                }
              const u64 acc0 = block_scan(sh, s, &sum);
              u64 need_p = ~0ull;
              if (use_p) {
                need_p = scaled(use_k ? sum : all, p, &more);
                need_p += more;
                need_p = need_p ? need_p : 1;
              }
              // kept: what lies before it is short of need_p, and w >= least;
              // the last kept token in sorted order is the cut
              u64 acc = acc0;
              int kept_n = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                kept_n += w[e] >= least && acc < need_p;
                acc += w[e];
              }
              if (__syncthreads_count(kept_n > 0) == (int)threadIdx.x + 1)
                sh.cut = sh.cand[threadIdx.x * 4 + kept_n - 1];
              __syncthreads();
              const u64 cut_at = sh.cut;
              s = 0;
              weigh4(listed, nc, cut_at, w);
#pragma unroll
              for (int e = 0; e < 4; ++e) s += w[e];
              acc = block_scan(sh, s, &sum);
              const u64 target = u >= 1.f ? sum - 1 : u > 0.f ? scaled(sum, u, &more) : 0ull;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (acc <= target && target < acc + w[e])
                  P.tokens[row] = (int)(uint32_t)listed[threadIdx.x * 4 + e];
                acc += w[e];
              }
            }
          }
          if (small) return;                          // only the first block's memory is in use
          cluster_barrier();
          cut = true;
          cut_key = (uint32_t)(sh.cut >> 32);
          last = (int)(uint32_t)sh.cut;
        }
      }
    }
    if (wide) {
      cluster_barrier();                              // the histograms have been read
      u64 cut_left = 0;                               // tokens kept at cut_key
      use_k = k > 0 && k < P.vocab;
      if (use_k) cut_key = radix_select<T, false>(sh, x, n, rank, C, (u64)k, sc, -1, 0, 0, &cut_left);
      if (use_p) {
        const int64_t above = use_k ? (int64_t)cut_key : -1;
        const u64 tie = use_k ? cut_left * weight(value_of(cut_key), sc, sh.table) : 0ull;
        u64 total;
        cluster_sum(sh, 0, x, n, rank, C, [&](float xa, int, float xb, int, u64 &wa, u64 &wb) {
          weight2(xa, xb, sc, sh.table, wa, wb);       // 0 at -inf
          if ((int64_t)key_of(xa) <= above) wa = 0;
          if ((int64_t)key_of(xb) <= above) wb = 0;
        }, &total);
        total += tie;
        bool more;
        u64 need = scaled(total, p, &more);
        need += more;
        u64 left;
        cut_key = radix_select<T, true>(sh, x, n, rank, C, need ? need : 1, sc, above, cut_key, tie, &left);
        const u64 one = weight(value_of(cut_key), sc, sh.table);
        cut_left = (left + one - 1) / one;
      }
      cut = true;
      auto is_tie = [&](float xa, int, float xb, int b, u64 &wa, u64 &wb) {
        wa = key_of(xa) == cut_key;
        wb = b >= 0 && key_of(xb) == cut_key;
      };
      u64 ties;
      const u64 before = cluster_sum(sh, 1, x, n, rank, C, is_tie, &ties);
      if (ties > cut_left) {                          // the same in every block
        ordered_find(sh, 1, x, n, before, cut_left - 1, is_tie, [&](int i) {
          for (int c = 0; c < C; ++c) remote_store(&sh.cut, c, (u64)(lo + i));
        });
        cluster_barrier();
        last = (int)sh.cut;
      }
    }
  }
  auto keeps = [&](float v, int i) -> bool {
    const uint32_t key = key_of(v);
    return key > cut_key || (key == cut_key && lo + i <= last);
  };
  auto kept = [&](float xa, int a, float xb, int b, u64 &wa, u64 &wb) {
    wa = wb = 0;
    const bool ka = !cut || keeps(xa, a), kb = !cut || keeps(xb, b);   // -inf weighs 0 anyway
    if (!ka && !kb) return;
    weight2(xa, xb, sc, sh.table, wa, wb);
    if (!ka || wa < least) wa = 0;
    if (!kb || wb < least) wb = 0;
  };
  u64 total;
  const u64 before = cluster_sum(sh, 2, x, n, rank, C, kept, &total);
  bool more;
  const u64 target = u >= 1.f ? total - 1 : u > 0.f ? scaled(total, u, &more) : 0ull;
  ordered_find(sh, 2, x, n, before, target, kept, [&](int i) { P.tokens[row] = lo + i; });
  cluster_barrier();                                  // its shared memory has been read
}

template <typename T>
static size_t smem_bytes(int slice) {
  const size_t tokens = (size_t)slice * sizeof(T), list = kCand * sizeof(u64);   // the list takes the slice's place
  return (sizeof(Shared) + 15) / 16 * 16 + (tokens > list ? tokens : list);
}

template <typename T>
static cudaError_t run(const Params &P, int n_rows, int C, cudaStream_t s) {
  static PerDeviceOnce attr;
  cudaError_t e = attr.run([](int) {
    return cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<T>(CB_MAX_SAMPLE_VOCAB / kMaxCluster));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n_rows * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<T>(P.slice);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, P);
  if (e != cudaSuccess) return e;
  return launched(1);
}

}  // namespace smp

cudaError_t launch_sample(const void *logits, int64_t ld, int n_rows, int vocab, cb_dtype dt, const float *u,
                          const float *temperature, const int32_t *top_k, const float *top_p,
                          const float *min_p, int32_t *tokens, cudaStream_t s) {
  using namespace smp;
  if (n_rows == 0) return cudaSuccess;
  int C = 1;
  while (C < kMaxCluster && vocab > C * 4096) C *= 2;
  Params P;
  P.logits = logits;
  P.ld = ld;
  P.vocab = vocab;
  P.slice = ((vocab + C - 1) / C + 7) / 8 * 8;
  // sums of vocab weights of at most 2^S stay below 2^63
  P.shift = 46;
  while ((int64_t)vocab > ((int64_t)1 << (62 - P.shift))) --P.shift;
  P.u = u;
  P.temperature = temperature;
  P.top_p = top_p;
  P.min_p = min_p;
  P.top_k = top_k;
  P.tokens = tokens;
  return dt == CB_BF16 ? run<bf16>(P, n_rows, C, s) : run<float>(P, n_rows, C, s);
}

}  // namespace cb
