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
// fixed point numbers, w * 2^S rounded, with exp evaluated to about 2^-40:
// every sum is then exact and the same whatever its order, and a token can
// differ from the real-number definition only where u falls within about
// 2^-36 of a border.  Sums of float weights would err by 2^-24, which over
// 10^5 borders is a wrong token in every hundredth row.
//
// One cluster of C blocks holds a row in shared memory, C slices of it, so
// the logits are read once from device memory.  The two selections share one
// histogram over equal steps of x, from the maximum down to where weights
// vanish: the step at which the count reaches top_k, or the weight top_p, is
// found from its sums, and only the tokens that matter there are gathered and
// sorted exactly by (x, index):
//   small  all tokens down to that step (at most kCand): the cluster's first
//          block sorts them and finishes the row alone;
//   large  the step's own tokens: the exact cut goes back to the cluster,
//          whose blocks then draw from everything above it;
//   wide   more tokens in one step than kCand (long ties): a radix selection
//          over the keys finds the cut instead.
#include <math.h>

#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_tc.cuh"

namespace cb {
namespace smp {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;                 // steps of the histogram
constexpr int kCand = 2048;                 // tokens the sorter takes
constexpr int kMaxCluster = 8;
typedef unsigned long long u64;

// 2^(j / 64) * 2^62 for j = -32 .. 32, rounded.
__device__ const u64 kExp2Table[65] = {
    0x2d413cccfe779921ull, 0x2dbf6478ca345de4ull, 0x2e3eebd1d8bee7baull, 0x2ebfd6ac84cf917full,
    0x2f4228e7d6030db0ull, 0x2fc5e66d9e9cc421ull, 0x304b1332999c2516ull, 0x30d1b3368925d902ull,
    0x3159ca845541b6b7ull, 0x31e35d322aee6c57ull, 0x326e6f619b8bc9e9ull, 0x32fb053fbc9c9f17ull,
    0x3389230547e12039ull, 0x3418ccf6bbcac965ull, 0x34aa07647c4ab917ull, 0x353cd6aaf3fb7e88ull,
    0x35d13f32b5a75abdull, 0x366745709e2bf5edull, 0x36feede5f6bc8dd5ull, 0x37983d209783a449ull,
    0x383337bb0aa53844ull, 0x38cfe25cafa29694ull, 0x396e41b9df20d22aull, 0x3a0e5a940f12f71aull,
    0x3ab031b9f7490e4cull, 0x3b53cc07b6650ae1ull, 0x3bf92e66f736bd73ull, 0x3ca05dcf167fec4eull,
    0x3d495f454921b30bull, 0x3df437dcc2b44eeeull, 0x3ea0ecb6dc8a80cfull, 0x3f4f83033d21b05dull,
    0x4000000000000000ull, 0x40b268f9de0183baull, 0x4166c34c5615d0ecull, 0x421d1461d66f2023ull,
    0x42d561b3e6243d8aull, 0x438fb0cb4f468808ull, 0x444c0740496d4294ull, 0x450a6abaa4b77ecdull,
    0x45cae0f1f545eb73ull, 0x468d6fadbf2dd4f3ull, 0x47521cc5a2e6a9e0ull, 0x4818ee218a3358eeull,
    0x48e1e9b9d588e19bull, 0x49ad159789f37496ull, 0x4a7a77d47f7b84b1ull, 0x4b4a169b900c2d00ull,
    0x4c1bf828c6dc54b8ull, 0x4cf022c9905bfd32ull, 0x4dc69cdceaa72a9cull, 0x4e9f6cd3967fdba8ull,
    0x4f7a993048d088d7ull, 0x50582887dcb8a7e1ull, 0x513821818624b40cull, 0x521a8ad704f3404full,
    0x52ff6b54d8a89c75ull, 0x53e6c9da74b29ab5ull, 0x54d0ad5a753e077cull, 0x55bd1cdad49f699cull,
    0x56ac1f752150a563ull, 0x579dbc56b48521baull, 0x5891fac0e95612c8ull, 0x5988e20954889245ull,
    0x5a827999fcef3242ull,
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

// w * 2^S of one logit.  (x - X) log2(e) / t is formed as an unevaluated sum
// of two floats (the subtraction's and the product's errors are exact by
// two-sum and fma); its integer part becomes a shift, the next six bits a
// table entry, and the rest e (|e| <= 2^-7) enters 2^e - 1 = y + y^2/2 +
// y^3/6 + y^4/24, y = e ln 2, whose first term is again a two-float product.
__device__ __forceinline__ u64 weight(float x, const Scale &c, const u64 *table) {
  if (x == c.top) return 1ull << c.shift;
  const float dh = x - c.top;
  const float ph = dh * c.ch;
  if (!(ph > -(float)(c.shift + 2))) return 0ull;      // below half a unit; -inf
  const float bb = dh - x;
  const float dl = (x - (dh - bb)) + (-c.top - bb);
  float pl = fmaf(dh, c.ch, -ph);
  pl = fmaf(dh, c.cl, pl);
  pl = fmaf(dl, c.ch, pl);
  const float n = rintf(ph), f = ph - n;
  const float jf = rintf(f * 64.f);
  const float e = fmaf(jf, -1.f / 64.f, f);            // exact
  constexpr float kLn2h = 0x1.62e430p-1f, kLn2l = -1.9046543e-9f;   // ln 2
  const float yh = e * kLn2h;
  float yl = fmaf(e, kLn2h, -yh);
  yl = fmaf(e, kLn2l, yl);
  yl = fmaf(pl, kLn2h, yl);
  // yh on a grid of 2^-38, what is left of it to the small terms
  const float gh = rintf(yh * 0x1p38f);
  const float rest = fmaf(gh, -0x1p-38f, yh) + yl;
  const float y = yh + yl;
  const float q = fmaf(fmaf(y, 1.f / 24.f, 1.f / 6.f), y, 0.5f);
  const float small = fmaf(y * y, q, rest);            // |.| < 2^-14
  const long long m46 = (1ll << 46) + ((long long)(int)gh << 8) + (long long)(int)rintf(small * 0x1p46f);
  const u64 w60 = __umul64hi((u64)m46 << 16, table[(int)jf + 32]);   // 2^(f) * 2^60
  const int sh = 60 - c.shift - (int)n;
  return sh > 63 ? 0ull : (w60 + (1ull << (sh - 1))) >> sh;
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
  u64 table[65];
  u64 warp[kWarps];         // a pass's sum per warp
  u64 sum[3];               // this block's sums: weights to cut, ties, kept weights
  u64 best;                 // this block's largest (key, ~index)
  float least;              // and its smallest logit above -inf
  uint32_t n_cand;
  u64 left, total;          // a search's answer
  int bin, count;
  u64 cut;                  // the cut: key << 32 | last index kept with that key
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
// The same shared variable in block `rank` of the cluster.
__device__ __forceinline__ u64 remote(const u64 *p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];"
               : "=l"(v) : "r"(tcx::map_to_rank(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t remote(const uint32_t *p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(v) : "r"(tcx::map_to_rank(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ float remote(const float *p, uint32_t rank) {
  return __uint_as_float(remote(reinterpret_cast<const uint32_t *>(p), rank));
}
__device__ __forceinline__ void remote_store(u64 *p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tcx::map_to_rank(smem_u32(p), rank)), "l"(v)
               : "memory");
}
__device__ __forceinline__ uint32_t remote_add(uint32_t *p, uint32_t rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(old) : "r"(tcx::map_to_rank(smem_u32(p), rank)), "r"(v) : "memory");
  return old;
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
  u64 before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const u64 t = sh.warp[w];
    before += w < warp ? t : 0;
    all += t;
  }
  *total = all;
  return before + incl - v;
}

// Adds a weight to bin b of this block's histogram, in three 16-bit parts:
// their sums over a slice of at most 2^16 tokens stay below 2^32.
__device__ __forceinline__ void add_weight(Shared &sh, int b, u64 m) {
  atomicAdd(&sh.m0[b], (uint32_t)m & 0xffffu);
  const uint32_t hi = (uint32_t)(m >> 16) & 0xffffu, top = (uint32_t)(m >> 32);
  if (hi) atomicAdd(&sh.m1[b], hi);
  if (top) atomicAdd(&sh.m2[b], top);
}
__device__ __forceinline__ u64 remote_weight(const Shared &sh, int b, int rank) {
  return (u64)remote(&sh.m0[b], rank) + ((u64)remote(&sh.m1[b], rank) << 16) + ((u64)remote(&sh.m2[b], rank) << 32);
}

// The consecutive range of a block's n tokens that warp w owns.
__device__ __forceinline__ int warp_begin(int n, int w) {
  return min(n, w * (((n + kWarps - 1) / kWarps + 31) / 32 * 32));
}

// This block's sum of f(i) over its tokens, left in sh.sum[slot] and, per
// warp, in sh.warp; then meets the cluster.  Returns the sums of the blocks
// before this one, and of all in *total.
template <typename F>
__device__ __forceinline__ u64 cluster_sum(Shared &sh, int slot, int n, int rank, int C, F f, u64 *total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = warp_begin(n, warp + 1);
  u64 s = 0;
  for (int i = warp_begin(n, warp) + lane; i < e; i += 32) s += f(i);
  s = warp_sum64(s);
  __syncthreads();
  if (lane == 0) sh.warp[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    u64 t = 0;
    for (int w = 0; w < kWarps; ++w) t += sh.warp[w];
    sh.sum[slot] = t;
  }
  cluster_barrier();
  u64 before = 0, all = 0;
  for (int c = 0; c < C; ++c) {
    const u64 v = remote(&sh.sum[slot], c);
    if (c < rank) before += v;
    all += v;
  }
  *total = all;
  return before;
}

// After cluster_sum over the same f: the token at which the running sum over
// the cluster, `before` at this block's first token, first exceeds `target`
// is passed to found(i) by one thread of the block that holds it.
template <typename F, typename G>
__device__ __forceinline__ void ordered_find(const Shared &sh, int n, u64 before, u64 target, F f, G found) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  u64 acc = before;
  for (int w = 0; w < warp; ++w) acc += sh.warp[w];
  if (target < acc || target >= acc + sh.warp[warp]) return;
  const int e = warp_begin(n, warp + 1);
  for (int i0 = warp_begin(n, warp); i0 < e; i0 += 32) {
    u64 v = i0 + lane < e ? f(i0 + lane) : 0ull;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, acc + v > target);
    if (hit) {
      if (lane == __ffs(hit) - 1) found(i0 + lane);
      return;
    }
    acc += __shfl_sync(0xffffffffu, v, 31);
  }
}

// Sorts a[0 .. n) ascending (n a power of two); the block's threads all call.
__device__ __forceinline__ void sort_block(u64 *a, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      for (int t = threadIdx.x; t < n / 2; t += kThreads) {
        const int i = (t / j) * 2 * j + t % j, l = i + j;
        const u64 x = a[i], y = a[l];
        if ((x > y) == ((i & k) == 0)) {
          a[i] = y;
          a[l] = x;
        }
      }
      __syncthreads();
    }
}
// Sorts the first n gathered tokens (padded to a power of two); returns that
// power.
__device__ __forceinline__ int sort_cand(Shared &sh, int n) {
  int m = 2;
  while (m < n) m <<= 1;
  for (int i = n + threadIdx.x; i < m; i += kThreads) sh.cand[i] = ~0ull;
  __syncthreads();
  sort_block(sh.cand, m);
  return m;
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
      u64 s = 0;
      for (int c = 0; c < C; ++c) s += MASS ? remote_weight(sh, b, c) : (u64)remote(&sh.cnt[b], c);
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
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) {
      best = sh.warp[w] > best ? sh.warp[w] : best;
      mn = fminf(mn, wmin[w]);
    }
    sh.best = best;
    sh.least = mn;
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
  if (threadIdx.x < 65) sh.table[threadIdx.x] = kExp2Table[threadIdx.x];
  if (threadIdx.x == 0) sh.n_cand = 0;
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.cnt[i] = sh.m0[i] = sh.m1[i] = sh.m2[i] = 0;
  grid_dep_wait();
  grid_dep_launch();
  const float temp = P.temperature ? P.temperature[row] : 1.f;
  const int k = P.top_k ? P.top_k[row] : 0;
  const float p = P.top_p ? P.top_p[row] : 1.f;
  const float mp = P.min_p ? P.min_p[row] : 0.f;
  const float u = P.u[row];
  load_slice(sh, x, reinterpret_cast<const T *>(P.logits) + (int64_t)row * P.ld + lo, n, lo);
  cluster_barrier();
  u64 best = 0;
  float low = INFINITY;
  for (int c = 0; c < C; ++c) {
    const u64 t = remote(&sh.best, c);
    best = t > best ? t : best;
    low = fminf(low, remote(&sh.least, c));
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
  {
    // log2(e) / t as two floats; a temperature below 1e-30 acts as 1e-30
    const double c = 1.4426950408889634 / (double)fmaxf(temp, 1e-30f);
    sc.ch = (float)c;
    sc.cl = (float)(c - (double)sc.ch);
  }
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
    const float scale = (float)kBins / fmaxf(range * 1.0001f, 1e-35f);
    auto bin_of = [&](float v) -> int {               // monotone in v
      const float t = (sc.top - v) * scale;
      return t < (float)kBins ? (int)t : kBins;
    };
    wide = sc.top == INFINITY;                        // no distance to measure by
    if (!wide) {
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const float v = to_f(x[i]);
        const int b = bin_of(v);
        if (b >= kBins) continue;
        atomicAdd(&sh.cnt[b], 1u);
        if (use_p) {
          const u64 m = weight(v, sc, sh.table);
          if (m) add_weight(sh, b, m);
        }
      }
      cluster_barrier();
      const int per = kBins / C;
      for (int b = rank * per + threadIdx.x; b < (rank + 1) * per; b += kThreads) {
        u64 s = 0;
        uint32_t q = 0;
        for (int c = 0; c < C; ++c) {
          q += remote(&sh.cnt[b], c);
          if (use_p) s += remote_weight(sh, b, c);
        }
        sh.rmass[b] = s;
        sh.rcnt[b] = q;
      }
      cluster_barrier();
      // every block scans all bins, two per thread, from the maximum down
      static_assert(kBins == 2 * kThreads, "two bins per thread");
      const int b = threadIdx.x * 2;
      const uint32_t q0 = remote(&sh.rcnt[b], b / per), q1 = remote(&sh.rcnt[b + 1], b / per);
      u64 count, total = 0, w0 = 0, w1 = 0, wacc = 0;
      const u64 qacc = block_scan(sh, (u64)q0 + q1, &count);
      if (use_p) {
        w0 = remote(&sh.rmass[b], b / per);
        w1 = remote(&sh.rmass[b + 1], b / per);
        wacc = block_scan(sh, w0 + w1, &total);
      }
      use_k = use_k && (u64)k <= count;               // else only vanished weights fall to it
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
          for (int i0 = threadIdx.x & ~31; i0 < n; i0 += kThreads) {
            const int i = i0 + (threadIdx.x & 31);
            const float v = i < n ? to_f(x[i]) : -INFINITY;
            const int bi = i < n ? bin_of(v) : kBins;
            const bool take = small ? bi <= step : bi == step;
            const uint32_t mask = __ballot_sync(0xffffffffu, take);
            if (mask == 0) continue;
            uint32_t base = 0;
            const int leader = __ffs(mask) - 1, lane = threadIdx.x & 31;
            if (lane == leader) base = remote_add(&sh.n_cand, 0, __popc(mask));
            base = __shfl_sync(0xffffffffu, base, leader);
            if (take)
              remote_store(&sh.cand[base + __popc(mask & ((1u << lane) - 1))], 0, pack(key_of(v), lo + i));
          }
          cluster_barrier();
          if (rank == 0) {
            const int nc = small ? down : in_step;
            const u64 in_left = sh.left, all = sh.total;
            sort_cand(sh, nc);
            // thread t holds sorted tokens 4t .. 4t + 3 and their weights
            u64 w[4], s = 0, sum;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = threadIdx.x * 4 + e;
              w[e] = i < nc && (small || use_p) ? weight(value_of(packed_key(sh.cand[i])), sc, sh.table) : 0ull;
              s += w[e];
            }
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
              // kept: what lies before it is short of need_p, and w >= least
              u64 acc = acc0;
              u64 kept_n = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const bool keep = w[e] >= least && acc < need_p;
                acc += w[e];
                kept_n += keep;
              }
              u64 nm;
              block_scan(sh, kept_n, &nm);
              __syncthreads();
              // the kept tokens by index
              u64 item[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i = threadIdx.x * 4 + e;
                const u64 v = i < (int)nm ? sh.cand[i] : 0ull;
                item[e] = ((u64)(uint32_t)v << 32) | packed_key(v);
              }
              __syncthreads();
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((int)threadIdx.x * 4 + e < (int)nm) sh.cand[threadIdx.x * 4 + e] = item[e];
              __syncthreads();
              sort_cand(sh, (int)nm);
              s = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i = threadIdx.x * 4 + e;
                w[e] = i < (int)nm ? weight(value_of((uint32_t)sh.cand[i]), sc, sh.table) : 0ull;
                s += w[e];
              }
              acc = block_scan(sh, s, &sum);
              const u64 target = u >= 1.f ? sum - 1 : u > 0.f ? scaled(sum, u, &more) : 0ull;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (acc <= target && target < acc + w[e])
                  P.tokens[row] = (int)(sh.cand[threadIdx.x * 4 + e] >> 32);
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
        cluster_sum(sh, 0, n, rank, C, [&](int i) {
          const float v = to_f(x[i]);
          return (int64_t)key_of(v) > above ? weight(v, sc, sh.table) : 0ull;
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
      auto is_tie = [&](int i) { return key_of(to_f(x[i])) == cut_key ? 1ull : 0ull; };
      u64 ties;
      const u64 before = cluster_sum(sh, 1, n, rank, C, is_tie, &ties);
      if (ties > cut_left) {                          // the same in every block
        ordered_find(sh, n, before, cut_left - 1, is_tie, [&](int i) {
          for (int c = 0; c < C; ++c) remote_store(&sh.cut, c, (u64)(lo + i));
        });
        cluster_barrier();
        last = (int)sh.cut;
      }
    }
  }
  auto kept = [&](int i) {
    const float v = to_f(x[i]);
    if (cut) {
      const uint32_t key = key_of(v);
      if (key < cut_key || (key == cut_key && lo + i > last)) return 0ull;
    }
    const u64 w = weight(v, sc, sh.table);
    return w >= least ? w : 0ull;
  };
  u64 total;
  const u64 before = cluster_sum(sh, 2, n, rank, C, kept, &total);
  bool more;
  const u64 target = u >= 1.f ? total - 1 : u > 0.f ? scaled(total, u, &more) : 0ull;
  ordered_find(sh, n, before, target, kept, [&](int i) { P.tokens[row] = lo + i; });
  cluster_barrier();                                  // its shared memory has been read
}

template <typename T>
static size_t smem_bytes(int slice) {
  return (sizeof(Shared) + 15) / 16 * 16 + (size_t)slice * sizeof(T);
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
