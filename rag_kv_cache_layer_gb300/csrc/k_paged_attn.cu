// Paged attention's host side: which kernels a call runs, with which tiles and
// key splits, and the workspace they share.
#include "cb_common.cuh"
#include "cb_internal.h"
#include "cb_paged_attn.cuh"

namespace cb {
namespace paged {

// Tiles of R rows that n_rows rows over S sequences can make at most.
static int64_t tile_bound(int64_t n_rows, int S, int G, int R) {
  const int64_t a = (n_rows * G + (int64_t)S * (R - 1)) / R;
  const int64_t b = n_rows * ((G + R - 1) / R);
  return a < b ? a : b;
}

// How a call runs.
struct Plan {
  int few_R, hc;                          // few-rows kernel: rows per tile (0: not launched), heads per item
  int R;                                  // chunk kernel: rows per unit, 0: not launched
  int few_hi, rows_lo;                    // which sequences each takes
  int64_t tiles;                          // chunk units at most
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
// The model sees bounds: max_kv for every length, and up to a unit for every
// sequence.  A loose max_kv costs little (64 rows over 3200 keys: 15.6 us, 20.1 with
// a bound of 131,072; large chunks the same).  Single rows beside a chunk cost more:
// they count as units, so the chunk is split less or not at all, and the call lasts
// as long as its few CTAs (64 rows + 63 single rows, all over 16,384 keys: 894 us; as
// two calls 35 + 610).  The costs are those of head_dim 128; 64 is planned by them too.
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
// for.  Taken for single rows, one sequence's many rows are slower than through
// both kernels (128 over 8192 keys in 128 slots: 106 us and 88), and single rows
// are faster (64 over 2000 keys: 89 us and 94).
// The few-rows tile is 16, 32 or 64 rows by the average sequence, 16 where that
// exceeds 64.  The average is right for drafts alone and misleads in mixed calls,
// whose long sequences the chunk kernel takes (32/8 heads over 8192 keys unless
// stated; us with tiles of 16 / 32 / 64 rows, the rule's in brackets):
//   512 + 63 single rows                         435 / 442 / [701]
//   2048 + 63 single rows                      [618] / 624 / 877
//   512 + 32 drafts of 4, 16,384 keys          [484] / 490 / 752
//   512 + 16 drafts of 5 to 8, 64/8, 16,384    [712] / 644 / 618
// fp32 runs the few-rows kernel alone, whatever its rows.
static Plan plan(int64_t n_rows, int S, int max_kv, int G, int Hkv, int hd, cb_dtype dt) {
  Plan p = {};
  const int64_t all = n_rows * G, per_seq = (all + S - 1) / S;
  const bool few = dt == CB_F32 || all <= 64 || n_rows <= S;
  p.few_hi = 0x7fffffff;
  p.n_split = 1;
  if (few || S > 1) p.few_R = per_seq <= 16 ? 16 : per_seq <= 32 ? 32 : few || per_seq <= 64 ? 64 : 16;
  p.hc = p.few_R ? decode_heads(p.few_R, tile_bound(n_rows, S, G, p.few_R), Hkv) : 1;
  p.few_partials = p.few_R ? 2LL * decode_grid() * p.few_R * p.hc : 0;
  if (few) return p;
  if (S > 1) p.few_hi = p.rows_lo = 64;
  plan_chunk(p, n_rows, S, max_kv, G, Hkv, hd);
  p.partials = p.n_split == 1 ? 0 : p.tiles * Hkv * p.n_split * p.R;
  return p;
}

static size_t plan_bytes(const Plan &p, int hd) {
  const size_t row = hd * sizeof(float) + sizeof(float2);
  const size_t few = (size_t)p.few_partials * row + (p.few_R ? decode_grid() * sizeof(Join) : 0);
  const size_t rest = (size_t)p.partials * row;
  return few > rest ? few : rest;
}

// The partials of a launch reuse the workspace of the launch before it: each
// waits for its predecessor's end, and a merge has read them by then.
static cudaError_t run_plan(AttnParams P, const Plan &p, int hd, cb_dtype dt, void *ws, int *status,
                            cudaStream_t s) {
  auto bind = [&](int64_t partials) {
    P.part_o = reinterpret_cast<float *>(ws);
    P.part_ml = reinterpret_cast<float2 *>(P.part_o + (size_t)partials * hd);
    P.joins = reinterpret_cast<Join *>(P.part_ml + partials);
  };
  if (p.few_R) {
    bind(p.few_partials);
    const cudaError_t e = launch_decode(P, p.few_R, hd, dt, status, s);
    if (e != cudaSuccess) return e;
  }
  if (!p.R) return cudaSuccess;
  bind(p.partials);
  return launch_chunk(P, p.R, p.tiles, hd, status, s);
}

}  // namespace paged

size_t paged_attention_ws_bytes(int n_rows, int n_seq, int max_kv, int Hq, int Hkv, int hd, cb_dtype dt) {
  using namespace paged;
  if (n_rows <= 0 || n_seq <= 0) return 0;
  return plan_bytes(plan(n_rows, n_seq, max_kv, Hq / Hkv, Hkv, hd, dt), hd);
}

void paged_attention_plan(int n_rows, int n_seq, int max_kv, int Hq, int Hkv, int hd, cb_dtype dt, int64_t out[7]) {
  using namespace paged;
  const Plan p = plan(n_rows, n_seq, max_kv, Hq / Hkv, Hkv, hd, dt);
  const int64_t v[7] = {p.few_R, p.hc, decode_grid(), p.R, p.n_split, p.tiles, p.few_R ? p.few_hi : 0};
  for (int i = 0; i < 7; ++i) out[i] = v[i];
}

cudaError_t launch_paged_attention(const PagedKV &kv, const cb_paged_query &a, cb_dtype dt, int *status,
                                   cudaStream_t s) {
  using namespace paged;
  const int G = a.n_q_heads / a.n_kv_heads;
  const Plan p = plan(a.n_rows, kv.n_seq, a.max_kv_len, G, a.n_kv_heads, a.head_dim, dt);
  if (p.tiles * a.n_kv_heads * p.n_split > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  AttnParams P;
  P.kv = kv;
  P.q = a.q;
  P.out = a.out;
  P.ld_q = a.ld_q;
  P.ld_out = a.ld_out;
  P.n_rows = a.n_rows;
  P.G = G;
  P.Hkv = a.n_kv_heads;
  P.max_kv = a.max_kv_len;
  P.n_split = p.n_split;
  P.few_hi = p.few_hi;
  P.rows_lo = p.rows_lo;
  P.hc = p.hc;
  P.by_G = Divisor(G);
  P.by_quads = Divisor(a.n_kv_heads / p.hc);
  P.scale_log2 = a.scale * 1.4426950408889634f;
  return run_plan(P, p, a.head_dim, dt, a.ws, status, s);
}

}  // namespace cb
