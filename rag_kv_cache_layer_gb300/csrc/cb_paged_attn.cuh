// Parameters and variants of the paged attention, shared by its kernels.
#pragma once

#include "cb_common.cuh"
#include "cb_internal.h"

namespace cb {
namespace paged {

// An item of the few-rows kernel whose keys more than one block has: its rows
// (0: nothing to join), its first kv head, the last block with a piece, and whether the first
// block's piece is its second.
struct Join {
  int row0, l0, rows, g, last, second;
};

// x / d for 0 <= x < 2^31 by one product: m = ceil(2^s / d) with s = 31 +
// ceil(log2 d) is off by less than 2^(s - 31) / d.  The kernels' index
// arithmetic lies on every piece's path, where a division costs 20 dependent
// instructions.
struct Divisor {
  uint32_t d, m;
  int s;
  explicit Divisor(int by = 1) : d(by), s(31) {
    while ((1u << (s - 31)) < d) ++s;
    m = (uint32_t)(((1ull << s) + d - 1) / d);
  }
  __device__ __forceinline__ int div(int x) const { return (int)(((uint64_t)(uint32_t)x * m) >> s); }
};

struct AttnParams {
  PagedKV kv;
  const void *q;
  void *out;
  int64_t ld_q, ld_out;
  int n_rows, G, Hkv, max_kv;
  int n_split;                            // parts of a unit's key range (chunk kernel)
  // Sequences by rows (queries x G): the few-rows kernel takes those up to
  // few_hi, the chunk kernel those above rows_lo.
  int few_hi, rows_lo;
  int hc;                                 // kv heads per item of the few-rows kernel
  Divisor by_G, by_quads;                 // G; Hkv / hc
  float scale_log2;                       // softmax scale times log2(e)
  float *part_o;                          // unnormalised partial rows, HD floats each
  float2 *part_ml;                        // (m, l) of each partial row
  Join *joins;                            // one per block of the few-rows kernel
};

// Few rows per sequence, and all of fp32: R (16, 32 or 64) rows per tile.  The
// workspace holds 2 * decode_grid() * R * hc partial rows and decode_grid()
// joins.
int decode_grid();
int decode_heads(int R, int64_t tiles, int Hkv);   // hc, for that many tiles
cudaError_t launch_decode(const AttnParams &P, int R, int hd, cb_dtype dt, int *status, cudaStream_t s);

// bf16, many rows: units of R (128 or 256) rows, their keys in n_split parts;
// the workspace holds units * Hkv * n_split * R partial rows if n_split > 1.
cudaError_t launch_chunk(const AttnParams &P, int R, int64_t units, int hd, int *status, cudaStream_t s);

}  // namespace paged
}  // namespace cb
