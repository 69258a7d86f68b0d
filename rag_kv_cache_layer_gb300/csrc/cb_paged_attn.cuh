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
  // 4-bit cache (kv.k_pages: the pool, kv.page_stride in bytes)
  int head_bytes = 0;                     // of one head's block of a page
  int scale_exp = 0;                      // scale_log2 is to be multiplied by 2^that
  float v_mul = 1.f;                      // 2^v_exp
  int pad = 0;                            // units that a tile counts beyond its blocks
};

// Few rows per sequence, and all of fp32: R (16, 32 or 64) rows per tile.  The
// workspace holds 2 * decode_grid() * R * hc partial rows and decode_grid()
// joins.
int decode_grid();
int decode_heads(int R, int64_t tiles, int Hkv);   // hc, for that many tiles
cudaError_t launch_decode(const AttnParams &P, int R, int hd, cb_dtype dt, int *status, cudaStream_t s);

// bf16, many rows: units of R (128 or 256) rows, their keys in n_split parts;
// the workspace holds units * Hkv * n_split * R partial rows if n_split > 1.
// q4: over a 4-bit cache.
struct ChunkPlan {
  int R, n_split;
  int64_t units;
};
ChunkPlan plan_chunk(int64_t n_rows, int S, int max_kv, int G, int Hkv, int hd);
cudaError_t launch_chunk(const AttnParams &P, int R, int64_t units, int hd, int *status, cudaStream_t s,
                         bool q4 = false);

// Blocks of a kernel that the current device takes at once in clusters of 1, 2, 4, 8 and 16 (0:
// no group of its SMs holds one), asked once per device; nullptr without a device.  `prepare`
// sets the kernel's attributes.
struct ClusterRoom {
  PerDeviceOnce once;
  int blocks[kMaxDevices][5];
  template <typename Prepare, typename... Params>
  const int *of(void (*kernel)(Params...), int threads, size_t smem, Prepare &&prepare) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    const cudaError_t e = once.run([&](int d) {
      const cudaError_t e = prepare();
      for (int i = 0; i < 5 && e == cudaSuccess; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1 << i);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 1 << i;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
          n = 0;
          cudaGetLastError();                   // (a size that the device refuses)
        }
        blocks[d][i] = n << i;
      }
      return e;
    });
    return e == cudaSuccess ? blocks[dev] : nullptr;
  }
};

// Blocks that a plan counts on at once in clusters of c, per_sm of them an SM: a cluster lies in
// one group of SMs, and not all groups are multiples of it (as cudaOccupancyMaxActiveClusters
// counts them on 152 SMs: 144 of 152 for 4; 120, and 288 of 304, for 8; 112 and 224 for 16).
inline int64_t cluster_room(int sms, int per_sm, int c) {
  return (int64_t)sms * per_sm * (c <= 2 ? 100 : c == 4 || (c == 8 && per_sm > 1) ? 94 : c == 8 ? 78 : 73) / 100;
}

// Blocks of an item's cluster (up to `most`, of eight warps) where each of `items` items has
// `blocks` key blocks; 0: the line, `parts` blocks of four warps.  The warps' rounds over
// their keys may be one more than on the line, which costs a launch and more parts to join;
// lengths below the bound leave a cluster idle and the line not.  Measured, one row each of
// S requests of one length (32/8 heads of 128), line and cluster: 3000 keys, S = 1 11.2 and
// 8.8 us, S = 4 13.2 and 10.4, S = 16 21.6 and 17.1; 8000 keys, S = 1 15.5 and 11.1.
// room: from ClusterRoom, a device may take fewer clusters than that, or none of a size.
inline int plan_cluster(int64_t items, int64_t blocks, int sms, int per_sm, int parts, int most, const int *room) {
  auto fits = [&](int c) {
    const int i = c == 1 ? 0 : c == 2 ? 1 : c == 4 ? 2 : c == 8 ? 3 : 4;
    return items * c <= cluster_room(sms, per_sm, c) && (!room || items * c <= room[i]);
  };
  int c = 1;
  while (c < most && 8 * c < blocks) c <<= 1;
  while (c > 1 && !fits(c)) c >>= 1;
  if (!fits(c)) return 0;
  const int64_t rounds = (blocks + 8 * c - 1) / (8 * c), line = (items * blocks + 4 * parts - 1) / (4 * parts);
  return rounds <= line + 1 ? c : 0;
}

// Tiles of R rows that n_rows rows over S sequences can make at most.
inline int64_t tile_bound(int64_t n_rows, int S, int G, int R) {
  const int64_t a = (n_rows * G + (int64_t)S * (R - 1)) / R;
  const int64_t b = n_rows * ((G + R - 1) / R);
  return a < b ? a : b;
}

}  // namespace paged
}  // namespace cb
