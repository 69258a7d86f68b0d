// Stages and tensor core steps of the few-rows attention kernels over a cache of
// 16 or 32 bits: 16 query rows on the instruction's 16-row side.
#pragma once

#include "cb_common.cuh"

namespace cb {
namespace paged {

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

// 16 bytes to shared memory, or 16 zero bytes when `there` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
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

}  // namespace paged
}  // namespace cb
