// The 4-bit cache's format: 4-bit floats (sign, 2 exponent bits, 1 mantissa bit:
// 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one 8-bit float scale (4 exponent bits, 3
// mantissa bits) for 16 consecutive dimensions of a head: 4.5 bits a value.
//
// A page holds its kv heads one after the other; a head's block is
//   keys' codes [slot][hd / 2] | values' codes | keys' scales [slot][hd / 16] |
//   values' scales,
// so one head's part of a page is contiguous: the attention, which works head
// by head, reads whole lines whatever the page size is.
//
// A product code * scale has at most 2 + 4 significant bits and lies between
// 2^-10 and 2688: it is exact in fp16 (and in bf16).
#pragma once

#include <cuda_fp16.h>

#include "cb_common.cuh"

namespace cb {
namespace q4 {

constexpr int kGroup = 16;
constexpr float kMinScale = 0x1p-9f;        // the smallest scale: never zero

// Bytes of one head's block, and the places of its parts.
__host__ __device__ constexpr int head_bytes(int page, int hd) { return page * (hd + hd / 8); }
__host__ __device__ constexpr int codes_at(int page, int hd, bool v) { return v ? page * (hd / 2) : 0; }
__host__ __device__ constexpr int scales_at(int page, int hd, bool v) { return page * hd + (v ? page * (hd / 16) : 0); }

// Two codes of a byte, the low one first.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two scales of 16 bits, the low one first, as fp16.
__device__ __forceinline__ uint32_t decode_scales(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 s, t;\n\tmov.b32 {s, t}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// (v, v) of a pair's low or high half.
__device__ __forceinline__ uint32_t both(uint32_t h2, bool high) {
  uint32_t r;
  if (high) asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(h2));
  else asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(h2));
  return r;
}

// x / s toward zero with a sticky last bit (x, s finite, s > 0, q = 0 or
// normal): a further rounding to fewer bits then rounds the quotient itself.
__device__ __forceinline__ float divide_odd(float x, float s, float inv) {
  float q = x * inv;
  q = fmaf(fmaf(-q, s, x), inv, q);                   // within one step of x / s
  const float rest = fmaf(-q, s, x);                  // exact
  if (rest == 0.f) return q;
  uint32_t b = __float_as_uint(q);
  if ((rest < 0.f) != (x < 0.f)) --b;                 // |q| was too large
  return __uint_as_float(b | 1u);
}

__device__ __forceinline__ float reciprocal(float x) {      // to a step or two
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The scale of a group whose largest magnitude is a (as an 8-bit float): a / 6 to
// the nearest, ties to even, within [2^-9, 448]; and its value.
template <typename T>
__device__ __forceinline__ uint32_t scale_of(float a, float &value) {
  float r;
  if (sizeof(T) == 4 && a < 3e4f && a > 1e-6f) {
    r = divide_odd(a, 6.f, 1.f / 6.f);
  } else {
    // bf16: a has 8 bits, so a / 6 is a border between two scales (5 bits) or at least
    // 2^-9 of itself away from one: one correction makes a border exact, and the others'
    // rounding to fp32 does not matter (an infinity stays one by the choice of the larger)
    r = a * (1.f / 6.f);
    r = fmaxf(fmaf(fmaf(-r, 6.f, a), 1.f / 6.f, r), a > 1e30f ? a : 0.f);
  }
  uint32_t code;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(code) : "f"(0.f), "f"(r));
  code = max(code & 0xffu, 1u);
  value = __half2float(__ushort_as_half((unsigned short)(decode_scales(code) & 0xffffu)));
  return code;
}

// (x0, x1) in one register pair, and arithmetic on such pairs.
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ Pair fma_pair(Pair a, Pair b, Pair c) {
  Pair p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
  return p;
}
__device__ __forceinline__ Pair add_pair(Pair a, Pair b) {
  Pair p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
// Two 4-bit floats of a byte, x the low one.
__device__ __forceinline__ uint32_t encode2(float x, float y) {
  uint32_t two;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(two) : "f"(y), "f"(x));
  return two;
}
__device__ __forceinline__ uint32_t join4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Codes of 16 values x and their scale's code: codes[0] holds dimensions 0..7, the
// lowest four bits the first.  Each value is the 4-bit float nearest to x / scale
// (the quotient itself: ties go to the even code).
template <typename T>
__device__ __forceinline__ uint32_t quantise(float (&x)[kGroup], uint2 &codes) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < kGroup; ++i) a = fmaxf(a, fabsf(x[i]));
  float s;
  const uint32_t scale = scale_of<T>(a, s);
  if (a > 4096.f) {
    // far above 6 * 448, where every value saturates: keeps infinities out of the
    // quotient (NaN becomes a number too)
#pragma unroll
    for (int i = 0; i < kGroup; ++i) x[i] = fminf(fmaxf(x[i], -4096.f), 4096.f);
  }
  uint32_t two[8];
  if constexpr (sizeof(T) == 2) {
    // A value has 8 bits, border * scale at most 7: their quotient is a border (a multiple
    // of 1/4) or at least 2^-10 away from it.  Rounding to multiples of 2^-11, by adding
    // and taking off 1.5 * 2^12, restores met borders and keeps the others on their side.
    const float inv = reciprocal(s), big = 6144.f;
    const Pair inv2 = pair(inv, inv), up = pair(big, big), down = pair(-big, -big);
#pragma unroll
    for (int i = 0; i < kGroup; i += 2) {
      const Pair q = add_pair(fma_pair(pair(x[i], x[i + 1]), inv2, up), down);
      float q0, q1;
      asm("mov.b64 {%0, %1}, %2;" : "=f"(q0), "=f"(q1) : "l"(q));
      two[i / 2] = encode2(q0, q1);
    }
  } else {
    const float inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < kGroup; i += 2) {
      float q[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        q[k] = fabsf(x[i + k]) < 0.125f * s ? 0.f : divide_odd(x[i + k], s, inv);
      two[i / 2] = encode2(q[0], q[1]);
    }
  }
  codes = make_uint2(join4(two[0], two[1], two[2], two[3]), join4(two[4], two[5], two[6], two[7]));
  return scale;
}

// x a - y b (a, b fp32), correctly rounded to T: products and sum in pairs of floats, and an
// odd last bit in place of the rest where T has fewer.  The pair's own rounding loses up to
// 2^-46 of the larger product, which meets no border of bf16's values (8 bits); in fp32 it
// counts where the pair is close to the middle of two neighbours, as a value of few bits
// beside a tiny one may bring it: then `near` is set, and turned_near has the result.
template <typename T>
__device__ __forceinline__ float turned(float x, float a, float y, float b, bool &near) {
  // (__fmul_rn: a product that a sum took into an fma would not be the rounded one)
  const float h1 = __fmul_rn(x, a), l1 = fmaf(x, a, -h1), h2 = -__fmul_rn(y, b), l2 = fmaf(-y, b, -h2);
  const float s = h1 + h2, t = s - h1;
  const float e = (h1 - (s - t)) + (h2 - t) + (l1 + l2);
  const float hi = s + e, lo = e - (hi - s);
  uint32_t bits = __float_as_uint(hi);
  if (sizeof(T) == 4) {
    near = fmaf(lo, 1.f + 0x1p-18f, hi) != hi;  // lo is half a step, or nearly
    return hi;
  }
  if (lo != 0.f && hi != 0.f) {
    if ((lo < 0.f) != (hi < 0.f)) --bits;
    bits |= 1u;
  }
  return to_f(from_f<bf16>(__uint_as_float(bits)));
}
// x + y and what its rounding leaves.
__device__ __forceinline__ float add_rest(float x, float y, float &rest) {
  const float s = x + y, t = s - x;
  rest = (x - (s - t)) + (y - t);
  return s;
}
// x a - y b correctly rounded to fp32: all of the sum's rests, the last one as an odd bit.
__device__ __forceinline__ float turned_near(float x, float a, float y, float b) {
  const float h1 = __fmul_rn(x, a), l1 = fmaf(x, a, -h1), h2 = -__fmul_rn(y, b), l2 = fmaf(-y, b, -h2);
  float d, r1, r2;
  const float s = add_rest(h1, h2, d), l = add_rest(l1, l2, r1);
  float e = add_rest(d, l, r2);
  const float rest = r1 + r2;
  if (e == 0.f) {
    e = rest;
  } else if (rest != 0.f) {
    uint32_t bits = __float_as_uint(e);
    if ((rest < 0.f) != (e < 0.f)) --bits;
    e = __uint_as_float(bits | 1u);
  }
  return s + e;
}

// The power of two that brings a row's largest magnitude to [2^13, 2^14), as an exponent.
__device__ __forceinline__ int exponent_up(float top) { return top > 0.f ? 13 - ilogbf(top) : 0; }
// ... and what is left of the softmax's log2 scale, scale_log2 2^scale_exp: above 0, so that a
// masked -inf stays one (with a smaller scale every weight is 1 too), and finite, so that a
// score of 0 stays one (with a larger scale the largest score has all the weight too: scores
// differ by 2^-34 at least before it).  The cache's exponent is in scale_exp, since it may
// take the scale alone out of fp32 where a score is far inside.
__device__ __forceinline__ float scale_down(float scale_log2, int scale_exp, int up) {
  const int down = scale_exp - up;          // in two factors: 2^down may leave fp32
  return fminf(fmaxf(scale_log2 * ldexpf(1.f, down / 2) * ldexpf(1.f, down - down / 2), 0x1p-126f), 0x1.fffffep127f);
}
// A bf16 row (8 values each) to fp16 behind its power of two; the softmax's log2 scale of
// the row.
template <int N> __device__ __forceinline__ float scaled_row(uint4 (&v)[N], float scale_log2, int scale_exp) {
  __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 *e = reinterpret_cast<__nv_bfloat162 *>(v);
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) top2 = __hmax2(top2, __habs2(e[i]));
  const int up = exponent_up(fmaxf(__low2float(top2), __high2float(top2)));
  const float f1 = ldexpf(1.f, up / 2), f2 = ldexpf(1.f, up - up / 2);
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) {
    const float2 x = __bfloat1622float2(e[i]);
    const __half2 h = __floats2half2_rn(x.x * f1 * f2, x.y * f1 * f2);
    e[i] = *reinterpret_cast<const __nv_bfloat162 *>(&h);
  }
  return scale_down(scale_log2, scale_exp, up);
}

}  // namespace q4
}  // namespace cb
