// The 4-bit cache format shared by the append, the gather and the attention:
// blocks of 16 rows, 16 x 64 bytes of e2m1 codes then 16 x 8 e4m3 scales.
//
// e2m1 has two significant bits and e4m3 four, so code * scale has at most six:
// exact in bf16 and in fp16 (2^-10 .. 2688), which lets the attention feed the
// matrix instructions with 16-bit operands without rounding what is stored.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dd_common.cuh"

namespace dd {

constexpr int kRow4 = DD_KV4_ROW_BYTES;
constexpr int kBlk4 = 16 * kRow4;         // bytes of a block of 16 rows
constexpr int kBlk4Scales = 16 * 64;      // offset of its scales
constexpr int kMaxExp4 = 64;              // |e| of a head's 2^e

// 2^e for |e| <= 126, from the exponent's bits
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// The head's exponent, checked: one outside +-64 is reported and clamped.
__device__ __forceinline__ int head_exp(const int32_t *exps, int g, int32_t *status) {
  if (!exps) return 0;
  const int e = exps[g];
  if (e < -kMaxExp4 || e > kMaxExp4) {
    set_status(status, DD_ERR_DEVICE_CHECK);
    return e < 0 ? -kMaxExp4 : kMaxExp4;
  }
  return e;
}

// four bytes of codes -> four half2 (byte i: low nibble in .x, high nibble in .y)
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// two e4m3 scales (bytes of s) -> half2
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t s) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)s));
  return r;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A product with the reciprocal of a number is within 2^-22 of the quotient.  Where the
// numbers have 8 and 4 significant bits, the quotient is either a tie of the format that
// it is rounded to (at most five significant bits) or at least 2^-9 of it away, so
// rounding the product to 16 significant bits first puts every tie back in its place.
__device__ __forceinline__ float to_16_bits(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x80u) & ~0xFFu);
}

// Two groups' scales, the e4m3 numbers nearest to top / 6, at most 448 (0x7F, NaN, for a
// NaN group), and mul / scale (0 for a zero scale: all codes zero).  top: the largest
// magnitudes as bf16 bits, mul: a power of two that they are multiplied by first.
__device__ __forceinline__ void group_scales(uint32_t top_a, uint32_t top_b, float mul, uint32_t &sa, uint32_t &sb,
                                             float &inv_a, float &inv_b) {
  const float a = to_16_bits(__uint_as_float(top_a << 16) * mul * (1.f / 6.f));
  const float b = to_16_bits(__uint_as_float(top_b << 16) * mul * (1.f / 6.f));
  uint16_t s;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s) : "f"(b), "f"(a));
  sa = top_a > 0x7F80u ? 0x7Fu : (uint32_t)(s & 0xFF);
  sb = top_b > 0x7F80u ? 0x7Fu : (uint32_t)(s >> 8);
  const uint32_t h = e4m3x2_to_half2(s);
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  inv_a = f.x > 0.f ? __fdividef(1.f, f.x) * mul : 0.f;
  inv_b = f.y > 0.f ? __fdividef(1.f, f.y) * mul : 0.f;
}

// Eight bf16 values (x; v as they are) and mul / scale -> four bytes of codes.  The codes'
// ties are multiples of 1/4 and other quotients at least 2^-11 away from them, so
// rounding the product to multiples of 2^-13 puts every tie back in its place too, by two
// instructions of the FMA pipe: 1536 is added and taken away.  That loses the sign of a
// value that becomes 0, so the signs are taken from v.
__device__ __forceinline__ uint32_t encode8(const uint4 &v, const float (&x)[8], float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fadd_rn(fmaf(x[i], inv, 1536.f), -1536.f);
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  // value k's sign is bit 7 of byte k; times 17 it lies in bits 3 and 7 of bytes 1 and 3
  const uint32_t a = (__byte_perm(v.x, v.y, 0x7531) & 0x80808080u) * 17u;
  const uint32_t b = (__byte_perm(v.z, v.w, 0x7531) & 0x80808080u) * 17u;
  return r | (__byte_perm(a, b, 0x7531) & 0x88888888u);
}

}  // namespace dd
