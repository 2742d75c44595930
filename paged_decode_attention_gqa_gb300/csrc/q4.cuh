// Rows of the 4-bit cache: their layout (described in include/zl_decode_attn.h)
// and the conversions in both directions.
#pragma once

#include "../../include/zl_decode_attn.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace zl {

constexpr int kQ4Row = ZL_Q4_ROW_BYTES;
constexpr int kQ4VCodes = 64;    // first byte of V's codes
constexpr int kQ4KScales = 128;  // of K's scales
constexpr int kQ4VScales = 136;  // of V's scales
constexpr uint32_t kQ4BadScale = 255;

// Quotients of numbers below 2^31 by a number d that the host knows: x mul >> shift, with
// mul = 2^shift / d rounded up and 2^(shift - 31) the least power not below d, so that what
// mul is too large by, less than d / d, adds less than 1 / d.
struct Divisor {
  uint32_t mul, shift;
  Divisor() = default;
  explicit Divisor(uint32_t d) : shift(31) {
    while ((UINT64_C(1) << (shift - 31)) < d) ++shift;
    mul = uint32_t(((UINT64_C(1) << shift) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t quotient(uint32_t x) const {
    return uint32_t((uint64_t(x) * mul) >> shift);
  }
};

// ------------------------------------------------------------------- writing
// The scale of a block whose largest magnitude is the bf16 number of bits amax
// (NaN and infinity: 0x7F80 and above).
struct Q4Scale {
  float s, r;     // the scale and 1 / s to an ulp (0 for scale 0)
  uint32_t byte;
};
__device__ __forceinline__ Q4Scale q4_scale(uint32_t amax) {
  Q4Scale q;
  const bool bad = amax >= 0x7F80u;
  const float a = __uint_as_float(amax << 16);
  // a / 6: the product with the rounded 1 / 6 lies on the same side of every
  // border as the quotient (a has 8 significant bits, a border 5: checked for
  // every a), so the rounding below is that of the exact quotient.
  const float top = fminf(__fmul_rn(a, 1.f / 6.f), 10240.f);
  // To 3 bits behind the leading one, from 2^-14 down to multiples of 2^-17: in a
  // sum with 1.5 * 2^23 steps a step is the last bit.
  const uint32_t e = max(__float_as_uint(top) & 0x7F800000u, 113u << 23);
  const float big = __uint_as_float((e + (20u << 23)) | 0x400000u);
  q.s = __fsub_rn(__fadd_rn(top, big), big);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(q.s));
  q.r = q.s > 0.f ? r : 0.f;
  q.byte = uint32_t(__half_as_ushort(__float2half_rn(q.s))) >> 7;
  if (bad) {
    q.r = 0.f;
    q.byte = kQ4BadScale;
  }
  return q;
}

// Codes of 8 bf16 elements (element 0 in the low half of x[0], nibble 0 of the
// word): x / s by one Newton step behind the product with r, so that a quotient that is
// halfway between two codes comes out exact (with the bare product some ties fall off it).
// In terms of -x, two elements at a time; a zero keeps x's sign in every step. The
// conversion rounds to nearest, ties to even, and saturates at 6.
__device__ __forceinline__ uint32_t q4_codes(const uint32_t (&x)[4], const Q4Scale& q) {
  const uint64_t s = pack_f32x2(q.s, q.s), r = pack_f32x2(-q.r, -q.r);
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = x[i] ^ 0x80008000u;
    const uint64_t minus =
        pack_f32x2(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    const uint64_t first = mul_f32x2(minus, r);
    const float2 v = unpack_f32x2(fma_f32x2(fma_f32x2(first, s, minus), r, first));
    y[2 * i] = v.x;
    y[2 * i + 1] = v.y;
  }
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return q.byte == kQ4BadScale ? 0u : w;
}

// Largest magnitude of 8 bf16 elements, as bits; NaN counts as the largest.
__device__ __forceinline__ uint32_t q4_amax8(const uint32_t (&x)[4]) {
  // as integers: magnitudes order as their bits do, NaN above infinity
  const uint32_t m = __vmaxu2(__vmaxu2(x[0] & 0x7FFF7FFFu, x[1] & 0x7FFF7FFFu),
                              __vmaxu2(x[2] & 0x7FFF7FFFu, x[3] & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

// ------------------------------------------------------------------- reading
// The four pairs of a word's codes as fp16 pairs: r[i] = elements 2 i (low half)
// and 2 i + 1.
__device__ __forceinline__ void q4_pairs(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace zl
