// MXFP4 on the device: blocks of 32 values share one power-of-two scale
// (E8M0, byte e + 127), each value one E2M1 code (sign, two exponent bits,
// one mantissa bit: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; the OCP
// microscaling formats), two codes a byte, the even value in the low nibble.
//
// Quantisation (of bf16 values): e is the smallest integer with
// max|x| <= 6 * 2^e, at most 125, so that every code times 2^e is finite in
// bf16 and no value saturates but those above 6 * 2^125 = 1.5 * 2^127; codes
// round x * 2^-e to nearest, ties to even.  x * 2^-e is exact in fp32 and every
// rounding border is a representable number, so codes and scales are defined bit
// for bit.
// Values (code * 2^e) are exact in bf16.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace csa {

constexpr int kMxBlock = 32;

// Scale byte of a block from the bf16 bits (sign cleared) of its largest
// magnitude.  amax = 1.f * 2^k <= 6 * 2^e = 1.5 * 2^(e+2): e = k - 2, one more
// when the fraction exceeds one half.  0 for a zero block; 255 (NaN) when a
// value is NaN or infinite; otherwise at most 252 (e = 126 would turn finite
// values into infinities: 4 * 2^126).
CSA_DEV uint32_t mx_scale_byte(uint32_t amax) {
  // (63 carries into the exponent where the fraction exceeds one half.)
  const int e = ((int)amax + 63 - 2 * 128) >> 7;
  return amax >= 0x7F80u ? 255u : (uint32_t)__vimin_s32_relu(e, 252);
}

// Eight fp32 values (pairs) -> eight codes, value i in bits 4i.
CSA_DEV uint32_t mx_codes8(const float2 (&x)[4]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x),
        "f"(x[3].y));
  return w;
}

// Eight bf16 values (pairs) of a block with scale byte `s` -> codes.
CSA_DEV uint32_t mx_quantise8(const uint32_t (&w)[4], uint32_t s) {
  // 2^(127 - s) brings the block into E2M1 range (s <= 252 for finite blocks).
  const float f = __uint_as_float((254u - min(s, 252u)) << 23);
  const float2 f2 = make_float2(f, f);
  float2 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = mul_f32x2(make_float2(bf16_lo(w[i]), bf16_hi(w[i])), f2);
  const uint32_t c = mx_codes8(x);
  return s == 255u ? 0u : c;  // a NaN block's codes are zero
}

// Largest magnitude of eight bf16 values, as bf16 bits (integer order of the
// magnitudes; NaN and infinity are the largest).
CSA_DEV uint32_t mx_amax8(const uint32_t (&w)[4]) {
  const uint32_t k = 0x7FFF7FFFu;
  const uint32_t a = __vmaxu2(__vmaxu2(w[0] & k, w[1] & k), __vmaxu2(w[2] & k, w[3] & k));
  return max(a & 0xFFFFu, a >> 16);
}

CSA_DEV uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Scale factors of a block as bf16 pairs.  A code's exponent and mantissa
// bits placed at bits 8..6 of a bf16 are its magnitude times 2^-126 (its zero
// exponent becomes a bf16 subnormal, which the multiply keeps), so the value
// is that times 2^126 * 2^(s-127) = 2^(s-1): one exact product for
// s <= 128, and a second factor 2^(s-128) (NaN for s = 255) above.
CSA_DEV uint32_t mx_bf16_lo(uint32_t s) { return ((min(s, 128u) + 126u) << 7) * 0x10001u; }
CSA_DEV uint32_t mx_bf16_hi(uint32_t s) {
  return (s == 255u ? 0x7FC0u : (max(s, 128u) - 1u) << 7) * 0x10001u;
}

// Eight codes (value i in bits 4i) -> eight bf16 values times `lo` as four
// pairs.  The high nibble of a byte of w << 4 (w) is the even (odd) code of
// its pair: one byte permute puts both into the high bytes of the two halves,
// sign in place and magnitude six bits too high.
CSA_DEV void mx_values8(uint32_t w, uint32_t lo, uint32_t (&o)[4]) {
  const uint32_t v = w << 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // bytes: 1 = byte i of v, 3 = byte i of w (0 and 2 are masked away)
    const uint32_t sel = (uint32_t)(i | (i << 4) | ((i + 4) << 8) | ((i + 4) << 12));
    const uint32_t r = __byte_perm(v, w, sel);
    o[i] = mul_bf16x2((r & 0x80008000u) | ((r >> 6) & 0x01C001C0u), lo);
  }
}

// The same in fp16, the form the attention's tensor cores take.  fp16 holds the
// codes and the factor 2^(s-127) of scale bytes 103 .. 142 (2^-24 .. 2^15): one
// conversion and one exact product a pair.  Values are exact from s = 104 to
// s = 140 (49152); a scale below 103 is zero.  Above 140 (where six times the
// scale passes fp16's range) the factor is NaN, whatever the block's codes:
// 255 is a NaN block, and an infinity could end as a weight of zero and be lost.
// The caller reports 141 .. 254.
constexpr uint32_t kMxF16Top = 140u;
CSA_DEV uint32_t mx_f16_scale(uint32_t s) {
  const float f = __uint_as_float(s << 23);  // 2^(s-127); 0 for s = 0
  return s > kMxF16Top ? 0x7FFF7FFFu : h2_bits(__floats2half2_rn(f, f));
}
CSA_DEV uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
CSA_DEV void mx_values8_f16(uint32_t w, uint32_t scale, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = mul_f16x2(o[i], scale);
}

}  // namespace csa
