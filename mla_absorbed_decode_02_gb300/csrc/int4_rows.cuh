// Cached tokens of 416 bytes: 512 four-bit codes n, 16 bf16 scales of 32 values each, 64 bf16 RoPE values.
//
// value = (n - 8) scale.  The scale has four significant bits and n - 8 three, so the value is a bf16 and one bf16 FMA finds
// it: 0x4300 | n are the bits of 128 + n, and (128 + n) s - 136 s has nothing to round (136 s has at most eight significant
// bits, 17 x 15 = 255).  Three instructions for two values.  E2M1 codes (FP4) take six (their magnitude and sign go to different
// places, and the exponent needs a product of its own), and the tensor cores take FP4 only with FP4 or FP8 on the other side,
// where the weights P are bf16.  On normal values the even steps are the closer ones, too: mean squared error 0.0073 against 0.0112 of
// the variance, with exact scales; rounding these up to four bits costs a tenth of that.
// A word holds the codes of eight dims, those of dims 2 i and 2 i + 1 16 bits apart: they come out as a pair.
#pragma once
#include "common.cuh"

namespace mla {

constexpr int kI4Row = 416;
constexpr int kI4Codes = 256, kI4Rope = kI4Codes + 32;  // offsets of the scales and of the RoPE values

// From 2^121 on 136 s is an infinity, which would make infinities of one sign of all codes: a product with a weight of 0, or a
// maximum, can lose those.  kI4Nan takes the place of such a scale, and every value is NaN.
__device__ __forceinline__ bool int4_scale_overflows(uint32_t s) { return (s & 0x7FFFu) >= 0x7C00u; }
constexpr uint32_t kI4Nan = 0x7FC07FC0u;
__device__ __forceinline__ uint32_t int4_offset(uint32_t s2) {  // -136 s of both halves
  uint32_t a2;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(a2) : "r"(s2), "r"(0xC308C308u));
  return a2;
}
// The eight values of a word, dims in order.  s2: the scale in both halves, a2 = int4_offset(s2).
__device__ __forceinline__ void expand_int4_word(uint32_t x, uint32_t s2, uint32_t a2, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = ((x >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o[i]) : "r"(v), "r"(s2), "r"(a2));
  }
}

// 16 latent values of a lane (bf16 numbers; lanes 2 k and 2 k + 1 share 32 values) -> two words of codes and the scale's
// bits: scale = amax / 7 rounded up to four significant bits, at least 2^-126 (1 for zeros); code = 8 + rint(x / scale), 1 .. 15.
// NaN in the place of the scale, codes of 8, where a value is not finite, or the scale above 2^119 (136 scale would overflow).
// The quotient is x r, r = 1 / scale, corrected once by its remainder (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990): correctly rounded for all 128 x 8 pairs of significands (tests/test_int4_rows.py), so
// that ties stay ties.  Outside (2^-60, 2^100) it is divided.
__device__ __forceinline__ void quantize_int4_16(const float (&x)[16], uint32_t (&code)[2], uint32_t& scale_bits) {
  uint32_t top = 0;  // of the magnitudes' bits: infinities and NaN are above all numbers
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  float scale = __uint_as_float((__float_as_uint(__uint_as_float(top) / 7.f) + 0xFFFFFu) & 0xFFF00000u);
  scale = fmaxf(scale, 0x1p-126f);
  const bool bad = top >= 0x7F800000u || scale > 0x1p119f;
  if (top == 0 || bad) scale = 1.f;
  scale_bits = bad ? 0x7FC0u : __float_as_uint(scale) >> 16;
  float z[16];
  if (__all_sync(0xffffffffu, scale > 0x1p-60f && scale < 0x1p100f)) {
    const float r = 1.f / scale;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float q = x[i] * r;
      z[i] = fmaf(fmaf(-q, scale, x[i]), r, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = x[i] / scale;
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    code[w] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // 1.5 x 2^23 + 8 + z: the sum is rounded to a whole number, whose last four bits are 8 + rint(z)
      const uint32_t n = __float_as_uint(z[8 * w + i] + 12582920.f) & 15u;
      code[w] |= n << (4 * (i >> 1) + 16 * (i & 1));
    }
    if (bad) code[w] = 0x88888888u;
  }
}

}  // namespace mla
