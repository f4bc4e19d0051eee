// fp8.hpp -- the arithmetic of an e4m3 block with its scale, shared by the
// quantisation kernels and the 8-bit products.
//
// A block with largest magnitude amax gets s = 2^n, the smallest power of two
// with amax <= 448 s (n >= -126), and codes rne_e4m3(x / s).  With amax = m 2^e,
// m in [1, 2), and 448 = 1.75 * 2^8: n = e - 8 + (m > 1.75), read off amax's bits.
// Multiplying by 2^-n is exact (a result below 2^-126 rounds to the code 0
// either way), so the codes are those of the exact quotient and do not depend
// on the hardware's division; a scale amax / 448 would give quotients that round
// twice, and gains at most one of e4m3's 18 binades.  Magnitudes are compared
// as integers (bits without the sign), where infinity and NaN are the largest:
// a block that holds one shows it in amax, and all its codes become NaN.
#pragma once

#include "common.hpp"

namespace tre {

constexpr int kBlock = 128;                   // elements a scale covers in a row
constexpr uint32_t kNan8 = 0x7F7F7F7Fu;       // four NaN codes

// Bits of the scale 2^n for a block whose largest magnitude has these bits,
// and of 2^-n.
__device__ __forceinline__ void power_scale(uint32_t amax, float& scale, float& inv, bool& finite) {
  finite = amax < 0x7F800000u;
  int n = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  n = n < -126 ? -126 : n;
  scale = __builtin_bit_cast(float, finite ? (uint32_t)(n + 127) << 23 : 0x7FC00000u);
  inv = __builtin_bit_cast(float, (uint32_t)(127 - (finite ? n : 0)) << 23);
}

__device__ __forceinline__ uint32_t pack_fp8x4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// Eight codes as bf16, which holds every e4m3 value exactly.
__device__ __forceinline__ bf16x8 fp8x8_to_bf16(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// silu(g) * u = g / (1 + e^-g) * u with the hardware's exponential (of two) and
// reciprocal, one step off each: 11 instructions instead of about 40 with expf
// and a division, which a tile of 128 x 288 values feels.  e^-g = 2^t (1 + r
// ln 2) for t = -g log2(e) as rounded and r what the rounding left out, so the
// error does not grow with |g|: at most 8 half steps in all (exponential 2, its
// correction 1, sum 1, reciprocal 2, products 2).  silu is formed first: it is
// at most |g|, where g u may leave float32 although the result does not.  The
// denominator is taken a fourth, so that its reciprocal stays a normal number
// up to the largest e^-g; past that (g < -88.72) it is infinite and silu a
// zero, as in the formula.  r is far below a half wherever e^-g is neither zero
// nor infinite; the limits keep a huge g's from making a NaN of those.
__device__ __forceinline__ float swiglu(float g, float u) {
  constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;
  const float t = g * -kLog2e;
  const float r = __builtin_amdgcn_fmed3f(fmaf(g, -kLog2eLow, fmaf(g, -kLog2e, -t)), -0.5f, 0.5f);
  const float quarter = fmaf(__builtin_amdgcn_exp2f(t), fmaf(r, 0.25f * kLn2, 0.25f), 0.25f);
  return 0.25f * g * __builtin_amdgcn_rcpf(quarter) * u;
}

}  // namespace tre
