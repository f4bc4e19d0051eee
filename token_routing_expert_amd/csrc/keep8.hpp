// keep8.hpp -- the arithmetic of an 8-bit checkpoint's block: 64 values as
// whole multiples of s = max(amax, 2^-100) / 127 (include/moe_training.h).
// Pre-activations that a backward computes again pass between its products in
// 16-bit codes of the same kind (whole multiples of amax / 32767): as many bytes
// as bf16, and 2e-5 of the values' size off instead of 1.7e-3, which showed in
// every gradient (0.34% off in the 2-norm, with codes 0.24%).
//
// Magnitudes are compared as integers (bits without the sign), where infinity
// and NaN are the largest, so a block that holds one shows it in amax and gets
// a NaN scale.  The floor keeps 127 / amax finite; what lies below it rounds to
// the code 0.  A quotient is formed with the hardware's reciprocal (one step
// off): a code differs from the exact quotient's only where that lies within
// 2^-15 of a half, by one.  That reciprocal has no subnormal results, so it is
// taken of 2^-8 amax: from 2^126 on it would be zero otherwise.
#pragma once

#include "common.hpp"

namespace tre {

// The scale of a block whose largest magnitude has these bits, and its inverse,
// for codes of 8 or 16 bits.
template <int BITS = 8>
__device__ __forceinline__ void keep_scale(uint32_t amax_bits, float& scale, float& inv) {
  constexpr uint32_t kFloor = (uint32_t)(127 - 100) << 23;   // 2^-100
  constexpr float kTop = (float)((1 << (BITS - 1)) - 1);
  const float amax = __builtin_bit_cast(float, amax_bits > kFloor ? amax_bits : kFloor);
  const bool finite = amax_bits < 0x7F800000u;
  scale = finite ? amax * (1.f / kTop) : __builtin_bit_cast(float, 0x7FC00000u);
  inv = finite ? kTop * 0x1p-8f * __builtin_amdgcn_rcpf(amax * 0x1p-8f) : 0.f;
}

// Four codes, the first in the lowest byte.  |v inv| <= 127 (1 + 2^-21), and
// adding 1.5 * 2^23 rounds it to the nearest whole number (ties to even), whose
// lowest byte is the code's two's complement.
__device__ __forceinline__ uint32_t keep_codes4(float a, float b, float c, float d, float inv) {
  constexpr float kRound = 12582912.f;
  const uint32_t ia = __builtin_bit_cast(uint32_t, fmaf(a, inv, kRound));
  const uint32_t ib = __builtin_bit_cast(uint32_t, fmaf(b, inv, kRound));
  const uint32_t ic = __builtin_bit_cast(uint32_t, fmaf(c, inv, kRound));
  const uint32_t id = __builtin_bit_cast(uint32_t, fmaf(d, inv, kRound));
  return __builtin_amdgcn_perm(ib, ia, 0x0c0c0400u) | __builtin_amdgcn_perm(id, ic, 0x04000c0cu);
}

// The values of four codes (the conversion takes a byte with its sign; the product
// is rounded once, and finite wherever the values that were kept are).
__device__ __forceinline__ void keep_values4(uint32_t codes, float s, float* v) {
  v[0] = (float)(int8_t)codes * s;
  v[1] = (float)(int8_t)(codes >> 8) * s;
  v[2] = (float)(int8_t)(codes >> 16) * s;
  v[3] = (float)(int8_t)(codes >> 24) * s;
}

// The same with two 16-bit codes a dword.
__device__ __forceinline__ uint32_t keep_codes2(float a, float b, float inv) {
  constexpr float kRound = 12582912.f;
  return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, fmaf(b, inv, kRound)),
                               __builtin_bit_cast(uint32_t, fmaf(a, inv, kRound)), 0x05040100u);
}
__device__ __forceinline__ void keep_values2(uint32_t codes, float s, float* v) {
  v[0] = (float)(int16_t)codes * s;
  v[1] = (float)(int16_t)(codes >> 16) * s;
}

// max over 16 consecutive lanes (quads, then mirrored halves)
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));    // lane ^ 1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));    // lane ^ 2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));   // mirror in 8 lanes
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));  // mirror in 16 lanes
}

// One block of a row's checkpoint by 16 lanes, four columns each (v[0] its gates,
// v[1] its ups, at column c of I): codes and scales, and of 8 bits h in bf16 or float32.
template <int BITS, typename H>
__device__ __forceinline__ void keep_block(const f32x4 (&v)[2], int64_t row, int c, int I, int l16, const Kept& kept,
                                           H* __restrict__ h) {
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, abs_bits(v[hf][i]));
    float s, inv;
    keep_scale<BITS>(max16(m), s, inv);
    const int64_t at = (row * 2 + hf) * I + c;
    if constexpr (BITS == 8)
      *(uint32_t*)(kept.q + at) = keep_codes4(v[hf][0], v[hf][1], v[hf][2], v[hf][3], inv);
    else
      *(uint2*)(kept.q + 2 * at) = make_uint2(keep_codes2(v[hf][0], v[hf][1], inv), keep_codes2(v[hf][2], v[hf][3], inv));
    if (l16 == 0) kept.s[(row * 2 + hf) * (I / kKeepBlock) + c / kKeepBlock] = s;
  }
  if constexpr (BITS == 8) {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[0][i] * __builtin_amdgcn_rcpf(1.f + __expf(-v[0][i])) * v[1][i];
    if constexpr (sizeof(H) == 4)
      *(f32x4*)(h + row * I + c) = f32x4{f[0], f[1], f[2], f[3]};
    else
      *(uint2*)(h + row * I + c) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  }
}

// A row of an MFMA result block: 32 columns in lanes l and l + 32, register q4
// holding columns 8 q4 + 4 (l / 32) .. +3 as one dword.  to_halves gives lane l
// the dwords of columns 16 (l / 32) .. +15 in order, from_halves takes them back.
__device__ __forceinline__ u32x4 to_halves(const uint32_t (&q)[4]) {
  const auto a = __builtin_amdgcn_permlane32_swap(q[0], q[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(q[1], q[3], false, false);
  return u32x4{a[0], a[1], b[0], b[1]};
}

__device__ __forceinline__ void from_halves(const u32x4& v, uint32_t (&q)[4]) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[1], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[2], v[3], false, false);
  q[0] = a[0];
  q[2] = a[1];
  q[1] = b[0];
  q[3] = b[1];
}

// The same for two bytes a column: lane l loaded columns 8 (l / 32) .. +7 of a
// 16-column half (four dwords); q[w][g], q[w][g + 1] get dword w of the half's
// two 4-column groups.
__device__ __forceinline__ void from_quarters(const u32x4& v, uint32_t (&q)[2][4], int g) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const auto a = __builtin_amdgcn_permlane32_swap(v[w], v[2 + w], false, false);
    q[w][g] = a[0];
    q[w][g + 1] = a[1];
  }
}

}  // namespace tre
