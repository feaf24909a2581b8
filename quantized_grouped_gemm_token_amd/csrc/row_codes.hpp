// Pairs of bf16; codes of a row's values from its scale: the rule of row_quant.hpp with one reciprocal
// per row in place of a division per value (few.hip, norm.hip, dense_i8.hip).
#pragma once

#include "common.hpp"

namespace w4a8 {

// two fp32 values -> bf16, round to nearest even (a NaN stays one), the first in the low half
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// x / s rounded to fp32 from r = 1 / s rounded: q = fl(x r), its residual x - q s in
// one FMA, and the corrected quotient, which is the correctly rounded one (Markstein's
// theorem where q is within an ulp; tests/test_few_division_cpu.py compares 2 10^7 pairs
// of an amax and a value below it, and 3.6 10^9 had no differing result).  3
// instructions instead of the ~10 of a division.
__device__ __forceinline__ float div_by(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

// the codes nearest to four quotients, the first in byte 0.  The FP8 conversion instruction rounds
// to nearest even like e4m3_encode (equal on every fp32 magnitude up to 448).  No clamp: a
// quotient is at most a rounding above 448 (127), which rounds to the largest code.
template <bool kInt8>
__device__ __forceinline__ uint32_t nearest4(float a, float b, float c, float d) {
  if constexpr (kInt8) {
    const float v[4] = {a, b, c, d};
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) o |= ((uint32_t)(int)rintf(v[i]) & 0xffu) << (8 * i);
    return o;
  } else {
    const int o = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, o, true);
  }
}
// four codes of four values of a row with scale s (r = 1 / s)
template <bool kInt8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s, float r) {
  return nearest4<kInt8>(div_by(a, s, r), div_by(b, s, r), div_by(c, s, r), div_by(d, s, r));
}

template <bool kInt8>
__device__ __forceinline__ float row_scale(float amax) {
  return amax > 0.0f ? amax / (kInt8 ? 127.0f : kFp8Max) : 1.0f;
}

// What a row is divided by: values and scale times `by`, a power of two that keeps 1 / s
// finite and the residual of div_by exact in rows of very small values; 1 in any other
// row.  s = 0 (amax below 2^-141): the codes do not matter, 0 times a finite one.
struct RowDivisor {
  float s, r, by;
};
__device__ __forceinline__ RowDivisor row_divisor(float scale) {
  RowDivisor d;
  d.by = scale < 0x1p-80f ? 0x1p100f : 1.0f;
  d.s = scale * d.by;
  d.r = d.s > 0.0f ? 1.0f / d.s : 0.0f;
  return d;
}
__device__ __forceinline__ bool rescaled(float by) { return __builtin_amdgcn_readfirstlane(__float_as_int(by)) != 0x3f800000; }

}  // namespace w4a8
