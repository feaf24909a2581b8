// 4-bit weights on the bf16 matrix cores, shared by the few-token layer
// (few.hip) and the matrix-vector product (matvec.hip).
//
// Both read every weight once for at most 16 activation rows, so they are bound
// by HBM and can afford the bf16 matrix cores, whose sums are fp32.  Largest and rms
// error over K = 128 in units of sum |products| (16 x 4096 outputs,
// test_one_group_on_the_bf16_matrix_cores), against a serial fp32 sum of the same:
//   activations                 INT4 (u and -8)           E2M1
//   normally distributed        9.7e-9, 6.2e-10           3.0e-8, 1.2e-9
//     a serial sum              9.7e-9, 4.9e-10           3.0e-8, 1.4e-9
//   spread over 24 binades      2.0e-7, 1.9e-8            1.8e-7, 2.9e-8
//     a serial sum              3.1e-7, 3.6e-8            4.5e-7, 4.9e-8
// The FP8 form that the grouped GEMMs use is off by up to 7.5e-6.  Every operand is
// exact in bf16: an FP8 or bf16 activation, an INT4 value u = q + 8 (0..15), an E2M1
// code times a power of two (below 2^128).
//
// The conversions are one instruction per two values at the rate of an FMA:
//   * INT4: two masks and a shift give the bytes u of a word; u read as E4M3 is
//     u 2^-9 (gemm_common.hpp), and the conversion's scale 2^9 makes it u.  The
//     offset leaves with a second product against a constant -8, the accumulator
//     input of the first: A x U + A x (-8) = A x Q;
//   * MXFP4: the conversion applies the block's E8M0 scale, exactly.
//
// Operand maps of v_mfma_f32_16x16x32_bf16: lane l supplies A row l % 16 and B
// column l % 16, K elements 8 (l / 16) .. +8; D lane l holds column l % 16, rows
// 4 (l / 16) .. +3.  A 128-wide K group takes four of them: with kq = l / 16,
// product c covers the K elements 32 kq + 8 c .. +8 of every lane, so a lane's 16
// weight bytes of a group (its 32 K elements from 32 kq) are its B operands in
// order, and the A side reads the same elements.
#pragma once

#include "gemm_common.hpp"

namespace w4a8 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma_bf16(i32x4 a, i32x4 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// eight E4M3 bytes -> eight bf16 values, times scale (a power of two)
__device__ __forceinline__ i32x4 e4m3x8_to_bf16(uint32_t lo, uint32_t hi, float scale) {
  i32x4 r;
  r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
  r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
  r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
  r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
  return r;
}

// eight INT4 values of one word as bf16 u = q + 8, in K order.  kRM: the word as
// stored (the nibble of k at bits 4 (k mod 8)); else the GEMM storage's order
// k0 k4 k1 k5 k2 k6 k3 k7.
template <bool kRM>
__device__ __forceinline__ i32x4 int4x8_to_bf16(uint32_t w) {
  uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  if constexpr (kRM) {                                        // lo: k0 k2 k4 k6, hi: k1 k3 k5 k7
    const uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u), b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
    lo = a;
    hi = b;
  }
  return e4m3x8_to_bf16(lo, hi, kUnitScale);
}

// the E8M0 byte b as the fp32 2^(b - 127) (b = 0 is a subnormal)
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// eight E2M1 codes of one word as bf16, times the block's scale
__device__ __forceinline__ i32x4 e2m1x8_to_bf16(uint32_t w, float scale) {
  i32x4 r;
  r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return r;
}

// orders LDS accesses of one wave's lanes (the LDS itself serves a wave in order)
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Loads of weights and scales through buffer resources: an offset past the resource's
// size reads as zero without touching memory, so a load of nothing (a wave's missing
// group, the step after the last) is the same instruction as any other, and a loop
// that refills registers as it uses them up needs no branch around its loads.  (With
// a branch, the compiler waits for each load at the branch's end.)  Weights are read
// once: without the hint (nt) the output head takes 75 instead of 67.5 us, gate/up of 16
// tokens 251 instead of 228; on scales, whose lines two blocks share, it only costs.
constexpr uint32_t kNowhere = 0x80000000u;                     // past every resource
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, int64_t bytes) {
  const int n = (int)(bytes < 0 ? 0 : bytes < 0x7fffffff ? bytes : 0x7fffffff);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, 0x00020000);   // gfx9: raw, untyped
}
__device__ __forceinline__ i32x4 buffer_load16_nt(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 2));   // 2: read once (nt)
}
__device__ __forceinline__ i32x4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ uint32_t buffer_load4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
}
__device__ __forceinline__ uint32_t buffer_load1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b8(r, (int)off, 0, 0);
}

// Scales come as one word per lane for four K groups: the word that lane group r of 16
// lanes holds (group 4 j + r, column l % 16) goes to every lane group of out[r], by
// three row swaps.  A load per group would cost as many load instructions as the
// weights themselves.
__device__ __forceinline__ void spread4(uint32_t v, uint32_t (&out)[4]) {
  const auto ab = __builtin_amdgcn_permlane16_swap(v, v, false, false);        // rows 0 0 2 2 | 1 1 3 3
  const auto a = __builtin_amdgcn_permlane32_swap(ab[0], ab[0], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(ab[1], ab[1], false, false);
  out[0] = a[0];
  out[1] = b[0];
  out[2] = a[1];
  out[3] = b[1];
}

// This workgroup's place in an order in which neighbours share an XCD (workgroups go to the
// 8 XCDs in turn).  Two neighbouring blocks of 16 columns share every 128-byte line of their
// scales, which the one L2 then reads once.
__device__ __forceinline__ int xcd_order() {
  const int n = gridDim.x, b = blockIdx.x;
  return n & 7 ? b : (b & 7) * (n >> 3) + (b >> 3);
}

constexpr int kMinus8 = (int)0xc100c100u;                      // two bf16 -8

// A x (-8) over one K group: what A x U is too large by
__device__ __forceinline__ v4f minus8_product(const i32x4 (&a)[4]) {
  const i32x4 m = {kMinus8, kMinus8, kMinus8, kMinus8};
  v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 4; ++c) d = mfma_bf16(a[c], m, d);
  return d;
}

// A x W of one K group and one 16-column subtile added to acc.  w: the lane's 16
// weight bytes; bias: minus8_product(a) (INT4 forms).  s: the group's scale (the
// fp32 scale's bits, or the E8M0 byte of the lane's 32 elements; unused per channel).
template <int kForm, bool kRM>
__device__ __forceinline__ void group_product(const i32x4 (&a)[4], i32x4 w, uint32_t s, v4f bias, v4f& acc) {
  if constexpr (kForm == kFormMx) {
    const float f = e8m0_to_f32(s);
#pragma unroll
    for (int c = 0; c < 4; ++c) acc = mfma_bf16(a[c], e2m1x8_to_bf16((uint32_t)w[c], f), acc);
  } else {
    v4f d = bias;
#pragma unroll
    for (int c = 0; c < 4; ++c) d = mfma_bf16(a[c], int4x8_to_bf16<kRM>((uint32_t)w[c]), d);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc[r] = kForm == kFormG128 ? fmaf(__uint_as_float(s), d[r], acc[r]) : acc[r] + d[r];
  }
}

}  // namespace w4a8
