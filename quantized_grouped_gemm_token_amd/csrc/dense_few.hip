// Dense products in 8-bit integers, and the gated block on them, for 1 to 16 rows (w4a8_block.h).
//
// Bound by reading the weights once.  A step is 16 weight rows (8 gate and 8 up rows in the
// gated product); the 8 waves of a workgroup split its K, in units of 128 bytes.  Each wave
// streams its units through a ring of its own in LDS, filled by loads straight into LDS, kSlots
// units ahead and across steps, with no barrier: an instruction loads 8 rows of 128 bytes, whole
// cache lines (reading the 16 rows of a product's operand directly, 64 bytes of each to an
// instruction, the same stream reached 4.0 to 5.6 TB/s where whole lines reach 5.8 to 7.0).  The
// activations stay in registers as operands of 16x16x64 INT8 products; the eight partial 16x16
// tiles (int32, exact) are summed in LDS at the end of a step, with the workgroup's one barrier.
//
// One workgroup a CU, persistent.  131072 x 6144 with one row takes 115 us (7.0 TB/s, what a plain
// read of whole lines reaches); 6144 x 6144 9.2 us with one row and 10.6 with 16, of which 3 are the
// launch and the first loads' way; 12288 x 6144 14.4 us.  Weights in a cache and 16 rows of more than 8192 outputs
// would go faster in the tiled kernel (16 x 12288 x 6144 13.2 against 15.7 us); read from memory, as a
// model's weights are, they do not (17.4 against 16.6; 16 x 24576 x 6144 31.9 against 27.3).  Half of the
// LDS cycles are bank conflicts: the operand reads take chunks q and 4 + q of a row, where dense_i8.hip's 2 q
// and 2 q + 1 have none.  A unit's two reads a wave hide behind its weights (the head reads at memory's rate).
//
// The gated block is two kernels: the gated product leaves act (fp32) and the maxima of 8
// columns of it; the down product's workgroups quantize act themselves, each wave its part of K,
// while their weights are in flight.
#include "block.hpp"
#include "gemm_common.hpp"
#include "lds_dma.hpp"
#include "row_codes.hpp"
#include "w4_bf16.hpp"

#include <type_traits>

namespace w4a8 {

namespace {

constexpr int kFewRowsWaves = 8;
constexpr int kFewRowsThreads = 64 * kFewRowsWaves;
constexpr int kUnit = 128;                   // K bytes of a unit: two products
constexpr int kUnitBytes = 16 * kUnit;

enum FewForm : int { kFewDense = 0, kFewGated = 1, kFewDown = 2 };

// |v| as an integer of its order, a NaN above infinity: a row with one gets a scale of NaN
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// (the swizzle of the tiled kernel's slots, dense_i8.hip)
__device__ __forceinline__ int few_swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

struct FewRowsArgs {
  DenseArgs d;            // gated: w13 with N = 2 I; down: w2, K = I, no a
  int64_t I;              // gated
  float* act;             // gated: written, down: read, [M][I]
  uint32_t* pmax;         // [M][I / 8]: magnitudes
};

// 16 values in scalar registers (uniform p): lane c's.  Scalar loads leave the ring's count of
// vector loads alone.
__device__ __forceinline__ float pick16(const float* p, int c) {
  const __attribute__((address_space(4))) float* u = (const __attribute__((address_space(4))) float*)(uintptr_t)p;
  float v = u[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) v = c == i ? u[i] : v;
  return v;
}

// LDS of a wave: its ring, then two buffers of partial tiles [16][16].  The down product
// converts act to codes, a unit at a time, in the second part (before it is used for tiles; next
// to them where a step goes over parts of K).
constexpr int kCodePitch = kUnit + 16;       // (16 bytes more: the rows of an operand start in different banks)
template <int kForm, bool kParts>
struct FewLds {
  static constexpr int kSlots = 4;
  static constexpr int kRing = kSlots * kUnitBytes, kTiles = 2 * 1024;
  static constexpr int kCodes = kForm == kFewDown ? 16 * kCodePitch : 0;
  static constexpr int kRegion = kParts ? kTiles + kCodes : kTiles > kCodes ? kTiles : kCodes;
  static constexpr int kBytes = kFewRowsWaves * (kRing + kRegion);
};

// GW: units of a wave held at once; kParts: K is longer than 8 GW units, and a step goes over parts
// of K and fetches each part's activations again.
template <int kForm, int GW, bool kParts>
__global__ __launch_bounds__(kFewRowsThreads) void dense_few_kernel(const FewRowsArgs f) {
  constexpr bool kGated = kForm == kFewGated, kDown = kForm == kFewDown;
  constexpr int kRows = kGated ? 8 : 16;       // outputs of a step
  using Lds = FewLds<kForm, kParts>;
  constexpr int kFewSlots = Lds::kSlots;
  __shared__ __attribute__((aligned(16))) uint8_t sm[Lds::kBytes];   // the rings, then the waves' regions
  __shared__ float row_s[16], row_f[16][3];   // down: a row's scale, what its values are divided by
  uint8_t* regions = sm + kFewRowsWaves * Lds::kRing;
  const DenseArgs& d = f.d;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int K = (int)d.K, M = (int)d.M;
  const int units = (K + kUnit - 1) / kUnit;
  const int nch = kParts ? (units + kFewRowsWaves * GW - 1) / (kFewRowsWaves * GW) : 1;
  const int64_t outs = kGated ? f.I : d.N;
  const int steps = (int)((outs + kRows - 1) / kRows);
  uint8_t* ring = sm + wave * Lds::kRing;

  // the wave's units of a part of K: g0 .. g0 + ng - 1
  auto units_of = [&](int ch, int& g0, int& ng) {
    const int all = min(kFewRowsWaves * GW, units - ch * kFewRowsWaves * GW);
    const int each = (all + kFewRowsWaves - 1) / kFewRowsWaves;
    g0 = ch * kFewRowsWaves * GW + wave * each;
    ng = max(0, min(each, all - wave * each));
  };
  // ---- the stream of weights: unit lu of part lch of step ls is the next one to load, into slot lslot
  // Neighbouring steps of a round run on one XCD (its L2 joins their short pieces of y's lines: 16
  // rows of 131072 outputs 124 against 132 us), those of a last round that is not whole on all.
  auto step_of = [&](int base) { return base + (base + (int)gridDim.x <= steps ? xcd_order() : (int)blockIdx.x); };
  int lbase = 0, ls = step_of(0), lch = 0, lu = 0, lslot = 0, lg0, lng;
  __amdgpu_buffer_rsrc_t r0, r1;
  const int lrow = lane >> 3;                  // rows lrow and lrow + 8 of the step: chunk lane % 8, swizzled
  const uint32_t woff0 = (uint32_t)(lrow * K + 16 * ((lane & 7) ^ few_swz(lrow)));
  const uint32_t woff1 = (uint32_t)((kGated ? lrow : lrow + 8) * K + 16 * ((lane & 7) ^ few_swz(lrow + 8)));
  auto point = [&]() {                         // (rows past the end are past the resource)
    const int64_t n0 = (int64_t)ls * kRows;
    if constexpr (kGated) {
      r0 = buffer_of(d.w + n0 * K, 8 * K);
      r1 = buffer_of(d.w + (f.I + n0) * K, 8 * K);
    } else {
      r0 = r1 = buffer_of(d.w + n0 * K, (d.N - n0 < 16 ? d.N - n0 : 16) * K);
    }
  };
  units_of(0, lg0, lng);
  // the first unit at or after (ls, lch, lu)
  auto settle = [&]() {
    while (ls < steps && lu >= lng) {
      lu = 0;
      if (kParts && ++lch < nch) {
        units_of(lch, lg0, lng);
      } else {
        lch = 0;
        lbase += (int)gridDim.x;
        ls = step_of(lbase);
        if (kParts) units_of(0, lg0, lng);
        if (ls < steps && lng > 0) point();
        if (!kParts && lng == 0) ls = steps;   // a wave without units
      }
    }
  };
  auto load = [&]() {
    const uint32_t k = (uint32_t)((lg0 + lu) * kUnit);
    uint8_t* to = ring + lslot * kUnitBytes;
    dma16_nt(r0, woff0, k, to);
    dma16_nt(r1, woff1, k, to + 8 * kUnit);
    lslot = lslot + 1 == kFewSlots ? 0 : lslot + 1;
    ++lu;
    settle();
  };

  i32x4 av[GW][2];
  const __amdgpu_buffer_rsrc_t ra = buffer_of(d.a, kDown ? 0 : (int64_t)(M - 1) * d.ld_a + K);
  auto load_a = [&](int g0, int ng) {          // (zeros past K and past the wave's units)
#pragma unroll
    for (int u = 0; u < GW; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (g0 + u) * kUnit + 16 * (4 * h + q);
        av[u][h] = buffer_load16(ra, u < ng && k < K ? (uint32_t)(min(col, M - 1) * (int)d.ld_a + k) : kNowhere);
      }
  };
  // down: act of unit g of every row, two rows an instruction, and its codes as operands
  uint8_t* mine = regions + wave * Lds::kRegion + (kParts ? Lds::kTiles : 0);
  auto fetch = [&](float4 (&v)[8], int g) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (2 * i < M)
        v[i] = *reinterpret_cast<const float4*>(f.act + (int64_t)min(2 * i + (lane >> 5), M - 1) * K + g * kUnit +
                                                4 * (lane & 31));
  };
  auto convert = [&](const float4 (&v)[8], i32x4 (&to)[2]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int m = 2 * i + (lane >> 5);
      if (2 * i < M) {
        const float s = row_f[m][0], r = row_f[m][1], by = row_f[m][2];
        *reinterpret_cast<uint32_t*>(mine + m * kCodePitch + 4 * (lane & 31)) =
            codes4<true>(v[i].x * by, v[i].y * by, v[i].z * by, v[i].w * by, s, r);
      }
    }
    wave_lds_fence();
#pragma unroll
    for (int h = 0; h < 2; ++h)
      to[h] = *reinterpret_cast<const i32x4*>(mine + min(col, M - 1) * kCodePitch + 16 * (4 * h + q));
    wave_lds_fence();
  };
  float4 av4[2][8];
  auto convert_all = [&](int g0, int ng) {     // (unit g0 is fetched; zeros past the wave's units)
#pragma unroll
    for (int u = 0; u < GW; ++u) {
      if (u < ng) {
        if (u + 1 < ng) fetch(av4[(u + 1) & 1], g0 + u + 1);
        convert(av4[u & 1], av[u]);
      }
    }
  };

  if (ls < steps && lng > 0) point();
  settle();
#pragma unroll
  for (int i = 0; i < kFewSlots; ++i)
    if (ls < steps) load();
  int g0, ng;
  units_of(0, g0, ng);
  if constexpr (kDown) {
    if (ng > 0) fetch(av4[0], g0);
    // the rows' scales: 32 threads a row over its maxima, four at a time
    const int m = threadIdx.x >> 5, fours = K >> 5;
    uint32_t top = 0;
    if (m < M)
#pragma unroll 2
      for (int c = threadIdx.x & 31; c < fours; c += 32) {
        const uint4 v = reinterpret_cast<const uint4*>(f.pmax + (int64_t)m * (K >> 3))[c];
        top = max(max(top, v.x), max(max(v.y, v.z), v.w));
      }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
    if ((threadIdx.x & 31) == 0) {
      const float scale = top == 0 ? 1.0f : __uint_as_float(top) / 127.0f;
      const RowDivisor v = row_divisor(scale);
      row_s[m] = scale, row_f[m][0] = v.s, row_f[m][1] = v.r, row_f[m][2] = v.by;
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);
    barrier_loads_in_flight();
    if constexpr (!kParts) convert_all(g0, ng);
  } else if constexpr (!kParts) {
    load_a(g0, ng);
  }
  // this thread's output of a step: row m, column c
  const int c = threadIdx.x & (kRows - 1), m = threadIdx.x / kRows;
  const float sa = kDown ? row_s[min(m, 15)] : d.a_scale[min(m, M - 1)];

  constexpr int kStride = Lds::kRegion / 4;    // words from one wave's tiles to the next's
  const int rd = col * kUnit, sw = few_swz(col);
  int slot = 0, buf = 0;
  for (int base = 0; base < steps; base += gridDim.x, buf ^= 1) {
    const int step = step_of(base);
    if (step >= steps) break;                  // (the same for the workgroup)
    i32x4 acc = {0, 0, 0, 0};
    for (int ch = 0; ch < nch; ++ch) {
      if constexpr (kParts) {                  // the activations of this part (from the cache)
        units_of(ch, g0, ng);
        if constexpr (kDown) {
          if (ng > 0) fetch(av4[0], g0);
          convert_all(g0, ng);
        } else {
          load_a(g0, ng);
        }
      }
#pragma unroll
      for (int u = 0; u < GW; ++u) {
        if (u < ng) {
          // the unit has landed when only the loads of the kFewSlots - 1 after it are in flight
          if (ls < steps) __builtin_amdgcn_s_waitcnt(0x0F70 | (2 * (kFewSlots - 1)));
          else __builtin_amdgcn_s_waitcnt(0x0F70);
          asm volatile("" ::: "memory");
          const uint8_t* at = ring + slot * kUnitBytes + rd;
          const i32x4 w0 = lds_load<i32x4>(at + 16 * (q ^ sw)), w1 = lds_load<i32x4>(at + 16 * ((4 + q) ^ sw));
          acc = mfma_i8_16x16x64(av[u][0], w0, acc);
          acc = mfma_i8_16x16x64(av[u][1], w1, acc);
          __builtin_amdgcn_s_waitcnt(0xC07F);  // (the slot is read)
          slot = slot + 1 == kFewSlots ? 0 : slot + 1;
          if (ls < steps) load();
        }
      }
    }
    int* part = reinterpret_cast<int*>(regions) + buf * 256;
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave * kStride + (4 * q + r) * 16 + col] = acc[r];
    __builtin_amdgcn_s_waitcnt(0xC07F);
    barrier_loads_in_flight();                 // one per step: the other buffer's readers passed the last one
    const int64_t n0 = (int64_t)step * kRows, n = n0 + c;
    if (m < M && n < outs) {
      const int* at = part + m * 16 + c;
      if constexpr (kGated) {
        int g = 0, u = 0;
#pragma unroll
        for (int w = 0; w < kFewRowsWaves; ++w) {
          g += at[w * kStride];
          u += at[w * kStride + 8];
        }
        const float v = silu_mul((float)g * sa * d.w_scale[n], (float)u * sa * d.w_scale[f.I + n]);
        f.act[(int64_t)m * f.I + n] = v;
        uint32_t top = magnitude(v);
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
        if (c == 0) f.pmax[(int64_t)m * (f.I >> 3) + step] = top;
      } else {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kFewRowsWaves; ++w) sum += at[w * kStride];
        const bool whole = n0 + 16 <= d.N;     // (the same for the workgroup)
        float v = (float)sum * sa * (whole ? pick16(d.w_scale + n0, c) : d.w_scale[n]);
        if (d.bias) v += whole ? pick16(d.bias + n0, c) : d.bias[n];
        const int64_t o = (int64_t)m * d.N + n;
        if (d.y_bf16) {
          if (d.add) v += __uint_as_float((uint32_t)static_cast<const uint16_t*>(d.add)[o] << 16);
          static_cast<uint16_t*>(d.y)[o] = __builtin_bit_cast(uint16_t, (__bf16)v);
        } else {
          if (d.add) v += static_cast<const float*>(d.add)[o];
          static_cast<float*>(d.y)[o] = v;
        }
      }
    }
  }
}

template <int kForm, int GW, bool kParts>
hipError_t launch_few_steps(const FewRowsArgs& f, hipStream_t stream) {
  const int64_t outs = kForm == kFewGated ? f.I : f.d.N, rows = kForm == kFewGated ? 8 : 16;
  const int64_t steps = (outs + rows - 1) / rows;
  auto kernel = dense_few_kernel<kForm, GW, kParts>;
  // One workgroup on a CU at most, each the same number of steps: a second one would fetch the
  // activations again (16 x 6144 x 6144 10.5 against 12.6 us with two, 9000 x 5120 11.0 against
  // 12.6; 6144 x 2048 5.2 against 4.9).  Rings of 5, 6 or 8 units changed nothing.
  const int64_t rounds = (steps + 255) / 256;
  hipLaunchKernelGGL(kernel, dim3((unsigned)((steps + rounds - 1) / rounds)), dim3(kFewRowsThreads), 0, stream, f);
  return hipGetLastError();
}

template <int kForm>
hipError_t launch_few_rows(const FewRowsArgs& f, hipStream_t stream) {
  const int64_t each = ((f.d.K + kUnit - 1) / kUnit + kFewRowsWaves - 1) / kFewRowsWaves;   // units per wave
  if (each <= 2) return launch_few_steps<kForm, 2, false>(f, stream);
  if (each <= 4) return launch_few_steps<kForm, 4, false>(f, stream);
  if (each <= 6) return launch_few_steps<kForm, 6, false>(f, stream);
  if (each <= 8) return launch_few_steps<kForm, 8, false>(f, stream);
  if (each <= 12) return launch_few_steps<kForm, 12, false>(f, stream);
  if (each <= 16) return launch_few_steps<kForm, 16, false>(f, stream);
  return launch_few_steps<kForm, 8, true>(f, stream);
}

}  // namespace

bool dense_few_fits(int64_t M, int64_t ld_a) { return M <= 16 && M * ld_a < ((int64_t)1 << 31); }

hipError_t launch_dense_few(const DenseArgs& d, hipStream_t stream) {
  return launch_few_rows<kFewDense>(FewRowsArgs{d, 0, nullptr, nullptr}, stream);
}

hipError_t launch_gated_few(const DenseArgs& d, int64_t I, float* act, uint32_t* pmax, hipStream_t stream) {
  return launch_few_rows<kFewGated>(FewRowsArgs{d, I, act, pmax}, stream);
}

hipError_t launch_down_few(const DenseArgs& d, float* act, uint32_t* pmax, hipStream_t stream) {
  return launch_few_rows<kFewDown>(FewRowsArgs{d, d.K, act, pmax}, stream);
}

}  // namespace w4a8
