// Dense products in 8-bit integers and the gated feed-forward block on them (w4a8_block.h).
//
// One workgroup of four waves computes a tile of 128 rows x 128 weight rows (output
// columns), each wave 64 x 64 of it in 16x16x64 INT8 products with int32 sums.  K goes in
// steps of 128 bytes through two LDS slots, filled by loads straight into LDS.
#include "block.hpp"
#include "gemm_common.hpp"
#include "lds_dma.hpp"
#include "row_codes.hpp"

namespace w4a8 {

namespace {

constexpr int kBM = 128, kBN = 128, kBK = 128;

__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// kGated: the tile's columns are 64 gate rows and the 64 up rows of the same act columns, by
// 16 in turn, and the result is act = silu(gate) up, fp32 [M][I]; otherwise y.
template <bool kGated>
__global__ __launch_bounds__(256) void dense_i8_kernel(const DenseArgs d, int64_t I, float* __restrict__ act) {
  __shared__ __attribute__((aligned(16))) uint8_t sm[2][(kBM + kBN) * kBK];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * kBM, n0 = (int64_t)blockIdx.x * kBN;
  const int K = (int)d.K;
  const int rows = (int)min((int64_t)kBM, d.M - m0);
  const int cols = (int)min((int64_t)kBN, d.N - n0);
  const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(d.a + m0 * d.ld_a, (uint32_t)((rows - 1) * d.ld_a + K));
  // weight rows: 64 gate and 64 up rows, or 128 in a row
  const int64_t c0 = kGated ? n0 / 2 : n0;
  const int wrows = kGated ? cols / 2 : cols;
  const __amdgpu_buffer_rsrc_t rg = buffer_rsrc(d.w + c0 * K, (uint32_t)(wrows * K));
  const __amdgpu_buffer_rsrc_t ru = buffer_rsrc(d.w + ((kGated ? I : 0) + c0) * K, (uint32_t)(wrows * K));

  const int steps = (K + kBK - 1) / kBK;
  // an instruction loads 8 rows of 128 bytes; wave w loads the rows 32 w .. +31 of each side.  A row or chunk
  // past the operand is never read (its offset is past the resource) and never matters: rows past the end give
  // outputs that are not stored, bytes past K are taken out of a below.
  auto stage = [&](int s, int kt) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 32 * wave + 8 * q + (lane >> 3);
      const int c = (lane & 7) ^ swz(r);
      dma16(ra, (uint32_t)(r * (int)d.ld_a + 16 * c), (uint32_t)(kt * kBK), &sm[s][(32 * wave + 8 * q) * kBK]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 32 * wave + 8 * q + (lane >> 3);
      const int c = (lane & 7) ^ swz(r);
      const int wr = kGated ? 16 * (r >> 5) + (r & 15) : r;
      if (kGated && ((2 * wave + (q >> 1)) & 1))
        dma16(ru, (uint32_t)(wr * K + 16 * c), (uint32_t)(kt * kBK), &sm[s][(kBM + 32 * wave + 8 * q) * kBK]);
      else
        dma16(rg, (uint32_t)(wr * K + 16 * c), (uint32_t)(kt * kBK), &sm[s][(kBM + 32 * wave + 8 * q) * kBK]);
    }
  };
  const int wm = 64 * (wave >> 1), wn = 64 * (wave & 1);
  i32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  stage(0, 0);
  for (int kt = 0; kt < steps; ++kt) {
    const int s = kt & 1;
    __builtin_amdgcn_s_waitcnt(0x0F70);                      // vmcnt(0): this step's loads
    barrier_loads_in_flight();
    if (kt + 1 < steps) stage(s ^ 1, kt + 1);                // (its readers passed the barrier)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 a[4], b[4];
      const uint32_t off = 16u * (uint32_t)((4 * h + lq) ^ swz(lr));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = lds_load<i32x4>(&sm[s][(wm + 16 * i + lr) * kBK + off]);
        b[i] = lds_load<i32x4>(&sm[s][(kBM + wn + 16 * i + lr) * kBK + off]);
      }
      if (kt * kBK + 64 * h + 16 * lq >= K) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma_i8_16x16x64(a[i], b[j], acc[i][j]);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);                      // lgkmcnt(0)
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t m = m0 + wm + 16 * i + 4 * lq + v;
      if (m >= d.M) continue;
      const float sa = d.a_scale[m];
      if constexpr (kGated) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int64_t n = c0 + wn / 2 + 16 * j + lr;
          if (n < I) {
            const float g = (float)acc[i][2 * j][v] * sa * d.w_scale[n];
            const float u = (float)acc[i][2 * j + 1][v] * sa * d.w_scale[I + n];
            act[m * I + n] = silu_mul(g, u);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t n = n0 + wn + 16 * j + lr;
          if (n >= d.N) continue;
          float y = (float)acc[i][j][v] * sa * d.w_scale[n];
          if (d.bias) y += d.bias[n];
          const int64_t o = m * d.N + n;
          if (d.y_bf16) {
            if (d.add) y += __uint_as_float((uint32_t)static_cast<const uint16_t*>(d.add)[o] << 16);
            static_cast<uint16_t*>(d.y)[o] = __builtin_bit_cast(uint16_t, (__bf16)y);
          } else {
            if (d.add) y += static_cast<const float*>(d.add)[o];
            static_cast<float*>(d.y)[o] = y;
          }
        }
      }
    }
  }
}

// |v| as an integer of its order, a NaN above infinity: a row with one gets a scale of NaN
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t wave_max_uint(uint32_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, kWave));
  return v;
}

// codes of act rows, one workgroup a row
__global__ __launch_bounds__(256) void act_quant_kernel(const float* __restrict__ act, int64_t I,
                                                        uint8_t* __restrict__ q, float* __restrict__ s) {
  __shared__ uint32_t red[4];
  const float4* ar = reinterpret_cast<const float4*>(act + blockIdx.x * I);
  uint32_t m = 0;
  for (int c = threadIdx.x; c < (int)(I >> 2); c += 256) {
    const float4 v = ar[c];
    m = max(max(m, magnitude(v.x)), max(max(magnitude(v.y), magnitude(v.z)), magnitude(v.w)));
  }
  m = wave_max_uint(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(red[0], red[1]), max(red[2], red[3]));
  const float scale = m == 0 ? 1.0f : __uint_as_float(m) / 127.0f;
  const RowDivisor d = row_divisor(scale);
  uint32_t* qr = reinterpret_cast<uint32_t*>(q + blockIdx.x * I);
  for (int c = threadIdx.x; c < (int)(I >> 2); c += 256) {
    const float4 v = ar[c];
    qr[c] = codes4<true>(v.x * d.by, v.y * d.by, v.z * d.by, v.w * d.by, d.s, d.r);
  }
  if (threadIdx.x == 0) s[blockIdx.x] = scale;
}

}  // namespace

int64_t dense_i8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_dense_i8(const DenseArgs& d, hipStream_t stream) {
  const dim3 grid((unsigned)((d.N + kBN - 1) / kBN), (unsigned)((d.M + kBM - 1) / kBM));
  hipLaunchKernelGGL(dense_i8_kernel<false>, grid, dim3(256), 0, stream, d, (int64_t)0, (float*)nullptr);
  return hipGetLastError();
}

// act fp32 [M][I], codes [M][I], scales [M]
int64_t mlp_i8_workspace_bytes(int64_t M, int64_t, int64_t I) { return M * (5 * I + 4); }

hipError_t launch_mlp_i8(const MlpArgs& p, hipStream_t stream) {
  float* act = static_cast<float*>(p.workspace);
  uint8_t* q = reinterpret_cast<uint8_t*>(act + p.M * p.I);
  float* s = reinterpret_cast<float*>(q + p.M * p.I);
  DenseArgs up{p.a, p.a_scale, p.M, p.H, p.ld_a, p.w13, p.s13, nullptr, 2 * p.I, nullptr, nullptr, 0, nullptr};
  const dim3 grid((unsigned)((2 * p.I + kBN - 1) / kBN), (unsigned)((p.M + kBM - 1) / kBM));
  hipLaunchKernelGGL(dense_i8_kernel<true>, grid, dim3(256), 0, stream, up, p.I, act);
  hipLaunchKernelGGL(act_quant_kernel, dim3((unsigned)p.M), dim3(256), 0, stream, act, p.I, q, s);
  const DenseArgs down{reinterpret_cast<int8_t*>(q), s, p.M, p.I, p.I, p.w2, p.s2, nullptr, p.H, p.add, p.y, p.y_bf16,
                       nullptr};
  return launch_dense_i8(down, stream);
}

}  // namespace w4a8
