// Matrix-vector products with 4-bit weights: y[t, n] = sum_k x[t, k] w[n, k] for
// 1 to 16 bf16 activation rows, the activations as they are (no quantization).
//
// Bound by reading the weights once.  A workgroup owns 16 NS weight rows (output
// columns) and its 8 waves split K: wave v takes the K groups v gpw .. +gpw of
// every subtile, so a projection of a few thousand outputs still puts 8 loads
// in flight for every 16 rows.  Each wave multiplies on the bf16 matrix cores
// (w4_bf16.hpp); the eight partial 16x16 tiles meet in LDS and are summed in wave
// order (fp32; the same bits at every run).
// The activation rows come from the cache for each group: 64 bytes per lane, rows
// past T repeating row T - 1 (their products are never stored).
#include "kernels.hpp"
#include "w4_bf16.hpp"

namespace w4a8 {

constexpr int kMvWaves = 8;
constexpr int kMvThreads = 64 * kMvWaves;

template <int kForm, bool kRM, int NS>
__global__ __launch_bounds__(kMvThreads) void matvec_kernel(const uint16_t* __restrict__ x, int T, int64_t K,
                                                            int64_t ld, const uint8_t* __restrict__ w,
                                                            const uint32_t* __restrict__ s, int64_t N,
                                                            void* __restrict__ y, int y_bf16) {
  constexpr int kBatch = 4;                    // groups loaded together
  __shared__ float red[kMvWaves][NS][16][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NS);
  const int G = (int)((K + kGroup - 1) / kGroup);
  const int gpw = (G + kMvWaves - 1) / kMvWaves;
  const int g_begin = wave * gpw, g_end = min(G, g_begin + gpw);

  // the lane's weight bytes of subtile s and group g: pw[s] + g kGStride
  constexpr int kGStride = kRM ? 64 : 1024;
  const uint8_t* pw[NS];
  int64_t nrow[NS];                            // the lane's weight row (clamped: a row past N is not stored)
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int64_t n = n0 + 16 * i + col;
    nrow[i] = n < N ? n : N - 1;
    if constexpr (kRM) pw[i] = w + nrow[i] * (K >> 1) + kq * 16;
    else pw[i] = w + ((nrow[i] - (nrow[i] & 15)) * (K >> 1)) + (nrow[i] & 15) * 64 + kq * 16;
  }
  const uint16_t* xr = x + (int64_t)min(col, T - 1) * ld + 32 * kq;

  v4f acc[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int g0 = g_begin; g0 < g_end; g0 += kBatch) {
    i32x4 wv[kBatch][NS], av[kBatch][4];
    uint32_t sv[kBatch][NS];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int g = g0 + b;
      // a lane past K (a last group that is not whole) multiplies zeros
      const bool in = g < g_end && (int64_t)g * kGroup + 32 * kq < K;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        wv[b][i] = in ? __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pw[i] + (int64_t)g * kGStride))
                      : i32x4{0, 0, 0, 0};
        if constexpr (kForm == kFormG128)
          sv[b][i] = in ? s[kRM ? nrow[i] * G + g : (int64_t)g * N + nrow[i]] : 0u;
        else if constexpr (kForm == kFormMx)
          sv[b][i] = in ? reinterpret_cast<const uint8_t*>(s)[kRM ? nrow[i] * (K >> 5) + 4 * g + kq
                                                                  : ((int64_t)g * N + nrow[i]) * 4 + kq]
                        : 127u;
        else sv[b][i] = 0u;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        av[b][c] = in ? *reinterpret_cast<const i32x4*>(xr + (int64_t)g * kGroup + 8 * c) : i32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const v4f bias = kForm == kFormMx ? v4f{0.f, 0.f, 0.f, 0.f} : minus8_product(av[b]);
#pragma unroll
      for (int i = 0; i < NS; ++i) group_product<kForm, kRM>(av[b], wv[b][i], sv[b][i], bias, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][i][4 * kq + r][col] = acc[i][r];
  __syncthreads();
  for (int v = threadIdx.x; v < T * 16 * NS; v += kMvThreads) {
    const int c = v & 15, i = (v >> 4) % NS, t = (v >> 4) / NS;
    const int64_t n = n0 + 16 * i + c;
    if (n >= N) continue;
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kMvWaves; ++u) sum += red[u][i][t][c];
    if constexpr (kForm == kFormChannel) sum *= __uint_as_float(s[n]);
    if (y_bf16) static_cast<uint16_t*>(y)[(int64_t)t * N + n] = __builtin_bit_cast(uint16_t, (__bf16)sum);
    else static_cast<float*>(y)[(int64_t)t * N + n] = sum;
  }
}

template <int kForm, bool kRM>
static void launch_matvec_form(const MatvecArgs& a, hipStream_t stream) {
  constexpr int NS = 1;
  hipLaunchKernelGGL((matvec_kernel<kForm, kRM, NS>), dim3((unsigned)((a.N + 16 * NS - 1) / (16 * NS))),
                     dim3(kMvThreads), 0, stream, a.x, (int)a.T, a.K, a.ld, static_cast<const uint8_t*>(a.w),
                     static_cast<const uint32_t*>(a.s), a.N, a.y, a.y_bf16);
}

hipError_t launch_matvec(const MatvecArgs& a, hipStream_t stream) {
  if (a.form == kFormMx) a.row_major ? launch_matvec_form<kFormMx, true>(a, stream)
                                     : launch_matvec_form<kFormMx, false>(a, stream);
  else if (a.form == kFormChannel) a.row_major ? launch_matvec_form<kFormChannel, true>(a, stream)
                                               : launch_matvec_form<kFormChannel, false>(a, stream);
  else a.row_major ? launch_matvec_form<kFormG128, true>(a, stream)
                   : launch_matvec_form<kFormG128, false>(a, stream);
  return hipGetLastError();
}

}  // namespace w4a8
