// Matrix-vector products with 4-bit weights: y[t, n] = sum_k x[t, k] w[n, k] for
// 1 to 16 bf16 activation rows, the activations as they are (no quantization).
//
// Bound by reading the weights once.  A step is 16 NS weight rows (output columns);
// the 8 waves of a workgroup split its K: wave v takes up to GW K groups of every
// subtile, so a projection of a few thousand outputs still puts 8 waves on every 16
// rows.  The workgroups walk the steps; a wave holds its part of the activations in
// registers as matrix-core operands (w4_bf16.hpp) for all of them, and refills each
// weight register with the next step's as it is used up, so that a step's loads are
// in flight while the one before is multiplied and summed.  The eight partial 16x16
// tiles meet in LDS and are summed in wave order (fp32; the same bits at every run).
// Rows of A past T repeat row T - 1; their products are never stored.
//
// Measured (group 128, GEMM storage; kernel times): 1 x 131072 x 6144 67 us (428 MB, 6.4
// TB/s), 16 x 65536 x 6144 40.5 us (5.3 TB/s), 16 x 12288 x 6144 13.8 us (41 MB, 3.0 TB/s; 13.4
// with the weights of three matrices in turn, which the 256 MB last-level cache holds),
// 1 x 4096 x 6144 8.3 us (7.3 from the cache), 1 x 2048 x 2048 4.1 us (from the cache): up to
// some 20 MB the start bounds it (the launch, one trip to memory for the weights, which the
// turn of x waits for as they are issued first, the exchange in LDS).  A call from the host
// takes about 7 us, so the smallest are bound by that.
#include "kernels.hpp"
#include "w4_bf16.hpp"

namespace w4a8 {

constexpr int kMvWaves = 8;
constexpr int kMvThreads = 64 * kMvWaves;
constexpr int kMvPitch = 272;                // bytes of a row of activations on its way to operand order

// kParts: K is longer than the 8 GW groups held at once; a step then goes over parts of
// K and fetches each part's activations again (a path of its own: their loads would
// otherwise be waited for in every step).
template <int kForm, bool kRM, int GW, int NS, bool kParts>
__global__ __launch_bounds__(kMvThreads) void matvec_kernel(const uint16_t* __restrict__ x, int T, int64_t K,
                                                            int64_t ld, const uint8_t* __restrict__ w,
                                                            const uint8_t* __restrict__ s, int64_t N,
                                                            void* __restrict__ y, int y_bf16) {
  constexpr bool kMx = kForm == kFormMx;
  __shared__ float red[2][kMvWaves][NS][16][16];
  // The wave's activations of one group on their way to operand order, T rows of 256 bytes.  A row is 16 bytes
  // longer so that the 16 rows an operand read covers start in different banks.
  constexpr int kPitch = kMvPitch;
  extern __shared__ __attribute__((aligned(16))) unsigned char a_sm[];   // [waves][T][kPitch]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int G = (int)((K + kGroup - 1) / kGroup);
  const uint32_t row_bytes = (uint32_t)(K >> 1);
  const int steps = (int)((N + 16 * NS - 1) / (16 * NS));
  const int nch = kParts ? (G + kMvWaves * GW - 1) / (kMvWaves * GW) : 1;   // parts of K

  // the wave's groups of a part of K: g0 .. g0 + ng - 1
  auto groups_of = [&](int ch, int& g0, int& ng) {
    const int all = min(kMvWaves * GW, G - ch * kMvWaves * GW);
    const int gpw = (all + kMvWaves - 1) / kMvWaves;
    g0 = ch * kMvWaves * GW + wave * gpw;
    ng = max(0, min(gpw, all - wave * gpw));
  };
  auto inside = [&](int g) { return g * kGroup + 32 * kq < K; };   // of stored MXFP4 rows, a last group that is not whole

  // Scales: a word per lane for four groups (spread4), or for the bytes of stored MXFP4
  // rows, which need not be aligned to words, one per group.
  constexpr bool kBytes = kMx && kRM;
  constexpr int SP = kBytes ? 1 : 4, SW = (GW + SP - 1) / SP;  // groups per scale word
  i32x4 av[GW][4], wv[GW][NS];
  uint32_t sv[SW][NS];
  v4f bias[GW];
  // A row's 256 bytes of a group are read by 16 lanes side by side (an operand's lanes read 16 rows 16 bytes at a
  // time: 64 cache lines an instruction, four times over), then change places through LDS.
  unsigned char* a_mine = a_sm + (size_t)wave * T * kPitch;
  auto load_a = [&](int g0, int ng) {
#pragma unroll
    for (int i = 0; i < GW; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {                            // rows 4 j + lane / 16
        if (4 * j < T) {
          const int k = (g0 + i) * kGroup + 8 * col;
          av[i][j] = i < ng && k < K ? *reinterpret_cast<const i32x4*>(x + (int64_t)min(4 * j + kq, T - 1) * ld + k)
                                     : i32x4{0, 0, 0, 0};
        }
      }
    }
  };
  auto turn_a = [&](int ng) {
    const int row = min(col, T - 1);
#pragma unroll
    for (int i = 0; i < GW; ++i) {
      if (i < ng) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * j + kq < T) *reinterpret_cast<i32x4*>(a_mine + (4 * j + kq) * kPitch + 16 * col) = av[i][j];
        wave_lds_fence();
#pragma unroll
        for (int c = 0; c < 4; ++c) av[i][c] = *reinterpret_cast<const i32x4*>(a_mine + row * kPitch + 64 * kq + 16 * c);
        wave_lds_fence();
      }
    }
  };
  __amdgpu_buffer_rsrc_t rw = buffer_of(w, 0), rs = buffer_of(s, 0);
  int lg0 = 0, lng = 0;                                        // the groups being loaded
  auto point = [&](int step, int ch) {                         // the weights of (step, part); none past the last step
    groups_of(ch, lg0, lng);
    const int64_t n0 = (int64_t)step * (16 * NS);
    const int64_t rows = step < steps ? (N - n0 < 16 * NS ? N - n0 : 16 * NS) : 0;
    rw = buffer_of(w + n0 * row_bytes, rows * row_bytes);
    if constexpr (kForm == kFormG128) {
      if constexpr (kRM) rs = buffer_of(s + n0 * G * 4, rows * G * 4);
      else rs = buffer_of(s + ((int64_t)lg0 * N + n0) * 4, rows ? ((int64_t)(G - lg0) * N - n0) * 4 : 0);
    } else if constexpr (kMx) {
      if constexpr (kRM) rs = buffer_of(s + n0 * (K >> 5), rows * (K >> 5));
      else rs = buffer_of(s + ((int64_t)lg0 * N + n0) * 4, rows ? ((int64_t)(G - lg0) * N - n0) * 4 : 0);
    }
  };
  auto load_w = [&](int i) {
    const bool on = i < lng;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const uint32_t g = (uint32_t)(lg0 + i);
      const uint32_t wo = kRM ? (16 * j + col) * row_bytes + 64 * g + 16 * kq
                              : 16 * j * row_bytes + 1024 * g + 64 * col + 16 * kq;
      wv[i][j] = buffer_load16_nt(rw, on ? wo : kNowhere);
    }
  };
  auto load_s = [&](int m) {                                   // scale word m, before its groups' weights
    if constexpr (kForm != kFormChannel) {
      const int i = SP * m + (kBytes ? 0 : kq);                // the lane's group
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const uint32_t so = kBytes ? (16 * j + col) * (uint32_t)(K >> 5) + 4 * (lg0 + i) + kq
                            : kRM  ? ((16 * j + col) * G + lg0 + i) * 4
                                   : (uint32_t)(i * N + 16 * j + col) * 4;
        if constexpr (kBytes) sv[m][j] = buffer_load1(rs, i < lng ? so : kNowhere);
        else sv[m][j] = buffer_load4(rs, i < lng ? so : kNowhere);
      }
    }
  };

  int step = xcd_order(), buf = 0, g0, ng;
  point(step, 0);
#pragma unroll
  for (int i = 0; i < GW; ++i) {
    if (i % SP == 0) load_s(i / SP);
    load_w(i);
  }
  groups_of(0, g0, ng);
  load_a(g0, ng);
  turn_a(ng);
  auto all_bias = [&]() {
    if constexpr (!kMx) {
#pragma unroll
      for (int i = 0; i < GW; ++i)
        if (i < ng) bias[i] = minus8_product(av[i]);
    }
  };
  all_bias();
  for (; step < steps; step += gridDim.x, buf ^= 1) {
    v4f acc[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int ch = 0; ch < nch; ++ch) {
      if constexpr (kParts) {                                  // the activations of this part (from the cache)
        groups_of(ch, g0, ng);
        load_a(g0, ng);
        turn_a(ng);
        all_bias();
      }
      const bool last = ch + 1 == nch;
      point(last ? step + (int)gridDim.x : step, last ? 0 : ch + 1);
      uint32_t s4[NS][4];
#pragma unroll
      for (int i = 0; i < GW; ++i) {
        if (i % SP == 0) {
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            if constexpr (kBytes) s4[j][0] = sv[i][j];
            else if constexpr (kForm != kFormChannel) spread4(sv[i / SP][j], s4[j]);
          }
          load_s(i / SP);
        }
        if (i < ng) {
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            uint32_t f = 0;
            if constexpr (kForm == kFormG128) f = s4[j][i & 3];
            else if constexpr (kMx) f = kRM ? (inside(g0 + i) ? s4[j][0] : 127u) : (s4[j][i & 3] >> (8 * kq)) & 0xffu;
            group_product<kForm, kRM>(av[i], wv[i][j], f, kMx ? v4f{0.f, 0.f, 0.f, 0.f} : bias[i], acc[j]);
          }
        }
        load_w(i);
      }
    }
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[buf][wave][j][4 * kq + r][col] = acc[j][r];
    __syncthreads();                                           // one per step: the other buffer's readers passed the last one
    const int v = threadIdx.x;
    if (v < T * 16 * NS) {
      const int c = v & 15, j = (v >> 4) % NS, t = (v >> 4) / NS;
      const int64_t n = (int64_t)step * (16 * NS) + 16 * j + c;
      if (n < N) {
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < kMvWaves; ++u) sum += red[buf][u][j][t][c];
        if constexpr (kForm == kFormChannel) sum *= reinterpret_cast<const float*>(s)[n];
        if (y_bf16) static_cast<uint16_t*>(y)[(int64_t)t * N + n] = __builtin_bit_cast(uint16_t, (__bf16)sum);
        else static_cast<float*>(y)[(int64_t)t * N + n] = sum;
      }
    }
  }
}

// One workgroup on each CU: 256 against 512 at 16 x 12288 x 6144 13.7 against 20.1 us, 1 x
// 131072 x 6144 67.5 against 69.9; the same where K is 2048.
constexpr int64_t kMvGrid = 256;

template <int kForm, bool kRM, int GW, bool kParts = false>
static void launch_matvec_steps(const MatvecArgs& a, hipStream_t stream) {
  auto go = [&](auto kernel, int ns) {
    const int64_t steps = (a.N + 16 * ns - 1) / (16 * ns);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(steps < kMvGrid ? steps : kMvGrid)), dim3(kMvThreads),
                       (size_t)(kMvWaves * a.T * kMvPitch), stream, a.x, (int)a.T, a.K, a.ld,
                       static_cast<const uint8_t*>(a.w), static_cast<const uint8_t*>(a.s), a.N, a.y, a.y_bf16);
  };
  // Steps of 32 outputs (whole lines of scales, half the exchanges) from two steps of them per workgroup on: K
  // 4096, N 32768 15.1 against 16.3 us, N 4096 7.0 against 6.3.  With K in parts from one on, as each step fetches
  // the activations again: 8192 x 16384 21.6 against 26.7 us (group 128).
  if (a.N >= (kParts ? 32 : 64) * kMvGrid) go(matvec_kernel<kForm, kRM, GW, 2, kParts>, 2);
  else go(matvec_kernel<kForm, kRM, GW, 1, kParts>, 1);
}

// K above 6144 goes in parts, at a cost: a part's activations are fetched behind its weights, and waiting for them
// drains the prefetch; the MXFP4 form also spills registers (10 to 12 of 256 in steps of 16 outputs, 103 to 125 in
// steps of 32).  1 / 16 rows of 8192 x 8192: group 128 14.9 / 18.7 us, per channel 14.9 / 17.5, MXFP4 30.4 / 42.9; of
// 6144 x 12288: 19.7 / 27.6, 19.6 / 27.1 and 28.2 / 45.1, against 13.8 for 16 rows of 12288 x 6144.
template <int kForm, bool kRM>
static void launch_matvec_form(const MatvecArgs& a, hipStream_t stream) {
  const int64_t gpw = ((a.K + kGroup - 1) / kGroup + kMvWaves - 1) / kMvWaves;   // K groups per wave
  if (gpw <= 2) launch_matvec_steps<kForm, kRM, 2>(a, stream);
  else if (gpw <= 4) launch_matvec_steps<kForm, kRM, 4>(a, stream);
  else if (gpw <= 6) launch_matvec_steps<kForm, kRM, 6>(a, stream);
  else launch_matvec_steps<kForm, kRM, 6, true>(a, stream);
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
