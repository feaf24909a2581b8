// Norms before and after a block (w4a8_block.h): RMS norm of a row with its 8-bit codes; and
// the residual sum of a block's result, normed and gated, followed by the next block's norm.
//
// A row is read once and held in registers by a group of threads (a wave for up to 2048
// values, 256 threads up to 16384, 1024 up to 32768), 8 values to a chunk of 16 or 32 bytes:
//   before: n = weight x rsqrt(mean x^2 + eps); max |n|; codes.
//   after:  p = post y rsqrt(mean y^2 + eps); out = r_scale r + token_gate gate p; then the
//           same of out.
// Each mean, and the maximum, is one reduction over the group.  Sums are fp32; a row whose
// sum of squares is not below infinity is summed again times 2^-80, where 32768 squares of
// the largest fp32 values stay finite (eps no longer matters then).
#include "block.hpp"
#include "row_codes.hpp"

namespace w4a8 {

// all values of a group of kThr threads; a buffer serves one reduction
template <int kThr, typename F>
__device__ __forceinline__ float group_reduce(float v, float* red, F wave, float (*join)(float, float)) {
  v = wave(v);
  if constexpr (kThr > kWave) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < kThr / kWave; ++w) v = join(v, red[w]);
  }
  return v;
}
__device__ __forceinline__ float join_sum(float a, float b) { return a + b; }
__device__ __forceinline__ float join_max(float a, float b) { return fmaxf(a, b); }
template <int kThr>
__device__ __forceinline__ float group_sum(float v, float* red) {
  return group_reduce<kThr>(v, red, [](float x) { return wave_sum(x); }, join_sum);
}
template <int kThr>
__device__ __forceinline__ float group_max(float v, float* red) {
  return group_reduce<kThr>(v, red, [](float x) { return wave_max(x); }, join_max);
}

// 8 values of a row as they lie in memory, and as fp32
struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ Raw load_raw(const void* row, int bf16, int chunk) {
  Raw v;
  if (bf16) {
    v.a = static_cast<const uint4*>(row)[chunk];
    v.b = make_uint4(0u, 0u, 0u, 0u);
  } else {
    v.a = static_cast<const uint4*>(row)[2 * chunk];
    v.b = static_cast<const uint4*>(row)[2 * chunk + 1];
  }
  return v;
}
__device__ __forceinline__ void widen(const Raw& v, int bf16, float (&f)[8]) {
  const uint32_t a[4] = {v.a.x, v.a.y, v.a.z, v.a.w}, b[4] = {v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      f[2 * i] = bf16_lo(a[i]);
      f[2 * i + 1] = bf16_hi(a[i]);
    } else {
      f[i] = __uint_as_float(a[i]);
      f[4 + i] = __uint_as_float(b[i]);
    }
  }
}
__device__ __forceinline__ void load_vector(const float* v, int chunk, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(v)[2 * chunk], b = reinterpret_cast<const float4*>(v)[2 * chunk + 1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ uint4 bf16x8(const float (&f)[8]) {
  return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

// the values of a row times 1 / sqrt(mean square + eps) and times `weight`; false where the
// row holds a NaN or an infinity
template <int kThr, int kPer>
__device__ __forceinline__ bool normalize(float (&v)[kPer][8], int chunks, int tid, float H, float eps,
                                          const float* weight, float* red, float* red2) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  ss = group_sum<kThr>(ss, red);
  float f;
  if (ss < INFINITY) {
    f = __builtin_amdgcn_rsqf(ss / H + eps);
  } else {                                                  // (the same for the whole group)
    constexpr float kDown = 0x1p-80f;
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] *= kDown;
        ss = fmaf(v[i][j], v[i][j], ss);
      }
    ss = group_sum<kThr>(ss, red2);
    f = __builtin_amdgcn_rsqf(ss / H);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = tid + kThr * i;
    if (c < chunks) {
      float w[8];
      load_vector(weight, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * f * w[j];
    }
  }
  return ss < INFINITY;
}

// kRes: with r (the residual form).  A block holds one group, or four of a wave.
template <int kThr, int kPer, bool kRes, int kCodes>
__global__ __launch_bounds__(kThr < 256 ? 256 : kThr) void norm_kernel(const NormArgs n) {
  __shared__ float red[5][16];
  constexpr int kGroups = kThr < 256 ? 256 / kThr : 1;
  const int tid = kGroups > 1 ? threadIdx.x % kThr : threadIdx.x;
  const int64_t t = (int64_t)blockIdx.x * kGroups + (kGroups > 1 ? threadIdx.x / kThr : 0);
  if (kGroups > 1 && t >= n.T) return;                      // (groups of a wave meet no barrier)
  const int chunks = (int)(n.H >> 3);
  const float H = (float)n.H;
  const char* xr = static_cast<const char*>(n.x) + t * n.ld_x * (n.x_bf16 ? 2 : 4);
  float v[kPer][8];
  Raw raw[kPer], raw_r[kRes ? kPer : 1];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = tid + kThr * i;
    raw[i] = c < chunks ? load_raw(xr, n.x_bf16, c) : Raw{};
  }
  if constexpr (kRes) {
    const char* rr = static_cast<const char*>(n.r) + t * n.ld_r * (n.r_bf16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = tid + kThr * i;
      raw_r[i] = c < chunks ? load_raw(rr, n.r_bf16, c) : Raw{};
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) widen(raw[i], n.x_bf16, v[i]);
  bool fine = true;
  if constexpr (kRes) {
    if (n.post) fine = normalize<kThr, kPer>(v, chunks, tid, H, n.eps, n.post, red[0], red[1]);
    const float tg = n.token_gate ? n.token_gate[t] : 1.0f;
    char* outr = static_cast<char*>(n.out) + t * n.ld_out * (n.r_bf16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = tid + kThr * i;
      if (c < chunks) {
        float r[8], g[8];
        widen(raw_r[i], n.r_bf16, r);
        if (n.gate) load_vector(n.gate, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float p = v[i][j];
          if (n.gate) p *= g[j];
          if (n.token_gate) p *= tg;
          v[i][j] = fmaf(n.r_scale, r[j], p);
        }
        if (n.r_bf16) {
          reinterpret_cast<uint4*>(outr)[c] = bf16x8(v[i]);
        } else {
          reinterpret_cast<float4*>(outr)[2 * c] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
          reinterpret_cast<float4*>(outr)[2 * c + 1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
        }
      }
    }
    if (!n.weight) return;
  }
  fine &= normalize<kThr, kPer>(v, chunks, tid, H, n.eps, n.weight, red[2], red[3]);
  if (n.xn) {
    uint4* xnr = reinterpret_cast<uint4*>(n.xn + t * n.H);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (tid + kThr * i < chunks) xnr[tid + kThr * i] = bf16x8(v[i]);
  }
  if constexpr (kCodes != kCodesNone) {
    constexpr bool kInt8 = kCodes == kCodesI8;
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));    // (0 past the row)
    m = group_max<kThr>(m, red[4]);
    const float scale = row_scale<kInt8>(m);
    const RowDivisor d = row_divisor(scale);
    uint2* qr = reinterpret_cast<uint2*>(n.q + t * n.H);
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = tid + kThr * i;
      if (c < chunks) {
        if (d.by != 1.0f) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] *= d.by;
        }
        const uint2 q = make_uint2(codes4<kInt8>(v[i][0], v[i][1], v[i][2], v[i][3], d.s, d.r),
                                   codes4<kInt8>(v[i][4], v[i][5], v[i][6], v[i][7], d.s, d.r));
        if constexpr (kInt8) sum = __builtin_amdgcn_sdot4(q.x, 0x01010101, __builtin_amdgcn_sdot4(q.y, 0x01010101, sum, false), false);
        qr[c] = q;
      }
    }
    if (tid == 0) n.s[t] = fine ? scale : __uint_as_float(0x7fc00000u);
    if constexpr (kInt8) {
      if (n.rowsum) {                                        // (the same for the whole launch)
        sum = wave_sum_int(sum);
        if constexpr (kThr > kWave) {
          int* reds = reinterpret_cast<int*>(red[0]);       // its readers are past later barriers
          if ((threadIdx.x & 63) == 0) reds[threadIdx.x >> 6] = sum;
          __syncthreads();
          sum = 0;
#pragma unroll
          for (int w = 0; w < kThr / kWave; ++w) sum += reds[w];
        }
        if (tid == 0) n.rowsum[t] = sum;
      }
    }
  }
}

template <int kThr, int kPer>
static void launch_norm_form(const NormArgs& n, hipStream_t stream) {
  constexpr int kGroups = kThr < 256 ? 256 / kThr : 1;
  const dim3 grid((unsigned)((n.T + kGroups - 1) / kGroups)), block(kThr * kGroups);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, n); };
  if (n.r) {
    if (n.codes == kCodesFp8) go(norm_kernel<kThr, kPer, true, kCodesFp8>);
    else if (n.codes == kCodesI8) go(norm_kernel<kThr, kPer, true, kCodesI8>);
    else go(norm_kernel<kThr, kPer, true, kCodesNone>);
  } else {
    if (n.codes == kCodesFp8) go(norm_kernel<kThr, kPer, false, kCodesFp8>);
    else if (n.codes == kCodesI8) go(norm_kernel<kThr, kPer, false, kCodesI8>);
    else go(norm_kernel<kThr, kPer, false, kCodesNone>);
  }
}

hipError_t launch_norm(const NormArgs& n, hipStream_t stream) {
  if (n.T == 0) return hipSuccess;
  if (n.H <= 512) launch_norm_form<64, 1>(n, stream);
  else if (n.H <= 1024) launch_norm_form<64, 2>(n, stream);
  else if (n.H <= 2048) launch_norm_form<64, 4>(n, stream);
  else if (n.H <= 4096) launch_norm_form<256, 2>(n, stream);
  else if (n.H <= 6144) launch_norm_form<256, 3>(n, stream);
  else if (n.H <= 8192) launch_norm_form<256, 4>(n, stream);
  else if (n.H <= 16384) launch_norm_form<256, 8>(n, stream);
  else launch_norm_form<1024, 4>(n, stream);
  return hipGetLastError();
}

}  // namespace w4a8
