// Norms before and after a block (w4a8_block.h): RMS norm of a row with its 8-bit codes; and
// the residual sum of a block's result, normed and gated, followed by the next block's norm.
//
// A row is read once and held in registers by a group of threads (a wave for up to 1024
// values, 128 to 1024 threads beyond), 8 values to a chunk of 16 or 32 bytes:
//   before: n = weight x / sqrt(mean x^2 + eps); max |n|; codes.
//   after:  p = post y / sqrt(mean y^2 + eps); out = r_scale r + token_gate gate p; then the
//           same of out.
// Each mean, and the maximum, is one reduction over the group.  Sums are fp32; a row whose
// mean square and eps are not below infinity is summed again times 2^-80, where 32768 squares of
// the largest fp32 values stay finite (an eps that is lost by that does not matter next to them).
//
// Bound by the bytes of the rows where they are many (16384 rows of 6144 bf16, norm and codes: 503 MB in
// 89 us, 5.7 TB/s, above a copy's 5.15), by a launch, one trip to memory and two reductions where they are
// few (one row 3.6 to 3.9 us; 128 rows between two blocks 5.9 to 6.2 us).
#include "block.hpp"
#include "row_codes.hpp"

namespace w4a8 {

// A value of another lane of the row of 16 (DPP).
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, false));
}
struct Sum {
  static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct Max {
  static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};
// The reduction of kLanes neighbouring lanes, in registers: quads by their permutations, rows of 16 by
// mirrors, rows by swaps (with shuffles through LDS a norm of one row takes 4.8 us, so 3.7).  In every
// step two lanes read each other and add the same two values, so all lanes end with the same bits, which
// row_norm's branch and the codes rely on.  (Rows turned by 4 and 8 in place of the mirrors would add the
// quads in two orders: fp32 sums that differ.)
template <typename Op, int kLanes>
__device__ __forceinline__ float lanes_reduce(float v) {
  if constexpr (kLanes > 1) v = Op::of(v, dpp<0xB1>(v));
  if constexpr (kLanes > 2) v = Op::of(v, dpp<0x4E>(v));
  if constexpr (kLanes > 4) v = Op::of(v, dpp<0x141>(v));
  if constexpr (kLanes > 8) v = Op::of(v, dpp<0x140>(v));
  if constexpr (kLanes > 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = Op::of(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  if constexpr (kLanes > 32) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = Op::of(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  return v;
}

// all values of a group of kThr threads; a buffer serves one reduction
template <int kThr, typename Op>
__device__ __forceinline__ float group_reduce(float v, float* red) {
  v = lanes_reduce<Op, kWave>(v);
  if constexpr (kThr > kWave) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lanes_reduce<Op, kThr / kWave>(red[threadIdx.x % (kThr / kWave)]);
  }
  return v;
}
template <int kThr>
__device__ __forceinline__ float group_sum(float v, float* red) {
  return group_reduce<kThr, Sum>(v, red);
}

// 8 values of a row as they lie in memory, and as fp32
struct Raw {
  u32x4 a, b;
};
// kNt: read once
template <bool kNt>
__device__ __forceinline__ u32x4 load16(const u32x4* p) {
  return kNt ? __builtin_nontemporal_load(p) : *p;
}
template <bool kNt>
__device__ __forceinline__ Raw load_raw(const void* row, int bf16, int chunk) {
  const u32x4* p = static_cast<const u32x4*>(row);
  Raw v;
  if (bf16) {
    v.a = load16<kNt>(p + chunk);
    v.b = u32x4{0u, 0u, 0u, 0u};
  } else {
    v.a = load16<kNt>(p + 2 * chunk);
    v.b = load16<kNt>(p + 2 * chunk + 1);
  }
  return v;
}
template <bool kNt, int kThr, int kPer>
__device__ __forceinline__ void load_row(Raw (&raw)[kPer], const void* row, int bf16, int tid, int chunks) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = tid + kThr * i;
    raw[i] = c < chunks ? load_raw<kNt>(row, bf16, c) : Raw{};
  }
}
template <bool kNt, typename T>
__device__ __forceinline__ void store(T* p, T v) {
  if constexpr (kNt) __builtin_nontemporal_store(v, p);
  else *p = v;
}
__device__ __forceinline__ void widen(const Raw& v, int bf16, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      f[2 * i] = bf16_lo(v.a[i]);
      f[2 * i + 1] = bf16_hi(v.a[i]);
    } else {
      f[i] = __uint_as_float(v.a[i]);
      f[4 + i] = __uint_as_float(v.b[i]);
    }
  }
}
__device__ __forceinline__ void load_vector(const float* v, int chunk, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(v)[2 * chunk], b = reinterpret_cast<const float4*>(v)[2 * chunk + 1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ u32x4 bf16x8(const float (&f)[8]) {
  return u32x4{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
}

// What a row is multiplied by for its norm (weights apart): 1 / sqrt(mean square + eps); not fine
// where the row holds a NaN or an infinity.  The values may be scaled on the way, the factor too.
struct RowNorm {
  float f;
  bool fine;
};
template <int kThr, int kPer>
__device__ __forceinline__ RowNorm row_norm(float (&v)[kPer][8], float H, float eps, float* red, float* red2) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  ss = group_sum<kThr>(ss, red);
  const float mean = ss / H + eps;
  if (mean < INFINITY) return RowNorm{__builtin_amdgcn_rsqf(mean), true};
  constexpr float kDown = 0x1p-80f;                         // (the whole group comes here, or none: one sum)
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] *= kDown;
      ss = fmaf(v[i][j], v[i][j], ss);
    }
  ss = group_sum<kThr>(ss, red2);
  return RowNorm{__builtin_amdgcn_rsqf(ss / H + eps * kDown * kDown), ss < INFINITY};
}

// the largest value of a group, held as a sum of two: the larger m, of equal ones the larger rest,
// which is only asked for where m is a wave's largest
template <int kThr, typename F>
__device__ __forceinline__ float2 group_max_pair(float m, F rest_of, float* red) {
  float top = lanes_reduce<Max, kWave>(m);
  float rest = lanes_reduce<Max, kWave>(m == top ? rest_of(m) : -INFINITY);
  if constexpr (kThr > kWave) {
    float2* r = reinterpret_cast<float2*>(red);
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = make_float2(top, rest);
    __syncthreads();
    const float2 o = r[threadIdx.x % (kThr / kWave)];
    top = lanes_reduce<Max, kThr / kWave>(o.x);
    rest = lanes_reduce<Max, kThr / kWave>(o.x == top ? o.y : -INFINITY);
  }
  return make_float2(top, rest);
}

// kRes: with r (the residual form).  kNt: rows and results are marked as read and written once.  A
// block holds one group, or four of a wave.
template <int kThr, int kPer, bool kRes, int kCodes, bool kNt>
__global__ __launch_bounds__(kThr == kWave ? 4 * kWave : kThr) void norm_kernel(const NormArgs n) {
  __shared__ __attribute__((aligned(8))) float red[6][16];    // (the last two for one reduction of pairs)
  constexpr int kGroups = kThr == kWave ? 4 : 1;
  const int tid = kGroups > 1 ? threadIdx.x % kThr : threadIdx.x;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t t = block * kGroups + (kGroups > 1 ? threadIdx.x / kThr : 0);
  if (t >= n.T) return;                                     // (a whole block, or groups that meet no barrier)
  const int chunks = (int)(n.H >> 3);
  const float H = (float)n.H;
  const char* xr = static_cast<const char*>(n.x) + t * n.ld_x * (n.x_bf16 ? 2 : 4);
  float v[kPer][8];
  // Rows beyond 16384 do not fit in the registers of 1024 threads with all that is known of them: their
  // chunks of r are read as they are needed, and the weight twice for the products' second parts
  // (2000 bf16 rows of 24576 between two blocks 124 against 164 us; rows of 8192 to 16384 would lose, 89
  // to 116).
  constexpr bool kHold = kThr * kPer <= 2048;
  Raw raw[kPer], raw_r[kRes && kHold ? kPer : 1];
  const char* rr = static_cast<const char*>(n.r) + t * n.ld_r * (n.r_bf16 ? 2 : 4);
  load_row<kNt, kThr>(raw, xr, n.x_bf16, tid, chunks);
  if constexpr (kRes && kHold) load_row<kNt, kThr>(raw_r, rr, n.r_bf16, tid, chunks);
#pragma unroll
  for (int i = 0; i < kPer; ++i) widen(raw[i], n.x_bf16, v[i]);
  bool fine = true;
  if constexpr (kRes) {
    if (n.post) {
      const RowNorm r = row_norm<kThr, kPer>(v, H, n.eps, red[0], red[1]);
      fine = r.fine;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int c = tid + kThr * i;
        if (c < chunks) {
          float w[8];
          load_vector(n.post, c, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r.f * w[j];
        }
      }
    }
    const float tg = n.token_gate ? n.token_gate[t] : 1.0f;
    char* outr = static_cast<char*>(n.out) + t * n.ld_out * (n.r_bf16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = tid + kThr * i;
      if (c < chunks) {
        float r[8], g[8];
        widen(kHold ? raw_r[kHold ? i : 0] : load_raw<kNt>(rr, n.r_bf16, c), n.r_bf16, r);
        if (n.gate) load_vector(n.gate, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float p = v[i][j];
          if (n.gate) p *= g[j];
          if (n.token_gate) p *= tg;
          v[i][j] = fmaf(n.r_scale, r[j], p);
        }
        if (n.r_bf16) {
          store<kNt>(reinterpret_cast<u32x4*>(outr) + c, bf16x8(v[i]));
        } else {
          reinterpret_cast<float4*>(outr)[2 * c] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
          reinterpret_cast<float4*>(outr)[2 * c + 1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
        }
      }
    }
    if (!n.weight) return;
  }
  // n = f x weight, with f = g 2^e: the products (2^e x) weight are taken exactly, as a sum of two
  // fp32 values, and g, which every quotient n / max |n| lacks, only enters xn and the scale.  The
  // largest product is taken exactly too, and a quotient that fp32 rounds to a border between two
  // codes leaves it for its own side.  So a code is the nearest to the row's true quotient
  // (rounded products and quotients put 0.8 of a million on the other side of a border).
  const RowNorm r = row_norm<kThr, kPer>(v, H, n.eps, red[2], red[3]);
  fine &= r.fine;
  const float e2 = __uint_as_float(__float_as_uint(r.f) & 0x7f800000u), g = r.f / e2;
  float lo[kCodes != kCodesNone && kHold ? kPer : 1][8], top_of[kPer], m = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = tid + kThr * i;
    top_of[i] = 0.0f;
    if (c < chunks) {
      float w[8], o[8];
      load_vector(n.weight, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[i][j] * e2, p = x * w[j];
        if constexpr (kCodes != kCodesNone) {
          if constexpr (kHold) lo[i][j] = fmaf(x, w[j], -p);
          top_of[i] = fmaxf(top_of[i], fabsf(p));
        }
        v[i][j] = kHold ? p : x;
        o[j] = p * g;
      }
      if (n.xn) store<kNt>(reinterpret_cast<u32x4*>(n.xn + t * n.H) + c, bf16x8(o));
    }
  }
  if constexpr (kCodes != kCodesNone) {
    constexpr bool kInt8 = kCodes == kCodesI8;
    constexpr float kTop = kInt8 ? 127.0f : kFp8Max;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = fmaxf(m, top_of[i]);
    // chunk i's products, as sums of two
    auto products = [&](int i, float (&p)[8], float (&l)[8]) {
      float w[8];
      if constexpr (!kHold) load_vector(n.weight, tid + kThr * i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = kHold ? v[i][j] : v[i][j] * w[j];
        l[j] = kHold ? lo[kHold ? i : 0][j] : fmaf(v[i][j], w[j], -p[j]);
      }
    };
    const float2 largest = group_max_pair<kThr>(m, [&](float at) {
      float rest = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (top_of[i] == at && tid + kThr * i < chunks) {
          float p[8], l[8];
          products(i, p, l);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (fabsf(p[j]) == at) rest = fmaxf(rest, p[j] < 0.0f ? -l[j] : l[j]);
        }
      return rest;
    }, red[4]);
    m = largest.x;
    const float scale = row_scale<kInt8>(m * g);
    // kTop / m as a sum of two as well, to 2^-44 of it; rows of very small or large values are scaled
    // first, where a reciprocal would not be finite or normal
    const float by = m < 0x1p-80f ? 0x1p100f : m > 0x1p80f ? 0x1p-100f : 1.0f, top = m * by;
    const float c = top > 0.0f ? __builtin_amdgcn_rcpf(top) : 0.0f, c0 = kTop * c;
    const float c1 = fmaf(-c0, largest.y * by, fmaf(-c0, top, kTop)) * c;
    uint64_t* qr = reinterpret_cast<uint64_t*>(n.q + t * n.H);
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = tid + kThr * i;
      if (c < chunks) {
        float p[8], l[8], o[8];
        products(i, p, l);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] *= by, l[j] *= by;
          o[j] = fmaf(p[j], c0, fmaf(p[j], c1, l[j] * c0));
        }
        // (a border has 8 leading bits at most, of E4M3 5; zeros and the largest value need no care)
        constexpr int kLead = kInt8 ? 16 : 13;
        uint32_t low = ~0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) low = min(low, __float_as_uint(o[j]) << kLead);
        if (low == 0) {
          bool near = false;
          auto at_border = [&](int j) {
            return __float_as_uint(o[j]) << kLead == 0 && o[j] != 0.0f && fabsf(o[j]) < kTop;
          };
#pragma unroll
          for (int j = 0; j < 8; ++j) near |= at_border(j);
          if (near) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float over = fmaf(p[j], c0, -o[j]) + fmaf(p[j], c1, l[j] * c0);     // (of a tie, 2^-44 of o may be left)
              const uint32_t u = __float_as_uint(o[j]);
              if (at_border(j) && fabsf(over) > 0x1p-43f * fabsf(o[j]))
                o[j] = __uint_as_float((over > 0.0f) == (o[j] > 0.0f) ? u + 1 : u - 1);
            }
          }
        }
        const uint2 q = make_uint2(nearest4<kInt8>(o[0], o[1], o[2], o[3]), nearest4<kInt8>(o[4], o[5], o[6], o[7]));
        if constexpr (kInt8) sum = __builtin_amdgcn_sdot4(q.x, 0x01010101, __builtin_amdgcn_sdot4(q.y, 0x01010101, sum, false), false);
        store<kNt>(qr + c, q.x | (uint64_t)q.y << 32);
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

// kBoth, or the norms alone, or the residual forms alone
enum Forms : int { kBoth = 0, kNorms = 1, kResiduals = 2 };
template <int kThr, int kPer, bool kNt, int kForms = kBoth>
static void launch_norm_form(const NormArgs& n, hipStream_t stream) {
  constexpr int kGroups = kThr == kWave ? 4 : 1;
  // (a launch has fewer than 2^32 threads in x)
  constexpr int64_t kWide = (int64_t)1 << 21;
  const int64_t blocks = (n.T + kGroups - 1) / kGroups;
  const dim3 grid((unsigned)(blocks < kWide ? blocks : kWide), (unsigned)((blocks + kWide - 1) / kWide)), block(kThr * kGroups);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, n); };
  if constexpr (kForms != kNorms) {
    if (n.r) {
      if (n.codes == kCodesFp8) go(norm_kernel<kThr, kPer, true, kCodesFp8, kNt>);
      else if (n.codes == kCodesI8) go(norm_kernel<kThr, kPer, true, kCodesI8, kNt>);
      else go(norm_kernel<kThr, kPer, true, kCodesNone, kNt>);
    }
  }
  if constexpr (kForms != kResiduals) {
    if (!n.r) {
      if (n.codes == kCodesFp8) go(norm_kernel<kThr, kPer, false, kCodesFp8, kNt>);
      else if (n.codes == kCodesI8) go(norm_kernel<kThr, kPer, false, kCodesI8, kNt>);
      else go(norm_kernel<kThr, kPer, false, kCodesNone, kNt>);
    }
  }
}

// A row has as many threads as keep it in a few registers: 256 of bf16, 512 where fp32 is among the
// rows (norms on both sides of 8192 rows of 6144, fp32: 149 against 158 us; 16384 bf16 rows, norm
// alone: 89 against 86; 4 us more each since codes are exact).  While there is a CU for every row, as many as it has chunks, up to 1024 (128
// rows of 6144: the norm 3.6 against 4.0 us with 256, between two blocks 5.5 against 7.0).  Rows of 1025
// to 2048 have 128 (24000 bf16 rows of 2048 between two blocks: 95 against 107 us with a wave each);
// the residual forms, which hold two rows, 1024 beyond 8192 (4000 bf16 rows of 12288: 108 against 155
// with 256, fp32 185 against 201 with 512; the norm alone is the faster with few, 93 against 107).
constexpr int64_t kFewRows = 256;
template <bool kNt>
static void launch_bf16_rows(const NormArgs& n, hipStream_t stream) {
  if (n.H <= 4096) launch_norm_form<256, 2, kNt>(n, stream);
  else if (n.H <= 6144) launch_norm_form<256, 3, kNt>(n, stream);
  else if (n.H <= 8192) launch_norm_form<256, 4, kNt>(n, stream);
  else if (n.r) launch_norm_form<1024, 2, kNt, kResiduals>(n, stream);
  else launch_norm_form<256, 8, kNt, kNorms>(n, stream);
}

// From here on bf16 rows and their results are marked as read or written once: they would only push
// each other out of the 256 MB last-level cache (16384 rows of 6144 90 against 97 us; norm, a
// product of 6144 outputs and the residual of 8192 rows 327 against 341 us).  Below, the reader of
// the results finds them there (2048 rows 90 against 98 us).  fp32 rows gain nothing.
constexpr int64_t kStreamBytes = (int64_t)192 << 20;

hipError_t launch_norm(const NormArgs& n, hipStream_t stream) {
  if (n.T == 0) return hipSuccess;
  const bool bf16 = n.x_bf16 && (!n.r || n.r_bf16);
  const int64_t bytes = n.T * n.H * (2 + (n.r ? 4 : 0) + (n.xn ? 2 : 0) + (n.q ? 1 : 0));
  if (n.H <= 512) launch_norm_form<64, 1, false>(n, stream);
  else if (n.H <= 1024) launch_norm_form<64, 2, false>(n, stream);
  else if (n.H <= 2048) launch_norm_form<128, 2, false>(n, stream);
  else if (n.H > 16384) launch_norm_form<1024, 4, false>(n, stream);
  else if (n.T <= kFewRows && n.H <= 8192) launch_norm_form<1024, 1, false>(n, stream);
  else if (n.T <= kFewRows) launch_norm_form<1024, 2, false>(n, stream);
  else if (bf16 && bytes > kStreamBytes) launch_bf16_rows<true>(n, stream);
  else if (bf16) launch_bf16_rows<false>(n, stream);
  else if (n.H <= 4096) launch_norm_form<512, 1, false>(n, stream);
  else if (n.H <= 8192) launch_norm_form<512, 2, false>(n, stream);
  else if (n.r) launch_norm_form<1024, 2, false, kResiduals>(n, stream);
  else launch_norm_form<512, 4, false, kNorms>(n, stream);
  return hipGetLastError();
}

}  // namespace w4a8
