// The whole routed-expert layer for a few tokens (1 to 16) in two kernels, on the
// GEMM storage.
//
//   few_gate_up: route and quantize the tokens, then gate/up and SwiGLU:
//     act[f, i] = silu(gate) up for every routed index f = t k + j;
//   few_down: requantize act per row, then down and the routing-weighted sum:
//     y[t, n] = sum_j w[t, j] sa[f] sum_i qa[f, i] q2[e, n, i] s2.
//
// With so few tokens a step is one read of the touched experts' weights plus the
// time to start: launches, and loads that wait for one another.  So:
//   * routing and quantization are repeated by every workgroup of the first kernel
//     (a logits row and an activation row come from the cache) instead of being a
//     launch of their own; the requantization likewise in the second;
//   * all T tokens are the rows of one 16-row matrix-core block, whichever expert is
//     multiplied: the A operand is the same for every expert, needs no gather, and
//     each token keeps only the columns of the experts it is routed to;
//   * an expert that several tokens picked is read once: the workgroups go over the
//     distinct experts;
//   * the 8 waves of a workgroup split K (gate/up) or the (expert, K chunk) pieces
//     (down), so that even one token puts enough loads in flight; their partial
//     tiles meet in LDS and are summed in wave order: the same bits at every run.
// The products run on the bf16 matrix cores (w4_bf16.hpp; INT8 form: the INT8 ones,
// exact), so act and y carry fp32 rounding only.
#include "kernels.hpp"
#include "w4_bf16.hpp"

#include <type_traits>

namespace w4a8 {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = 64 * kFewWaves;
constexpr int kFewDownGroups = 4;              // K groups of one (expert, K chunk) piece of the down product

// ---- values -----------------------------------------------------------------
// x / s rounded to fp32 from r = 1 / s rounded: q = fl(x r) is within an ulp, its
// residual x - q s is exact in an FMA, and the corrected quotient is the correctly
// rounded one (Markstein's theorem; no differing result in 10^9 random pairs of an
// amax and a value below it).  3 instructions instead of the ~10 of a division.
__device__ __forceinline__ float div_by(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

// four codes of four values of a row with scale s (r = 1 / s), the first in byte 0.
// The FP8 conversion instruction rounds to nearest even like e4m3_encode (equal on
// every fp32 magnitude up to 448).  No clamp: a quotient is at most a rounding above
// 448 (127), which rounds to the largest code.
template <bool kInt8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s, float r) {
  const float v[4] = {div_by(a, s, r), div_by(b, s, r), div_by(c, s, r), div_by(d, s, r)};
  if constexpr (kInt8) {
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) o |= ((uint32_t)(int)rintf(v[i]) & 0xffu) << (8 * i);
    return o;
  } else {
    const int o = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], o, true);
  }
}

template <bool kInt8>
__device__ __forceinline__ float row_scale(float amax) {
  return amax > 0.0f ? amax / (kInt8 ? 127.0f : kFp8Max) : 1.0f;
}

// orders LDS accesses of one wave's lanes (the LDS itself serves a wave in order)
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---- routing of one token by one wave ---------------------------------------
// fp32 -> uint32 with the order of the values (-0 as +0); 0 is below every value
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return k > 1u ? k : 1u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
// the largest key of the wave, as a uniform value
__device__ __forceinline__ uint32_t wave_max_key(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));   // row_shr:1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));   // row_shr:2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));   // row_shr:4
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));   // row_shr:8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));   // row_bcast:15
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));   // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

constexpr int kRouteSlots = 16;                // 1024 experts

// The k experts of a logits row and their weights, with the order, ties and sums of
// w4a8_moe_route (the same bits): slot s of lane l is expert l + 64 s.  Every id
// written is in [0, E), whatever the logits hold.
// v: the row's logits, loaded before.  picked: a bit for each expert.
template <int S>
__device__ __forceinline__ void route_token(const float (&v)[kRouteSlots], int E, int k, int renormalize, int* ids,
                                            float* w, uint32_t* picked) {
  const int lane = threadIdx.x & 63;
  uint32_t key[S];
#pragma unroll
  for (int s = 0; s < S; ++s) key[s] = lane + s * kWave < E ? order_key(v[s]) : 0u;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int s = 1; s < S; ++s) best = max(best, key[s]);
    best = wave_max_key(best);
    // the lowest expert that holds it: the first slot with a match, its lowest lane
    int id = 0;
    bool found = false;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const uint64_t hit = __ballot(key[s] == best);
      if (!found && hit) {
        found = true;
        const int l = __builtin_ctzll(hit);
        id = s * kWave + l;
        if (lane == l) key[s] = 0u;
      }
    }
    if (lane == 0) {
      ids[j] = id;
      w[j] = key_value(best);
      atomicOr(&picked[id >> 5], 1u << (id & 31));
    }
  }
  wave_lds_fence();
  const float m = w[0];
  float denom = 0.0f;
  if (renormalize) {
    for (int j = lane; j < k; j += kWave) denom += expf(w[j] - m);
  } else {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (lane + s * kWave < E) denom += expf(v[s] - m);
  }
  denom = wave_sum(denom);
  wave_lds_fence();
  for (int j = lane; j < k; j += kWave) w[j] = expf(w[j] - m) / denom;
}

// ---- what the first kernel leaves for the second ------------------------------
// Views into the caller's workspace (16-byte aligned): the number of distinct
// experts, the experts, the routed index of (expert, token) or -1, the routing
// weights, act [R][I] and the maxima of |act| over its 16-column blocks [R][I/16].
struct FewWorkspace {
  int32_t* count;
  int32_t* experts;       // [kFewMaxRows]
  int16_t* slot;          // [kFewMaxRows][16]
  float* weights;         // [kFewMaxRows]
  float* act;
  float* pmax;
};
__device__ __host__ __forceinline__ FewWorkspace few_workspace(void* p, int64_t R, int64_t I) {
  unsigned char* b = static_cast<unsigned char*>(p);
  FewWorkspace v;
  v.count = reinterpret_cast<int32_t*>(b);
  v.experts = reinterpret_cast<int32_t*>(b + 16);
  v.weights = reinterpret_cast<float*>(b + 16 + 4 * kFewMaxRows);
  v.slot = reinterpret_cast<int16_t*>(b + 16 + 8 * kFewMaxRows);
  v.act = reinterpret_cast<float*>(b + kFewHeadBytes);
  v.pmax = v.act + R * I;
  return v;
}

// A x W of one K group for one 16-column subtile: a the lane's 32 activation codes,
// w its 16 weight bytes.  INT8 form: int32 sums, the -8 rowsum(a) included.
template <int kForm>
struct FewProduct {
  static constexpr bool kInt8 = kForm == kFormChannel;
  using Acc = std::conditional_t<kInt8, i32x4, v4f>;
  i32x4 ab[4];            // FP8 forms: the codes as bf16 operands
  v8i ai;                 // INT8 form: the codes
  Acc bias;
  __device__ __forceinline__ void set_codes(v8i a) {
    if constexpr (kInt8) {
      ai = a;
      const i32x4 m = {(int)0xf8f8f8f8, (int)0xf8f8f8f8, (int)0xf8f8f8f8, (int)0xf8f8f8f8};   // -8
      bias = mfma_i8_16x16x64(a.hi, m, mfma_i8_16x16x64(a.lo, m, i32x4{0, 0, 0, 0}));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) ab[c] = e4m3x8_to_bf16((uint32_t)a[2 * c], (uint32_t)a[2 * c + 1], 1.0f);
      set_bias();
    }
  }
  __device__ __forceinline__ void set_bias() {
    if constexpr (kForm == kFormG128) bias = minus8_product(ab);
    else bias = Acc{0, 0, 0, 0};
  }
  __device__ __forceinline__ void add(i32x4 w, uint32_t s, Acc& acc) const {
    if constexpr (kInt8) {
      const v8i b = nibbles_to_fp8(w);         // the bytes u, read as INT8
      const i32x4 d = mfma_i8_16x16x64(ai.hi, b.hi, mfma_i8_16x16x64(ai.lo, b.lo, bias));
      acc += d;
    } else {
      group_product<kForm, false>(ab, w, s, bias, acc);
    }
  }
};

// ---- kernel 1: routing, quantization, gate/up, SwiGLU -----------------------
// A task is 16 columns of act for one distinct expert: 16 gate and 16 up rows of
// w13, K split over the 8 waves.  The workgroups walk the tasks; a wave refills each
// weight register with the next task's as it uses it up.
// GW: the most K groups of a wave (H <= 1024 GW).  S: logits per lane (E <= 64 S).
template <int kForm, int GW, int S>
__global__ __launch_bounds__(kFewThreads) void few_gate_up_kernel(const uint16_t* __restrict__ x, int T, int64_t H,
                                                                  int64_t ld, const float* __restrict__ logits, int E,
                                                                  int k, int renormalize,
                                                                  const uint8_t* __restrict__ w13,
                                                                  const uint8_t* __restrict__ s13, int64_t I,
                                                                  int32_t* __restrict__ ids_out,
                                                                  float* __restrict__ w_out, void* workspace) {
  using P = FewProduct<kForm>;
  using Acc = typename P::Acc;
  constexpr bool kInt8 = P::kInt8;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ int ids[kFewMaxRows];
  __shared__ float wts[kFewMaxRows];
  __shared__ int experts[kFewMaxRows];
  __shared__ __attribute__((aligned(16))) int16_t slot[kFewMaxRows][kFewMaxTokens];
  __shared__ float wave_amax[kFewMaxTokens][kFewWaves];
  __shared__ uint32_t picked[32];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int G = (int)(H >> 7), R = T * k;
  uint8_t* codes = smem;                                          // [G][4][T][32]
  float* red = reinterpret_cast<float*>(smem + (size_t)T * H);    // [2][waves][2][T][16]; int32 for INT8

  // The waves share the rows of x, wpr waves to a row; every load of the prologue that
  // depends on nothing is issued here.
  const int wpr = T == 1 ? 8 : T == 2 ? 4 : T <= 4 ? 2 : 1;       // waves per row
  const int rows_at_once = kFewWaves / wpr;                       // T <= 16: at most two rows per wave
  const int part = wave % wpr;
  const int chunks = (int)(H >> 3);                               // of 8 elements
  float lg[kRouteSlots];
  const bool routes = wave < T;                                   // waves 0 .. T-1 route (and wave + 8 for T > 8)
#pragma unroll
  for (int s = 0; s < S; ++s) lg[s] = routes && lane + s * kWave < E ? logits[(int64_t)wave * E + lane + s * kWave] : 0.0f;
  if (threadIdx.x < 32) picked[threadIdx.x] = 0u;
  for (int i = threadIdx.x; i < R * kFewMaxTokens / 2; i += kFewThreads) reinterpret_cast<int*>(slot)[i] = -1;
  for (int t0 = 0; t0 < T; t0 += rows_at_once) {                  // row maxima of x
    const int t = t0 + wave / wpr;
    if (t < T) {
      const uint4* xr = reinterpret_cast<const uint4*>(x + (int64_t)t * ld);
      float amax = 0.0f;
#pragma unroll 4
      for (int c = part * 64 + lane; c < chunks; c += 64 * wpr) {
        const uint4 v = xr[c];
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(u[i])), fabsf(bf16_hi(u[i]))));
      }
      amax = wave_max(amax);
      if (lane == 0) wave_amax[t][part] = amax;
    }
  }
  __syncthreads();                                                // picked and slot are set
  if (routes) route_token<S>(lg, E, k, renormalize, ids + wave * k, wts + wave * k, picked);
  if (wave + kFewWaves < T) {
    const int t = wave + kFewWaves;
#pragma unroll
    for (int s = 0; s < S; ++s) lg[s] = lane + s * kWave < E ? logits[(int64_t)t * E + lane + s * kWave] : 0.0f;
    route_token<S>(lg, E, k, renormalize, ids + t * k, wts + t * k, picked);
  }
  __syncthreads();                                                // ids, weights, picked and row maxima are there

  // The distinct experts in ascending order: expert e is number (bits of picked below e).
  // Lane l holds word l and the bits in the words before it.
  const uint32_t word = lane < 32 ? picked[lane] : 0u;
  int below = __builtin_popcount(word);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up(below, off, kWave);
    if (lane >= off) below += o;
  }
  const int D = __builtin_amdgcn_readlane(below, 31);
  below -= __builtin_popcount(word);
  const int f = threadIdx.x;                                      // R <= 256 < 512 threads
  {
    const int e = f < R ? ids[f] : 0;
    const uint32_t we = (uint32_t)__shfl((int)word, e >> 5, kWave);
    const int number = __shfl(below, e >> 5, kWave) + __builtin_popcount(we & ((1u << (e & 31)) - 1u));
    if (f < R) {
      slot[number][f / k] = (int16_t)f;
      experts[number] = e;                                        // the same value from every token that picked it
    }
  }
  __syncthreads();

  const FewWorkspace ws = few_workspace(workspace, R, I);
  const int blocks = (int)(I >> 4);                               // column blocks of act
  const int ntasks = D * blocks;
  const int gpw = (G + kFewWaves - 1) / kFewWaves;                // <= GW
  const int g0 = wave * gpw, ng = max(0, min(gpw, G - g0));
  i32x4 wg[GW], wu[GW];
  uint32_t sg[GW], su[GW];
  __amdgpu_buffer_rsrc_t rg = buffer_of(w13, 0), ru = rg, rs = buffer_of(s13, 0);
  auto point = [&](int task) {                                    // the task's weights of this wave; none past the last task
    const bool on = task < ntasks && ng > 0;
    const int d = on ? task / blocks : 0, cb = on ? task - d * blocks : 0;
    const int64_t e = __builtin_amdgcn_readfirstlane(experts[d]);
    const uint8_t* p = w13 + ((e * (I >> 3) + cb) * G + g0) * 1024;
    rg = buffer_of(p, on ? ng * 1024 : 0);
    ru = buffer_of(p + (I >> 4) * G * 1024, on ? ng * 1024 : 0);
    if constexpr (!kInt8) rs = buffer_of(s13 + (((e * G + g0) * 2 * I) + 16 * cb) * 4, on ? ((int64_t)ng * 2 * I - 16 * cb) * 4 : 0);
  };
  auto load = [&](int i) {
    wg[i] = buffer_load16_nt(rg, col * 64 + kq * 16 + i * 1024);
    wu[i] = buffer_load16_nt(ru, col * 64 + kq * 16 + i * 1024);
    if constexpr (!kInt8) {
      sg[i] = buffer_load4(rs, (uint32_t)(i * 2 * I + col) * 4);
      su[i] = buffer_load4(rs, (uint32_t)(i * 2 * I + I + col) * 4);
    }
  };
  int task = blockIdx.x, buf = 0;
  point(task);
#pragma unroll
  for (int i = 0; i < GW; ++i) load(i);

  if (blockIdx.x == 0) {                                          // the routing, for the second kernel and the caller
    if (f == 0) *ws.count = D;
    if (f < D) ws.experts[f] = experts[f];
    if (f < R) {
      ws.weights[f] = wts[f];
      if (ids_out) ids_out[f] = ids[f];
      if (w_out) w_out[f] = wts[f];
    }
    for (int i = threadIdx.x; i < D * kFewMaxTokens / 2; i += kFewThreads)
      reinterpret_cast<int*>(ws.slot)[i] = reinterpret_cast<const int*>(slot)[i];
  }

  // the codes, in operand order: byte o of lane group kq of row t, group g
  for (int t0 = 0; t0 < T; t0 += rows_at_once) {
    const int t = t0 + wave / wpr;
    if (t < T) {
      float amax = 0.0f;
      for (int p = 0; p < wpr; ++p) amax = fmaxf(amax, wave_amax[t][p]);
      const float sc = row_scale<kInt8>(amax), rc = 1.0f / sc;
      const uint4* xr = reinterpret_cast<const uint4*>(x + (int64_t)t * ld);
      for (int c = part * 64 + lane; c < chunks; c += 64 * wpr) {
        const uint4 v = xr[c];
        uint2 o;
        o.x = codes4<kInt8>(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), sc, rc);
        o.y = codes4<kInt8>(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), sc, rc);
        // elements 8 c .. +7: group c / 16, lane group (c / 4) % 4, byte 8 (c % 4)
        *reinterpret_cast<uint2*>(codes + ((size_t)(c >> 2) * T + t) * 32 + 8 * (c & 3)) = o;
      }
    }
  }
  __syncthreads();

  const uint8_t* arow = codes + ((size_t)(4 * g0 + kq) * T + min(col, T - 1)) * 32;
  const size_t astep = (size_t)128 * T;
  // this thread's token scale (threads below 16 T finish the tiles: token threadIdx.x / 16)
  float sx = 1.0f;
  if ((int)threadIdx.x < 16 * T) {
    float amax = 0.0f;
    for (int p = 0; p < wpr; ++p) amax = fmaxf(amax, wave_amax[threadIdx.x >> 4][p]);
    sx = row_scale<kInt8>(amax);
  }
  for (; task < ntasks; task += gridDim.x, buf ^= 1) {
    point(task + (int)gridDim.x);
    Acc ag = Acc{0, 0, 0, 0}, au = Acc{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < GW; ++i) {
      if (i < ng) {
        P p;
        p.set_codes(*reinterpret_cast<const v8i*>(arow + i * astep));
        uint32_t fg = 0, fu = 0;
        if constexpr (!kInt8) {
          fg = kForm == kFormMx ? (sg[i] >> (8 * kq)) & 0xffu : sg[i];
          fu = kForm == kFormMx ? (su[i] >> (8 * kq)) & 0xffu : su[i];
        }
        p.add(wg[i], fg, ag);
        p.add(wu[i], fu, au);
      }
      load(i);
    }
    // the partial tiles: red[buf][wave][gate, up][t][col]
    float* rb = red + (size_t)buf * kFewWaves * 2 * T * 16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 4 * kq + r;
      if (t < T) {
        float* at = rb + ((size_t)wave * 2 * T + t) * 16 + col;
        if constexpr (kInt8) {
          at[0] = __int_as_float(ag[r]);
          at[T * 16] = __int_as_float(au[r]);
        } else {
          at[0] = ag[r];
          at[T * 16] = au[r];
        }
      }
    }
    __syncthreads();       // one per task: the other buffer's readers passed the last one
    if ((int)threadIdx.x < 16 * T) {
      const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
      const int d = task / blocks, cb = task - d * blocks;
      const int fr = slot[d][t];
      float gate, up;
      const float* at = rb + (size_t)t * 16 + c;
      if constexpr (kInt8) {
        int ig = 0, iu = 0;
#pragma unroll
        for (int v = 0; v < kFewWaves; ++v) {
          ig += __float_as_int(at[(size_t)v * 2 * T * 16]);
          iu += __float_as_int(at[(size_t)(v * 2 + 1) * T * 16]);
        }
        const float* sw = reinterpret_cast<const float*>(s13) + (int64_t)experts[d] * 2 * I + 16 * cb + c;
        gate = (float)ig * sx * sw[0];
        up = (float)iu * sx * sw[I];
      } else {
        gate = 0.0f;
        up = 0.0f;
#pragma unroll
        for (int v = 0; v < kFewWaves; ++v) {
          gate += at[(size_t)v * 2 * T * 16];
          up += at[(size_t)(v * 2 + 1) * T * 16];
        }
        gate *= sx;
        up *= sx;
      }
      const float a = silu_mul(gate, up);
      const float m = max16(fabsf(a));
      if (fr >= 0) {
        ws.act[(int64_t)fr * I + 16 * cb + c] = a;
        if (c == 0) ws.pmax[(int64_t)fr * blocks + cb] = m;
      }
    }
  }
}

// ---- kernel 2: requantization, down, the routing-weighted sum ----------------
// A workgroup owns 16 columns of y for every token.  Its waves take the (distinct
// expert, 4-group K chunk) pieces in turn: each requantizes the act of the expert's
// tokens over those K elements into LDS of its own, up to 4 tokens at a time as rows
// 0..3 of the A operand (an expert has one or two of the few tokens as a rule; the
// weights stay in registers for the next 4), multiplies, and adds the rows with the
// factors w[t, j] sa[f] to its own sums of y in LDS.  The next piece's weights, and
// the act of its first two tokens, are loaded meanwhile.
// The FP8 codes are held as the bf16 values they stand for: converting them once per
// token and piece instead of once per operand read takes 16 of about 80 instructions
// out of a K group's product, which are what bounds this kernel besides HBM.
template <int kForm>
__global__ __launch_bounds__(kFewThreads) void few_down_kernel(int T, int64_t H, int k, const uint8_t* __restrict__ w2,
                                                               const uint8_t* __restrict__ s2, int64_t I,
                                                               const void* __restrict__ workspace,
                                                               void* __restrict__ y, int y_bf16) {
  using P = FewProduct<kForm>;
  using Acc = typename P::Acc;
  constexpr bool kInt8 = P::kInt8;
  constexpr int CG = kFewDownGroups;
  constexpr int kRows = 4;                                               // rows of A in use
  constexpr int kQuads = CG * kGroup / 4 / 64;                           // float4 of act per lane, token and piece
  // the wave's A rows: FP8 forms [CG][4 products][4 lane groups][rows][16 bytes], INT8 form [CG][4][rows][32 bytes]
  __shared__ __attribute__((aligned(16))) uint8_t a_sm[kFewWaves][CG * kGroup * kRows * (kInt8 ? 1 : 2)];
  __shared__ float scale[kFewMaxRows], factor[kFewMaxRows];              // sa[f], w[f] sa[f]
  __shared__ int experts[kFewMaxRows];
  __shared__ uint32_t routed[kFewMaxRows];                               // bit t: token t picked the expert
  __shared__ __attribute__((aligned(16))) int16_t slot[kFewMaxRows][kFewMaxTokens];
  extern __shared__ float y_sm[];                                        // [waves][T][16]

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int G = (int)(I >> 7), R = T * k;
  const int nch = (G + CG - 1) / CG;                                     // K chunks of an expert
  const int64_t cb = blockIdx.x;
  const FewWorkspace ws = few_workspace(const_cast<void*>(workspace), R, I);

  // The weights of a piece, and the act of two of its tokens.  Loads past the last piece,
  // or of a token that is not there, read nothing.
  i32x4 w[CG];
  uint32_t s[CG];
  float4 av0[kQuads], av1[kQuads];
  __amdgpu_buffer_rsrc_t rw, rs;
  auto point = [&](int64_t e, int g0, bool on) {
    const int n = min(CG, G - g0);
    rw = buffer_of(w2 + ((e * (H >> 4) + cb) * G + g0) * 1024, on ? n * 1024 : 0);
    if constexpr (!kInt8) rs = buffer_of(s2 + ((e * G + g0) * H + 16 * cb) * 4, on ? (n * H - 16 * cb) * 4 : 0);
  };
  auto load = [&](int i) {
    w[i] = buffer_load16_nt(rw, col * 64 + kq * 16 + i * 1024);
    if constexpr (!kInt8) s[i] = buffer_load4(rs, (uint32_t)(i * H + col) * 4);
  };
  auto load_act = [&](float4 (&v)[kQuads], int f, int g0) {              // f < 0: nothing
    const __amdgpu_buffer_rsrc_t ra = buffer_of(ws.act + (int64_t)max(f, 0) * I + (int64_t)g0 * kGroup,
                                                f >= 0 ? min(CG, G - g0) * kGroup * 4 : 0);
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
      v[q] = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(ra, (lane + 64 * q) * 16, 0, 0));
  };
  // the first piece of the wave, from what the first kernel left in memory
  const int items = __builtin_amdgcn_readfirstlane(*ws.count) * nch;
  {
    const bool on = wave < items;
    const int d = on ? wave / nch : 0, g0 = on ? (wave - d * nch) * CG : 0;
    const int e = __builtin_amdgcn_readfirstlane(ws.experts[d]);
    const int f = ws.slot[(int64_t)d * kFewMaxTokens + col];
    const uint32_t any = (uint32_t)__ballot(f >= 0) & 0xffffu, rest = any & (any - 1);
    const int f0 = __builtin_amdgcn_readlane(f, any ? __builtin_ctz(any) : 0);
    const int f1 = __builtin_amdgcn_readlane(f, rest ? __builtin_ctz(rest) : 0);
    load_act(av0, on && any ? f0 : -1, g0);
    load_act(av1, on && rest ? f1 : -1, g0);
    point(e, g0, on);
#pragma unroll
    for (int i = 0; i < CG; ++i) load(i);
  }
  const int D = items / nch;
  for (int i = threadIdx.x; i < D; i += kFewThreads) experts[i] = ws.experts[i];
  for (int i = threadIdx.x; i < D * kFewMaxTokens; i += kFewThreads) {   // 16 lanes per expert
    const int f = ws.slot[i];
    slot[i >> 4][i & 15] = (int16_t)f;
    const uint64_t any = __ballot(f >= 0);
    if ((i & 15) == 0) routed[i >> 4] = (uint32_t)(any >> (lane & 48)) & 0xffffu;
  }
  const int blocks = (int)(I >> 4);
  for (int f = wave; f < R; f += kFewWaves) {                            // the row maxima
    float m = 0.0f;
    for (int b = lane; b < blocks; b += 64) m = fmaxf(m, ws.pmax[(int64_t)f * blocks + b]);
    m = wave_max(m);
    if (lane == 0) {
      const float sa = row_scale<kInt8>(m);
      scale[f] = sa;
      factor[f] = ws.weights[f] * sa;
    }
  }
  for (int i = threadIdx.x; i < kFewWaves * T * 16; i += kFewThreads) y_sm[i] = 0.0f;
  __syncthreads();

  uint8_t* mine = a_sm[wave];
  float* ymine = y_sm + (size_t)wave * T * 16;
  auto put = [&](const float4 (&v)[kQuads], int row, int f) {            // one token's codes of a piece
    const float sc = scale[f], rc = 1.0f / sc;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      // 4 elements: group q / 32, lane group (q / 8) % 4, elements 4 (q % 8) of its 32 (past the piece's
      // groups: zeros, which nothing reads)
      const int q = lane + 64 * i;
      const uint32_t c4 = codes4<kInt8>(v[i].x, v[i].y, v[i].z, v[i].w, sc, rc);
      if constexpr (kInt8) {
        *reinterpret_cast<uint32_t*>(mine + ((q >> 3) * kRows + row) * 32 + 4 * (q & 7)) = c4;
      } else {
        uint2 b;
        b.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c4, 1.0f, false));
        b.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c4, 1.0f, true));
        const int g = q >> 5, c = (q & 7) >> 1, l = (q >> 3) & 3;
        *reinterpret_cast<uint2*>(mine + (((g * 4 + c) * 4 + l) * kRows + row) * 16 + 8 * (q & 1)) = b;
      }
    }
  };
  // rows of A: the tokens of `set` from row `row` on, their act loaded here
  auto put_rest = [&](uint32_t set, int d, int row, int g0) {
    for (; set && row < kRows; set &= set - 1, ++row) {
      const int f = __builtin_amdgcn_readfirstlane((int)slot[d][__builtin_ctz(set)]);
      load_act(av0, f, g0);
      put(av0, row, f);
    }
    return set;
  };
  auto product = [&](int i, Acc& acc, int rows) {
    const int row = col < rows ? col : 0;
    P p;
    if constexpr (kInt8) {
      p.set_codes(*reinterpret_cast<const v8i*>(mine + ((i * 4 + kq) * kRows + row) * 32));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        p.ab[c] = *reinterpret_cast<const i32x4*>(mine + (((i * 4 + c) * 4 + kq) * kRows + row) * 16);
      p.set_bias();
    }
    uint32_t fs = 0;
    if constexpr (!kInt8) fs = kForm == kFormMx ? (s[i] >> (8 * kq)) & 0xffu : s[i];
    p.add(w[i], fs, acc);
  };
  // row r of the tile (lanes 0..15) to the sums of the r-th token of `set`
  auto add_rows = [&](const Acc& acc, uint32_t set, int d) {
    float ws_n = 1.0f;
    if constexpr (kInt8) ws_n = reinterpret_cast<const float*>(s2)[(int64_t)experts[d] * H + 16 * cb + col];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (set) {
        const int t = __builtin_ctz(set);
        set &= set - 1;
        if (lane < 16) {
          float* at = ymine + t * 16 + col;
          *at = fmaf(factor[slot[d][t]], kInt8 ? (float)acc[r] * ws_n : (float)acc[r], *at);
        }
      }
    }
  };
  for (int it = wave; it < items; it += kFewWaves) {
    const int d = it / nch, g0 = (it - d * nch) * CG, ng = min(CG, G - g0);
    uint32_t tokens = __builtin_amdgcn_readfirstlane(routed[d]);         // at least one bit
    int rows = min(__builtin_popcount(tokens), kRows);
    put(av0, 0, __builtin_amdgcn_readfirstlane((int)slot[d][__builtin_ctz(tokens)]));
    uint32_t next = tokens & (tokens - 1);
    if (next) {
      put(av1, 1, __builtin_amdgcn_readfirstlane((int)slot[d][__builtin_ctz(next)]));
      next = put_rest(next & (next - 1), d, 2, g0);
    }
    while (next) {                                                       // more than 4 tokens: the same weights again
      // (opaque here: hoisted out of the loop, the unpacked weights would take a third more registers)
#pragma unroll
      for (int i = 0; i < CG; ++i) asm volatile("" : "+v"(w[i]));
      wave_lds_fence();
      Acc acc = Acc{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < CG; ++i)
        if (i < ng) product(i, acc, rows);
      add_rows(acc, tokens, d);
      wave_lds_fence();
      tokens = next;
      rows = min(__builtin_popcount(tokens), kRows);
      next = put_rest(tokens, d, 0, g0);
    }
    wave_lds_fence();
    {
      const int nx = it + kFewWaves;
      const bool on = nx < items;
      const int dn = on ? nx / nch : 0, gn = on ? (nx - dn * nch) * CG : 0;
      const uint32_t tn = __builtin_amdgcn_readfirstlane(routed[dn]), rest = tn & (tn - 1);
      const int f0 = __builtin_amdgcn_readfirstlane((int)slot[dn][__builtin_ctz(tn)]);
      const int f1 = __builtin_amdgcn_readfirstlane((int)slot[dn][rest ? __builtin_ctz(rest) : 0]);
      load_act(av0, on ? f0 : -1, gn);
      load_act(av1, on && rest ? f1 : -1, gn);
      point(__builtin_amdgcn_readfirstlane(experts[dn]), gn, on);
    }
    Acc acc = Acc{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      if (i < ng) product(i, acc, rows);
      load(i);
    }
    add_rows(acc, tokens, d);
    wave_lds_fence();
  }
  __syncthreads();
  if ((int)threadIdx.x < 16 * T) {
    const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < kFewWaves; ++v) sum += y_sm[((size_t)v * T + t) * 16 + c];
    if (y_bf16) static_cast<uint16_t*>(y)[(int64_t)t * H + 16 * cb + c] = __builtin_bit_cast(uint16_t, (__bf16)sum);
    else static_cast<float*>(y)[(int64_t)t * H + 16 * cb + c] = sum;
  }
}

// ---- launches ------------------------------------------------------------------
template <int kForm, int GW, int S>
static hipError_t launch_few_form(const FewArgs& a, hipStream_t stream) {
  const int64_t R = a.T * a.k;
  const int64_t tasks = (R < a.E ? R : a.E) * (a.I >> 4);                // at most
  const unsigned grid = (unsigned)(tasks < 512 ? tasks : 512);
  const size_t smem = (size_t)few_gate_up_smem(a.T, a.H);
  hipLaunchKernelGGL((few_gate_up_kernel<kForm, GW, S>), dim3(grid), dim3(kFewThreads), smem, stream, a.x, (int)a.T, a.H,
                     a.ld, a.logits, a.E, a.k, a.renormalize, static_cast<const uint8_t*>(a.w13),
                     static_cast<const uint8_t*>(a.s13), a.I, a.ids, a.w, a.workspace);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const size_t smem2 = (size_t)kFewWaves * a.T * 16 * sizeof(float);
  hipLaunchKernelGGL((few_down_kernel<kForm>), dim3((unsigned)(a.H >> 4)), dim3(kFewThreads), smem2, stream, (int)a.T,
                     a.H, a.k, static_cast<const uint8_t*>(a.w2), static_cast<const uint8_t*>(a.s2), a.I,
                     a.workspace, a.y, a.y_bf16);
  return hipGetLastError();
}

template <int kForm, int GW>
static hipError_t launch_few_experts(const FewArgs& a, hipStream_t stream) {
  if (a.E <= 256) return launch_few_form<kForm, GW, 4>(a, stream);
  return launch_few_form<kForm, GW, kRouteSlots>(a, stream);
}

template <int kForm>
static hipError_t launch_few_groups(const FewArgs& a, hipStream_t stream) {
  const int64_t gpw = (a.H / kGroup + kFewWaves - 1) / kFewWaves;
  if (gpw <= 2) return launch_few_experts<kForm, 2>(a, stream);
  if (gpw <= 4) return launch_few_experts<kForm, 4>(a, stream);
  if (gpw <= 6) return launch_few_experts<kForm, 6>(a, stream);
  return launch_few_experts<kForm, 8>(a, stream);
}

hipError_t launch_few(const FewArgs& a, hipStream_t stream) {
  if (a.form == kFormMx) return launch_few_groups<kFormMx>(a, stream);
  if (a.form == kFormChannel) return launch_few_groups<kFormChannel>(a, stream);
  return launch_few_groups<kFormG128>(a, stream);
}

}  // namespace w4a8
