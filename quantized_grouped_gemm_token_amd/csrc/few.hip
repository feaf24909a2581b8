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
// every fp32 magnitude up to 448); quotients a rounding above 448 are clamped.
template <bool kInt8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s, float r) {
  const float v[4] = {div_by(a, s, r), div_by(b, s, r), div_by(c, s, r), div_by(d, s, r)};
  if constexpr (kInt8) {
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o |= ((uint32_t)(int)fminf(fmaxf(rintf(v[i]), -127.0f), 127.0f) & 0xffu) << (8 * i);
    return o;
  } else {
    float u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = fminf(fmaxf(v[i], -kFp8Max), kFp8Max);
    int o = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], o, true);
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

// The k experts of a logits row and their weights, with the order, ties and sums of
// w4a8_moe_route (the same bits): slot s of lane l is expert l + 64 s.  Every id
// written is in [0, E), whatever the logits hold.
template <int S>
__device__ __forceinline__ void route_token(const float* __restrict__ lr, int E, int k, int renormalize, int* ids,
                                            float* w) {
  const int lane = threadIdx.x & 63;
  float v[S];
  uint32_t key[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = lane + s * kWave;
    v[s] = e < E ? lr[e] : 0.0f;
    key[s] = e < E ? order_key(v[s]) : 0u;
  }
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

__device__ __forceinline__ void route_any(const float* __restrict__ lr, int E, int k, int renormalize, int* ids,
                                          float* w) {
  if (E <= 64) route_token<1>(lr, E, k, renormalize, ids, w);
  else if (E <= 128) route_token<2>(lr, E, k, renormalize, ids, w);
  else if (E <= 256) route_token<4>(lr, E, k, renormalize, ids, w);
  else if (E <= 512) route_token<8>(lr, E, k, renormalize, ids, w);
  else route_token<16>(lr, E, k, renormalize, ids, w);
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
  __device__ __forceinline__ void set_a(v8i a) {
    if constexpr (kInt8) {
      ai = a;
      const i32x4 m = {(int)0xf8f8f8f8, (int)0xf8f8f8f8, (int)0xf8f8f8f8, (int)0xf8f8f8f8};   // -8
      bias = mfma_i8_16x16x64(a.hi, m, mfma_i8_16x16x64(a.lo, m, i32x4{0, 0, 0, 0}));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) ab[c] = e4m3x8_to_bf16((uint32_t)a[2 * c], (uint32_t)a[2 * c + 1], 1.0f);
      if constexpr (kForm == kFormG128) bias = minus8_product(ab);
      else bias = Acc{0, 0, 0, 0};
    }
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
// w13, K split over the 8 waves.  The grid walks the tasks; a wave has all of a
// task's loads in flight, and issues the next task's as it uses them up.
// GW: the most K groups of a wave (H <= 1024 GW).
template <int kForm, int GW>
__global__ __launch_bounds__(kFewThreads) void few_gate_up_kernel(const uint16_t* __restrict__ x, int T, int64_t H,
                                                                  int64_t ld, const float* __restrict__ logits, int E,
                                                                  int k, int renormalize,
                                                                  const uint8_t* __restrict__ w13,
                                                                  const uint32_t* __restrict__ s13, int64_t I,
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
  __shared__ int distinct, wave_firsts[kFewWaves];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int G = (int)(H >> 7), R = T * k;
  uint8_t* codes = smem;                                          // [G][4][T][32]
  float* red = reinterpret_cast<float*>(smem + (size_t)T * H);    // [2][waves][2][T][16]; int32 for INT8
  int* first = reinterpret_cast<int*>(red);                       // [max(E, R)], before red is used

  // row maxima of x: the waves share the rows, wpr waves to a row
  const int wpr = T == 1 ? 8 : T == 2 ? 4 : T <= 4 ? 2 : 1;       // waves per row
  const int rows_at_once = kFewWaves / wpr;
  const int part = wave % wpr;
  const int chunks = (int)(H >> 3);
  for (int t0 = 0; t0 < T; t0 += rows_at_once) {
    const int t = t0 + wave / wpr;
    if (t < T) {
      const uint4* xr = reinterpret_cast<const uint4*>(x + (int64_t)t * ld);
      float amax = 0.0f;
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
  for (int t = wave; t < T; t += kFewWaves)
    route_any(logits + (int64_t)t * E, E, k, renormalize, ids + t * k, wts + t * k);
  for (int e = threadIdx.x; e < E; e += kFewThreads) first[e] = 0x7fffffff;
  for (int i = threadIdx.x; i < R * kFewMaxTokens / 2; i += kFewThreads) reinterpret_cast<int*>(slot)[i] = -1;
  __syncthreads();

  // the distinct experts in the order of their first routed index
  const int f = threadIdx.x;                                      // R <= 256 < 512 threads
  if (f < R) atomicMin(&first[ids[f]], f);
  __syncthreads();
  const bool is_first = f < R && first[ids[f]] == f;
  const uint64_t ball = __ballot(is_first);
  if (lane == 0) wave_firsts[wave] = __builtin_popcountll(ball);
  __syncthreads();
  int before = __builtin_popcountll(ball & ((1ull << lane) - 1)), all = 0;
#pragma unroll
  for (int v = 0; v < kFewWaves; ++v) {
    before += v < wave ? wave_firsts[v] : 0;
    all += wave_firsts[v];
  }
  int my_first = 0;
  if (f < R) my_first = first[ids[f]];
  __syncthreads();                                                // first[] read by everyone: reuse it as index of f
  if (is_first) {
    experts[before] = ids[f];
    first[f] = before;                                            // position of the expert first seen at f
  }
  if (threadIdx.x == 0) distinct = all;
  __syncthreads();
  if (f < R) slot[first[my_first]][f / k] = (int16_t)f;
  if (blockIdx.x == 0) {
    const FewWorkspace ws = few_workspace(workspace, R, I);
    if (f == 0) *ws.count = all;
    if (f < all) ws.experts[f] = experts[f];
    if (f < R) {
      ws.weights[f] = wts[f];
      if (ids_out) ids_out[f] = ids[f];
      if (w_out) w_out[f] = wts[f];
    }
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
  const int D = distinct;
  if (blockIdx.x == 0) {
    const FewWorkspace ws = few_workspace(workspace, R, I);
    for (int i = threadIdx.x; i < D * kFewMaxTokens / 2; i += kFewThreads)
      reinterpret_cast<int*>(ws.slot)[i] = reinterpret_cast<const int*>(slot)[i];
  }

  const FewWorkspace ws = few_workspace(workspace, R, I);
  const int blocks = (int)(I >> 4);                               // column blocks of act
  const int ntasks = D * blocks;
  const int gpw = (G + kFewWaves - 1) / kFewWaves;                // <= GW
  const int g0 = wave * gpw, ng = max(0, min(gpw, G - g0));
  const uint8_t* arow = codes + ((size_t)(4 * g0 + kq) * T + min(col, T - 1)) * 32;
  const size_t astep = (size_t)128 * T;

  i32x4 wg[GW], wu[GW];
  uint32_t sg[GW], su[GW];
  const uint8_t *pg = nullptr, *pu = nullptr;
  const uint32_t* ps = nullptr;
  auto point = [&](int task) {                                    // the task's weights of this wave
    const int d = task / blocks, cb = task - d * blocks;
    const int64_t e = experts[d];
    pg = w13 + ((e * (I >> 3) + cb) * G + g0) * 1024 + col * 64 + kq * 16;
    pu = pg + (I >> 4) * G * 1024;
    if constexpr (!kInt8) ps = s13 + (e * G + g0) * 2 * I + 16 * cb + col;
  };
  auto load = [&](int i) {
    wg[i] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pg + i * 1024));
    wu[i] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pu + i * 1024));
    if constexpr (!kInt8) {
      sg[i] = ps[(int64_t)i * 2 * I];
      su[i] = ps[(int64_t)i * 2 * I + I];
    }
  };
  // this thread's token scale (threads below 16 T finish the tiles: token threadIdx.x / 16)
  float sx = 1.0f;
  if ((int)threadIdx.x < 16 * T) {
    float amax = 0.0f;
    for (int p = 0; p < wpr; ++p) amax = fmaxf(amax, wave_amax[threadIdx.x >> 4][p]);
    sx = row_scale<kInt8>(amax);
  }
  int task = blockIdx.x, buf = 0;
  if (task < ntasks) {
    point(task);
#pragma unroll
    for (int i = 0; i < GW; ++i)
      if (i < ng) load(i);
  }
  for (; task < ntasks; task += gridDim.x, buf ^= 1) {
    const bool more = task + (int)gridDim.x < ntasks;
    if (more) point(task + gridDim.x);
    Acc ag = Acc{0, 0, 0, 0}, au = Acc{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < GW; ++i) {
      if (i < ng) {
        P p;
        p.set_a(*reinterpret_cast<const v8i*>(arow + i * astep));
        uint32_t fg = 0, fu = 0;
        if constexpr (!kInt8) {
          fg = kForm == kFormMx ? (sg[i] >> (8 * kq)) & 0xffu : sg[i];
          fu = kForm == kFormMx ? (su[i] >> (8 * kq)) & 0xffu : su[i];
        }
        p.add(wg[i], fg, ag);
        p.add(wu[i], fu, au);
        if (more) load(i);
      }
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
// expert, 4-group K chunk) pieces in turn: each requantizes its routed tokens' act
// of those K elements into LDS of its own, multiplies, and adds the result to its
// 16x16 tile of y with the factor w[t, j] sa[f] of each routed token.
template <int kForm>
__global__ __launch_bounds__(kFewThreads) void few_down_kernel(int T, int64_t H, int k, const uint8_t* __restrict__ w2,
                                                               const uint32_t* __restrict__ s2, int64_t I,
                                                               const void* __restrict__ workspace,
                                                               void* __restrict__ y, int y_bf16) {
  using P = FewProduct<kForm>;
  using Acc = typename P::Acc;
  constexpr bool kInt8 = P::kInt8;
  constexpr int CG = kFewDownGroups;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];   // [waves][CG][4][T][32], then [waves][T][16] floats
  __shared__ float scale[kFewMaxRows], factor[kFewMaxRows];              // sa[f], w[f] sa[f]
  __shared__ __attribute__((aligned(16))) int16_t slot[kFewMaxRows][kFewMaxTokens];
  __shared__ int experts[kFewMaxRows];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int G = (int)(I >> 7), R = T * k;
  const int64_t cb = blockIdx.x;
  const FewWorkspace ws = few_workspace(const_cast<void*>(workspace), R, I);
  const int D = *ws.count;
  for (int i = threadIdx.x; i < D; i += kFewThreads) experts[i] = ws.experts[i];
  for (int i = threadIdx.x; i < D * kFewMaxTokens / 2; i += kFewThreads)
    reinterpret_cast<int*>(slot)[i] = reinterpret_cast<const int*>(ws.slot)[i];
  const int blocks = (int)(I >> 4);
  for (int f = wave; f < R; f += kFewWaves) {                     // the row maxima
    float m = 0.0f;
    for (int b = lane; b < blocks; b += 64) m = fmaxf(m, ws.pmax[(int64_t)f * blocks + b]);
    m = wave_max(m);
    if (lane == 0) {
      const float sa = row_scale<kInt8>(m);
      scale[f] = sa;
      factor[f] = ws.weights[f] * sa;
    }
  }
  __syncthreads();

  const int nch = (G + CG - 1) / CG;                              // K chunks of an expert
  const int items = D * nch;
  uint8_t* mine = smem + (size_t)wave * CG * 128 * T;             // this wave's codes
  const uint8_t* arow = mine + ((size_t)kq * T + min(col, T - 1)) * 32;

  i32x4 w[CG], wn[CG];
  uint32_t s[CG], sn[CG];
  auto load = [&](int it, i32x4 (&wv)[CG], uint32_t (&sv)[CG]) {
    const int d = it / nch, g0 = (it - d * nch) * CG;
    const int64_t e = experts[d];
    const uint8_t* p = w2 + ((e * (H >> 4) + cb) * G + g0) * 1024 + col * 64 + kq * 16;
    const uint32_t* ps = s2 + (e * G + g0) * H + 16 * cb + col;
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      if (g0 + i < G) {
        wv[i] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(p + i * 1024));
        if constexpr (!kInt8) sv[i] = ps[(int64_t)i * H];
      }
    }
  };
  v4f yacc = {0.f, 0.f, 0.f, 0.f};
  if (wave < items) load(wave, w, s);
  for (int it = wave; it < items; it += kFewWaves) {
    const int d = it / nch, g0 = (it - d * nch) * CG, ng = min(CG, G - g0);
    if (it + kFewWaves < items) load(it + kFewWaves, wn, sn);
    for (int t = 0; t < T; ++t) {
      const int f = __builtin_amdgcn_readfirstlane((int)slot[d][t]);
      if (f < 0) continue;
      const float sc = scale[f], rc = 1.0f / sc;
      const float4* ar = reinterpret_cast<const float4*>(ws.act + (int64_t)f * I + (int64_t)g0 * kGroup);
      for (int q = lane; q < ng * 32; q += 64) {                  // 4 elements each: group q / 32, lane group (q / 8) % 4
        const float4 v = ar[q];
        *reinterpret_cast<uint32_t*>(mine + ((size_t)(q >> 3) * T + t) * 32 + 4 * (q & 7)) =
            codes4<kInt8>(v.x, v.y, v.z, v.w, sc, rc);
      }
    }
    wave_lds_fence();
    Acc acc = Acc{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      if (i < ng) {
        P p;
        p.set_a(*reinterpret_cast<const v8i*>(arow + (size_t)i * 128 * T));
        uint32_t fs = 0;
        if constexpr (!kInt8) fs = kForm == kFormMx ? (s[i] >> (8 * kq)) & 0xffu : s[i];
        p.add(w[i], fs, acc);
      }
    }
    float ws_n = 1.0f;
    if constexpr (kInt8) ws_n = reinterpret_cast<const float*>(s2)[(int64_t)experts[d] * H + 16 * cb + col];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 4 * kq + r;
      const int f = t < T ? (int)slot[d][t] : -1;
      // a token that did not pick the expert multiplied whatever the LDS held: dropped here
      if (f >= 0) yacc[r] = fmaf(factor[f], kInt8 ? (float)acc[r] * ws_n : (float)acc[r], yacc[r]);
    }
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      w[i] = wn[i];
      s[i] = sn[i];
    }
  }
  __syncthreads();                                                // the codes are done with: reuse the LDS
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (4 * kq + r < T) red[((size_t)wave * T + 4 * kq + r) * 16 + col] = yacc[r];
  __syncthreads();
  if ((int)threadIdx.x < 16 * T) {
    const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < kFewWaves; ++v) sum += red[((size_t)v * T + t) * 16 + c];
    if (y_bf16) static_cast<uint16_t*>(y)[(int64_t)t * H + 16 * cb + c] = __builtin_bit_cast(uint16_t, (__bf16)sum);
    else static_cast<float*>(y)[(int64_t)t * H + 16 * cb + c] = sum;
  }
}

// ---- launches ------------------------------------------------------------------
template <int kForm, int GW>
static hipError_t launch_few_form(const FewArgs& a, hipStream_t stream) {
  const int64_t R = a.T * a.k;
  const int64_t tasks = (R < a.E ? R : (int64_t)a.E) * (a.I >> 4);       // at most
  const unsigned grid = (unsigned)(tasks < 512 ? tasks : 512);
  const size_t smem = (size_t)few_gate_up_smem(a.T, a.H);
  hipLaunchKernelGGL((few_gate_up_kernel<kForm, GW>), dim3(grid), dim3(kFewThreads), smem, stream, a.x, (int)a.T, a.H,
                     a.ld, a.logits, a.E, a.k, a.renormalize, static_cast<const uint8_t*>(a.w13),
                     static_cast<const uint32_t*>(a.s13), a.I, a.ids, a.w, a.workspace);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const size_t smem2 = (size_t)kFewWaves * kFewDownGroups * 128 * a.T;
  hipLaunchKernelGGL((few_down_kernel<kForm>), dim3((unsigned)(a.H >> 4)), dim3(kFewThreads), smem2, stream, (int)a.T,
                     a.H, a.k, static_cast<const uint8_t*>(a.w2), static_cast<const uint32_t*>(a.s2), a.I,
                     a.workspace, a.y, a.y_bf16);
  return hipGetLastError();
}

template <int kForm>
static hipError_t launch_few_groups(const FewArgs& a, hipStream_t stream) {
  const int64_t gpw = (a.H / kGroup + kFewWaves - 1) / kFewWaves;
  if (gpw <= 1) return launch_few_form<kForm, 1>(a, stream);
  if (gpw <= 2) return launch_few_form<kForm, 2>(a, stream);
  if (gpw <= 4) return launch_few_form<kForm, 4>(a, stream);
  if (gpw <= 6) return launch_few_form<kForm, 6>(a, stream);
  return launch_few_form<kForm, 8>(a, stream);
}

hipError_t launch_few(const FewArgs& a, hipStream_t stream) {
  if (a.form == kFormMx) return launch_few_groups<kFormMx>(a, stream);
  if (a.form == kFormChannel) return launch_few_groups<kFormChannel>(a, stream);
  return launch_few_groups<kFormG128>(a, stream);
}

}  // namespace w4a8
