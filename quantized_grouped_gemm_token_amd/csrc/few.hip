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
//
// Measured (H 6144, I 2048, 256 experts, 8 picks; kernel times, weights and scales read):
//             gate/up                  down
//   1 token   23.6 us (107 MB, 4.5 TB/s)  16.0 us (54 MB, 3.3 TB/s)   group 128
//   4 tokens  70 us (408 MB, 5.8 TB/s)    40 us (204 MB, 5.1 TB/s)    MXFP4
//   16 tokens 226 us (1.36 GB, 6.0 TB/s)  131 us (0.68 GB, 5.2 TB/s)  group 128
// against about 6.5 TB/s that a long read reaches.  With one token the start bounds both
// (launch; logits and x, then the picks one after the other, then the first weights; count,
// act, then weights): a layer with next to no bytes takes 9.3 and 8.7 us (16 tokens, 8
// experts of I 128).
#include "kernels.hpp"
#include "row_codes.hpp"
#include "w4_bf16.hpp"

#include <type_traits>

namespace w4a8 {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = 64 * kFewWaves;

// ---- routing of one token by one wave ---------------------------------------
// fp32 -> uint32 with the order of the values (-0 as +0); NaN is below -infinity, 0 below both
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return v == v ? k : 1u;
}
// The key of -infinity.  An expert whose key is not above it is masked: it can be picked (where fewer
// than k are not masked), with weight 0, and is not routed, as in the separate steps, so nothing of
// it reaches y.
constexpr uint32_t kMaskedKey = 0x007fffffu;
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

// The k experts of a logits row in descending order, equal logits by the lower expert
// (the order of w4a8_moe_route): slot s of lane l is expert l + 64 s, v its logit.  Every
// id written is in [0, E), whatever the logits hold.  keys: the picks' order keys;
// picked: a bit for each expert that is routed to.  A round is one DPP maximum of the wave, then the
// lowest slot and lane that hold it; picks stay in registers (lane j holds pick j) and
// reach LDS 64 at a time.
template <int S>
__device__ __forceinline__ void pick_experts(const float (&v)[kRouteSlots], int E, int k, int* ids, uint32_t* keys,
                                             uint32_t* picked) {
  const int lane = threadIdx.x & 63;
  uint32_t key[S];
#pragma unroll
  for (int s = 0; s < S; ++s) key[s] = lane + s * kWave < E ? order_key(v[s]) : 0u;
  for (int j0 = 0; j0 < k; j0 += kWave) {
    int my_id = 0;
    uint32_t my_key = 0u;
    const int n = min(k - j0, kWave);
    for (int j = 0; j < n; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int s = 1; s < S; ++s) best = max(best, key[s]);
      best = wave_max_key(best);
      int id = 0;
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        const uint64_t hit = __ballot(key[s] == best);
        id = hit ? s * kWave + __builtin_ctzll(hit) : id;
      }
#pragma unroll
      for (int s = 0; s < S; ++s) key[s] = lane + s * kWave == id ? 0u : key[s];
      my_id = lane == j ? id : my_id;
      my_key = lane == j ? best : my_key;
    }
    if (lane < n) {
      ids[j0 + lane] = my_id;
      keys[j0 + lane] = my_key;
      if (my_key > kMaskedKey) atomicOr(&picked[my_id >> 5], 1u << (my_id & 31));
    }
  }
}

// The routing weights of one row from its picks' logits, by one wave, with the sums of
// w4a8_moe_route (the same bits); 0 for a masked expert.  lr: the logits row.
__device__ __forceinline__ void route_weights(const uint32_t* keys, const float* __restrict__ lr, int E, int k,
                                              int renormalize, float* __restrict__ w, float* __restrict__ w_out) {
  const int lane = threadIdx.x & 63;
  const float m = key_value(keys[0]);
  float denom = 0.0f;
  if (renormalize) {
    for (int j = lane; j < k; j += kWave) denom += keys[j] > kMaskedKey ? expf(key_value(keys[j]) - m) : 0.0f;
  } else {
    for (int e = lane; e < E; e += kWave) denom += expf(lr[e] - m);
  }
  denom = wave_sum(denom);
  for (int j = lane; j < k; j += kWave) {
    const float p = keys[j] > kMaskedKey ? expf(key_value(keys[j]) - m) / denom : 0.0f;
    w[j] = p;
    if (w_out) w_out[j] = p;
  }
}

// ---- what the first kernel leaves for the second ------------------------------
// Views into the caller's workspace (16-byte aligned): the number of distinct experts (0: every
// logit is masked); of each, the expert (10 bits), the routed indices of its first two tokens (8 bits each; one:
// the second counts nothing) and the set of its tokens; the routed index of (expert, token)
// or -1; the routing weights, act [R][I] and the maxima of |act| over its 16-column blocks
// [R][I/16]; then what the second kernel's workgroups leave for each other: their sums of a
// column block that they share, [workgroup][2][T][32], and a count of arrivals for each of
// the H/32 column blocks (set to zero by the first kernel).
struct FewWorkspace {
  int32_t* count;
  uint32_t* experts;      // [kFewMaxRows] expert | first routed index << 10 | second << 18
  uint32_t* tokens;       // [kFewMaxRows] bit t: token t picked the expert
  int16_t* slot;          // [kFewMaxRows][16]
  float* weights;         // [kFewMaxRows]
  float* act;
  float* pmax;
  float* partial;
  uint32_t* arrived;
};
__device__ __forceinline__ FewWorkspace few_workspace(void* p, int64_t T, int64_t R, int64_t I) {
  unsigned char* b = static_cast<unsigned char*>(p);
  FewWorkspace v;
  v.count = reinterpret_cast<int32_t*>(b);
  v.experts = reinterpret_cast<uint32_t*>(b + 16);
  v.weights = reinterpret_cast<float*>(b + 16 + 4 * kFewMaxRows);
  v.tokens = reinterpret_cast<uint32_t*>(b + 16 + 8 * kFewMaxRows);
  v.slot = reinterpret_cast<int16_t*>(b + 16 + 12 * kFewMaxRows);
  v.act = reinterpret_cast<float*>(b + kFewHeadBytes);
  v.pmax = v.act + R * I;
  v.partial = v.pmax + R * (I >> 4);
  v.arrived = reinterpret_cast<uint32_t*>(v.partial + kFewDownMaxGrid * 2 * T * 32);
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
// A task is 16 NC columns of act for one distinct expert: NC tiles of 16 gate rows of w13
// and NC of up rows, K split over the 8 waves.  The workgroups walk the tasks; a wave
// refills each weight register with the next task's as it uses it up.
// NC = 2 uses an operand and its -8 products four times, and reads whole lines of scales,
// but the first product waits for twice the weights and the last ends later.
// GW: the most K groups of a wave (H <= 1024 GW).  S: logits per lane (E <= 64 S).
template <int kForm, int GW, int S, int NC>
__global__ __launch_bounds__(kFewThreads, 2) void few_gate_up_kernel(const uint16_t* __restrict__ x, int T, int64_t H,
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
  __shared__ uint32_t keys[kFewMaxRows];
  __shared__ int experts[kFewMaxRows];
  __shared__ __attribute__((aligned(16))) int16_t slot[kFewMaxRows][kFewMaxTokens];
  __shared__ float wave_amax[kFewMaxTokens][kFewWaves];
  __shared__ uint32_t picked[32];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int G = (int)(H >> 7), R = T * k;
  uint8_t* codes = smem;                                          // [G][4][2][T][16]
  float* red = reinterpret_cast<float*>(smem + (size_t)T * H);    // NC = 1: [2][waves][gate, up][T][16], NC = 2: [waves][gate, up][T][32]; int32 for INT8

  // The waves share the first 8 rows of x, wpr waves to a row, and wave v takes row v + 8.
  // A part of a row that is short enough stays in registers until the weights are on
  // their way (up to 4 tokens, or rows of 2048); the others are read twice before that.
  const int wpr = T == 1 ? 8 : T == 2 ? 4 : T <= 4 ? 2 : 1;       // waves per row
  const int part = wave % wpr, row = wave / wpr;
  const int chunks = (int)(H >> 3);                               // of 8 elements
  constexpr int XC = GW <= 2 ? 2 * GW : GW;                       // chunks per lane held; a whole row has 2 GW
  const bool has_row = row < T && (GW <= 2 || wpr > 1);
  const bool routes = wave < T, routes2 = wave + 8 < T;           // wave v routes rows v and v + 8
  float lg[kRouteSlots], lg2[kRouteSlots];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = lane + s * kWave;
    lg[s] = routes && e < E ? logits[(int64_t)wave * E + e] : 0.0f;
    lg2[s] = routes2 && e < E ? logits[(int64_t)(wave + 8) * E + e] : 0.0f;
  }
  const __amdgpu_buffer_rsrc_t rx = buffer_of(x + (int64_t)(has_row ? row : 0) * ld, has_row ? chunks * 16 : 0);
  uint4 xv[XC];
#pragma unroll
  for (int i = 0; i < XC; ++i)                                    // past the row: zeros, which count nothing in the maximum
    xv[i] = __builtin_bit_cast(uint4, buffer_load16(rx, (part * 64 + lane + 64 * wpr * i) * 16));
  uint4 xv2[GW <= 2 ? XC : 1];                                    // row v + 8, where rows are short
  if constexpr (GW <= 2) {
    const __amdgpu_buffer_rsrc_t rx2 = buffer_of(x + (int64_t)(routes2 ? wave + 8 : 0) * ld, routes2 ? chunks * 16 : 0);
#pragma unroll
    for (int i = 0; i < XC; ++i) xv2[i] = __builtin_bit_cast(uint4, buffer_load16(rx2, (lane + 64 * i) * 16));
  }
  if (threadIdx.x < 32) picked[threadIdx.x] = 0u;
  for (int i = threadIdx.x; i < R * kFewMaxTokens / 2; i += kFewThreads) reinterpret_cast<int*>(slot)[i] = -1;
  auto amax8 = [](float m, uint4 v) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(u[i])), fabsf(bf16_hi(u[i]))));
    return m;
  };
  // the codes of chunk c of row t, in operand order: elements 8 c .. +7 are group c / 16, lane group
  // (c / 4) % 4, bytes 8 (c % 4) .. +7 of its 32, which are kept in two halves (16 lanes then read 256
  // bytes side by side)
  auto times2 = [](uint32_t v, float by) {                        // both bf16 of a word times a power of two (exact)
    return (__float_as_uint(bf16_hi(v) * by) & 0xffff0000u) | __float_as_uint(bf16_lo(v) * by) >> 16;
  };
  auto put_codes = [&](uint4 v, int c, int t, RowDivisor d) {
    if (rescaled(d.by)) v = make_uint4(times2(v.x, d.by), times2(v.y, d.by), times2(v.z, d.by), times2(v.w, d.by));
    uint2 o;
    o.x = codes4<kInt8>(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), d.s, d.r);
    o.y = codes4<kInt8>(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), d.s, d.r);
    *reinterpret_cast<uint2*>(codes + ((size_t)(c >> 1) * T + t) * 16 + 8 * (c & 1)) = o;
  };
  __syncthreads();                                                // picked and slot are set
  if (routes) pick_experts<S>(lg, E, k, ids + wave * k, keys + wave * k, picked);
  auto quantize_row = [&](int t) {
    const __amdgpu_buffer_rsrc_t rt = buffer_of(x + (int64_t)t * ld, chunks * 16);
    float m = 0.0f;
    for (int c = lane; c < chunks; c += 256) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint4, buffer_load16(rt, (c + 64 * i) * 16));
#pragma unroll
      for (int i = 0; i < 4; ++i) m = amax8(m, v[i]);
    }
    m = wave_max(m);
    if (lane == 0) wave_amax[t][0] = m;
    const RowDivisor d = row_divisor(row_scale<kInt8>(m));
    for (int c = lane; c < chunks; c += 256) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint4, buffer_load16(rt, (c + 64 * i) * 16));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + 64 * i < chunks) put_codes(v[i], c + 64 * i, t, d);
    }
  };
  if (GW > 2 && wpr == 1 && wave < T) quantize_row(wave);
  if (routes2) {
    pick_experts<S>(lg2, E, k, ids + (wave + 8) * k, keys + (wave + 8) * k, picked);
    if constexpr (GW <= 2) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < XC; ++i) m = amax8(m, xv2[i]);
      m = wave_max(m);
      if (lane == 0) wave_amax[wave + 8][0] = m;
      const RowDivisor d = row_divisor(row_scale<kInt8>(m));
#pragma unroll
      for (int i = 0; i < XC; ++i)
        if (lane + 64 * i < chunks) put_codes(xv2[i], lane + 64 * i, wave + 8, d);
    } else {
      quantize_row(wave + 8);
    }
  }
  __syncthreads();                                                // ids and picked are there

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
    if (f < R && keys[f] > kMaskedKey) {
      slot[number][f / k] = (int16_t)f;
      experts[number] = e;                                        // the same value from every token that picked it
    }
  }
  __syncthreads();

  const FewWorkspace ws = few_workspace(workspace, T, R, I);
  constexpr int kCols = 16 * NC, NT = 2 * NC;                     // tiles: gate, then up
  const int blocks = (int)(I / kCols);                            // column blocks of act
  const int ntasks = D * blocks;
  const int gpw = (G + kFewWaves - 1) / kFewWaves;                // <= GW
  const int g0 = wave * gpw, ng = max(0, min(gpw, G - g0));
  constexpr int SW = (GW + 3) / 4;                                // scale words: one for four groups
  i32x4 w[GW][NT];
  uint32_t sc[SW][NT];
  __amdgpu_buffer_rsrc_t rw[NT], rs;
  auto point = [&](int task) {                                    // the task's weights of this wave; none past the last task
    const bool on = task < ntasks && ng > 0;
    const int d = on ? task / blocks : 0, cb = on ? task - d * blocks : 0;
    const int64_t e = __builtin_amdgcn_readfirstlane(experts[d]);
    const uint8_t* p = w13 + ((e * (I >> 3) + NC * cb) * G + g0) * 1024;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      rw[n] = buffer_of(p + (n % NC + n / NC * (I >> 4)) * G * 1024, on ? ng * 1024 : 0);
    rs = buffer_of(s13 + (((e * G + g0) * 2 * I) + kCols * cb) * 4,
                   !kInt8 && on ? ((int64_t)ng * 2 * I - kCols * cb) * 4 : 0);
  };
  auto load = [&](int i) {
#pragma unroll
    for (int n = 0; n < NT; ++n) w[i][n] = buffer_load16_nt(rw[n], col * 64 + kq * 16 + i * 1024);
  };
  auto load_scales = [&](int j) {                                 // of the groups 4 j .. 4 j + 3; before their weights
    if constexpr (!kInt8) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        sc[j][n] = buffer_load4(rs, (uint32_t)((4 * j + kq) * 2 * I + n / NC * I + 16 * (n % NC) + col) * 4);
    }
  };
  int task = xcd_order(), buf = 0;
  point(task);
#pragma unroll
  for (int i = 0; i < GW; ++i) {
    if ((i & 3) == 0) load_scales(i >> 2);
    load(i);
  }

  {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < XC; ++i) m = amax8(m, xv[i]);
    m = wave_max(m);
    if (has_row && lane == 0) wave_amax[row][part] = m;           // (wave v's own row otherwise, below)
      // (opaque: the fp32 values of the maxima are not kept for the codes, they would take twice the registers)
#pragma unroll
    for (int i = 0; i < XC; ++i) asm volatile("" : "+v"(xv[i].x), "+v"(xv[i].y), "+v"(xv[i].z), "+v"(xv[i].w));
  }
  __syncthreads();                                                // the row maxima are there
  if (has_row) {                                                  // the codes of the rows in registers
    float m = 0.0f;
    for (int p = 0; p < wpr; ++p) m = fmaxf(m, wave_amax[row][p]);
    const RowDivisor d = row_divisor(row_scale<kInt8>(m));
#pragma unroll
    for (int i = 0; i < XC; ++i) {
      const int c = part * 64 + lane + 64 * wpr * i;
      if (c < chunks) put_codes(xv[i], c, row, d);
      __builtin_amdgcn_sched_barrier(0);                          // one chunk at a time: few values live
    }
  }
  if (blockIdx.x == 0) {                                          // the routing, for the second kernel and the caller
    for (int t = wave; t < T; t += kFewWaves)
      route_weights(keys + t * k, logits + (int64_t)t * E, E, k, renormalize, ws.weights + t * k,
                    w_out ? w_out + t * k : nullptr);
    if (f == 0) *ws.count = D;
    if (f < D) {
      uint32_t set = 0, fa = 0, fb = 0;
      for (int t = T - 1; t >= 0; --t) {
        const int v = slot[f][t];
        if (v >= 0) {
          set |= 1u << t;
          fb = fa;
          fa = (uint32_t)v;
        }
      }
      ws.experts[f] = (uint32_t)experts[f] | fa << 10 | fb << 18;
      ws.tokens[f] = set;
    }
    if (f < R && ids_out) ids_out[f] = ids[f];
    for (int i = threadIdx.x; i < D * kFewMaxTokens / 2; i += kFewThreads)
      reinterpret_cast<int*>(ws.slot)[i] = reinterpret_cast<const int*>(slot)[i];
    for (int i = threadIdx.x; i < (int)(H >> 5); i += kFewThreads) ws.arrived[i] = 0u;
  }
  __syncthreads();

  const uint8_t* arow = codes + ((size_t)(8 * g0 + 2 * kq) * T + min(col, T - 1)) * 16;
  const size_t astep = (size_t)128 * T;
  // this thread's token scale (threads below 16 NC T finish the tiles: token ft, column fc)
  const int ft = threadIdx.x / kCols, fc = threadIdx.x % kCols;
  float sx = 1.0f;
  if (ft < T) {
    float amax = 0.0f;
    for (int p = 0; p < wpr; ++p) amax = fmaxf(amax, wave_amax[ft][p]);
    sx = row_scale<kInt8>(amax);
  }
  for (; task < ntasks; task += gridDim.x, buf ^= 1) {
    point(task + (int)gridDim.x);
    Acc acc[NT] = {};
    uint32_t s4[NT][4];
#pragma unroll
    for (int i = 0; i < GW; ++i) {
      if (!kInt8 && (i & 3) == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) spread4(sc[i >> 2][n], s4[n]);
        load_scales(i >> 2);
      }
      if (i < ng) {
        P p;
        v8i a;
        a.lo = *reinterpret_cast<const i32x4*>(arow + i * astep);
        a.hi = *reinterpret_cast<const i32x4*>(arow + i * astep + 16 * T);
        p.set_codes(a);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t f = 0;
          if constexpr (!kInt8) f = kForm == kFormMx ? (s4[n][i & 3] >> (8 * kq)) & 0xffu : s4[n][i & 3];
          p.add(w[i][n], f, acc[n]);
        }
      }
      load(i);
    }
    // the partial tiles: one barrier per task where there are two buffers (the other's readers passed the last one)
    const size_t step = (size_t)T * kCols;                        // gate to up, up to the next wave's gate
    float* rb = red + (NC == 1 ? buf * kFewWaves * 2 * step : 0);
    if constexpr (NC > 1) __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 4 * kq + r;
      if (t < T) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float* at = rb + (wave * 2 + n / NC) * step + t * kCols + 16 * (n % NC) + col;
          if constexpr (kInt8) *at = __int_as_float(acc[n][r]);
          else *at = acc[n][r];
        }
      }
    }
    __syncthreads();
    if (ft < T) {
      const int d = task / blocks, cb = task - d * blocks;
      const int fr = slot[d][ft];
      float gate, up;
      const float* at = rb + (size_t)ft * kCols + fc;
      if constexpr (kInt8) {
        int ig = 0, iu = 0;
#pragma unroll
        for (int v = 0; v < kFewWaves; ++v) {
          ig += __float_as_int(at[2 * v * step]);
          iu += __float_as_int(at[(2 * v + 1) * step]);
        }
        const float* sw = reinterpret_cast<const float*>(s13) + (int64_t)experts[d] * 2 * I + kCols * cb + fc;
        gate = (float)ig * sx * sw[0];
        up = (float)iu * sx * sw[I];
      } else {
        gate = 0.0f;
        up = 0.0f;
#pragma unroll
        for (int v = 0; v < kFewWaves; ++v) {
          gate += at[2 * v * step];
          up += at[(2 * v + 1) * step];
        }
        gate *= sx;
        up *= sx;
      }
      const float a = silu_mul(gate, up);
      const float m = max16(fabsf(a));
      if (fr >= 0) {
        ws.act[(int64_t)fr * I + kCols * cb + fc] = a;
        if ((fc & 15) == 0) ws.pmax[(int64_t)fr * NC * blocks + NC * cb + (fc >> 4)] = m;
      }
    }
  }
}

// ---- kernel 2: requantization, down, the routing-weighted sum ----------------
// The work is a row of pieces: for each block of 16 NB columns of y, the (distinct expert, K
// chunk of up to 8 / NB groups) products that its columns sum; a piece is 8 KB of weights.
// The workgroups take equal ranges of that row, of whole rounds of their 8 waves (H/32
// blocks are rarely a multiple of the CUs), so a workgroup has pieces of at most two
// blocks.  It leaves its sums of a block that it shares in memory and counts itself on the
// block's counter; the one that arrives last adds them in workgroup order (the same bits
// whichever that is) and writes y.  Nothing waits on a counter.  Where that saves no more
// than a round, a workgroup takes a whole block (few_down_range).
//
// A wave takes pieces in turn: it requantizes the act of the expert's tokens over those K
// elements into LDS of its own, up to 4 tokens at a time as rows 0 to 3 of the A operand (an
// expert has one or two of the few tokens as a rule; for more than 4 the weights stay in
// registers), multiplies, and adds the rows with the factors w[t, j] sa[f] to its own sums
// in LDS.  The next piece's weights, and the act of its first two tokens, are loaded
// meanwhile.  The FP8 codes are held as the bf16 values they stand for, converted once per
// token and piece.
//
// NB = 2: codes, their operands and the -8 products serve two tiles, and the scales of a
// group are a whole line of memory (NB = 1 at H 6144: 17.1 against 16.0 us for 1 token).
// Whole blocks of 32 columns fill too few CUs where there are few of them: NB = 1 (H 2048, I
// 768, 8 MXFP4 experts: 128 blocks of 16 7.5 us, 64 of 32 8.5 us).  One workgroup of 8 waves
// on a CU, with the registers for it, reads no slower than two with half of them.
__device__ __forceinline__ void store_y(void* y, int y_bf16, int64_t at, float v) {
  if (y_bf16) static_cast<uint16_t*>(y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
  else static_cast<float*>(y)[at] = v;
}
template <int NB>
struct FewDownShape {
  static constexpr int kCols = 16 * NB;
  static constexpr int kGroups = 8 / NB;
};
// Pieces of a workgroup: total in all, M of a block.  A shared block costs about a round, so
// whole blocks where equal ranges save no more: 192 blocks of 32 pieces 16.0 against 16.6 us,
// 64 of 16 8.5 against 8.6; 64 of 28 to 32 (4 rounds or 1) 11.9 against 10.0.
__host__ __device__ inline int few_down_range(int total, int M) {
  const int per = (total + kFewDownMaxGrid * kFewWaves - 1) / (kFewDownMaxGrid * kFewWaves) * kFewWaves;
  return M <= per + kFewWaves ? M : per;
}
template <int kForm, int NB>
__global__ __launch_bounds__(kFewThreads, 2) void few_down_kernel(int T, int64_t H, int k,
                                                                  const uint8_t* __restrict__ w2,
                                                                  const uint8_t* __restrict__ s2, int64_t I,
                                                                  void* __restrict__ workspace, void* __restrict__ y,
                                                                  int y_bf16) {
  using P = FewProduct<kForm>;
  using Acc = typename P::Acc;
  constexpr bool kInt8 = P::kInt8;
  constexpr int W = kFewWaves;
  constexpr int CG = FewDownShape<NB>::kGroups;
  constexpr int kDownCols = FewDownShape<NB>::kCols;
  constexpr int kRows = 4;                                               // rows of A in use
  constexpr int SW = (CG + 3) / 4;                                       // scale words per lane and tile
  constexpr int kQuads = CG * kGroup / 4 / 64;                           // float4 of act per lane, token and piece
  // the wave's A rows: FP8 forms [CG][4 products][4 lane groups][rows][16 bytes], INT8 form [CG][4][rows][32 bytes]
  __shared__ __attribute__((aligned(16))) uint8_t a_sm[W][CG * kGroup * kRows * (kInt8 ? 1 : 2)];
  __shared__ int last_sm[2];
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];   // few_down_smem bytes

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  const int G = (int)(I >> 7), R = T * k, cols = (int)(H / kDownCols);
  float4* row_sm = reinterpret_cast<float4*>(smem);                      // [R] of routed index f: sa and 1 / sa to divide by, w sa, `by`
  int16_t(*slot)[kFewMaxTokens] = reinterpret_cast<int16_t(*)[kFewMaxTokens]>(row_sm + R);   // [R]
  uint32_t* experts = reinterpret_cast<uint32_t*>(slot + R);             // [R] as in the workspace
  uint32_t* routed = experts + R;                                        // [R] bit t: token t picked the expert
  float* y_sm = reinterpret_cast<float*>(routed + R);                    // [W][2 blocks][T][kDownCols]
  const int nch = (G + CG - 1) / CG, cg = (G + nch - 1) / nch;           // K chunks of an expert, groups of a chunk
  const FewWorkspace ws = few_workspace(workspace, T, R, I);

  // The block maxima of act, 16 lanes to a row: the first 2 float4 per lane of rows f0 + 4 W u
  // go out before the weights (the rest, for I > 2048 or R > 128, after them).
  const int quads = (int)(I >> 6);                                       // float4 of maxima per row
  const int f0 = threadIdx.x >> 4;
  auto pmax_at = [&](int f, int j) {
    return f < R && j < quads ? reinterpret_cast<const float4*>(ws.pmax)[(int64_t)f * quads + j]
                              : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 pm[4][2];
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int j = 0; j < 2; ++j) pm[u][j] = pmax_at(f0 + 4 * W * u, col + 16 * j);

  // every distinct expert's words, lane l holding numbers l, l + 64, ..: with the count they are one round trip to
  // memory before the first weights (words past the count are not used)
  uint32_t pe[kFewMaxRows / 64], pt[kFewMaxRows / 64];
#pragma unroll
  for (int i = 0; i < kFewMaxRows / 64; ++i) {
    pe[i] = lane + 64 * i < R ? ws.experts[lane + 64 * i] : 0u;
    pt[i] = lane + 64 * i < R ? ws.tokens[lane + 64 * i] : 0u;
  }

  // the workgroup's pieces: lo .. hi - 1 of block * M + (expert number * nch + chunk); those below
  // `second` are of block c0, the others of c0 + 1 (a range is at most M long)
  const int D = __builtin_amdgcn_readfirstlane(*ws.count);
  if (D == 0) {                                                          // nothing is routed: y is zero
    for (int i = (int)(blockIdx.x * kFewThreads + threadIdx.x); i < T * (int)H; i += (int)gridDim.x * kFewThreads)
      store_y(y, y_bf16, i, 0.0f);
    return;
  }
  const int M = D * nch, total = cols * M;
  const int per = NB == 1 ? M : few_down_range(total, M);                // pieces of a workgroup
  const int lo = (NB == 1 ? xcd_order() : (int)blockIdx.x) * per, hi = min(lo + per, total);
  if (lo >= total) return;
  const int c0 = lo / M, second = (c0 + 1) * M;

  // The weights of a piece, and the act of its first two tokens.  Loads past the last piece,
  // or of a token that is not there, read nothing.
  struct Piece {
    int d, g0, ng, block;  // ng = 0: none
    uint32_t tokens;       // bit t: token t picked the expert
    int fa, fb;            // routed indices of the first two, -1: none
  };
  i32x4 w[NB][CG];
  uint32_t s[NB][SW];
  float4 av[2][kQuads];
  __amdgpu_buffer_rsrc_t rw[NB], rs;
  auto piece_at = [&](int it) {
    Piece p;
    const bool on = it < hi;
    const int b = on && it >= second ? 1 : 0, m = on ? it - (c0 + b) * M : 0;
    p.block = b;
    p.d = m / nch;
    p.g0 = (m - p.d * nch) * cg;
    p.ng = on ? min(cg, G - p.g0) : 0;
    return p;
  };
  auto set_tokens = [&](Piece& p, uint32_t expert, uint32_t tokens) {
    p.tokens = tokens;
    p.fa = p.ng ? (int)(expert >> 10 & 0xffu) : -1;
    p.fb = p.ng && (tokens & (tokens - 1)) ? (int)(expert >> 18 & 0xffu) : -1;
  };
  auto point = [&](int64_t e, const Piece& p) {
    const int cb = c0 + p.block;
#pragma unroll
    for (int j = 0; j < NB; ++j)
      rw[j] = buffer_of(w2 + ((e * (H >> 4) + NB * cb + j) * G + p.g0) * 1024, p.ng * 1024);
    if constexpr (kInt8) rs = buffer_of(s2 + (e * H + kDownCols * cb) * 4, p.ng ? kDownCols * 4 : 0);
    else rs = buffer_of(s2 + ((e * G + p.g0) * H + kDownCols * cb) * 4, p.ng ? ((int)H * p.ng - kDownCols * cb) * 4 : 0);
  };
  auto load = [&](int i) {
#pragma unroll
    for (int j = 0; j < NB; ++j) w[j][i] = buffer_load16_nt(rw[j], col * 64 + kq * 16 + i * 1024);
  };
  // before the weights.  INT8 form: the scale of the column that the lane adds up (add_rows)
  auto load_scales = [&]() {
    if constexpr (kInt8) {
      s[0][0] = buffer_load4(rs, (lane & (kDownCols - 1)) * 4);
    } else {
#pragma unroll
      for (int m = 0; m < SW; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j) s[j][m] = buffer_load4(rs, (uint32_t)((4 * m + kq) * (int)H + 16 * j + col) * 4);
    }
  };
  auto load_act = [&](int a, int f, const Piece& p) {                    // f < 0: nothing
    const __amdgpu_buffer_rsrc_t ra = buffer_of(ws.act + (int64_t)max(f, 0) * I + p.g0 * kGroup,
                                                f >= 0 ? p.ng * kGroup * 4 : 0);
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
      av[a][q] = __builtin_bit_cast(float4, buffer_load16(ra, (lane + 64 * q) * 16));
  };
  // the first piece of the wave, from what the first kernel left in memory
  Piece cur = piece_at(lo + wave);
  {
    uint32_t e = 0, set = 0;
#pragma unroll
    for (int i = 0; i < kFewMaxRows / 64; ++i) {
      if (cur.d >> 6 == i) {
        e = (uint32_t)__builtin_amdgcn_readlane((int)pe[i], cur.d & 63);
        set = (uint32_t)__builtin_amdgcn_readlane((int)pt[i], cur.d & 63);
      }
    }
    set_tokens(cur, e, set);
    load_act(0, cur.fa, cur);
    load_act(1, cur.fb, cur);
    point(e & 0x3ffu, cur);
    load_scales();
#pragma unroll
    for (int i = 0; i < CG; ++i) load(i);
  }
  for (int fu = f0; fu < R; fu += 16 * W) {                              // the row scales
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int f = fu + 4 * W * u;
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) m = fmaxf(m, fmaxf(fmaxf(pm[u][j].x, pm[u][j].y), fmaxf(pm[u][j].z, pm[u][j].w)));
      for (int j = col + 32; j < quads; j += 16) {
        const float4 v = pmax_at(f, j);
        m = fmaxf(m, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
      }
      m = max16(m);
      if (col == 0 && f < R) {
        const float sa = row_scale<kInt8>(m);
        const RowDivisor d = row_divisor(sa);
        row_sm[f] = make_float4(d.s, d.r, ws.weights[f] * sa, d.by);
      }
    }
    if (fu + 16 * W < R) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) pm[u][j] = pmax_at(fu + 16 * W + 4 * W * u, col + 16 * j);
    }
  }
#pragma unroll
  for (int i = 0; i < kFewMaxRows / 64; ++i) {
    if (wave == i && lane + 64 * i < R) {
      experts[lane + 64 * i] = pe[i];
      routed[lane + 64 * i] = pt[i];
    }
  }
  for (int i = threadIdx.x; i < D * kFewMaxTokens / 2; i += kFewThreads)
    reinterpret_cast<int*>(slot)[i] = reinterpret_cast<const int*>(ws.slot)[i];
  for (int i = threadIdx.x; i < W * 2 * T * kDownCols; i += kFewThreads) y_sm[i] = 0.0f;
  __syncthreads();

  uint8_t* mine = a_sm[wave];
  // Where the lane's quad i of a piece goes, row 0: quad q = lane + 64 i holds the elements 4 (q % 8) .. +3 of
  // lane group (q / 8) % 4 of group q / 32 (past the piece's groups: zeros, which nothing reads)
  uint8_t* put_at = mine + (kInt8 ? (lane >> 3) * kRows * 32 + 4 * (lane & 7)
                                  : (((lane >> 5) * 4 + ((lane & 7) >> 1)) * 4 + ((lane >> 3) & 3)) * kRows * 16 + 8 * (lane & 1));
  constexpr int kPutStep = kInt8 ? 8 * kRows * 32 : 2 * 16 * kRows * 16;  // two groups on
  const int r0 = NB == 2 ? 2 * (lane >> 5) : kq;                         // see add_rows
  float fac[NB];                                                         // w sa of the rows r0 and (NB = 2) r0 + 1
  auto put = [&](int row, int a, int f) {                                // one token's codes of a piece, from av[a]
    const float4 r4 = row_sm[f];
    fac[row % NB] = row < NB || r0 == row / NB * NB ? r4.z : fac[row % NB];
    if (rescaled(r4.w)) {                                                // (a subnormal sa can be too small by half: clamped)
      const float top = (kInt8 ? 127.0f : kFp8Max) * r4.x;
      auto in = [&](float v) { return fminf(fmaxf(v * r4.w, -top), top); };
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
        av[a][i] = make_float4(in(av[a][i].x), in(av[a][i].y), in(av[a][i].z), in(av[a][i].w));
    }
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const uint32_t c4 = codes4<kInt8>(av[a][i].x, av[a][i].y, av[a][i].z, av[a][i].w, r4.x, r4.y);
      if constexpr (kInt8) {
        *reinterpret_cast<uint32_t*>(put_at + i * kPutStep + row * 32) = c4;
      } else {
        uint2 b;
        b.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c4, 1.0f, false));
        b.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c4, 1.0f, true));
        *reinterpret_cast<uint2*>(put_at + i * kPutStep + row * 16) = b;
      }
    }
  };
  uint32_t s4[NB][SW][4];
  auto product = [&](int i, Acc (&acc)[NB]) {                             // lane row col of A is row col % 4 of LDS
    P p;
    if constexpr (kInt8) {
      p.set_codes(*reinterpret_cast<const v8i*>(mine + ((i * 4 + kq) * kRows + (col & 3)) * 32));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        p.ab[c] = *reinterpret_cast<const i32x4*>(mine + (((i * 4 + c) * 4 + kq) * kRows + (col & 3)) * 16);
      p.set_bias();
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      uint32_t fs = 0;
      if constexpr (!kInt8) fs = kForm == kFormMx ? (s4[j][i >> 2][i & 3] >> (8 * kq)) & 0xffu : s4[j][i >> 2][i & 3];
      p.add(w[j][i], fs, acc[j]);
    }
  };
  // Rows 0 to 3 to the sums of the first four tokens of `set`.  A row stands in every lane group's tiles
  // (register r: row r).  NB = 2: lane group q takes tile q % 2 and the rows r0 = 2 (q / 2) and r0 + 1; NB = 1: row q.
  auto add_rows = [&](const Acc (&acc)[NB], uint32_t set) {
    const uint32_t set1 = set & (set - 1), set2 = set1 & (set1 - 1), set3 = set2 & (set2 - 1);
    float* base = y_sm + ((size_t)(wave * 2 + cur.block) * T) * kDownCols + (lane & (kDownCols - 1));
    auto add = [&](uint32_t from, float f, float v) {                    // to the lowest token of `from`
      if constexpr (kInt8) v *= __uint_as_float(s4[0][0][0]);
      if (from) {
        float* at = base + (__builtin_ctz(from | 0x80000000u) & 15) * kDownCols;
        *at = fmaf(f, v, *at);
      }
    };
    if constexpr (NB == 2) {
      const bool odd = kq & 1;
      const auto a0 = odd ? acc[1][0] : acc[0][0], a1 = odd ? acc[1][1] : acc[0][1];
      const auto a2 = odd ? acc[1][2] : acc[0][2], a3 = odd ? acc[1][3] : acc[0][3];
      add(r0 ? set2 : set, fac[0], (float)(r0 ? a2 : a0));
      add(r0 ? set3 : set1, fac[1], (float)(r0 ? a3 : a1));
    } else {
      const auto a01 = kq & 1 ? acc[0][1] : acc[0][0], a23 = kq & 1 ? acc[0][3] : acc[0][2];
      const uint32_t s01 = kq & 1 ? set1 : set, s23 = kq & 1 ? set3 : set2;
      add(kq & 2 ? s23 : s01, fac[0], (float)(kq & 2 ? a23 : a01));
    }
  };
  for (int it = lo + wave; it < hi; it += W) {
    if constexpr (kInt8) {
      s4[0][0][0] = s[0][0];
    } else {
#pragma unroll
      for (int m = 0; m < SW; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j) spread4(s[j][m], s4[j][m]);
    }
    uint32_t tokens = cur.tokens, next = tokens;                         // at least one bit
    int fa = cur.fa, fb = cur.fb;                                        // the tokens whose act av holds
    auto take = [&]() {                                                  // the routed index of the next token, -1: none
      const int f = next ? __builtin_amdgcn_readfirstlane((int)slot[cur.d][__builtin_ctz(next | 0x80000000u) & 15]) : -1;
      next &= next - 1;
      return f;
    };
    next &= next - 1;
    next &= next - 1;
    for (;;) {
      put(0, 0, fa);
      if (fb >= 0) put(1, 1, fb);
      if (next) {
        const int fc = take(), fd = take();
        load_act(0, fc, cur);
        load_act(1, fd, cur);
        put(2, 0, fc);
        if (fd >= 0) put(3, 1, fd);
      }
      wave_lds_fence();
      if (!next) break;
      // more than 4 tokens: the same weights again
      // (opaque here: hoisted out of the loop, the unpacked weights would take a third more registers)
#pragma unroll
      for (int i = 0; i < CG; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) asm volatile("" : "+v"(w[j][i]));
      const uint32_t rest = next;
      fa = take();
      fb = take();
      load_act(0, fa, cur);
      load_act(1, fb, cur);
      Acc acc[NB] = {};
#pragma unroll
      for (int i = 0; i < CG; ++i)
        if (i < cur.ng) product(i, acc);
      add_rows(acc, tokens);
      wave_lds_fence();
      tokens = rest;
    }
    const int ng = cur.ng;
    Piece nx = piece_at(it + W);
    {
      const uint32_t e = (uint32_t)__builtin_amdgcn_readfirstlane((int)experts[nx.d]);
      set_tokens(nx, e, (uint32_t)__builtin_amdgcn_readfirstlane((int)routed[nx.d]));
      load_act(0, nx.fa, nx);
      load_act(1, nx.fb, nx);
      point(e & 0x3ffu, nx);
    }
    load_scales();
    Acc acc[NB] = {};
#pragma unroll
    for (int i = 0; i < CG; ++i) {
      if (i < ng) product(i, acc);
      load(i);
    }
    add_rows(acc, tokens);
    wave_lds_fence();
    cur = nx;
  }
  __syncthreads();

  // The blocks' sums: a thread per (token, column) of each.
  const int t = threadIdx.x / kDownCols, c = threadIdx.x % kDownCols;
  if constexpr (NB == 1) {
    if (t < T) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < W; ++v) sum += y_sm[((size_t)(v * 2) * T + t) * kDownCols + c];
      store_y(y, y_bf16, (int64_t)t * H + kDownCols * c0 + c, sum);
    }
    return;
  }
  float sum[2] = {0.0f, 0.0f};
  bool here[2], whole[2], writes[2];                                     // the workgroup has some of the block, all of it
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    here[b] = b == 0 || hi > second;
    whole[b] = here[b] && lo <= second - M + b * M && hi >= second + b * M;
    writes[b] = t < T && whole[b];
    if (t < T && here[b]) {
#pragma unroll
      for (int v = 0; v < W; ++v) sum[b] += y_sm[((size_t)(v * 2 + b) * T + t) * kDownCols + c];
    }
  }
  if (!whole[0] || here[1]) {                                            // (the same for every thread) a block is shared
    // The sums go to and come from the point where all XCDs' caches meet (device-scope accesses, which no cache
    // holds back), so the order "sums, then the count" needs the stores to be done and no cache to be written
    // back or dropped: a device-scope fence in its place took 170 us of a 50 us launch.
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if (t < T && here[b] && !whole[b])
        __hip_atomic_store(&ws.partial[((int64_t)(blockIdx.x * 2 + b) * T + t) * kDownCols + c], sum[b], __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x < 2) {
      const int b = threadIdx.x, first = second - M + b * M;
      const bool shared = b ? here[1] && !whole[1] : !whole[0];
      // the workgroups with pieces of the block: first / per .. (first + M - 1) / per
      last_sm[b] = shared && __hip_atomic_fetch_add(&ws.arrived[c0 + b], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                                 (uint32_t)((first + M - 1) / per - first / per);
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (t < T && here[b] && !whole[b] && last_sm[b]) {
        const int first = second - M + b * M;
        writes[b] = true;
        sum[b] = 0.0f;
        for (int wg = first / per; wg <= (first + M - 1) / per; ++wg) {  // (the block is the second one of a range that starts before it)
          const int half = wg * per < first ? 1 : 0;
          sum[b] += __hip_atomic_load(&ws.partial[((int64_t)(wg * 2 + half) * T + t) * kDownCols + c], __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < 2; ++b)
    if (writes[b]) store_y(y, y_bf16, (int64_t)t * H + kDownCols * (c0 + b) + c, sum[b]);
}

// ---- launches ------------------------------------------------------------------
// Fewer whole blocks of 32 columns than this: blocks of 16 (see FewDownShape).
constexpr int64_t kFewMinBlocks = 128;

template <int kForm, int NB>
static void launch_few_down(const FewArgs& a, unsigned grid, hipStream_t stream) {
  const int64_t R = a.T * a.k;
  // dynamic LDS: per routed row its scales, slots, expert and token set, then the waves' sums
  const size_t smem = (size_t)(56 * R + kFewWaves * 2 * a.T * FewDownShape<NB>::kCols * 4);
  hipLaunchKernelGGL((few_down_kernel<kForm, NB>), dim3(grid), dim3(kFewThreads), smem, stream, (int)a.T, a.H, a.k,
                     static_cast<const uint8_t*>(a.w2), static_cast<const uint8_t*>(a.s2), a.I, a.workspace, a.y, a.y_bf16);
}

// One workgroup of the first kernel on each CU: two make the CU route and quantize twice.  Gate/up, 256
// against 512 workgroups: 1 token (H 6144, I 2048) 24.5 against 27.0 us, 8 tokens (H 4096, I 1024, 64
// experts) 28.5 against 32.4, 16 tokens 243 against 259; 4 tokens MXFP4 71.3 against 69.9.
constexpr int64_t kFewGrid = 256;

// From this many tokens on, tasks of 32 columns where every workgroup has one (16 tokens, 8 experts of I 128:
// 32 tasks 10.1 us, 64 of 16 columns 9.9).  Gate/up, 32 against 16: 16 tokens (H 6144, I 2048, group
// 128) 227 against 246 us, 12 tokens 185 against 199, 12 tokens MXFP4 177 against 179, 16 tokens (H 4096,
// I 1024, 64 experts) 46.5 against 44.8; 8 tokens 132 against 136, (H 4096, I 1024) 32.0 against 29.4; 1 token 26.7
// against 24.6.  So the rule takes the slower form, by 3 to 4 %, at 16 tokens of the smaller layer and at 8 of
// the larger: what decides may be the tasks per workgroup rather than the tokens.
constexpr int64_t kFewWideTokens = 9;

template <int kForm, int GW, int S, int NC>
static void launch_few_gate_up(const FewArgs& a, hipStream_t stream) {
  const int64_t R = a.T * a.k, tasks = (R < a.E ? R : a.E) * (a.I / (16 * NC));   // at most
  hipLaunchKernelGGL((few_gate_up_kernel<kForm, GW, S, NC>), dim3((unsigned)(tasks < kFewGrid ? tasks : kFewGrid)),
                     dim3(kFewThreads), (size_t)few_gate_up_smem(a.T, a.H), stream, a.x, (int)a.T, a.H, a.ld, a.logits,
                     a.E, a.k, a.renormalize, static_cast<const uint8_t*>(a.w13), static_cast<const uint8_t*>(a.s13),
                     a.I, a.ids, a.w, a.workspace);
}

template <int kForm, int GW, int S>
static hipError_t launch_few_form(const FewArgs& a, hipStream_t stream) {
  const int64_t R = a.T * a.k;
  const bool wide = a.T >= kFewWideTokens && (R < a.E ? R : a.E) * (a.I >> 5) >= kFewGrid;
  if (!wide) launch_few_gate_up<kForm, GW, S, 1>(a, stream);
  else launch_few_gate_up<kForm, GW, S, 2>(a, stream);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  // at most M pieces of each of `cols` blocks of 32 columns
  const int64_t groups = FewDownShape<2>::kGroups, nch = (a.I / kGroup + groups - 1) / groups;
  const int64_t M = (R < a.E ? R : a.E) * nch, cols = a.H / FewDownShape<2>::kCols;
  if (cols < kFewMinBlocks && few_down_range((int)(cols * M), (int)M) == M) {
    launch_few_down<kForm, 1>(a, (unsigned)(a.H / 16), stream);
  } else {
    // whatever the number of distinct experts, ranges are whole blocks or whole rounds of the waves
    const int64_t rounds = (cols * M + kFewWaves - 1) / kFewWaves, wgs = rounds > cols ? rounds : cols;
    launch_few_down<kForm, 2>(a, (unsigned)(wgs < kFewDownMaxGrid ? wgs : kFewDownMaxGrid), stream);
  }
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
