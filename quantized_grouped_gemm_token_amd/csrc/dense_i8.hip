// Dense products in 8-bit integers and the gated feed-forward block on them (w4a8_block.h).
//
// One workgroup of kWM x kWN waves computes a tile of kBM rows x kBN weight rows (output
// columns), in 16x16x64 INT8 products with int32 sums (exact, so K may be taken in any order).  K
// goes in steps of 128 bytes, a cache line of each row, through a ring of kSlots slots in LDS that
// loads straight into LDS fill kSlots - 1 steps ahead; operands are read from LDS four blocks of
// 16 rows ahead of their products, with one barrier a step.  Workgroups stay for all their tiles
// (a multiple of 256): a tile's first loads are issued ahead of the last one's epilogue.
//
// What bounds it.  Many rows (256 x 256): the card's power.  The INT8 products alone, from registers
// of random codes, run at 3250 to 3750 TOP/s (4530 to 4670 on zeros, the clock being held); 8192 x
// 12288 x 6144 takes 436 to 481 us, 2570 to 2840 TOP/s with loads, LDS and epilogue, the matrix
// cores busy 67% of the cycles at 1.9 GHz.
// The smaller tiles: what a CU gets from its L2 (130 to 150 GB/s), 100 to 300 rows the latency of the
// loads at a step each (128 x 6144 x 6144 11.5 us in 192 tiles of 64 x 64).  Weights that come
// from memory reach one CU at 25 to 35 GB/s.
//
// Measured and not taken, 8192 x 12288 x 6144 unless named: 4 waves of 128 x 128 (593 against 532
// us at that stage), steps of 64 bytes in 4 slots (half lines double the L2's requests: 503
// against 484), lines touched ahead into L2 (482 against 472), wave priorities, XCDs out of step and
// nontemporal stores (nothing); K split over workgroups with a second kernel for the sums (128 x
// 6144 x 6144 16.4 against 11.7, weights in a cache); tiles of 128 x 32 in a ring of 4 (the same 14.2 against
// 11.7, from memory 21.4 against 18.5), of 64 x 128 and 128 x 256.
#include "block.hpp"
#include "gemm_common.hpp"
#include "lds_dma.hpp"
#include "row_codes.hpp"

#include <type_traits>

namespace w4a8 {

namespace {

constexpr int kBK = 128;             // K bytes of a step

// Row r of a slot keeps its 16-byte chunk c at 16 (c ^ swz(r)): the operand reads (lane l: row
// l % 16, chunk 2 (l / 16) + h of half h) are then free of bank conflicts.  Which K elements a
// half takes does not matter, as both operands take the same.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// a buffer resource in scalar registers (64-bit comparisons leave uniform values in vector ones)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, int bytes) {
  const uint64_t p = (uint64_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)p);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32));
  return buffer_rsrc(reinterpret_cast<const void*>(((uint64_t)hi << 32) | lo), (uint32_t)__builtin_amdgcn_readfirstlane(bytes));
}

// what a tile leaves: y (fp32 or bf16), or act of the gated product
enum Out : int { kOutF32 = 0, kOutBf16 = 1, kOutAct = 2 };

// s_waitcnt's field for at most n vector memory operations in flight (n < 64), with lgkmcnt(l)
constexpr int vm_wait(int n, int l) { return (n & 15) | ((n >> 4) << 14) | 0x70 | (l << 8); }

// kOutAct: the tile's columns are 16 gate rows and the 16 up rows of the same act columns in
// turn, and the result is act = silu(gate) up, fp32 [M][I]; otherwise y, with an addend (kAdd).
template <int kBM, int kBN, int kWM, int kWN, int kSlots, int kOut, bool kAdd>
__global__ __launch_bounds__(64 * kWM * kWN) void dense_i8_kernel(const DenseArgs d, int64_t I,
                                                                  float* __restrict__ act, int mblocks, int nblocks) {
  constexpr bool kGated = kOut == kOutAct;
  constexpr int kWaves = kWM * kWN;
  constexpr int WM = kBM / kWM, WN = kBN / kWN, FM = WM / 16, FN = WN / 16;
  constexpr int kSlot = (kBM + kBN) * kBK;
  constexpr int kALoads = kBM / 8 / kWaves, kWLoads = kBN / 8 / kWaves;    // instructions of 8 rows per wave
  constexpr int kCols = kBN < 64 ? 64 : kBN;
  constexpr int kScaleBytes = 4 * (2 * kCols + kBM);                       // w_scale, bias, a_scale of a tile
  __shared__ __attribute__((aligned(16))) uint8_t sm[kSlots * kSlot + 2 * kScaleBytes];   // the slots, two tiles' scales
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int K = (int)d.K, steps = (K + kBK - 1) / kBK;
  const int total = mblocks * nblocks;

  // Loads of 8 rows of 128 bytes.  A row or chunk past the operand is never read (its offset is
  // past the resource) and never matters: rows past the end give outputs that are not stored,
  // bytes past K are taken out of a in the last step.
  uint32_t aoff[kALoads], woff[kWLoads];
#pragma unroll
  for (int q = 0; q < kALoads; ++q) {
    const int r = 8 * (kALoads * wave + q) + (lane >> 3);
    aoff[q] = (uint32_t)(r * (int)d.ld_a + 16 * ((lane & 7) ^ swz(r)));
  }
#pragma unroll
  for (int q = 0; q < kWLoads; ++q) {
    const int r = 8 * (kWLoads * wave + q) + (lane >> 3);
    const int wr = kGated ? 16 * (r >> 5) + (r & 15) : r;
    woff[q] = (uint32_t)(wr * K + 16 * ((lane & 7) ^ swz(r)));
  }
  // gated: a wave's loads go two by two over gate and up rows, or are all of one kind
  constexpr bool kBoth = kGated && kWLoads % 4 == 0;
  static_assert(kBoth || !kGated || kWLoads <= 2, "gate and up rows");
  __amdgpu_buffer_rsrc_t ra, rw0, rw1;
  int64_t m0 = 0, n0 = 0;
  // Column blocks of the largest tiles begin at K steps of their own, each one further, and turn
  // over K (sums of integers do not care): their loads then meet on fewer memory channels.  8192 x
  // 12288 x 6144 462 to 454 us, 4096 x 6144 x 6144 133 to 131; the smaller tiles lose 1 to 4%.
  constexpr bool kTurns = kBM * kBN == 65536;
  int turn = 0;

  // Tile t of the workgroups' order: workgroups go to the 8 XCDs in turn, and each XCD takes a
  // window of neighbouring tiles.  The tiles go in groups of 4 row blocks that walk the column
  // blocks side by side, so that 32 tiles of an XCD at a time share 4 row and 8 column blocks
  // in its L2.
  auto point = [&](int t, int par) {
    const int per = 4 * nblocks, group = t / per, gm = min(4, mblocks - 4 * group), in = t - group * per;
    m0 = (int64_t)(4 * group + in % gm) * kBM, n0 = (int64_t)(in / gm) * kBN;
    if (kTurns && K % kBK == 0) turn = (in / gm) % steps;      // (a part of a step stays the last)
    const int rows = (int)min((int64_t)kBM, d.M - m0), cols = (int)min((int64_t)kBN, d.N - n0);
    ra = uniform_rsrc(d.a + m0 * d.ld_a, (rows - 1) * (int)d.ld_a + K);
    const int64_t c0 = kGated ? n0 / 2 : n0;
    const int wrows = kGated ? cols / 2 : cols;
    const bool up = kGated && !kBoth && ((kWLoads * wave) >> 1) % 2;
    rw0 = uniform_rsrc(d.w + ((up ? I : 0) + c0) * K, wrows * K);
    if (kBoth) rw1 = uniform_rsrc(d.w + (I + c0) * K, wrows * K);
    // scales of the tile: 64 words to an instruction
    uint8_t* sc = &sm[kSlots * kSlot + par * kScaleBytes];
    for (int c = wave; c < kCols / 64; c += kWaves) {
      // gated: the gate and up rows 32 c .. +31 of the tile's act columns, by 16
      const uint32_t o = kGated ? (uint32_t)(32 * c + 16 * (lq >> 1) + lr + (lq & 1) * (int)I) * 4u
                                : (uint32_t)(64 * c + lane) * 4u;
      const int bytes = kGated ? (int)(I + wrows) * 4 : cols * 4;
      dma4(uniform_rsrc(d.w_scale + c0, bytes), o, 0, sc + 256 * c);
      if (!kGated && d.bias) dma4(uniform_rsrc(d.bias + n0, cols * 4), o, 0, sc + 4 * kCols + 256 * c);
    }
    for (int c = wave; c < kBM / 64; c += kWaves)
      dma4(uniform_rsrc(d.a_scale + m0, rows * 4), (uint32_t)(64 * c + lane) * 4u, 0, sc + 8 * kCols + 256 * c);
  };
  constexpr int kLoads = kALoads + kWLoads;
  auto load = [&](int kt, int q) {                            // load q of the wave's kLoads of step kt
    const uint32_t k = (uint32_t)((kTurns && kt + turn >= steps ? kt + turn - steps : kt + turn) * kBK);
    uint8_t* slot = &sm[(kt % kSlots) * kSlot];
    if (q < kALoads) {
      dma16(ra, aoff[q], k, slot + 8 * (kALoads * wave + q) * kBK);
    } else {
      const int u = q - kALoads;
      uint8_t* to = slot + (kBM + 8 * (kWLoads * wave + u)) * kBK;
      if (kBoth && ((u >> 1) & 1)) dma16(rw1, woff[u], k, to);
      else dma16(rw0, woff[u], k, to);
    }
  };
  // The first loads of a tile: those that the steps before would have issued.  A step kt issues
  // the rest of step kt + kSlots - 1, and from its barrier on the first kEarly of step kt + kSlots.
  constexpr int kAhead = FM < 4 ? FM : 4, kPerRegion = (kLoads + 2 * kAhead - 1) / (2 * kAhead), kEarly = kAhead * kPerRegion;
  auto begin = [&]() {
    for (int kt = 0; kt < min(kSlots - 1, steps); ++kt)
#pragma unroll
      for (int q = 0; q < kLoads; ++q) load(kt, q);
    if (kSlots - 1 < steps) {
#pragma unroll
      for (int q = 0; q < kEarly; ++q) load(kSlots - 1, q);
    }
  };
  const int wm = WM * (wave / kWN), wn = WN * (wave % kWN);
  const int fs = swz(lr);

  const int grid = gridDim.x;
  const int window = (grid + 7) >> 3;
  const int first = (blockIdx.x & 7) * window + (blockIdx.x >> 3);    // (grid % 8 == 0, or one round)
  const int start = grid % 8 == 0 ? first : (int)blockIdx.x;
  int par = 0;
  if (!kGated && !d.bias) {                                    // a bias of zero
    for (int c = tid; c < 2 * kCols; c += 64 * kWaves)
      reinterpret_cast<float*>(&sm[kSlots * kSlot + (c / kCols) * kScaleBytes])[kCols + c % kCols] = 0.0f;
    __builtin_amdgcn_s_waitcnt(0xC07F);                        // (read after the barriers of the first tile)
  }
  point(start, par);
  begin();
  for (int t = start; t < total; t += grid, par ^= 1) {
    i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    // A step is 2 FM regions: the products of one block of 16 rows and half a step's K with the
    // FN column blocks.  Region r reads the row block of region r + kAhead, and in the last
    // kAhead regions of a half the column blocks of the next.  Before region kLast the wave's
    // reads of the slot are done and the loads of the next step (in the other slot) have landed;
    // one barrier, and from there on the next step's operands are read, at the pace of the
    // others, and the slot is filled again.
    constexpr int kRegions = 2 * FM, kLast = kRegions - kAhead, kPerA = (FN + kAhead - 1) / kAhead;
    constexpr int kHeld = kRegions < 8 ? kRegions : 8;
    static_assert(FM % kAhead == 0 && kRegions % kHeld == 0 && FN % 2 == 0, "regions");
    i32x4 a[kHeld], b[2][FN];
    auto read_a = [&](int s, int r) {
      a[r % kHeld] = lds_load<i32x4>(&sm[s * kSlot + (wm + lr + 16 * (r % FM)) * kBK + 16 * ((2 * lq + r / FM) ^ fs)]);
    };
    auto read_b = [&](int s, int h, int j) {
      b[h][j] = lds_load<i32x4>(&sm[s * kSlot + (kBM + wn + lr + 16 * j) * kBK + 16 * ((2 * lq + h) ^ fs)]);
    };
    // step 0 has landed when only the loads after it are in flight (and stores of the last tile)
    if (steps >= kSlots) __builtin_amdgcn_s_waitcnt(vm_wait((kSlots - 2) * kLoads + kEarly, 15));
    else __builtin_amdgcn_s_waitcnt(vm_wait(0, 15));
    barrier_loads_in_flight();
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      read_a(0, r);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        if (j / kPerA == r) read_b(0, 0, j);
    }
    __builtin_amdgcn_sched_barrier(0);
    const int64_t tm0 = m0, tn0 = n0;                         // (the last step points to the next tile)
    // kPhase: 0 while a step issues loads of both later steps, 1 the one that issues the last
    // loads, 2 those after it, 3 the tile's last step (where bytes past K are zeros)
    auto step = [&](auto Phase_, int kt) {
      constexpr int kPhase = decltype(Phase_)::value;
      const int s = kt % kSlots, next = (kt + 1) % kSlots;
#pragma unroll
      for (int r = 0; r < kRegions; ++r) {
        const int h = r / FM, i = r % FM;
        if (r == kLast) {
          // (of the steps after the next one, all loads may be in flight)
          __builtin_amdgcn_s_waitcnt(vm_wait(kPhase == 3 ? 63 : kPhase == 2 ? 0 : (kSlots - 2) * kLoads, 0));
          barrier_loads_in_flight();
          if (kPhase == 3 && t + grid < total) {              // the next tile's first loads
            point(t + grid, par ^ 1);
            begin();
          }
        }
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
          if (kPhase < 2 && r < kLast && q >= kEarly && (q - kEarly) / kPerRegion == r) load(kt + kSlots - 1, q);
          if (kPhase < 1 && r >= kLast && q < kEarly && q / kPerRegion == r - kLast) load(kt + kSlots, q);
        }
        if (r < kLast) read_a(s, r + kAhead);
        else if (kPhase < 3) read_a(next, r - kLast);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if (r >= FM - kAhead && r < FM && j / kPerA == r - (FM - kAhead)) read_b(s, 1, j);
          if (kPhase < 3 && r >= kLast && j / kPerA == r - kLast) read_b(next, 0, j);
        }
        if (kPhase == 3 && kt * kBK + 16 * (2 * lq + h) >= K) a[r % kHeld] = i32x4{0, 0, 0, 0};
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma_i8_16x16x64(b[h][j], a[r % kHeld], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int kt = 0;
    for (; kt + kSlots < steps; ++kt) step(std::integral_constant<int, 0>{}, kt);
    for (; kt + kSlots == steps; ++kt) step(std::integral_constant<int, 1>{}, kt);
    if constexpr (kSlots > 2)
      for (; kt + 1 < steps; ++kt) step(std::integral_constant<int, 2>{}, kt);
    step(std::integral_constant<int, 3>{}, steps - 1);
    // ---- epilogue: D lane holds row lr of its row block, outputs 4 lq .. +3 of its column block
    // (lane roles taken afresh: addresses built from them are not kept through the products)
    int lr = lane & 15, lq = lane >> 4;
    asm volatile("" : "+v"(lr), "+v"(lq));
    const float* sc = reinterpret_cast<const float*>(&sm[kSlots * kSlot + par * kScaleBytes]) + wn + 4 * lq;
    const float* as = reinterpret_cast<const float*>(&sm[kSlots * kSlot + par * kScaleBytes]) + 2 * kCols + wm + lr;
    const int mleft = (int)min(d.M - tm0 - wm, (int64_t)WM);  // rows of the wave
    const int nleft = (int)min(d.N - tn0 - wn, (int64_t)WN);  // columns of the wave
    const int64_t row0 = tm0 + wm + lr;
    float sa[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = as[16 * i];
    constexpr bool kBf16 = kOut == kOutBf16;
    using E = std::conditional_t<kBf16, uint16_t, float>;
    using Four = std::conditional_t<kBf16, uint2, f32x4>;      // 4 values of y's type
    // (the column blocks of a row one after the other: whole lines of y and of the addend, 8192 x
    // 6144 x 1024 54.6 us, row blocks one after the other 62.2; with an addend 88.7 and 94.9.
    // Addends read 2 to 8 blocks ahead, or touched during the products, gave 92 to 104: they
    // come at the rate that memory has for them and the results together.)
    f32x4 ws[FN], bs[kGated ? 1 : FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      ws[j] = lds_load<f32x4>(sc + 16 * j);
      if constexpr (!kGated) bs[j] = lds_load<f32x4>(sc + kCols + 16 * j);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const bool live = 16 * i + lr < mleft;
#pragma unroll
      for (int j = 0; j < FN; j += 2) {                        // two column blocks: gate and up, or 32 outputs
        const bool whole = 16 * j + 32 <= nleft;               // (the same for the whole wave)
        if constexpr (kGated) {
          f32x4 o;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            o[v] = silu_mul((float)acc[i][j][v] * sa[i] * ws[j][v], (float)acc[i][j + 1][v] * sa[i] * ws[j + 1][v]);
          // (a block of 32 columns is all inside the 2 I, or none)
          if (live && whole)
            *reinterpret_cast<f32x4*>(act + (row0 + 16 * i) * I + (tn0 + wn) / 2 + 8 * j + 4 * lq) = o;
        } else {
          const int64_t at = (row0 + 16 * i) * d.N + tn0 + wn + 16 * j;
          const E* add = static_cast<const E*>(d.add) + at;
          E* y = static_cast<E*>(d.y) + at;
          f32x4 o[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int v = 0; v < 4; ++v) o[e][v] = (float)acc[i][j + e][v] * sa[i] * ws[j + e][v] + bs[j + e][v];
          if (whole) {
            if constexpr (kAdd) {
              Four w[2];
              if (live) {
                __builtin_memcpy(&w[0], add + 4 * lq, sizeof(Four));
                __builtin_memcpy(&w[1], add + 16 + 4 * lq, sizeof(Four));
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if constexpr (kBf16) {
                  o[e][0] += bf16_lo(w[e].x), o[e][1] += bf16_hi(w[e].x), o[e][2] += bf16_lo(w[e].y), o[e][3] += bf16_hi(w[e].y);
                } else {
#pragma unroll
                  for (int v = 0; v < 4; ++v) o[e][v] += w[e][v];
                }
              }
            }
            if constexpr (kBf16) {
              // neighbouring groups of 16 lanes trade halves: 8 outputs of one block each
              const auto s0 = __builtin_amdgcn_permlane16_swap(bf16_pair(o[0][0], o[0][1]), bf16_pair(o[1][0], o[1][1]),
                                                               false, false);
              const auto s1 = __builtin_amdgcn_permlane16_swap(bf16_pair(o[0][2], o[0][3]), bf16_pair(o[1][2], o[1][3]),
                                                               false, false);
              const uint4 v = make_uint4(s0[0], s1[0], s0[1], s1[1]);
              if (live) __builtin_memcpy(y + 16 * (lq & 1) + 8 * (lq >> 1), &v, 16);
            } else if (live) {
#pragma unroll
              for (int e = 0; e < 2; ++e) __builtin_memcpy(y + 16 * e + 4 * lq, &o[e], 16);
            }
          } else if (live) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const int c = 16 * e + 4 * lq + v;
                if (16 * j + c < nleft) {
                  float r = o[e][v];
                  if constexpr (kBf16) {
                    if (kAdd) r += __uint_as_float((uint32_t)add[c] << 16);
                    y[c] = __builtin_bit_cast(uint16_t, (__bf16)r);
                  } else {
                    y[c] = kAdd ? r + add[c] : r;
                  }
                }
              }
          }
        }
        __builtin_amdgcn_sched_barrier(0);                     // one row block at a time: few temporaries
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
__global__ __launch_bounds__(256) void act_quant_kernel(const float* __restrict__ act, int64_t M, int64_t I,
                                                        uint8_t* __restrict__ q, float* __restrict__ s) {
  __shared__ uint32_t red[4];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= M) return;
  const float4* ar = reinterpret_cast<const float4*>(act + row * I);
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
  uint32_t* qr = reinterpret_cast<uint32_t*>(q + row * I);
  for (int c = threadIdx.x; c < (int)(I >> 2); c += 256) {
    const float4 v = ar[c];
    qr[c] = codes4<true>(v.x * d.by, v.y * d.by, v.z * d.by, v.w * d.by, d.s, d.r);
  }
  if (threadIdx.x == 0) s[row] = scale;
}

template <int kBM, int kBN, int kWM, int kWN, int kSlots, int kPerCu, int kOut, bool kAdd>
hipError_t launch_tiles(const DenseArgs& d, int64_t I, float* act, hipStream_t stream) {
  const int64_t mb = (d.M + kBM - 1) / kBM, nb = (d.N + kBN - 1) / kBN;
  auto kernel = dense_i8_kernel<kBM, kBN, kWM, kWN, kSlots, kOut, kAdd>;
  static_assert(kPerCu * (kSlots * (kBM + kBN) * kBK + 2 * 4 * (2 * (kBN < 64 ? 64 : kBN) + kBM)) <= 160 * 1024, "LDS");
  const int64_t slots = 256 * kPerCu, tiles = mb * nb;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles < slots ? tiles : slots)), dim3(64 * kWM * kWN), 0, stream, d, I,
                     act, (int)mb, (int)nb);
  return hipGetLastError();
}

// The tile that ends first: the tiles go over the 256 CUs in rounds, and a round costs the tile's
// time per step.  Measured at K = 6144 (us a step, one tile on each CU): 64 x 32 0.19, 64 x 64 0.20, 128 x 64
// 0.33, 128 x 128 0.46, 256 x 128 0.63 to 0.84, 256 x 256 1.15 to 1.35 (the larger the nearer to
// the card's power limit).  A CU reads weights from memory at 25 to 35 GB/s however many loads it
// has in flight, so the narrow tile, up to one for each CU, is for few rows: 64 x 6144 x 6144 10.8 us against 11.7 with
// 64 x 64, and 15.0 against 18.7 where the weights come from memory and not from a cache (20 rows 11.4
// against 15.9; of 8, 6 and 4 slots, 8).  6144 outputs (us; the tile chosen first, then the next best): 128 rows
// 11.7 with 64 x 64, 16.4 with 128 x 64; 256 rows 17.2 with 128 x 64, 19.5 with 64 x 64; 512 rows
// 22.8 with 128 x 128, 32.7 with 128 x 64; 1024 rows 37.8 with 256 x 128, 42.3 with 128 x 128; 2048
// rows 64.9 with 256 x 256, 73.3 with 128 x 128; 3000 rows 113.7 with 256 x 128, 129.9 with 256 x 256.
template <int kOut, bool kAdd>
hipError_t launch_product(const DenseArgs& d, int64_t I, float* act, hipStream_t stream) {
  auto cost = [&](int bm, int bn, double step) {
    return step * (double)((((d.M + bm - 1) / bm) * ((d.N + bn - 1) / bn) + 255) / 256);
  };
  const double c[6] = {cost(64, 32, 0.19),   cost(64, 64, 0.20),   cost(128, 64, 0.33),
                       cost(128, 128, 0.46), cost(256, 128, 0.75), cost(256, 256, 1.32)};
  int best = 0;
  for (int i = 1; i < 6; ++i)
    if (c[i] < c[best]) best = i;
  switch (best) {
    case 0: return launch_tiles<64, 32, 4, 1, 8, 1, kOut, kAdd>(d, I, act, stream);
    case 1: return launch_tiles<64, 64, 2, 2, 4, 2, kOut, kAdd>(d, I, act, stream);
    case 2: return launch_tiles<128, 64, 2, 2, 4, 1, kOut, kAdd>(d, I, act, stream);
    case 3: return launch_tiles<128, 128, 2, 2, 4, 1, kOut, kAdd>(d, I, act, stream);
    case 4: return launch_tiles<256, 128, 4, 2, 3, 1, kOut, kAdd>(d, I, act, stream);
    default: return launch_tiles<256, 256, 2, 4, 2, 1, kOut, kAdd>(d, I, act, stream);
  }
}

}  // namespace

hipError_t launch_dense_i8(const DenseArgs& d, hipStream_t stream) {
  if (dense_few_fits(d.M, d.ld_a)) return launch_dense_few(d, stream);
  if (d.y_bf16)
    return d.add ? launch_product<kOutBf16, true>(d, 0, nullptr, stream)
                 : launch_product<kOutBf16, false>(d, 0, nullptr, stream);
  return d.add ? launch_product<kOutF32, true>(d, 0, nullptr, stream)
               : launch_product<kOutF32, false>(d, 0, nullptr, stream);
}

// act fp32 [M][I], then codes [M][I] and scales [M], or the maxima of 8 columns of act [M][I / 8]
int64_t mlp_i8_workspace_bytes(int64_t M, int64_t, int64_t I) { return M * (5 * I + 4); }

hipError_t launch_mlp_i8(const MlpArgs& p, hipStream_t stream) {
  float* act = static_cast<float*>(p.workspace);
  uint8_t* q = reinterpret_cast<uint8_t*>(act + p.M * p.I);
  float* s = reinterpret_cast<float*>(q + p.M * p.I);
  const DenseArgs up{p.a, p.a_scale, p.M, p.H, p.ld_a, p.w13, p.s13, nullptr, 2 * p.I, nullptr, nullptr, 0};
  const DenseArgs down{reinterpret_cast<int8_t*>(q), s, p.M, p.I, p.I, p.w2, p.s2, nullptr, p.H, p.add, p.y, p.y_bf16};
  if (dense_few_fits(p.M, p.ld_a)) {
    uint32_t* pmax = reinterpret_cast<uint32_t*>(q);
    if (const hipError_t e = launch_gated_few(up, p.I, act, pmax, stream); e != hipSuccess) return e;
    return launch_down_few(down, act, pmax, stream);
  }
  if (const hipError_t e = launch_product<kOutAct, false>(up, p.I, act, stream); e != hipSuccess) return e;
  constexpr int64_t kWide = (int64_t)1 << 23;                 // (a launch has fewer than 2^32 threads in x)
  const dim3 grid((unsigned)(p.M < kWide ? p.M : kWide), (unsigned)((p.M + kWide - 1) / kWide));
  hipLaunchKernelGGL(act_quant_kernel, grid, dim3(256), 0, stream, act, p.M, p.I, q, s);
  return launch_dense_i8(down, stream);
}

}  // namespace w4a8
