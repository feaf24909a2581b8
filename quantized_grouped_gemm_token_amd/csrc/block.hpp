// Internal launchers of the operators around the experts (called by abi_block.cpp after it
// has validated every argument on the host).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a8 {

// y [M][N] = a [M][K] x w [N][K]^T in int8, scaled (dense_i8.hip)
constexpr int64_t kDenseMaxK = (int64_t)1 << 17;    // (exclusive) 2^14 K < 2^31: exact int32 sums of any codes
constexpr int64_t kDenseMaxN = (int64_t)1 << 24;
constexpr int64_t kDenseMaxLd = (int64_t)1 << 22;   // 32-bit offsets within 256 rows
constexpr int64_t kDenseMaxOut = (int64_t)1 << 40;  // M N: tile numbers stay below 2^31
constexpr int64_t kMlpMaxI = 65536;
struct DenseArgs {
  const int8_t* a;
  const float* a_scale;
  int64_t M, K, ld_a;
  const int8_t* w;
  const float* w_scale;
  const float* bias;      // or null
  int64_t N;
  const void* add;        // or null
  void* y;
  int y_bf16;
};
hipError_t launch_dense_i8(const DenseArgs& d, hipStream_t stream);

struct MlpArgs {
  const int8_t* a;
  const float* a_scale;
  int64_t M, H, ld_a;
  const int8_t* w13;
  const float* s13;
  const int8_t* w2;
  const float* s2;
  int64_t I;
  const void* add;        // or null
  void* y;
  int y_bf16;
  void* workspace;
};
int64_t mlp_i8_workspace_bytes(int64_t M, int64_t H, int64_t I);
hipError_t launch_mlp_i8(const MlpArgs& m, hipStream_t stream);

// the same for 1 to 16 rows (dense_few.hip); the gated product (d: w13, N = 2 I) leaves act [M][I] and
// pmax [M][I / 8], bit patterns of the maxima of 8 columns of |act|; the down product (d: w2, K = I, a
// unused) quantizes act itself
bool dense_few_fits(int64_t M, int64_t ld_a);
hipError_t launch_dense_few(const DenseArgs& d, hipStream_t stream);
hipError_t launch_gated_few(const DenseArgs& d, int64_t I, float* act, uint32_t* pmax, hipStream_t stream);
hipError_t launch_down_few(const DenseArgs& d, float* act, uint32_t* pmax, hipStream_t stream);

// norms before and after a block (norm.hip).  Without r: the norm of x.  With it: out from x
// (the block's result) and r, and, where `weight` is set, the norm of out.
constexpr int64_t kNormMaxH = 32768;     // 1024 threads, 4 chunks of 8 values each
constexpr float kNormMinEps = 0x1p-100f;
enum NormCodes : int { kCodesNone = 0, kCodesFp8 = 1, kCodesI8 = 2 };
struct NormArgs {
  const void* x;
  int x_bf16;
  int64_t ld_x, T, H;
  const float* weight;
  float eps;
  int codes;              // NormCodes
  uint16_t* xn;           // or null
  uint8_t* q;             // or null, with s
  float* s;
  int32_t* rowsum;        // or null
  const void* r;          // or null
  int r_bf16;
  int64_t ld_r;
  const float* post;      // or null
  const float* gate;      // or null
  const float* token_gate;  // or null
  float r_scale;
  void* out;
  int64_t ld_out;
};
hipError_t launch_norm(const NormArgs& n, hipStream_t stream);

}  // namespace w4a8
