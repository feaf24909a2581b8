// C ABI of the operators around the experts (w4a8_block.h): host-side argument checks, then
// kernel launches on the caller's stream, as in abi.cpp.
#include "w4a8_block.h"

#include <cmath>

#include "abi_common.hpp"
#include "block.hpp"

using namespace w4a8::abi;
typedef long long ll;

namespace {

bool is_dtype(int32_t d) { return d == W4A8_Y_F32 || d == W4A8_Y_BF16; }
int64_t element(int32_t d) { return d == W4A8_Y_F32 ? 4 : 2; }

int check_dense(const char* name, int64_t M, int64_t N, int64_t K, int64_t ld_a, int32_t y_dtype) {
  if (M < 0 || M >= kMaxRows) return fail(W4A8_ERR_SHAPE, "%s: %lld rows out of range", name, (ll)M);
  if (N <= 0 || N > w4a8::kDenseMaxN)
    return fail(W4A8_ERR_SHAPE, "%s: N=%lld must be in 1..%lld", name, (ll)N, (ll)w4a8::kDenseMaxN);
  if (K <= 0 || K % 16 || K >= w4a8::kDenseMaxK)
    return fail(W4A8_ERR_SHAPE, "%s: row length %lld must be a positive multiple of 16 below %lld", name, (ll)K,
                (ll)w4a8::kDenseMaxK);
  if (ld_a < K || ld_a % 16 || ld_a > w4a8::kDenseMaxLd)
    return fail(W4A8_ERR_SHAPE, "%s: ld_a=%lld must be >= %lld, a multiple of 16 and at most %lld", name, (ll)ld_a,
                (ll)K, (ll)w4a8::kDenseMaxLd);
  if (M * N > w4a8::kDenseMaxOut)
    return fail(W4A8_ERR_SHAPE, "%s: %lld x %lld outputs are too many", name, (ll)M, (ll)N);
  if (!is_dtype(y_dtype))
    return fail(W4A8_ERR_SHAPE, "%s: y_dtype=%d must be W4A8_Y_F32 or W4A8_Y_BF16", name, y_dtype);
  return W4A8_OK;
}

int check_workspace(const char* name, const void* ws, int64_t bytes, int64_t need) {
  if (need == 0) return W4A8_OK;
  if (!ws) return fail(W4A8_ERR_NULL, "%s: null workspace", name);
  if (bytes < need)
    return fail(W4A8_ERR_WORKSPACE, "%s: workspace of %lld bytes, need %lld", name, (ll)bytes, (ll)need);
  if (!aligned(ws, 16)) return fail(W4A8_ERR_ALIGN, "%s: the workspace must be 16-byte aligned", name);
  return W4A8_OK;
}

// rows of a [T][ld] array of this type
int check_rows(const char* name, const char* what, int64_t H, int64_t ld, int32_t dtype) {
  if (!is_dtype(dtype))
    return fail(W4A8_ERR_SHAPE, "%s: the type of %s, %d, must be W4A8_Y_F32 or W4A8_Y_BF16", name, what, dtype);
  if (ld < H || (ld * element(dtype)) % 16 || ld > (int64_t)1 << 40)
    return fail(W4A8_ERR_SHAPE, "%s: ld=%lld of %s must be >= H and a whole number of 16 bytes", name, (ll)ld, what);
  return W4A8_OK;
}

int check_norm_sizes(const char* name, int64_t T, int64_t H, float eps) {
  if (T < 0 || T >= kMaxRows) return fail(W4A8_ERR_SHAPE, "%s: T=%lld out of range", name, (ll)T);
  if (H <= 0 || H % 8 || H > w4a8::kNormMaxH)
    return fail(W4A8_ERR_SHAPE, "%s: H=%lld must be a positive multiple of 8 up to %lld", name, (ll)H,
                (ll)w4a8::kNormMaxH);
  if (!(eps >= w4a8::kNormMinEps) || !std::isfinite(eps))
    return fail(W4A8_ERR_SHAPE, "%s: eps=%g must be finite and at least 2^-100", name, (double)eps);
  return W4A8_OK;
}

// the outputs of a norm before a block
int check_codes(const char* name, const float* weight, const void* xn, const void* q, const float* s,
                const int32_t* rowsum) {
  if (!weight || (!xn && !q) || (q == nullptr) != (s == nullptr) || (rowsum && !q))
    return fail(W4A8_ERR_NULL, "%s: null weight, no output, or codes without scales", name);
  if (!aligned(weight, 16) || !aligned(xn, 16) || !aligned(q, 8) || !aligned(s, 4) || !aligned(rowsum, 4))
    return fail(W4A8_ERR_ALIGN, "%s: the weight and xn must be 16-byte, codes 8-byte, scales and sums 4-byte aligned",
                name);
  return W4A8_OK;
}

int run_norm(const char* name, int codes, const void* x, int32_t x_dtype, int64_t T, int64_t H, int64_t ld_x,
             const float* weight, float eps, uint16_t* xn, void* q, float* s, int32_t* rowsum, void* stream) {
  if (int st = check_norm_sizes(name, T, H, eps)) return st;
  if (int st = check_rows(name, "x", H, ld_x, x_dtype)) return st;
  if (T == 0) return ok();
  if (!x) return fail(W4A8_ERR_NULL, "%s: null x", name);
  if (int st = check_codes(name, weight, xn, q, s, rowsum)) return st;
  if (!aligned(x, 16)) return fail(W4A8_ERR_ALIGN, "%s: x must be 16-byte aligned", name);
  if (int st = check_device()) return st;
  (void)hipGetLastError();
  w4a8::NormArgs n{};
  n.x = x, n.x_bf16 = x_dtype == W4A8_Y_BF16, n.ld_x = ld_x, n.T = T, n.H = H, n.weight = weight, n.eps = eps;
  n.codes = q ? codes : w4a8::kCodesNone, n.xn = xn, n.q = static_cast<uint8_t*>(q), n.s = s, n.rowsum = rowsum;
  return launched(w4a8::launch_norm(n, as_stream(stream)), name);
}

int run_residual(const char* name, int codes, const void* y, int32_t y_dtype, int64_t ld_y, const void* r,
                 int32_t r_dtype, int64_t ld_r, int64_t T, int64_t H, const float* post, const float* gate,
                 const float* token_gate, float r_scale, float eps, void* out, int64_t ld_out, const float* weight,
                 uint16_t* xn, void* q, float* s, int32_t* rowsum, void* stream) {
  if (int st = check_norm_sizes(name, T, H, eps)) return st;
  if (int st = check_rows(name, "y", H, ld_y, y_dtype)) return st;
  if (int st = check_rows(name, "r", H, ld_r, r_dtype)) return st;
  if (int st = check_rows(name, "out", H, ld_out, r_dtype)) return st;
  if (!std::isfinite(r_scale)) return fail(W4A8_ERR_SHAPE, "%s: r_scale=%g must be finite", name, (double)r_scale);
  if (T == 0) return ok();
  if (!y || !r || !out) return fail(W4A8_ERR_NULL, "%s: null pointer", name);
  if (codes != w4a8::kCodesNone)
    if (int st = check_codes(name, weight, xn, q, s, rowsum)) return st;
  if (!aligned(y, 16) || !aligned(r, 16) || !aligned(out, 16) || !aligned(post, 16) || !aligned(gate, 16) ||
      !aligned(token_gate, 4))
    return fail(W4A8_ERR_ALIGN, "%s: y, r, out and the vectors over H must be 16-byte aligned, token_gate 4-byte",
                name);
  if (int st = check_device()) return st;
  (void)hipGetLastError();
  w4a8::NormArgs n{};
  n.x = y, n.x_bf16 = y_dtype == W4A8_Y_BF16, n.ld_x = ld_y, n.T = T, n.H = H, n.weight = weight, n.eps = eps;
  n.codes = q ? codes : w4a8::kCodesNone, n.xn = xn, n.q = static_cast<uint8_t*>(q), n.s = s, n.rowsum = rowsum;
  n.r = r, n.r_bf16 = r_dtype == W4A8_Y_BF16, n.ld_r = ld_r, n.post = post, n.gate = gate;
  n.token_gate = token_gate, n.r_scale = r_scale, n.out = out, n.ld_out = ld_out;
  return launched(w4a8::launch_norm(n, as_stream(stream)), name);
}

}  // namespace

extern "C" {

int w4a8_moe_dense_i8(const int8_t* a, const float* a_scale, int64_t M, int64_t K, int64_t ld_a, const int8_t* w,
                      const float* w_scale, const float* bias, int64_t N, const void* add, void* y, int32_t y_dtype,
                      void* stream) {
  if (int st = check_dense("dense_i8", M, N, K, ld_a, y_dtype)) return st;
  if (M == 0) return ok();
  if (!a || !a_scale || !w || !w_scale || !y) return fail(W4A8_ERR_NULL, "dense_i8: null pointer");
  const uintptr_t e = (uintptr_t)element(y_dtype);
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
      !aligned(add, e) || !aligned(y, e))
    return fail(W4A8_ERR_ALIGN, "dense_i8: a and w must be 16-byte aligned, the rest to their elements");
  if (int st = check_device()) return st;
  (void)hipGetLastError();
  const w4a8::DenseArgs d{a, a_scale, M, K, ld_a, w, w_scale, bias, N, add, y, y_dtype == W4A8_Y_BF16};
  return launched(w4a8::launch_dense_i8(d, as_stream(stream)), "dense_i8");
}

static int check_mlp(int64_t M, int64_t H, int64_t I, int64_t ld_a, int32_t y_dtype) {
  if (I <= 0 || I % 128 || I > w4a8::kMlpMaxI)
    return fail(W4A8_ERR_SHAPE, "mlp_i8: I=%lld must be a positive multiple of 128 up to %lld", (ll)I,
                (ll)w4a8::kMlpMaxI);
  if (int st = check_dense("mlp_i8", M, 2 * I, H, ld_a, y_dtype)) return st;
  return check_dense("mlp_i8", M, H, I, I, y_dtype);
}

int64_t w4a8_moe_mlp_i8_workspace_bytes(int64_t M, int64_t H, int64_t I) {
  if (check_mlp(M, H, I, H, W4A8_Y_F32) != W4A8_OK) return -1;
  return w4a8::mlp_i8_workspace_bytes(M, H, I);
}

int w4a8_moe_mlp_i8(const int8_t* a, const float* a_scale, int64_t M, int64_t H, int64_t ld_a, const int8_t* w13,
                    const float* s13, const int8_t* w2, const float* s2, int64_t I, const void* add, void* y,
                    int32_t y_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  if (int st = check_mlp(M, H, I, ld_a, y_dtype)) return st;
  if (M == 0) return ok();
  if (!a || !a_scale || !w13 || !s13 || !w2 || !s2 || !y) return fail(W4A8_ERR_NULL, "mlp_i8: null pointer");
  const uintptr_t e = (uintptr_t)element(y_dtype);
  if (!aligned(a, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(a_scale, 4) || !aligned(s13, 4) ||
      !aligned(s2, 4) || !aligned(add, e) || !aligned(y, e))
    return fail(W4A8_ERR_ALIGN, "mlp_i8: a and the weights must be 16-byte aligned, the rest to their elements");
  if (int st = check_workspace("mlp_i8", workspace, workspace_bytes, w4a8::mlp_i8_workspace_bytes(M, H, I))) return st;
  if (int st = check_device()) return st;
  (void)hipGetLastError();
  const w4a8::MlpArgs m{a, a_scale, M, H, ld_a, w13, s13, w2, s2, I, add, y, y_dtype == W4A8_Y_BF16, workspace};
  return launched(w4a8::launch_mlp_i8(m, as_stream(stream)), "mlp_i8");
}

int w4a8_moe_norm_quant(const void* x, int32_t x_dtype, int64_t T, int64_t H, int64_t ld_x, const float* weight,
                        float eps, uint16_t* xn_bf16, uint8_t* qx, float* sx, void* stream) {
  return run_norm("norm_quant", w4a8::kCodesFp8, x, x_dtype, T, H, ld_x, weight, eps, xn_bf16, qx, sx, nullptr,
                  stream);
}

int w4a8_moe_norm_quant_i8(const void* x, int32_t x_dtype, int64_t T, int64_t H, int64_t ld_x, const float* weight,
                           float eps, uint16_t* xn_bf16, int8_t* qx, float* sx, int32_t* rowsum, void* stream) {
  return run_norm("norm_quant_i8", w4a8::kCodesI8, x, x_dtype, T, H, ld_x, weight, eps, xn_bf16, qx, sx, rowsum,
                  stream);
}

int w4a8_moe_residual_norm(const void* y, int32_t y_dtype, int64_t ld_y, const void* r, int32_t r_dtype, int64_t ld_r,
                           int64_t T, int64_t H, const float* post_weight, const float* gate, const float* token_gate,
                           float r_scale, float eps, void* out, int64_t ld_out, void* stream) {
  return run_residual("residual_norm", w4a8::kCodesNone, y, y_dtype, ld_y, r, r_dtype, ld_r, T, H, post_weight, gate,
                      token_gate, r_scale, eps, out, ld_out, nullptr, nullptr, nullptr, nullptr, nullptr, stream);
}

int w4a8_moe_residual_norm_quant(const void* y, int32_t y_dtype, int64_t ld_y, const void* r, int32_t r_dtype,
                                 int64_t ld_r, int64_t T, int64_t H, const float* post_weight, const float* gate,
                                 const float* token_gate, float r_scale, float eps, void* out, int64_t ld_out,
                                 const float* next_weight, uint16_t* xn_bf16, uint8_t* qx, float* sx, void* stream) {
  return run_residual("residual_norm_quant", w4a8::kCodesFp8, y, y_dtype, ld_y, r, r_dtype, ld_r, T, H, post_weight,
                      gate, token_gate, r_scale, eps, out, ld_out, next_weight, xn_bf16, qx, sx, nullptr, stream);
}

int w4a8_moe_residual_norm_quant_i8(const void* y, int32_t y_dtype, int64_t ld_y, const void* r, int32_t r_dtype,
                                    int64_t ld_r, int64_t T, int64_t H, const float* post_weight, const float* gate,
                                    const float* token_gate, float r_scale, float eps, void* out, int64_t ld_out,
                                    const float* next_weight, uint16_t* xn_bf16, int8_t* qx, float* sx,
                                    int32_t* rowsum, void* stream) {
  return run_residual("residual_norm_quant_i8", w4a8::kCodesI8, y, y_dtype, ld_y, r, r_dtype, ld_r, T, H, post_weight,
                      gate, token_gate, r_scale, eps, out, ld_out, next_weight, xn_bf16, qx, sx, rowsum, stream);
}

}  // extern "C"
