// Host side of the C ABIs declared in include/atom_mxfp4.h and include/atom_norm.h: argument validation (all of
// it before any HIP call), then the kernel launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "host_checks.h"
#include "serve_internal.h"

namespace {

using namespace atom::check;

uint64_t groups_of(int32_t K) { return ((uint64_t)K + ATOM_MX_GROUP - 1) / ATOM_MX_GROUP; }
uint64_t row_bytes4(int32_t K) { return groups_of(K) * (ATOM_MX_GROUP / 2); }
uint64_t code_bytes(int32_t rows, int32_t K) { return (uint64_t)rows * row_bytes4(K); }
uint64_t scale_bytes(int32_t rows, int32_t K) { return (uint64_t)rows * groups_of(K) * 8; }

// The plan of a valid shape with as much scratch memory; false where no launch would hold it.
bool plan_of(int32_t M, int32_t N, int32_t K, atom::MxPlan& plan, int64_t scratch = INT64_MAX) {
  if (!valid_gemm8(M, N, K)) return false;
  plan = atom::mx_plan(M, N, K, scratch);
  return plan.tiles > 0;
}
int64_t linear_bytes(int32_t M, int32_t K, const atom::MxPlan& plan) {
  return (int64_t)(code_bytes(M, K) + up16(scale_bytes(M, K))) + atom::mx_workspace_bytes(plan);
}

// The checks that both norms share; `codes` and `scales`: bytes of their outputs.
int check_norm(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* W, double eps, int32_t dtype, int32_t rows,
               int32_t K, const void* H, int64_t ldh, const void* Xq, const void* sx, uint64_t (*codes)(int32_t, int32_t),
               uint64_t (*scales)(int32_t, int32_t)) {
  if (!X || !W || !Xq || !sx || (R && !H)) return ATOM_E_NULL;
  if (!valid_k8(K) || !valid_rows(rows) || !valid_dtype(dtype) || (H && !R) || !(eps > 0.0) || !(eps < 1e300)) return ATOM_E_SHAPE;
  if (!aligned(X, 2) || !aligned(R, 2) || !aligned(W, 2) || !aligned(H, 2) || !aligned16(Xq) || !aligned16(sx)) return ATOM_E_ALIGN;
  if (!valid_x(X, ldx, rows, K) || (R && (!valid_x(R, ldr, rows, K) || !valid_x(H, ldh, rows, K)))) return ATOM_E_SHAPE;
  const Range x = range_of(X, x_bytes(ldx, rows, K)), w = range_of(W, (uint64_t)K * 2);
  const Range out[3] = {range_of(Xq, codes(rows, K)), range_of(sx, scales(rows, K)), range_of(H, R ? x_bytes(ldh, rows, K) : 0)};
  const Range r = range_of(R, R ? x_bytes(ldr, rows, K) : 0);
  const Range in[3] = {x, w, r};
  if (int s = check_overlap(in, R ? 3 : 2, out, 2)) return s;
  if (!R) return ATOM_OK;
  if (int s = check_overlap(out, 2, out + 2, 1)) return s;
  // the sum may take the place of one of its terms, row for row
  const bool on_x = H == X && (rows == 1 || ldh == ldx), on_r = H == R && (rows == 1 || ldh == ldr);
  if ((!on_x && overlap(out[2], x)) || (!on_r && overlap(out[2], r)) || overlap(out[2], w)) return ATOM_E_OVERLAP;
  return ATOM_OK;
}

uint64_t codes8(int32_t rows, int32_t K) { return (uint64_t)rows * row_bytes8(K); }
uint64_t scales8(int32_t rows, int32_t) { return (uint64_t)rows * 4; }

int rmsnorm(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* W, double eps, int32_t dtype, int32_t rows,
            int32_t K, void* H, int64_t ldh, void* Xq, void* sx, bool mx, void* stream) {
  const int s = mx ? check_norm(X, ldx, R, ldr, W, eps, dtype, rows, K, H, ldh, Xq, sx, code_bytes, scale_bytes)
                   : check_norm(X, ldx, R, ldr, W, eps, dtype, rows, K, H, ldh, Xq, sx, codes8, scales8);
  if (s) return s;
  const atom::NormCall n = {static_cast<const uint16_t*>(X), ldx, static_cast<const uint16_t*>(R), ldr,
                            static_cast<const uint16_t*>(W), eps, dtype == ATOM_BF16, rows, K, static_cast<uint16_t*>(H), ldh,
                            static_cast<uint8_t*>(Xq), sx};
  return hip_status(atom::launch_rmsnorm(n, mx, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int64_t atom_mxfp4_row_bytes(int32_t K) { return valid_k8(K) ? (int64_t)row_bytes4(K) : -(int64_t)ATOM_E_SHAPE; }
int32_t atom_mxfp4_groups(int32_t K) { return valid_k8(K) ? (int32_t)groups_of(K) : -(int32_t)ATOM_E_SHAPE; }

int atom_quantize_mxfp4(const void* X, int64_t ldx, int32_t dtype, int32_t rows, int32_t K, void* Xq, void* sx,
                        void* stream) {
  if (!X || !Xq || !sx) return ATOM_E_NULL;
  if (!valid_k8(K) || !valid_rows(rows) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  if (!valid_x(X, ldx, rows, K)) return aligned(X, 2) ? ATOM_E_SHAPE : ATOM_E_ALIGN;
  if (!aligned16(Xq) || !aligned16(sx)) return ATOM_E_ALIGN;
  const Range in[1] = {range_of(X, x_bytes(ldx, rows, K))};
  const Range out[2] = {range_of(Xq, code_bytes(rows, K)), range_of(sx, scale_bytes(rows, K))};
  if (int s = check_overlap(in, 1, out, 2)) return s;
  return hip_status(atom::launch_quantize_mxfp4(static_cast<const uint16_t*>(X), ldx, dtype == ATOM_BF16, rows, K,
                                                static_cast<uint8_t*>(Xq), static_cast<uint8_t*>(sx),
                                                static_cast<hipStream_t>(stream)));
}

int atom_dequantize_mxfp4(const void* Xq, const void* sx, int32_t rows, int32_t K, int32_t dtype, void* X, void* stream) {
  if (!X || !Xq || !sx) return ATOM_E_NULL;
  if (!valid_k8(K) || !valid_rows(rows) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  if (!aligned16(X) || !aligned16(Xq) || !aligned16(sx)) return ATOM_E_ALIGN;
  const Range in[2] = {range_of(Xq, code_bytes(rows, K)), range_of(sx, scale_bytes(rows, K))};
  const Range out[1] = {range_of(X, (uint64_t)rows * (uint64_t)K * 2)};
  if (int s = check_overlap(in, 2, out, 1)) return s;
  return hip_status(atom::launch_dequantize_mxfp4(static_cast<const uint8_t*>(Xq), static_cast<const uint8_t*>(sx), rows, K,
                                                  dtype == ATOM_BF16, static_cast<uint16_t*>(X),
                                                  static_cast<hipStream_t>(stream)));
}

int64_t atom_gemm_mxfp4_workspace_bytes(int32_t M, int32_t N, int32_t K) {
  atom::MxPlan plan;
  if (!plan_of(M, N, K, plan)) return -(int64_t)ATOM_E_SHAPE;
  return atom::mx_workspace_bytes(plan);
}

int atom_gemm_mxfp4(const void* Xq, const void* sx, const void* Wq, const void* sw, const void* bias, int32_t M, int32_t N,
                    int32_t K, int32_t dtype, void* Y, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!Xq || !sx || !Wq || !sw || !Y) return ATOM_E_NULL;
  atom::MxPlan plan;
  if (!plan_of(M, N, K, plan, workspace ? workspace_bytes : 0) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  if (!aligned16(Xq) || !aligned16(sx) || !aligned16(Wq) || !aligned16(sw) || !aligned16(bias) || !aligned16(Y))
    return ATOM_E_ALIGN;
  const int64_t need = atom::mx_workspace_bytes(plan);
  if (need > 0 && !aligned16(workspace)) return ATOM_E_ALIGN;
  const Range in[5] = {range_of(Xq, code_bytes(M, K)), range_of(sx, scale_bytes(M, K)), range_of(Wq, code_bytes(N, K)),
                       range_of(sw, scale_bytes(N, K)), range_of(bias, bias ? (uint64_t)N * 2 : 0)};
  const Range out[2] = {range_of(Y, (uint64_t)M * N * 2), range_of(workspace, (uint64_t)need)};
  if (int s = check_overlap(in, bias ? 5 : 4, out, need > 0 ? 2 : 1)) return s;
  return hip_status(atom::launch_gemm_mxfp4(static_cast<const uint8_t*>(Xq), static_cast<const uint8_t*>(sx),
                                            static_cast<const uint8_t*>(Wq), static_cast<const uint8_t*>(sw),
                                            static_cast<const uint16_t*>(bias), M, N, K, dtype == ATOM_BF16,
                                            static_cast<uint16_t*>(Y), need > 0 ? static_cast<float*>(workspace) : nullptr,
                                            plan, static_cast<hipStream_t>(stream)));
}

int64_t atom_linear_mxfp4_workspace_bytes(int32_t M, int32_t N, int32_t K) {
  if (!valid_gemm8(M, N, K)) return -(int64_t)ATOM_E_SHAPE;
  if (atom::mx_one_launch(M, N, K)) return 0;
  atom::MxPlan plan;
  return plan_of(M, N, K, plan) ? linear_bytes(M, K, plan) : -(int64_t)ATOM_E_SHAPE;
}

int atom_linear_mxfp4(const void* X, int64_t ldx, int32_t dtype, const void* Wq, const void* sw, const void* bias, int32_t M,
                      int32_t N, int32_t K, void* Y, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!X || !Wq || !sw || !Y) return ATOM_E_NULL;
  if (!valid_gemm8(M, N, K) || !valid_dtype(dtype)) return ATOM_E_SHAPE;
  const bool one = atom::mx_one_launch(M, N, K);
  atom::MxPlan plan = {};
  if (!one && !plan_of(M, N, K, plan)) return ATOM_E_SHAPE;
  if (!valid_x(X, ldx, M, K)) return aligned(X, 2) ? ATOM_E_SHAPE : ATOM_E_ALIGN;
  const int64_t need = one ? 0 : linear_bytes(M, K, plan);
  if (need > 0 && !workspace) return ATOM_E_NULL;
  if (workspace_bytes < need) return ATOM_E_SHAPE;
  if (!aligned16(Wq) || !aligned16(sw) || !aligned16(bias) || !aligned16(Y) || (need > 0 && !aligned16(workspace)))
    return ATOM_E_ALIGN;
  const Range in[4] = {range_of(X, x_bytes(ldx, M, K)), range_of(Wq, code_bytes(N, K)), range_of(sw, scale_bytes(N, K)),
                       range_of(bias, bias ? (uint64_t)N * 2 : 0)};
  const Range out[2] = {range_of(Y, (uint64_t)M * N * 2), range_of(workspace, (uint64_t)need)};
  if (int s = check_overlap(in, bias ? 4 : 3, out, need > 0 ? 2 : 1)) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const uint8_t *wq = static_cast<const uint8_t*>(Wq), *ws = static_cast<const uint8_t*>(sw);
  if (one)
    return hip_status(atom::launch_linear_rows_mxfp4(static_cast<const uint16_t*>(X), ldx, wq, ws,
                                                     static_cast<const uint16_t*>(bias), M, N, K, dtype == ATOM_BF16,
                                                     static_cast<uint16_t*>(Y), st));
  uint8_t* xq = static_cast<uint8_t*>(workspace);
  uint8_t* sx = xq + code_bytes(M, K);
  float* part = reinterpret_cast<float*>(sx + up16(scale_bytes(M, K)));
  const hipError_t e = atom::launch_quantize_mxfp4(static_cast<const uint16_t*>(X), ldx, dtype == ATOM_BF16, M, K, xq, sx, st);
  if (e != hipSuccess) return ATOM_E_HIP;
  return hip_status(atom::launch_gemm_mxfp4(xq, sx, wq, ws, static_cast<const uint16_t*>(bias), M, N, K, dtype == ATOM_BF16,
                                            static_cast<uint16_t*>(Y), part, plan, st));
}

int atom_rmsnorm_w8a8(const void* X, int64_t ldx, const void* residual, int64_t ldr, const void* weight, double eps,
                      int32_t dtype, int32_t rows, int32_t K, void* H, int64_t ldh, void* Xq, float* sx, void* stream) {
  return rmsnorm(X, ldx, residual, ldr, weight, eps, dtype, rows, K, H, ldh, Xq, sx, false, stream);
}

int atom_rmsnorm_mxfp4(const void* X, int64_t ldx, const void* residual, int64_t ldr, const void* weight, double eps,
                       int32_t dtype, int32_t rows, int32_t K, void* H, int64_t ldh, void* Xq, void* sx, void* stream) {
  return rmsnorm(X, ldx, residual, ldr, weight, eps, dtype, rows, K, H, ldh, Xq, sx, true, stream);
}

}  // extern "C"
