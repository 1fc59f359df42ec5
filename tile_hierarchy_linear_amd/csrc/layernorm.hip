// layernorm.hip -- the layer norm of each token (centred, with weight and
// bias), the residual's addition before it and its output in 32, 16, 8 or 4
// bits, and its gradient.
//
//   s = x + r,   mu = mean(s),   rho = 1 / sqrt(mean((s - mu)^2) + eps)
//   h = (s - mu) * rho,   y_i = q(h_i * w_i + b_i)
//
// with q as in norm.hip.  Gradient: with t = w * dy,
//   dx = rho * (t - mean(t) - h * mean(t * h)) + dr
//   dw = sum over tokens of dy * h,   db = sum over tokens of dy.
//
// The kernels are norm.hip's (norm_kernels.hpp), bound by HBM like them.  A
// token is in registers, so its mean is found first and the squares are of
// differences from it: one more sum over the workgroup, and no cancellation.
//
// Measured on bf16: the norm of 16,384 tokens of 4,096 features with residual
// 100 us (5.4 TB/s; a large copy runs at 5.0), of eight tokens of 8,192 4.6 us (a
// launch alone takes 3.9); the gradient of 8,192 tokens of 4,096 features 58 us
// (5.2 TB/s with the partial sums of dw and db, an eighth of the traffic).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "../../include/thl.h"
#include "host_checks.hpp"
#include "norm_kernels.hpp"

namespace thl {
namespace {

// Workgroups of the gradient: the other norm's, or as many fewer as take the same
// number of rounds.
int64_t rows_of(int64_t m, int64_t n) {
  const int64_t rows = grad_rows(m, n);
  if (m <= 512) return rows;  // (four tokens a workgroup)
  const int64_t rounds = (n + rows - 1) / rows;
  return (n + rounds - 1) / rounds;
}

}  // namespace
}  // namespace thl

using namespace thl;

extern "C" {

thl_status thl_layernorm(int64_t m, int64_t n, const void* X, int64_t ldx, const void* R, int64_t ldr, void* S,
                         int64_t lds, const void* W, const void* B, float eps, float y_scale, void* Y, int64_t ldy,
                         uint8_t* sfy, int64_t ld_sfy, const thl_norm_types* ty, struct ihipStream_t* stream) {
  // ---- arguments
  if (!ty || m < 0 || n < 0) return THL_ERR_INVALID;
  if (m > kMaxFeatures || big(n) || big(ldx) || big(ldr) || big(lds) || big(ldy) || big(ld_sfy)) return THL_ERR_UNSUPPORTED;
  if (!is_float_io(ty->x) || ((W || B) && !is_float_io(ty->w))) return THL_ERR_UNSUPPORTED;
  if (R && ty->r != ty->x && ty->r != THL_F32) return THL_ERR_UNSUPPORTED;
  const bool fp8 = ty->y == THL_E4M3 || ty->y == THL_E5M2, fp4 = ty->y == THL_E2M1X2;
  if (!is_float_io(ty->y) && !fp8 && !fp4) return THL_ERR_UNSUPPORTED;
  const bool mx = sfy != nullptr;
  if (is_float_io(ty->y) ? mx : (fp4 && !mx)) return THL_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || std::isinf(eps)) return THL_ERR_INVALID;
  const float inv_scale = 1.0f / y_scale;
  if (!(y_scale > 0.0f) || std::isinf(y_scale) || std::isinf(inv_scale)) return THL_ERR_INVALID;
  if (y_scale != 1.0f && (!fp8 || mx)) return THL_ERR_UNSUPPORTED;
  if (bad_ld(ldx, m) || bad_ld(ldy, m)) return THL_ERR_INVALID;
  if (fp4 && ldy % 2 != 0) return THL_ERR_INVALID;
  if (R ? (bad_ld(ldr, m) || (S && bad_ld(lds, m))) : S != nullptr) return THL_ERR_INVALID;
  if (mx && ld_sfy < (m + 31) / 32) return THL_ERR_INVALID;
  if (m == 0 || n == 0) return THL_OK;
  if (!X || !Y) return THL_ERR_INVALID;
  if (misaligned(X, ty->x) || (W && misaligned(W, ty->w)) || (B && misaligned(B, ty->w)) ||
      (is_float_io(ty->y) && misaligned(Y, ty->y)) || (R && (misaligned(R, ty->r) || misaligned(S, ty->r))))
    return THL_ERR_MISALIGNED;

  // ---- overlap: S may be X or R exactly, Y may be X exactly
  const Range rx = matrix_range(X, ty->x, m, n, ldx);
  const Range rw = W ? matrix_range(W, ty->w, m, 1, m) : Range{}, rb = B ? matrix_range(B, ty->w, m, 1, m) : Range{};
  const Range rr = R ? matrix_range(R, ty->r, m, n, ldr) : Range{};
  const Range rs = R ? matrix_range(S, ty->r, m, n, lds) : Range{};
  const Range ry = matrix_range(Y, ty->y, m, n, ldy);
  const Range rf = mx ? matrix_range(sfy, THL_E8M0, (m + 31) / 32, n, ld_sfy) : Range{};
  const bool s_is_x = S == X && lds == ldx && ty->r == ty->x, s_is_r = S == R && lds == ldr;
  const bool y_is_x = Y == X && ldy == ldx && ty->y == ty->x;
  if ((!s_is_x && overlaps(rs, rx)) || (!s_is_r && overlaps(rs, rr)) || (!y_is_x && overlaps(ry, rx)) ||
      overlaps(ry, rr) || overlaps(ry, rs))
    return THL_ERR_INVALID;
  for (const Range& o : {rw, rb})
    if (overlaps(rs, o) || overlaps(ry, o) || overlaps(rf, o)) return THL_ERR_INVALID;
  for (const Range& o : {rx, rr, rs, ry})
    if (overlaps(rf, o)) return THL_ERR_INVALID;

  NormArgs a{};
  a.x = X, a.r = R, a.s = S, a.w = W, a.b = B, a.y = Y, a.sf = sfy;
  a.ldx = ldx, a.ldr = ldr, a.lds = lds, a.ldy = ldy, a.ld_sf = ld_sfy;
  a.n = n, a.m = static_cast<int32_t>(m), a.eps = eps, a.inv_scale = inv_scale;
  a.x_type = ty->x, a.r_type = ty->r, a.w_type = ty->w, a.y_type = ty->y;
  a.y_mode = mx ? Y_MX : (fp8 ? Y_FP8 : Y_FLOAT);
  return launch_norm<true>(a, stream) == hipSuccess ? THL_OK : THL_ERR_HIP;
}

size_t thl_layernorm_backward_workspace(int64_t m, int64_t n) {
  if (m <= 0 || n <= 0) return 0;
  return 2 * static_cast<size_t>(rows_of(m, n)) * static_cast<size_t>(m) * sizeof(float);
}

thl_status thl_layernorm_backward(int64_t m, int64_t n, const void* S, int64_t lds, const void* DY, int64_t lddy,
                                  const void* DR, int64_t lddr, const void* W, float eps, void* DX, int64_t lddx,
                                  void* DW, void* DB, void* workspace, size_t workspace_bytes,
                                  const thl_norm_grad_types* ty, struct ihipStream_t* stream) {
  if (!ty || m < 0 || n < 0) return THL_ERR_INVALID;
  if (m > kMaxFeatures || big(n) || big(lds) || big(lddy) || big(lddr) || big(lddx)) return THL_ERR_UNSUPPORTED;
  if (!is_float_io(ty->s) || (W && !is_float_io(ty->w)) || !is_float_io(ty->g)) return THL_ERR_UNSUPPORTED;
  if ((DW || DB) && ty->dw != THL_F32 && (!W || ty->dw != ty->w)) return THL_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || std::isinf(eps)) return THL_ERR_INVALID;
  if (bad_ld(lds, m) || bad_ld(lddy, m) || bad_ld(lddx, m) || (DR && bad_ld(lddr, m))) return THL_ERR_INVALID;
  if (m == 0) return THL_OK;
  if ((DW && misaligned(DW, ty->dw)) || (DB && misaligned(DB, ty->dw))) return THL_ERR_MISALIGNED;
  const Range rd = DW ? matrix_range(DW, ty->dw, m, 1, m) : Range{}, re = DB ? matrix_range(DB, ty->dw, m, 1, m) : Range{};
  if (overlaps(rd, re)) return THL_ERR_INVALID;
  const size_t need = DW || DB ? thl_layernorm_backward_workspace(m, n) : 0;
  if (n > 0) {
    if (!S || !DY || !DX) return THL_ERR_INVALID;
    if (need && (!workspace || workspace_bytes < need)) return THL_ERR_INVALID;
    if (misaligned(S, ty->s) || misaligned(DY, ty->g) || (W && misaligned(W, ty->w)) || misaligned(DX, ty->g) ||
        misaligned(DR, ty->g) || (need && reinterpret_cast<uintptr_t>(workspace) % 4 != 0))
      return THL_ERR_MISALIGNED;
    // DX may be DY, DR or S exactly; nothing else may overlap an output
    const Range rs = matrix_range(S, ty->s, m, n, lds), rg = matrix_range(DY, ty->g, m, n, lddy);
    const Range rr = matrix_range(DR, ty->g, m, n, lddr), rw = W ? matrix_range(W, ty->w, m, 1, m) : Range{};
    const Range rx = matrix_range(DX, ty->g, m, n, lddx);
    const Range rp = need ? vector_range(workspace, static_cast<int64_t>(need), 1) : Range{};
    if ((overlaps(rx, rs) && !(DX == S && lddx == lds && ty->g == ty->s)) ||
        (overlaps(rx, rg) && !(DX == DY && lddx == lddy)) || (overlaps(rx, rr) && !(DX == DR && lddx == lddr)) ||
        overlaps(rx, rw))
      return THL_ERR_INVALID;
    for (const Range& o : {rs, rg, rr, rw, rx})
      if (overlaps(rd, o) || overlaps(re, o) || overlaps(rp, o)) return THL_ERR_INVALID;
    if (overlaps(rd, rp) || overlaps(re, rp)) return THL_ERR_INVALID;
  }

  hipError_t e = hipSuccess;
  const int64_t rows = n > 0 ? rows_of(m, n) : 0;
  if (n > 0) {
    NormGradArgs a{};
    a.s = S, a.dy = DY, a.dr = DR, a.w = W, a.dx = DX, a.part = need ? static_cast<float*>(workspace) : nullptr;
    a.lds = lds, a.lddy = lddy, a.lddr = lddr, a.lddx = lddx;
    a.n = n, a.m = static_cast<int32_t>(m), a.eps = eps;
    a.s_type = ty->s, a.g_type = ty->g, a.w_type = ty->w;
    e = launch_grad<true>(a, rows, stream);
  }
  if (e == hipSuccess && (DW || DB))
    e = launch_grad_reduce(static_cast<const float*>(workspace), rows, 2 * m, m, DW, DB, ty->dw, stream);
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

}  // extern "C"
