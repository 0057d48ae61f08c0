// C ABI of the norm (include/eqnorm.h): argument validation and dispatch.
// Every check runs before the first HIP call.
#include <float.h>
#include <string.h>

#include <new>

#include "eqnorm_internal.h"

namespace {

constexpr int64_t MAX_ROWS = ((int64_t)1 << 31) - 1;
constexpr int64_t MAX_T = 16;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

eqlinear_status_t hip_status(const char* what, hipError_t e) {
  if (e == hipSuccess) return EQL_OK;
  eql::set_last_error(what, e);
  return EQL_ERR_HIP;
}

}  // namespace

extern "C" {

eqlinear_status_t eqnorm_plan_create(int64_t C, int64_t T, double eps, eqlinear_dtype_t dtype_arg,
                                     eqnorm_plan_t* out) {
  if (out == nullptr) return EQL_ERR_INVALID_ARG;
  *out = nullptr;
  if (C <= 0 || !(eps >= 0 && eps <= FLT_MAX) || (eps > 0 && (float)eps == 0.f)) return EQL_ERR_INVALID_ARG;
  const int dv = eql::enum_value(dtype_arg);
  if (dv != EQL_F32 && dv != EQL_F16) return EQL_ERR_UNSUPPORTED;
  if (T < 1 || T > MAX_T || C > EQNORM_MAX_FEATURES / T) return EQL_ERR_UNSUPPORTED;
  eqnorm_plan* p = new (std::nothrow) eqnorm_plan;
  if (p == nullptr) return EQL_ERR_ALLOC;
  p->C = C;
  p->T = T;
  p->eps = eps;
  p->dtype = (eqlinear_dtype_t)dv;
  p->esize = dv == EQL_F16 ? 2 : 4;
  *out = p;
  return EQL_OK;
}

eqlinear_status_t eqnorm_plan_destroy(eqnorm_plan_t p) {
  delete p;
  return EQL_OK;
}

eqlinear_status_t eqnorm_forward(eqnorm_plan_t p, const void* x, const void* gamma,
                                 const void* beta, void* y, float* mean, float* rstd, int64_t N,
                                 void* stream) {
  if (p == nullptr || N < 0 || N > MAX_ROWS) return EQL_ERR_INVALID_ARG;
  if (N == 0) return EQL_OK;
  if (x == nullptr || y == nullptr) return EQL_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(gamma) || !aligned16(beta) ||
      !aligned16(mean) || !aligned16(rstd))
    return EQL_ERR_MISALIGNED;
  return hip_status("norm forward launch", eql::launch_norm_forward(p, x, gamma, beta, y, mean, rstd,
                                                                    N, (hipStream_t)stream));
}

size_t eqnorm_backward_workspace(eqnorm_plan_t p, int64_t N) {
  if (p == nullptr || N <= 0 || N > MAX_ROWS) return 0;
  return (size_t)eql::norm_parts(p, N) * 2 * (size_t)p->C * sizeof(float);
}

eqlinear_status_t eqnorm_backward(eqnorm_plan_t p, const void* x, const void* dy,
                                  const void* gamma, const float* mean, const float* rstd, void* dx,
                                  float* dgamma, float* dbeta, int64_t N, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (p == nullptr || N < 0 || N > MAX_ROWS) return EQL_ERR_INVALID_ARG;
  if (N > 0 && (x == nullptr || dy == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr))
    return EQL_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(dy) || !aligned16(gamma) || !aligned16(mean) || !aligned16(rstd) ||
      !aligned16(dx) || !aligned16(dgamma) || !aligned16(dbeta) || !aligned16(workspace))
    return EQL_ERR_MISALIGNED;
  const size_t need = eqnorm_backward_workspace(p, N);
  if ((dgamma != nullptr || dbeta != nullptr) && need > 0 &&
      (workspace == nullptr || workspace_bytes < need))
    return EQL_ERR_WORKSPACE;
  return hip_status("norm backward launch",
                    eql::launch_norm_backward(p, x, dy, gamma, mean, rstd, dx, dgamma, dbeta, N,
                                              workspace, (hipStream_t)stream));
}

}  // extern "C"
