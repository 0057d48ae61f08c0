/*
 * eqnorm.h -- C ABI of the layer norm over a token's channels and group values
 * in libeqlinear (AMD MI355X, gfx950): forward, and backward with the
 * reductions of the affine gradients.
 *
 * The operation.  A row x[n] holds C channels of T group values.  With the
 * mean and the variance of all C * T values of the row,
 *
 *     xhat[n,c,t] = (x[n,c,t] - mean[n]) * rstd[n],  rstd = 1 / sqrt(var + eps)
 *     y[n,c,t]    = xhat[n,c,t] * gamma[c] + beta[c]
 *
 * The affine parameters are one per channel, equal on its T group values: the
 * statistics do not change when a group element permutes the values of every
 * channel, and neither do gamma and beta, so the norm commutes with the group
 * as the layers of eqlinear.h do, for the cyclic and the dihedral groups.
 * T = 1 is the layer norm of C features.
 *
 * Backward.  With g = dy * gamma and F = C * T,
 *
 *     dx[n,c,t] = rstd[n] * (g - sum(g)/F - xhat * sum(g * xhat)/F)   (sums over the row)
 *     dgamma[c] = sum_{n,t} dy[n,c,t] * xhat[n,c,t]                   (binary32)
 *     dbeta[c]  = sum_{n,t} dy[n,c,t]                                 (binary32)
 *
 * Arithmetic.  Rows are held in binary32 once loaded; the variance is the mean
 * of squared differences from the mean (no cancellation); y and dx are rounded
 * once.  The reductions over rows run in a fixed order: the same call gives
 * the same bits.  A NaN or infinity in a row makes that row's outputs NaN as
 * the formulas do, and no other row's.
 *
 * Layouts (dense, row-major, group index fastest; every pointer 16-byte
 * aligned, EQL_ERR_MISALIGNED otherwise):
 *     x, y, dy, dx : [N][C][T] in the plan dtype     gamma, beta : [C] in the plan dtype
 *     mean, rstd : [N] binary32                      dgamma, dbeta : [C] binary32
 * y may be x and dx may be dy (in place); other overlaps are not allowed.
 *
 * Ownership, streams, errors and concurrency are as in eqlinear.h: buffers
 * belong to the caller, every call is asynchronous on the given HIP stream,
 * allocates nothing and can be captured in a graph, and arguments are checked
 * on the host before any HIP call.
 */
#ifndef EQNORM_H
#define EQNORM_H

#include <stddef.h>
#include <stdint.h>

#include "eqlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most features C * T of a row: a row is kept by one work-group, in registers up to
 * 8192 features and partly in scratch memory backward above. */
#define EQNORM_MAX_FEATURES 16384

typedef struct eqnorm_plan* eqnorm_plan_t; /* opaque */

/* Create a plan for rows of C channels of T group values, 1 <= T <= 16.
 * EQL_ERR_INVALID_ARG: C <= 0, eps negative or not finite or (unless 0) outside
 * binary32, out == NULL;
 * EQL_ERR_UNSUPPORTED: T or dtype out of range, C * T > EQNORM_MAX_FEATURES.
 * Host-only: allocates no device memory. */
eqlinear_status_t eqnorm_plan_create(int64_t C, int64_t T, double eps, eqlinear_dtype_t dtype,
                                     eqnorm_plan_t* out);

/* Destroy a plan (NULL is a no-op). */
eqlinear_status_t eqnorm_plan_destroy(eqnorm_plan_t plan);

/* y, and the rows' mean and rstd (each NULL = not wanted), of x.  gamma NULL is
 * all ones, beta NULL all zeros.  N = 0 is a successful no-op. */
eqlinear_status_t eqnorm_forward(eqnorm_plan_t plan, const void* x, const void* gamma,
                                 const void* beta, void* y, float* mean, float* rstd, int64_t N,
                                 void* stream);

/* Bytes of device workspace eqnorm_backward needs for N rows (0 for an invalid
 * plan or N <= 0): partial sums of dgamma and dbeta. */
size_t eqnorm_backward_workspace(eqnorm_plan_t plan, int64_t N);

/* dx, dgamma and dbeta (the latter two NULL = not wanted) from dy, the
 * forward's input x and its mean and rstd.  Outputs are overwritten, not
 * accumulated into.  The workspace may be NULL where neither dgamma nor dbeta
 * is wanted; otherwise EQL_ERR_WORKSPACE if NULL or too small.  N = 0 writes
 * zeros to dgamma and dbeta. */
eqlinear_status_t eqnorm_backward(eqnorm_plan_t plan, const void* x, const void* dy,
                                  const void* gamma, const float* mean, const float* rstd, void* dx,
                                  float* dgamma, float* dbeta, int64_t N, void* workspace,
                                  size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EQNORM_H */
