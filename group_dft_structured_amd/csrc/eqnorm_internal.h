// Host-side internals of the norm: the plan object and kernel launchers.
#pragma once

#include "../../include/eqnorm.h"
#include "eql_internal.h"

struct eqnorm_plan {
  int64_t C, T;
  double eps;
  eqlinear_dtype_t dtype;
  size_t esize;
};

namespace eql {

// Most work-groups of a pass: those that find a place on the chip at once, five a
// compute unit forward and three backward, by their registers at three vectors of
// binary16 a lane (384 and 768 features, where it was measured).  Other widths find
// other numbers of places, so that their last turn may be a part of one: at four
// vectors a lane (1024, 4096 features) four a compute unit forward and two backward,
// two backward in binary32 at three vectors, and two or one above 4096 features.
constexpr int64_t FWD_BLOCKS = 1280, BWD_BLOCKS = 768;

// Work-groups, and so partial sums, of a backward pass over N rows.
int norm_parts(const eqnorm_plan* p, int64_t N);

hipError_t launch_norm_forward(const eqnorm_plan* p, const void* x, const void* gamma,
                               const void* beta, void* y, float* mean, float* rstd, int64_t N,
                               hipStream_t s);
hipError_t launch_norm_backward(const eqnorm_plan* p, const void* x, const void* dy,
                                const void* gamma, const float* mean, const float* rstd, void* dx,
                                float* dgamma, float* dbeta, int64_t N, void* ws, hipStream_t s);

}  // namespace eql
