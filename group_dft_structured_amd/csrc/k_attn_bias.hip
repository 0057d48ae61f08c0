// The bias table's gradient from the sums over offsets that the backward pass's
// work-groups left: [parts][heads][2 span + 1], first over the parts (of the slots of
// tiles, those up to the last sequence's end), in a few
// slices, then over the slices and over the offsets of a bucket, in binary64: one
// far bucket may hold most pairs of tokens, with both signs.  Fixed orders
// throughout.  A few megabytes, bound by two launches: 5 + 5 us after the 236 us of
// a backward pass over 16 documents, 12 heads, 257 offsets.
#include "eqattn_internal.h"

namespace eql {
namespace attn {
namespace {

// Slices of the first sum: enough work-groups for many parts, and few partial
// sums for the second kernel.
constexpr int MAX_SLICES = 16;
int slices_of(int parts) {
  const int n = parts / 32;
  return n < 1 ? 1 : n > MAX_SLICES ? MAX_SLICES : n;
}

__global__ __launch_bounds__(1024) void k_bias_slices(const float* __restrict__ hist,
                                                      double* __restrict__ slices, int parts, int cols,
                                                      const int32_t* __restrict__ cu_q, int seqs,
                                                      int total_q, int slot_rows) {
  __shared__ double s[16][64];
  int first = 0;
  if (slot_rows > 0 && parts > 0) {
    const int start = cu_q[0], end = cu_q[seqs];
    first = (start < 0 ? 0 : start > total_q ? total_q : start) / slot_rows;
    const int behind = (end < 0 ? 0 : end > total_q ? total_q : end) / slot_rows + seqs;
    parts = behind < parts ? behind : parts;
  }
  const int col = blockIdx.x * 64 + (threadIdx.x & 63), sub = threadIdx.x >> 6;
  double v = 0.0;
  if (col < cols) {
#pragma unroll 8
    for (int p = first + blockIdx.y * 16 + sub; p < parts; p += 16 * gridDim.y) v += hist[(int64_t)p * cols + col];
  }
  s[sub][threadIdx.x & 63] = v;
  __syncthreads();
  if (sub != 0 || col >= cols) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
  slices[(int64_t)blockIdx.y * cols + col] = v;
}

// A work-group a head and 32 buckets: the sums of all offsets in LDS, then eight
// lanes a bucket.
__global__ __launch_bounds__(256) void k_bias_buckets(const double* __restrict__ slices,
                                                      const int32_t* __restrict__ map,
                                                      float* __restrict__ dtable, int heads, int width,
                                                      int buckets, int count) {
  __shared__ double sum[2 * EQATTN_MAX_SPAN + 1];
  __shared__ int bucket[2 * EQATTN_MAX_SPAN + 1];
  const int head = blockIdx.x;
  for (int r = threadIdx.x; r < width; r += 256) {
    double v = 0.0;
#pragma unroll 16
    for (int s = 0; s < count; ++s) v += slices[((int64_t)s * heads + head) * width + r];
    sum[r] = v;
    bucket[r] = map[r];
  }
  __syncthreads();
  const int b = blockIdx.y * 32 + threadIdx.x / 8;
  double v = 0.0;
#pragma unroll 4
  for (int r = threadIdx.x & 7; r < width; r += 8) v += bucket[r] == b ? sum[r] : 0.0;
#pragma unroll
  for (int d = 1; d < 8; d *= 2) v += __shfl_xor(v, d);
  if ((threadIdx.x & 7) == 0 && b < buckets) dtable[(int64_t)b * heads + head] = (float)v;
}

}  // namespace

size_t slices_bytes(const eqattn_plan* p) {
  return (size_t)MAX_SLICES * p->H * (2 * (size_t)p->span + 1) * sizeof(double);
}

hipError_t launch_bias_finish(const Common& c, const float* hist, int parts, double* slices,
                              float* dtable, hipStream_t st) {
  const int width = 2 * c.span + 1, cols = c.H * width, count = slices_of(parts);
  hipLaunchKernelGGL(k_bias_slices, dim3((unsigned)((cols + 63) / 64), count), dim3(1024), 0, st, hist,
                     slices, parts, cols, c.cu_q, c.seqs, c.total_q, c.slot_rows);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_bias_buckets, dim3((unsigned)c.H, (unsigned)((c.buckets + 31) / 32)), dim3(256), 0, st, slices, c.map, dtable, c.H,
                     width, c.buckets, count);
  return hipGetLastError();
}

}  // namespace attn
}  // namespace eql
