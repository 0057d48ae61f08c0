// Sums of the attention backward passes: products with a factor of any size, and
// the sums of ds over offsets.
//
// The sums over offsets lie in LDS: where positions are given, one copy for each
// half of each wave, where they follow from indices, one for each wave (Diagonals
// below).  The lanes of one half hold one key and 32 queries; where the queries' positions
// differ, no two lanes of an addition meet in one place, so a read, an add and a
// write do, in the order of the instructions.  (LDS float atomics took 250 cycles
// a wave and instruction: 632 us against 182 us of the other pass for 4096
// windows of 49 tokens and 6 heads.)  Where positions repeat, which the wave
// finds out at its start, atomics add.  Clamped offsets, where many would meet,
// are summed in registers.
#pragma once

#include "attn_device.h"

namespace eql {
namespace attn {
namespace {

// A running sum of products whose second operand is rounded to T.  In binary16
// each lane's column (a query in the first pass, a key in the second) has a power
// of two that brings the largest factor met so far to 2^12 .. 2^15: gradients
// have any size, and binary16 loses bits below 2^-14.  The sum is rescaled when
// a factor outgrows it and divided by the scale at the end.
template <typename T, int HD>
struct ScaledSum {
  floatx16 acc[HD / 32];
  float scale;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int db = 0; db < HD / 32; ++db) acc[db] = zero16();
    scale = sizeof(T) == 2 ? 0x1p100f : 1.f;
  }
  __device__ __forceinline__ void add(const char* tile, int row0, floatx16 d) {
    if constexpr (sizeof(T) == 2) {
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, __builtin_fabsf(d[e]));
      top = pair_max(top);
      const bool over = top * scale > 32768.f;
      if (__any(over)) {
        const int e = clamp_int(12 - __builtin_amdgcn_frexp_expf(top), -100, 100);
        const float next = over ? __builtin_ldexpf(1.f, e) : scale;
        const float f = next / scale;
        scale = next;
#pragma unroll
        for (int db = 0; db < HD / 32; ++db)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[db][i] *= f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) d[e] *= scale;
    }
    mma_cols<T, HD>(tile, row0, ColFrag<T>(d), acc);
    reads_ahead<Reads<T, HD>::COL, Reads<T, HD>::COL_MMA, 8>();
  }
};

// Whether two lanes of a half that count hold the same value.
__device__ __forceinline__ bool repeats(int v, bool counts) {
  bool same = false;
  const int tid = unknown_thread();  // or its 31 neighbours are kept, in scratch memory
#pragma unroll
  for (int d = 1; d < 32; ++d) {
    const int from = (tid & 32) | ((tid + d) & 31);
    same |= __shfl(v, from) == v && __shfl((int)counts, from) != 0;
  }
  return __any(same && counts);
}

// Adds v[e] to the sum of offset off[e]; clamped ones to below and above.  hist
// has one place more than offsets, where the additions of clamped ones go, and
// those of lanes without a query (width 0, v zero): they must not write over a
// sum that another lane adds to.
__device__ __forceinline__ void add_offsets(float* hist, const int (&off)[16], const floatx16& v,
                                            int width, int lane_width, bool repeated, float& below,
                                            float& above) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    below += off[e] < 0 ? v[e] : 0.f;
    above += off[e] >= width ? v[e] : 0.f;
  }
  if (repeated) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if ((unsigned)off[e] < (unsigned)width)
        __hip_atomic_fetch_add(hist + off[e], v[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float* at = hist + ((unsigned)off[e] < (unsigned)lane_width ? off[e] : width);
      *at += v[e];
      wave_order();
    }
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// The same for blocks whose offsets follow from indices (result row k, lane q:
// offset base + k - q): the sums along their 63 diagonals.  Each lane writes its
// sixteen values to row q of a scratch tile, at column k - q + 31 (put); then
// sixteen lanes sum four columns each, the four groups of sixteen a quarter of the
// rows each, and meet in registers, a column a lane (finish).  A wave's blocks
// follow each other 32 offsets apart, so that the upper 32 columns go on in the
// lower ones of the next block: they are carried in a register, and a column is
// written and never read.  The cells beside a row's 32 values are never written
// and stay zero.  (Sixteen dependent reads, adds and writes a block made the query
// pass of packed prompts a third slower.)
constexpr int DIAG_PITCH = 64, DIAG = 32 * DIAG_PITCH;  // floats
struct Diagonals {
  float carry;
  __device__ __forceinline__ void put(float* scratch, const floatx16& v) const {
    const int lane = threadIdx.x & 63, q = lane & 31, h = lane >> 5;
    float* mine = scratch + q * (DIAG_PITCH - 1) + 31 + 4 * h;
#pragma unroll
    for (int e = 0; e < 16; ++e) mine[8 * (e >> 2) + (e & 3)] = v[e];
    wave_order();
  }
  __device__ __forceinline__ void finish(float* hist, const float* scratch) {
    const int lane = threadIdx.x & 63, group = lane >> 4, col = 4 * (lane & 15);
    const float* rows = scratch + 8 * group * DIAG_PITCH + col;
    floatx4 sum = *reinterpret_cast<const floatx4*>(rows);
#pragma unroll
    for (int r = 1; r < 8; ++r) sum += *reinterpret_cast<const floatx4*>(rows + r * DIAG_PITCH);
    wave_order();
    // rows of 16 lanes: 0 and 1, 2 and 3; then the halves.  Group g is left with column g.
    const float a = row_pair(sum[0], sum[1]), b = row_pair(sum[2], sum[3]);
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(int, a), __builtin_bit_cast(int, b),
                                                    false, false);
    const float total = __builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]) + carry;
    hist[col + group] = total;
    carry = __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, total), 0x128, 0xf, 0x3, false));
  }
  // x summed over two rows in the even one, y in the odd one
  static __device__ __forceinline__ float row_pair(float x, float y) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(int, x), __builtin_bit_cast(int, y),
                                                    false, false);
    return __builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]);
  }
};

// Sums of `copies` of hist, `stride` apart, and of the waves' clamped ends, through
// LDS `ends` of 2 NW binary64 values that nothing else uses, to out.
template <int NW>
__device__ __forceinline__ void join_offsets(const float* hist, int copies, int stride, int width,
                                             double low, double high, double* ends, float* out) {
  const int wave = threadIdx.x >> 6;
  low = wave_sum(low);
  high = wave_sum(high);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    ends[wave] = low;
    ends[NW + wave] = high;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += 64 * NW) {
    double v = 0.0;
    for (int n = 0; n < copies; ++n) v += hist[n * stride + i];
#pragma unroll
    for (int n = 0; n < NW; ++n) {
      if (i == 0) v += ends[n];
      if (i == width - 1) v += ends[NW + n];
    }
    out[i] = (float)v;
  }
}

}  // namespace
}  // namespace attn
}  // namespace eql
