// Layer norm over a token's channels and group values: forward and backward.
//
//     forward   y = (x - mean) rstd gamma[c] + beta[c]     rstd = 1 / sqrt(var + eps)
//     backward  xhat = (x - mean) rstd, g = dy gamma[c]
//               dx = rstd (g - avg(g) - xhat avg(g xhat))
//               dgamma[c] = sum dy xhat, dbeta[c] = sum dy   (rows and group values)
//
// Both passes are bound by HBM bytes (a few operations per value), so each
// value is loaded once and kept in registers until its row's sums are known: the
// variance is the mean square of the differences, not a difference of squares.
// A row is spread over LPR lanes with NV vectors of four values a lane: LPR is a
// power of two up to one wave (several rows a wave) for short rows and a whole
// work-group of 256 or 512 lanes for long ones.  Work-groups walk the rows
// with a fixed stride and load the next row before they reduce the present one.
// A lane keeps the same columns for every row it sees, so its gamma and beta
// are loaded once, and in the backward pass it sums dgamma and dbeta of its
// columns in registers; the work-group then joins its rows and a channel's T
// group values in LDS in a fixed order and writes one partial per channel, and
// a second launch adds the partials, again in a fixed order (atomics would make
// the last bits depend on timing).
//
// Measured (kernel times, steady state), binary16: 12608 rows of 384 forward 8.4 us
// (19.5 MB) and backward 12.1 + 3.8 us (29.2 MB) from the memory-side cache, where 64
// rows take 2.4 us: 10.4 and 20.0 + 3.8 us in binary32; 200704 rows of 768 backward 166 +
// 5 us (926 MB: 5.4 TB/s, the rate of a large copy), binary32 348 + 5 us.  12608 rows of
// 4096: 49 us forward (4.3 TB/s), 62 + 5 us backward (5.0 TB/s).  Above 8192 features the
// backward pass does not fit the registers (4096 rows of 16384: 207 + 6 us, 1.9 TB/s).
#include <type_traits>

#include "eqnorm_internal.h"

#include "eql_device.h"

namespace eql {
namespace {

constexpr int WG = 256;

// Values a lane holds side by side, in both types: 16 bytes of binary32.  With
// 16 bytes of binary16 a lane's eight columns, and their gamma and sums in
// binary32, took 300 registers in the backward pass at 768 features (one wave a
// SIMD, 442 us at 200704 rows).
constexpr int VN = 4;

template <typename T>
struct Vec {
  // rows of an odd size start at any element, and the hardware loads a vector
  // from any element address
  typedef T raw __attribute__((ext_vector_type(VN), aligned(sizeof(T))));
  typedef uint32_t bits __attribute__((ext_vector_type(VN * sizeof(T) / 4)));
};

// Values f0 .. f0 + VN - 1 of a row of F, as stored (converted where they are
// used, so that a row waits in half the registers in binary16): zeros past the
// row's end.
template <typename T>
__device__ __forceinline__ typename Vec<T>::bits load_row(const T* row, int f0, int F) {
  typename Vec<T>::raw v;
  if (f0 + VN <= F) {
    v = *reinterpret_cast<const typename Vec<T>::raw*>(row + f0);
  } else {
#pragma unroll
    for (int e = 0; e < VN; ++e) v[e] = f0 + e < F ? row[f0 + e] : (T)0.f;
  }
  return __builtin_bit_cast(typename Vec<T>::bits, v);
}

template <typename T>
__device__ __forceinline__ float value(const typename Vec<T>::bits& v, int e) {
  return (float)__builtin_bit_cast(typename Vec<T>::raw, v)[e];
}

template <typename T>
__device__ __forceinline__ void store_row(T* row, int f0, int F, const float (&v)[VN]) {
  if (f0 + VN <= F) {
    typename Vec<T>::raw r;
#pragma unroll
    for (int e = 0; e < VN; ++e) r[e] = (T)v[e];
    *reinterpret_cast<typename Vec<T>::raw*>(row + f0) = r;
  } else {
#pragma unroll
    for (int e = 0; e < VN; ++e)
      if (f0 + e < F) row[f0 + e] = (T)v[e];
  }
}

// Per-channel parameter at values f0 .. f0 + VN - 1 of a row (past its end: any).
// Loads without conditions, so that they are all on their way at once.
template <typename T>
__device__ __forceinline__ void load_channels(const T* p, int f0, int F, int group, float other,
                                              float (&v)[VN]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < VN; ++e) v[e] = other;
    return;
  }
  const int first = f0 < F ? f0 : F - 1;
  int c = first / group, r = first - c * group;
  if (group % VN == 0) {  // the values of a vector share a channel
    v[0] = (float)p[c];
#pragma unroll
    for (int e = 1; e < VN; ++e) v[e] = v[0];
    return;
  }
  const int last = F / group - 1;
  T t[VN];
#pragma unroll
  for (int e = 0; e < VN; ++e) {
    t[e] = p[c < last ? c : last];
    const bool next = ++r == group;
    r = next ? 0 : r;
    c += next ? 1 : 0;
  }
#pragma unroll
  for (int e = 0; e < VN; ++e) v[e] = (float)t[e];
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true);
  return v + __builtin_bit_cast(float, o);
}

// Sum over the LPR lanes of a row, in all of them (a butterfly: every lane adds
// the same pairs, so all hold the same bits).  Rows of a whole work-group go on
// through LDS; `slot` alternates so that one barrier a sum is enough.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* lds, int& slot) {
  v = dpp_add<0xB1>(v);                                  // lanes 1 apart
  v = dpp_add<0x4E>(v);                                  // 2 apart
  v = dpp_add<0x141>(v);                                 // the other four of eight
  if constexpr (LPR >= 16) v = dpp_add<0x140>(v);        // the other eight of sixteen
  if constexpr (LPR >= 32) v += __shfl_xor(v, 16);
  if constexpr (LPR >= 64) v += __shfl_xor(v, 32);
  if constexpr (LPR > 64) {
    constexpr int W = LPR / 64;
    float* s = lds + slot * W;
    slot = slot == 3 ? 0 : slot + 1;
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += s[w];
  }
  return v;
}

template <typename T, int LPR, int NV>
__global__ __launch_bounds__(LPR > WG ? LPR : WG) void k_norm_fwd(
    const T* x, const T* gamma, const T* beta, T* y, float* mean_out, float* rstd_out, int64_t N,
    int F, int group, float eps) {
  typedef typename Vec<T>::bits Bits;
  constexpr int BLOCK = LPR > WG ? LPR : WG, RPB = BLOCK / LPR;
  constexpr bool AHEAD = LPR < 512;  // up to 32 values a lane leave no registers for a second row
  __shared__ float lds[LPR > 64 ? 4 * LPR / 64 : 1];
  int slot = 0;
  const int lane = threadIdx.x % LPR;
  const float width = (float)F;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  Bits cur[NV], next[NV];
  if (row < N) {
#pragma unroll
    for (int i = 0; i < NV; ++i) cur[i] = load_row(x + row * F, (lane + LPR * i) * VN, F);
  }
  float g[NV][VN], b[NV][VN];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_channels(gamma, (lane + LPR * i) * VN, F, group, 1.0f, g[i]);
    load_channels(beta, (lane + LPR * i) * VN, F, group, 0.0f, b[i]);
  }
  for (; row < N; row += step) {
    if (AHEAD && row + step < N) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        next[i] = load_row(x + (row + step) * F, (lane + LPR * i) * VN, F);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VN; ++e) s += value<T>(cur[i], e);
    // a quotient, not a product with 1 / F, which the compiler would merge into
    // x - mean unrounded: a row of equal values then has differences of zero
    const float mean = row_sum<LPR>(s, lds, slot) / width;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VN; ++e) {
        const float d = value<T>(cur[i], e) - mean;
        q = (lane + LPR * i) * VN + e < F ? __builtin_fmaf(d, d, q) : q;
      }
    const float rstd = 1.0f / sqrtf(row_sum<LPR>(q, lds, slot) / width + eps);
    if (lane == 0) {
      if (mean_out != nullptr) mean_out[row] = mean;
      if (rstd_out != nullptr) rstd_out[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[VN];
#pragma unroll
      for (int e = 0; e < VN; ++e)
        o[e] = __builtin_fmaf((value<T>(cur[i], e) - mean) * rstd, g[i][e], b[i][e]);
      if ((lane + LPR * i) * VN < F) store_row(y + row * F, (lane + LPR * i) * VN, F, o);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (AHEAD) cur[i] = next[i];
      else if (row + step < N) cur[i] = load_row(x + (row + step) * F, (lane + LPR * i) * VN, F);
    }
  }
}

// partial: [work-groups][2][C] (dgamma, dbeta), or nullptr
template <typename T, int LPR, int NV>
__global__ __launch_bounds__(LPR > WG ? LPR : WG) void k_norm_bwd(
    const T* x, const T* dy, const T* gamma, const float* mean_in, const float* rstd_in, T* dx,
    float* partial, int64_t N, int F, int group) {
  typedef typename Vec<T>::bits Bits;
  constexpr int BLOCK = LPR > WG ? LPR : WG, RPB = BLOCK / LPR;
  constexpr bool AHEAD = LPR < 512;  // up to 32 values a lane leave no registers for a second row
  constexpr int COLS = LPR * NV * VN;                 // columns of a row, padded
  constexpr int COPIES = LPR > 64 ? 1 : BLOCK / 64;    // waves that hold the same columns
  __shared__ float lds[LPR > 64 ? 4 * LPR / 64 : 1];
  __shared__ float joined[COPIES * COLS];
  int slot = 0;
  const int lane = threadIdx.x % LPR;
  const float inv = 1.0f / (float)F;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  Bits xc[NV], xn[NV], dc[NV], dn[NV];
  float mean = 0.f, rstd = 0.f, mean_n = 0.f, rstd_n = 0.f;
  if (row < N) {
    mean = mean_in[row];
    rstd = rstd_in[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xc[i] = load_row(x + row * F, (lane + LPR * i) * VN, F);
      dc[i] = load_row(dy + row * F, (lane + LPR * i) * VN, F);
    }
  }
  float g[NV][VN], dg[NV][VN], db[NV][VN];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_channels(gamma, (lane + LPR * i) * VN, F, group, 1.0f, g[i]);
#pragma unroll
    for (int e = 0; e < VN; ++e) dg[i][e] = db[i][e] = 0.f;
  }
  for (; row < N; row += step) {
    if (AHEAD && row + step < N) {
      mean_n = mean_in[row + step];
      rstd_n = rstd_in[row + step];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xn[i] = load_row(x + (row + step) * F, (lane + LPR * i) * VN, F);
        dn[i] = load_row(dy + (row + step) * F, (lane + LPR * i) * VN, F);
      }
    }
    float a = 0.f, q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VN; ++e) {
        // past the row's end dy is zero: both sums and both columns get nothing
        const float xh = (value<T>(xc[i], e) - mean) * rstd, d = value<T>(dc[i], e);
        const float gd = d * g[i][e];
        a += gd;
        q = __builtin_fmaf(gd, xh, q);
        dg[i][e] = __builtin_fmaf(d, xh, dg[i][e]);
        db[i][e] += d;
      }
    a = row_sum<LPR>(a, lds, slot) * inv;
    q = row_sum<LPR>(q, lds, slot) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[VN];
#pragma unroll
      for (int e = 0; e < VN; ++e) {
        const float xh = (value<T>(xc[i], e) - mean) * rstd;
        o[e] = rstd * (__builtin_fmaf(-xh, q, value<T>(dc[i], e) * g[i][e]) - a);
      }
      if ((lane + LPR * i) * VN < F) store_row(dx + row * F, (lane + LPR * i) * VN, F, o);
    }
    if (AHEAD) {
      mean = mean_n;
      rstd = rstd_n;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xc[i] = xn[i];
        dc[i] = dn[i];
      }
    } else if (row + step < N) {
      mean = mean_in[row + step];
      rstd = rstd_in[row + step];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xc[i] = load_row(x + (row + step) * F, (lane + LPR * i) * VN, F);
        dc[i] = load_row(dy + (row + step) * F, (lane + LPR * i) * VN, F);
      }
    }
  }
  if (partial == nullptr) return;
  const int C = F / group;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VN; ++e) {
        float v = which == 0 ? dg[i][e] : db[i][e];
        // rows of one wave first
        if constexpr (LPR <= 8) v = dpp_add<0x128>(v);  // lanes 8 apart
        if constexpr (LPR <= 16) v += __shfl_xor(v, 16);
        if constexpr (LPR <= 32) v += __shfl_xor(v, 32);
        const int col = (lane + LPR * i) * VN + e;
        if (LPR > 64 || (threadIdx.x & 63) < LPR)
          joined[(LPR > 64 ? 0 : threadIdx.x / 64 * COLS) + col] = v;
      }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += BLOCK) {
      float v = 0.f;
      for (int t = 0; t < group; ++t)
#pragma unroll
        for (int w = 0; w < COPIES; ++w) v += joined[w * COLS + c * group + t];
      partial[((int64_t)blockIdx.x * 2 + which) * C + c] = v;
    }
  }
}

// Column sums of the partials [parts][2 C]: a work-group takes 32 columns, its
// 32 slices of 32 lanes every 32nd partial each.
__global__ __launch_bounds__(1024) void k_norm_finish(const float* __restrict__ partial,
                                                      float* __restrict__ dgamma,
                                                      float* __restrict__ dbeta, int parts, int C) {
  __shared__ float s[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float v = 0.f;
  if (col < 2 * C) {
#pragma unroll 4
    for (int p = slice; p < parts; p += 32) v += partial[(int64_t)p * 2 * C + col];
  }
  s[slice][threadIdx.x & 31] = v;
  __syncthreads();
  if (slice == 0 && col < 2 * C) {
    v = 0.f;
#pragma unroll
    for (int p = 0; p < 32; ++p) v += s[p][threadIdx.x];
    if (col < C) {
      if (dgamma != nullptr) dgamma[col] = v;
    } else if (dbeta != nullptr) {
      dbeta[col - C] = v;
    }
  }
}

// Lanes and vectors a lane of a row of V vectors: the fewest idle lanes, and of
// equal ones the fewest vectors a lane.  Up to one wave that leaves a power of
// two of lanes with one vector, or three vectors (widths of 3 * 2^k are usual).
struct Split {
  int lpr, nv;
};
Split split_of(int V) {
  if (V > 1024) return {512, (V + 1023) / 1024 * 2};
  if (V > 256) return {256, (V + 255) / 256};
  if (V > 96) return {64, (V + 63) / 64};
  if (V > 64) return {32, 3};
  if (V > 48) return {64, 1};
  if (V > 32) return {16, 3};
  if (V > 24) return {32, 1};
  if (V > 16) return {8, 3};
  return {V > 8 ? 16 : 8, 1};
}

int rows_per_block(const Split& s) { return s.lpr > WG ? 1 : WG / s.lpr; }

// Work-groups for N rows: at most `most`, and as many as give each of them the same
// number of rows (12608 rows of 384 binary16 features forward: 1576 work-groups, of
// which a fifth waited for a place, took 11.6 us).
int64_t groups_of(const Split& s, int64_t N) {
  return (N + rows_per_block(s) - 1) / rows_per_block(s);
}
int64_t blocks_for(const Split& s, int64_t N, int64_t most) {
  const int64_t groups = groups_of(s, N);
  if (groups == 0) return 0;
  const int64_t turns = (groups + most - 1) / most;
  return (groups + turns - 1) / turns;
}

template <int V>
using Int = std::integral_constant<int, V>;

template <typename F>
hipError_t with_split(const Split& s, F&& f) {
  switch (s.lpr * 16 + s.nv) {
    case 8 * 16 + 1: return f(Int<8>{}, Int<1>{});
    case 8 * 16 + 3: return f(Int<8>{}, Int<3>{});
    case 16 * 16 + 1: return f(Int<16>{}, Int<1>{});
    case 16 * 16 + 3: return f(Int<16>{}, Int<3>{});
    case 32 * 16 + 1: return f(Int<32>{}, Int<1>{});
    case 32 * 16 + 3: return f(Int<32>{}, Int<3>{});
    case 64 * 16 + 1: return f(Int<64>{}, Int<1>{});
    case 64 * 16 + 2: return f(Int<64>{}, Int<2>{});
    case 64 * 16 + 3: return f(Int<64>{}, Int<3>{});
    case 64 * 16 + 4: return f(Int<64>{}, Int<4>{});
    case 256 * 16 + 2: return f(Int<256>{}, Int<2>{});
    case 256 * 16 + 3: return f(Int<256>{}, Int<3>{});
    case 256 * 16 + 4: return f(Int<256>{}, Int<4>{});
    case 512 * 16 + 4: return f(Int<512>{}, Int<4>{});
    case 512 * 16 + 6: return f(Int<512>{}, Int<6>{});
    case 512 * 16 + 8: return f(Int<512>{}, Int<8>{});
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t forward(const eqnorm_plan* p, const void* x, const void* gamma, const void* beta, void* y,
                   float* mean, float* rstd, int64_t N, hipStream_t s) {
  const int F = (int)(p->C * p->T);
  const Split sp = split_of((F + VN - 1) / VN);
  const unsigned grid = (unsigned)blocks_for(sp, N, FWD_BLOCKS);
  return with_split(sp, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, NV = decltype(v)::value;
    hipLaunchKernelGGL((k_norm_fwd<T, L, NV>), dim3(grid), dim3(L > WG ? L : WG), 0, s,
                       (const T*)x, (const T*)gamma, (const T*)beta, (T*)y, mean, rstd, N, F,
                       (int)p->T, (float)p->eps);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t backward(const eqnorm_plan* p, const void* x, const void* dy, const void* gamma,
                    const float* mean, const float* rstd, void* dx, float* dgamma, float* dbeta,
                    int64_t N, void* ws, hipStream_t s) {
  const int F = (int)(p->C * p->T);
  const Split sp = split_of((F + VN - 1) / VN);
  const int parts = norm_parts(p, N);
  float* partial = dgamma != nullptr || dbeta != nullptr ? (float*)ws : nullptr;
  if (parts > 0) {
    const hipError_t e = with_split(sp, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, NV = decltype(v)::value;
      hipLaunchKernelGGL((k_norm_bwd<T, L, NV>), dim3((unsigned)parts), dim3(L > WG ? L : WG), 0, s,
                         (const T*)x, (const T*)dy, (const T*)gamma, mean, rstd, (T*)dx, partial, N,
                         F, (int)p->T);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (dgamma == nullptr && dbeta == nullptr) return hipSuccess;
  hipLaunchKernelGGL(k_norm_finish, dim3((unsigned)((2 * p->C + 31) / 32)), dim3(1024), 0, s,
                     (const float*)ws, dgamma, dbeta, parts, (int)p->C);
  return hipGetLastError();
}

}  // namespace

int norm_parts(const eqnorm_plan* p, int64_t N) {
  const Split sp = split_of(((int)(p->C * p->T) + VN - 1) / VN);
  // many rows: two a compute unit, whose partial sums are fewer (200704 rows of 768
  // binary16 features: 171 us for 181 us); else as many as find a place at once
  // (12608 rows of 384: three even turns, 17 us for 19 us)
  const int64_t most = groups_of(sp, N) > 8 * BWD_BLOCKS ? BWD_BLOCKS * 2 / 3 : BWD_BLOCKS;
  return (int)blocks_for(sp, N, most);
}

hipError_t launch_norm_forward(const eqnorm_plan* p, const void* x, const void* gamma,
                               const void* beta, void* y, float* mean, float* rstd, int64_t N,
                               hipStream_t s) {
  return p->dtype == EQL_F16 ? forward<_Float16>(p, x, gamma, beta, y, mean, rstd, N, s)
                             : forward<float>(p, x, gamma, beta, y, mean, rstd, N, s);
}

hipError_t launch_norm_backward(const eqnorm_plan* p, const void* x, const void* dy,
                                const void* gamma, const float* mean, const float* rstd, void* dx,
                                float* dgamma, float* dbeta, int64_t N, void* ws, hipStream_t s) {
  return p->dtype == EQL_F16
             ? backward<_Float16>(p, x, dy, gamma, mean, rstd, dx, dgamma, dbeta, N, ws, s)
             : backward<float>(p, x, dy, gamma, mean, rstd, dx, dgamma, dbeta, N, ws, s);
}

}  // namespace eql
