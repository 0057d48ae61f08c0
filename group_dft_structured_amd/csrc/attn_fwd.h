// Attention, forward: one pass over a sequence's keys with the running maximum
// and sum of the softmax (included by one file per type).
//
// A work-group of NW waves takes 32 NW query rows of one sequence and head, each
// wave 32 of them; keys and values go through LDS in tiles.  Per tile a wave
// computes the scores transposed (keys x its 32 queries), adds the bias, and
// multiplies exp(score - maximum) from the registers with the transposed values; a lane holds one query's column, so its
// maximum and sum need one exchange between the two halves of the wave.
//
// The maximum moves only when a tile exceeds it by more than 8 ln 2: until then the
// factors are at most 2^8 times 2^SHIFT and the output registers need no
// rescaling.  SHIFT = 7 places binary16 factors in [.., 2^15]: the normal range
// then reaches down to 2^-21 of the largest factor, and a rounding to 11 bits is
// the only loss; the sum of the softmax adds the factors before rounding.
//
// With few query rows (a new token against its cache) the query heads that share
// a key/value head are packed into the rows of one work-group, so keys and values
// are read once, and the keys are split over work-groups that leave maximum, sum
// and unnormalised output for k_attn_join.
//
// Tiles of 64 keys in binary16: two blocks of scores in flight a wave hide each
// other's exponentials; four waves share a tile, so LDS is read once a 128 queries.
// Measured (kernel times, steady state), binary16: 12 packed prompts of 65 to 2048
// tokens, 16 heads of 128 on 4, causal with a bias, 132 us, 126 without the bias (76.7
// GFLOP: 580 TFLOP/s; 16 full sequences of 2048 run at 860 TFLOP/s, causal 760): what
// lacks are the start of a work-group (queries, first tile, bias: 9 us with its end)
// and the unequal lengths.  Binary32: 900 us.  One token for 48 caches of up to 8192,
// 32 heads of 128 on 8: 165 + 6 us (817 MB: 4.9 TB/s, near a copy's 5.1); binary32 300 +
// 6 us (5.4 TB/s).  One token for one cache of 32768, 16 heads of 64 on 4: 11 + 6 us
// (33.6 MB from the memory-side cache; two launches' starts); binary32 27 + 5 us.
#pragma once

#include "attn_device.h"
#include "attn_short.h"

namespace eql {
namespace attn {
namespace {

template <typename T, int HD, int NW>
struct FwdLds {
  static constexpr int BUFS = NW > 1 ? 2 : 1;  // one wave waits for nobody
  static constexpr int TILES = 2 * BUFS * Tile<T, HD>::BYTES;
  static constexpr int POS = BUFS * Tile<T, HD>::ROWS * 4;
};

// Waves a SIMD that the registers are held to (with more than 256 registers a
// wave the products' results go to accumulation registers and are moved back).
// Two waves a work-group hold twice the next tile's rows each: one wave a SIMD
// fewer from dimension 64 on, where they would need scratch memory (512 sequences
// of 40 to 64 tokens, 8 heads of 128 on 2: 4% less time).
template <typename T, int HD, int NW>
struct FwdWaves {
  static constexpr int f16 = (HD == 32 ? 4 : HD == 64 ? 3 : 2) - (NW == 2 && HD >= 64 ? 1 : 0);
  static constexpr int value = NW == 1 ? 1 : sizeof(T) == 2 ? f16 : HD == 128 ? 1 : 2;
};

template <typename T, int HD, int NW, int BIAS>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(FwdWaves<T, HD, NW>::value))) void k_attn_fwd(const FwdArgs a) {
  typedef Tile<T, HD> Tl;
  typedef FwdLds<T, HD, NW> Lds;
  constexpr int BN = Tl::ROWS, KB = Tl::BLOCKS, ROWS = 32 * NW, NT = 64 * NW;
  constexpr float SHIFT = sizeof(T) == 2 ? 7.f : 0.f, SLACK = 5.5f;  // below 8 ln 2
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const Common& c = a.c;
  Where w;
  if (!locate(c, w)) return;
  const int gp = a.packed ? c.G : 1;
  // the last tiles of a causal sequence see the most keys: they go first
  const int split = w.rest % a.splits;
  int rest = w.rest / a.splits;
  const int heads = c.G / gp, head0 = w.hk * c.G + (rest % heads) * gp;
  const int tile = a.tiles - 1 - rest / heads;

  int q0, lq, k0, lk;
  bounds(c.cu_q, w.seq, c.total_q, q0, lq);
  bounds(c.cu_k, w.seq, c.total_k, k0, lk);
  const int r0 = tile * ROWS;
  const int64_t rows64 = (int64_t)lq * gp;
  const int rows = rows64 - r0 < ROWS ? (int)(rows64 - r0) : ROWS;  // rows of this work-group
  if (rows <= 0) return;
  const int shift = lk - lq;  // query i sits at position i + shift of the keys

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, h = lane >> 5;
  // this lane's query
  const int row = r0 + wave * 32 + (lane & 31);
  const bool valid = row - r0 < rows;
  const int token = gp == 1 ? row : row / gp;
  const int g = gp == 1 ? 0 : row - token * gp;
  const int head = head0 + g;
  int klim = 0;  // keys it sees
  if (valid) klim = c.causal && token + shift < lk ? (token + shift + 1 > 0 ? token + shift + 1 : 0) : lk;
  // and the wave's queries: the first one sees the fewest keys, the last one the most
  const int wrow0 = wave * 32, wrow1 = wrow0 + 31 < rows - 1 ? wrow0 + 31 : rows - 1;
  const bool working = wrow0 < rows;
  const int tok0 = (r0 + wrow0) / gp, tok1 = (r0 + wrow1) / gp, tokl = (r0 + rows - 1) / gp;
  auto sees = [&](int t) {
    return !c.causal ? lk : clamp_int(t + shift + 1, 0, lk);
  };
  const int wmin = working ? sees(tok0) : 0, wmax = working ? sees(tok1) : 0;
  const int kend = sees(tokl);
  int t0 = 0, t1 = (kend + BN - 1) / BN;
  if (a.splits > 1) {
    // tiles of the whole sequence are dealt out: every split of a row has its place
    const int per = ((lk + BN - 1) / BN + a.splits - 1) / a.splits;
    t0 = split * per;
    t1 = t1 < t0 + per ? t1 : t0 + per;
  }

  RowFrag<T, HD> qf;
  qf.load(a.q.data + ((int64_t)(q0 + token) * a.q.ts + (int64_t)head * a.q.hs) * Tl::ES, c.dim, valid);

  float* lut = reinterpret_cast<float*>(smem + Lds::TILES + (BIAS == BIAS_POSITIONS ? Lds::POS : 0));
  const int width = bias_width<BIAS>(c.span);
  const float* lut_row = lut + g * width;
  int pq = token + shift;  // position of this lane's query
  if constexpr (BIAS == BIAS_POSITIONS) pq = valid ? c.pos_q[q0 + token] : 0;

  floatx16 acc[HD / 32];
#pragma unroll
  for (int db = 0; db < HD / 32; ++db) acc[db] = zero16();
  float m = -EQL_INF, l = 0.f;

  Stage<T, HD, NT> sk, sv;
  int pos_next = 0;
  const char* kp = a.k.data + ((int64_t)k0 * a.k.ts + (int64_t)w.hk * a.k.hs) * Tl::ES;
  const char* vp = a.v.data + ((int64_t)k0 * a.v.ts + (int64_t)w.hk * a.v.hs) * Tl::ES;
  auto fetch = [&](int t) {
    const int first = t * BN;
    sk.load(kp + (int64_t)first * a.k.ts * Tl::ES, a.k.ts, lk - first, c.dim);
    sv.load(vp + (int64_t)first * a.v.ts * Tl::ES, a.v.ts, lk - first, c.dim);
    if constexpr (BIAS == BIAS_POSITIONS) {
      if (threadIdx.x < BN && first + (int)threadIdx.x < lk) pos_next = c.pos_k[k0 + first + threadIdx.x];
    }
  };
  if (t0 < t1) fetch(t0);
  // behind the loads of the first tile, so that those are on their way meanwhile
  if constexpr (BIAS != BIAS_NONE) fill_bias<T, BIAS>(lut, c, head0, gp);

  for (int t = t0; t < t1; ++t) {
    const int buf = Lds::BUFS == 2 ? (t - t0) & 1 : 0;
    char* tk = smem + buf * 2 * Tl::BYTES;
    char* tv = tk + Tl::BYTES;
    int* tp = reinterpret_cast<int*>(smem + Lds::TILES) + buf * BN;
    // With two buffers, one barrier a tile: whoever passes the barrier of tile t
    // has left tile t - 1, so the buffer of tile t - 1 is free for tile t + 1.
    if constexpr (Lds::BUFS == 1) __syncthreads();
    sk.store(tk);
    sv.store(tv);
    if constexpr (BIAS == BIAS_POSITIONS) {
      if (threadIdx.x < BN) tp[threadIdx.x] = pos_next;
    }
    __syncthreads();
    if (t + 1 < t1) fetch(t + 1);
    const int key0 = t * BN;
    if (key0 >= wmax) continue;

    floatx16 s[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) s[kb] = mma_rows<T, HD>(tk, 32 * kb, qf, zero16());
    reads_ahead<KB * Reads<T, HD>::ROW, KB * Reads<T, HD>::ROW_MMA, 8>();

    // scores with the bias
    if constexpr (BIAS == BIAS_NONE) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) scale_scores(s[kb], c.scale);
    } else {
      bool far = false;
      float fb = 0.f;
      if constexpr (BIAS == BIAS_INDEX) {  // a tile beyond the span on one side has one bias
        if (key0 + BN - 1 - (tok0 + shift) <= -c.span) {
          far = true;
          fb = lut_row[0];
        } else if (key0 - (tok1 + shift) >= c.span) {
          far = true;
          fb = lut_row[width - 1];
        }
      }
      if (far) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[kb][e] = __builtin_fmaf(s[kb][e], c.scale, fb);
      } else if constexpr (BIAS == BIAS_INDEX) {
        const float* at = lut_row + (key0 + 4 * h - pq + c.span + PAD);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) add_bias_row<1>(s[kb], c.scale, at + 32 * kb);
      } else {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          int off[16];
#pragma unroll
          for (int e4 = 0; e4 < 4; ++e4) {
            const i32x4 pk = *reinterpret_cast<const i32x4*>(tp + 32 * kb + 8 * e4 + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) off[4 * e4 + e] = pk[e] - pq + c.span;
          }
          add_bias_offsets(s[kb], c.scale, lut_row, off, width);
        }
      }
    }
    if (key0 + BN > wmin) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (key0 + 32 * kb + 8 * (e >> 2) + 4 * h + (e & 3) >= klim) s[kb][e] = -EQL_INF;
    }

    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[kb][e]);
    top = pair_max(top);
    if (__any(top > m + SLACK)) {
      const float mn = fmaxf(m, top);
      const float f = mn == -EQL_INF ? 1.f : __builtin_amdgcn_exp2f((m - mn) * LOG2E);
      m = mn;
      l *= f;
#pragma unroll
      for (int db = 0; db < HD / 32; ++db)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[db][e] *= f;
    }
    const float base = m == -EQL_INF ? 0.f : m;  // nothing seen: every factor is 2^-inf
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][e] - base, LOG2E, SHIFT));
        s[kb][e] = p;
        l += p;
      }
      mma_cols<T, HD>(tv, 32 * kb, ColFrag<T>(s[kb]), acc);
    }
    reads_ahead<KB * Reads<T, HD>::COL, KB * Reads<T, HD>::COL_MMA, 16>();
  }

  l = pair_sum(l);
  const int64_t out_row = (int64_t)head * c.total_q + q0 + token;
  if (a.splits > 1) {
    if (!valid) return;
    const int64_t at = (int64_t)split * c.H * c.total_q + out_row;
    store_column<float, HD>(reinterpret_cast<char*>(a.part_o + at * c.dim), acc, 1.f, c.dim);
    if (h == 0) {
      a.part_ml[2 * at] = m;
      a.part_ml[2 * at + 1] = l;
    }
    return;
  }
  // a sum of zero: no key was seen (l is at least 2^SHIFT where one was)
  const float inv = l == 0.f ? 0.f : 1.f / l;
  char* out = a.o.data + ((int64_t)q0 * a.o.ts + (int64_t)head0 * a.o.hs) * Tl::ES;
  if (gp == 1) {
    __syncthreads();  // the tiles are done
    if (!working) return;
    store_rows<T, HD>(smem + wave * 32 * HD * Tl::ES, out + (int64_t)(r0 + wrow0) * a.o.ts * Tl::ES, a.o.ts,
                      rows - wrow0, acc, inv, c.dim);
  } else if (valid) {
    store_column<T, HD>(out + ((int64_t)token * a.o.ts + (int64_t)g * a.o.hs) * Tl::ES, acc, inv, c.dim);
  }
  if (a.lse != nullptr && valid && h == 0)
    a.lse[out_row] = l == 0.f ? -EQL_INF : __builtin_fmaf(__builtin_amdgcn_logf(l) - SHIFT, LN2, m);
}

// Joins the splits of every row: a work-group a row.  A lane takes a split for
// the maximum and the weights (at most MAX_SPLITS = 128 of them), then each wave
// every fourth split of the outputs, two values a lane, and the waves' sums are
// added in LDS.  (One wave a row that walked the splits waited for each of them:
// 100 us of 122 us at 128 splits.)
template <typename T>
__global__ __launch_bounds__(256) void k_attn_join(const FwdArgs a, int max_q) {
  const Common& c = a.c;
  constexpr float SHIFT = sizeof(T) == 2 ? 7.f : 0.f;
  __shared__ float weight[MAX_SPLITS], part[4][EQATTN_MAX_DIM];
  const int64_t id = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int head = (int)(id % c.H), token = (int)(id / c.H % max_q), seq = (int)(id / c.H / max_q);
  int q0, lq;
  bounds(c.cu_q, seq, c.total_q, q0, lq);
  if (token >= lq) return;
  const int64_t row = (int64_t)head * c.total_q + q0 + token, stride = (int64_t)c.H * c.total_q;
  float mv[MAX_SPLITS / 64], lv[MAX_SPLITS / 64], m = -EQL_INF;
#pragma unroll
  for (int i = 0; i < MAX_SPLITS / 64; ++i) {
    const int s = lane + 64 * i;
    const bool in = s < a.splits;
    mv[i] = in ? a.part_ml[2 * (s * stride + row)] : -EQL_INF;
    lv[i] = in ? a.part_ml[2 * (s * stride + row) + 1] : 0.f;
    m = fmaxf(m, mv[i]);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
  const float base = m == -EQL_INF ? 0.f : m;
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < MAX_SPLITS / 64; ++i) {
    const float f = lv[i] == 0.f ? 0.f : __builtin_amdgcn_exp2f((mv[i] - base) * LOG2E);  // 0: saw no key
    l = __builtin_fmaf(f, lv[i], l);
    if (wave == 0) weight[lane + 64 * i] = f;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) l += __shfl_xor(l, d);
  __syncthreads();
  const float* po = a.part_o + row * c.dim + 2 * lane;
  float x = 0.f, y = 0.f;
  if (2 * lane < c.dim) {
#pragma unroll 8
    for (int s = wave; s < a.splits; s += 4) {
      // a split that saw no key left zeros
      const float2 v = *reinterpret_cast<const float2*>(po + s * stride * c.dim);
      x = __builtin_fmaf(weight[s], v.x, x);
      y = __builtin_fmaf(weight[s], v.y, y);
    }
    part[wave][2 * lane] = x;
    part[wave][2 * lane + 1] = y;
  }
  __syncthreads();
  if (wave != 0) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = reinterpret_cast<T*>(a.o.data) + (int64_t)(q0 + token) * a.o.ts + (int64_t)head * a.o.hs;
#pragma unroll
  for (int i = 0; i < EQATTN_MAX_DIM / 64; ++i) {
    const int d = lane + 64 * i;
    if (d < c.dim) out[d] = (T)((part[0][d] + part[1][d] + part[2][d] + part[3][d]) * inv);
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[row] = l == 0.f ? -EQL_INF : __builtin_fmaf(__builtin_amdgcn_logf(l) - SHIFT, LN2, m);
}

template <typename T, int HD, int NW, int BIAS>
hipError_t run_fwd(const FwdArgs& a, int64_t grid, hipStream_t st) {
  typedef FwdLds<T, HD, NW> Lds;
  const size_t lds = Lds::TILES + (BIAS == BIAS_POSITIONS ? Lds::POS : 0) +
                     (BIAS == BIAS_NONE ? 0 : (size_t)(a.packed ? a.c.G : 1) * bias_width<BIAS>(a.c.span) * 4);
  const auto kernel = k_attn_fwd<T, HD, NW, BIAS>;
  const hipError_t e = allow_lds(kernel, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * NW), lds, st, a);
  return hipGetLastError();
}

template <typename T, int HD, int NW>
hipError_t run_fwd_bias(const FwdArgs& a, int64_t grid, hipStream_t st) {
  if (a.c.buckets == 0) return run_fwd<T, HD, NW, BIAS_NONE>(a, grid, st);
  if (a.c.pos_q == nullptr) return run_fwd<T, HD, NW, BIAS_INDEX>(a, grid, st);
  return run_fwd<T, HD, NW, BIAS_POSITIONS>(a, grid, st);
}

template <typename T, int HD>
hipError_t run_fwd_waves(const FwdArgs& a, int waves, int64_t grid, hipStream_t st) {
  if (waves == 1) return run_fwd_bias<T, HD, 1>(a, grid, st);
  if (waves == 2) return run_fwd_bias<T, HD, 2>(a, grid, st);
  return run_fwd_bias<T, HD, 4>(a, grid, st);
}

template <typename T>
hipError_t launch_fwd(FwdArgs a, const FwdShape& s, int max_q, hipStream_t st) {
  if (s.chunks > 0) {
    if constexpr (sizeof(T) == 2) {
      if (a.c.dim > 32) return launch_short_fwd<T, 64>(a, st);
    }
    return launch_short_fwd<T, 32>(a, st);
  }
  const int64_t heads = a.packed ? 1 : a.c.G;
  const int64_t grid = spread(a.c, heads * s.tiles * s.splits, s.tiles == 1);
  if (grid <= 0) return hipErrorInvalidValue;
  hipError_t e;
  if (a.c.dim <= 32) e = run_fwd_waves<T, 32>(a, s.waves, grid, st);
  else if (a.c.dim <= 64) e = run_fwd_waves<T, 64>(a, s.waves, grid, st);
  else e = run_fwd_waves<T, 128>(a, s.waves, grid, st);
  if (e != hipSuccess || s.splits == 1) return e;
  const int64_t rows = (int64_t)a.c.seqs * a.c.H * max_q;
  if (rows > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_attn_join<T>), dim3((unsigned)rows), dim3(256), 0, st, a, max_q);
  return hipGetLastError();
}

}  // namespace
}  // namespace attn
}  // namespace eql
