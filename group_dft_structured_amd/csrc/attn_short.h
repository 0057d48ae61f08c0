// Attention over short sequences (at most 64 queries and 64 keys, a head of its
// own for every query head, rows of at most 128 bytes): the windows of a vision
// transformer, thousands of them.  Included by one file per type.
//
// Such a sequence is one tile, and the long kernels would spend their time on
// its chain of loads (offsets, bias, tile) and on reading every operand twice in
// the backward pass.  Here a work-group of two waves keeps its head and walks
// sequences chunk, chunk + chunks, ...: it loads the next sequence's rows into
// registers while it works on the present one, keeps the bias of its 32 x 64
// scores a wave in registers for as long as the positions stay the same, and in
// the backward pass sums ds in registers over the sequences just as long, before
// the sums go to their offsets.  The backward pass reads every operand once and
// computes every score once: a wave takes 32 queries against all keys (dq, and p
// and ds to LDS), then 32 keys against all queries (dk and dv from p and ds).
//
// Measured (kernel times, steady state), 4096 windows of 49 tokens, 6 heads of 32, bias
// over the grid, binary16: forward 71 us (313 MB: 4.4 TB/s; the long kernel 160 us),
// backward 174 us (621 MB: 3.6 TB/s; the long passes 490 us); binary32 163 us and 539
// us (two work-groups a compute unit by their LDS).  The forward pass is bound by its loads and
// stores of 64 bytes a row and head; the backward pass by the instructions around
// its small products: 49 tokens fill 59% of a 64 x 64 tile.  Four waves of 32 x 32
// scores, with four barriers a sequence instead of three: 201 us.
#pragma once

#include "attn_device.h"
#include "attn_sums.h"

namespace eql {
namespace attn {
namespace {

constexpr int SHORT = 64;  // rows of a tile

struct Span {  // a sequence's tokens
  int q0, lq, k0, lk;
  __device__ __forceinline__ int nq() const { return lq < SHORT ? lq : SHORT; }
  __device__ __forceinline__ int nk() const { return lk < SHORT ? lk : SHORT; }
};

// A sequence's offsets on their way: vector loads, although they are uniform.  The
// wait for a scalar load is the wait for all LDS reads too, so a scalar load ahead
// would hold up every product of the present sequence.
struct SpanLoad {
  int q[2], k[2];
  __device__ __forceinline__ void start(const Common& c, int seq) {
    const int bytes = (c.seqs + 1) * 4;
    const Buffer bq = __builtin_amdgcn_make_buffer_rsrc(const_cast<int32_t*>(c.cu_q), (short)0, bytes, 0x00020000);
    const Buffer bk = __builtin_amdgcn_make_buffer_rsrc(const_cast<int32_t*>(c.cu_k), (short)0, bytes, 0x00020000);
    const uint32_t at = seq < c.seqs ? (uint32_t)seq * 4 : NO_ROW;  // none: four zeros
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q[i] = __builtin_amdgcn_raw_buffer_load_b32(bq, (int)(at + 4 * i), 0, 0);
      k[i] = __builtin_amdgcn_raw_buffer_load_b32(bk, (int)(at + 4 * i), 0, 0);
    }
  }
  __device__ __forceinline__ Span take(const Common& c) const {
    Span s;
    clip(__builtin_amdgcn_readfirstlane(q[0]), __builtin_amdgcn_readfirstlane(q[1]), c.total_q, s.q0, s.lq);
    clip(__builtin_amdgcn_readfirstlane(k[0]), __builtin_amdgcn_readfirstlane(k[1]), c.total_k, s.k0, s.lk);
    return s;
  }
};

// Word l of `words` words from a uniform address, 0 behind them.  (Addresses of 64
// bits a lane, kept over the loop, went to scratch memory, and their way back waited
// for all loads of the next sequence: 198 us for 182 us.)
__device__ __forceinline__ int lane_word(const void* from, int words, int tid) {
  return __builtin_amdgcn_raw_buffer_load_b32(rows_of<float>(static_cast<const char*>(from), words, 1, 1),
                                              (tid & 63) * 4, 0, 0);
}

// Offsets of the wave's scores (register e of block kb: key 32 kb + row(e, h), the
// lane's query), for the bias and for the sums over offsets.
template <int BIAS>
__device__ __forceinline__ void short_offsets(int (&off)[16], const int* pos, int kb, int pq, int span) {
  const int h = (unknown_thread() >> 5) & 1;
#pragma unroll
  for (int e4 = 0; e4 < 4; ++e4) {
    const int k = 32 * kb + 8 * e4 + 4 * h;
    i32x4 pk = {k, k + 1, k + 2, k + 3};
    if constexpr (BIAS == BIAS_POSITIONS) pk = *reinterpret_cast<const i32x4*>(pos + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) off[4 * e4 + e] = pk[e] - pq + span;
  }
}

// What the wave's offsets and masks depend on: they are kept while it stays.
struct ShortKey {
  int klim, shift, pq, pk;  // of the lane; pk: position of key l
  __device__ __forceinline__ bool differs(int klim_, int shift_, int pq_, int pk_) const {
    return __any(klim != klim_ || shift != shift_ || pq != pq_ || pk != pk_);
  }
};

// Bias and mask of the wave's scores.
template <int BIAS>
__device__ __forceinline__ void short_bias(floatx16 (&bias)[2], const float* lut, const int* pos, int pq,
                                           int span, int klim) {
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    const int left = klim - 32 * kb - 4 * ((unknown_thread() >> 5) & 1);
    int off[16];
    if constexpr (BIAS != BIAS_NONE) short_offsets<BIAS>(off, pos, kb, pq, span);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float b = 0.f;
      if constexpr (BIAS != BIAS_NONE) b = lut[clamp_int(off[e], 0, 2 * span)];
      bias[kb][e] = 8 * (e >> 2) + (e & 3) < left ? b : -EQL_INF;
    }
  }
}

// Work-group id to (chunk of sequences, head): the heads of a chunk on one XCD
// side by side, since short heads share cache lines.
__device__ __forceinline__ bool short_place(const Common& c, int chunks, int& chunk, int& head) {
  const int id = blockIdx.x;
  chunk = id / (8 * c.H) * 8 + (id & 7);
  head = (id >> 3) % c.H;
  return chunk < chunks;
}

template <typename T, int HD, int BIAS>
__global__ __launch_bounds__(128) __attribute__((amdgpu_waves_per_eu(HD * sizeof(T) <= 64 ? 3 : 2))) void k_attn_short_fwd(const FwdArgs a) {
  typedef Tile<T, HD, SHORT> Tl;
  constexpr float SHIFT = sizeof(T) == 2 ? 7.f : 0.f;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const Common& c = a.c;
  int chunk, head;
  if (!short_place(c, a.chunks, chunk, head)) return;
  char *tk = smem, *tv = smem + Tl::BYTES, *tq = smem + 2 * Tl::BYTES, *rows = smem + 3 * Tl::BYTES;
  int* pos = reinterpret_cast<int*>(smem + 4 * Tl::BYTES);
  float* lut = reinterpret_cast<float*>(pos + SHORT);
  if constexpr (BIAS != BIAS_NONE) fill_bias<T, BIAS_POSITIONS>(lut, c, head, 1);

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, h = lane >> 5, row = wave * 32 + (lane & 31);
  SpanLoad next;
  next.start(c, chunk);
  Span now = next.take(c);
  Stage<T, HD, 128, SHORT> sq, sk, sv;
  int pqn = 0, pkn = 0;
  auto fetch = [&](const Span& s) {
    sk.load(a.k.data + ((int64_t)s.k0 * a.k.ts + (int64_t)head * a.k.hs) * Tl::ES, a.k.ts, s.nk(), c.dim);
    sv.load(a.v.data + ((int64_t)s.k0 * a.v.ts + (int64_t)head * a.v.hs) * Tl::ES, a.v.ts, s.nk(), c.dim);
    sq.load(a.q.data + ((int64_t)s.q0 * a.q.ts + (int64_t)head * a.q.hs) * Tl::ES, a.q.ts, s.nq(), c.dim);
    if constexpr (BIAS == BIAS_POSITIONS) {
      if (row < s.nq()) pqn = c.pos_q[s.q0 + row];
      if (lane < s.nk()) pkn = c.pos_k[s.k0 + lane];
    }
  };
  fetch(now);
  next.start(c, chunk + a.chunks);
  ShortKey kept{-1, 0, 0, 0};
  floatx16 bias[2];

  for (int seq = chunk; seq < c.seqs; seq += a.chunks) {
    __syncthreads();  // the sequence before has been read
    sq.store(tq);
    sk.store(tk);
    sv.store(tv);
    if constexpr (BIAS == BIAS_POSITIONS) {
      if (wave == 0) pos[lane] = pkn;
    }
    const int lk = now.nk(), lq = now.nq(), shift = now.lk - now.lq, q0 = now.q0;
    const int pq = BIAS == BIAS_POSITIONS ? pqn : row + shift, pk = pkn;
    __syncthreads();
    now = next.take(c);
    fetch(now);
    next.start(c, seq + 2 * a.chunks);
    if (wave * 32 >= lq) continue;

    const bool valid = row < lq;
    const int klim = c.causal ? clamp_int(row + shift + 1, 0, lk) : lk;
    if (kept.differs(klim, shift, pq, pk)) {
      kept = ShortKey{klim, shift, pq, pk};
      short_bias<BIAS>(bias, lut, pos, pq, c.span, klim);
    }
    RowFrag<T, HD> qf;
    qf.read(tq, 32 * wave);
    floatx16 s[2];
    float m = -EQL_INF, l = 0.f;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      s[kb] = mma_rows<T, HD>(tk, 32 * kb, qf, zero16());
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[kb][e] = __builtin_fmaf(s[kb][e], c.scale, bias[kb][e]);
        m = fmaxf(m, s[kb][e]);
      }
    }
    m = pair_max(m);
    const float base = m == -EQL_INF ? 0.f : m;
    floatx16 acc[HD / 32];
#pragma unroll
    for (int db = 0; db < HD / 32; ++db) acc[db] = zero16();
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[kb][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][e] - base, LOG2E, SHIFT));
        l += s[kb][e];
      }
      mma_cols<T, HD>(tv, 32 * kb, ColFrag<T>(s[kb]), acc);
    }
    reads_ahead<2 * Reads<T, HD>::COL, 2 * Reads<T, HD>::COL_MMA, 8>();
    l = pair_sum(l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    store_rows<T, HD>(rows + wave * 32 * HD * Tl::ES,
                      a.o.data + ((int64_t)(q0 + 32 * wave) * a.o.ts + (int64_t)head * a.o.hs) * Tl::ES, a.o.ts,
                      lq - 32 * wave, acc, inv, c.dim);
    if (a.lse != nullptr && valid && h == 0)
      a.lse[(int64_t)head * c.total_q + q0 + row] =
          l == 0.f ? -EQL_INF : __builtin_fmaf(__builtin_amdgcn_logf(l) - SHIFT, LN2, m);
  }
}

template <typename T, int HD, int BIAS>
__global__ __launch_bounds__(128) __attribute__((amdgpu_waves_per_eu(HD * sizeof(T) <= 64 ? 2 : 1))) void k_attn_short_bwd(const BwdArgs a) {
  typedef Tile<T, HD, SHORT> Tl;
  // p <= 1 up to the rounding of lse: normal in binary16 down to 2^-26
  constexpr float P_SCALE = sizeof(T) == 2 ? 0x1p12f : 1.f;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const Common& c = a.c;
  int chunk, head;
  if (!short_place(c, a.chunks, chunk, head)) return;
  typedef Tile<T, SHORT, SHORT> Sq;  // p and ds: [queries][keys]
  char *tq = smem, *td = smem + Tl::BYTES, *tk = smem + 2 * Tl::BYTES, *tv = smem + 3 * Tl::BYTES;
  char *tp = smem + 4 * Tl::BYTES, *ts = tp + Sq::BYTES;
  float* row_lse = reinterpret_cast<float*>(ts + Sq::BYTES);
  float* row_delta = row_lse + SHORT;
  float* ds_scale = row_lse + 2 * SHORT;  // of each wave's queries
  int* pos_k = reinterpret_cast<int*>(row_lse + 3 * SHORT);
  int* pos_q = pos_k + SHORT;
  int* kept_pos = pos_q + SHORT;  // [2][SHORT]
  double* ends = reinterpret_cast<double*>(kept_pos + 2 * SHORT);
  float* lut = reinterpret_cast<float*>(ends + 4);
  const int width = 2 * c.span + 1;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, h = lane >> 5, row = wave * 32 + (lane & 31);
  float* hist = lut + width + (wave * 2 + h) * (width + 1);
  const bool summing = BIAS != BIAS_NONE && a.hist != nullptr;
  if constexpr (BIAS != BIAS_NONE) {
    fill_bias<T, BIAS_POSITIONS>(lut, c, head, 1);
    if (summing)
      for (int i = threadIdx.x; i < 4 * (width + 1); i += 128) lut[width + i] = 0.f;
  }

  SpanLoad next;
  next.start(c, chunk);
  Span now = next.take(c);
  Stage<T, HD, 128, SHORT> sq, sd, so, sk, sv;
  int lse_n = 0, pqn = 0, pkn = 0;
  auto fetch = [&](const Span& s, int tid) {
    const int64_t q0 = s.q0, k0 = s.k0;
    sq.load(a.q.data + (q0 * a.q.ts + (int64_t)head * a.q.hs) * Tl::ES, a.q.ts, s.nq(), c.dim, tid);
    sd.load(a.dout.data + (q0 * a.dout.ts + (int64_t)head * a.dout.hs) * Tl::ES, a.dout.ts, s.nq(), c.dim, tid);
    so.load(a.o.data + (q0 * a.o.ts + (int64_t)head * a.o.hs) * Tl::ES, a.o.ts, s.nq(), c.dim, tid);
    sk.load(a.k.data + (k0 * a.k.ts + (int64_t)head * a.k.hs) * Tl::ES, a.k.ts, s.nk(), c.dim, tid);
    sv.load(a.v.data + (k0 * a.v.ts + (int64_t)head * a.v.hs) * Tl::ES, a.v.ts, s.nk(), c.dim, tid);
    lse_n = lane_word(a.lse + (int64_t)head * c.total_q + q0, s.nq(), tid);
    if constexpr (BIAS == BIAS_POSITIONS) {
      pqn = lane_word(c.pos_q + q0, s.nq(), tid);
      pkn = lane_word(c.pos_k + k0, s.nk(), tid);
    }
  };
  fetch(now, threadIdx.x);
  next.start(c, chunk + a.chunks);

  // Bias and mask of the wave's scores, and the sums of ds over the sequences that
  // share them; the sums go to their offsets when these change.
  ShortKey kept{-1, 0, 0, 0};
  bool kept_valid = false;
  floatx16 bias[2], sums[2];
  double low = 0.0, high = 0.0;
  sums[0] = sums[1] = zero16();
  auto flush = [&]() {
    if constexpr (BIAS != BIAS_NONE) {
      if (__all(kept.klim < 0)) return;  // nothing yet
      const bool repeated = BIAS == BIAS_POSITIONS && repeats(kept.pq, kept_valid);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        int off[16];
        short_offsets<BIAS>(off, kept_pos + wave * SHORT, kb, kept.pq, c.span);
        float below = 0.f, above = 0.f;
        add_offsets(hist, off, sums[kb], width, kept_valid ? width : 0, repeated, below, above);
        low += below;
        high += above;
        sums[kb] = zero16();
      }
    }
  };

  // a block of p or ds (keys 32 kb .., the wave's queries) to its rows, and the
  // block of queries 32 qb .. and a wave's keys as the second operand of a product
  auto store_block = [&](char* tile, int kb, const floatx16& v, int tid) {
    const int row = wave * 32 + (tid & 31), h = (tid >> 5) & 1;
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4) {
      const floatx4 x = {v[4 * e4], v[4 * e4 + 1], v[4 * e4 + 2], v[4 * e4 + 3]};
      const int key = 32 * kb + 8 * e4 + 4 * h;
      *reinterpret_cast<typename Elem<T>::quad*>(tile + Sq::at(row, key / Sq::EPC) +
                                                 key % Sq::EPC * Sq::ES) = Elem<T>::pack(x);
    }
  };
  auto read_block = [&](const char* tile, int qb, int kb, int tid) {
    ColFrag<T> f;
    if constexpr (sizeof(T) == 2) {
      f.v[0] = read_col16<T, SHORT>(tile, 32 * qb, kb, 0, tid);
      f.v[1] = read_col16<T, SHORT>(tile, 32 * qb, kb, 1, tid);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) f.v[e] = read_col32<SHORT>(tile, 32 * qb, kb, e, tid);
    }
    return f;
  };

  for (int seq = chunk; seq < c.seqs; seq += a.chunks) {
    const int tid = unknown_thread();
    __syncthreads();  // the sequence before has been read
    sq.store(tq, tid);
    sd.store(td, tid);
    sk.store(tk, tid);
    sv.store(tv, tid);
    {
      // delta: products of the chunks that lie in the same thread, summed over the
      // threads of a row
      typedef T chunk_t __attribute__((ext_vector_type(16 / sizeof(T))));
#pragma unroll
      for (int n = 0; n < Stage<T, HD, 128, SHORT>::N; ++n) {
        const chunk_t x = __builtin_bit_cast(chunk_t, so.r[n]), y = __builtin_bit_cast(chunk_t, sd.r[n]);
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < Tl::EPC; ++e) d = __builtin_fmaf((float)x[e], (float)y[e], d);
#pragma unroll
        for (int i = 1; i < Tl::CPR; i *= 2) d += __shfl_xor(d, i);
        if (threadIdx.x % Tl::CPR == 0) row_delta[threadIdx.x / Tl::CPR + n * (128 / Tl::CPR)] = d;
      }
      if (wave == 0) {
        row_lse[lane] = lane < now.nq() ? __builtin_bit_cast(float, lse_n) : -EQL_INF;
        if constexpr (BIAS == BIAS_POSITIONS) {
          pos_k[lane] = pkn;
          pos_q[lane] = pqn;
        }
      }
    }
    const int lk = now.nk(), lq = now.nq(), shift = now.lk - now.lq, pk_lane = pkn;
    const int64_t q0 = now.q0, k0 = now.k0;
    __syncthreads();
    now = next.take(c);
    fetch(now, tid);
    next.start(c, seq + 2 * a.chunks);

    // ---- 32 queries a wave: dq, and ds for the bias ----
    floatx16 dq[HD / 32];
    float scale = 1.f, own = 1.f;  // of ds, for dk and for dq
    if (wave * 32 < lq) {
      const bool valid = row < lq;
      const int pq = BIAS == BIAS_POSITIONS ? pos_q[row] : row + shift;
      const int klim = valid ? (c.causal ? clamp_int(row + shift + 1, 0, lk) : lk) : 0;
      if (kept.differs(klim, shift, pq, pk_lane)) {
        if (summing) flush();
        kept = ShortKey{klim, shift, pq, pk_lane};
        kept_valid = valid;
        if constexpr (BIAS == BIAS_POSITIONS) kept_pos[wave * SHORT + lane] = pk_lane;
        short_bias<BIAS>(bias, lut, pos_k, pq, c.span, klim);
      }
      RowFrag<T, HD> qf, df;
      qf.read(tq, 32 * wave, tid);
      df.read(td, 32 * wave, tid);
      const float delta = row_delta[row];
      float lse = row_lse[row];
      if (lse == -EQL_INF) lse = EQL_INF;  // rows that saw nothing: every p is 2^-inf
      floatx16 ds[2];
      float top = 0.f;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        floatx16 s = mma_rows<T, HD>(tk, 32 * kb, qf, zero16(), tid);
        ds[kb] = mma_rows<T, HD>(tv, 32 * kb, df, zero16(), tid);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p = __builtin_amdgcn_exp2f((__builtin_fmaf(s[e], c.scale, bias[kb][e]) - lse) * LOG2E);
          ds[kb][e] = p * (ds[kb][e] - delta);
          if constexpr (BIAS != BIAS_NONE) sums[kb][e] += ds[kb][e];
          if constexpr (sizeof(T) == 2) top = fmaxf(top, __builtin_fabsf(ds[kb][e]));
          s[e] = p * P_SCALE;
        }
        store_block(tp, kb, s, tid);
      }
      // one power of two for the wave's 32 queries: ds of binary16 in 2^14 .. 2^15
      // at the largest, and normal down to 2^-28 of it, for dk; for dq a query whose
      // own largest would be below 2 gets a power of its own
      bool apart = false;
      if constexpr (sizeof(T) == 2) {
        top = pair_max(top);
        top = top < EQL_INF ? top : 0.f;  // a query of infinities has no say
        const float mine = top;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
        scale = own = __builtin_ldexpf(1.f, clamp_int(15 - __builtin_amdgcn_frexp_expf(top), -100, 100));
        apart = __any(mine > 0.f && mine * 0x1p13f < top);
        if (apart) own = __builtin_ldexpf(1.f, clamp_int(15 - __builtin_amdgcn_frexp_expf(mine), -100, 100));
      }
#pragma unroll
      for (int db = 0; db < HD / 32; ++db) dq[db] = zero16();
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
        for (int e = 0; e < 16; ++e) ds[kb][e] *= scale;
        ColFrag<T> f(ds[kb]);
        store_block(ts, kb, ds[kb], tid);
        if (apart) {
          const float more = own / scale;
#pragma unroll
          for (int e = 0; e < 16; ++e) ds[kb][e] *= more;
          f = ColFrag<T>(ds[kb]);
        }
        mma_cols<T, HD>(tk, 32 * kb, f, dq, tid);
      }
      if (lane == 0) ds_scale[wave] = scale;
    }
    __syncthreads();
    // keys and values are done: their tiles hold the rows to store, each wave's its own
    char* rows = tk + wave * 32 * HD * Tl::ES;
    if (wave * 32 < lq)
      store_rows<T, HD>(rows, a.dq.data + ((q0 + 32 * wave) * a.dq.ts + (int64_t)head * a.dq.hs) * Tl::ES,
                        a.dq.ts, lq - 32 * wave, dq, c.scale / own, c.dim, tid);

    // ---- 32 keys a wave: dk and dv ----
    if (wave * 32 < lk) {
      floatx16 dk[HD / 32], dv[HD / 32];
#pragma unroll
      for (int db = 0; db < HD / 32; ++db) dk[db] = dv[db] = zero16();
#pragma unroll
      for (int qb = 0; qb < 2; ++qb) {
        if (32 * qb >= lq) break;
        mma_cols<T, HD>(td, 32 * qb, read_block(tp, qb, wave, tid), dv, tid);
        floatx16 part[HD / 32];
#pragma unroll
        for (int db = 0; db < HD / 32; ++db) part[db] = zero16();
        mma_cols<T, HD>(tq, 32 * qb, read_block(ts, qb, wave, tid), part, tid);
        const float f = 1.f / ds_scale[qb];
#pragma unroll
        for (int db = 0; db < HD / 32; ++db)
#pragma unroll
          for (int e = 0; e < 16; ++e) dk[db][e] = __builtin_fmaf(part[db][e], f, dk[db][e]);
      }
      store_rows<T, HD>(rows, a.dk.data + ((k0 + 32 * wave) * a.dk.ts + (int64_t)head * a.dk.hs) * Tl::ES,
                        a.dk.ts, lk - 32 * wave, dk, c.scale, c.dim, tid);
      store_rows<T, HD>(rows, a.dv.data + ((k0 + 32 * wave) * a.dv.ts + (int64_t)head * a.dv.hs) * Tl::ES,
                        a.dv.ts, lk - 32 * wave, dv, 1.f / P_SCALE, c.dim, tid);
    }
  }
  if constexpr (BIAS != BIAS_NONE) {
    if (!summing) return;
    flush();
    join_offsets<2>(lut + width, 4, width + 1, width, low, high, ends,
                    a.hist + ((int64_t)chunk * c.H + head) * width);
  }
}

template <typename T, int HD, int BIAS>
hipError_t run_short_fwd(const FwdArgs& a, unsigned grid, hipStream_t st) {
  const size_t lds = 4 * Tile<T, HD, SHORT>::BYTES + SHORT * 4 + (size_t)(2 * a.c.span + 1) * 4;
  const auto kernel = k_attn_short_fwd<T, HD, BIAS>;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(128), lds, st, a);
  return hipGetLastError();
}

template <typename T, int HD, int BIAS>
hipError_t run_short_bwd(const BwdArgs& a, unsigned grid, hipStream_t st) {
  const size_t width = 2 * a.c.span + 1;
  const size_t lds = 4 * Tile<T, HD, SHORT>::BYTES + 2 * Tile<T, SHORT, SHORT>::BYTES + 7 * SHORT * 4 + 4 * 8 +
                     (BIAS == BIAS_NONE ? 0 : width * 4 + (a.hist != nullptr ? 4 * (width + 1) * 4 : 0));
  const auto kernel = k_attn_short_bwd<T, HD, BIAS>;
  const hipError_t e = allow_lds(kernel, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(128), lds, st, a);
  return hipGetLastError();
}

inline unsigned short_grid(int heads, int chunks) { return (unsigned)((chunks + 7) / 8 * 8 * heads); }

template <typename T, int HD>
hipError_t launch_short_fwd(const FwdArgs& a, hipStream_t st) {
  const unsigned grid = short_grid(a.c.H, a.chunks);
  if (a.c.buckets == 0) return run_short_fwd<T, HD, BIAS_NONE>(a, grid, st);
  if (a.c.pos_q == nullptr) return run_short_fwd<T, HD, BIAS_INDEX>(a, grid, st);
  return run_short_fwd<T, HD, BIAS_POSITIONS>(a, grid, st);
}

template <typename T, int HD>
hipError_t launch_short_bwd(const BwdArgs& a, hipStream_t st) {
  const unsigned grid = short_grid(a.c.H, a.chunks);
  if (a.c.buckets == 0) return run_short_bwd<T, HD, BIAS_NONE>(a, grid, st);
  if (a.c.pos_q == nullptr) return run_short_bwd<T, HD, BIAS_INDEX>(a, grid, st);
  return run_short_bwd<T, HD, BIAS_POSITIONS>(a, grid, st);
}

}  // namespace
}  // namespace attn
}  // namespace eql
