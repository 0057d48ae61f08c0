// Attention, backward (included by one file per type).
//
// Two passes recompute the scores from lse instead of storing them.  The first
// is the forward pass's: a work-group keeps 32 NW queries of one head, walks the
// keys, and sums dq; it also computes delta for the second pass and, of the bias
// table, the sum of ds over every offset.  The second keeps 32 NW keys of one
// key/value head, walks the queries of all heads of its group, and sums dk and
// dv in registers, so that shared heads need no further sum.  Both products of a
// pass with p and ds take them from the score registers.  Seven products of the
// size of the forward's instead of five in one pass, where dq would have to be
// summed by atomics, whose order would change the last bits.
//
// The sums over offsets: attn_sums.h.
//
// Measured (kernel times, steady state): 16 packed documents of 33 to 2048 tokens, 12
// heads of 64 on 4, causal with a bias, binary16: 110 us queries (76 us without the
// bias: its sums, and LDS for two work-groups a compute unit where three would run) +
// 126 us keys (118); 67.5 GFLOP of five products, 94.5 of the seven: 400 TFLOP/s.  16
// full sequences of 2048: 570 TFLOP/s (five products), causal 420.  64 images of 197
// tokens, 6 heads of 64, binary32: 80 + 102 us (9.5 GFLOP of five products, 20 of seven
// on 197 tokens padded to 224 queries or 256 keys: 110 TFLOP/s of 152 by the matrix
// cores).
#pragma once

#include "attn_device.h"
#include "attn_short.h"
#include "attn_sums.h"

namespace eql {
namespace attn {
namespace {

template <typename T, int HD, int NW>
struct BwdLds {
  static constexpr int TILES = 4 * Tile<T, HD>::BYTES;  // two buffers of two tiles
  static constexpr int ROWS = 2 * 4 * Tile<T, HD>::ROWS; // one value a row, two buffers
};

// Waves a SIMD that the registers of the query pass are held to, as in the forward
// pass: the most that need little or no scratch memory.
template <typename T, int HD, int NW, int BIAS>
struct BwdWaves {
  static constexpr bool three = sizeof(T) == 2 && (HD == 32 || (HD == 64 && NW == 4 && BIAS != BIAS_POSITIONS));
  // dimension 128 with the sums over offsets: their LDS leaves one work-group anyway;
  // two waves a work-group hold twice the next tile's rows each (512 sequences of 40
  // to 64 tokens, 8 heads on 2, no bias: 92 us, with 200 bytes of scratch 133 us)
  static constexpr int q = three ? 3 : HD == 128 && (sizeof(T) == 4 || BIAS != BIAS_NONE || NW == 2) ? 1 : 2;
};

template <typename T, int HD, int NW, int BIAS>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(BwdWaves<T, HD, NW, BIAS>::q))) void k_attn_bwd_q(const BwdArgs a) {
  typedef Tile<T, HD> Tl;
  typedef BwdLds<T, HD, NW> Lds;
  constexpr int BN = Tl::ROWS, KB = Tl::BLOCKS, ROWS = 32 * NW, NT = 64 * NW;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const Common& c = a.c;
  Where w;
  if (!locate(c, w)) return;
  const int head = w.hk * c.G + w.rest % c.G, tile = a.tiles - 1 - w.rest / c.G;
  const int width = 2 * c.span + 1;

  int q0, lq, k0, lk;
  bounds(c.cu_q, w.seq, c.total_q, q0, lq);
  bounds(c.cu_k, w.seq, c.total_k, k0, lk);
  const int r0 = tile * ROWS;
  const int rows = lq - r0 < ROWS ? lq - r0 : ROWS;
  float* hist_out = nullptr;
  if constexpr (BIAS != BIAS_NONE) {
    if (a.hist != nullptr) {
      // the tile's slot; the last tile, or the first one of an empty sequence, clears
      // the slot behind it that is no other's
      const int64_t slot = (int64_t)(q0 / ROWS) + w.seq + tile, pitch = (int64_t)c.H * width;
      hist_out = a.hist + slot * pitch + (int64_t)head * width;
      const bool first = tile == 0 && lq == 0, last = rows > 0 && r0 + ROWS >= lq;
      const int64_t next = slot + (last ? 1 : 0);
      if ((first || last) && next < (int64_t)((q0 + lq) / ROWS) + w.seq + 1)
        for (int i = threadIdx.x; i < width; i += NT) a.hist[next * pitch + (int64_t)head * width + i] = 0.f;
    }
  }
  if (rows <= 0) return;
  const int shift = lk - lq;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int token = r0 + wave * 32 + (lane & 31);
  const bool valid = token - r0 < rows;
  auto sees = [&](int t) { return !c.causal ? lk : clamp_int(t + shift + 1, 0, lk); };
  const int klim = valid ? sees(token) : 0;
  const int wrow0 = wave * 32, wrow1 = wrow0 + 31 < rows - 1 ? wrow0 + 31 : rows - 1;
  const bool working = wrow0 < rows;
  const int tok0 = r0 + wrow0, tok1 = r0 + wrow1;
  const int wmin = working ? sees(tok0) : 0, wmax = working ? sees(tok1) : 0;
  const int t1 = (sees(r0 + rows - 1) + BN - 1) / BN;

  RowFrag<T, HD> qf, df;
  const int64_t tok = q0 + token;
  qf.load(a.q.data + (tok * a.q.ts + (int64_t)head * a.q.hs) * Tl::ES, c.dim, valid);
  df.load(a.dout.data + (tok * a.dout.ts + (int64_t)head * a.dout.hs) * Tl::ES, c.dim, valid);
  RowFrag<T, HD> of;
  of.load(a.o.data + (tok * a.o.ts + (int64_t)head * a.o.hs) * Tl::ES, c.dim, valid);
  const int64_t row_at = (int64_t)head * c.total_q + tok;
  float lse = valid ? a.lse[row_at] : -EQL_INF;
  if (lse == -EQL_INF) lse = EQL_INF;  // rows that saw nothing: every p is 2^-inf

  ScaledSum<T, HD> dq;
  dq.clear();
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
  // All first loads on their way before the bias's, which follow each other; at
  // dimension 128 after delta, since the registers do not hold them beside o.
  if (HD < 128 && t1 > 0) fetch(0);

  int* pos = reinterpret_cast<int*>(smem + Lds::TILES);
  float* lut = reinterpret_cast<float*>(smem + Lds::TILES + (BIAS == BIAS_POSITIONS ? Lds::ROWS : 0));
  // sums over offsets: a copy a wave of the padded offsets, and a scratch tile a
  // wave; or a copy a half of a wave, with the place of clamped ones
  const int bw = bias_width<BIAS>(c.span);
  float* hists = lut + (bw + 3) / 4 * 4;
  constexpr int COPIES = BIAS == BIAS_INDEX ? NW : 2 * NW;
  const int stride = BIAS == BIAS_INDEX ? (bw + 3) / 4 * 4 : width + 1;
  float* hist = hists + (BIAS == BIAS_INDEX ? wave : wave * 2 + h) * stride;
  float* scratch = hists + COPIES * stride + wave * DIAG;
  // Sums of clamped offsets: in a long sequence nearly all of them, with both
  // signs, so the blocks' sums are added in binary64.
  double low = 0.0, high = 0.0;
  int pq = token + shift;
  bool repeated = false;
  Diagonals diagonals = {0.f};
  if constexpr (BIAS != BIAS_NONE) {
    fill_bias<T, BIAS>(lut, c, head, 1);
    if (hist_out != nullptr)
      for (int i = threadIdx.x; i < COPIES * stride + (BIAS == BIAS_INDEX ? NW * DIAG : 0); i += NT)
        hists[i] = 0.f;
    if constexpr (BIAS == BIAS_POSITIONS) {
      pq = valid ? c.pos_q[tok] : 0;
      repeated = hist_out != nullptr && repeats(pq, valid);
    }
  }

  float delta = 0.f;
  {
#pragma unroll
    for (int s = 0; s < Tl::STEPS; ++s) {
      typedef T chunk __attribute__((ext_vector_type(16 / sizeof(T))));
      const chunk x = __builtin_bit_cast(chunk, of.c[s]), y = __builtin_bit_cast(chunk, df.c[s]);
#pragma unroll
      for (int e = 0; e < Tl::EPC; ++e) delta = __builtin_fmaf((float)x[e], (float)y[e], delta);
    }
    delta = pair_sum(delta);
    if (valid && h == 0) a.delta[row_at] = delta;
  }

  if (HD == 128 && t1 > 0) fetch(0);

  for (int t = 0; t < t1; ++t) {
    char* tk = smem + (t & 1) * 2 * Tl::BYTES;
    char* tv = tk + Tl::BYTES;
    int* tp = pos + (t & 1) * BN;
    sk.store(tk);
    sv.store(tv);
    if constexpr (BIAS == BIAS_POSITIONS) {
      if (threadIdx.x < BN) tp[threadIdx.x] = pos_next;
    }
    __syncthreads();  // one a tile: see the forward pass
    if (t + 1 < t1) fetch(t + 1);
    const int key0 = t * BN;
    if (key0 >= wmax) continue;
    int side = 0;  // -1, 1: every offset of the tile is clamped to that end
    if constexpr (BIAS == BIAS_INDEX) {
      if (key0 + BN - 1 - (tok0 + shift) <= -c.span) side = -1;
      else if (key0 - (tok1 + shift) >= c.span) side = 1;
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      floatx16 s = mma_rows<T, HD>(tk, 32 * kb, qf, zero16());
      floatx16 dp = mma_rows<T, HD>(tv, 32 * kb, df, zero16());
      reads_ahead<2 * Reads<T, HD>::ROW, 2 * Reads<T, HD>::ROW_MMA, 8>();
      int off[16];
      if constexpr (BIAS != BIAS_NONE) {
        if (side != 0) {
          const float b = lut[side < 0 ? 0 : bw - 1];
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e] = __builtin_fmaf(s[e], c.scale, b);
        } else if constexpr (BIAS == BIAS_INDEX) {
          add_bias_row<1>(s, c.scale, lut + (key0 + 32 * kb + 4 * h - pq + c.span + PAD));
        } else {
#pragma unroll
          for (int e4 = 0; e4 < 4; ++e4) {
            const i32x4 pk = *reinterpret_cast<const i32x4*>(tp + 32 * kb + 8 * e4 + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) off[4 * e4 + e] = pk[e] - pq + c.span;
          }
          add_bias_offsets(s, c.scale, lut, off, width);
        }
      } else {
        scale_scores(s, c.scale);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) dp[e] = __builtin_amdgcn_exp2f((s[e] - lse) * LOG2E) * (dp[e] - delta);
      if (key0 + BN > wmin) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (key0 + 32 * kb + 8 * (e >> 2) + 4 * h + (e & 3) >= klim) dp[e] = 0.f;
      }
      if constexpr (BIAS != BIAS_NONE) {
        if (hist_out != nullptr) {
          if (side == 0 && BIAS == BIAS_INDEX) {
            diagonals.put(scratch, dp);
          } else if (side == 0) {
            float below = 0.f, above = 0.f;
            add_offsets(hist, off, dp, width, valid ? width : 0, repeated, below, above);
            low += below;
            high += above;
          } else {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) sum += dp[e];
            if (side < 0) low += sum;
            else high += sum;
          }
        }
      }
      dq.add(tk, 32 * kb, dp);
      if constexpr (BIAS == BIAS_INDEX) {
        if (hist_out != nullptr && side == 0)
          diagonals.finish(hist + (key0 + 32 * kb - (tok0 + shift) - 31 + c.span + PAD), scratch);
      }
    }
  }

  __syncthreads();  // the tiles are done
  if (working)
    store_rows<T, HD>(smem + wave * 32 * HD * Tl::ES,
                      a.dq.data + ((int64_t)(q0 + tok0) * a.dq.ts + (int64_t)head * a.dq.hs) * Tl::ES, a.dq.ts,
                      rows - wrow0, dq.acc, c.scale / dq.scale, c.dim);
  if constexpr (BIAS != BIAS_NONE) {
    if (hist_out == nullptr) return;
    if constexpr (BIAS == BIAS_INDEX) {  // the padding belongs to the ends
      for (int i = lane; i < PAD; i += 64) {
        low += hist[i];
        high += hist[PAD + width + i];
      }
    }
    // nor are the rows above after its first barrier
    join_offsets<NW>(hists + (BIAS == BIAS_INDEX ? PAD : 0), COPIES, stride, width, low, high,
                     reinterpret_cast<double*>(smem), hist_out);
  }
}

template <typename T, int HD, int QT>
struct KvLds {
  typedef Tile<T, HD, 32 * QT> Tl;
  static constexpr int TILES = 4 * Tl::BYTES;     // two buffers of two tiles
  static constexpr int ROWS = 2 * 4 * Tl::ROWS;   // one value a row, two buffers
};

// KW blocks of 32 keys and QW QB blocks of 32 queries a step, a wave for each key
// block and QB query blocks; the sums of the QW waves of a key block meet at the
// end.  The steps of a work-group follow each other, and the first keys of a long
// causal sequence have the most of them, with shared heads as many times more: one
// wave a key block made the whole pass wait for them (packed documents of up to
// 2048 tokens, three query heads of 64 a key/value head: 211 us, with 60 us of work,
// in binary16, 1254 us for 770 us with two in binary32).  Two query blocks a wave
// and step halve the barriers (155 -> 136 us there).
template <typename T, int HD, int KW, int QW, int QB, int BIAS>
__global__ __launch_bounds__(64 * KW * QW) __attribute__((amdgpu_waves_per_eu(HD <= 64 ? 2 : 1))) void k_attn_bwd_kv(
    const BwdArgs a) {
  typedef KvLds<T, HD, QW * QB> Lds;
  typedef typename Lds::Tl Tl;
  constexpr int BM = Tl::ROWS, KEYS = 32 * KW, NT = 64 * KW * QW;
  // p <= 1 up to the rounding of lse: 2^12 keeps factors down to 2^-26 normal in binary16
  constexpr float SHIFT = sizeof(T) == 2 ? 12.f : 0.f, UNSHIFT = sizeof(T) == 2 ? 0x1p-12f : 1.f;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const Common& c = a.c;
  Where w;
  if (!locate(c, w)) return;
  int q0, lq, k0, lk;
  bounds(c.cu_q, w.seq, c.total_q, q0, lq);
  bounds(c.cu_k, w.seq, c.total_k, k0, lk);
  const int n0 = w.rest * KEYS;  // the first keys of a causal sequence are seen by the most queries
  if (n0 >= lk) return;
  const int shift = lk - lq;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave / KW, block = wave % KW;  // queries of a tile; keys
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int kw = n0 + block * 32;  // the wave's first key
  const int key = kw + (lane & 31);
  const bool valid = key < lk;

  RowFrag<T, HD> kf, vf;
  const int64_t tok = k0 + key;
  kf.load(a.k.data + (tok * a.k.ts + (int64_t)w.hk * a.k.hs) * Tl::ES, c.dim, valid);
  vf.load(a.v.data + (tok * a.v.ts + (int64_t)w.hk * a.v.hs) * Tl::ES, c.dim, valid);
  int pk = key;
  if constexpr (BIAS == BIAS_POSITIONS) pk = valid ? c.pos_k[tok] : 0;

  // query tiles from the first query that sees key n0
  const int qt0 = c.causal && n0 > shift ? (n0 - shift) / BM : 0;
  const int nqt = (lq + BM - 1) / BM - qt0;
  const int steps = nqt > 0 ? nqt * c.G : 0;

  float* row_lse = reinterpret_cast<float*>(smem + Lds::TILES);
  float* row_delta = row_lse + 2 * BM;
  int* row_pos = reinterpret_cast<int*>(row_delta + 2 * BM);
  float* luts = reinterpret_cast<float*>(row_pos + (BIAS == BIAS_POSITIONS ? 2 * BM : 0));
  const int bw = bias_width<BIAS>(c.span);

  ScaledSum<T, HD> dk, dv;
  dk.clear();
  dv.clear();
  Stage<T, HD, NT, BM> sq, sd;
  float lse_next = EQL_INF, delta_next = 0.f;
  int pos_next = 0;
  auto fetch = [&](int head, int first) {
    const int64_t t = q0 + first;
    sq.load(a.q.data + (t * a.q.ts + (int64_t)head * a.q.hs) * Tl::ES, a.q.ts, lq - first, c.dim);
    sd.load(a.dout.data + (t * a.dout.ts + (int64_t)head * a.dout.hs) * Tl::ES, a.dout.ts, lq - first,
            c.dim);
    if (threadIdx.x < BM) {
      lse_next = EQL_INF;  // rows past the end, and rows that saw nothing
      delta_next = 0.f;
      if (first + (int)threadIdx.x < lq) {
        const int64_t at = (int64_t)head * c.total_q + t + threadIdx.x;
        const float v = a.lse[at];
        if (v != -EQL_INF) lse_next = v;
        delta_next = a.delta[at];
        if constexpr (BIAS == BIAS_POSITIONS) pos_next = c.pos_q[t + threadIdx.x];
      }
    }
  };
  if (steps > 0) {
    fetch(w.hk * c.G, qt0 * BM);
    if constexpr (BIAS != BIAS_NONE) fill_bias<T, BIAS>(luts, c, w.hk * c.G, 1);
  }

  int g = 0, qt = 0;
  for (int n = 0; n < steps; ++n) {
    const int buf = n & 1;
    char* tq = smem + buf * 2 * Tl::BYTES;
    char* td = tq + Tl::BYTES;
    const float* lut = luts + (g & 1) * bw;
    sq.store(tq);
    sd.store(td);
    if (threadIdx.x < BM) {
      row_lse[buf * BM + threadIdx.x] = lse_next;
      row_delta[buf * BM + threadIdx.x] = delta_next;
      if constexpr (BIAS == BIAS_POSITIONS) row_pos[buf * BM + threadIdx.x] = pos_next;
    }
    __syncthreads();
    if constexpr (BIAS != BIAS_NONE) {
      // the next head's bias, in the place of the last one's: whoever passes a head's
      // first barrier has left the head before
      if (qt == 0 && g + 1 < c.G) fill_bias<T, BIAS>(luts + ((g + 1) & 1) * bw, c, w.hk * c.G + g + 1, 1);
    }
    const int tile0 = (qt0 + qt) * BM;
    if (++qt == nqt) {
      qt = 0;
      ++g;
    }
    if (n + 1 < steps) fetch(w.hk * c.G + g, (qt0 + qt) * BM);
    if (kw >= lk) continue;
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
      const int row0 = 32 * (part * QB + qb), first = tile0 + row0;  // the block's first query
      if (first >= lq || (c.causal && first + 31 + shift < kw)) continue;
      floatx16 s = mma_rows<T, HD>(tq, row0, kf, zero16());
      floatx16 dp = mma_rows<T, HD>(td, row0, vf, zero16());
      reads_ahead<2 * Reads<T, HD>::ROW, 2 * Reads<T, HD>::ROW_MMA, 8>();
      if constexpr (BIAS == BIAS_INDEX) {
        if (kw + 31 - (first + shift) <= -c.span || kw - (first + 31 + shift) >= c.span) {
          const float b = lut[kw < first + shift ? 0 : bw - 1];
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e] = __builtin_fmaf(s[e], c.scale, b);
        } else {
          add_bias_row<-1>(s, c.scale, lut + (pk - (first + 4 * h + shift) + c.span + PAD));
        }
      } else if constexpr (BIAS == BIAS_POSITIONS) {
        int off[16];
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          const i32x4 pq = *reinterpret_cast<const i32x4*>(row_pos + buf * BM + row0 + 8 * e4 + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) off[4 * e4 + e] = pk - pq[e] + c.span;
        }
        add_bias_offsets(s, c.scale, lut, off, 2 * c.span + 1);
      } else {
        scale_scores(s, c.scale);
      }
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const int r = buf * BM + row0 + 8 * e4 + 4 * h;
        const floatx4 l4 = *reinterpret_cast<const floatx4*>(row_lse + r);
        const floatx4 d4 = *reinterpret_cast<const floatx4*>(row_delta + r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[4 * e4 + e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * e4 + e] - l4[e], LOG2E, SHIFT));
          dp[4 * e4 + e] = s[4 * e4 + e] * (dp[4 * e4 + e] - d4[e]);
        }
      }
      if (c.causal && first + shift < kw + 31) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (first + 8 * (e >> 2) + 4 * h + (e & 3) + shift < key) s[e] = dp[e] = 0.f;
      }
      mma_cols<T, HD>(td, row0, ColFrag<T>(s), dv.acc);
      reads_ahead<Reads<T, HD>::COL, Reads<T, HD>::COL_MMA, 8>();
      dk.add(tq, row0, dp);
    }
  }

  // the parts' sums to the first one, in their order, through LDS (the tiles are done)
  constexpr int SUM = HD / 32 * 16 * 64;  // values of a wave
  float* meet = reinterpret_cast<float*>(smem) + block * SUM + lane;
  static_assert((QW == 1 || KW * SUM * 4 <= Lds::TILES) && KW * 32 * HD * Tl::ES <= Lds::TILES,
                "the sums of a part, and the rows to store, fit the tiles");
  const float fk = c.scale * UNSHIFT / dk.scale;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    floatx16(&acc)[HD / 32] = which == 0 ? dk.acc : dv.acc;
    const float f = which == 0 ? fk : UNSHIFT;
#pragma unroll
    for (int db = 0; db < HD / 32; ++db)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[db][e] *= f;
#pragma unroll
    for (int p = 1; p < QW; ++p) {
      __syncthreads();
      if (part == p) {
#pragma unroll
        for (int db = 0; db < HD / 32; ++db)
#pragma unroll
          for (int e = 0; e < 16; ++e) meet[(db * 16 + e) * 64] = acc[db][e];
      }
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int db = 0; db < HD / 32; ++db)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[db][e] += meet[(db * 16 + e) * 64];
      }
    }
    const View& out = which == 0 ? a.dk : a.dv;
    __syncthreads();
    if (part == 0 && kw < lk)
      store_rows<T, HD>(smem + block * 32 * HD * Tl::ES,
                        out.data + ((int64_t)(k0 + kw) * out.ts + (int64_t)w.hk * out.hs) * Tl::ES, out.ts,
                        lk - kw, acc, 1.f, c.dim);
  }
}

template <typename T, int HD, int NW, int BIAS>
hipError_t run_bwd_q(const BwdArgs& a, int64_t grid, hipStream_t st) {
  typedef BwdLds<T, HD, NW> Lds;
  size_t lds = Lds::TILES + (BIAS == BIAS_POSITIONS ? Lds::ROWS : 0);
  if (BIAS != BIAS_NONE) {
    const size_t bw = (bias_width<BIAS>(a.c.span) + 3) / 4 * 4;
    lds += bw * 4;
    if (a.hist != nullptr)
      lds += BIAS == BIAS_INDEX ? NW * (bw + DIAG) * 4 : (size_t)2 * NW * (2 * a.c.span + 2) * 4;
  }
  const auto kernel = k_attn_bwd_q<T, HD, NW, BIAS>;
  const hipError_t e = allow_lds(kernel, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * NW), lds, st, a);
  return hipGetLastError();
}

template <typename T, int HD, int KW, int QW, int QB, int BIAS>
hipError_t run_bwd_kv(const BwdArgs& a, int64_t grid, hipStream_t st) {
  typedef KvLds<T, HD, QW * QB> Lds;
  size_t lds = Lds::TILES + (BIAS == BIAS_POSITIONS ? 3 : 2) * Lds::ROWS;
  if (BIAS != BIAS_NONE) lds += 2 * (size_t)bias_width<BIAS>(a.c.span) * 4;
  const auto kernel = k_attn_bwd_kv<T, HD, KW, QW, QB, BIAS>;
  const hipError_t e = allow_lds(kernel, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * KW * QW), lds, st, a);
  return hipGetLastError();
}

template <typename T, int HD, int BIAS>
hipError_t run_bwd(BwdArgs a, const BwdShape& s, hipStream_t st) {
  hipError_t e;
  if (s.tiles_q > 0) {
    const int64_t grid = spread(a.c, (int64_t)a.c.G * s.tiles_q, s.tiles_q == 1);
    if (grid <= 0) return hipErrorInvalidValue;
    a.tiles = s.tiles_q;
    e = s.waves_q == 2 ? run_bwd_q<T, HD, 2, BIAS>(a, grid, st) : run_bwd_q<T, HD, 4, BIAS>(a, grid, st);
    if (e != hipSuccess) return e;
  }
  if (s.tiles_k == 0) return hipSuccess;
  const int64_t grid = spread(a.c, s.tiles_k, s.tiles_k == 1);
  if (grid <= 0) return hipErrorInvalidValue;
  if constexpr (sizeof(T) == 2) {
    if constexpr (HD <= 64) {
      if (s.keys == 128) return run_bwd_kv<T, HD, 4, 1, 2, BIAS>(a, grid, st);
      return run_bwd_kv<T, HD, 2, 2, 2, BIAS>(a, grid, st);
    } else {
      if (s.keys == 128) return run_bwd_kv<T, HD, 4, 1, 2, BIAS>(a, grid, st);
      return run_bwd_kv<T, HD, 2, 2, 1, BIAS>(a, grid, st);
    }
  } else {
    if (s.keys == 64) return run_bwd_kv<T, HD, 2, 2, 1, BIAS>(a, grid, st);
    return run_bwd_kv<T, HD, 4, 1, 1, BIAS>(a, grid, st);
  }
}

template <typename T, int HD>
hipError_t run_bwd_bias(const BwdArgs& a, const BwdShape& s, hipStream_t st) {
  if (a.c.buckets == 0) return run_bwd<T, HD, BIAS_NONE>(a, s, st);
  if (a.c.pos_q == nullptr) return run_bwd<T, HD, BIAS_INDEX>(a, s, st);
  return run_bwd<T, HD, BIAS_POSITIONS>(a, s, st);
}

template <typename T>
hipError_t launch_bwd(const BwdArgs& a, const BwdShape& s, hipStream_t st) {
  if (s.chunks > 0) {
    if constexpr (sizeof(T) == 2) {
      if (a.c.dim > 32) return launch_short_bwd<T, 64>(a, st);
    }
    return launch_short_bwd<T, 32>(a, st);
  }
  if (a.c.dim <= 32) return run_bwd_bias<T, 32>(a, s, st);
  if (a.c.dim <= 64) return run_bwd_bias<T, 64>(a, s, st);
  return run_bwd_bias<T, 128>(a, s, st);
}

}  // namespace
}  // namespace attn
}  // namespace eql
