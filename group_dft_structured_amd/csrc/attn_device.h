// Device pieces shared by the attention kernels (gfx950).
//
// Every matrix product runs on the 32 x 32 matrix-core block of eql_device.h,
// whose result has its column in the lane (l % 32) and sixteen rows in the
// lane's registers, row(e, h) = 8 (e / 4) + 4 h + e % 4 with h = l / 32.  Scores
// are computed transposed in the passes that reduce over keys (rows are keys,
// the column is the lane's query), so that softmax statistics are reductions
// inside a lane and across one lane pair, and the score registers are already
// the second operand of the next product: its reduction index may come in any
// order as long as both operands agree, so the order is the one in which the
// result registers hold the rows.  The first operand of that product is the
// transpose of a tile that lies row by row in LDS: ds_read_b64_tr_b16 reads it in
// binary16 (four rows of one column in a lane), single 4-byte reads in binary32.
//
// A tile holds ROWS tokens of HD values (the head dimension padded to 32, 64 or
// 128) in 16-byte chunks; chunk c of row r lies at c ^ swizzle(r), which spreads
// both kinds of reads over the banks.
#pragma once

#include "eql_device.h"
#include "eqattn_internal.h"

namespace eql {
namespace attn {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Scores, their maxima and lse are kept in base e, and only differences of them go
// to base 2: a score and a maximum of the same size then cancel exactly.  (lse times
// log2 e is off by half a unit of its own last place, which at 10^9, a usual mask
// value, is 2^6 in the exponent: gradients of infinity, or of zero.)
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
#define EQL_INF __builtin_inff()

enum { BIAS_NONE = 0, BIAS_INDEX = 1, BIAS_POSITIONS = 2 };

// Work-group id to (sequence, key/value head, rest).  Consecutive ids go to
// consecutive XCDs, each with its own L2, so the ids of one cluster of units,
// which read the same keys and values (or, for heads shorter than a cache line,
// the same lines), are those of one XCD, one cluster after the other.  (All
// clusters' largest pieces of work first balances better, but the keys and values
// of many units do not stay in one L2: 10% more time on packed prompts.)
struct Where {
  int seq, hk, rest;
};

// The sequence whose length (in keys) is the r-th largest of up to 64.  Ragged
// sequences go longest first, so that no long one starts last.  (Packed prompts of
// 167 to 2048 tokens in the order given: the last work-groups end at 1.4 times the
// mean of the chip's, sorted and dealt out to the XCDs to and fro at 1.12.)
__device__ __forceinline__ int ranked(const Common& c, int r) {
  const int lane = threadIdx.x & 63;
  const int len = lane < c.seqs ? c.cu_k[lane + 1] - c.cu_k[lane] : -1;
  int rank = 0;
  for (int j = 0; j < c.seqs; ++j) {
    const int other = __builtin_amdgcn_readlane(len, j);
    rank += other > len || (other == len && j < lane) ? 1 : 0;
  }
  const uint64_t mask = __ballot(lane < c.seqs && rank == r);
  return __builtin_ctzll(mask | (1ull << 63));
}

__device__ __forceinline__ bool locate(const Common& c, Where& w) {
  const int id = blockIdx.x, units = c.seqs * c.Hk;
  int unit;
  if (c.cluster > 0) {
    const int slot = id >> 3, per = c.cluster * c.per_unit;
    int cl = slot / per, in = slot - cl * per;
    // heads of a cluster side by side, so that lines are shared while they are hot
    w.rest = in / c.cluster;
    in -= w.rest * c.cluster;
    cl = cl * 8 + ((cl & 1) != 0 ? 7 - (id & 7) : id & 7);
    if (cl >= c.clusters) return false;
    unit = cl * c.cluster + in;
  } else {
    unit = id / c.per_unit;
    w.rest = id - unit * c.per_unit;
  }
  if (unit >= units) return false;
  w.seq = unit / c.Hk;
  w.hk = unit - w.seq * c.Hk;
  if (c.sorted) w.seq = ranked(c, w.seq);
  return true;
}

// First token and length of a sequence, inside [0, total] whatever the offsets say.
__device__ __forceinline__ void clip(int a, int b, int total, int& start, int& len) {
  start = a < 0 ? 0 : a > total ? total : a;
  const int end = b < start ? start : b > total ? total : b;
  len = end - start;
}
__device__ __forceinline__ void bounds(const int32_t* cu, int seq, int total, int& start, int& len) {
  clip(cu[seq], cu[seq + 1], total, start, len);
}

// A thread's index of which the compiler knows nothing: what is computed from it in
// a loop stays in the loop.  (Addresses of a dozen tiles, taken out of the loop over
// short sequences, filled the registers.)
__device__ __forceinline__ int unknown_thread() {
  int v = threadIdx.x;
  asm volatile("" : "+v"(v));
  return v;
}

// ---- tiles ------------------------------------------------------------------
template <typename T, int HD, int R = sizeof(T) == 2 ? 64 : 32>
struct Tile {
  static constexpr int ES = sizeof(T);
  static constexpr int EPC = 16 / ES;          // values of a chunk
  static constexpr int CPR = HD * ES / 16;     // chunks of a row
  static constexpr int ROWS = R;
  static constexpr int BLOCKS = ROWS / 32;
  static constexpr int BYTES = ROWS * HD * ES;
  static constexpr int STEPS = CPR / 2;        // chunk pairs of a row: one a lane half

  static __device__ __forceinline__ int swizzle(int r) {
    const int k0 = r & 1, k1 = (r >> 1) & 1, k2 = (r >> 2) & 1;
    if constexpr (ES == 4) return r & 7;
    if constexpr (CPR == 4) return k1 | (k2 << 1);
    if constexpr (CPR == 8) return (k0 << 2) | k1 | (k2 << 1);
    return (k1 << 3) | (k0 << 2) | (k1 << 1) | k2;
  }
  static __device__ __forceinline__ int at(int row, int chunk) {
    return (row * CPR + (chunk ^ swizzle(row))) * 16;
  }
};

// A buffer over `rows` rows of `ts` elements from `base`: what lies behind the
// last row's dim values reads as zero.  (A tile may end inside a sequence's last
// rows: what follows belongs to another sequence, and not even an infinity of it
// may reach a product.)  Token strides are at least dim and at most
// MAX_TOKEN_STRIDE, so that offsets of a tile's rows stay below 2^31; the base
// carries the 64-bit part of an address.
typedef __amdgpu_buffer_rsrc_t Buffer;
template <typename T>
__device__ __forceinline__ Buffer rows_of(const char* base, int rows, int64_t ts, int dim) {
  const int bytes = rows > 0 ? ((rows - 1) * (int)ts + dim) * (int)sizeof(T) : 0;
  // uniform, and said to be: where the compiler cannot see it, it loops over the lanes
  const uint64_t at = (uint64_t)(uintptr_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)((uint64_t)hi << 32 | lo), (short)0,
                                           __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
constexpr uint32_t NO_ROW = 0xc0000000u;  // beyond every buffer, also after adding a tile's offsets

__device__ __forceinline__ u32x4 load16(Buffer b, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0);
}

// Registers between global memory and LDS: the rows of a tile, zeros behind `left`.
template <typename T, int HD, int NT, int R = Tile<T, HD>::ROWS>
struct Stage {
  typedef Tile<T, HD, R> Tl;
  static constexpr int N = Tl::ROWS * Tl::CPR / NT, STEP = NT / Tl::CPR;
  static_assert(N > 0 && Tl::ROWS * Tl::CPR % NT == 0 && NT % Tl::CPR == 0,
                "every thread takes the same chunk of N rows");
  u32x4 r[N];
  __device__ __forceinline__ void load(const char* base, int64_t ts, int left, int dim,
                                       int tid = threadIdx.x) {
    const int row = tid / Tl::CPR, ch = tid % Tl::CPR;
    const Buffer b = rows_of<T>(base, left < R ? left : R, ts, dim);
    const uint32_t pitch = (uint32_t)ts * Tl::ES;
    const uint32_t off = ch * Tl::EPC < dim ? row * pitch + ch * 16 : NO_ROW;
#pragma unroll
    for (int n = 0; n < N; ++n) r[n] = load16(b, off + n * (STEP * pitch));
  }
  __device__ __forceinline__ void store(char* lds, int tid = threadIdx.x) const {
    const int row = tid / Tl::CPR, ch = tid % Tl::CPR;
#pragma unroll
    for (int n = 0; n < N; ++n)
      *reinterpret_cast<u32x4*>(lds + Tl::at(row + n * STEP, ch)) = r[n];
  }
};

// ---- operands ---------------------------------------------------------------
// Lane l's part of a row of 32 rows (the token of column or row l % 32): chunks
// 2 s + h of the row, s < STEPS.  Both operands use it, so the order in which
// the reduction runs over the head dimension is the same in both.
template <typename T, int HD>
struct RowFrag {
  u32x4 c[Tile<T, HD>::STEPS];
  // from global memory; zeros past the head dimension or where !valid
  __device__ __forceinline__ void load(const char* row, int dim, bool valid) {
    typedef Tile<T, HD> Tl;
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int s = 0; s < Tl::STEPS; ++s) {
      const int ch = 2 * s + h;
      if (valid && ch * Tl::EPC < dim)
        c[s] = *reinterpret_cast<const u32x4*>(row + ch * 16);
      else
        c[s] = u32x4{0, 0, 0, 0};
    }
  }
  // row row0 + l % 32 of a tile in LDS
  __device__ __forceinline__ void read(const char* tile, int row0, int tid = threadIdx.x) {
    typedef Tile<T, HD> Tl;
    const int lane = tid & 63;
#pragma unroll
    for (int s = 0; s < Tl::STEPS; ++s)
      c[s] = *reinterpret_cast<const u32x4*>(tile + row0 * HD * Tl::ES +
                                             Tl::at(lane & 31, 2 * s + (lane >> 5)));
  }
};

template <typename T>
__device__ __forceinline__ floatx16 mma_chunk(u32x4 a, u32x4 b, floatx16 acc) {
  if constexpr (sizeof(T) == 2) {
    return Mma<_Float16>::mma(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), acc);
  } else {
    const floatx4 x = __builtin_bit_cast(floatx4, a), y = __builtin_bit_cast(floatx4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = Mma<float>::mma(x[e], y[e], acc);
    return acc;
  }
}

// rows row0 .. row0 + 31 of an LDS tile times the lane's column vector
template <typename T, int HD>
__device__ __forceinline__ floatx16 mma_rows(const char* tile, int row0, const RowFrag<T, HD>& b,
                                             floatx16 acc, int tid = threadIdx.x) {
  typedef Tile<T, HD> Tl;
  const int lane = tid & 63;
#pragma unroll
  for (int s = 0; s < Tl::STEPS; ++s) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(tile + row0 * HD * Tl::ES +
                                                    Tl::at(lane & 31, 2 * s + (lane >> 5)));
    acc = mma_chunk<T>(a, b.c[s], acc);
  }
  return acc;
}

// Sixteen result registers as the second operand of a product over their rows.
template <typename T>
struct ColFrag;
template <>
struct ColFrag<float> {
  floatx16 v;
  __device__ __forceinline__ ColFrag() {}
  __device__ __forceinline__ explicit ColFrag(const floatx16& p) : v(p) {}
};
template <>
struct ColFrag<_Float16> {
  half8 v[2];
  __device__ __forceinline__ ColFrag() {}
  __device__ __forceinline__ explicit ColFrag(const floatx16& p) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e >> 3][e & 7] = (_Float16)p[e];
  }
};

// Values 32 db + l % 32 of rows row0 .. row0 + 31 of a tile, transposed: the lane's
// column of the block, its rows in the order of the result registers.  As the first
// operand of a product over the tile's rows, and as the second one of a matrix that
// lies in LDS by rows.
template <typename T, int HD>
__device__ __forceinline__ half8 read_col16(const char* tile, int row0, int db, int s,
                                            int tid = threadIdx.x) {
  typedef Tile<T, HD> Tl;
  typedef __attribute__((address_space(3))) s16x4 lds4;
  const int lane = tid & 63;
  const int k = 4 * (lane >> 5) + ((lane & 15) >> 2);
  const int ch = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  const char* base = tile + (row0 + 16 * s) * HD * 2 + Tl::at(k, 4 * db + ch) + (lane & 1) * 8;
  const half4 lo = __builtin_bit_cast(half4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)base));
  const half4 hi =
      __builtin_bit_cast(half4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(base + 8 * HD * 2)));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int HD>
__device__ __forceinline__ float read_col32(const char* tile, int row0, int db, int e,
                                            int tid = threadIdx.x) {
  const int lane = tid & 63, r = 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
  return *reinterpret_cast<const float*>(tile + row0 * HD * 4 +
                                         Tile<float, HD>::at(r, 8 * db + ((lane & 31) >> 2)) +
                                         (lane & 3) * 4);
}

// acc[db] += (rows row0 .. row0 + 31 of the tile, values 32 db ..)' times p
template <typename T, int HD>
__device__ __forceinline__ void mma_cols(const char* tile, int row0, const ColFrag<T>& p,
                                         floatx16 (&acc)[HD / 32], int tid = threadIdx.x) {
#pragma unroll
  for (int db = 0; db < HD / 32; ++db) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        acc[db] = Mma<_Float16>::mma(read_col16<T, HD>(tile, row0, db, s, tid), p.v[s], acc[db]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        acc[db] = Mma<float>::mma(read_col32<HD>(tile, row0, db, e, tid), p.v[e], acc[db]);
    }
  }
}

// Asks the scheduler for LDS reads ahead of the products that use them: AHEAD reads
// first, then products with the other reads between them.  (Left alone it places
// a read right before its product, and every product waits for LDS: a tile of the
// forward pass at dimension 128 took twice the cycles of its instructions.)
template <int READS, int PRODUCTS, int AHEAD>
__device__ __forceinline__ void reads_ahead() {
  constexpr int FIRST = AHEAD < READS ? AHEAD : READS, REST = READS - FIRST;
  constexpr int GROUPS = REST > 0 && REST < PRODUCTS ? REST : PRODUCTS;  // of products
  constexpr int MFMA = PRODUCTS / GROUPS, READ = (REST + GROUPS - 1) / GROUPS;
  __builtin_amdgcn_sched_group_barrier(0x100, FIRST, 0);
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, MFMA, 0);
    if (REST > 0) __builtin_amdgcn_sched_group_barrier(0x100, READ, 0);
  }
}
// of mma_rows and mma_cols of a block
template <typename T, int HD>
struct Reads {
  static constexpr int ROW = Tile<T, HD>::STEPS, ROW_MMA = ROW * (sizeof(T) == 2 ? 1 : 4);
  static constexpr int COL = HD / 32 * (sizeof(T) == 2 ? 4 : 16), COL_MMA = HD / 32 * (sizeof(T) == 2 ? 2 : 16);
};

// ---- small things -------------------------------------------------------------
// the two halves of a wave hold rows of the same column: lane l and l ^ 32
__device__ __forceinline__ float pair_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(int, v),
                                                  __builtin_bit_cast(int, v), false, false);
  return fmaxf(__builtin_bit_cast(float, (int)r[0]), __builtin_bit_cast(float, (int)r[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(int, v),
                                                  __builtin_bit_cast(int, v), false, false);
  return __builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]);
}

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// Offsets that follow from indices: a block of scores meets at most 63 + 31
// consecutive ones, and the tiles that are not wholly beyond the span on one side
// meet the span, so a bias with PAD copies of its ends on both sides needs no
// clamping, and a lane's reads are a fixed distance from its first one.
constexpr int PAD = 96;
template <int BIAS>
__host__ __device__ constexpr int bias_width(int span) {
  return 2 * span + 1 + (BIAS == BIAS_INDEX ? 2 * PAD : 0);
}

// The bias of every offset for heads head0 .. head0 + n - 1.
// Four offsets a thread at a time: the buckets of all four, then their values head by
// head, are on their way together.  (One value after the other, bucket and then value,
// took half of a new token's pass over a cache of 32768 with four heads of 257 offsets
// a work-group of one wave: 20.6 us for 10.5 us without a bias.)
template <typename T, int BIAS>
__device__ __forceinline__ void fill_bias(float* lut, const Common& c, int head0, int n) {
  const int width = bias_width<BIAS>(c.span), threads = blockDim.x;
  for (int i0 = threadIdx.x; i0 < width; i0 += 4 * threads) {
    const T* from[4];
    bool in[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int b = c.map[clamp_int(i0 + u * threads - (BIAS == BIAS_INDEX ? PAD : 0), 0, 2 * c.span)];
      in[u] = b >= 0 && b < c.buckets;
      from[u] = (const T*)c.table + (int64_t)(in[u] ? b : 0) * c.H + head0;
    }
#pragma unroll 4
    for (int g = 0; g < n; ++g) {
      float t[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) t[u] = (float)from[u][g];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * threads < width) lut[g * width + i0 + u * threads] = in[u] ? t[u] : 0.f;
    }
  }
}

// Scores of a block, scaled, each rounded before a maximum or lse is taken from it:
// merged with that into one operation, a score of 10^9 would differ from itself by up
// to 2^5.
__device__ __forceinline__ void scale_scores(floatx16& s, float scale) {
#pragma clang fp contract(off)
#pragma unroll
  for (int e = 0; e < 16; ++e) s[e] = s[e] * scale;
}

// Scores of a block, scaled, with the bias of the lane's row of offsets: INDEX,
// at[e] for result row 8 (e / 4) + e % 4 above the lane's first (at: PAD included;
// step -1 where rows are queries); POSITIONS, offsets off.
template <int STEP>
__device__ __forceinline__ void add_bias_row(floatx16& s, float scale, const float* at) {
  float b[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) b[e] = at[STEP * (8 * (e >> 2) + (e & 3))];
#pragma unroll
  for (int e = 0; e < 16; ++e) s[e] = __builtin_fmaf(s[e], scale, b[e]);
}
__device__ __forceinline__ void add_bias_offsets(floatx16& s, float scale, const float* lut,
                                                 const int (&off)[16], int width) {
  float b[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) b[e] = lut[clamp_int(off[e], 0, width - 1)];
#pragma unroll
  for (int e = 0; e < 16; ++e) s[e] = __builtin_fmaf(s[e], scale, b[e]);
}

// Values of a result column (d = 32 db + 8 g + 4 h + 0..3) to a row of the output.
template <typename T, int HD>
__device__ __forceinline__ void store_column(char* row, const floatx16 (&acc)[HD / 32], float f,
                                             int dim) {
  const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
  for (int db = 0; db < HD / 32; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * db + 8 * g + 4 * h;
      if (d < dim) {
        floatx4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = acc[db][4 * g + e] * f;
        *reinterpret_cast<typename Elem<T>::quad*>(row + d * sizeof(T)) = Elem<T>::pack(o);
      }
    }
}

// One wave's LDS operations run in the order of its instructions, so what a lane
// has written another lane reads without a wait; the compiler, which looks at one
// lane, has to keep that order.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The 32 result columns of a wave (rows of the output, `rows` of them from `out`) by
// way of `scratch`, 32 HD values of the wave's own LDS: straight from the registers
// a store would touch 32 rows with 8 bytes a lane, and those short writes were 40%
// of a window's time in the forward pass.
template <typename T, int HD>
__device__ __forceinline__ void store_rows(char* scratch, char* out, int64_t ts, int rows,
                                           const floatx16 (&acc)[HD / 32], float f, int dim,
                                           int tid = threadIdx.x) {
  typedef Tile<T, HD, 32> Tl;
  const int lane = tid & 63, h = lane >> 5;
#pragma unroll
  for (int db = 0; db < HD / 32; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = 32 * db + 8 * g + 4 * h;
      floatx4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = acc[db][4 * g + e] * f;
      *reinterpret_cast<typename Elem<T>::quad*>(scratch + Tl::at(lane & 31, d / Tl::EPC) +
                                                 d % Tl::EPC * Tl::ES) = Elem<T>::pack(o);
    }
  wave_order();
  constexpr int N = 32 * Tl::CPR / 64, STEP = 64 / Tl::CPR;
  const int row = lane / Tl::CPR, ch = lane % Tl::CPR;
  char* p = out + (row * ts + ch * Tl::EPC) * Tl::ES;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(scratch + Tl::at(row + n * STEP, ch));
    if (row + n * STEP < rows && ch * Tl::EPC < dim)
      *reinterpret_cast<u32x4*>(p + (int64_t)n * STEP * ts * Tl::ES) = v;
  }
  wave_order();
}

// Lets a kernel have more than 64 KB of LDS.  Always the same number, a work-group's
// most: the attribute belongs to the kernel, not to the call, and calls of several
// threads set it with sizes of their own in mind.
constexpr int LDS_BYTES = 163840;
template <typename K>
hipError_t allow_lds(K kernel, size_t lds) {
  if (lds <= 65536) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, LDS_BYTES);
}

__device__ __forceinline__ floatx16 zero16() {
  floatx16 z;
#pragma unroll
  for (int e = 0; e < 16; ++e) z[e] = 0.f;
  return z;
}

}  // namespace attn
}  // namespace eql
