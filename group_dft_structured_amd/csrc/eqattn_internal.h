// Host-side internals of attention: the plan object, the arguments of the
// kernels and their launchers.
#pragma once

#include "../../include/eqattn.h"
#include "eql_internal.h"

struct eqattn_plan {
  int H, Hk, dim;
  int causal, buckets, span;
  double scale;
  eqlinear_dtype_t dtype;
  size_t esize;
};

namespace eql {
namespace attn {

// A tensor of [tokens][heads][dim]; strides in elements.
struct View {
  char* data;
  int64_t ts, hs;
};

// What every kernel of a call sees.
struct Common {
  int H, Hk, G, dim, esize;  // G = H / Hk query heads share a key/value head
  int causal, buckets, span;
  float scale;
  int seqs, total_q, total_k, max_k;
  const int32_t *cu_q, *cu_k, *pos_q, *pos_k;
  const void* table;
  const int32_t* map;
  // work-groups: per (sequence, key/value head) unit, and how units go to XCDs
  int per_unit, cluster, clusters, sorted;
  int slot_rows;  // queries of a part of BwdArgs::hist; 0: a part is a chunk
};

struct FwdArgs {
  Common c;
  View q, k, v, o;
  float* lse;
  int tiles, packed, splits;
  int chunks;  // short sequences (attn_short.h): work-groups of a head
  float *part_o, *part_ml;  // splits > 1: [splits][H][total_q] rows of dim values; of (max, sum)
};

struct BwdArgs {
  Common c;
  View dout, q, k, v, o, dq, dk, dv;
  const float* lse;
  float* delta;  // [H][total_q]
  float* hist;   // [slots of tiles] or [chunks], [H][2 span + 1]: partial sums of dtable, or nullptr
  int tiles;
  int chunks;
};

// Largest token stride in elements: a tile's 64 rows lie within 2^30 bytes.
constexpr int64_t MAX_TOKEN_STRIDE = EQATTN_MAX_TOKEN_STRIDE;

// Most pieces that the keys of a forward pass are split into.
constexpr int MAX_SPLITS = 128;

// Waves of a work-group and work-groups of a pass.
struct FwdShape {
  int chunks;  // > 0: short sequences, and the others are not used
  int waves, packed, tiles, splits;
};
FwdShape forward_shape(const eqattn_plan* p, const eqattn_packing_t* b);
size_t forward_workspace(const eqattn_plan* p, const eqattn_packing_t* b, const FwdShape& s);

struct BwdShape {
  int chunks;
  int waves_q, tiles_q, keys, tiles_k;  // keys: of a work-group of the key pass
};
BwdShape backward_shape(const eqattn_plan* p, const eqattn_packing_t* b);
size_t delta_bytes(const eqattn_plan* p, const eqattn_packing_t* b);
size_t hist_parts(const eqattn_packing_t* b, const BwdShape& s);
size_t hist_bytes(const eqattn_plan* p, const eqattn_packing_t* b, const BwdShape& s);
size_t slices_bytes(const eqattn_plan* p);

// One file per type (k_attn_*_f16.hip, k_attn_*_f32.hip).
hipError_t launch_fwd_f16(const FwdArgs& a, const FwdShape& s, int max_q,
                          hipStream_t st);
hipError_t launch_fwd_f32(const FwdArgs& a, const FwdShape& s, int max_q,
                          hipStream_t st);
hipError_t launch_bwd_f16(const BwdArgs& a, const BwdShape& s, hipStream_t st);
hipError_t launch_bwd_f32(const BwdArgs& a, const BwdShape& s, hipStream_t st);
// dtable from the partial sums of `parts` work-groups of each head
hipError_t launch_bias_finish(const Common& c, const float* hist, int parts, double* slices,
                              float* dtable, hipStream_t st);

// Spreads the units of a pass over the chip (sets c.per_unit, cluster, clusters,
// sorted) and returns the number of work-groups, -1 for too many.
int64_t spread(Common& c, int64_t per_unit, bool one_tile);

}  // namespace attn
}  // namespace eql
