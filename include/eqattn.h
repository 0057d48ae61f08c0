/*
 * eqattn.h -- C ABI of attention over packed sequences with grouped heads and a
 * learned relative position bias by buckets, forward and backward, in
 * libeqlinear (AMD MI355X, gfx950).
 *
 * The operation.  Tokens of several sequences of different lengths lie one
 * after the other (packed); sequence b has Lq queries and Lk keys.  With H query
 * heads, Hk key/value heads (H a multiple of Hk; query head h reads key/value
 * head h / (H / Hk)) and head dimension D, for query i and key j of a sequence
 *
 *     s[i,j] = scale * sum_d q[i,h,d] * k[j,h',d] + table[map[r(i,j)], h]
 *     r(i,j) = clamp(pos_k[j] - pos_q[i], -span, span) + span
 *     o[i,h] = sum_j softmax_j(s[i,:])[j] * v[j,h']
 *     lse[i,h] = log sum_j exp(s[i,j])
 *
 * Causal plans let query i see the keys j <= i + Lk - Lq (the last query sees
 * every key): Lq = Lk is a whole prompt, Lq = 1 one new token against a cache.
 * A query that sees no key gives o = 0 and lse = -infinity.
 *
 * Equivariance.  A token's C channels of T group values, cut into heads of
 * C / H channels, are H vectors of D = (C / H) * T values: the score sums over a
 * channel's group values, so a permutation of the group axis common to q, k and
 * v leaves the scores alone and permutes o.
 *
 * Bias.  map gives the bucket of every clamped offset and table the learned
 * value of every bucket and head.  Positions default to the token's index in its
 * sequence (queries at the end of the keys), so a map over offsets makes any
 * one-dimensional bucketing.  For a grid of W columns, positions
 * row * (2 W - 1) + column make the offsets of the plane distinct and the map
 * gives one bucket to each.  An offset whose bucket is outside [0, buckets)
 * gets no bias.  A table value of -infinity removes its offsets.
 *
 * Backward.  With p = exp(s - lse) and delta[i] = sum_d do[i,d] * o[i,d],
 *     ds = p * (do . v - delta)      dq = scale * ds k      dk = scale * ds' q
 *     dv = p' do                     dtable[map[r], h] = sum of ds      (binary32)
 * where dk and dv also sum over the query heads that share a key/value head.
 *
 * Arithmetic.  Scores, softmax statistics, delta and every sum are binary32.  A
 * finite table value of any size leaves results finite (beside it a score keeps
 * what binary32 has room for).  In
 * binary16 plans the factors p and ds of the matrix products are rounded to
 * binary16, scaled by a power of two (per query for dq, per key for dk; for dk of
 * sequences of at most 64 tokens per 32 queries, so that a key whose every ds is
 * below 2^-28 of their largest loses digits) that keeps them in its normal range;
 * o, dq, dk and dv are rounded once.  Every sum has a fixed order,
 * so the same call gives the same bits (dtable: where the positions of a
 * sequence's queries are distinct).  Sequences do not see each other's values,
 * infinities and NaN included.  Within a sequence a key or value that is not
 * finite may also reach queries that do not see it, as it does where the mask is
 * applied to the scores alone.
 *
 * Layouts.  A view names the first element, and the strides in elements between
 * tokens and between heads; the D values of a head are contiguous.  Views may be
 * parts of one larger tensor (queries, keys and values side by side).  Every
 * view starts on 16 bytes and its strides are multiples of 16 bytes
 * (EQL_ERR_MISALIGNED otherwise).  The token stride is at least D
 * (EQL_ERR_INVALID_ARG) and at most EQATTN_MAX_TOKEN_STRIDE
 * (EQL_ERR_UNSUPPORTED), the head stride of outputs at least D and that of inputs
 * at least 0 (one head for all).  Strides over a single token or head are not
 * read.  Tensors may be larger than 4 GiB.
 *     q, o, do, dq : [total_q] tokens x [H] heads      k, v, dk, dv : [total_k] x [Hk]
 *     lse : [H][total_q] binary32, contiguous
 *     table : [buckets][H] in the plan dtype           map : [2 span + 1] int32
 *     dtable : [buckets][H] binary32
 *     cu_q, cu_k : [sequences + 1] int32, token offsets, non-decreasing from 0
 *     pos_q : [total_q] int32, pos_k : [total_k] int32 (both or neither NULL)
 * Offsets are read on the GPU and clamped to the token counts.  A sequence longer
 * than max_q or max_k says, or offsets that decrease, give unspecified outputs, inside
 * the tensors.  Outputs of tokens that belong to no sequence are left alone.
 * Positions and their differences must stay within 31 bits.
 *
 * Caches with room behind their tokens: the room is a sequence of its own without
 * queries, so that cu_k is 0, len0, room, room + len1, 2 room, ... and cu_q 0, 1, 1,
 * 2, 2, ...  (Keys are split over work-groups by the number of sequences, these
 * among them: half as many pieces as packed caches get.)
 *
 * Ownership, streams, errors and concurrency are as in eqlinear.h: buffers
 * belong to the caller, every call is asynchronous on the given HIP stream,
 * allocates nothing and can be captured in a graph, and arguments are checked
 * on the host before any HIP call.
 */
#ifndef EQATTN_H
#define EQATTN_H

#include <stddef.h>
#include <stdint.h>

#include "eqlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EQATTN_MAX_DIM 128
#define EQATTN_MAX_SPAN 1023
#define EQATTN_MAX_HEADS 1024
#define EQATTN_MAX_TOKEN_STRIDE 4194304

typedef struct eqattn_plan* eqattn_plan_t; /* opaque */

typedef struct {
  void* data; /* read only where the view is an input */
  int64_t token_stride, head_stride; /* elements */
} eqattn_view_t;

/* How tokens are packed into sequences. */
typedef struct {
  int64_t sequences, total_q, total_k;
  int64_t max_q, max_k; /* at least the longest sequence's queries and keys */
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* pos_q; /* NULL: index in the sequence, queries at the end of the keys */
  const int32_t* pos_k;
} eqattn_packing_t;

/* Create a plan for `heads` query heads on `kv_heads` key/value heads of `dim`
 * values.  dim is a multiple of 8 up to EQATTN_MAX_DIM.  scale is positive and
 * finite in binary32.  buckets = 0 is a plan without a bias (span must be 0); otherwise
 * offsets are clamped to [-span, span], 0 <= span <= EQATTN_MAX_SPAN, and the
 * table has `buckets` <= 65536 rows.  EQL_ERR_INVALID_ARG: heads, kv_heads, dim,
 * buckets or span negative (or 0 where at least 1 is needed), scale, heads not a
 * multiple of kv_heads, out == NULL; EQL_ERR_UNSUPPORTED: dtype, or sizes above
 * those stated.  Host-only: allocates no device memory. */
eqlinear_status_t eqattn_plan_create(int64_t heads, int64_t kv_heads, int64_t dim, double scale,
                                     int causal, int64_t buckets, int64_t span,
                                     eqlinear_dtype_t dtype, eqattn_plan_t* out);

/* Destroy a plan (NULL is a no-op). */
eqlinear_status_t eqattn_plan_destroy(eqattn_plan_t plan);

/* Bytes of device workspace eqattn_forward needs (0 for invalid arguments, and
 * where none is needed): with few query rows against long sequences the keys are
 * split over work-groups, whose partial results are joined by a second kernel. */
size_t eqattn_forward_workspace(eqattn_plan_t plan, const eqattn_packing_t* packing);

/* o, and lse (NULL = not wanted).  table and map are NULL exactly for a plan
 * without a bias.  No query is a successful no-op.  EQL_ERR_UNSUPPORTED: more than
 * 2^24 work-groups (sequences x heads x tiles of 32 to 128 queries of the longest);
 * so does the backward pass. */
eqlinear_status_t eqattn_forward(eqattn_plan_t plan, const eqattn_packing_t* packing,
                                 const eqattn_view_t* q, const eqattn_view_t* k,
                                 const eqattn_view_t* v, const void* table, const int32_t* map,
                                 const eqattn_view_t* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Bytes of device workspace eqattn_backward needs (0 for invalid arguments):
 * delta of every query row, and the partial sums of dtable: about
 * heads * (2 span + 1) * 4 bytes for every 64 or 128 queries and every sequence. */
size_t eqattn_backward_workspace(eqattn_plan_t plan, const eqattn_packing_t* packing);

/* The same where dtable is NULL: delta alone. */
size_t eqattn_backward_workspace_no_dtable(eqattn_plan_t plan, const eqattn_packing_t* packing);

/* dq, dk, dv and dtable (NULL = not wanted; NULL for a plan without a bias) from
 * the forward pass's inputs, its o and lse, and dout, the gradient of o.
 * Outputs are overwritten, not accumulated into. */
eqlinear_status_t eqattn_backward(eqattn_plan_t plan, const eqattn_packing_t* packing,
                                  const eqattn_view_t* dout, const eqattn_view_t* q,
                                  const eqattn_view_t* k, const eqattn_view_t* v,
                                  const eqattn_view_t* o, const float* lse, const void* table,
                                  const int32_t* map, const eqattn_view_t* dq,
                                  const eqattn_view_t* dk, const eqattn_view_t* dv, float* dtable,
                                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EQATTN_H */
