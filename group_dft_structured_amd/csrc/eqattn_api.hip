// C ABI of attention (include/eqattn.h): argument validation, the shapes of a
// pass (waves, tiles, splits) and dispatch.  Every check runs before the first
// HIP call.
#include <float.h>
#include <string.h>

#include <new>

#include "eqattn_internal.h"

namespace {

using namespace eql::attn;

constexpr int64_t MAX_TOKENS = ((int64_t)1 << 31) - 256;
constexpr int64_t MAX_SEQUENCES = 1 << 24, MAX_BUCKETS = 65536;
// a launch has fewer than 2^32 threads, at most 256 in a work-group here
constexpr int64_t MAX_GRID = ((int64_t)1 << 24) - 1;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t ru256(size_t v) { return (v + 255) / 256 * 256; }

eqlinear_status_t hip_status(const char* what, hipError_t e) {
  if (e == hipSuccess) return EQL_OK;
  eql::set_last_error(what, e);
  return EQL_ERR_HIP;
}

bool sizes_ok(const eqattn_packing_t* b) {
  if (b == nullptr || b->sequences < 0 || b->total_q < 0 || b->total_k < 0 || b->max_q < 0 ||
      b->max_k < 0)
    return false;
  return b->sequences <= MAX_SEQUENCES && b->total_q <= MAX_TOKENS && b->total_k <= MAX_TOKENS;
}

eqlinear_status_t check_packing(const eqattn_packing_t* b) {
  if (!sizes_ok(b)) return EQL_ERR_INVALID_ARG;
  if (b->sequences > 0 && (b->cu_q == nullptr || b->cu_k == nullptr)) return EQL_ERR_INVALID_ARG;
  const void* const each[] = {b->cu_q, b->cu_k, b->pos_q, b->pos_k};
  for (const void* a : each)
    if (((uintptr_t)a & 3u) != 0) return EQL_ERR_MISALIGNED;
  // positions of tokens that exist come for queries and keys alike
  const bool pq = b->pos_q != nullptr || b->total_q == 0, pk = b->pos_k != nullptr || b->total_k == 0;
  if ((b->pos_q != nullptr && !pk) || (b->pos_k != nullptr && !pq)) return EQL_ERR_INVALID_ARG;
  return EQL_OK;
}

// A view of `tokens` x `heads` rows.  A stride over a single token or head is
// not used and may be anything.
eqlinear_status_t check_view(const eqattn_plan* p, const eqattn_view_t* v, int64_t tokens, int64_t heads,
                             bool output, View* out) {
  if (v == nullptr) return EQL_ERR_INVALID_ARG;
  int64_t ts = tokens > 1 ? v->token_stride : 0, hs = heads > 1 ? v->head_stride : 0;
  if (tokens > 0 && v->data == nullptr) return EQL_ERR_INVALID_ARG;
  if ((tokens > 1 && ts < p->dim) || (heads > 1 && hs < (output ? p->dim : 0))) return EQL_ERR_INVALID_ARG;
  if (ts > MAX_TOKEN_STRIDE) return EQL_ERR_UNSUPPORTED;
  const int64_t per = 16 / (int64_t)p->esize;
  if (!aligned16(v->data) || ts % per != 0 || hs % per != 0) return EQL_ERR_MISALIGNED;
  *out = View{(char*)v->data, ts, hs};
  return EQL_OK;
}

int64_t max_q_of(const eqattn_packing_t* b) { return b->max_q < b->total_q ? b->max_q : b->total_q; }
int64_t max_k_of(const eqattn_packing_t* b) { return b->max_k < b->total_k ? b->max_k : b->total_k; }

eqlinear_status_t check_bias(const eqattn_plan* p, const void* table, const int32_t* map) {
  if (p->buckets == 0) return table == nullptr && map == nullptr ? EQL_OK : EQL_ERR_INVALID_ARG;
  if (table == nullptr || map == nullptr) return EQL_ERR_INVALID_ARG;
  return aligned16(table) && aligned16(map) ? EQL_OK : EQL_ERR_MISALIGNED;
}

void fill_common(Common* c, const eqattn_plan* p, const eqattn_packing_t* b, const void* table,
                 const int32_t* map) {
  memset(c, 0, sizeof(*c));
  c->H = p->H;
  c->Hk = p->Hk;
  c->G = p->H / p->Hk;
  c->dim = p->dim;
  c->esize = (int)p->esize;
  c->causal = p->causal;
  c->buckets = p->buckets;
  c->span = p->span;
  c->scale = (float)p->scale;
  c->seqs = (int)b->sequences;
  c->total_q = (int)b->total_q;
  c->total_k = (int)b->total_k;
  c->max_k = (int)max_k_of(b);
  c->cu_q = b->cu_q;
  c->cu_k = b->cu_k;
  c->pos_q = b->pos_q;
  c->pos_k = b->pos_k;
  c->table = table;
  c->map = map;
}

}  // namespace

namespace eql {
namespace attn {

// Work-groups of a head for sequences of one tile (attn_short.h), 0 for others: as
// many as find a place on the chip at once, `places` a compute unit over all heads,
// with the same number of sequences each (with a third of them waiting for a place,
// 4096 windows took 102 us for 90 us forward and 231 us for 203 us backward).  They
// go round the XCDs, so that it is an XCD's 32 compute units that hold them: six
// heads on two places, 84 work-groups a head, left two of 66 waiting on half of the
// XCDs (877 us for 559 us, binary32 backward).  Shared key/value heads and wider rows
// take the long kernels: the same windows with 6 heads on 3 take 88 us forward and
// 383 us backward for 76 us and 183 us.
int short_chunks(const eqattn_plan* p, const eqattn_packing_t* b, int places) {
  if (p->H != p->Hk || p->dim * p->esize > 128 || max_q_of(b) > 64 || max_k_of(b) > 64) return 0;
  const int64_t an_xcd = 32 * places / p->H, most = 8 * (an_xcd < 1 ? 1 : an_xcd);
  const int64_t turns = ceil_div(b->sequences, most);
  return turns > 0 ? (int)ceil_div(b->sequences, turns) : 0;
}

FwdShape forward_shape(const eqattn_plan* p, const eqattn_packing_t* b) {
  const int64_t max_q = max_q_of(b), max_k = max_k_of(b);
  const int G = p->H / p->Hk;
  FwdShape s;
  memset(&s, 0, sizeof(s));
  s.splits = 1;
  s.chunks = max_q > 0 ? short_chunks(p, b, p->dim * p->esize <= 64 ? 6 : 4) : 0;
  if (s.chunks > 0) return s;
  // Up to 16 queries a sequence the heads that share a key/value head share a
  // work-group, whose rows they would not fill one by one.  Their biases lie in
  // LDS side by side, which bounds them.
  s.packed = G > 1 && max_q <= 16 && (int64_t)G * (2 * p->span + 256) <= 8192;
  const int64_t rows = max_q * (s.packed ? G : 1);
  s.waves = rows <= 32 ? 1 : rows <= 64 ? 2 : 4;
  s.tiles = (int)ceil_div(rows, 32 * s.waves);
  const int64_t groups = b->sequences * p->Hk * (s.packed ? 1 : G) * s.tiles;
  s.splits = 1;
  // Fewer work-groups than the chip holds: the keys are split, down to pieces
  // whose partial results (8 bytes a row and value, written and read) stay small
  // against the keys and values read.
  const int64_t least = 8 * 32 * s.waves;
  if (groups > 0 && groups < 1024 && max_k >= 2 * least) {
    int64_t n = ceil_div(2048, groups);
    if (n > max_k / least) n = max_k / least;
    s.splits = (int)(n > MAX_SPLITS ? MAX_SPLITS : n);
  }
  return s;
}

size_t forward_workspace(const eqattn_plan* p, const eqattn_packing_t* b, const FwdShape& s) {
  if (s.splits <= 1) return 0;
  return (size_t)s.splits * p->H * (size_t)b->total_q * (size_t)(p->dim + 2) * sizeof(float);
}

BwdShape backward_shape(const eqattn_plan* p, const eqattn_packing_t* b) {
  const int64_t max_q = max_q_of(b), max_k = max_k_of(b);
  BwdShape s;
  memset(&s, 0, sizeof(s));
  s.chunks = max_q > 0 || max_k > 0 ? short_chunks(p, b, p->dim * p->esize <= 64 ? 4 : 2) : 0;
  if (s.chunks > 0) return s;
  s.waves_q = max_q <= 64 ? 2 : 4;
  s.tiles_q = (int)ceil_div(max_q, 32 * s.waves_q);
  // The key pass (attn_bwd.h).  The steps of a work-group follow each other: `chain`
  // of them for 128 keys that every query sees, against `mean` for a compute unit.
  // 128 keys where there is work enough (16 sequences of 2048, 16 heads of 64,
  // causal, binary16: 841 us backward for 922 us with 64; 64 sequences of 197, 6
  // heads, binary32: 112 us for 137 us), 64 keys and twice the queries a step where
  // the longest work-group would end last (16 documents of up to 2048 tokens, 12
  // heads on 4: 156 us for 206 us in binary16, 770 us for 1254 us in binary32).
  const double chain = (double)(p->H / p->Hk) * (double)max_q / 64.0;
  const double mean = (double)p->H * (double)b->total_k / 128.0 * (double)b->total_q / 64.0 /
                      (double)(b->sequences > 0 ? b->sequences : 1) * (p->causal ? 0.5 : 1.0) / 256.0;
  s.keys = max_k <= 64 || chain > 0.75 * mean ? 64 : 128;
  s.tiles_k = (int)ceil_div(max_k, s.keys);
  return s;
}

size_t delta_bytes(const eqattn_plan* p, const eqattn_packing_t* b) {
  return ru256((size_t)p->H * (size_t)b->total_q * sizeof(float));
}

// Parts of the sums over offsets.  Tile t of sequence b has slot
// cu_q[b] / rows + b + t: a sequence's next slot is at most two behind its last, so
// that there are total_q / rows + sequences of them whatever the longest sequence.
// (One for every sequence and tile of the longest: 2 GiB for 256 sequences of 262144
// tokens in all, the longest of 8192, 16 heads, span 1023; 300 MB so.)
size_t hist_parts(const eqattn_packing_t* b, const BwdShape& s) {
  if (s.chunks > 0) return (size_t)s.chunks;
  if (b->sequences == 0 || s.tiles_q == 0) return 0;
  return (size_t)(b->total_q / (32 * s.waves_q) + b->sequences);
}

size_t hist_bytes(const eqattn_plan* p, const eqattn_packing_t* b, const BwdShape& s) {
  if (p->buckets == 0) return 0;
  return ru256(hist_parts(b, s) * p->H * (2 * (size_t)p->span + 1) * sizeof(float));
}

int64_t spread(Common& c, int64_t per_unit, bool one_tile) {
  const int64_t units = (int64_t)c.seqs * c.Hk;
  if (per_unit > MAX_GRID || units > MAX_GRID) return -1;
  c.per_unit = (int)per_unit;
  // one XCD takes whole units, or, of sequences of one tile whose heads share cache
  // lines, all heads of a sequence.  Few units go round the XCDs one work-group at
  // a time.
  c.cluster = one_tile && c.dim * c.esize < 128 ? c.Hk : 1;
  const int64_t clusters = units / c.cluster;
  // lengths that differ: the mean at most nine tenths of the longest (up to 64
  // sequences, a lane each; more of them go in the order given)
  c.sorted = per_unit > 1 && c.seqs > 1 && c.seqs <= 64 &&
             (int64_t)c.total_k * 10 < (int64_t)c.seqs * c.max_k * 9;
  if (clusters < 32 && clusters % 8 != 0) {
    c.cluster = 0;
    return units * per_unit <= MAX_GRID ? units * per_unit : -1;
  }
  c.clusters = (int)clusters;
  const int64_t grid = ceil_div(clusters, 8) * 8 * c.cluster * per_unit;
  return grid <= MAX_GRID ? grid : -1;
}

}  // namespace attn
}  // namespace eql

extern "C" {

eqlinear_status_t eqattn_plan_create(int64_t heads, int64_t kv_heads, int64_t dim, double scale,
                                     int causal, int64_t buckets, int64_t span,
                                     eqlinear_dtype_t dtype_arg, eqattn_plan_t* out) {
  if (out == nullptr) return EQL_ERR_INVALID_ARG;
  *out = nullptr;
  if (heads <= 0 || kv_heads <= 0 || dim <= 0 || heads % kv_heads != 0) return EQL_ERR_INVALID_ARG;
  if (!(scale > 0 && scale <= FLT_MAX) || buckets < 0 || span < 0 || (buckets == 0 && span != 0))
    return EQL_ERR_INVALID_ARG;
  const int dv = eql::enum_value(dtype_arg);
  if (dv != EQL_F32 && dv != EQL_F16) return EQL_ERR_UNSUPPORTED;
  if (heads > EQATTN_MAX_HEADS || dim > EQATTN_MAX_DIM || dim % 8 != 0 || buckets > MAX_BUCKETS ||
      span > EQATTN_MAX_SPAN)
    return EQL_ERR_UNSUPPORTED;
  eqattn_plan* p = new (std::nothrow) eqattn_plan;
  if (p == nullptr) return EQL_ERR_ALLOC;
  p->H = (int)heads;
  p->Hk = (int)kv_heads;
  p->dim = (int)dim;
  p->causal = causal != 0;
  p->buckets = (int)buckets;
  p->span = (int)span;
  p->scale = scale;
  p->dtype = (eqlinear_dtype_t)dv;
  p->esize = dv == EQL_F16 ? 2 : 4;
  *out = p;
  return EQL_OK;
}

eqlinear_status_t eqattn_plan_destroy(eqattn_plan_t p) {
  delete p;
  return EQL_OK;
}

size_t eqattn_forward_workspace(eqattn_plan_t p, const eqattn_packing_t* b) {
  if (p == nullptr || !sizes_ok(b)) return 0;
  return forward_workspace(p, b, forward_shape(p, b));
}

eqlinear_status_t eqattn_forward(eqattn_plan_t p, const eqattn_packing_t* b, const eqattn_view_t* q,
                                 const eqattn_view_t* k, const eqattn_view_t* v, const void* table,
                                 const int32_t* map, const eqattn_view_t* o, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (p == nullptr) return EQL_ERR_INVALID_ARG;
  eqlinear_status_t st = check_packing(b);
  if (st != EQL_OK) return st;
  FwdArgs a;
  memset(&a, 0, sizeof(a));
  if ((st = check_view(p, q, b->total_q, p->H, false, &a.q)) != EQL_OK) return st;
  if ((st = check_view(p, k, b->total_k, p->Hk, false, &a.k)) != EQL_OK) return st;
  if ((st = check_view(p, v, b->total_k, p->Hk, false, &a.v)) != EQL_OK) return st;
  if ((st = check_view(p, o, b->total_q, p->H, true, &a.o)) != EQL_OK) return st;
  if ((st = check_bias(p, table, map)) != EQL_OK) return st;
  if (!aligned16(lse) || !aligned16(workspace)) return EQL_ERR_MISALIGNED;
  const FwdShape s = forward_shape(p, b);
  const size_t need = forward_workspace(p, b, s);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return EQL_ERR_WORKSPACE;
  if (b->sequences == 0 || (s.chunks == 0 && s.tiles == 0)) return EQL_OK;
  fill_common(&a.c, p, b, table, map);
  a.lse = lse;
  a.tiles = s.tiles;
  a.packed = s.packed;
  a.splits = s.splits;
  a.chunks = s.chunks;
  a.part_o = (float*)workspace;
  a.part_ml = a.part_o + (size_t)s.splits * p->H * (size_t)b->total_q * (size_t)p->dim;
  Common probe = a.c;
  if (s.chunks == 0 &&
      spread(probe, (int64_t)(s.packed ? 1 : a.c.G) * s.tiles * s.splits, s.tiles == 1) < 0)
    return EQL_ERR_UNSUPPORTED;
  return hip_status("attention forward launch",
                    p->dtype == EQL_F16
                        ? launch_fwd_f16(a, s, (int)max_q_of(b), (hipStream_t)stream)
                        : launch_fwd_f32(a, s, (int)max_q_of(b), (hipStream_t)stream));
}

size_t eqattn_backward_workspace(eqattn_plan_t p, const eqattn_packing_t* b) {
  if (p == nullptr || !sizes_ok(b)) return 0;
  return delta_bytes(p, b) + hist_bytes(p, b, backward_shape(p, b)) +
         (p->buckets > 0 ? slices_bytes(p) : 0);
}

size_t eqattn_backward_workspace_no_dtable(eqattn_plan_t p, const eqattn_packing_t* b) {
  return p == nullptr || !sizes_ok(b) ? 0 : delta_bytes(p, b);
}

eqlinear_status_t eqattn_backward(eqattn_plan_t p, const eqattn_packing_t* b,
                                  const eqattn_view_t* dout, const eqattn_view_t* q,
                                  const eqattn_view_t* k, const eqattn_view_t* v,
                                  const eqattn_view_t* o, const float* lse, const void* table,
                                  const int32_t* map, const eqattn_view_t* dq,
                                  const eqattn_view_t* dk, const eqattn_view_t* dv, float* dtable,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (p == nullptr) return EQL_ERR_INVALID_ARG;
  eqlinear_status_t st = check_packing(b);
  if (st != EQL_OK) return st;
  BwdArgs a;
  memset(&a, 0, sizeof(a));
  const struct {
    const eqattn_view_t* from;
    int64_t tokens, heads;
    bool output;
    View* to;
  } views[] = {{dout, b->total_q, p->H, false, &a.dout}, {q, b->total_q, p->H, false, &a.q},
               {k, b->total_k, p->Hk, false, &a.k},      {v, b->total_k, p->Hk, false, &a.v},
               {o, b->total_q, p->H, false, &a.o},       {dq, b->total_q, p->H, true, &a.dq},
               {dk, b->total_k, p->Hk, true, &a.dk},     {dv, b->total_k, p->Hk, true, &a.dv}};
  for (const auto& w : views)
    if ((st = check_view(p, w.from, w.tokens, w.heads, w.output, w.to)) != EQL_OK) return st;
  if ((st = check_bias(p, table, map)) != EQL_OK) return st;
  if ((b->total_q > 0 && lse == nullptr) || (p->buckets == 0 && dtable != nullptr))
    return EQL_ERR_INVALID_ARG;
  if (!aligned16(lse) || !aligned16(dtable) || !aligned16(workspace)) return EQL_ERR_MISALIGNED;
  const size_t need =
      dtable != nullptr ? eqattn_backward_workspace(p, b) : eqattn_backward_workspace_no_dtable(p, b);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return EQL_ERR_WORKSPACE;
  const BwdShape s = backward_shape(p, b);
  fill_common(&a.c, p, b, table, map);
  a.lse = lse;
  a.delta = (float*)workspace;
  float* hist = (float*)((char*)workspace + delta_bytes(p, b));
  double* slices = (double*)((char*)hist + hist_bytes(p, b, s));
  a.hist = dtable != nullptr ? hist : nullptr;
  a.chunks = s.chunks;
  a.c.slot_rows = s.chunks > 0 ? 0 : 32 * s.waves_q;
  if (b->sequences > 0) {
    Common probe = a.c;
    if (spread(probe, (int64_t)a.c.G * s.tiles_q, s.tiles_q == 1) < 0 ||
        spread(probe, s.tiles_k, s.tiles_k == 1) < 0)
      return EQL_ERR_UNSUPPORTED;
    st = hip_status("attention backward launch",
                    p->dtype == EQL_F16 ? launch_bwd_f16(a, s, (hipStream_t)stream)
                                        : launch_bwd_f32(a, s, (hipStream_t)stream));
    if (st != EQL_OK) return st;
  }
  if (dtable == nullptr) return EQL_OK;
  return hip_status("bias gradient launch",
                    launch_bias_finish(a.c, hist, (int)hist_parts(b, s), slices, dtable,
                                       (hipStream_t)stream));
}

}  // extern "C"
