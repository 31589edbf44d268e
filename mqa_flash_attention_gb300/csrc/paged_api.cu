// C ABI of the paged cache and of the norm (declared in include/ds4a.h):
// argument checks, work splitting and launches.  No device memory is
// allocated here; every buffer belongs to the caller.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "ds4a.h"
#include "host.h"
#include "internal.h"
#include "paged_params.h"
#include "step_params.h"

namespace {

using ds4a::HostDevice;
using ds4a::PagedSeg;

constexpr unsigned long long kTimeoutNs = 2000000000ull;  // 2 s per wait
constexpr int64_t kMostBytes = 1LL << 39;  // of any stride
constexpr int32_t kMostRows = 1 << 30;     // rows of a sequence
constexpr int32_t kMostSeqs = 1 << 20;
constexpr int32_t kMostTokens = 1 << 20;   // new tokens of a call
constexpr float kLog2e = 1.4426950408889634f;

cudaStream_t as_cuda(ds4a_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool stride_ok(int64_t s, int64_t least, int64_t step) { return s >= least && s % step == 0 && s < kMostBytes; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Byte range [lo, hi) of `rows` rows of `row_bytes` at `stride`.
struct Span {
  uintptr_t lo, hi;
};
Span span(const void *p, int64_t rows, int64_t stride, int64_t row_bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, p != nullptr && rows > 0 ? lo + (uintptr_t)((rows - 1) * stride + row_bytes) : lo};
}
bool meet(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }
// A written range against one read: the same range at the same stride, or apart.
bool same_or_apart(Span a, int64_t stride_a, Span b, int64_t stride_b) {
  return !meet(a, b) || (a.lo == b.lo && stride_a == stride_b);
}

// n whole numbers in a row (none: a range that meets nothing).
Span ints(const int32_t *p, int64_t n) { return p != nullptr && n > 0 ? span(p, 1, 0, 4 * n) : Span{0, 0}; }
// Every output apart from every input and from every other output.
bool apart(const Span *out, int n_out, const Span *in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (meet(out[i], in[j])) return false;
    for (int j = i + 1; j < n_out; ++j)
      if (meet(out[i], out[j])) return false;
  }
  return true;
}

bool has_rows(const ds4a_paged_rows *r) { return r->max_pages > 0; }

// The pool of a segment (not its table).
bool pool_ok(const ds4a_paged_rows *r, bool need_v) {
  const bool e4m3 = r->k_scale != nullptr || r->v_scale != nullptr;
  const int64_t row = e4m3 ? DS4A_HEAD_DIM : DS4A_ROW_BYTES;
  if (r->page_rows < 1 || r->n_pages < 1 || r->page_rows > kMostRows) return false;
  if (r->k == nullptr || !aligned(r->k, 16)) return false;
  if (need_v && (r->v == nullptr || !aligned(r->v, 16))) return false;
  if (!stride_ok(r->row_stride, row, 16)) return false;
  // A page's rows lie within the page.
  if (r->page_stride % 16 != 0 || r->page_stride >= kMostBytes ||
      r->page_stride < (int64_t)(r->page_rows - 1) * r->row_stride + row)
    return false;
  if (e4m3 && (r->k_scale == nullptr || !aligned(r->k_scale, 4))) return false;
  if (e4m3 && need_v && (r->v_scale == nullptr || !aligned(r->v_scale, 4))) return false;
  return true;
}

bool table_ok(const ds4a_paged_rows *r) {
  if (r->table == nullptr || !aligned(r->table, 4)) return false;
  if (!stride_ok(r->table_stride, 4LL * r->max_pages, 4)) return false;
  return (int64_t)r->max_pages * r->page_rows <= kMostRows;
}

// The pools, scales and table of a segment with rows.
constexpr int kSegSpans = 5;
int seg_spans(const ds4a_paged_rows *r, int32_t n_seq, Span *out) {
  const bool e4m3 = r->k_scale != nullptr;
  const int64_t page = (int64_t)(r->page_rows - 1) * r->row_stride + (e4m3 ? DS4A_HEAD_DIM : DS4A_ROW_BYTES);
  const int64_t scales = 4LL * r->page_rows;
  int n = 0;
  for (const void *pool : {r->k, r->v}) out[n++] = span(pool, r->n_pages, r->page_stride, page);
  if (e4m3)
    for (const float *scale : {r->k_scale, r->v_scale}) out[n++] = span(scale, r->n_pages, scales, scales);
  out[n++] = span(r->table, n_seq, r->table_stride, 4LL * r->max_pages);
  return n;
}

// The exponent of a power of two, -1 otherwise.
int log2_of(int n) {
  for (int i = 0; i < 31; ++i)
    if (n == 1 << i) return i;
  return -1;
}

PagedSeg seg_of(const ds4a_paged_rows *r) {
  PagedSeg s;
  std::memset(&s, 0, sizeof(s));
  s.page_rows = 1;
  s.k = static_cast<const uint8_t *>(r->k);
  s.v = static_cast<const uint8_t *>(r->v);
  s.row_stride = r->row_stride;
  s.page_stride = r->page_stride;
  s.page_rows = r->page_rows;
  s.page_shift = log2_of(r->page_rows);
  s.n_pages = r->n_pages;
  s.k_scale = r->k_scale;
  s.v_scale = r->v_scale;
  s.table = r->table;
  s.table_stride = r->table_stride / 4;
  s.max_rows = r->max_pages * r->page_rows;
  return s;
}

PagedSeg no_rows() {
  PagedSeg s;
  std::memset(&s, 0, sizeof(s));
  s.page_rows = 1;
  return s;
}

ds4a_status check_batch(int32_t n_seq, const ds4a_layout *shape, const int32_t *seq_geom) {
  if (shape->window < 1 || !std::isfinite(shape->scale * kLog2e) || shape->ratio < 1) return DS4A_ERR_INVALID_ARG;
  if (seq_geom == nullptr || !aligned(seq_geom, 16)) return DS4A_ERR_INVALID_ARG;
  return n_seq > (1 << 20) ? DS4A_ERR_INVALID_ARG : DS4A_OK;
}

bool q_ok(const void *q, int64_t stride) {
  return q != nullptr && aligned(q, 16) && stride_ok(stride, 64LL * DS4A_ROW_BYTES, 16);
}

// Rows of a run that TMA copies at once: the largest power of two that divides
// a page's rows, 128 at most; 0 (all rows gathered) below 8.
int run_rows_of(int page_rows) {
  const int run = page_rows & -page_rows;
  return run > 128 ? 128 : run < 8 ? 0 : run;
}

// The tensor maps of the compressed rows, when their pages allow them.
ds4a_status encode_comp(ds4a::PagedAttnParams &p, const ds4a_paged_rows *r, bool need_v) {
  p.run_rows = has_rows(r) ? run_rows_of(r->page_rows) : 0;
  if (p.run_rows == 0) return DS4A_OK;
  p.run_shift = log2_of(p.run_rows);
  const bool e4m3 = r->k_scale != nullptr;
  // Rows further apart (one layer of a pool that interleaves several): a run's
  // block would bring more of other rows than of these.
  const int64_t row = e4m3 ? DS4A_HEAD_DIM : DS4A_ROW_BYTES;
  if (r->row_stride <= 2 * row) p.run_bytes = (uint32_t)((p.run_rows - 1) * r->row_stride + row);
  ds4a_status st = ds4a::host_encode_pages(&p.tm_k, r->k, e4m3, r->page_rows, r->n_pages, r->row_stride,
                                           r->page_stride, p.run_rows);
  if (st == DS4A_OK && need_v)
    st = ds4a::host_encode_pages(&p.tm_v, r->v, e4m3, r->page_rows, r->n_pages, r->row_stride, r->page_stride,
                                 p.run_rows);
  return st;
}

int64_t tiles_of(int64_t rows) { return (rows + 127) / 128; }

// A slot per CTA and one more per sequence, and the plan of the merge.
size_t decode_workspace(int32_t n_seq, int ctas) {
  const size_t slots = (size_t)n_seq + ctas;
  return slots * DS4A_HEADS * (DS4A_HEAD_DIM * sizeof(float) + sizeof(float2)) + (size_t)n_seq * sizeof(int2);
}

// The workspace of the attention of several new tokens: the plan, then partial
// results of two items of two tokens per pair of CTAs.
struct TreeSpace {
  int clusters, max_units;
  size_t start, unit, seq, ml, o, bytes;
};
TreeSpace tree_space(int32_t n_seq, int32_t n_tok, int ctas) {
  TreeSpace t;
  t.clusters = ctas / 2;
  t.max_units = (int)(((int64_t)n_tok + n_seq) / 2 + 1);
  const size_t slots = 4 * (size_t)t.clusters;
  t.start = 256;
  t.unit = t.start + align256(4 * ((size_t)t.clusters + 1));
  t.seq = t.unit + align256(128 * (size_t)t.max_units);
  t.ml = t.seq + align256(4 * (size_t)n_seq);
  t.o = t.ml + align256(slots * DS4A_HEADS * sizeof(float2));
  t.bytes = t.o + slots * DS4A_HEADS * DS4A_HEAD_DIM * sizeof(float);
  return t;
}

int device_sms() {
  int sms = 152, dev = -1, v = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0)
    sms = v;
  return sms;
}

}  // namespace

extern "C" {

size_t ds4a_attn_decode_paged_workspace_size(int32_t n_seq) {
  if (n_seq <= 0) return 0;
  return decode_workspace(n_seq, device_sms());
}

ds4a_status ds4a_attn_decode_paged(int32_t n_seq, const ds4a_layout *shape, const int32_t *seq_geom,
                                   const ds4a_paged_batch *X, void *workspace, size_t workspace_bytes,
                                   ds4a_stream_t stream) {
  if (n_seq < 0 || shape == nullptr || X == nullptr) return DS4A_ERR_INVALID_ARG;
  if (n_seq == 0) return DS4A_OK;
  ds4a_status st = check_batch(n_seq, shape, seq_geom);
  if (st != DS4A_OK) return st;
  if (!q_ok(X->q, X->q_seq_stride) || !q_ok(X->o, X->o_seq_stride)) return DS4A_ERR_INVALID_ARG;
  if (X->lse != nullptr && !aligned(X->lse, 4)) return DS4A_ERR_INVALID_ARG;
  bool e4m3 = false, any = false, shared = true;
  int64_t most = 0;  // rows a token can see
  for (const ds4a_paged_rows *r : {&X->raw, &X->comp}) {
    if (r->max_pages < 0) return DS4A_ERR_INVALID_ARG;
    if (!has_rows(r)) continue;
    if (!pool_ok(r, true) || !table_ok(r)) return DS4A_ERR_INVALID_ARG;
    const bool f8 = r->k_scale != nullptr;
    if (any && f8 != e4m3) return DS4A_ERR_INVALID_ARG;  // one format for both segments
    e4m3 = f8;
    any = true;
    shared = shared && r->k == r->v && r->k_scale == r->v_scale;
    const int64_t rows = (int64_t)r->max_pages * r->page_rows;
    most += r == &X->raw && rows > shape->window ? shape->window : rows;
  }
  const int64_t tiles = n_seq * tiles_of(most);
  if (most > kMostRows || tiles > (1 << 29)) return DS4A_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < ds4a_attn_decode_paged_workspace_size(n_seq))
    return DS4A_ERR_WORKSPACE;
  HostDevice d;
  st = ds4a::host_device(&d);
  if (st != DS4A_OK) return st;
  ds4a::PagedAttnParams p;
  std::memset(&p, 0, sizeof(p));
  st = ds4a::host_encode_q(&p.tm_q, X->q, n_seq, X->q_seq_stride);
  if (st != DS4A_OK) return st;
  st = encode_comp(p, &X->comp, true);
  if (st != DS4A_OK) return st;
  p.seg[0] = has_rows(&X->raw) ? seg_of(&X->raw) : no_rows();
  p.seg[1] = has_rows(&X->comp) ? seg_of(&X->comp) : no_rows();
  p.geom = reinterpret_cast<const int4 *>(seq_geom);
  p.n_seq = n_seq;
  p.ratio = shape->ratio;
  p.window = shape->window;
  p.scale_log2 = shape->scale * kLog2e;
  p.o = static_cast<__half *>(X->o);
  p.o_stride = X->o_seq_stride / 2;
  p.lse = X->lse;
  const int ctas = d.sm_count;
  const size_t slots = (size_t)n_seq + ctas;
  p.ws_o = static_cast<float *>(workspace);
  p.ws_ml = reinterpret_cast<float2 *>(p.ws_o + slots * DS4A_HEADS * DS4A_HEAD_DIM);
  p.ws_plan = reinterpret_cast<int2 *>(p.ws_ml + slots * DS4A_HEADS);
  p.timeout_ns = kTimeoutNs;
  p.err = d.err;
  const int grid = (int)(tiles < 1 ? 1 : tiles < ctas ? tiles : ctas);
  st = ds4a::host_launched(ds4a::launch_paged_decode(p, e4m3, any && shared, grid, as_cuda(stream)));
  if (st != DS4A_OK) return st;
  return ds4a::host_launched(ds4a::launch_paged_merge(p, as_cuda(stream)));
}

ds4a_status ds4a_attn_weights_paged(int32_t n_seq, const ds4a_layout *shape, const int32_t *seq_geom,
                                    const ds4a_paged_batch *X, const float *weights, int64_t weight_stride,
                                    float decay, float *out, int64_t out_stride, ds4a_stream_t stream) {
  if (n_seq < 0 || shape == nullptr || X == nullptr) return DS4A_ERR_INVALID_ARG;
  if (n_seq == 0) return DS4A_OK;
  ds4a_status st = check_batch(n_seq, shape, seq_geom);
  if (st != DS4A_OK) return st;
  if (!std::isfinite(decay) || X->comp.max_pages < 0) return DS4A_ERR_INVALID_ARG;
  if (!has_rows(&X->comp)) return DS4A_OK;
  if (!q_ok(X->q, X->q_seq_stride) || X->lse == nullptr || !aligned(X->lse, 4)) return DS4A_ERR_INVALID_ARG;
  ds4a_paged_rows rows = X->comp;
  rows.v = rows.k;
  rows.v_scale = rows.k_scale;
  if (!pool_ok(&rows, false) || !table_ok(&rows)) return DS4A_ERR_INVALID_ARG;
  const int64_t cols = (int64_t)rows.max_pages * rows.page_rows;
  if (out == nullptr || !aligned(out, 4) || !stride_ok(out_stride, 4 * cols, 4)) return DS4A_ERR_INVALID_ARG;
  if (weights != nullptr) {
    if (!aligned(weights, 4) || !stride_ok(weight_stride, 4 * cols, 4)) return DS4A_ERR_INVALID_ARG;
    if (!same_or_apart(span(out, n_seq, out_stride, 4 * cols), out_stride,
                       span(weights, n_seq, weight_stride, 4 * cols), weight_stride))
      return DS4A_ERR_INVALID_ARG;
  }
  const int64_t tiles = n_seq * tiles_of(cols);
  if (tiles > (1 << 29)) return DS4A_ERR_INVALID_ARG;
  HostDevice d;
  st = ds4a::host_device(&d);
  if (st != DS4A_OK) return st;
  ds4a::PagedAttnParams p;
  std::memset(&p, 0, sizeof(p));
  st = ds4a::host_encode_q(&p.tm_q, X->q, n_seq, X->q_seq_stride);
  if (st != DS4A_OK) return st;
  st = encode_comp(p, &rows, false);
  if (st != DS4A_OK) return st;
  p.seg[0] = no_rows();
  p.seg[1] = seg_of(&rows);
  p.geom = reinterpret_cast<const int4 *>(seq_geom);
  p.n_seq = n_seq;
  p.ratio = shape->ratio;
  p.window = shape->window;
  p.scale_log2 = shape->scale * kLog2e;
  p.lse_in = X->lse;
  p.acc_in = weights;
  p.acc_in_stride = weights != nullptr ? weight_stride / 4 : 0;
  p.acc_out = out;
  p.acc_out_stride = out_stride / 4;
  p.decay = decay;
  p.timeout_ns = kTimeoutNs;
  p.err = d.err;
  const int grid = (int)(tiles < d.sm_count ? tiles : d.sm_count);
  return ds4a::host_launched(ds4a::launch_paged_weights(p, rows.k_scale != nullptr, grid, as_cuda(stream)));
}

size_t ds4a_evict_paged_workspace_size(int32_t n_seq, int32_t n_keep) {
  if (n_seq <= 0 || n_keep <= 0) return 0;
  const size_t words = ((size_t)n_keep + 31) / 32;
  return align256(8 * (size_t)n_seq) + 4 * (size_t)n_seq * (2 * (size_t)n_keep + words);
}

ds4a_status ds4a_evict_paged(int32_t n_seq, const ds4a_layout *shape, const int32_t *seq_geom,
                             const ds4a_paged_rows *rows, const ds4a_eviction *E, void *workspace,
                             size_t workspace_bytes, ds4a_stream_t stream) {
  if (n_seq < 0 || shape == nullptr || rows == nullptr || E == nullptr) return DS4A_ERR_INVALID_ARG;
  if (n_seq == 0) return DS4A_OK;
  if (E->n_keep < 1 || E->n_keep > kMostRows || E->n_first < 0 || E->n_recent < 0 || shape->ratio < 1 ||
      n_seq > (1 << 20))
    return DS4A_ERR_INVALID_ARG;
  if (seq_geom == nullptr || !aligned(seq_geom, 16)) return DS4A_ERR_INVALID_ARG;
  if (rows->max_pages < 1 || !pool_ok(rows, true) || !table_ok(rows)) return DS4A_ERR_INVALID_ARG;
  const int64_t cols = (int64_t)rows->max_pages * rows->page_rows;
  if (E->weights == nullptr || !aligned(E->weights, 4) || !stride_ok(E->weight_stride, 4 * cols, 4))
    return DS4A_ERR_INVALID_ARG;
  if ((E->ids == nullptr) != (E->ids_out == nullptr)) return DS4A_ERR_INVALID_ARG;
  if (E->kept == nullptr || !aligned(E->kept, 4) || !stride_ok(E->kept_stride, 4LL * E->n_keep, 4))
    return DS4A_ERR_INVALID_ARG;
  if (E->n_out == nullptr || !aligned(E->n_out, 4) || !stride_ok(E->n_out_stride, 4, 4)) return DS4A_ERR_INVALID_ARG;
  const Span in_w = span(E->weights, n_seq, E->weight_stride, 4 * cols);
  if (E->weights_out != nullptr &&
      (!aligned(E->weights_out, 4) || !stride_ok(E->weight_out_stride, 4 * cols, 4) ||
       !same_or_apart(span(E->weights_out, n_seq, E->weight_out_stride, 4 * cols), E->weight_out_stride, in_w,
                      E->weight_stride)))
    return DS4A_ERR_INVALID_ARG;
  if (E->ids != nullptr &&
      (!aligned(E->ids, 4) || !stride_ok(E->id_stride, 4 * cols, 4) || !aligned(E->ids_out, 4) ||
       !stride_ok(E->id_out_stride, 4 * cols, 4) ||
       !same_or_apart(span(E->ids_out, n_seq, E->id_out_stride, 4 * cols), E->id_out_stride,
                      span(E->ids, n_seq, E->id_stride, 4 * cols), E->id_stride)))
    return DS4A_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < ds4a_evict_paged_workspace_size(n_seq, E->n_keep))
    return DS4A_ERR_WORKSPACE;
  if (n_seq * ((cols + 7) / 8) > INT32_MAX || n_seq * ((E->n_keep + 255LL) / 256) > INT32_MAX)
    return DS4A_ERR_INVALID_ARG;  // blocks of the move kernel
  HostDevice d;
  const ds4a_status st = ds4a::host_device(&d);
  if (st != DS4A_OK) return st;
  ds4a::EvictParams p;
  p.geom = reinterpret_cast<const int4 *>(seq_geom);
  p.n_seq = n_seq;
  p.ratio = shape->ratio;
  p.rows = seg_of(rows);
  p.weights = E->weights;
  p.weight_stride = E->weight_stride / 4;
  p.ids = E->ids;
  p.id_stride = E->ids != nullptr ? E->id_stride / 4 : 0;
  p.n_keep = E->n_keep;
  p.n_first = E->n_first;
  p.n_recent = E->n_recent;
  p.kept = E->kept;
  p.kept_stride = E->kept_stride / 4;
  p.weights_out = E->weights_out;
  p.weight_out_stride = E->weights_out != nullptr ? E->weight_out_stride / 4 : 0;
  p.ids_out = E->ids_out;
  p.id_out_stride = E->ids_out != nullptr ? E->id_out_stride / 4 : 0;
  p.n_out = reinterpret_cast<uint8_t *>(E->n_out);
  p.n_out_stride = E->n_out_stride;
  p.n_moves = static_cast<int2 *>(workspace);
  p.from = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + align256(8 * (size_t)n_seq));
  p.to = p.from + (size_t)n_seq * E->n_keep;
  p.stay_words = (E->n_keep + 31) / 32;
  p.stay = reinterpret_cast<uint32_t *>(p.to + (size_t)n_seq * E->n_keep);
  p.cached = ds4a::evict_cached_keys(p.rows.max_rows, ds4a::evict_cluster(p.rows.max_rows));
  return ds4a::host_launched(ds4a::launch_evict(p, as_cuda(stream)));
}

ds4a_status ds4a_append_paged(const ds4a_paged_rows *rows, int32_t n, const void *k, const void *v,
                              int64_t new_row_stride, const int32_t *slots, ds4a_stream_t stream) {
  if (n < 0 || rows == nullptr) return DS4A_ERR_INVALID_ARG;
  if (n == 0) return DS4A_OK;
  if (!pool_ok(rows, true)) return DS4A_ERR_INVALID_ARG;
  const bool one = rows->v == rows->k;
  if (k == nullptr || !aligned(k, 16) || !stride_ok(new_row_stride, DS4A_ROW_BYTES, 16)) return DS4A_ERR_INVALID_ARG;
  if (!one && (v == nullptr || !aligned(v, 16))) return DS4A_ERR_INVALID_ARG;
  if (slots == nullptr || !aligned(slots, 4)) return DS4A_ERR_INVALID_ARG;
  const int64_t row = rows->k_scale != nullptr ? DS4A_HEAD_DIM : DS4A_ROW_BYTES;
  const int64_t page = (int64_t)(rows->page_rows - 1) * rows->row_stride + row;
  // A row's K and V have a scale each, unless they are one row.
  const int64_t scales = 4LL * rows->page_rows;
  const Span ks = span(rows->k_scale, rows->n_pages, scales, scales);
  const Span vs = span(rows->v_scale, rows->n_pages, scales, scales);
  if (meet(ks, vs) && !(one && rows->k_scale == rows->v_scale)) return DS4A_ERR_INVALID_ARG;
  for (const void *pool : {rows->k, rows->v})
    for (const void *in : {k, one ? k : v})
      if (meet(span(pool, rows->n_pages, rows->page_stride, page), span(in, n, new_row_stride, DS4A_ROW_BYTES)))
        return DS4A_ERR_INVALID_ARG;
  HostDevice d;
  const ds4a_status st = ds4a::host_device(&d);
  if (st != DS4A_OK) return st;
  ds4a::AppendParams p;
  ds4a_paged_rows pool = *rows;
  pool.max_pages = 0;
  p.rows = seg_of(&pool);
  p.k = static_cast<const uint8_t *>(k);
  p.v = static_cast<const uint8_t *>(one ? k : v);
  p.new_stride = new_row_stride;
  p.slots = slots;
  p.n = n;
  return ds4a::host_launched(ds4a::launch_append(p, as_cuda(stream)));
}

size_t ds4a_page_tables_workspace_size(int32_t n_seq) {
  return n_seq <= 0 ? 0 : ((size_t)n_seq + 1) * sizeof(ds4a::PagePlan);
}

ds4a_status ds4a_page_tables(int32_t n_seq, const ds4a_page_lists *X, void *workspace, size_t workspace_bytes,
                             ds4a_stream_t stream) {
  if (n_seq < 0 || X == nullptr) return DS4A_ERR_INVALID_ARG;
  if (n_seq == 0) return DS4A_OK;
  if (n_seq > kMostSeqs || X->max_pages < 1 || X->page_rows < 1 || X->n_pages < 1 || X->n_slots < 0 ||
      (int64_t)X->max_pages * X->page_rows > kMostRows || (int64_t)X->n_pages * X->page_rows > INT32_MAX)
    return DS4A_ERR_INVALID_ARG;
  if (X->table == nullptr || !aligned(X->table, 4) || !stride_ok(X->table_stride, 4LL * X->max_pages, 4))
    return DS4A_ERR_INVALID_ARG;
  for (const int32_t *p : {(const int32_t *)X->free_pages, (const int32_t *)X->n_free, X->have, X->want,
                           (const int32_t *)X->first, (const int32_t *)X->n_short})
    if (p == nullptr || !aligned(p, 4)) return DS4A_ERR_INVALID_ARG;
  if (!aligned(X->drop, 4) || !aligned(X->slots, 4) || (X->n_slots > 0 && X->slots == nullptr))
    return DS4A_ERR_INVALID_ARG;
  const Span out[6] = {span(X->table, n_seq, X->table_stride, 4LL * X->max_pages), ints(X->free_pages, X->n_pages),
                       ints(X->n_free, 1), ints(X->slots, X->n_slots), ints(X->first, (int64_t)n_seq + 1),
                       ints(X->n_short, 1)};
  const Span in[3] = {ints(X->have, n_seq), ints(X->want, n_seq), ints(X->drop, n_seq)};
  if (!apart(out, 6, in, 3)) return DS4A_ERR_INVALID_ARG;
  const int64_t need = (int64_t)ds4a_page_tables_workspace_size(n_seq);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < (size_t)need) return DS4A_ERR_WORKSPACE;
  // The second kernel reads the counts again, and the plan that the first left.
  const Span ws = span(workspace, 1, 0, need);
  if (!apart(&ws, 1, in, 3) || !apart(&ws, 1, out, 6)) return DS4A_ERR_INVALID_ARG;
  HostDevice d;
  const ds4a_status st = ds4a::host_device(&d);
  if (st != DS4A_OK) return st;
  ds4a::PageTablesParams p;
  p.n_seq = n_seq;
  p.max_pages = X->max_pages;
  p.page_rows = X->page_rows;
  p.n_pages = X->n_pages;
  p.n_slots = X->n_slots;
  p.table = X->table;
  p.table_stride = X->table_stride / 4;
  p.free_pages = X->free_pages;
  p.n_free = X->n_free;
  p.slots = X->slots;
  p.first = X->first;
  p.n_short = X->n_short;
  p.have = X->have;
  p.want = X->want;
  p.drop = X->drop;
  p.plan = static_cast<ds4a::PagePlan *>(workspace);
  return ds4a::host_launched(ds4a::launch_page_tables(p, as_cuda(stream)));
}

size_t ds4a_attn_tree_paged_workspace_size(int32_t n_seq, int32_t n_tok) {
  if (n_seq <= 0 || n_tok <= 0) return 0;
  return tree_space(n_seq, n_tok, device_sms()).bytes;
}

ds4a_status ds4a_attn_tree_paged(int32_t n_seq, int32_t n_tok, const ds4a_layout *shape, const int32_t *seq_geom,
                                 const ds4a_paged_tree *X, void *workspace, size_t workspace_bytes,
                                 ds4a_stream_t stream) {
  if (n_seq < 0 || n_tok < 0 || shape == nullptr || X == nullptr) return DS4A_ERR_INVALID_ARG;
  if (n_seq == 0 || n_tok == 0) return DS4A_OK;
  ds4a_status st = check_batch(n_seq, shape, seq_geom);
  if (st != DS4A_OK) return st;
  if (n_tok > kMostTokens) return DS4A_ERR_INVALID_ARG;
  if (!q_ok(X->q, X->q_tok_stride) || !q_ok(X->o, X->o_tok_stride)) return DS4A_ERR_INVALID_ARG;
  if (!aligned(X->lse, 4) || X->first == nullptr || !aligned(X->first, 4) || !aligned(X->parent, 4))
    return DS4A_ERR_INVALID_ARG;
  bool e4m3 = false, any = false;
  int64_t most = 0;  // rows of a sequence
  for (const ds4a_paged_rows *r : {&X->raw, &X->comp}) {
    if (r->max_pages < 0) return DS4A_ERR_INVALID_ARG;
    if (!has_rows(r)) continue;
    if (!pool_ok(r, true) || !table_ok(r)) return DS4A_ERR_INVALID_ARG;
    const bool f8 = r->k_scale != nullptr;
    if (any && f8 != e4m3) return DS4A_ERR_INVALID_ARG;  // one format for both segments
    e4m3 = f8;
    any = true;
    most += (int64_t)r->max_pages * r->page_rows;
  }
  if (most > kMostRows) return DS4A_ERR_INVALID_ARG;
  // Other units still read q and the rows, and the merge the plan, when a unit's output is written.
  const Span out[3] = {span(X->o, n_tok, X->o_tok_stride, (int64_t)DS4A_HEADS * DS4A_ROW_BYTES),
                       span(X->lse, n_tok, 4 * DS4A_HEADS, 4 * DS4A_HEADS),
                       span(workspace, 1, 0, (int64_t)ds4a_attn_tree_paged_workspace_size(n_seq, n_tok))};
  Span in[4 + 2 * kSegSpans] = {span(X->q, n_tok, X->q_tok_stride, (int64_t)DS4A_HEADS * DS4A_ROW_BYTES),
                                ints(X->first, (int64_t)n_seq + 1), ints(X->parent, n_tok), ints(seq_geom, 4LL * n_seq)};
  int n_in = 4;
  for (const ds4a_paged_rows *r : {&X->raw, &X->comp})
    if (has_rows(r)) n_in += seg_spans(r, n_seq, in + n_in);
  if (!apart(out, 3, in, n_in)) return DS4A_ERR_INVALID_ARG;
  // Tiles of 256 rows, of pairs of tokens.
  if ((((int64_t)n_tok + n_seq) / 2 + 1) * ((most + 255) / 256 + 1) > (1 << 30)) return DS4A_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < ds4a_attn_tree_paged_workspace_size(n_seq, n_tok))
    return DS4A_ERR_WORKSPACE;
  HostDevice d;
  st = ds4a::host_device(&d);
  if (st != DS4A_OK) return st;
  ds4a::TreeAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.seg[0] = has_rows(&X->raw) ? seg_of(&X->raw) : no_rows();
  p.seg[1] = has_rows(&X->comp) ? seg_of(&X->comp) : no_rows();
  p.geom = reinterpret_cast<const int4 *>(seq_geom);
  p.first = X->first;
  p.parent = X->parent;
  p.n_seq = n_seq;
  p.n_tok = n_tok;
  p.ratio = shape->ratio;
  p.window = shape->window;
  p.scale_log2 = shape->scale * kLog2e;
  p.o = static_cast<__half *>(X->o);
  p.o_stride = X->o_tok_stride / 2;
  p.lse = X->lse;
  st = ds4a::host_encode_q(&p.tm_q, X->q, n_tok, X->q_tok_stride);
  if (st != DS4A_OK) return st;
  // Rows of a copy that lies within a page: 16 or 8 of either segment, and of the
  // compressed ones up to 64.  (Pages of other sizes are gathered row by row.)
  int grain = 16;
  for (const ds4a_paged_rows *r : {&X->raw, &X->comp})
    if (has_rows(r) && run_rows_of(r->page_rows) < grain) grain = run_rows_of(r->page_rows);
  p.grain = any ? grain : 0;
  if (p.grain > 0) {
    p.grain_shift = p.run_shift = log2_of(grain);
    const ds4a_paged_rows *segs[2] = {&X->raw, &X->comp};
    for (int i = 0; i < 2 && st == DS4A_OK; ++i) {
      const ds4a_paged_rows *r = segs[i];
      if (!has_rows(r)) continue;
      st = ds4a::host_encode_pages(&p.tm_kg[i], r->k, e4m3, r->page_rows, r->n_pages, r->row_stride, r->page_stride,
                                   grain, 1);
      if (st == DS4A_OK)
        st = ds4a::host_encode_pages(&p.tm_vg[i], r->v, e4m3, r->page_rows, r->n_pages, r->row_stride,
                                     r->page_stride, grain, 2);
    }
    if (st == DS4A_OK && has_rows(&X->comp)) {
      const ds4a_paged_rows *r = &X->comp;
      const int run = run_rows_of(r->page_rows) > 64 ? 64 : run_rows_of(r->page_rows);  // (a part of V has 64 rows)
      p.run_shift = log2_of(run);
      st = ds4a::host_encode_pages(&p.tm_k, r->k, e4m3, r->page_rows, r->n_pages, r->row_stride, r->page_stride, run, 1);
      if (st == DS4A_OK)
        st = ds4a::host_encode_pages(&p.tm_v, r->v, e4m3, r->page_rows, r->n_pages, r->row_stride, r->page_stride,
                                     run, 2);
    }
    if (st != DS4A_OK) return st;
  }
  const TreeSpace t = tree_space(n_seq, n_tok, d.sm_count);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.clusters = t.clusters;
  p.max_units = t.max_units;
  p.ws_head = reinterpret_cast<int4 *>(ws);
  p.ws_start = reinterpret_cast<int *>(ws + t.start);
  p.ws_unit = ws + t.unit;
  p.ws_seq = reinterpret_cast<int *>(ws + t.seq);
  p.ws_ml = reinterpret_cast<float2 *>(ws + t.ml);
  p.ws_o = reinterpret_cast<float *>(ws + t.o);
  p.timeout_ns = kTimeoutNs;
  p.err = d.err;
  return ds4a::host_launched(ds4a::launch_tree_attn(p, e4m3, as_cuda(stream)));
}

ds4a_status ds4a_tree_accept(int32_t n_seq, int32_t n_tok, const int32_t *first, const int32_t *parent,
                             const int32_t *token, const int32_t *target, const int32_t *prev, int32_t *path,
                             int64_t path_stride, int32_t width, int32_t *n_accepted, int32_t *next,
                             ds4a_stream_t stream) {
  if (n_seq < 0 || n_tok < 0 || width < 0) return DS4A_ERR_INVALID_ARG;
  if (n_seq == 0) return DS4A_OK;
  if (n_seq > kMostSeqs || n_tok > kMostRows || width > kMostRows) return DS4A_ERR_INVALID_ARG;
  for (const int32_t *p : {first, (const int32_t *)n_accepted, (const int32_t *)next})
    if (p == nullptr || !aligned(p, 4)) return DS4A_ERR_INVALID_ARG;
  if (n_tok > 0 && (token == nullptr || target == nullptr)) return DS4A_ERR_INVALID_ARG;
  if (!aligned(parent, 4) || !aligned(token, 4) || !aligned(target, 4) || !aligned(prev, 4))
    return DS4A_ERR_INVALID_ARG;
  if (width > 0 && (path == nullptr || !aligned(path, 4) || !stride_ok(path_stride, 4LL * width, 4)))
    return DS4A_ERR_INVALID_ARG;
  const Span out[3] = {span(path, width > 0 ? n_seq : 0, path_stride, 4LL * width), ints(n_accepted, n_seq),
                       ints(next, n_seq)};
  const Span in[5] = {ints(first, (int64_t)n_seq + 1), ints(parent, n_tok), ints(token, n_tok), ints(target, n_tok),
                      ints(prev, n_seq)};
  if (!apart(out, 3, in, 5)) return DS4A_ERR_INVALID_ARG;
  HostDevice d;
  const ds4a_status st = ds4a::host_device(&d);
  if (st != DS4A_OK) return st;
  ds4a::AcceptParams p;
  p.n_seq = n_seq;
  p.n_tok = n_tok;
  p.width = width;
  p.first = first;
  p.parent = parent;
  p.token = token;
  p.target = target;
  p.prev = prev;
  p.path = path;
  p.path_stride = path_stride / 4;
  p.n_accepted = n_accepted;
  p.next = next;
  return ds4a::host_launched(ds4a::launch_accept(p, as_cuda(stream)));
}

ds4a_status ds4a_commit_paged(int32_t n_seq, const ds4a_paged_rows *rows, const int32_t *seq_geom,
                              const int32_t *path, int64_t path_stride, int32_t width, const int32_t *n_accepted,
                              ds4a_stream_t stream) {
  if (n_seq < 0 || rows == nullptr || width < 0) return DS4A_ERR_INVALID_ARG;
  if (n_seq == 0 || width == 0) return DS4A_OK;
  if (n_seq > kMostSeqs || width > kMostRows) return DS4A_ERR_INVALID_ARG;
  if (rows->max_pages < 1 || !pool_ok(rows, true) || !table_ok(rows)) return DS4A_ERR_INVALID_ARG;
  // K and V apart have a scale array each.
  const int64_t scales = 4LL * rows->page_rows;
  if (rows->k != rows->v && rows->k_scale != nullptr &&
      meet(span(rows->k_scale, rows->n_pages, scales, scales), span(rows->v_scale, rows->n_pages, scales, scales)))
    return DS4A_ERR_INVALID_ARG;
  if (seq_geom == nullptr || !aligned(seq_geom, 16) || n_accepted == nullptr || !aligned(n_accepted, 4))
    return DS4A_ERR_INVALID_ARG;
  if (path == nullptr || !aligned(path, 4) || !stride_ok(path_stride, 4LL * width, 4)) return DS4A_ERR_INVALID_ARG;
  HostDevice d;
  const ds4a_status st = ds4a::host_device(&d);
  if (st != DS4A_OK) return st;
  ds4a::CommitParams p;
  p.rows = seg_of(rows);
  p.n_seq = n_seq;
  p.width = width;
  p.geom = reinterpret_cast<const int4 *>(seq_geom);
  p.path = path;
  p.path_stride = path_stride / 4;
  p.n_accepted = n_accepted;
  return ds4a::host_launched(ds4a::launch_commit(p, as_cuda(stream)));
}

ds4a_status ds4a_rmsnorm_fp8(const ds4a_norm *N, ds4a_stream_t stream) {
  if (N == nullptr) return DS4A_ERR_INVALID_ARG;
  if (N->n < 0 || N->n > kMostRows || N->width < 8 || N->width > 32768 || N->width % 8 != 0) return DS4A_ERR_INVALID_ARG;
  if (N->group != 0 && N->group != 32 && N->group != 64 && N->group != 128 && N->group != 256)
    return DS4A_ERR_INVALID_ARG;
  if (!(N->eps >= FLT_MIN) || !std::isfinite(N->eps)) return DS4A_ERR_INVALID_ARG;
  if (N->n == 0) return DS4A_OK;  // (the pointers of empty tensors say nothing)
  if (N->codes == nullptr && N->y == nullptr) return DS4A_ERR_INVALID_ARG;
  if ((N->codes == nullptr) != (N->scales == nullptr)) return DS4A_ERR_INVALID_ARG;
  if ((N->residual == nullptr) != (N->residual_out == nullptr)) return DS4A_ERR_INVALID_ARG;
  const int64_t row = (N->x_fp32 ? 4LL : 2LL) * N->width;
  const int64_t groups = N->group == 0 ? 1 : (N->width + N->group - 1) / N->group;
  if (N->x == nullptr || !aligned(N->x, 16) || !stride_ok(N->x_stride, row, 16)) return DS4A_ERR_INVALID_ARG;
  if (N->weight == nullptr || !aligned(N->weight, 16)) return DS4A_ERR_INVALID_ARG;
  if (N->residual != nullptr && (!aligned(N->residual, 16) || !stride_ok(N->residual_stride, row, 16) ||
                                 !aligned(N->residual_out, 16) || !stride_ok(N->residual_out_stride, row, 16)))
    return DS4A_ERR_INVALID_ARG;
  if (N->codes != nullptr && (!aligned(N->codes, 8) || !stride_ok(N->code_stride, N->width, 8) ||
                              !aligned(N->scales, 4) || !stride_ok(N->scale_stride, 4 * groups, 4)))
    return DS4A_ERR_INVALID_ARG;
  if (N->y != nullptr && (!aligned(N->y, 16) || !stride_ok(N->y_stride, 2LL * N->width, 16)))
    return DS4A_ERR_INVALID_ARG;
  const Span in[3] = {span(N->x, N->n, N->x_stride, row), span(N->residual, N->n, N->residual_stride, row),
                      span(N->weight, 1, 0, 4LL * N->width)};
  const Span out[4] = {span(N->residual_out, N->n, N->residual_out_stride, row),
                       span(N->codes, N->n, N->code_stride, N->width),
                       span(N->scales, N->n, N->scale_stride, 4 * groups),
                       span(N->y, N->n, N->y_stride, 2LL * N->width)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j) {
      const bool in_place = i == 0 && j < 2 && out[0].lo == in[j].lo &&
                            N->residual_out_stride == (j == 0 ? N->x_stride : N->residual_stride);
      if (!in_place && meet(out[i], in[j])) return DS4A_ERR_INVALID_ARG;
    }
    for (int j = i + 1; j < 4; ++j)
      if (meet(out[i], out[j])) return DS4A_ERR_INVALID_ARG;
  }
  HostDevice d;
  const ds4a_status st = ds4a::host_device(&d);
  if (st != DS4A_OK) return st;
  ds4a::NormParams p;
  p.n = N->n;
  p.width = N->width;
  p.x = static_cast<const uint8_t *>(N->x);
  p.x_stride = N->x_stride;
  p.res = static_cast<const uint8_t *>(N->residual);
  p.res_stride = N->residual_stride;
  p.res_out = static_cast<uint8_t *>(N->residual_out);
  p.res_out_stride = N->residual_out_stride;
  p.weight = N->weight;
  p.eps = N->eps;
  p.inv_width = 1.0f / (float)N->width;
  p.group = N->group;
  p.codes = N->codes;
  p.code_stride = N->code_stride;
  p.scales = N->scales;
  p.scale_stride = N->codes != nullptr ? N->scale_stride / 4 : 0;
  p.y = static_cast<uint8_t *>(N->y);
  p.y_stride = N->y_stride;
  return ds4a::host_launched(ds4a::launch_norm(p, N->x_fp32 != 0, d.sm_count, as_cuda(stream)));
}

}  // extern "C"
