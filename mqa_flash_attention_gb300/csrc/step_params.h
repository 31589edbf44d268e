// Launch parameters of the kernels of a step with several new tokens per
// sequence, shared by the host code that fills them and by the kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "paged_params.h"

namespace ds4a {

// Where a sequence's tables stand: pages it needs in all sequences before it,
// and new rows there (workspace of the page tables).
struct PagePlan {
  long long pages, rows;
};

struct PageTablesParams {
  int n_seq, max_pages, page_rows, n_pages, n_slots;
  int32_t *table;
  long long table_stride;  // elements
  int32_t *free_pages, *n_free, *slots, *first, *n_short;
  const int32_t *have, *want, *drop;
  PagePlan *plan;          // workspace: [n_seq + 1]; the last one: the list's top before any page is taken, all new rows
};
cudaError_t launch_page_tables(const PageTablesParams &p, cudaStream_t s);

struct AcceptParams {
  int n_seq, n_tok, width;
  const int32_t *first, *parent, *token, *target, *prev;
  int32_t *path;
  long long path_stride;   // elements
  int32_t *n_accepted, *next;
};
cudaError_t launch_accept(const AcceptParams &p, cudaStream_t s);

struct CommitParams {
  PagedSeg rows;
  int n_seq, width;
  const int4 *geom;
  const int32_t *path;
  long long path_stride;   // elements
  const int32_t *n_accepted;
};
cudaError_t launch_commit(const CommitParams &p, cudaStream_t s);

constexpr int kTreeTokens = 128;

struct TreeAttnParams {
  CUtensorMap tm_q;        // 4-D {64, 64 heads, n_tok, 8 dim blocks}, box {64, 64, 1, 8}
  // K by 64 dims and V by 128: fp16 5-D {64 dims, 8 rows, 8 blocks, page_rows / 8,
  // pages}, box {64, 8, 1 or 2, rows / 8, 1}; codes 3-D {512, page_rows, pages}, box
  // {64 or 128, rows, 1}.  Compressed rows by runs of 2^run_shift rows (at most 64),
  // and rows of either segment by grains of 8 or 16.
  CUtensorMap tm_k, tm_v, tm_kg[2], tm_vg[2];
  int grain, grain_shift, run_shift;  // grain 0: pages that TMA cannot copy
  PagedSeg seg[2];         // raw, compressed
  const int4 *geom;        // (q_pos, n_raw, raw_pos0, n_comp) per sequence
  const int32_t *first, *parent;
  int n_seq, n_tok, ratio, window;
  float scale_log2;
  __half *o;
  long long o_stride;      // elements
  float *lse;
  int clusters, max_units;
  // Workspace.
  int4 *ws_head;           // (tiles, tiles of a cluster, units, -)
  int *ws_start;           // [clusters] unit of a cluster's first tile
  void *ws_unit;           // [max_units] 128 bytes each
  int *ws_seq;             // [n_seq] units before
  float2 *ws_ml;           // [4 clusters][64] (m in log2 units, l)
  float *ws_o;             // [4 clusters][64][512] normalised partial outputs
  unsigned long long timeout_ns;
  unsigned int *err;
};
cudaError_t launch_tree_attn(const TreeAttnParams &p, bool e4m3, cudaStream_t s);
cudaError_t prepare_tree_kernels();

cudaError_t preload_step_kernels();

}  // namespace ds4a
