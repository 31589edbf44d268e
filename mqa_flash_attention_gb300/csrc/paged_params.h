// Launch parameters of the kernels around the paged K/V cache and of the
// norm, shared by the host code that fills them and by the kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace ds4a {

// One segment of a paged cache (raw or compressed rows).  Offsets in bytes.
struct PagedSeg {
  const uint8_t *k, *v;
  long long row_stride, page_stride;
  int page_rows, n_pages;
  int page_shift;                  // log2 of page_rows, or -1
  const float *k_scale, *v_scale;  // E4M3 rows: [n_pages][page_rows]
  const int32_t *table;
  long long table_stride;          // elements
  int max_rows;                    // rows a table can name (0: no rows)
};

struct PagedAttnParams {
  CUtensorMap tm_q;        // 4-D {64, 64 heads, n_seq, 8 dim blocks}, box {64, 64, 1, 8}
  // Compressed rows by runs of run_rows rows: fp16 5-D {64 dims, 8 rows, 8
  // blocks, page_rows / 8, pages}, box {64, 8, 2, run_rows / 8, 1}; codes 3-D
  // {512, page_rows, pages}, box {128, run_rows, 1}.
  CUtensorMap tm_k, tm_v;
  int run_rows, run_shift; // 8 .. 128, a power of two, and its log2; 0: no TMA loads
  uint32_t run_bytes;      // of a run, first row to last, or 0: not worth a prefetch as one block
  PagedSeg seg[2];         // raw, compressed
  const int4 *geom;        // (q_pos, n_raw, raw_pos0, n_comp) per sequence
  int n_seq, ratio, window;
  float scale_log2;
  __half *o;
  long long o_stride;      // elements
  float *lse;              // decode: written, or NULL
  float *ws_o;             // [slots][64][512] normalised partial outputs
  float2 *ws_ml;           // [slots][64] (m in log2 units, l)
  int2 *ws_plan;           // [n_seq] (first slot, slots) of the sequences split over several CTAs
  const float *lse_in;     // weights: [n_seq][64]
  const float *acc_in;     // weights: what rows received before, or NULL
  long long acc_in_stride; // elements
  float *acc_out;
  long long acc_out_stride;
  float decay;
  unsigned long long timeout_ns;
  unsigned int *err;
};
cudaError_t prepare_paged_kernels();  // shared-memory opt-in and code of the paged attention kernels
cudaError_t launch_paged_decode(const PagedAttnParams &p, bool e4m3, bool shared, int grid, cudaStream_t s);
cudaError_t launch_paged_merge(const PagedAttnParams &p, cudaStream_t s);
cudaError_t launch_paged_weights(const PagedAttnParams &p, bool e4m3, int grid, cudaStream_t s);

struct EvictParams {
  const int4 *geom;
  int n_seq, ratio;
  PagedSeg rows;
  const float *weights;
  long long weight_stride;
  const int32_t *ids;
  long long id_stride;
  int n_keep, n_first, n_recent;
  int32_t *kept;
  long long kept_stride;
  float *weights_out;
  long long weight_out_stride;
  int32_t *ids_out;
  long long id_out_stride;
  uint8_t *n_out;
  long long n_out_stride;  // bytes
  int2 *n_moves;           // workspace: [n_seq] (rows moved, n')
  uint32_t *stay;          // workspace: [n_seq][stay_words] a bit per slot below n': its row stays
  int stay_words;          // ceil(n_keep / 32)
  int32_t *from, *to;      // workspace: [n_seq][n_keep] slots of the moved rows, and the freed slots they take
  int cached;              // keys of a CTA's rows kept in shared memory (0: recomputed from the weights)
  int move_here;           // set by launch_evict: the selection moves the rows, too
};
int evict_cluster(int max_rows);
int evict_cached_keys(int max_rows, int cluster);
cudaError_t launch_evict(EvictParams p, cudaStream_t s);
cudaError_t prepare_cache_kernels();

struct AppendParams {
  PagedSeg rows;
  const uint8_t *k, *v;
  long long new_stride;
  const int32_t *slots;
  int n;
};
cudaError_t launch_append(const AppendParams &p, cudaStream_t s);

struct NormParams {
  int n, width;
  const uint8_t *x, *res;
  uint8_t *res_out;
  long long x_stride, res_stride, res_out_stride;  // bytes
  const float *weight;
  float eps, inv_width;
  int group;   // values per scale, 0: the row
  uint8_t *codes;
  long long code_stride;
  float *scales;
  long long scale_stride;  // elements
  uint8_t *y;
  long long y_stride;
};
cudaError_t launch_norm(const NormParams &p, bool fp32, int sm_count, cudaStream_t s);
cudaError_t preload_norm_kernels();

}  // namespace ds4a
