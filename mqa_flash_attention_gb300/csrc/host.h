// Host helpers of the C ABI shared by its translation units (defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "ds4a.h"

namespace ds4a {

struct HostDevice {
  int sm_count;
  unsigned int *err;  // device error word
};
// The current device, its kernels prepared; DS4A_ERR_UNSUPPORTED off sm_103a.
ds4a_status host_device(HostDevice *out);
// A launch's result as a status, the CUDA error kept for ds4a_last_cuda_error.
ds4a_status host_launched(cudaError_t e);
// Q [n][64][512]: the eight [64 heads][64 dims] boxes of a token per copy.
ds4a_status host_encode_q(CUtensorMap *m, const void *base, int n, int64_t stride);
// Paged rows in runs of run_rows rows and `blocks` blocks of 64 dims (see
// PagedAttnParams and TreeAttnParams).
ds4a_status host_encode_pages(CUtensorMap *m, const void *base, bool e4m3, int page_rows, int n_pages,
                              int64_t row_stride, int64_t page_stride, int run_rows, int blocks = 2);

}  // namespace ds4a
