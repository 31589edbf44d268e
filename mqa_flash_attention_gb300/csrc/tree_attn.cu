// Attention of several new tokens per sequence over a paged K/V cache.
//
//   o[t][h] = sum_j softmax_j(scale q[t][h].k_j) v_j over the cached raw rows of
//             token t's window, the rows of t and its ancestors, and the
//             compressed rows whose span has ended
//
// (64 query heads over one K/V row of 512; "DwarfStar 4 (DS4) - DeepSeek V4 Flash
// Inference Engine", "Fixed Model Shape" and "Layer Compression".)
//
// A warp per token and head goes through the rows once, with the running maximum
// and sum of the softmax; a lane holds 16 dims of q and o.
#include "attn_params.h"
#include "internal.h"
#include "ptx.cuh"
#include "step_params.h"

namespace ds4a {

namespace {

constexpr int kWarps = 8;

template <bool E4M3>
__device__ __forceinline__ void row16(const uint8_t *row, int lane, float (&x)[16]) {
  if (E4M3) {
    const uint4 c = *reinterpret_cast<const uint4 *>(row + 16 * lane);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
    const uint4 a = reinterpret_cast<const uint4 *>(row + 32 * lane)[0], b = reinterpret_cast<const uint4 *>(row + 32 * lane)[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) tree_attn_kernel(const TreeAttnParams p) {
  const int lane = threadIdx.x & 31, h = (blockIdx.x % (kH / kWarps)) * kWarps + (threadIdx.x >> 5);
  const int at = blockIdx.x / (kH / kWarps);
  grid_launch_dependents();
  grid_dependency_wait();
  // The sequence of token `at`: the last one that begins at or before it.
  int lo = 0, hi = p.n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (min(max(p.first[mid], 0), p.n_tok) <= at) lo = mid; else hi = mid;
  }
  const int b = lo, t0 = min(max(p.first[b], 0), p.n_tok);
  if (at < t0 || at >= min(max(p.first[b + 1], t0), p.n_tok)) return;
  const int t = at - t0;
  const int4 g = p.geom[b];
  const long long pos0 = max(g.x, 0), raw_pos0 = max(g.z, 0);
  const int n_raw = min(max(g.y, 0), p.seg[0].max_rows), n_comp = min(max(g.w, 0), p.seg[1].max_rows);
  auto parent_of = [&](int u) {
    if (p.parent == nullptr) return u - 1;
    const int v = p.parent[t0 + u];
    return v >= 0 && v < u ? v : -1;
  };
  int depth = 0;
  if (p.parent == nullptr)
    depth = t;
  else
    for (int u = parent_of(t); u >= 0; u = parent_of(u)) ++depth;
  const long long pos = pos0 + depth;
  float q[16], o[16], m = -INFINITY, l = 0.f;
  row16<false>(p.q + at * p.q_stride + h * 1024, lane, q);
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  auto take = [&](int sg, long long row) {
    const PagedSeg &s = p.seg[sg];
    if (row >= s.max_rows) return;
    const int pi = (int)row / s.page_rows, page = s.table[b * s.table_stride + pi], slot = (int)row - pi * s.page_rows;
    if ((unsigned)page >= (unsigned)s.n_pages) return;
    const long long off = page * s.page_stride + slot * s.row_stride, sr = (long long)page * s.page_rows + slot;
    float k[16], v[16], x = 0.f;
    row16<E4M3>(s.k + off, lane, k);
    row16<E4M3>(s.v + off, lane, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= p.scale_log2 * (E4M3 ? s.k_scale[sr] : 1.f);
    const float next = fmaxf(m, x);
    const float a = m == next ? 1.f : exp2f(m - next), w = exp2f(x - next);
    m = next;
    l = fmaf(l, a, w);
    const float wv = w * (E4M3 ? s.v_scale[sr] : 1.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = fmaf(o[i], a, wv * v[i]);
  };
  if (p.parent == nullptr || t < kTreeTokens) {
    const int nc = (int)min((long long)n_comp, (pos + 1) / p.ratio);
    for (int c = 0; c < nc; ++c) take(1, c);
    const long long r0 = max(0ll, pos - p.window + 1 - raw_pos0), r1 = min((long long)n_raw, pos + 1 - raw_pos0);
    for (long long i = r0; i < r1; ++i) take(0, i);
    int far = 0;
    for (int u = t; u >= 0 && far < p.window; u = parent_of(u), ++far) take(0, (long long)n_raw + u);
  }
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  __half2 out[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = __floats2half2_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
  uint4 *dst = reinterpret_cast<uint4 *>(p.o + at * p.o_stride + h * kD + 16 * lane);
  dst[0] = reinterpret_cast<const uint4 *>(out)[0];
  dst[1] = reinterpret_cast<const uint4 *>(out)[1];
  if (lane == 0 && p.lse != nullptr) p.lse[(long long)at * kH + h] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

cudaError_t launch_tree_attn(const TreeAttnParams &p, bool e4m3, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_tok * (kH / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return e4m3 ? cudaLaunchKernelEx(&cfg, tree_attn_kernel<true>, p)
              : cudaLaunchKernelEx(&cfg, tree_attn_kernel<false>, p);
}

cudaError_t prepare_tree_kernels() {
  for (const void *f : {(const void *)tree_attn_kernel<true>, (const void *)tree_attn_kernel<false>}) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ds4a
