// Root-mean-square norm with the residual's addition, quantised to E4M3.
//
//   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * weight,
//   scale_g = max_g |y| / 448,  code = E4M3(y * (448 / max_g |y|))
//
// ("DwarfStar 4 (DS4) - DeepSeek V4 Flash Inference Engine", section
// "Whole-Model Graph Execution": projections with a fused RMS norm; the code
// is that of quantize_fp8_kernel.)  No contraction: a row is read once, kept
// in registers over both reductions (the square sum, then a group's largest
// magnitude), and written once, so memory bounds it.
//
// A thread holds V vectors of 8 values.  A group of 32, 64, 128 or 256 values
// is 4, 8, 16 or 32 consecutive vectors, held by as many consecutive lanes of
// one warp, so a group's maximum is a few shuffles.  Rows of up to 512 values
// take one warp each (no block barrier); longer ones a block.
#include "internal.h"
#include "paged_params.h"
#include "ptx.cuh"

namespace ds4a {

namespace {

constexpr int kWarpRows = 4;         // rows per block of the warp-per-row form
constexpr int kWarpRowWidth = 512;   // widest row a warp takes: two vectors a lane
constexpr float kLeastMax = 7.8886090522101181e-31f;  // 2^-100: 448 / max stays finite far above it

template <typename T>
__device__ __forceinline__ void load8(const uint8_t *row, int vec, float (&v)[8]) {
  if (sizeof(T) == 2) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(row) + vec);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(row) + 2 * vec);
    const float4 b = __ldg(reinterpret_cast<const float4 *>(row) + 2 * vec + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

__device__ __forceinline__ uint4 pack_half8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ void store8(uint8_t *row, int vec, const float (&v)[8]) {
  if (sizeof(T) == 2) {
    reinterpret_cast<uint4 *>(row)[vec] = pack_half8(v);
  } else {
    reinterpret_cast<float4 *>(row)[2 * vec] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(row)[2 * vec + 1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Non-negative floats order like their bit patterns.
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

template <typename T, int V, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kWarpRows) rmsnorm_fp8_kernel(const NormParams p) {
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int threads = BLOCK ? blockDim.x : 32;  // of a row
  const int tid = BLOCK ? threadIdx.x : lane;
  const long long r = BLOCK ? (long long)blockIdx.x : (long long)blockIdx.x * kWarpRows + warp;
  grid_launch_dependents();
  grid_dependency_wait();
  if (r >= p.n) return;  // a whole warp or a whole block: no barrier is left waiting
  const int vecs = p.width >> 3;
  const uint8_t *xrow = p.x + r * p.x_stride;
  const uint8_t *rrow = p.res != nullptr ? p.res + r * p.res_stride : nullptr;
  float h[V][8];
  float w[V][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = tid + i * threads;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = w[i][e] = 0.f;
    if (vec < vecs) {
      load8<T>(xrow, vec, h[i]);
      load8<float>(reinterpret_cast<const uint8_t *>(p.weight), vec, w[i]);
    }
  }
  if (rrow != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = tid + i * threads;
      if (vec < vecs) {
        float q[8];
        load8<T>(rrow, vec, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += q[e];
        store8<T>(p.res_out + r * p.res_out_stride, vec, h[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
  ss = warp_sum(ss);
  if (BLOCK) {
    if (lane == 0) red[0][warp] = ss;
    __syncthreads();
    ss = warp_sum(lane < (threads >> 5) ? red[0][lane] : 0.f);
  }
  const float rs = __frsqrt_rn(__fdiv_rn(ss, (float)p.width) + p.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = tid + i * threads;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * rs * w[i][e];
    if (p.y != nullptr && vec < vecs) reinterpret_cast<uint4 *>(p.y + r * p.y_stride)[vec] = pack_half8(h[i]);
  }
  if (p.codes == nullptr) return;
  float m[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    m[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m[i] = fmaxf(m[i], fabsf(h[i][e]));
  }
  if (p.group == 0) {
    float t = m[0];
#pragma unroll
    for (int i = 1; i < V; ++i) t = fmaxf(t, m[i]);
    t = warp_max(t);
    if (BLOCK) {
      if (lane == 0) red[1][warp] = t;
      __syncthreads();
      t = warp_max(lane < (threads >> 5) ? red[1][lane] : 0.f);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) m[i] = t;
  } else {
    const int span = p.group >> 3;  // lanes of a group
#pragma unroll
    for (int i = 0; i < V; ++i)
      for (int o = 1; o < span; o <<= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
  }
  float *srow = p.scales + r * p.scale_stride;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = tid + i * threads;
    if (vec >= vecs) continue;
    uint32_t out[2] = {0u, 0u};
    const bool some = m[i] > kLeastMax;
    if (some) {
      const float inv = __fdiv_rn(448.f, m[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
            : "=h"(c)
            : "f"(__fmul_rn(h[i][2 * k + 1], inv)), "f"(__fmul_rn(h[i][2 * k], inv)));
        out[k >> 1] |= static_cast<uint32_t>(c) << (16 * (k & 1));
      }
    }
    reinterpret_cast<uint2 *>(p.codes + r * p.code_stride)[vec] = make_uint2(out[0], out[1]);
    const bool first = p.group == 0 ? vec == 0 : (vec & ((p.group >> 3) - 1)) == 0;
    if (first) srow[p.group == 0 ? 0 : vec / (p.group >> 3)] = some ? __fdiv_rn(m[i], 448.f) : 0.f;
  }
}

template <typename T>
const void *norm_kernel(int v, bool block) {
  if (!block) return (const void *)rmsnorm_fp8_kernel<T, 2, false>;
  return v == 1 ? (const void *)rmsnorm_fp8_kernel<T, 1, true>
                : v == 2 ? (const void *)rmsnorm_fp8_kernel<T, 2, true> : (const void *)rmsnorm_fp8_kernel<T, 4, true>;
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, bool fp32, cudaStream_t s) {
  const int vecs = p.width / 8;
  const bool block = p.width > kWarpRowWidth;
  const int v = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
  const int threads = block ? ((vecs + v - 1) / v + 31) / 32 * 32 : 32 * kWarpRows;
  const void *f = fp32 ? norm_kernel<float>(v, block) : norm_kernel<__half>(v, block);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(block ? p.n : (p.n + kWarpRows - 1) / kWarpRows);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *args[] = {const_cast<NormParams *>(&p)};
  return cudaLaunchKernelExC(&cfg, f, args);
}

cudaError_t preload_norm_kernels() {
  for (int block = 0; block < 2; ++block)
    for (int v = 1; v <= 4; v *= 2)
      for (const void *f : {norm_kernel<float>(v, block), norm_kernel<__half>(v, block)}) {
        cudaFuncAttributes a;
        const cudaError_t e = cudaFuncGetAttributes(&a, f);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

}  // namespace ds4a
