// Root-mean-square norm with the residual's addition, quantised to E4M3.
//
//   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * weight,
//   scale_g = max_g |y| / 448,  code = E4M3(y * (448 / max_g |y|))
//
// ("DwarfStar 4 (DS4) - DeepSeek V4 Flash Inference Engine", section
// "Whole-Model Graph Execution": projections with a fused RMS norm; the code
// is that of quantize_fp8_kernel.)  No contraction: a row is read once, kept
// in registers over both reductions (the square sum, then a group's largest
// magnitude), and written once.  2,048 rows of 4,096 fp16 values with a residual:
// 12.0 us, of which the issue slots of its 9.9 M warp instructions are 8.6 (all 59
// MB fit in L2); one row: 2.0 us on the device, 2.3 us of host time.
//
// A thread holds V vectors of 8 values.  A group of 32, 64, 128 or 256 values
// is 4, 8, 16 or 32 consecutive vectors, held by as many consecutive lanes of
// one warp, so a group's maximum is a few shuffles.  Rows of up to 512 values
// take one warp each (no block barrier); longer ones a block.  Blocks stay for
// many rows: the weight is read once per block and not once per row (it is
// as large as x and the residual together), and the next row's values are on
// their way while a row is reduced and written.
#include "internal.h"
#include "paged_params.h"
#include "ptx.cuh"

namespace ds4a {

namespace {

constexpr int kWarpRows = 4;         // rows per block of the warp-per-row form
constexpr int kWarpRowWidth = 512;   // widest row a warp takes: two vectors a lane
constexpr float kLeastMax = 7.8886090522101181e-31f;  // 2^-100: 448 / max stays finite far above it

// Eight values of a row as they are stored.
template <typename T>
struct Raw {
  uint4 a[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const uint8_t *row, int vec) {
  Raw<T> v;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    v.a[i] = __ldcs(reinterpret_cast<const uint4 *>(row) + sizeof(T) / 2 * vec + i);
  return v;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw<T> &raw, float (&v)[8]) {
  if (sizeof(T) == 2) {
    const uint32_t w[4] = {raw.a[0].x, raw.a[0].y, raw.a[0].z, raw.a[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 q = raw.a[i < (int)sizeof(T) / 2 ? i : 0];
      v[4 * i] = __uint_as_float(q.x);
      v[4 * i + 1] = __uint_as_float(q.y);
      v[4 * i + 2] = __uint_as_float(q.z);
      v[4 * i + 3] = __uint_as_float(q.w);
    }
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

// MAXT: threads of a block at most.  Rows of up to 4096 values (512 threads)
// leave room for three blocks an SM.
template <typename T, int V, bool BLOCK, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 512 ? 3 : 1) rmsnorm_fp8_kernel(const NormParams p) {
  __shared__ float red[2][2][32];  // by row parity: square sums, magnitudes
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int threads = BLOCK ? blockDim.x : 32;  // of a row
  const int tid = BLOCK ? threadIdx.x : lane;
  const int step = BLOCK ? gridDim.x : gridDim.x * kWarpRows;
  const int vecs = p.width >> 3;
  int r = BLOCK ? blockIdx.x : blockIdx.x * kWarpRows + warp;
  const bool res = p.res != nullptr;
  const int span = p.group >> 3;  // lanes of a group
  grid_launch_dependents();
  grid_dependency_wait();
  Raw<T> x[V], q[V];
  const uint8_t *xrow = p.x + r * p.x_stride, *rrow = p.res + r * p.res_stride;
  auto fetch = [&]() {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = tid + i * threads;
      if (vec < vecs) {
        x[i] = load_raw<T>(xrow, vec);
        if (res) q[i] = load_raw<T>(rrow, vec);
      }
    }
    xrow += step * p.x_stride;
    rrow += step * p.res_stride;
  };
  constexpr bool kAhead = V == 1 || !BLOCK;  // wider rows have no registers to spare for the next one
  if (kAhead && r < p.n) fetch();
  float w[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = tid + i * threads;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = 0.f;
    if (vec < vecs) {
      const float4 a = reinterpret_cast<const float4 *>(p.weight)[2 * vec];
      const float4 b = reinterpret_cast<const float4 *>(p.weight)[2 * vec + 1];
      w[i][0] = a.x; w[i][1] = a.y; w[i][2] = a.z; w[i][3] = a.w;
      w[i][4] = b.x; w[i][5] = b.y; w[i][6] = b.z; w[i][7] = b.w;
    }
  }
  int parity = 0;
  for (; r < p.n; r += step, parity ^= 1) {  // the same rows for a whole warp or block: no barrier is left waiting
    float h[V][8];  // x + residual, then that times the weight
    float m[V];
    float ss = 0.f;
    if (!kAhead) fetch();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = tid + i * threads;
      m[i] = 0.f;
      if (vec < vecs) {
        unpack8<T>(x[i], h[i]);
        if (res) {
          float y[8];
          unpack8<T>(q[i], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[i][e] += y[e];
          store8<T>(p.res_out + r * p.res_out_stride, vec, h[i]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(h[i][e], h[i][e], ss);
          h[i][e] *= w[i][e];
          m[i] = fmaxf(m[i], fabsf(h[i][e]));
        }
      }
    }
    if (kAhead && r + step < p.n) fetch();
    ss = warp_sum(ss);
    if (BLOCK && lane == 0) red[parity][0][warp] = ss;
    // The largest |h w| of each group.  The row's factor 1 / rms scales y and
    // m alike, so the codes do not need it: only the scales and y wait for the
    // sum over the row.
    if (span == 0) {
      float t = m[0];
#pragma unroll
      for (int i = 1; i < V; ++i) t = fmaxf(t, m[i]);
      t = warp_max(t);
      if (BLOCK && lane == 0) red[parity][1][warp] = t;
      m[0] = t;
    } else {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
        if (o < span)
#pragma unroll
          for (int i = 0; i < V; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
    }
    if (BLOCK) {
      __syncthreads();
      const bool have = lane < (threads >> 5);
      ss = warp_sum(have ? red[parity][0][lane] : 0.f);
      if (span == 0) m[0] = warp_max(have ? red[parity][1][lane] : 0.f);
    }
    const float rs = rsqrtf(fmaf(ss, p.inv_width, p.eps));
    if (span == 0)
#pragma unroll
      for (int i = 1; i < V; ++i) m[i] = m[0];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = tid + i * threads;
      if (vec >= vecs) continue;
      float f = rs;  // what h and m still lack
      if (m[i] <= kLeastMax) {  // 448 / m would overflow: apply the factor first
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] *= rs;
        m[i] *= rs;
        f = 1.f;
      }
      if (p.codes != nullptr) {
        const bool some = m[i] > kLeastMax && rs > 0.f;  // (rs is 0 when the sum of squares overflowed)
        const float inv = __fdiv_rn(448.f, m[i]);  // exactly rounded: an error here moves codes that lie near a tie
        uint32_t out[2] = {0u, 0u};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint16_t c;
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(h[i][2 * k + 1] * inv), "f"(h[i][2 * k] * inv));
          out[k >> 1] |= static_cast<uint32_t>(c) << (16 * (k & 1));
        }
        reinterpret_cast<uint2 *>(p.codes + r * p.code_stride)[vec] = some ? make_uint2(out[0], out[1]) : make_uint2(0u, 0u);
        if (span == 0 ? vec == 0 : (vec & (span - 1)) == 0)
          p.scales[r * p.scale_stride + (span == 0 ? 0 : vec / span)] = some ? m[i] * f * (1.f / 448.f) : 0.f;
      }
      if (p.y != nullptr) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[i][e] * f;
        reinterpret_cast<uint4 *>(p.y + r * p.y_stride)[vec] = pack_half8(y);
      }
    }
  }
}

constexpr int kShapes = 5;

// By width: a warp per row; one vector per thread, up to 512 and up to 1024
// threads; two and four vectors per thread.
template <typename T>
const void *norm_kernel(int shape) {
  switch (shape) {
    case 0: return (const void *)rmsnorm_fp8_kernel<T, 2, false, 32 * kWarpRows>;
    case 1: return (const void *)rmsnorm_fp8_kernel<T, 1, true, 512>;
    case 2: return (const void *)rmsnorm_fp8_kernel<T, 1, true, 1024>;
    case 3: return (const void *)rmsnorm_fp8_kernel<T, 2, true, 1024>;
    default: return (const void *)rmsnorm_fp8_kernel<T, 4, true, 1024>;
  }
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, bool fp32, int sm_count, cudaStream_t s) {
  const int vecs = p.width / 8;
  const int shape = p.width <= kWarpRowWidth ? 0 : vecs <= 512 ? 1 : vecs <= 1024 ? 2 : vecs <= 2048 ? 3 : 4;
  const bool block = shape > 0;
  const int v = shape == 4 ? 4 : shape == 3 ? 2 : 1;
  const int threads = block ? ((vecs + v - 1) / v + 31) / 32 * 32 : 32 * kWarpRows;
  const void *f = fp32 ? norm_kernel<float>(shape) : norm_kernel<__half>(shape);
  cudaLaunchConfig_t cfg = {};
  // About as many blocks as are resident at once (1536 threads an SM).
  const int rows = block ? p.n : (p.n + kWarpRows - 1) / kWarpRows;
  const int most = sm_count * (threads >= 1536 ? 1 : 1536 / threads);
  cfg.gridDim = dim3(rows < most ? rows : most);
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
  for (int shape = 0; shape < kShapes; ++shape)
    for (const void *f : {norm_kernel<float>(shape), norm_kernel<__half>(shape)}) {
      cudaFuncAttributes a;
      const cudaError_t e = cudaFuncGetAttributes(&a, f);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace ds4a
