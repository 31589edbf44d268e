// Writing and thinning a paged K/V cache: new rows into their slots, and the
// eviction of the rows that received the least attention weight.
#include <cooperative_groups.h>

#include "internal.h"
#include "paged_params.h"
#include "ptx.cuh"

namespace ds4a {

namespace cg = cooperative_groups;

namespace {

// ------------------------------------------------------------------ append
// One warp per new row and pool: 16 values a lane, copied, or quantised as
// quantize_fp8_kernel does (scale = absmax / 448, code = E4M3(x * (448 /
// absmax)), quotients and product rounded to nearest in fp32).  A row is 1 KB
// in and at most 1 KB out: memory latency for a decode step's rows.

constexpr int kAppendWarps = 4;

__global__ void __launch_bounds__(32 * kAppendWarps) append_paged_kernel(const AppendParams p, int pools) {
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  grid_launch_dependents();
  grid_dependency_wait();
  if (i >= (long long)p.n * pools) return;
  const bool is_v = i >= p.n;
  const int r = (int)(is_v ? i - p.n : i);
  const uint4 *src = reinterpret_cast<const uint4 *>((is_v ? p.v : p.k) + r * p.new_stride) + 2 * lane;
  const int slot = __ldg(p.slots + r);
  const uint4 a = __ldg(src), b = __ldg(src + 1);
  if (slot < 0) return;
  const int page = slot / p.rows.page_rows, row = slot - page * p.rows.page_rows;
  if (page >= p.rows.n_pages) return;
  uint8_t *dst = const_cast<uint8_t *>(is_v ? p.rows.v : p.rows.k) + page * p.rows.page_stride +
                 row * p.rows.row_stride;
  if (p.rows.k_scale == nullptr) {
    reinterpret_cast<uint4 *>(dst)[2 * lane] = a;
    reinterpret_cast<uint4 *>(dst)[2 * lane + 1] = b;
    return;
  }
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float x[16];
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  uint32_t out[4] = {0u, 0u, 0u, 0u};
  if (amax > 0.f) {
    const float inv = __fdiv_rn(448.f, amax);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint16_t h;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(h)
          : "f"(__fmul_rn(x[2 * k + 1], inv)), "f"(__fmul_rn(x[2 * k], inv)));
      out[k >> 1] |= static_cast<uint32_t>(h) << (16 * (k & 1));
    }
  }
  reinterpret_cast<uint4 *>(dst)[lane] = make_uint4(out[0], out[1], out[2], out[3]);
  if (lane == 0)
    const_cast<float *>(is_v ? p.rows.v_scale : p.rows.k_scale)[(long long)page * p.rows.page_rows + row] =
        amax > 0.f ? __fdiv_rn(amax, 448.f) : 0.f;
}

// ------------------------------------------------------------------ eviction: choosing the rows
// A cluster of CTAs per sequence; each CTA owns a contiguous range of slots
// and each of its warps a contiguous part of that.  An exact radix select
// over order-preserving 32-bit keys, four digits of 8 bits from the top, finds
// the smallest kept key and how many rows of that key stay (the lowest slots);
// the cluster adds its histograms through distributed shared memory.  Three
// walks of the keys follow: equal keys per warp; with their prefix every row
// knows whether it stays, so kept rows at or above n' and freed slots below it
// are counted; with the prefix of those each row writes its own entry.  The
// h-th of either list pairs up in the move kernel.  All integer work: the
// result does not depend on any order of execution.

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;
constexpr int kMaxCachedKeys = 49152;  // 192 KB of keys beside the histogram

struct SelShared {
  unsigned hist[kBins];
  unsigned warp_sum[kSelWarps];
  unsigned warp_sum2[kSelWarps];
  unsigned total[3];  // this CTA's counts, read by the other CTAs
  unsigned digit, left;
};

// Order-preserving key: larger weight, larger key; NaN as -inf, -0 as +0.
// Protected rows come above every weight.
__device__ __forceinline__ uint32_t evict_key(float x, bool safe) {
  if (safe) return 0xFFFFFFFFu;
  if (x != x) x = -INFINITY;
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix over the block's warps of a per-warp count; total = sum.
__device__ __forceinline__ unsigned warps_before(unsigned mine, unsigned *sums, int warp, int lane, unsigned &total) {
  __syncthreads();
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  const unsigned v = sums[lane];
  unsigned inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  total = __shfl_sync(0xffffffffu, inc, 31);
  return __shfl_sync(0xffffffffu, inc - v, warp);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ SelShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / C;
  grid_dependency_wait();
  const int4 g = __ldg(p.geom + b);
  const int n = min(max(g.w, 0), p.rows.max_rows);
  const int n_out = min(n, p.n_keep);
  const float *w = p.weights + b * p.weight_stride;
  const int32_t *ids = p.ids != nullptr ? p.ids + b * p.id_stride : nullptr;
  int32_t *kept = p.kept + b * p.kept_stride;
  float *w_out = p.weights_out != nullptr ? p.weights_out + b * p.weight_out_stride : nullptr;
  int32_t *ids_out = p.ids_out != nullptr ? p.ids_out + b * p.id_out_stride : nullptr;
  const int per = ((n + C - 1) / C + 31) / 32 * 32;
  const int lo = min(n, rank * per), hi = min(n, lo + per);
  for (int i = n_out + rank * kSelThreads + tid; i < p.n_keep; i += C * kSelThreads) kept[i] = -1;
  if (n == n_out) {  // everything stays
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      kept[j] = j;
      if (w_out != nullptr) w_out[j] = w[j];
      if (ids_out != nullptr) ids_out[j] = ids[j];
    }
    if (rank == 0 && tid == 0) {
      p.n_moves[b] = 0;
      *reinterpret_cast<int32_t *>(p.n_out + b * p.n_out_stride) = n_out;
    }
    return;
  }
  const long long recent = ((long long)max(g.x, 0) + 1) / p.ratio - p.n_recent;
  auto key_at = [&](int j) -> uint32_t {
    const int id = ids != nullptr ? ids[j] : j;
    return evict_key(w[j], id < p.n_first || id >= recent);
  };
  if (p.cached > 0)
    for (int j = lo + tid; j < hi; j += kSelThreads) keys[j - lo] = key_at(j);
  auto key = [&](int j) -> uint32_t { return p.cached > 0 ? keys[j - lo] : key_at(j); };

  // The n'-th largest key, digit by digit.
  uint32_t prefix = 0, mask = 0;
  unsigned left = (unsigned)n_out;  // rows still to take among those that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < kBins) sh.hist[tid] = 0;
    __syncthreads();
    for (int base = lo; base < hi; base += kSelThreads) {
      const int j = base + tid;
      uint32_t k = 0;
      const bool in = j < hi && (((k = key(j)) ^ prefix) & mask) == 0;
      const unsigned who = __ballot_sync(0xffffffffu, in);
      if (who == 0) continue;
      const uint32_t d = (k >> shift) & 0xFFu;
      // Rows of one digit (all-equal weights) are added once per warp.
      int same = 0;
      if (who == 0xffffffffu) __match_all_sync(0xffffffffu, d, &same);
      if (same) {
        if (lane == 0) atomicAdd(&sh.hist[d], 32u);
      } else if (in) {
        atomicAdd(&sh.hist[d], 1u);
      }
    }
    cluster.sync();
    unsigned c = 0, above = 0;
    if (tid < kBins) {  // thread t: the bin t from the top
      const int bin = kBins - 1 - tid;
      for (int r = 0; r < C; ++r) c += cluster.map_shared_rank(sh.hist, r)[bin];
      unsigned inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
      }
      if (lane == 31) sh.warp_sum[warp] = inc;
      above = inc - c;
    }
    __syncthreads();
    if (tid < kBins) {
      for (int i = 0; i < warp; ++i) above += sh.warp_sum[i];
      if (above < left && left <= above + c) {  // exactly one thread
        sh.digit = kBins - 1 - tid;
        sh.left = left - above;
      }
    }
    cluster.sync();  // every CTA has read the histograms; digit and left are set
    prefix |= sh.digit << shift;
    mask |= 0xFFu << shift;
    left = sh.left;
  }
  const uint32_t T = prefix;  // rows above T stay, and the first `left` of T

  const int sub = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(hi, lo + warp * sub), w1 = min(hi, w0 + sub);
  unsigned eq = 0;
  for (int base = w0; base < w1; base += 32) {
    const int j = base + lane;
    eq += __popc(__ballot_sync(0xffffffffu, j < w1 && key(j) == T));
  }
  unsigned total;
  unsigned eq_before = warps_before(eq, sh.warp_sum, warp, lane, total);
  if (tid == 0) sh.total[0] = total;
  cluster.sync();
  for (int r = 0; r < rank; ++r) eq_before += *cluster.map_shared_rank(&sh.total[0], r);

  const unsigned below = (1u << lane) - 1u;
  auto stays = [&](int j, unsigned &seen) -> bool {  // `seen`: equal keys before this step's 32 rows
    const uint32_t k = j < w1 ? key(j) : 0u;
    const bool is_eq = j < w1 && k == T;
    const unsigned bal = __ballot_sync(0xffffffffu, is_eq);
    const bool in = j < w1 && (k > T || (is_eq && seen + __popc(bal & below) < left));
    seen += __popc(bal);
    return in;
  };
  unsigned movers = 0, holes = 0, seen = eq_before;
  for (int base = w0; base < w1; base += 32) {
    const int j = base + lane;
    const bool in = stays(j, seen);
    movers += __popc(__ballot_sync(0xffffffffu, in && j >= n_out));
    holes += __popc(__ballot_sync(0xffffffffu, !in && j < w1 && j < n_out));
  }
  unsigned tm, th;
  unsigned m_at = warps_before(movers, sh.warp_sum, warp, lane, tm);
  unsigned h_at = warps_before(holes, sh.warp_sum2, warp, lane, th);
  if (tid == 0) {
    sh.total[1] = tm;
    sh.total[2] = th;
  }
  cluster.sync();
  unsigned all = 0;
  for (int r = 0; r < C; ++r) {
    const unsigned t1 = *cluster.map_shared_rank(&sh.total[1], r);
    all += t1;
    if (r < rank) {
      m_at += t1;
      h_at += *cluster.map_shared_rank(&sh.total[2], r);
    }
  }
  int32_t *from = p.from + (long long)b * p.n_keep, *to = p.to + (long long)b * p.n_keep;
  seen = eq_before;
  for (int base = w0; base < w1; base += 32) {
    const int j = base + lane;
    const bool in = stays(j, seen);
    const bool mover = in && j >= n_out, hole = !in && j < w1 && j < n_out;
    const unsigned bm = __ballot_sync(0xffffffffu, mover), bh = __ballot_sync(0xffffffffu, hole);
    if (mover) from[m_at + __popc(bm & below)] = j;
    if (hole) to[h_at + __popc(bh & below)] = j;
    if (in && j < n_out) {
      kept[j] = j;
      if (w_out != nullptr) w_out[j] = w[j];
      if (ids_out != nullptr) ids_out[j] = ids[j];
    }
    m_at += __popc(bm);
    h_at += __popc(bh);
  }
  if (rank == 0 && tid == 0) {
    p.n_moves[b] = (int)all;
    *reinterpret_cast<int32_t *>(p.n_out + b * p.n_out_stride) = n_out;
  }
  cluster.sync();  // no CTA leaves while another reads its counts
}

// ------------------------------------------------------------------ eviction: moving the rows
// One warp per move: the K and the V row (and the scales of an E4M3 pool) of
// the h-th kept row above n' into the h-th freed slot below it.  Sources and
// destinations never meet, so the moves need no order.  Bound by memory: two
// rows read and two written per move.

constexpr int kMoveWarps = 8;

__global__ void __launch_bounds__(32 * kMoveWarps) evict_move_kernel(const EvictParams p, int blocks_per_seq) {
  const int b = blockIdx.x / blocks_per_seq, lane = threadIdx.x & 31;
  const int h = (blockIdx.x - b * blocks_per_seq) * kMoveWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (h >= p.n_moves[b]) return;
  const int src = p.from[(long long)b * p.n_keep + h], dst = p.to[(long long)b * p.n_keep + h];
  const PagedSeg &s = p.rows;
  const int32_t *table = s.table + b * s.table_stride;
  const int sp = src / s.page_rows, dp = dst / s.page_rows;
  const int from_page = __ldg(table + sp), to_page = __ldg(table + dp);
  if (lane == 0) p.kept[b * p.kept_stride + dst] = src;
  if (lane == 1 && p.weights_out != nullptr)
    p.weights_out[b * p.weight_out_stride + dst] = p.weights[b * p.weight_stride + src];
  if (lane == 2 && p.ids_out != nullptr) p.ids_out[b * p.id_out_stride + dst] = p.ids[b * p.id_stride + src];
  if ((unsigned)from_page >= (unsigned)s.n_pages || (unsigned)to_page >= (unsigned)s.n_pages) return;
  const int ss = src - sp * s.page_rows, ds = dst - dp * s.page_rows;
  const long long so = from_page * s.page_stride + ss * s.row_stride, d = to_page * s.page_stride + ds * s.row_stride;
  const bool both = s.v != s.k;
  uint8_t *kd = const_cast<uint8_t *>(s.k), *vd = const_cast<uint8_t *>(s.v);
  if (s.k_scale != nullptr) {
    const uint4 a = *(reinterpret_cast<const uint4 *>(s.k + so) + lane);
    uint4 c = a;
    if (both) c = *(reinterpret_cast<const uint4 *>(s.v + so) + lane);
    const long long sr = (long long)from_page * s.page_rows + ss, dr = (long long)to_page * s.page_rows + ds;
    if (lane == 0) const_cast<float *>(s.k_scale)[dr] = s.k_scale[sr];
    if (lane == 1 && s.v_scale != s.k_scale) const_cast<float *>(s.v_scale)[dr] = s.v_scale[sr];
    *(reinterpret_cast<uint4 *>(kd + d) + lane) = a;
    if (both) *(reinterpret_cast<uint4 *>(vd + d) + lane) = c;
    return;
  }
  const uint4 *ks = reinterpret_cast<const uint4 *>(s.k + so), *vs = reinterpret_cast<const uint4 *>(s.v + so);
  const uint4 a0 = ks[lane], a1 = ks[lane + 32];
  uint4 c0 = a0, c1 = a1;
  if (both) {
    c0 = vs[lane];
    c1 = vs[lane + 32];
  }
  reinterpret_cast<uint4 *>(kd + d)[lane] = a0;
  reinterpret_cast<uint4 *>(kd + d)[lane + 32] = a1;
  if (both) {
    reinterpret_cast<uint4 *>(vd + d)[lane] = c0;
    reinterpret_cast<uint4 *>(vd + d)[lane + 32] = c1;
  }
}

}  // namespace

int evict_cluster(int max_rows) { return max_rows <= 8192 ? 1 : 8; }

int evict_cached_keys(int max_rows, int cluster) {
  const long long per = (((long long)max_rows + cluster - 1) / cluster + 31) / 32 * 32;
  return per <= kMaxCachedKeys ? (int)per : 0;
}

cudaError_t launch_evict(const EvictParams &p, cudaStream_t s) {
  const int C = evict_cluster(p.rows.max_rows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_seq * C);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = 4 * (size_t)p.cached;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
  if (e != cudaSuccess) return e;
  const int spare = p.rows.max_rows - p.n_keep;  // kept rows above n' are at most this many
  const int moves = spare < p.n_keep ? spare : p.n_keep;
  if (moves <= 0) return cudaSuccess;
  const int blocks = (moves + kMoveWarps - 1) / kMoveWarps;
  cfg.gridDim = dim3(p.n_seq * blocks);
  cfg.blockDim = dim3(32 * kMoveWarps);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, p, blocks);
}

cudaError_t launch_append(const AppendParams &p, cudaStream_t s) {
  const int pools = p.rows.v != p.rows.k ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)p.n * pools + kAppendWarps - 1) / kAppendWarps));
  cfg.blockDim = dim3(32 * kAppendWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_paged_kernel, p, pools);
}

// The shared-memory opt-in of the selection, and the code of every kernel here.
cudaError_t prepare_cache_kernels() {
  cudaError_t e = cudaFuncSetAttribute((const void *)evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       4 * kMaxCachedKeys);
  for (const void *f : {(const void *)append_paged_kernel, (const void *)evict_select_kernel,
                        (const void *)evict_move_kernel}) {
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, f);
  }
  return e;
}

}  // namespace ds4a
