// Writing and thinning a paged K/V cache: new rows into their slots, and the
// eviction of the rows that received the least attention weight.
#include <cooperative_groups.h>

#include <type_traits>

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
// in and at most 1 KB out: 64 rows of E4M3 pools take 1.5 us on the device, the
// latency of a slot and a row, and 2.6 us of host time; 2,048 fp16 rows 3.0 us.

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
  const int slot = p.slots[r];
  const uint4 a = src[0], b = src[1];
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
  // Rows that serve as K and V may have a scale array for each: both get this row's.
  const float *scales = is_v || (lane == 1 && pools == 1) ? p.rows.v_scale : p.rows.k_scale;
  if (lane <= (pools == 1 && p.rows.v_scale != p.rows.k_scale))
    const_cast<float *>(scales)[(long long)page * p.rows.page_rows + row] = amax > 0.f ? __fdiv_rn(amax, 448.f) : 0.f;
}

// ------------------------------------------------------------------ eviction: choosing the rows
// A cluster of CTAs per sequence (one CTA for up to 8192 rows, eight for up to
// 65536, else sixteen);
// each CTA owns a contiguous range of slots and each of its warps a contiguous
// part of that.  An exact radix select over order-preserving 32-bit keys, in
// digits of 11, 11 and 10 bits (the first spans sign, exponent and two mantissa
// bits, so that rows of like weight still spread over bins and the shared
// atomics rarely collide), finds the smallest kept key T and how many rows of
// that key stay (the lowest slots).  CTAs of a cluster add their histograms
// through distributed shared memory.  One walk
// then counts, per warp and apart below and above n', the rows over T and at
// T; their prefixes give every warp its first entry of the two lists (kept rows
// at or above n', freed slots below), and a last walk writes them, and a bit
// per slot below n' that tells whether its row stays there.  The h-th of either
// list pairs up in the move kernel.  All integer work: the result does not
// depend on any order of execution.

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCachedKeys = 45056;  // 176 KB of keys beside the histograms
constexpr int kBatch = 8;              // rows of a thread (or a warp's steps) loaded ahead

struct Counts {  // rows over T and at T, in slots below n' and from n' on
  unsigned gt_lo, eq_lo, gt_hi, eq_hi;
};

struct SelShared {
  unsigned hist[kBins];    // of this CTA's keys
  unsigned warp_sum[kSelWarps];
  Counts warp[kSelWarps];
  unsigned digit, left;
};
struct ClusterShared : SelShared {
  unsigned sum[3][kBins];  // of the cluster's keys, by digit
  unsigned share[kBins / 8];
  Counts cta[16];          // every CTA's counts
};

// Order-preserving key: larger weight, larger key; NaN as -inf, -0 as +0.
// Protected rows come above every weight.
__device__ __forceinline__ uint32_t evict_key(float x, bool safe) {
  if (safe) return 0xFFFFFFFFu;
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0xFF800000u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ unsigned warp_add(unsigned v) { return __reduce_add_sync(0xffffffffu, v); }

__device__ __forceinline__ unsigned scan_lanes(unsigned v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// Of rows over / at T, how many of those at T are taken when `seen` rows at T
// come before and `left` are taken in all.
__device__ __forceinline__ unsigned taken(unsigned eq, unsigned seen, unsigned left) {
  return seen >= left ? 0u : min(eq, left - seen);
}

template <bool CLUSTER, typename Shared>
__device__ __forceinline__ void select_rows(const EvictParams &p, uint32_t *keys, Shared &sh) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / C;
  for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
  if constexpr (CLUSTER) {
    static_assert(kBins == 2 * kSelThreads, "two bins per thread");
    for (int i = tid; i < 3 * kBins; i += kSelThreads) sh.sum[0][i] = 0;
    if (tid < kBins / 8) sh.share[tid] = 0;
    cluster.sync();  // clear before any CTA adds to them
  }
  grid_launch_dependents();
  grid_dependency_wait();
  const int4 g = p.geom[b];
  const int n = min(max(g.w, 0), p.rows.max_rows);
  const int n_out = min(n, p.n_keep);
  const float *w = p.weights + b * p.weight_stride;
  const int32_t *ids = p.ids != nullptr ? p.ids + b * p.id_stride : nullptr;
  uint32_t *stay = p.stay + (long long)b * p.stay_words;
  const int per = ((n + C - 1) / C + 31) / 32 * 32;
  const int lo = min(n, rank * per), hi = min(n, lo + per);
  if (n == n_out) {  // everything stays
    for (int i = lo / 32 + tid; 32 * i < hi; i += kSelThreads) stay[i] = 0xFFFFFFFFu;
    if (rank == 0 && tid == 0) {
      p.n_moves[b] = make_int2(0, n_out);
      *reinterpret_cast<int32_t *>(p.n_out + b * p.n_out_stride) = n_out;
    }
    return;
  }
  // Ids over `old` are protected; it lies in -2^31 .. 2^31 - 1.
  const int old = (int)(((long long)max(g.x, 0) + 1) / p.ratio - p.n_recent - 1);
  auto key_at = [&](int j) -> uint32_t {
    const int id = ids != nullptr ? ids[j] : j;
    return evict_key(w[j], id < p.n_first || id > old);
  };
  auto key = [&](int j) -> uint32_t { return p.cached > 0 ? keys[j - lo] : key_at(j); };
  if (p.cached > 0) {  // kBatch loads of a thread in flight at a time
    for (int base = lo + tid; base < hi; base += kBatch * kSelThreads) {
      float x[kBatch];
      int id[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = base + i * kSelThreads;
        x[i] = j < hi ? w[j] : 0.f;
        id[i] = j < hi && ids != nullptr ? ids[j] : j;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = base + i * kSelThreads;
        if (j < hi) keys[j - lo] = evict_key(x[i], id[i] < p.n_first || id[i] > old);
      }
    }
  }

  // The n'-th largest key, digit by digit.
  uint32_t prefix = 0, mask = 0;
  unsigned left = (unsigned)n_out;  // rows still to take among those that match the prefix
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    const uint32_t digits = (1u << bits) - 1u;
    __syncthreads();  // the histogram is clear
    for (int base = lo; base < hi; base += kSelThreads) {
      const int j = base + tid;
      uint32_t k = 0;
      bool in = j < hi;
      if (in) {
        k = key(j);
        in = ((k ^ prefix) & mask) == 0;
      }
      if (!__any_sync(0xffffffffu, in)) continue;
      const uint32_t d = (k >> shift) & digits, d0 = __shfl_sync(0xffffffffu, d, 0);
      // Rows of one digit (all-equal weights) are added once per warp.
      if (__all_sync(0xffffffffu, in && d == d0)) {
        if (lane == 0) atomicAdd(&sh.hist[d], 32u);
      } else if (in) {
        atomicAdd(&sh.hist[d], 1u);
      }
    }
    __syncthreads();
    if constexpr (CLUSTER) {
      if (pass != 1) {
        // Few bins hold keys of this CTA (like exponents in the first digit,
        // the last survivors in the third): each is added to the sums of
        // every CTA at once.
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int bin = tid + u * kSelThreads;
          const unsigned v = sh.hist[bin];
          if (v != 0)
            for (int r = 0; r < C; ++r) atomicAdd(cluster.map_shared_rank(&sh.sum[pass][bin], (rank + r) % C), v);
        }
      } else {
        // Mantissa bits spread over the bins: each CTA adds up its share of
        // them and hands the sums to every CTA (16 CTAs, 131,072 rows: 5,800
        // cycles against 10,800 as above).
        cluster.sync();
        const int share = kBins / C;
        unsigned v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = tid + u * kSelThreads;
          v[u] = cluster.map_shared_rank(sh.hist, i / share)[rank * share + i % share];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (v[u] != 0) atomicAdd(&sh.share[(tid + u * kSelThreads) % share], v[u]);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = tid + u * kSelThreads;
          cluster.map_shared_rank(sh.sum[pass], i / share)[rank * share + i % share] = sh.share[i % share];
        }
      }
      cluster.sync();
    }
    // Thread t: the two bins 2t, 2t + 1 counted from the top.
    const unsigned *total = sh.hist;
    if constexpr (CLUSTER) total = sh.sum[pass];
    const int top = kBins - 1 - 2 * tid;
    const unsigned c0 = total[top], c1 = total[top - 1];
    const unsigned inc = scan_lanes(c0 + c1, lane);
    if (lane == 31) sh.warp_sum[warp] = inc;
    __syncthreads();
    const unsigned before = warp_add(lane < warp ? sh.warp_sum[lane] : 0u);
    const unsigned above0 = before + inc - c0 - c1, above1 = above0 + c0;
    if (above0 < left && left <= above1) {  // one thread of one of the two lines
      sh.digit = top;
      sh.left = left - above0;
    } else if (above1 < left && left <= above1 + c1) {
      sh.digit = top - 1;
      sh.left = left - above1;
    }
    sh.hist[2 * tid] = sh.hist[2 * tid + 1] = 0;
    __syncthreads();
    prefix |= sh.digit << shift;
    mask |= digits << shift;
    left = sh.left;
  }
  const uint32_t T = prefix;  // rows above T stay, and the first `left` of T

  const int sub = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(hi, lo + warp * sub), w1 = min(hi, w0 + sub);
  Counts c = {0u, 0u, 0u, 0u};
  for (int j = w0 + lane; j < w1; j += 32) {
    const uint32_t k = key(j);
    const unsigned gt = k > T, eq = k == T, low = j < n_out;
    c.gt_lo += gt & low;
    c.eq_lo += eq & low;
    c.gt_hi += gt & ~low & 1u;
    c.eq_hi += eq & ~low & 1u;
  }
  c.gt_lo = warp_add(c.gt_lo);
  c.eq_lo = warp_add(c.eq_lo);
  c.gt_hi = warp_add(c.gt_hi);
  c.eq_hi = warp_add(c.eq_hi);
  if (lane == 0) sh.warp[warp] = c;
  __syncthreads();
  // Lane l: warp l's counts, its rows at T before it in this CTA.
  const Counts wc = sh.warp[lane];
  const unsigned wc_eq = wc.eq_lo + wc.eq_hi;
  const unsigned eq_inc = scan_lanes(wc_eq, lane);
  if constexpr (CLUSTER) {
    if (warp == 0) {
      const Counts t = {warp_add(wc.gt_lo), warp_add(wc.eq_lo), warp_add(wc.gt_hi), warp_add(wc.eq_hi)};
      if (lane < C) *cluster.map_shared_rank(&sh.cta[rank], lane) = t;
    }
    cluster.sync();
  }
  // Entries of the lists, and rows at T, of the CTAs before this one.
  unsigned eq_before = 0, m_before = 0, h_before = 0, m_all = 0;
  auto lists_of = [&](const Counts &x, int slots_lo, unsigned seen, unsigned &movers, unsigned &holes) {
    holes = slots_lo - x.gt_lo - taken(x.eq_lo, seen, left);
    movers = x.gt_hi + taken(x.eq_hi, seen + x.eq_lo, left);
  };
  if constexpr (CLUSTER) {  // lane r: CTA r
    const Counts none = {0u, 0u, 0u, 0u};
    const Counts x = lane < C ? sh.cta[lane] : none;
    const int r0 = min(n, lane * per), r1 = lane < C ? min(n, r0 + per) : r0;
    const unsigned eq_all = x.eq_lo + x.eq_hi, eq_upto = scan_lanes(eq_all, lane);
    unsigned m, h;
    lists_of(x, min(max(n_out - r0, 0), r1 - r0), eq_upto - eq_all, m, h);
    const bool before = lane < rank;
    eq_before = warp_add(before ? eq_all : 0u);
    m_before = warp_add(before ? m : 0u);
    h_before = warp_add(before ? h : 0u);
    m_all = warp_add(m);
  }
  // The same for the warps of this CTA (lane l: warp l).
  unsigned m_mine, h_mine;
  {
    const int r0 = min(hi, lo + lane * sub), r1 = min(hi, r0 + sub);
    lists_of(wc, min(max(n_out - r0, 0), r1 - r0), eq_before + eq_inc - wc_eq, m_mine, h_mine);
  }
  const unsigned m_inc = scan_lanes(m_mine, lane), h_inc = scan_lanes(h_mine, lane);
  if (!CLUSTER) m_all = __shfl_sync(0xffffffffu, m_inc, 31);
  unsigned m_at = m_before + __shfl_sync(0xffffffffu, m_inc - m_mine, warp);
  unsigned h_at = h_before + __shfl_sync(0xffffffffu, h_inc - h_mine, warp);
  unsigned seen = eq_before + __shfl_sync(0xffffffffu, eq_inc - wc_eq, warp);
  const unsigned below = (1u << lane) - 1u;
  int32_t *from = p.from + (long long)b * p.n_keep, *to = p.to + (long long)b * p.n_keep;
  for (int base = w0; base < w1; base += 32) {
    const int j = base + lane;
    const uint32_t k = j < w1 ? key(j) : 0u;
    const bool eq = j < w1 && k == T;
    const unsigned be = __ballot_sync(0xffffffffu, eq);
    const bool in = j < w1 && (k > T || (eq && seen + __popc(be & below) < left));
    const bool low = j < n_out;
    const unsigned bm = __ballot_sync(0xffffffffu, in && !low);
    const unsigned bh = __ballot_sync(0xffffffffu, !in && j < w1 && low);
    if (lane == 0 && base < n_out) stay[base >> 5] = ~bh;
    if ((bm >> lane) & 1u) from[m_at + __popc(bm & below)] = j;
    if ((bh >> lane) & 1u) to[h_at + __popc(bh & below)] = j;
    seen += __popc(be);
    m_at += __popc(bm);
    h_at += __popc(bh);
  }
  if (rank == 0 && tid == 0) {
    p.n_moves[b] = make_int2((int)m_all, n_out);
    *reinterpret_cast<int32_t *>(p.n_out + b * p.n_out_stride) = n_out;
  }
}

// ------------------------------------------------------------------ eviction: moving the rows
// One warp per move: the K and the V row (and the scales of an E4M3 pool) of
// the h-th kept row above n' into the h-th freed slot below it.  Sources and
// destinations never meet, so the moves need no order.  One thread per slot
// below n_keep: kept, weights and ids of the row that stays in it.

__device__ __forceinline__ void keep_slot(const EvictParams &p, int b, int j, int n_out) {
  int32_t *kept = p.kept + b * p.kept_stride;
  if (j >= n_out) {
    kept[j] = -1;
  } else if ((p.stay[(long long)b * p.stay_words + (j >> 5)] >> (j & 31)) & 1u) {
    kept[j] = j;
    if (p.weights_out != nullptr) p.weights_out[b * p.weight_out_stride + j] = p.weights[b * p.weight_stride + j];
    if (p.ids_out != nullptr) p.ids_out[b * p.id_out_stride + j] = p.ids[b * p.id_stride + j];
  }
}

__device__ __forceinline__ void move_row(const EvictParams &p, int b, int h, int lane) {
  const int src = p.from[(long long)b * p.n_keep + h], dst = p.to[(long long)b * p.n_keep + h];
  const PagedSeg &s = p.rows;
  const int32_t *table = s.table + b * s.table_stride;
  const int sp = src / s.page_rows, dp = dst / s.page_rows;
  const int from_page = table[sp], to_page = table[dp];
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

// With few rows to move (p.move_here) the CTA that chose them moves them too.
template <bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ typename std::conditional<CLUSTER, ClusterShared, SelShared>::type sh;
  select_rows<CLUSTER>(p, keys, sh);
  if (CLUSTER || !p.move_here) return;
  const int b = blockIdx.x;
  __syncthreads();  // its lists are written
  const int2 plan = p.n_moves[b];
  for (int h = threadIdx.x >> 5; h < plan.x; h += kSelWarps) move_row(p, b, h, threadIdx.x & 31);
  for (int j = threadIdx.x; j < p.n_keep; j += kSelThreads) keep_slot(p, b, j, plan.y);
}

// Bound by memory: two rows read and two written per move.  The blocks of a
// sequence share out its slots, too.
constexpr int kMoveWarps = 8;
constexpr int kMoveSlots = 32 * kMoveWarps;  // slots of a block, one per thread

__global__ void __launch_bounds__(32 * kMoveWarps) evict_move_kernel(const EvictParams p, int blocks_per_seq) {
  const int b = blockIdx.x / blocks_per_seq, part = blockIdx.x - b * blocks_per_seq;
  const int h = part * kMoveWarps + (threadIdx.x >> 5), j = part * kMoveSlots + threadIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  const int2 plan = p.n_moves[b];  // (moves, n')
  if (j < p.n_keep) keep_slot(p, b, j, plan.y);
  if (h < plan.x) move_row(p, b, h, threadIdx.x & 31);
}

}  // namespace

int evict_cluster(int max_rows) { return max_rows <= 8192 ? 1 : max_rows <= 65536 ? 8 : 16; }

int evict_cached_keys(int max_rows, int cluster) {
  const long long per = (((long long)max_rows + cluster - 1) / cluster + 31) / 32 * 32;
  return per <= kMaxCachedKeys ? (int)per : 0;
}

// With up to so many rows that a table can name beyond n_keep (as many can have
// to move; a page of 64, say) the CTA of a sequence moves the rows itself.  64
// sequences that lose 1, 16 or 64 rows of 1,088: 7.5, 8.2 and 11.4 us, with a
// second kernel 9.5, 10.5 and 11.9; one sequence that loses 64: 11.2 us, and 9.4;
// 64 sequences with 128 rows beyond: 15.6, and 13.3.
constexpr int kMovesHere = 64, kSlotsHere = 8192;

cudaError_t launch_evict(EvictParams p, cudaStream_t s) {
  const int C = evict_cluster(p.rows.max_rows);
  const int spare = p.rows.max_rows - p.n_keep;  // kept rows above n' are at most this many
  const int moves = spare < 0 ? 0 : spare < p.n_keep ? spare : p.n_keep;
  p.move_here = C == 1 && moves <= kMovesHere && p.n_keep <= kSlotsHere;
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
  cfg.numAttrs = C > 1 ? 2 : 1;
  const cudaError_t e = C > 1 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<true>, p)
                              : cudaLaunchKernelEx(&cfg, evict_select_kernel<false>, p);
  if (e != cudaSuccess || p.move_here) return e;
  const int move_blocks = (moves + kMoveWarps - 1) / kMoveWarps, slot_blocks = (p.n_keep + kMoveSlots - 1) / kMoveSlots;
  const int blocks = move_blocks > slot_blocks ? move_blocks : slot_blocks;
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
  cudaError_t e = cudaSuccess;
  for (const void *f : {(const void *)evict_select_kernel<false>, (const void *)evict_select_kernel<true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMaxCachedKeys);
  if (e == cudaSuccess)  // clusters of sixteen
    e = cudaFuncSetAttribute((const void *)evict_select_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (const void *f : {(const void *)append_paged_kernel, (const void *)evict_select_kernel<false>,
                        (const void *)evict_select_kernel<true>, (const void *)evict_move_kernel}) {
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, f);
  }
  return e;
}

}  // namespace ds4a
