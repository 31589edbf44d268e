// Attention of one new token per sequence over a paged K/V cache, and the
// weight that each cached row received in it (tcgen05 + TMEM).
//
//   decode   o[b][h] = sum_j softmax_j(scale q[b][h].k_j) v_j over the raw
//            window rows and the compressed rows that sequence b's token sees
//   weights  w[b][c] = sum_h exp(scale q[b][h].k_c - lse[b][h])
//
// (64 query heads over one K/V row of 512, "DwarfStar 4 (DS4) - DeepSeek V4
// Flash Inference Engine", sections "Fixed Model Shape", "Layer Compression"
// and "KV Cache Design"; the visibility rule is that of attn_kernel.cuh.)
//
// Work.  A sequence's visible rows, compressed then raw, form one list, cut
// into tiles of 128 rows; row j of the list is found through the page table,
// so pages of any size, tiles that span pages and pages that end inside a tile
// are all alike.  A CTA's tiles of one sequence are an item.  With c the least
// number for which the items ceil(tiles / c) of all sequences number at most
// the CTAs, each CTA gets one item of at most c tiles.  Where c would be over
// a + min(2, a - 1), with a the average ceil(total / CTAs), or there is none
// (more sequences than CTAs), the tiles of all sequences are numbered through
// instead and CTA i takes a of them in a row, several items.  So no CTA has more
// than the average and two tiles, whatever the lengths; one item per CTA costs one
// drain of the pipeline and fewer partial results.  Averages of 3 to 12 tiles,
// fp16: items one tile above the average 28.5 and 32.0 us, numbered 28.6 and
// 34.3; two above 34.3 to 51.9, numbered 36.8 to 51.3; four above 37.7 to 74.9,
// numbered 32.0 to 67.4; an average of 2, items of 4: 29.1, numbered 26.0; 149
// sequences of one tile and one of 48, items of 16: 69.4, numbered 25.7.
// An item that holds the whole sequence
// writes its output; otherwise it leaves its normalised output (fp32) and
// (m, l) in a slot of the workspace, slot CTA, or CTA + sequence with several
// items per CTA (unique, since along the tiles either number grows), and the
// merge kernel joins the slots of a sequence.
//
// Per tile, as in attn_kernel.cuh, the rows are on the M side of every MMA:
//   S^T[128 rows][64 heads]  = K_tile[128][512] . Q^T
//   O^T[512 dims][64 heads] += V_tile^T . P^T
// with S^T and O^T in TMEM.
//
// Loads.  A stage of the ring holds 128 dims of a tile.  A tile of 128
// compressed rows whose pages all exist is loaded by TMA, one copy per run of
// rows that one page holds (the largest power of two that divides the page's
// rows, 8 at least and 128 at most), issued by the loader warps in turn: a
// thread's bulk copies start some 700 cycles apart.  Every other tile (a sequence's last rows, the window rows, absent
// pages, pages of odd sizes) is gathered with 16-byte cp.async by all loader
// threads, an absent row zero-filled (a copy with no source bytes): nothing a
// page holds beyond the rows in use can reach a product, not even as 0 * NaN.
//
// Warps (512 threads, one CTA per SM): 0-7 softmax and epilogue, 8-14 loaders,
// 15 TMEM allocation and MMA issue.  Ring order: K(0), then K(j+1) and V(j) for
// each tile j, so the next scores are computed while the softmax works.  Where K
// and V are the same rows, a tile is loaded once: its four parts stay in the four
// stages from QK^T to PV, and the next tile, whose rows are in L2 by then, follows
// as each PV frees its stage (24 sequences of 17 to 65 E4M3 tiles: 46 us, 52 us
// with the rows loaded twice).  Half tiles, two of them in the ring, took 49 us: a
// product of 64 rows costs the tensor core as much as one of 128.  With E4M3 rows, warps 8, 13 and 14 load codes into
// the upper half of a stage and warps 9-12 widen them in place, exactly.
//
// A stage's fp16 layout is rows in groups of 8: [16 groups][2 blocks of 64
// dims][8 rows][128 bytes], 128-byte swizzle: a TMA box of any number of
// 8-row groups lands contiguously, and the distance between row groups
// is one constant for the MMA descriptors.  With E4M3 rows it is [2 blocks][128
// rows][128 bytes], where a row's codes sit in bytes that only its own values
// replace.
//
// E4M3 scales.  K's multiplies the scores.  V's scale c_j is folded into the
// exponent: p'_j = 2^(s_j + log2 c_j - m') with m' the running maximum of that
// sum, so the fp16 p' that feeds the MMA has full precision whatever the size
// of the scales; the sum of weights adds p'_j / c_j.
//
// What bounds it.  One sequence of 262,144 fp16 rows: HBM (537 MB in 95 us with the
// merge, 83% of the measured copy rate).  Batches with K = V: the chain of a tile,
// some 7,600 cycles from one tile's first load to the next's: 1,100 until the first
// part is there and 2,200 for 128 KB at the 64 bytes a clock of an SM's port to
// L2, the last part's QK^T 630, softmax 1,800, PV 430 to the first freed stage; 64
// sequences take 40 us, 24 of E4M3 rows 43 us, where widening (read once, written
// twice as wide) and the products' operands share the bandwidth of shared memory.
// Weights of 16 sequences of E4M3 rows, 88 MB: 26 us, bound by the same.
#include "attn_params.h"
#include "internal.h"
#include "paged_params.h"
#include "ptx.cuh"

namespace ds4a {

namespace {

constexpr int kLists = 4;  // row lists in flight
constexpr int kTries = 3;  // sizes tried for one item per CTA: the average number of tiles, one and two more
constexpr float kLeastLog2Scale = -40.f;  // V scales below 2^-40 count as 0: such rows round to 0 in fp16

// Low bits of a list entry (rows are 16-byte aligned).  A slot without a row
// holds the address of a row that exists, copied with no source bytes.
constexpr unsigned long long kSegBit = 1, kNoRow = 2;
// A tile within its item (the CTA's tiles of one sequence).
constexpr int kFirst = 1, kLast = 2, kWhole = 4;  // kWhole: the item holds all tiles of the sequence

// Wait sites of this kernel.
enum : unsigned int {
  PSITE_Q_EMPTY = 0x60, PSITE_KV_EMPTY, PSITE_Q_FULL, PSITE_S_EMPTY, PSITE_KV_FULL, PSITE_P_FULL, PSITE_O_EMPTY,
  PSITE_S_FULL, PSITE_P_EMPTY, PSITE_O_FULL, PSITE_DRAIN, PSITE_CODE_FULL, PSITE_LIST_FULL, PSITE_LIST_EMPTY
};

// The rows sequence b's token sees: compressed rows [0, nc), then raw rows
// [raw_lo, raw_lo + nr).  The weights need the compressed ones only.
struct SeqRows {
  int raw_lo, nr, nc;
  __device__ __forceinline__ int tiles() const { return (nr + nc + kTile - 1) / kTile; }
};

// A CTA's tiles: n of them, from tile `tile` of sequence `seq` on.  The slot of
// an item is CTA + slot_step * sequence.
struct CtaPlan {
  int n, seq, tile, slot_step;
  SeqRows rows;  // of sequence `seq`
};

struct PMisc {
  alignas(16) unsigned long long row[kLists][kTile];  // K address | kSegBit | kNoRow
  alignas(16) float ksc[kLists][kTile];   // E4M3: scale * log2(e) * K scale
  alignas(16) float lvs[kLists][kTile];   // E4M3: log2 of the V scale (of 2^-40 at least)
  alignas(16) float ivs[kLists][kTile];   // E4M3: 2^-lvs
  int2 box[kLists][kTile / 8];            // (page, slot) of the runs of a tile that TMA loads
  alignas(16) float red[4][kH];
  alignas(16) float m_use[kH];  // reference of each head (weights: its lse), log2 units
  alignas(16) float m_lim[kH];  // largest score under that reference
  alignas(16) float alpha[kH];
  alignas(16) float inv_l[kH];
  alignas(8) uint64_t q_full, q_empty;
  uint64_t kv_full[kStages], kv_empty[kStages], code_full[kStages];
  uint64_t list_full[kLists], list_empty[kLists];
  int gathered[kLists];  // of the lists' tiles: rows come by cp.async
  int seq[kLists], flags[kLists], base[kLists], end[kLists];  // of the lists' tiles: sequence, kFirst | ..,
                                                              // first row of the tile, rows of the sequence
  uint64_t s_full[2], s_empty[2];
  uint64_t o_full[4];
  uint64_t p_full, p_empty, o_empty, mma_done;
  unsigned scan[kThreads / 32];
  CtaPlan plan;
  int fits[kTries];
  uint32_t tmem_base;
  int abort_flag;
};
constexpr uint32_t kPagedSmem = kOffMisc + ((sizeof(PMisc) + 127) / 128) * 128 + 1024;
static_assert(kPagedSmem <= 232448, "shared memory of one CTA");

// Bytes between 8-row groups and between the two 64-dim blocks of a stage.
template <bool FP8>
__host__ __device__ constexpr uint32_t group_stride() { return FP8 ? 1024u : 2048u; }
template <bool FP8>
__host__ __device__ constexpr uint32_t block_stride() { return FP8 ? kBoxBytes : 1024u; }

template <bool FP8>
__host__ __device__ constexpr int loader_threads() { return FP8 ? kLoaderThreads - kTile : kLoaderThreads; }

// ------------------------------------------------------------------ small tools

struct StageRing {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void advance() {
    if (++st == kStages) {
      st = 0;
      ph ^= 1;
    }
  }
};

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void bar_sync_id(uint32_t id, uint32_t count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
// 16 bytes global -> shared; `bytes` of 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Starts bringing `bytes` (a multiple of 16) at a 16-byte aligned address into L2.
__device__ __forceinline__ void l2_prefetch(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrives (as one of the expected arrivals) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void load_row32(const float *src, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 x = reinterpret_cast<const float4 *>(src)[i];
    v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
  }
}

// Lane l ends with the max (or sum) over the warp's 32 rows of head l of s[0..31]:
// at each of five steps a lane keeps one half of its values and gets the
// other lane's part of them.
template <bool kMax>
__device__ __forceinline__ float reduce_heads(const float (&s)[32], int lane) {
  float a[16];
  {
    const bool up = lane & 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float send = up ? s[i] : s[i + 16], keep = up ? s[i + 16] : s[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, 16);
      a[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
#pragma unroll
  for (int half = 8; half >= 1; half >>= 1) {
    const bool up = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? a[i] : a[i + half], keep = up ? a[i + half] : a[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, half);
      a[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  return a[0];
}

// ------------------------------------------------------------------ plan

template <bool WEIGHTS>
__device__ __forceinline__ SeqRows seq_rows(const PagedAttnParams &p, int b) {
  const int4 g = p.geom[b];
  const int pos = max(g.x, 0), raw_pos0 = max(g.z, 0);
  const int n_raw = min(max(g.y, 0), p.seg[0].max_rows), n_comp = min(max(g.w, 0), p.seg[1].max_rows);
  SeqRows s;
  s.raw_lo = s.nr = 0;
  if (!WEIGHTS) {
    const long long lo = max((long long)pos - p.window + 1 - raw_pos0, 0ll);
    const long long hi = min((long long)pos + 1 - raw_pos0, (long long)n_raw);
    s.raw_lo = (int)min(lo, (long long)n_raw);
    s.nr = hi > lo ? (int)(hi - lo) : 0;
  }
  s.nc = (int)min((unsigned)n_comp, ((unsigned)pos + 1u) / (unsigned)p.ratio);
  return s;
}

// A CTA's tiles in order.
template <bool WEIGHTS>
struct Walk {
  int b, j, n;   // sequence, tile within it, its tiles
  SeqRows rows;
  bool first, last;  // of this CTA's tiles of the sequence (an item)
  int left;      // tiles of the CTA from this one on
  __device__ __forceinline__ void start(const CtaPlan &cp) {
    b = cp.seq;
    j = cp.tile;
    left = cp.n;
    if (left <= 0) return;
    rows = cp.rows;
    n = rows.tiles();
    first = true;
    last = j == n - 1 || left == 1;
  }
  __device__ __forceinline__ void next(const PagedAttnParams &p) {
    if (--left <= 0) return;
    first = false;
    if (++j == n) {
      do {
        rows = seq_rows<WEIGHTS>(p, ++b);
        n = rows.tiles();
      } while (n == 0 && b + 1 < p.n_seq);
      j = 0;
      first = true;
    }
    last = j == n - 1 || left == 1;
  }
  __device__ __forceinline__ int flags() {
    if (first) first_j = j;
    return (first ? kFirst : 0) | (last ? kLast : 0) | (last && first_j == 0 && j == n - 1 ? kWhole : 0);
  }
  int first_j;   // tile the item began with
};

__device__ __forceinline__ int scan_warp(int n, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) n += t;
  }
  return n;
}


// The plan of this CTA, by one warp alone: lane l has kMost sequences in a
// row.  Every warp computes it for itself (no block barrier stands between the
// geometry and the first load); `writes`: this one writes each sequence's slots
// for the merge.
template <bool WEIGHTS, int kMost>
__device__ __forceinline__ CtaPlan plan_warp(const PagedAttnParams &p, int lane, bool writes) {
  const int G = gridDim.x, cta = blockIdx.x;
  const SeqRows none = {0, 0, 0};
  SeqRows rows[kMost];
  int n[kMost], sum = 0;
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    const int b = lane * kMost + u;
    rows[u] = b < p.n_seq ? seq_rows<WEIGHTS>(p, b) : none;
    n[u] = rows[u].tiles();
    sum += n[u];
  }
  const int total = __reduce_add_sync(0xffffffffu, sum), per = (total + G - 1) / G;
  int c = per, items = G + 1;
  for (int t = 0; t < kTries && t < per; ++t, ++c) {
    int k = 0;
#pragma unroll
    for (int u = 0; u < kMost; ++u) k += (unsigned)(n[u] + c - 1) / (unsigned)c;
    items = __reduce_add_sync(0xffffffffu, k);
    if (items <= G) break;
  }
  const bool one = items <= G;  // one item per CTA
  int count[kMost], mine = 0;   // of the unit that is dealt out: items, or tiles
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    count[u] = one ? (int)((unsigned)(n[u] + c - 1) / (unsigned)c) : n[u];
    mine += count[u];
  }
  int at = scan_warp(mine, lane) - mine;  // items or tiles before this lane's sequences
  const int g0 = one ? cta : min(total, cta * per), g1 = one ? cta + 1 : min(total, g0 + per);
  CtaPlan cp = {0, 0, 0, one ? 0 : 1, none};
  bool found = false;
#pragma unroll
  for (int u = 0; u < kMost; ++u) {
    const int b = lane * kMost + u;
    if (count[u] > 0 && at <= g0 && g0 < at + count[u] && g1 > g0) {
      found = true;
      cp.seq = b;
      cp.rows = rows[u];
      if (one) {
        const unsigned i = g0 - at, k = count[u];
        cp.tile = (int)(i * (unsigned)n[u] / k);
        cp.n = (int)((i + 1) * (unsigned)n[u] / k) - cp.tile;
      } else {
        cp.tile = g0 - at;
        cp.n = g1 - g0;
      }
    }
    if (writes && b < p.n_seq) {
      int2 slots = make_int2(at, count[u]);
      if (!one) {
        const int c0 = n[u] > 0 ? at / per : 0, c1 = n[u] > 0 ? (at + n[u] - 1) / per : -1;
        slots = make_int2(c0 + b, c1 - c0 + 1);
      }
      p.ws_plan[b] = slots;
    }
    at += count[u];
  }
  const unsigned who = __ballot_sync(0xffffffffu, found);
  const int src = who != 0 ? __ffs(who) - 1 : 0;
  cp.n = __shfl_sync(0xffffffffu, cp.n, src);
  cp.seq = __shfl_sync(0xffffffffu, cp.seq, src);
  cp.tile = __shfl_sync(0xffffffffu, cp.tile, src);
  cp.rows.raw_lo = __shfl_sync(0xffffffffu, cp.rows.raw_lo, src);
  cp.rows.nr = __shfl_sync(0xffffffffu, cp.rows.nr, src);
  cp.rows.nc = __shfl_sync(0xffffffffu, cp.rows.nc, src);
  return cp;
}

// The same for a single sequence: nothing to add up.
template <bool WEIGHTS>
__device__ __forceinline__ CtaPlan plan_one(const PagedAttnParams &p, bool writes) {
  const SeqRows rows = seq_rows<WEIGHTS>(p, 0);
  const unsigned n = rows.tiles(), G = gridDim.x, i = blockIdx.x;
  const unsigned c = (n + G - 1) / G, k = n > 0 ? (n + c - 1) / c : 0;  // tiles of an item, items
  CtaPlan cp = {0, 0, 0, 0, rows};
  if (i < k) {
    cp.tile = (int)(i * n / k);
    cp.n = (int)((i + 1) * n / k) - cp.tile;
  }
  if (writes && threadIdx.x == 0) p.ws_plan[0] = make_int2(0, (int)k);
  return cp;
}

// The same for more sequences, by the whole block: thread t counts sequence t
// of every round of 512.  `counts`: 512 ints of shared memory, free until the
// caller's barrier, which publishes the result (ms.plan).
template <bool WEIGHTS>
__device__ __forceinline__ void plan_block(const PagedAttnParams &p, PMisc &ms, int *counts) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = gridDim.x, cta = blockIdx.x;
  const SeqRows none = {0, 0, 0};
  // Sum over the warps before this one, and over all, of `inc` in lane 31.
  auto before_warp = [&](int inc, int &all) {
    if (lane == 31) ms.scan[warp] = inc;
    __syncthreads();
    const int v = lane < kWarps ? (int)ms.scan[lane] : 0;
    all = __reduce_add_sync(0xffffffffu, v);
    return __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
  };
  SeqRows rows = tid < p.n_seq ? seq_rows<WEIGHTS>(p, tid) : none;
  int n = rows.tiles(), mine = n, total;
  for (int b = tid + kThreads; b < p.n_seq; b += kThreads) mine += seq_rows<WEIGHTS>(p, b).tiles();
  counts[tid] = n;
  int inc = scan_warp(mine, lane);
  int before = before_warp(inc, total);
  const int per = (total + G - 1) / G;
  if (p.n_seq <= kThreads && total > 0) {
    static_assert(kTries <= kWarps, "a warp per item size");
    if (warp < kTries) {
      int items = 0;
      for (int b = lane; b < p.n_seq; b += 32) items += (counts[b] + per + warp - 1) / (per + warp);
      items = __reduce_add_sync(0xffffffffu, items);
      if (lane == 0) ms.fits[warp] = warp < per && items <= G;
    }
    __syncthreads();
    const unsigned fit = __ballot_sync(0xffffffffu, lane < kTries && ms.fits[lane < kTries ? lane : 0]);
    if (fit != 0) {
      const int c = per + __ffs(fit) - 1, k = (n + c - 1) / c;
      int all;
      inc = scan_warp(k, lane);
      const int first = before_warp(inc, all) + inc - k;  // CTA of the sequence's first item
      if (cta >= all && tid == 0) ms.plan.n = 0;
      if (k > 0 && first <= cta && cta < first + k) {
        const unsigned i = cta - first;
        const int j0 = (int)(i * (unsigned)n / (unsigned)k);
        ms.plan = CtaPlan{(int)((i + 1) * (unsigned)n / (unsigned)k) - j0, tid, j0, 0, rows};
      }
      if (!WEIGHTS && cta == 0 && tid < p.n_seq) p.ws_plan[tid] = make_int2(first, k);
      return;
    }
  }
  const int g0 = min(total, cta * per), g1 = min(total, g0 + per);
  if (tid == 0 && g1 == g0) ms.plan.n = 0;
  int carry = 0;
  for (int b0 = 0; b0 < p.n_seq; b0 += kThreads) {
    const int b = b0 + tid;
    if (p.n_seq > kThreads) {  // several rounds: scan each by itself
      rows = b < p.n_seq ? seq_rows<WEIGHTS>(p, b) : none;
      n = rows.tiles();
      inc = scan_warp(n, lane);
      int all;
      __syncthreads();
      before = carry + before_warp(inc, all);
      carry += all;
    }
    const int at = before + inc - n;  // tiles before sequence b
    if (n > 0 && at <= g0 && g0 < at + n && g1 > g0) ms.plan = CtaPlan{g1 - g0, b, g0 - at, 1, rows};
    if (!WEIGHTS && cta == 0 && b < p.n_seq) {
      const int c0 = n > 0 ? at / per : 0, c1 = n > 0 ? (at + n - 1) / per : -1;
      p.ws_plan[b] = make_int2(c0 + b, c1 - c0 + 1);
    }
  }
}

// The geometry and the page tables, into L2 while the previous kernel still
// runs: each CTA a part of them.  (Only L2: what they hold then does not matter.)
template <bool WEIGHTS>
__device__ __forceinline__ void prefetch_tables(const PagedAttnParams &p) {
  auto lines = [&](const void *at, long long bytes, long long line) {
    if (line * 128 < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(at) + line * 128));
  };
  lines(p.geom, 16ll * p.n_seq, threadIdx.x);
  const long long line = (long long)blockIdx.x * kThreads + threadIdx.x;
#pragma unroll
  for (int i = WEIGHTS ? 1 : 0; i < 2; ++i)
    if (p.seg[i].max_rows > 0) lines(p.seg[i].table, 4ll * p.seg[i].table_stride * (p.n_seq - 1) + 4, line);
}

// ------------------------------------------------------------------ loaders

// Lists run ahead of the copies: while the rows of tile g are issued, its scales
// and the page ids of tile g + 1 are on their way in registers, so neither
// latency stands between tiles.  One loop holds the code of every step once, in
// the order in which the first tile runs through it: the code is cold when a CTA
// starts, and each further copy of a step in its way cost some 1,000 cycles.
template <bool FP8, bool WEIGHTS, bool SHARED>
__device__ __forceinline__ void load_role(const PagedAttnParams &p, const CtaPlan &cp, uint32_t sbase, PMisc &ms,
                                          int ltid) {
  constexpr int kGroup = loader_threads<FP8>();
  constexpr int kRowStep = kGroup / 8, kWarps = kGroup / 32;
  constexpr int kMine = (kTile + kGroup - 1) / kGroup;  // list rows of a thread
  volatile int *abrt = &ms.abort_flag;
  const int gtid = (FP8 && ltid >= 32) ? ltid - kTile : ltid;  // 0 .. kGroup - 1
  const int c8 = gtid & 7, rsub = gtid >> 3;
  const uint32_t b_q_full = smem_u32(&ms.q_full), b_q_empty = smem_u32(&ms.q_empty);
  const long long vdelta0 = p.seg[0].v - p.seg[0].k, vdelta1 = p.seg[1].v - p.seg[1].k;
  const int pad_seg = p.seg[1].max_rows > 0 ? 1 : 0;
  const unsigned long long pad_row = reinterpret_cast<unsigned long long>(p.seg[pad_seg].k) | pad_seg | kNoRow;
  StageRing ring;
  bool ok = true;
  bool q_issued = cp.n > 0;  // (the first Q by the kernel's thread 0)
  uint32_t n_item = 1, q_par = 0;
  uint32_t filled = 0, last_par = 0;  // TMA stages this thread issued, and their phases
  int turn = 0;                       // warp of the next part's first run
  const int nt = cp.n;

  Walk<WEIGHTS> w;     // at the tile whose page ids are fetched next
  w.start(cp);
  // Tile whose page ids are in flight, then tile whose scales are.
  int a_row[kMine], a_page[kMine], a_seq = 0, a_flags = 0, a_base = 0, a_end = 0;
  bool a_full = false, b_full = false;  // 128 compressed rows in runs that TMA can copy
  unsigned long long b_at[kMine];
  int b_page[kMine], b_slot[kMine];
  bool b_tma = false;
  float b_ks[kMine], b_vs[kMine];
  int b_seq = 0, b_flags = 0, b_base = 0, b_end = 0;

  // A field of segment sg: a choice of two constants (weights of 16 sequences of
  // E4M3 rows 25.7 us; the same with indexed loads of the parameters).
  auto of = [&](int sg, auto field) { return sg != 0 ? p.seg[1].*field : p.seg[0].*field; };
  auto fetch_pages = [&]() {
    a_seq = w.b;
    a_flags = w.flags();
    a_base = w.j * kTile;
    a_end = w.rows.nc + w.rows.nr;
    a_full = p.run_rows > 0 && a_base + kTile <= w.rows.nc;
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      const int r = gtid + u * kGroup, x = a_base + r;
      a_row[u] = -1;
      a_page[u] = -1;
      if (r < kTile && x < a_end) {
        const int sg = WEIGHTS || x < w.rows.nc ? 1 : 0;
        const int row = sg == 0 ? w.rows.raw_lo + x - w.rows.nc : x;
        const int shift = of(sg, &PagedSeg::page_shift), per = of(sg, &PagedSeg::page_rows);
        const int pi = shift >= 0 ? row >> shift : row / per;
        a_page[u] = of(sg, &PagedSeg::table)[w.b * of(sg, &PagedSeg::table_stride) + pi];
        a_row[u] = 2 * (row - pi * per) + sg;
      }
    }
    w.next(p);
  };
  auto fetch_scales = [&](bool ahead) {
    b_seq = a_seq;
    b_flags = a_flags;
    b_base = a_base;
    b_end = a_end;
    b_full = a_full;
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      b_at[u] = pad_row;
      b_page[u] = a_page[u];
      b_slot[u] = a_row[u] >> 1;
      b_ks[u] = 0.f;
      b_vs[u] = 1.f;
      const int sg = WEIGHTS ? 1 : a_row[u] & 1;
      if (a_row[u] >= 0 && (unsigned)a_page[u] < (unsigned)of(sg, &PagedSeg::n_pages)) {
        const int slot = a_row[u] >> 1;
        b_at[u] = reinterpret_cast<unsigned long long>(of(sg, &PagedSeg::k) + a_page[u] * of(sg, &PagedSeg::page_stride) +
                                                       slot * of(sg, &PagedSeg::row_stride)) |
                  sg;
        if (SHARED && ahead && a_full && p.run_bytes > 0 && ((gtid + u * kGroup) & (p.run_rows - 1)) == 0)
          l2_prefetch(reinterpret_cast<const void *>(b_at[u] & ~15ull), p.run_bytes);
        if (FP8) {
          const long long sr = (long long)a_page[u] * of(sg, &PagedSeg::page_rows) + slot;
          b_ks[u] = of(sg, &PagedSeg::k_scale)[sr];
          if (!WEIGHTS) b_vs[u] = of(sg, &PagedSeg::v_scale)[sr];
        }
      }
    }
  };
  // The rows of tile g, complete for the whole group; all go on or none.
  // Returns whether TMA loads the tile.
  auto store_list = [&](int g) -> bool {
    const int buf = g % kLists;
    const bool full = b_full;
    bool absent = false;
    b_tma = false;
    if (ok && !mbar_wait(smem_u32(&ms.list_empty[buf]), ((g / kLists) & 1) ^ 1, abrt, p.timeout_ns, p.err,
                         PSITE_LIST_EMPTY))
      ok = false;
    if (ok) {
#pragma unroll
      for (int u = 0; u < kMine; ++u) {
        const int r = gtid + u * kGroup;
        if (r < kTile) {
          ms.row[buf][r] = b_at[u];
          absent = absent || (b_at[u] & kNoRow);
          if (full && (r & (p.run_rows - 1)) == 0) ms.box[buf][r >> p.run_shift] = make_int2(b_page[u], b_slot[u]);
        }
      }
    }
    __syncwarp();  // the barrier below is one of whole warps
    const bool odd = bar_red_or(2, kGroup, !ok || (full && absent));
    if (odd) ok = !bar_red_or(2, kGroup, !ok);
    b_tma = full && !odd;
    return b_tma;
  };
  // The rest of it, once its rows are on their way: what the other warps need.
  auto finish_list = [&](int g) {
    const int buf = g % kLists;
    if (ok) {
      if (FP8) {
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
          const int r = gtid + u * kGroup;
          if (r < kTile) {
            ms.ksc[buf][r] = p.scale_log2 * b_ks[u];
            if (!WEIGHTS) {
              const float lv = fmaxf(__log2f(b_vs[u]), kLeastLog2Scale);
              ms.lvs[buf][r] = lv;
              ms.ivs[buf][r] = exp2f(-lv);
            }
          }
        }
      }
      if (gtid == 0) {
        ms.gathered[buf] = !b_tma;
        ms.seq[buf] = b_seq;
        ms.flags[buf] = b_flags;
        ms.base[buf] = b_base;
        ms.end[buf] = b_end;
      }
    }
    mbar_arrive(smem_u32(&ms.list_full[buf]));
  };
  // One part of tile g into the next stage (parts 0-3: K dims 128 part .., 4-7: V).
  auto emit = [&](int g, int part, bool tma) -> bool {
    const uint32_t stage = sbase + kOffKV + ring.st * kStageBytes;
    const uint32_t b_full_bar = smem_u32(FP8 ? &ms.code_full[ring.st] : &ms.kv_full[ring.st]);
    const uint32_t b_empty = smem_u32(&ms.kv_empty[ring.st]), ph = ring.ph ^ 1, st_bit = 1u << ring.st;
    ring.advance();
    // Every thread waits for every fill of a stage, whoever loads it: a parity
    // wait is only right for a thread that has seen the phase before.
    if (!mbar_wait(b_empty, ph, abrt, p.timeout_ns, p.err, PSITE_KV_EMPTY)) return false;
    if (tma) {
      // Run i of a part goes to one lane of warp (turn + i) % warps, so that
      // the warps share the copies of a part and of successive parts; lane 0
      // of each warp arrives for all its lanes.
      const int lane = ltid & 31, runs = kTile >> p.run_shift;
      const int first = gtid / 32 - turn, i = (first < 0 ? first + kWarps : first) + lane * kWarps;
      turn = (turn + runs) % kWarps;
      if (lane == 0) {
        if (gtid == 0) mbar_arrive_expect_tx(b_full_bar, FP8 ? kBoxBytes : kStageBytes);
        mbar_arrive_cnt(b_full_bar, gtid == 0 ? 31 : 32);
      }
      if (i < runs) {
        filled |= st_bit;
        last_par = ph ? last_par & ~st_bit : last_par | st_bit;
        const uint32_t at = (i << p.run_shift) * (FP8 ? 128u : 256u);
        const CUtensorMap *m = part >= 4 ? &p.tm_v : &p.tm_k;
        const int2 x = ms.box[g % kLists][i];
        if (FP8)
          tma_load_3d(stage + kBoxBytes + at, m, b_full_bar, 128 * (part & 3), x.y, x.x);
        else
          tma_load_5d(stage + at, m, b_full_bar, 0, 0, 2 * (part & 3), x.y >> 3, x.x);
      }
      return true;
    }
    const unsigned long long *list = ms.row[g % kLists];
    const int dim = (FP8 ? 128 : 256) * (part & 3) + 16 * c8;  // bytes
    const long long off0 = part >= 4 ? vdelta0 + dim : dim, off1 = part >= 4 ? vdelta1 + dim : dim;
#pragma unroll
    for (int it = 0; it < (kTile + kRowStep - 1) / kRowStep; ++it) {
      const int row = kRowStep * it + rsub;
      if (kTile % kRowStep != 0 && row >= kTile) break;
      const unsigned long long e = list[row];
      const uint32_t n = (e & kNoRow) ? 0u : 16u;
      const uint8_t *src = reinterpret_cast<const uint8_t *>(e & ~15ull) + ((e & kSegBit) ? off1 : off0);
      if (FP8) {
        cp_async16z(stage + kBoxBytes + row * 128 + 16 * c8, src, n);
      } else {
        const uint32_t dst = stage + (row >> 3) * group_stride<FP8>() + (row & 7) * 128 + ((c8 ^ (row & 7)) << 4);
        cp_async16z(dst, src, n);                              // dims 0-63 of the part
        cp_async16z(dst + block_stride<FP8>(), src + 128, n);  // dims 64-127
      }
    }
    cp_async_arrive(b_full_bar);
    return true;
  };
  auto load_q = [&](int b) {
    if (ltid == 0 && ok) {
      if (!mbar_wait(b_q_empty, (n_item & 1) ^ 1, abrt, p.timeout_ns, p.err, PSITE_Q_EMPTY)) {
        ok = false;
      } else {
        mbar_arrive_expect_tx(b_q_full, kQBytes);
        tma_load_4d(sbase + kOffQ, &p.tm_q, b_q_full, 0, 0, b, 0);
        q_issued = true;
        q_par = n_item & 1;
      }
    }
    ++n_item;
  };

  if (nt > 0) fetch_pages();
  bool tma = false, tma_v;  // whether TMA loads tile g, and tile g - 1
  for (int g = 0; nt > 0 && (g < nt || (!WEIGHTS && !SHARED && g == nt)); ++g) {
    tma_v = tma;
    if (g < nt) {
      // The first tile's rows before the prefetch of the second's: every SM wants
      // its first tile at the same time.
      if (SHARED && g == 1)
        mbar_wait(smem_u32(FP8 ? &ms.code_full[kStages - 1] : &ms.kv_full[kStages - 1]), 0, abrt, p.timeout_ns, p.err,
                  FP8 ? PSITE_CODE_FULL : PSITE_KV_FULL);
      fetch_scales(g > 0);
      if (g + 1 < nt) fetch_pages();
      tma = store_list(g);
      if (g > 0 && (b_flags & kFirst)) load_q(b_seq);
      for (int part = 0; part < 4 && ok; ++part) ok = emit(g, part, tma);
      finish_list(g);
    } else {
      __syncwarp();
      ok = !bar_red_or(2, kGroup, !ok);
    }
    if (!WEIGHTS && !SHARED && g > 0)
      for (int part = 4; part < 8 && ok; ++part) ok = emit(g - 1, part, tma_v);
  }
  // No copy may still be landing at exit.  (When every wait succeeded the MMA
  // thread has seen all stages land.)
  cp_async_done();
  volatile int never = 0;
  if (*abrt != 0)
    for (int st = 0; st < kStages; ++st)
      if (filled & (1u << st))
        mbar_wait(smem_u32(FP8 ? &ms.code_full[st] : &ms.kv_full[st]), (last_par >> st) & 1, &never, 100000000ull,
                  p.err, PSITE_DRAIN);
  if (ltid == 0 && q_issued) mbar_wait(b_q_full, q_par, &never, 100000000ull, p.err, PSITE_DRAIN);
}

// Warps 9-12 with E4M3 rows: every stage's codes (upper half), one row per
// thread, widened exactly to fp16 in the swizzled layout.  Row r's values
// overwrite only row r's own codes, which its thread has read first.
template <int PARTS>
__device__ __forceinline__ void convert_role(const PagedAttnParams &p, const CtaPlan &cp, uint32_t sbase, PMisc &ms,
                                             int row) {
  volatile int *abrt = &ms.abort_flag;
  StageRing ring;
  const long long parts = (long long)cp.n * PARTS;
  for (long long i = 0; i < parts; ++i) {
    if (!mbar_wait(smem_u32(&ms.code_full[ring.st]), ring.ph, abrt, p.timeout_ns, p.err, PSITE_CODE_FULL)) return;
    const uint32_t stage = sbase + kOffKV + ring.st * kStageBytes;
    uint4 raw[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t a = stage + kBoxBytes + row * 128 + 16 * ((k + row) & 7);
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(raw[k].x), "=r"(raw[k].y), "=r"(raw[k].z), "=r"(raw[k].w)
                   : "r"(a));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = (k + row) & 7;
      const uint32_t w4[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[2 * e] = e4m3x2_to_f16x2(static_cast<uint16_t>(w4[e] & 0xFFFFu));
        h[2 * e + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w4[e] >> 16));
      }
      const uint32_t drow = stage + (c >> 2) * kBoxBytes + row * 128;
      const int col = 2 * (c & 3);
      sts_v4(drow + ((col ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
      sts_v4(drow + (((col + 1) ^ (row & 7)) << 4), h[4], h[5], h[6], h[7]);
    }
    mbar_arrive(smem_u32(&ms.kv_full[ring.st]));
    ring.advance();
  }
}

// ------------------------------------------------------------------ MMA issue

// The whole warp walks the tiles, so that descriptors are warp-uniform values,
// and one elected lane issues (47 cycles per 128 x 64 x 16 MMA in a row; 61
// when a single lane runs the role).  Waits are joined over the warp: all lanes go
// on or none.
template <bool FP8, bool WEIGHTS, bool SHARED>
__device__ __forceinline__ void mma_role_paged(const PagedAttnParams &p, const CtaPlan &cp, uint32_t sbase,
                                               uint32_t tmem, PMisc &ms) {
  volatile int *abrt = &ms.abort_flag;
  constexpr uint32_t kIdescQK = idesc_f16_f32(128, 64, false, false);
  constexpr uint32_t kIdescPV = idesc_f16_f32(128, 64, true, true);
  // K tiles and Q: K-major.  V tiles: MN-major, LBO = distance of the 64-dim
  // blocks, SBO = distance of 8-row groups.  P^T: one 64-head MN atom.
  constexpr uint32_t kGrp = group_stride<FP8>(), kBlk = block_stride<FP8>();
  const uint64_t k_desc = sdesc_sw128(sbase + kOffKV, 16, kGrp);
  const uint64_t v_desc = sdesc_sw128(sbase + kOffKV, kBlk, kGrp);
  const uint64_t q_desc = sdesc_sw128(sbase + kOffQ, 16, 1024);
  const uint64_t p_desc = sdesc_sw128(sbase + kOffP, 16, 1024);
  StageRing ring;
  const int nt = cp.n;
  uint32_t q_item = 0, o_item = 0;
  bool ok = true;
  auto wait = [&](uint64_t &bar, uint32_t parity, unsigned int site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity, abrt, p.timeout_ns, p.err, site));
  };
  auto commit = [&](uint64_t &bar) {
    if (elect_lane()) umma_commit(smem_u32(&bar));
  };
  // Gathered rows (cp.async) and widened ones are generic-proxy writes: the fence
  // makes the landed stage visible to the tensor core (here one warp's, which took
  // 2% less of E4M3 decodes than one by every converter).  TMA writes need none.  No tcgen05 fence here: it is
  // for TMEM that other threads read or wrote.  fp16 stages are waited for two
  // at a time: behind the eight MMAs of one the warp would stand still until
  // they are done.  (E4M3 stages come one by one from the converters.)
  constexpr int kStep = FP8 ? 1 : 2;
  auto stages_ready = [&](int g) -> bool {
#pragma unroll
    for (int u = 0; u < kStep; ++u)
      if (!wait(ms.kv_full[ring.st + u], ring.ph, PSITE_KV_FULL)) return false;
    if (FP8 || ms.gathered[g % kLists]) fence_proxy_async_smem();
    return true;
  };
  auto qk = [&](int g, bool first, bool last) -> bool {
    if (first) {
      if (!wait(ms.q_full, q_item & 1, PSITE_Q_FULL)) return false;
      ++q_item;
    }
    const uint32_t sb = g & 1;
    if (!FP8 && !wait(ms.list_full[g % kLists], (g / kLists) & 1, PSITE_LIST_FULL)) return false;
    if (!wait(ms.s_empty[sb], ((g >> 1) & 1) ^ 1, PSITE_S_EMPTY)) return false;
    tc_fence_after();
    const uint32_t d_s = tmem + kTmemS + 64 * sb;
    for (int c = 0; c < 4; c += kStep) {
      if (!stages_ready(g)) return false;
      const uint64_t a0 = sdesc_add(k_desc, ring.st * kStageBytes);
      const uint64_t b0 = sdesc_add(q_desc, 2 * c * kQBoxBytes);
      if (elect_lane()) {
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
#pragma unroll
          for (int b2 = 0; b2 < 2; ++b2) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              const uint64_t a = sdesc_add(a0, u * kStageBytes + b2 * kBlk + ks * 32);
              const uint64_t b = sdesc_add(b0, (2 * u + b2) * kQBoxBytes + ks * 32);
              if (u == 0 && b2 == 0 && ks == 0)
                umma_f16(d_s, a, b, kIdescQK, c != 0 ? 1u : 0u);
              else
                umma_f16_acc(d_s, a, b, kIdescQK);
            }
          }
          if (!SHARED) umma_commit(smem_u32(&ms.kv_empty[ring.st + u]));
        }
        if (c + kStep == 4) umma_commit(smem_u32(&ms.s_full[sb]));
        if (c + kStep == 4 && last) umma_commit(smem_u32(&ms.q_empty));
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kStep; ++u) ring.advance();
    }
    return true;
  };
  auto pv = [&](int g, bool first, bool last) -> bool {
    if (!wait(ms.p_full, g & 1, PSITE_P_FULL)) return false;
    if (first) {
      if (!wait(ms.o_empty, (o_item & 1) ^ 1, PSITE_O_EMPTY)) return false;
      ++o_item;
    }
    tc_fence_after();
    for (int m = 0; m < 4; m += kStep) {
      // Shared rows: part m still lies in stage m, where QK^T read it.
      if (!SHARED && !stages_ready(g)) return false;
      const int st = SHARED ? m : (int)ring.st;
      const uint64_t a0 = sdesc_add(v_desc, st * kStageBytes);
      if (elect_lane()) {
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint64_t a = sdesc_add(a0, u * kStageBytes + ks * 2 * kGrp);
            const uint64_t b = sdesc_add(p_desc, ks * 2048);
            if (ks == 0)
              umma_f16(tmem + 64 * (m + u), a, b, kIdescPV, first ? 0u : 1u);
            else
              umma_f16_acc(tmem + 64 * (m + u), a, b, kIdescPV);
          }
          umma_commit(smem_u32(&ms.kv_empty[st + u]));
          if (last) umma_commit(smem_u32(&ms.o_full[m + u]));
        }
        if (m + kStep == 4) umma_commit(smem_u32(&ms.p_empty));
      }
      __syncwarp();
      if (!SHARED)
#pragma unroll
        for (int u = 0; u < kStep; ++u) ring.advance();
    }
    return true;
  };
  Walk<WEIGHTS> w;
  w.start(cp);
  if (nt > 0) ok = qk(0, true, w.last);
  for (int g = 0; g < nt && ok; ++g) {
    const bool first = w.first, last = w.last;
    if (SHARED) ok = pv(g, first, last);  // frees the stages of the next tile
    if (ok && g + 1 < nt) {
      w.next(p);
      ok = qk(g + 1, w.first, w.last);
    }
    if (!WEIGHTS && !SHARED) ok = ok && pv(g, first, last);
  }
  commit(ms.mma_done);
  volatile int never = 0;
  mbar_wait(smem_u32(&ms.mma_done), 0, &never, 100000000ull, p.err, PSITE_DRAIN);
  __syncwarp();
}

// ------------------------------------------------------------------ softmax and epilogue

// The reference of a head lies kLift below the largest score of the tile that
// set it, and moves only when a score passes it by kLift + kHold, so P is 2^15
// at most (fp16 holds 65504) and keeps fp16's full precision for rows down to
// 2^-(14 + kLift) of the largest weight; rows further down are off by half a
// step, 2^-(25 + kLift) of it.  (Without the lift a row of 2^-25 counted in the
// sum and not in the product: a long tail under one row lost 42% of its value.)
// While the reference holds (nearly always after a sequence's first tile) a
// tile needs no maximum over its rows: one vote of the block that no score is
// over.  kLift and kHold share out fp16's 15 bits above 1: 64 sequences of fp16
// and 24 of E4M3 rows take 0.5% and 0.2% longer with 10 + 5 than with 7 + 8, 5%
// and 7% longer with 12 + 3, where the reference moves often.  kNoRef stands for
// no reference yet: any score passes it, and absent rows (-inf) get weight 0
// under it.
constexpr float kLift = 10.f, kHold = 5.f;
constexpr float kNoRef = -3e38f;

template <bool FP8>
__device__ __forceinline__ void softmax_role(const PagedAttnParams &p, const CtaPlan &cp, uint8_t *smem, uint32_t tmem,
                                             PMisc &ms, int tid) {
  volatile int *abrt = &ms.abort_flag;
  const int wq = tid >> 5, l = tid & 31;
  const int q = wq & 3, hh = wq >> 2;  // TMEM lane quarter, head half
  const int r = 32 * q + l;            // row of the tile, or dim of a 128-dim block
  const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
  const uint32_t col0 = 32 * hh;
  const int nt = cp.n;
  bool bad = false;
  uint32_t n_item = 0;
  float m_ref = kNoRef, m_lim = kNoRef;  // reference of head `tid` (threads < 64), log2 units, and its limit
  float lpart[32];
  if (tid < kH) ms.m_use[tid] = ms.m_lim[tid] = kNoRef;
  bar_sync_id(1, kComputeThreads);
  for (int g = 0; g < nt; ++g) {
    const int buf = g % kLists;
    const uint32_t sb = g & 1;
    bad = bad || !mbar_wait(smem_u32(&ms.list_full[buf]), (g / kLists) & 1, abrt, p.timeout_ns, p.err, PSITE_LIST_FULL);
    const int flags = ms.flags[buf], seq = ms.seq[buf];
    if (flags & kFirst) {
#pragma unroll
      for (int h = 0; h < 32; ++h) lpart[h] = 0.f;
    }
    const bool vis = (ms.row[buf][r] & kNoRow) == 0;
    const float sl2 = FP8 ? ms.ksc[buf][r] : p.scale_log2;
    const float lvs = FP8 ? ms.lvs[buf][r] : 0.f;
    const float ivs = FP8 ? ms.ivs[buf][r] : 1.f;
    mbar_arrive(smem_u32(&ms.list_empty[buf]));
    bad = bad || !mbar_wait(smem_u32(&ms.s_full[sb]), (g >> 1) & 1, abrt, p.timeout_ns, p.err, PSITE_S_FULL);
    tc_fence_after();
    float s[32];
    tmem_ld32(tmem + kTmemS + 64 * sb + col0 + lane_base, s);
    tmem_wait_ld();
    tc_fence_before();
    mbar_arrive(smem_u32(&ms.s_empty[sb]));
    bool over = false;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float4 lim = reinterpret_cast<const float4 *>(ms.m_lim + col0)[c];
      const float li[4] = {lim.x, lim.y, lim.z, lim.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[4 * c + i] = vis ? fmaf(s[4 * c + i], sl2, lvs) : -INFINITY;
        over = over || s[4 * c + i] > li[i];
      }
    }
    bool resc = false;
    if (bar_red_or(1, kComputeThreads, over || bad)) {
      // Some head's reference moves: the tile's maxima over the rows.
      ms.red[q][col0 + l] = reduce_heads<true>(s, l);
      if (bar_red_or(1, kComputeThreads, bad)) break;
      if (tid < kH) {
        const float tmax = fmaxf(fmaxf(ms.red[0][tid], ms.red[1][tid]), fmaxf(ms.red[2][tid], ms.red[3][tid]));
        float alpha = 1.f;
        if (tmax > m_lim) {
          // Rounded so that P stays within 2^15 where scores are 16 and more apart.
          const float next = __fsub_ru(tmax, kLift);
          alpha = exp2f(m_ref - next);  // 0 while there was none
          m_ref = next;
          m_lim = __fadd_rd(m_ref, kLift + kHold);
        }
        ms.m_use[tid] = m_ref;
        ms.m_lim[tid] = m_lim;
        ms.alpha[tid] = alpha;
      }
      bar_sync_id(1, kComputeThreads);
      resc = true;
    }
    bad = bad || !mbar_wait(smem_u32(&ms.p_empty), (g & 1) ^ 1, abrt, p.timeout_ns, p.err, PSITE_P_EMPTY);
    {
      // P^T row r: heads 32hh .. +31 are 16-byte chunks 4hh .. 4hh+3 of its
      // 128 bytes, chunk c at c ^ (r & 7).  P is rounded once to fp16 for the
      // MMA, to 2^-11 of a weight (below 2^-(14 + kLift) of the largest, to half
      // a step); the row sums add it unrounded, so lse keeps fp32 precision.
      uint8_t *prow = smem + kOffP + r * 128;
      const bool dead = FP8 && lvs <= kLeastLog2Scale;  // a V scale of 0: weight, but no value
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 m0 = reinterpret_cast<const float4 *>(ms.m_use + col0)[2 * c];
        const float4 m1 = reinterpret_cast<const float4 *>(ms.m_use + col0)[2 * c + 1];
        const float mu[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
        if (resc) {
          const float4 a0 = reinterpret_cast<const float4 *>(ms.alpha + col0)[2 * c];
          const float4 a1 = reinterpret_cast<const float4 *>(ms.alpha + col0)[2 * c + 1];
          const float al[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) lpart[8 * c + i] *= al[i];
        }
        uint32_t w4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int h = 8 * c + 2 * i;
          const float e0 = exp2f(s[h] - mu[2 * i]), e1 = exp2f(s[h + 1] - mu[2 * i + 1]);
          lpart[h] = FP8 ? fmaf(e0, ivs, lpart[h]) : lpart[h] + e0;
          lpart[h + 1] = FP8 ? fmaf(e1, ivs, lpart[h + 1]) : lpart[h + 1] + e1;
          const __half2 hp = __floats2half2_rn(e0, e1);
          w4[i] = dead ? 0u : *reinterpret_cast<const uint32_t *>(&hp);
        }
        *reinterpret_cast<uint4 *>(prow + (((4 * hh + c) ^ (r & 7)) << 4)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
      }
    }
    if (resc && !(flags & kFirst)) {
      tc_fence_after();
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        float o[32];
        tmem_ld32(tmem + 64 * m + col0 + lane_base, o);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 a = reinterpret_cast<const float4 *>(ms.alpha + col0)[c];
          o[4 * c] *= a.x;
          o[4 * c + 1] *= a.y;
          o[4 * c + 2] *= a.z;
          o[4 * c + 3] *= a.w;
        }
        tmem_st32(tmem + 64 * m + col0 + lane_base, o);
      }
      tmem_wait_st();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    mbar_arrive(smem_u32(&ms.p_full));
    if (!(flags & kLast)) continue;

    // End of an item: row sums, then o block by block as the last PV finishes
    // them: fp16 and normalised for a whole sequence, else fp32 and normalised
    // by the item's own sum.
    const bool whole = flags & kWhole;
    const long long slot = (long long)blockIdx.x + (long long)cp.slot_step * seq;
    ms.red[q][col0 + l] = reduce_heads<false>(lpart, l);
    if (bar_red_or(1, kComputeThreads, bad)) break;
    if (tid < kH) {
      const float lsum = ms.red[0][tid] + ms.red[1][tid] + ms.red[2][tid] + ms.red[3][tid];
      // No weight at all: o = 0.  (A sum that is NaN is not that: it stays.)
      const bool none = lsum == 0.f;
      ms.inv_l[tid] = none ? 0.f : 1.f / lsum;
      if (!whole) {
        p.ws_ml[slot * kH + tid] = make_float2(none ? -INFINITY : m_ref, lsum);
      } else if (p.lse != nullptr) {
        p.lse[(long long)seq * kH + tid] = none ? -INFINITY : (m_ref + log2f(lsum)) * kLn2;
      }
    }
    bar_sync_id(1, kComputeThreads);
    float inv[32];
    load_row32(ms.inv_l + col0, inv);
#pragma unroll 1
    for (int m = 0; m < 4; ++m) {
      bad = bad || !mbar_wait(smem_u32(&ms.o_full[m]), n_item & 1, abrt, p.timeout_ns, p.err, PSITE_O_FULL);
      tc_fence_after();
      float o[32];
      tmem_ld32(tmem + 64 * m + col0 + lane_base, o);
      tmem_wait_ld();
      if (whole) {
        // Lanes 2k and 2k + 1 hold adjacent dims: they swap one value per pair
        // of heads and write half2.
        const bool odd = l & 1;
        __half *at = p.o + seq * p.o_stride + (long long)(col0 + (odd ? 1 : 0)) * kD + 128 * m + (r & ~1);
#pragma unroll
        for (int h = 0; h < 32; h += 2) {
          const float a = o[h] * inv[h], c = o[h + 1] * inv[h + 1];
          const float got = __shfl_xor_sync(0xffffffffu, odd ? a : c, 1);
          *reinterpret_cast<__half2 *>(at + h * kD) = odd ? __floats2half2_rn(got, c) : __floats2half2_rn(a, got);
        }
      } else {
        float *at = p.ws_o + (slot * kH + col0) * kD + 128 * m + r;
#pragma unroll
        for (int h = 0; h < 32; ++h) at[h * kD] = o[h] * inv[h];
      }
    }
    tc_fence_before();
    mbar_arrive(smem_u32(&ms.o_empty));
    ++n_item;
    m_ref = m_lim = kNoRef;
    if (tid < kH) ms.m_use[tid] = ms.m_lim[tid] = kNoRef;
    if (bar_red_or(1, kComputeThreads, bad)) break;
  }
}

// Weights: row r of a tile is TMEM lane r; each head half adds its 32 heads'
// exponentials in registers and the halves meet in shared memory.
template <bool FP8>
__device__ __forceinline__ void weights_role(const PagedAttnParams &p, const CtaPlan &cp, uint32_t tmem, PMisc &ms,
                                             int tid) {
  volatile int *abrt = &ms.abort_flag;
  const int wq = tid >> 5, l = tid & 31;
  const int q = wq & 3, hh = wq >> 2;
  const int r = 32 * q + l;
  const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
  const uint32_t col0 = 32 * hh;
  const int nt = cp.n;
  bool bad = false;
  float *part = &ms.red[0][0];  // [2][128] by tile parity (256 floats)
  for (int g = 0; g < nt; ++g) {
    const int buf = g % kLists;
    const uint32_t sb = g & 1;
    bad = bad || !mbar_wait(smem_u32(&ms.list_full[buf]), (g / kLists) & 1, abrt, p.timeout_ns, p.err, PSITE_LIST_FULL);
    // All go on or none: without the list its flags and sequence are what an
    // earlier kernel left here, and lead to barriers and addresses of their own.
    if (bar_red_or(1, kComputeThreads, bad)) break;
    const int seq = ms.seq[buf], c = ms.base[buf] + r;
    const bool mine = hh == 0 && c < ms.end[buf];
    const float before = mine && p.acc_in != nullptr ? p.acc_in[seq * p.acc_in_stride + c] : 0.f;
    if (ms.flags[buf] & kFirst) {
      // 2^(s - lse log2 e); a head whose lse is -inf gave no weight to anything.
      if (tid < kH) {
        const float v = p.lse_in[(long long)seq * kH + tid];
        ms.m_use[tid] = v == -INFINITY ? INFINITY : v * kLog2e;
      }
      bar_sync_id(1, kComputeThreads);
    }
    const bool vis = (ms.row[buf][r] & kNoRow) == 0;
    const float sl2 = FP8 ? ms.ksc[buf][r] : p.scale_log2;
    mbar_arrive(smem_u32(&ms.list_empty[buf]));
    bad = bad || !mbar_wait(smem_u32(&ms.s_full[sb]), (g >> 1) & 1, abrt, p.timeout_ns, p.err, PSITE_S_FULL);
    tc_fence_after();
    float s[32];
    tmem_ld32(tmem + kTmemS + 64 * sb + col0 + lane_base, s);
    tmem_wait_ld();
    tc_fence_before();
    mbar_arrive(smem_u32(&ms.s_empty[sb]));
    float ref[32];
    load_row32(ms.m_use + col0, ref);
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < 32; ++h) sum += exp2f(fmaf(s[h], sl2, -ref[h]));
    if (hh == 1) part[128 * (g & 1) + r] = sum;
    if (bar_red_or(1, kComputeThreads, bad)) break;
    if (mine) {
      const float got = vis ? sum + part[128 * (g & 1) + r] : 0.f;
      p.acc_out[seq * p.acc_out_stride + c] = fmaf(p.decay, before, got);
    }
  }
}

// ------------------------------------------------------------------ kernel

// SHARED: K and V are the same rows, loaded once.
template <bool FP8, bool WEIGHTS, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  PMisc &ms = *reinterpret_cast<PMisc *>(smem + kOffMisc);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&ms.q_full), 1);
    mbar_init(smem_u32(&ms.q_empty), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&ms.kv_full[s]), FP8 ? kTile : loader_threads<FP8>());
      mbar_init(smem_u32(&ms.kv_empty[s]), 1);
      mbar_init(smem_u32(&ms.code_full[s]), loader_threads<FP8>());
    }
    for (int s = 0; s < kLists; ++s) {
      mbar_init(smem_u32(&ms.list_full[s]), loader_threads<FP8>());
      mbar_init(smem_u32(&ms.list_empty[s]), kComputeThreads);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ms.s_full[s]), 1);
      mbar_init(smem_u32(&ms.s_empty[s]), kComputeThreads);
    }
    mbar_init(smem_u32(&ms.p_full), kComputeThreads);
    mbar_init(smem_u32(&ms.p_empty), 1);
    for (int m = 0; m < 4; ++m) mbar_init(smem_u32(&ms.o_full[m]), 1);
    mbar_init(smem_u32(&ms.o_empty), kComputeThreads);
    mbar_init(smem_u32(&ms.mma_done), 1);
    ms.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_q);
    if (p.run_rows > 0) {
      tma_prefetch_desc(&p.tm_k);
      if (!WEIGHTS) tma_prefetch_desc(&p.tm_v);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ms.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  prefetch_tables<WEIGHTS>(p);
  tc_fence_before();
  __syncthreads();  // barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  grid_launch_dependents();
  grid_dependency_wait();  // the plan reads the sequences' geometry
  CtaPlan cp;
  const bool writes = !WEIGHTS && blockIdx.x == 0 && warp == 0;
  if (p.n_seq == 1) {
    cp = plan_one<WEIGHTS>(p, writes);
  } else if (p.n_seq <= 32) {
    cp = plan_warp<WEIGHTS, 1>(p, threadIdx.x & 31, writes);
  } else if (p.n_seq <= 64) {
    cp = plan_warp<WEIGHTS, 2>(p, threadIdx.x & 31, writes);
  } else {
    // P's bytes: ordinary stores there are followed by ordinary stores only (the
    // ring's and Q's by TMA, whose writes a block barrier does not order after them).
    plan_block<WEIGHTS>(p, ms, reinterpret_cast<int *>(smem + kOffP));
    __syncthreads();
    cp = ms.plan;
  }
  // The first item's Q, by a thread of the compute warps (which wait for it);
  // the loaders issue those of further items.
  if (threadIdx.x == 0 && cp.n > 0) {
    mbar_arrive_expect_tx(smem_u32(&ms.q_full), kQBytes);
    tma_load_4d(sbase + kOffQ, &p.tm_q, smem_u32(&ms.q_full), 0, 0, cp.seq, 0);
  }
  if (warp < kComputeWarps) {
    if (WEIGHTS)
      weights_role<FP8>(p, cp, tmem, ms, threadIdx.x);
    else
      softmax_role<FP8>(p, cp, smem, tmem, ms, threadIdx.x);
  } else if (warp == kMmaWarp) {
    mma_role_paged<FP8, WEIGHTS, SHARED>(p, cp, sbase, tmem, ms);
  } else {
    const int ltid = threadIdx.x - 32 * kLoaderWarp0;
    if (FP8 && ltid >= 32 && ltid < 32 + kTile)
      convert_role<(WEIGHTS || SHARED) ? 4 : 8>(p, cp, sbase, ms, ltid - 32);
    else
      load_role<FP8, WEIGHTS, SHARED>(p, cp, sbase, ms, ltid);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ merge
// With M = max_s m_s and W_s = 2^(m_s - M) l_s over the slots of a sequence:
//   o = sum_s W_s o_s / L,  L = sum_s W_s,  lse = (M + log2 L) ln 2.
// A sequence that one CTA finished (one slot) is left alone; one without rows
// (no slot) gets o = 0 and lse = -inf.  A lane holds VEC float4 of a head
// (128 VEC dims a warp) and has kMergeLoads of them in flight; a warp's slots are
// loaded together with their (m, l), before the weights are known.

constexpr int kMergeLoads = 8;

template <int VEC>
struct Merged {
  float M, L;  // largest reference and sum of weights (relative to it) so far
  float4 acc[VEC];
};

// Slots first, first + step, .. below n of one head.
template <int VEC>
__device__ __forceinline__ Merged<VEC> merge_slots(const float2 *ml, const float4 *src, int n, int first, int step) {
  constexpr int kRound = kMergeLoads / VEC;
  constexpr long long kSlot = (long long)kH * kD / 4;  // float4 of a slot
  Merged<VEC> r;
  r.M = -INFINITY;
  r.L = 0.f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) r.acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = first; s0 < n; s0 += step * kRound) {
    float4 x[kRound][VEC];
    float2 q[kRound];
#pragma unroll
    for (int k = 0; k < kRound; ++k) {
      const int s = s0 + k * step;
      q[k] = s < n ? ml[(long long)s * kH] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        x[k][e] = s < n ? __ldcs(src + s * kSlot + 32 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = r.M;
#pragma unroll
    for (int k = 0; k < kRound; ++k) top = fmaxf(top, q[k].x);
    if (top == -INFINITY) continue;
    const float old = exp2f(r.M - top);  // 0 while nothing has been added
    r.M = top;
    r.L *= old;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      r.acc[e].x *= old;
      r.acc[e].y *= old;
      r.acc[e].z *= old;
      r.acc[e].w *= old;
    }
#pragma unroll
    for (int k = 0; k < kRound; ++k) {
      const float t = exp2f(q[k].x - top) * q[k].y;
      r.L += t;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        r.acc[e].x = fmaf(t, x[k][e].x, r.acc[e].x);
        r.acc[e].y = fmaf(t, x[k][e].y, r.acc[e].y);
        r.acc[e].z = fmaf(t, x[k][e].z, r.acc[e].z);
        r.acc[e].w = fmaf(t, x[k][e].w, r.acc[e].w);
      }
    }
  }
  return r;
}

__device__ __forceinline__ void store_half4(__half *at, const float4 &o, float f) {
  const __half2 a = __floats2half2_rn(o.x * f, o.y * f), c = __floats2half2_rn(o.z * f, o.w * f);
  *reinterpret_cast<uint2 *>(at) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&c));
}

// A block takes HEADS heads of one sequence, 128 VEC dims of each.  With HEADS
// = WARPS a warp joins a head by itself when the sequence has few slots (a
// batch: no barrier, every load in one or two rounds); otherwise, and with
// HEADS = 1 (few long sequences, up to a slot per SM), the warps share the
// slots of each head and meet in shared memory.
template <int VEC, int WARPS, int HEADS>
__global__ void __launch_bounds__(32 * WARPS) paged_merge_kernel(const PagedAttnParams p) {
  constexpr int kChunks = kD / (128 * VEC), kGroups = kH / HEADS;
  __shared__ float2 wl[WARPS];  // (M, L) of each warp's slots
  __shared__ float4 part[WARPS][32 * VEC];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int item = blockIdx.x / kChunks, chunk = blockIdx.x - item * kChunks;
  const int b = item / kGroups, h0 = (item - b * kGroups) * HEADS;
  const int2 plan = p.ws_plan[b];
  const int n = plan.y;
  if (n == 1) return;
  auto ml_of = [&](int h) { return p.ws_ml + (long long)plan.x * kH + h; };
  auto src_of = [&](int h) {
    return reinterpret_cast<const float4 *>(p.ws_o + ((long long)plan.x * kH + h) * kD + 128 * VEC * chunk) + lane;
  };
  auto out_of = [&](int h) { return p.o + b * p.o_stride + (long long)h * kD + 128 * VEC * chunk; };
  auto put_lse = [&](int h, float M, float L) {
    if (p.lse != nullptr && chunk == 0) p.lse[(long long)b * kH + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  };
  if (HEADS == WARPS && n <= 4 * kMergeLoads / VEC) {
    const int h = h0 + warp;
    const Merged<VEC> r = merge_slots<VEC>(ml_of(h), src_of(h), n, 0, 1);
    const float inv = r.L == 0.f ? 0.f : 1.f / r.L;
#pragma unroll
    for (int e = 0; e < VEC; ++e) store_half4(out_of(h) + 4 * (lane + 32 * e), r.acc[e], inv);
    if (lane == 0) put_lse(h, r.M, r.L);
    return;
  }
  for (int h = h0; h < h0 + HEADS; ++h) {
    const Merged<VEC> r = merge_slots<VEC>(ml_of(h), src_of(h), n, warp, WARPS);
    if (HEADS > 1) __syncthreads();  // the previous head has been read
    if (lane == 0) wl[warp] = make_float2(r.M, r.L);
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[warp][lane + 32 * e] = r.acc[e];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, wl[w].x);
    float t[WARPS];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      t[w] = M == -INFINITY ? 0.f : exp2f(wl[w].x - M);
      L = fmaf(t[w], wl[w].y, L);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    for (int v = threadIdx.x; v < 32 * VEC; v += 32 * WARPS) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4 y = part[w][v];
        o.x = fmaf(t[w], y.x, o.x);
        o.y = fmaf(t[w], y.y, o.y);
        o.z = fmaf(t[w], y.z, o.z);
        o.w = fmaf(t[w], y.w, o.w);
      }
      store_half4(out_of(h) + 4 * v, o, inv);
    }
    if (threadIdx.x == 0) put_lse(h, M, L);
  }
}

cudaError_t launch_pdl(const void *f, const PagedAttnParams &p, int grid, int threads, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *args[] = {const_cast<PagedAttnParams *>(&p)};
  return cudaLaunchKernelExC(&cfg, f, args);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedAttnParams &p, bool e4m3, bool shared, int grid, cudaStream_t s) {
  const void *f = e4m3 ? (shared ? (const void *)paged_attn_kernel<true, false, true>
                                 : (const void *)paged_attn_kernel<true, false, false>)
                       : (shared ? (const void *)paged_attn_kernel<false, false, true>
                                 : (const void *)paged_attn_kernel<false, false, false>);
  return launch_pdl(f, p, grid, kThreads, kPagedSmem, s);
}

// By the slots a sequence has on average, (CTAs + sequences) / sequences: four
// at most, a warp per head; up to twenty, a block per head; more, four.
cudaError_t launch_paged_merge(const PagedAttnParams &p, cudaStream_t s) {
  if (p.n_seq <= 8) return launch_pdl((const void *)paged_merge_kernel<1, 8, 1>, p, p.n_seq * kH * 4, 256, 0, s);
  if (p.n_seq < 48) return launch_pdl((const void *)paged_merge_kernel<4, 4, 1>, p, p.n_seq * kH, 128, 0, s);
  return launch_pdl((const void *)paged_merge_kernel<4, 4, 4>, p, p.n_seq * kH / 4, 128, 0, s);
}

cudaError_t launch_paged_weights(const PagedAttnParams &p, bool e4m3, int grid, cudaStream_t s) {
  return launch_pdl(e4m3 ? (const void *)paged_attn_kernel<true, true, false>
                         : (const void *)paged_attn_kernel<false, true, false>,
                    p, grid, kThreads, kPagedSmem, s);
}

cudaError_t prepare_paged_kernels() {
  for (const void *f :
       {(const void *)paged_attn_kernel<false, false, false>, (const void *)paged_attn_kernel<true, false, false>,
        (const void *)paged_attn_kernel<false, false, true>, (const void *)paged_attn_kernel<true, false, true>,
        (const void *)paged_attn_kernel<false, true, false>, (const void *)paged_attn_kernel<true, true, false>}) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPagedSmem);
    if (e != cudaSuccess) return e;
  }
  for (const void *f : {(const void *)paged_merge_kernel<1, 8, 1>, (const void *)paged_merge_kernel<4, 4, 1>,
                        (const void *)paged_merge_kernel<4, 4, 4>}) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ds4a
