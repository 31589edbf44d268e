// Attention of several new tokens per sequence over a paged K/V cache
// (tcgen05 + TMEM, two SMs to a product).
//
//   o[t][h] = sum_j softmax_j(scale q[t][h].k_j) v_j over the cached raw rows of
//             token t's window, the rows of t and its ancestors, and the
//             compressed rows whose span has ended
//
// (64 query heads over one K/V row of 512; "DwarfStar 4 (DS4) - DeepSeek V4 Flash
// Inference Engine", "Fixed Model Shape" and "Layer Compression".)
//
// Why two tokens and two SMs.  A product of one token's 64 heads with 128 rows
// reads 6 KB of operands from shared memory for 48 cycles' work that the tensor
// core could do in 32: shared memory bounds it, and the rows have to come in for
// each token anew.  Two CTAs of a cluster hold a token each and run every product
// as one MMA of M = 128 (2 x 64 heads) and N = 256 at the full rate (64 cycles for 16
// dims, 4096 multiply-adds per SM and cycle; measured), each SM bringing half of the
// rows' operand:
//   S[2 x 64 heads][256 rows]  = Q . K_tile^T     a CTA has rows 128c .. 128c+127 of K
//   O[2 x 64 heads][512 dims] += P . V_tile       and dims 128c .. +127 of each 256 of V
// so a row's K and V enter each SM half, and serve two tokens.  In such an MMA a CTA
// has its own 64 rows of D, N's lower half in TMEM lanes 0-63 and its upper half
// in lanes 64-127 (checked element by element on a GB300).  O takes 256 columns
// and S two buffers of 128; one score row lies in two lanes, so the softmax needs
// neither the other CTA nor exchanges between lanes but for a head's maximum.
//
// Work.  A unit is a pair of neighbouring tokens of a sequence.  The rows that
// either sees (compressed, cached raw, new) form a list, cut into tiles of 256.
// The tiles of all units are numbered through, and each cluster takes the same
// number of them in a row: whole units, and parts of the first and the last.  A
// part leaves its normalised output (fp32) and (m, l) in one of its cluster's two
// slots; a merge joins them.  Lengths are only known on the device: a small kernel
// counts the tiles first and writes down what each unit sees.
//
// Rows are found through the page tables.  Where all pages are whole grains of 8 or
// 16 rows, TMA brings K by grains and V by the grains of which every row is seen (in
// runs of up to 64 rows where a tile is seen in full); other rows of V, and all rows
// of other page sizes, are copied one by one, zeros in place of those that neither
// token sees.  What one of the two sees is masked for the other.  (Where the pages of
// either segment are no multiple of 8 rows, all rows of both are copied one by one: 2.2 to
// 2.7 times as long for trees and short lists, 3.3 times for 2,048 tokens over 7,680 rows.)
//
// What bounds it (GB300; the rates are this card's own, a cuBLAS product of bf16 at
// 1,878 TFLOP/s, at 1,702 where it runs for seconds under the power cap).  2,048 new
// tokens over 7,680 compressed rows: 1,320 us, 1,640 TFLOP/s, and 1,500 us under the
// power cap (clocks fall from 2,070 to 1,630 MHz).  A tile takes 6,200 cycles, of
// which the tensor core works 4,096, shared memory 5,100, and the warp that issues
// Q . K with its three stages all 6,200 (690 a part).  E4M3 rows: 9,100 cycles, 7,250 of
// them shared memory (each row is read as codes and written as values again); a slot
// of codes comes round in 3,300 and there is room for three.  Short lists (2,900
// tokens of 330 rows each in two tiles): 211 us; a tile takes 11,000 cycles, because
// an item's output has to leave TMEM before the next one's products, all clusters' at
// once (9.7 MB).  Few tokens (8 over 386 rows): 22.8 us, two launches and their round trips.
#include "attn_params.h"
#include "internal.h"
#include "ptx.cuh"
#include "ptx_async.cuh"
#include "step_params.h"

namespace ds4a {

namespace {

constexpr int kRows = 256;                  // of a tile
// A stage (a tile has 8 of K, 8 of V): 64 dims of 128 K rows, or 128 dims of 64 V rows.
constexpr uint32_t kPart = 16384;
constexpr uint32_t kCodePart = kPart / 2;
constexpr uint32_t kOffTP = kQBytes;        // P: 4 boxes [64 heads][64 rows]
constexpr uint32_t kPBox = 8192;
constexpr uint32_t kOffRing = kOffTP + 4 * kPBox;
constexpr uint32_t kRingBytes = 7 * kPart;
constexpr uint32_t kOffTMisc = kOffRing + kRingBytes;
constexpr uint32_t kTmemTS = 256;           // S buffers at columns 256 and 384
constexpr int kListsT = 3;

// K and V come through rings of their own, because their products are issued by
// warps of their own.  fp16 rows: three stages of K and four of V (four and three: 1,530
// against 1,449 us for 2,048 tokens when it was measured).  E4M3 rows: codes land in three
// slots for each and are widened into two stages for each (two slots and a third
// stage for K or V: 303 to 306 us against 301).
template <bool FP8>
constexpr int kKStages = FP8 ? 2 : 3;
template <bool FP8>
constexpr int kVStages = FP8 ? 2 : 4;
constexpr int kCodeSlots = 3;
static_assert(7 * kPart <= kRingBytes && 4 * kPart + 2 * kCodeSlots * kCodePart <= kRingBytes, "shared memory of the rings");
// Warps 0-7 softmax and epilogue; 13 finds the rows of the tiles; 12 and 14 issue P . V,
// a half of each 256 dims each, and 15 Q . K (in the CTA of rank 1 they report what has
// landed).  8-9 load K and 16-19 V (E4M3: 8 loads K and 11 V, 9-10 widen K and 16-19 V);
// 10-11 are idle with fp16 rows, because registers go to four warps at a time.  Every
// role is a loop over the tiles that meets the others at mbarriers only, and its code is
// kept small: what all roles run through in a tile has to stay in the instruction cache
// (128 KB on an SM).  What the numbers of warps are worth: two
// that issue P . V instead of one 1,446 -> 1,355 us (2,048 tokens), a third for K 1,449 ->
// 1,480; four that load V instead of two 329 -> 276 us (short lists); four that widen V
// instead of one 326 -> 301 us (E4M3).
constexpr int kTreeThreads = 640;
constexpr int kKLoadWarp0 = 8, kPvWarp1 = 12, kListWarp = 13, kPvWarp0 = 14, kQkWarp = 15;
constexpr int kWidenK0 = 9, kWidenV0 = 16, kWidenKWarps = 2, kWidenVWarps = 4;
template <bool FP8>
constexpr int kVLoadWarp0 = FP8 ? 11 : 16;
template <bool FP8>
constexpr int kKLoadWarps = FP8 ? 1 : 2;
template <bool FP8>
constexpr int kVLoadWarps = FP8 ? 1 : 4;

constexpr float kLeastLog2ScaleT = -40.f;  // V rows of a scale of 2^-40 or less count as 0: they round to 0 in fp16
constexpr unsigned long long kSegBitT = 1, kNoRowT = 2, kNoValue = 4;  // low bits of a list entry

// Of a tile within its item (the cluster's tiles of one unit); how its rows come; and
// from TF_PARTS on a bit for each 64 rows of which some token sees any.  (V's stages
// and products of the others are left out.)
enum : int { TF_FIRST = 1, TF_LAST = 2, TF_WHOLE = 4, TF_GATHERED = 8, TF_SPOILED = 16, TF_HEAD = 32, TF_FULL = 64 };
constexpr int TF_PARTS = 8;

enum : unsigned int {
  TSITE_Q_EMPTY = 0x80, TSITE_KV_EMPTY, TSITE_Q_FULL, TSITE_S_EMPTY, TSITE_KV_FULL, TSITE_P_FULL, TSITE_O_EMPTY,
  TSITE_S_FULL, TSITE_P_EMPTY, TSITE_O_FULL, TSITE_DRAIN, TSITE_CODE_FULL, TSITE_LIST_FULL, TSITE_LIST_EMPTY,
  TSITE_CODE_EMPTY
};

// What a cluster has to know of a unit, as 32 words (a warp reads one a lane).
struct UnitRec {
  int seq, t0, tiles, before;        // sequence, first token, tiles, tiles of all units before
  int nc, raw_at, raw0, len, n_raw;  // the list (UnitRows)
  int tok, two;                      // first token counted over all sequences; whether there is a second
  int nc_of[2], ra[2], rb[2];        // what either token sees: compressed rows below nc_of, cached rows ra .. rb - 1,
  int da[2], db[2];                  // new rows da .. db - 1 of a run,
  uint32_t anc[2][4];                // and of a tree those with a bit set
  int pad[3];
};
static_assert(sizeof(UnitRec) == 128, "a word per lane");

struct TMisc {
  alignas(16) unsigned long long row[kListsT][kRows];  // K address | bits (of gathered tiles)
  alignas(16) float ksc[kListsT][kRows];               // E4M3: scale * log2(e) * K scale
  alignas(16) float lvs[kListsT][kRows];               // E4M3: log2 of the V scale (of 2^-40 at least)
  alignas(16) float ivs[kListsT][kRows];               // E4M3: 2^-lvs
  int2 box[kListsT][kRows / 8];                        // (page, 2 * slot + segment) of the tile's grains
  uint32_t held[kListsT], live[kListsT];               // grains that have a page; whose rows all are seen by some token
  uint32_t mask[kListsT][kRows / 32];                  // rows that this CTA's token sees
  int flags[kListsT], tok[kListsT], q_tok[kListsT];    // TF_ bits; this CTA's token (-1: none); the one whose Q it loads
  alignas(16) float red[4][kH];
  alignas(8) uint64_t q_full, q_empty, peer_q_full;
  uint64_t kv_full[7], kv_empty[7];  // K's stages, then V's (rank 0's kv_full: of both CTAs)
  uint64_t code_full[2 * kCodeSlots], code_empty[2 * kCodeSlots];
  uint64_t list_full[kListsT], list_empty[kListsT];
  uint64_t s_full[2], s_empty[2], o_full[2];
  uint64_t p_full[4], p_empty[4], o_empty, mma_done;  // (P: by boxes of 64 rows)
  WaitBox wait;
  UnitRec unit;   // of the tile that is listed
  uint8_t odd_row[kRows];  // its rows that one token sees and the other does not
  uint32_t tmem_base;
};
constexpr uint32_t kTreeSmem = kOffTMisc + ((sizeof(TMisc) + 127) / 128) * 128 + 1024;
static_assert(kTreeSmem <= 232448, "shared memory of one CTA");

template <int N>
struct Ring {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void advance() {
    if (++st == N) {
      st = 0;
      ph ^= 1;
    }
  }
};

// ------------------------------------------------------------------ units

struct Span2 {
  int at, n;
};
__device__ __forceinline__ Span2 tokens_of(const TreeAttnParams &p, int b) {
  const int at = min(max(p.first[b], 0), p.n_tok);
  return Span2{at, min(max(p.first[b + 1], at), p.n_tok) - at};
}

// The rows that a unit's tokens t0 .. t1 see, as a list: compressed rows [0, nc), and
// from place raw_at on the raw rows raw0 .. (cached ones, then new ones, which follow
// them in the table).  raw_at and raw0 are whole grains, so that a grain of the list is
// one of a page.  (Of a tree, what any of its nodes could see: their depths are not
// known here.)
struct UnitRows {
  int nc, raw_at, raw0, len, n_raw;
  __device__ __forceinline__ int tiles() const { return max(1, (len + kRows - 1) / kRows); }
};

__device__ __forceinline__ UnitRows unit_rows(const TreeAttnParams &p, int4 g, int n, int t0, int t1) {
  const bool chain = p.parent == nullptr;
  const long long pos = max(g.x, 0), raw_pos0 = max(g.z, 0);
  const int n_comp = min(max(g.w, 0), p.seg[1].max_rows), grain = max(p.grain, 1);
  UnitRows r;
  r.n_raw = min(max(g.y, 0), p.seg[0].max_rows);
  r.nc = r.raw_at = r.raw0 = r.len = 0;
  if (!chain && t0 >= kTreeTokens) return r;  // nodes that see nothing
  const long long lo = chain ? pos + t0 : pos, hi = chain ? pos + t1 : pos + min(n, kTreeTokens) - 1;
  r.nc = (int)min((unsigned)n_comp, (unsigned)(hi + 1) / (unsigned)p.ratio);
  r.len = r.raw_at = (r.nc + grain - 1) / grain * grain;
  const int r0 = (int)min(max(lo - p.window + 1 - raw_pos0, 0ll), (long long)r.n_raw);
  const int r1 = (int)min(max(hi + 1 - raw_pos0, (long long)r0), (long long)r.n_raw);
  const int d1 = min(t1 + 1, p.seg[0].max_rows - r.n_raw), d0 = chain ? min(max(0, t0 - p.window + 1), d1) : 0;
  const int from = r1 > r0 ? r0 : r.n_raw + d0, to = d1 > d0 ? r.n_raw + d1 : r1;
  if (to > from) {
    r.raw0 = from / grain * grain;
    r.len += to - r.raw0;
  }
  return r;
}

// ------------------------------------------------------------------ plan

constexpr int kPlanThreads = 1024;

// Inclusive sum over the block; `all`: of all threads.  Two barriers.
__device__ __forceinline__ int block_scan(int v, int *warp_sum, int &all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  const int w = warp_sum[lane];
  all = __reduce_add_sync(0xffffffffu, w);
  v += __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  __syncthreads();
  return v;
}

__device__ __forceinline__ void unit_record(const TreeAttnParams &p, int seq, Span2 s, int4 g, int t0,
                                            const UnitRows &rows, UnitRec &r) {
  const bool chain = p.parent == nullptr;
  const int t1 = min(t0 + 1, s.n - 1);
  const long long pos = max(g.x, 0), raw_pos0 = max(g.z, 0);
  r.seq = seq;
  r.t0 = t0;
  r.tiles = rows.tiles();
  r.nc = rows.nc;
  r.raw_at = rows.raw_at;
  r.raw0 = rows.raw0;
  r.len = rows.len;
  r.n_raw = rows.n_raw;
  r.tok = s.at + t0;
  r.two = t1 > t0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = i == 0 ? t0 : t1;
    r.nc_of[i] = r.ra[i] = r.rb[i] = r.da[i] = r.db[i] = 0;
    r.anc[i][0] = r.anc[i][1] = r.anc[i][2] = r.anc[i][3] = 0;
    if (!chain && t0 >= kTreeTokens) continue;  // nodes that see nothing
    int depth = 0;
    if (chain) {
      depth = t;
      r.da[i] = max(0, t - p.window + 1);
      r.db[i] = t + 1;
    } else {
      for (int at = t;; ++depth) {  // up to the root, each step to an earlier node
        if (depth < p.window) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (at >> 5 == k) r.anc[i][k] |= 1u << (at & 31);
        }
        const int up = p.parent[s.at + at];
        if (up < 0 || up >= at) break;
        at = up;
      }
    }
    const long long at_pos = pos + depth;
    r.nc_of[i] = (int)min((unsigned)rows.nc, (unsigned)(at_pos + 1) / (unsigned)p.ratio);
    r.ra[i] = (int)min(max(at_pos - p.window + 1 - raw_pos0, 0ll), (long long)rows.n_raw);
    r.rb[i] = (int)min(max(at_pos + 1 - raw_pos0, 0ll), (long long)rows.n_raw);
  }
}

// Every block counts all tiles, which is quick, and writes the records of its share of
// the units, which is not (a tree's nodes climb to their roots): in one block, 1,470
// units took 31 us.
constexpr int kPlanUnits = 32;  // of a block, at least
constexpr int kPlanBlocks = 32;

__global__ void __launch_bounds__(kPlanThreads, 1) tree_plan_kernel(const TreeAttnParams p) {
  __shared__ int warp_sum[32], near[kPlanThreads];
  const int tid = threadIdx.x;
  int *units_before = p.n_seq <= kPlanThreads ? near : p.ws_seq;  // of each sequence (all blocks write the same)
  UnitRec *recs = static_cast<UnitRec *>(p.ws_unit);
  grid_launch_dependents();
  grid_dependency_wait();
  int units = 0;  // of the sequences before
  for (int b0 = 0; b0 < p.n_seq; b0 += kPlanThreads) {
    const int b = b0 + tid, n = b < p.n_seq ? (tokens_of(p, b).n + 1) / 2 : 0;
    int all;
    const int inc = block_scan(n, warp_sum, all);
    if (b < p.n_seq) units_before[b] = units + inc - n;
    units = min(units + all, 1 << 30);  // (only ranges that overlap name as many)
  }
  units = min(units, p.max_units);  // more than there is room for
  __syncthreads();
  const int share = (units + (int)gridDim.x - 1) / (int)gridDim.x, u_lo = (int)blockIdx.x * share;
  const int u_hi = min(u_lo + share, units);
  int tiles = 0, at = 0, n = 0;
  for (int u0 = 0; u0 < units; u0 += kPlanThreads) {
    const int u = u0 + tid;
    int here = 0, seq = 0, t0 = 0;
    Span2 toks = {0, 0};
    int4 g = make_int4(0, 0, 0, 0);
    UnitRows rows = {0, 0, 0, 0, 0};
    if (u < units) {
      int hi = p.n_seq;  // the last sequence whose units begin at or before u
      while (hi - seq > 1) {
        const int mid = (seq + hi) / 2;
        if (units_before[mid] <= u) seq = mid; else hi = mid;
      }
      t0 = 2 * (u - units_before[seq]);
      toks = tokens_of(p, seq);
      g = p.geom[seq];
      rows = unit_rows(p, g, toks.n, t0, min(t0 + 1, toks.n - 1));
      here = rows.tiles();
    }
    int all;
    const int inc = block_scan(here, warp_sum, all);
    if (u >= u_lo && u < u_hi) {
      UnitRec rec;
      unit_record(p, seq, toks, g, t0, rows, rec);
      rec.before = at = tiles + inc - here;
      n = here;
      rec.pad[0] = rec.pad[1] = rec.pad[2] = 0;
      recs[u] = rec;
    }
    tiles += all;
  }
  const int per = max(1, (tiles + p.clusters - 1) / p.clusters);
  if (blockIdx.x == 0 && tid == 0) p.ws_head[0] = make_int4(tiles, per, units, 0);
  __syncthreads();
  // The unit of each cluster's first tile.
  for (int u = tid; u < u_hi; u += kPlanThreads) {
    if (u < u_lo) continue;
    if (share > kPlanThreads) {  // (else this thread's only unit)
      at = recs[u].before;
      n = recs[u].tiles;
    }
    for (int i = (at + per - 1) / per; (long long)i * per < at + n; ++i) p.ws_start[i] = u;
  }
}

// Few sequences and units (one a lane of a warp): every CTA of the attention plans for
// itself, which is a launch less (8 tokens of one sequence: 23.4 us with the kernel above,
// 22.8 with this).  All write the same numbers to the workspace, each reads its own.
// (Not inlined: where its code lay among the roles', E4M3 rows took 277 us, not 270.)
__host__ __device__ __forceinline__ bool plans_itself(const TreeAttnParams &p) { return p.n_seq <= 32 && p.max_units <= 32; }

static __device__ __noinline__ void plan_by_warp(const TreeAttnParams &p, int lane) {
  auto sum_to = [&](int v) {  // over the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    return v;
  };
  const int ends = sum_to(lane < p.n_seq ? (tokens_of(p, lane).n + 1) / 2 : 0);  // units up to this sequence's last
  const int units = min(__shfl_sync(0xffffffffu, ends, 31), p.max_units);
  int seq = 0;  // the first whose units end behind this lane's
#pragma unroll
  for (int step = 16; step > 0; step >>= 1)
    if (__shfl_sync(0xffffffffu, ends, seq + step - 1) <= lane) seq += step;
  const int before = __shfl_sync(0xffffffffu, ends, max(seq - 1, 0));
  UnitRec rec;
  rec.tiles = 0;
  if (lane < units) {
    const Span2 toks = tokens_of(p, seq);
    const int4 g = p.geom[seq];
    const int t0 = 2 * (lane - (seq > 0 ? before : 0));
    unit_record(p, seq, toks, g, t0, unit_rows(p, g, toks.n, t0, min(t0 + 1, toks.n - 1)), rec);
  }
  const int end = sum_to(rec.tiles), tiles = __shfl_sync(0xffffffffu, end, 31);
  const int per = max(1, (tiles + p.clusters - 1) / p.clusters);
  if (lane < units) {
    rec.before = end - rec.tiles;
    rec.pad[0] = rec.pad[1] = rec.pad[2] = 0;
    static_cast<UnitRec *>(p.ws_unit)[lane] = rec;
    for (int i = (rec.before + per - 1) / per; (long long)i * per < end; ++i) p.ws_start[i] = lane;
  }
  if (lane == 0) p.ws_head[0] = make_int4(tiles, per, units, 0);
}

// ------------------------------------------------------------------ lists

// One warp goes ahead of all others and writes down, per tile, what is in it.  Where the
// pages allow TMA, a tile is a list of grains (8 or 16 rows, which one page holds): K
// comes by TMA wherever a grain has a page, since scores of rows that nobody sees are
// masked; V only where all rows of a grain are seen, and row by row elsewhere, zeros in
// place of the others.  Otherwise it is a list of the rows' addresses.
template <bool FP8>
__device__ __forceinline__ void tree_list_role(const TreeAttnParams &p, int nt, int cluster, uint32_t rank, TMisc &ms,
                                               int lane) {
  if (nt <= 0) return;
  const bool chain = p.parent == nullptr;
  const long long vdelta0 = p.seg[0].v - p.seg[0].k, vdelta1 = p.seg[1].v - p.seg[1].k;
  const int pad_seg = p.seg[1].max_rows > 0 ? 1 : 0;
  const unsigned long long pad_row = reinterpret_cast<unsigned long long>(p.seg[pad_seg].k) | pad_seg | kNoRowT;
  // Without grains every lane finds the pages of its own rows, as if each were one.
  const int grain = max(p.grain, 1), shift = p.grain > 0 ? p.grain_shift : 0;
  const int *recs = static_cast<const int *>(p.ws_unit);

  int u = p.ws_start[cluster], left = nt, j = 0, first_j = 0;
  int word = recs[32 * u + lane];  // of the unit that is entered next
  bool enter = true;
  UnitRec &r = ms.unit;
  const int32_t *table0 = nullptr, *table1 = nullptr;
  // Page and 2 * slot + segment of the list's place x (page -1: none).
  auto place = [&](int x) {
    int2 b = make_int2(-1, 0);
    if (x < r.len && (x < r.nc || x >= r.raw_at)) {
      const bool sg = x < r.raw_at;
      const int row = sg ? x : r.raw0 + (x - r.raw_at);
      const int s = sg ? p.seg[1].page_shift : p.seg[0].page_shift, per = sg ? p.seg[1].page_rows : p.seg[0].page_rows;
      const int pi = s >= 0 ? row >> s : row / per;
      b.x = (sg ? table1 : table0)[pi];
      b.y = 2 * (row - pi * per) + (sg ? 1 : 0);
      if ((unsigned)b.x >= (unsigned)(sg ? p.seg[1].n_pages : p.seg[0].n_pages)) b.x = -1;
    }
    return b;
  };
  auto address = [&](int2 b, int more) {  // of the K row `more` rows behind a place, with its segment's bit
    const bool sg = b.y & 1;
    return (reinterpret_cast<unsigned long long>(sg ? p.seg[1].k : p.seg[0].k) +
            b.x * (sg ? p.seg[1].page_stride : p.seg[0].page_stride) +
            ((b.y >> 1) + more) * (sg ? p.seg[1].row_stride : p.seg[0].row_stride)) |
           (sg ? kSegBitT : 0);
  };
  // Bits lo .. hi - 1 of a word (either may lie outside).
  auto range = [](int lo, int hi) -> unsigned {
    lo = max(lo, 0);
    hi = min(hi, 32);
    return lo < hi ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0;
  };
  // Which of places x .. x + 31 of the list token i sees.
  auto seen_word = [&](int i, int x) -> unsigned {
    const int to_row = r.raw0 - r.raw_at;  // from a place to a raw row
    unsigned m = range(-x, r.nc_of[i] - x);
    const int row = x + to_row;            // of the word's first bit, were it a raw one
    unsigned raw = range(r.ra[i] - row, r.rb[i] - row);
    const int d = r.n_raw - row;           // bit of the first new row
    if (chain) {
      raw |= range(r.da[i] + d, r.db[i] + d);
    } else if (d < 32 && d > -kTreeTokens) {
      // Bits d .. of the word are nodes 0 .. : two words of the ancestors, shifted.
      const int k = d >= 0 ? 0 : -d >> 5, off = d + 32 * k;  // 0 .. 31, or -31 .. 0
      const unsigned a0 = r.anc[i][k], a1 = k < 3 ? r.anc[i][k + 1] : 0;
      raw |= off >= 0 ? a0 << off : (a0 >> -off) | (a1 << (32 + off));
    }
    return m | (raw & range(r.raw_at - x, r.len - x));
  };
#pragma unroll 1
  for (int g = 0; g < nt; ++g) {
    const int buf = g % kListsT;
    if (enter) {
      __syncwarp();
      reinterpret_cast<int *>(&r)[lane] = word;
      __syncwarp();
      j = g == 0 ? cluster * p.ws_head[0].y - r.before : 0;
      if (left > r.tiles - j) word = recs[32 * (u + 1) + lane];
      table0 = p.seg[0].table + r.seq * p.seg[0].table_stride;
      table1 = p.seg[1].table + r.seq * p.seg[1].table_stride;
      enter = false;
    }
    const int base = j * kRows;
    // Compressed rows that both tokens see, in grains with pages: nothing to look through.
    bool full = p.grain > 0 && base + kRows <= min(r.nc_of[0], r.nc_of[1]), spoiled = false;
    int2 mine = make_int2(-1, 0);  // lane i: grain i
    unsigned held = 0, live = 0;
    if (p.grain > 0) {
      if (lane < kRows >> shift) mine = place(base + (lane << shift));
      held = __ballot_sync(0xffffffffu, mine.x >= 0);
      live = held;
      full = full && held == (kRows >> shift == 32 ? 0xffffffffu : (1u << (kRows >> shift)) - 1);
    }
    // Lane k: what either token sees of rows 32 k .. that have a page.
    unsigned see0 = 0xffffffffu, see1 = 0xffffffffu;
    if (!full && lane < kRows / 32) {
      unsigned there = 0xffffffffu;
      if (p.grain > 0) {
        there = 0;
#pragma unroll 1
        for (int k = 0; k < 32 >> shift; ++k)
          if ((held >> ((lane << (5 - shift)) + k)) & 1u) there |= ((1u << grain) - 1) << (k << shift);
      }
      see0 = seen_word(0, base + 32 * lane) & there;
      see1 = seen_word(1, base + 32 * lane) & there;
    }
    float ks[FP8 ? 8 : 1], vs[FP8 ? 8 : 1];
    if (FP8 && p.grain > 0) {
#pragma unroll
      for (int k = 0; k < (FP8 ? 8 : 1); ++k) {
        const int x = 32 * k + lane;
        const int page = __shfl_sync(0xffffffffu, mine.x, x >> shift), at = __shfl_sync(0xffffffffu, mine.y, x >> shift);
        const unsigned some = __shfl_sync(0xffffffffu, see0 | see1, k);
        ks[k] = 0.f;
        vs[k] = 1.f;
        if ((some >> lane) & 1u) {
          const bool sg = at & 1;
          const long long sr = (long long)page * (sg ? p.seg[1].page_rows : p.seg[0].page_rows) + (at >> 1) + (x & (grain - 1));
          ks[k] = (sg ? p.seg[1].k_scale : p.seg[0].k_scale)[sr];
          vs[k] = (sg ? p.seg[1].v_scale : p.seg[0].v_scale)[sr];
        }
      }
    }
    if (!__all_sync(0xffffffffu, wait_phase(smem_u32(&ms.list_empty[buf]), ((g / kListsT) & 1) ^ 1, TSITE_LIST_EMPTY,
                                            &ms.wait)))
      return;
    if (p.grain > 0) ms.box[buf][lane] = mine;
    if (p.grain == 0) {
      // Every row by itself.
#pragma unroll 1
      for (int k = 0; k < kRows / 32; ++k) {
        const int x = 32 * k + lane;
        const int2 b = place(base + x);
        const unsigned there = __ballot_sync(0xffffffffu, b.x >= 0);
        if (lane == k) {
          see0 &= there;
          see1 &= there;
        }
        const bool use = (__shfl_sync(0xffffffffu, see0 | see1, k) >> lane) & 1u;
        ms.row[buf][x] = use ? address(b, 0) : pad_row;
        if (FP8) {
          const bool sg = b.y & 1;
          const long long sr = (long long)b.x * (sg ? p.seg[1].page_rows : p.seg[0].page_rows) + (b.y >> 1);
          ms.ksc[buf][x] = use ? (sg ? p.seg[1].k_scale : p.seg[0].k_scale)[sr] : 0.f;
          ms.lvs[buf][x] = use ? (sg ? p.seg[1].v_scale : p.seg[0].v_scale)[sr] : 1.f;
        }
      }
    }
    if (lane < kRows / 32) ms.mask[buf][lane] = rank == 0 ? see0 : see1;
    unsigned parts = 15, bad_of = 0;  // rows whose V is left out of the product
    if (FP8) {
#pragma unroll
      for (int k = 0; k < (FP8 ? 8 : 1); ++k) {
        const float vv = p.grain > 0 ? vs[k] : ms.lvs[buf][32 * k + lane];
        const unsigned tiny = __ballot_sync(0xffffffffu, !(__log2f(vv) > kLeastLog2ScaleT));
        if (lane == k) bad_of = tiny;
        full = full && tiny == 0;
      }
    }
    if (!full) {
      const unsigned some = __ballot_sync(0xffffffffu, lane < kRows / 32 && (see0 | see1) != 0);
      parts = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) parts |= (some >> (2 * k)) & 3 ? 1u << k : 0;
      // A V row that one token sees and the other does not must be finite, because
      // its weight of 0 multiplies it all the same: the warp looks these few rows
      // through (new rows, edges of a window), eight lanes to a row.  One that is
      // not finite is left out of the product, and the token that sees it is marked.
      unsigned one = lane < kRows / 32 ? see0 ^ see1 : 0;
      int n_one = 0;
#pragma unroll 1
      for (unsigned words = __ballot_sync(0xffffffffu, one != 0); words != 0; words &= words - 1) {
        const int k = __ffs(words) - 1;
        const unsigned bits = __shfl_sync(0xffffffffu, one, k);
        if ((bits >> lane) & 1u) ms.odd_row[n_one + __popc(bits & ((1u << lane) - 1))] = (uint8_t)(32 * k + lane);
        n_one += __popc(bits);
      }
      __syncwarp();
#pragma unroll 1
      for (int i0 = 0; i0 < n_one; i0 += 4) {
        const int i = i0 + (lane >> 3), x = ms.odd_row[min(i, n_one - 1)];
        const unsigned long long e = p.grain > 0 ? address(ms.box[buf][x >> shift], x & (grain - 1)) : ms.row[buf][x];
        const uint4 *src = reinterpret_cast<const uint4 *>(e & ~15ull) + (lane & 7);
        src = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(src) + ((e & kSegBitT) ? vdelta1 : vdelta0));
        constexpr int kWords = FP8 ? 4 : 8;
        uint4 v[kWords];
#pragma unroll
        for (int w = 0; w < kWords; ++w) v[w] = src[8 * w];
        uint32_t odd = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const uint32_t y[4] = {v[w].x, v[w].y, v[w].z, v[w].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            odd |= FP8 ? ((y[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u   // a code of NaN: seven ones
                       : ((y[k] & 0x7C007C00u) + 0x04000400u) & 0x80008000u;  // an exponent of five ones
        }
        const unsigned who = __ballot_sync(0xffffffffu, odd != 0);
        if (who == 0) continue;
#pragma unroll 1
        for (int k = 0; k < 4 && i0 + k < n_one; ++k) {
          if (((who >> (8 * k)) & 255u) == 0) continue;
          const int y = ms.odd_row[i0 + k];
          if (lane == y >> 5) {
            bad_of |= 1u << (y & 31);
            spoiled = spoiled || (((rank == 0 ? see0 : see1) >> (y & 31)) & 1u) != 0;
          }
        }
      }
      spoiled = __any_sync(0xffffffffu, spoiled);
      if (p.grain > 0) {
        // Grains of which every row is seen and fit for the product; of the others the rows.
        const unsigned good = (see0 | see1) & ~bad_of;
        const unsigned bits = __shfl_sync(0xffffffffu, good, ((lane << shift) >> 5) & 7) >> ((lane << shift) & 31);
        const unsigned ones = (1u << grain) - 1, in_word = (1u << (32 >> shift)) - 1;
        live = __ballot_sync(0xffffffffu, mine.x >= 0 && lane < kRows >> shift && (bits & ones) == ones);
#pragma unroll 1
        for (int w = 0; w < kRows / 32; ++w) {
          if (((parts >> (w >> 1)) & 1u) == 0 || ((live >> (w << (5 - shift))) & in_word) == in_word) continue;
          const int x = 32 * w + lane;
          const bool use = (__shfl_sync(0xffffffffu, good, w) >> lane) & 1u;
          ms.row[buf][x] = use ? address(ms.box[buf][x >> shift], x & (grain - 1)) : pad_row;
        }
      } else {
#pragma unroll 1
        for (unsigned words = __ballot_sync(0xffffffffu, bad_of != 0); words != 0; words &= words - 1) {
          const int k = __ffs(words) - 1;
          if ((__shfl_sync(0xffffffffu, bad_of, k) >> lane) & 1u) ms.row[buf][32 * k + lane] |= kNoValue;
        }
      }
    }
    if (FP8) {
      uint32_t odd = 0;  // V scales that are not finite, by k
#pragma unroll
      for (int k = 0; k < (FP8 ? 8 : 1); ++k) {
        const int x = 32 * k + lane;
        const float kk = p.grain > 0 ? ks[k] : ms.ksc[buf][x], vv = p.grain > 0 ? vs[k] : ms.lvs[buf][x];
        odd |= (__float_as_uint(vv) & 0x7F800000u) == 0x7F800000u ? 1u << k : 0;
        ms.ksc[buf][x] = p.scale_log2 * kk;
        const float lv = fmaxf(__log2f(vv), kLeastLog2ScaleT);
        ms.lvs[buf][x] = lv;
        ms.ivs[buf][x] = exp2f(-lv);
      }
      if (__any_sync(0xffffffffu, odd != 0)) {
        // Such a row spoils who sees it; its weight counts all the same.
#pragma unroll 1
        for (int k = 0; k < kRows / 32; ++k) {
          const unsigned see = __shfl_sync(0xffffffffu, rank == 0 ? see0 : see1, k);
          if (((odd >> k) & 1u) == 0) continue;
          spoiled = spoiled || ((see >> lane) & 1u) != 0;
          ms.lvs[buf][32 * k + lane] = 0.f;
          ms.ivs[buf][32 * k + lane] = 1.f;
        }
        spoiled = __any_sync(0xffffffffu, spoiled);
      }
    }
    const bool head = g == 0 || j == 0, last = j == r.tiles - 1 || left == 1;
    if (head) first_j = j;
    if (lane == 0) {
      ms.held[buf] = held;
      ms.live[buf] = live;
      ms.flags[buf] = (head ? TF_FIRST : 0) | (last ? TF_LAST : 0) | (last && first_j == 0 && j == r.tiles - 1 ? TF_WHOLE : 0) |
                      (first_j == 0 ? TF_HEAD : 0) | (p.grain == 0 ? TF_GATHERED : 0) | (full ? TF_FULL : 0) |
                      (spoiled ? TF_SPOILED : 0) | (int)parts << TF_PARTS;
      ms.tok[buf] = rank == 0 ? r.tok : r.two ? r.tok + 1 : -1;
      ms.q_tok[buf] = rank == 0 || !r.two ? r.tok : r.tok + 1;
    }
    warp_arrive(smem_u32(&ms.list_full[buf]));
    --left;
    if (++j == r.tiles) {
      ++u;
      enter = true;
    }
  }
}

// ------------------------------------------------------------------ loaders

// The warps of K, or of V, load part after part into their ring: by TMA, a run or a
// grain per lane, or by 16-byte copies.  A warp stands some 600 cycles at a bulk copy,
// so the warps take the parts in turn, and nobody but a part's warp waits for its stage.
// (A parity tells a phase from the next one only.  Stages of K are freed in order, and
// a warp that waits for one has waited for another at most as many parts before as
// there are warps, fewer than stages.  V's halves are consumed by warps of their own,
// one up to a tile ahead of the other: there a stage is always the same warp's.)
template <bool FP8>
__device__ __forceinline__ void tree_load_role(const TreeAttnParams &p, int nt, uint32_t rank, uint32_t sbase, TMisc &ms,
                                               bool is_v, int tid) {
  if (nt <= 0) return;
  static_assert(kKLoadWarps<false> < kKStages<false> && kVLoadWarps<false> == kVStages<false> && kKLoadWarps<true> == 1 &&
                    kVLoadWarps<true> == 1,
                "whose turn a stage is");
  const int n_warps = is_v ? kVLoadWarps<FP8> : kKLoadWarps<FP8>;
  const int lane = tid & 31, warp = tid >> 5;
  const long long vdelta0 = p.seg[0].v - p.seg[0].k, vdelta1 = p.seg[1].v - p.seg[1].k;
  const uint32_t st0 = is_v ? (FP8 ? kCodeSlots : kKStages<false>) : 0;
  const uint32_t stages = FP8 ? kCodeSlots : is_v ? kVStages<false> : kKStages<false>;
  uint32_t at = 0, ph = 1, turn = 0;  // next stage of the ring and the parity to wait for; the warp whose turn is next
  uint32_t filled = 0, last_par = 0, n_item = 0;
  bool ok = true, q_issued = false;
#pragma unroll 1
  for (int g = 0; g < nt && ok; ++g) {
    const int buf = g % kListsT;
    if (!__all_sync(0xffffffffu, wait_phase(smem_u32(&ms.list_full[buf]), (g / kListsT) & 1, TSITE_LIST_FULL, &ms.wait))) break;
    const int flags = ms.flags[buf];
    if (!is_v && (flags & TF_FIRST)) {
      if (tid == 0) {
        if (!wait_phase(smem_u32(&ms.q_empty), (n_item & 1) ^ 1, TSITE_Q_EMPTY, &ms.wait)) {
          ok = false;
        } else {
          mbar_arrive_expect_tx(smem_u32(&ms.q_full), kQBytes);
          tma_load_4d(sbase, &p.tm_q, smem_u32(&ms.q_full), 0, 0, ms.q_tok[buf], 0);
          q_issued = true;
        }
      }
      ++n_item;
      if (__any_sync(0xffffffffu, !ok)) break;  // all lanes leave, or the votes below would miss one
    }
    // Grains that TMA brings (by runs of several where all are whole).
    const bool full = flags & TF_FULL, gathered = flags & TF_GATHERED;
    const uint32_t grains = is_v ? ms.live[buf] : ms.held[buf];
    const int shift = p.grain_shift, unit = full ? p.run_shift : shift;  // log2 of the rows of a copy
    const int rows = is_v ? 64 : 128;                                    // of a part
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      // Part c of K is dims 64 c .. of this CTA's rows; of V (kq, nb) dims 256 nb + 128 rank .. of rows 64 kq ..
      if (is_v && ((flags >> (TF_PARTS + (c >> 1))) & 1) == 0) continue;
      const bool mine = (int)turn == warp;
      const uint32_t st = st0 + at, par = ph;
      if ((int)++turn == n_warps) turn = 0;
      if (++at == stages) at = 0, ph ^= 1;
      if (!mine) continue;
      const int row0 = is_v ? 64 * (c >> 1) : 128 * (int)rank;
      const int dim0 = is_v ? 256 * (c & 1) + 128 * (int)rank : 64 * c;
      const uint32_t slot = sbase + kOffRing + (FP8 ? 4 * kPart + st * kCodePart : st * kPart);
      const uint32_t b_full = smem_u32(FP8 ? &ms.code_full[st] : &ms.kv_full[st]);
      if (!__all_sync(0xffffffffu, wait_phase(smem_u32(FP8 ? &ms.code_empty[st] : &ms.kv_empty[st]), par,
                                              FP8 ? TSITE_CODE_EMPTY : TSITE_KV_EMPTY, &ms.wait))) {
        ok = false;
        break;
      }
      // Grains of the part that TMA brings; of V, rows of the others are copied one by one.
      const uint32_t all = gathered ? 0 : 0xffffffffu >> (32 - (rows >> shift));
      const uint32_t here = gathered ? 0 : (grains >> (row0 >> shift)) & all;
      const bool by_rows = gathered || (is_v && here != all);
      if (!gathered) {
        // Rows that TMA brings here; fp16: the bytes of both CTAs count at rank 0's
        // barrier (of K, each has rows of its own), rank 1's has the issue only.
        if (lane == 0) {
          const uint32_t count = FP8 ? __popc(here) : is_v ? 2 * __popc(here) : __popc(grains);
          if (count != 0 && (FP8 || rank == 0))
            mbar_expect_tx(b_full, (count << shift) * (is_v ? 256u : 128u) / (FP8 ? 2u : 1u));
          if (!by_rows) mbar_arrive_cnt(b_full, 32);
        }
        const int row = lane << unit;  // within the part
        if (row < rows && ((here >> (row >> shift)) & 1u)) {
          const uint32_t dst = slot + row * (is_v ? (FP8 ? 128u : 256u) : (FP8 ? 64u : 128u));
          const int2 x = ms.box[buf][(row0 + row) >> shift];
          const CUtensorMap *m = full ? (is_v ? &p.tm_v : &p.tm_k)
                                      : (x.y & 1) ? (is_v ? &p.tm_vg[1] : &p.tm_kg[1]) : (is_v ? &p.tm_vg[0] : &p.tm_kg[0]);
          filled |= 1u << st;
          last_par = par ? last_par & ~(1u << st) : last_par | 1u << st;
          if (FP8)
            tma_load_3d(dst, m, b_full, dim0, x.y >> 1, x.x);
          else
            tma_load_5d_pair(dst, m, cluster_addr(b_full, 0), 0, 0, dim0 >> 6, x.y >> 4, x.x);
        }
        __syncwarp();
      }
      if (by_rows) {
        // 16-byte copies, eight lanes to a row (E4M3 codes of K: four), of the rows in
        // grains that TMA does not bring.
        const unsigned long long *list = ms.row[buf] + row0;
        auto src_of = [&](int row, int byte, uint32_t &bytes) {
          const unsigned long long e = list[row];
          const long long to_v = (e & kSegBitT) ? vdelta1 : vdelta0;
          bytes = (e & (is_v ? kNoRowT | kNoValue : kNoRowT)) ? 0u : 16u;
          return reinterpret_cast<const uint8_t *>(e & ~15ull) + (is_v ? to_v : 0) + byte;
        };
        // By eight rows, bit u: rows 8 u ..
        uint32_t todo = ~here & all;
        if (gathered) {
          todo = 0xffffffffu >> (32 - rows / 8);
        } else if (shift == 4) {  // 16 rows a grain
          todo = (todo | todo << 4) & 0x0f0f;
          todo = (todo | todo << 2) & 0x3333;
          todo = (todo | todo << 1) & 0x5555;
          todo |= todo << 1;
        }
        const int c8 = lane & 7;
#pragma unroll 1
        for (; todo != 0; todo &= todo - 1) {
          const int row = 8 * (__ffs(todo) - 1) + (lane >> 3);
          uint32_t n;
          if (FP8 && !is_v) {
            const int at_row = row - (lane >> 3) + (lane >> 2), byte = 16 * (lane & 3);
            const uint8_t *src = src_of(at_row, dim0 + byte, n);
            cp_async16z(slot + 64 * at_row + byte, src, n);
            continue;
          }
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            const uint8_t *src = src_of(row + k, (FP8 ? 1 : 2) * dim0 + 16 * c8, n);
            if (FP8) {
              cp_async16z(slot + 128 * (row + k) + 16 * c8, src, n);
              continue;
            }
            const int in8 = (row + k) & 7;
            const uint32_t dst = slot + (row >> 3) * (is_v ? 2048 : 1024) + in8 * 128 + ((c8 ^ in8) << 4);
            cp_async16z(dst, src, n);
            if (is_v) cp_async16z(dst + 1024, src + 128, n);
          }
        }
        cp_async_arrive(b_full);
      }
    }
    __syncwarp();
    if (ok) warp_arrive(smem_u32(&ms.list_empty[buf]));
  }
  // No copy may still be landing at exit.  (When every wait succeeded the MMA
  // warps have seen all stages land.)
  cp_async_done();
  if (ms.wait.abort_flag != 0) {
    volatile int never = 0;
    for (int st = 0; st < 7; ++st)
      if (filled & (1u << st))
        mbar_wait(smem_u32(FP8 ? &ms.code_full[st] : &ms.kv_full[st]), (last_par >> st) & 1, &never, 100000000ull,
                  p.err, TSITE_DRAIN);
    if (q_issued) mbar_wait(smem_u32(&ms.q_full), (n_item & 1) ^ 1, &never, 100000000ull, p.err, TSITE_DRAIN);
  }
}

// With E4M3 rows: a slot's codes widened exactly into the next stage, in the layout
// that the fp16 kernel's copies have.  A thread takes 16 codes at a time, at addresses
// that differ by constants; eight neighbouring threads meet every bank once, in codes
// and in values.
template <bool IS_V>
__device__ __forceinline__ void tree_widen_role(int nt, uint32_t sbase, TMisc &ms, int ct) {
  constexpr uint32_t kSlot0 = IS_V ? kCodeSlots : 0, kStage0 = IS_V ? kKStages<true> : 0;
  constexpr int kWarps = IS_V ? kWidenVWarps : kWidenKWarps, kTurns = 16 / kWarps;
  static_assert(kWidenVWarps % 2 == 0, "a turn is whole groups of eight rows");
  // K: 4 threads to a row.  V: 8 threads to a row, of which the first four take the left
  // half in even rows and the right half in odd ones.
  const int row = IS_V ? 2 * (ct >> 4) + ((ct >> 2) & 1) : ct >> 2;
  const int c = IS_V ? (ct & 3) | ((((ct >> 2) ^ (ct >> 3)) & 1) << 2) : ct & 3;  // chunks 2 c, 2 c + 1 of 8 values
  const uint32_t from = row * (IS_V ? 128 : 64) + 16 * c;
  const uint32_t to = (row >> 3) * (IS_V ? 2048 : 1024) + (row & 7) * 128 + (IS_V ? (c >> 2) * 1024 : 0);
  const uint32_t col0 = ((2 * (c & 3)) ^ (row & 7)) << 4, col1 = ((2 * (c & 3) + 1) ^ (row & 7)) << 4;
  Ring<kCodeSlots> codes;
  Ring<kKStages<true>> ring;
  int parts = 15;
#pragma unroll 1
  for (int i = 0; i < 8 * nt; ++i) {
    if (IS_V && (i & 7) == 0) {
      const int g = i >> 3, buf = g % kListsT;
      if (!__all_sync(0xffffffffu, wait_phase(smem_u32(&ms.list_full[buf]), (g / kListsT) & 1, TSITE_LIST_FULL, &ms.wait)))
        return;
      parts = ms.flags[buf] >> TF_PARTS;
      warp_arrive(smem_u32(&ms.list_empty[buf]));
    }
    if (((parts >> ((i & 7) >> 1)) & 1) == 0) continue;
    const uint32_t src = sbase + kOffRing + 4 * kPart + (kSlot0 + codes.st) * kCodePart + from;
    const uint32_t dst = sbase + kOffRing + (kStage0 + ring.st) * kPart + to;
    if (!__all_sync(0xffffffffu, wait_phase(smem_u32(&ms.code_full[kSlot0 + codes.st]), codes.ph, TSITE_CODE_FULL, &ms.wait) &&
                                     wait_phase(smem_u32(&ms.kv_empty[kStage0 + ring.st]), ring.ph ^ 1, TSITE_KV_EMPTY, &ms.wait)))
      return;
    uint4 raw[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(raw[k].x), "=r"(raw[k].y), "=r"(raw[k].z), "=r"(raw[k].w)
                   : "r"(src + k * 512 * kWarps));
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const uint32_t w4[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[2 * e] = e4m3x2_to_f16x2(static_cast<uint16_t>(w4[e] & 0xFFFFu));
        h[2 * e + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w4[e] >> 16));
      }
      sts_v4(dst + k * 1024 * kWarps + col0, h[0], h[1], h[2], h[3]);
      sts_v4(dst + k * 1024 * kWarps + col1, h[4], h[5], h[6], h[7]);
    }
    warp_arrive(smem_u32(&ms.code_empty[kSlot0 + codes.st]));
    if ((ct & 31) == 0) mbar_arrive(smem_u32(&ms.kv_full[kStage0 + ring.st]));
    codes.advance();
    ring.advance();
  }
}

// ------------------------------------------------------------------ MMA issue and relay

// The CTA of rank 1 has no MMA to issue: these warps (one lane) tell the other CTA
// what has landed here, stage by stage.  Gathered and widened rows are generic-proxy
// writes: the fence makes them visible to the tensor core before the news goes out.
template <bool FP8>
__device__ __forceinline__ void tree_relay_role(int nt, TMisc &ms, bool is_v, uint32_t half) {
  const uint32_t stage0 = is_v ? kKStages<FP8> : 0, stages = is_v ? kVStages<FP8> : kKStages<FP8>, step = is_v ? 2 : 1;
  uint32_t st = half, ph = 0, item = 0;
#pragma unroll 1
  for (int g = 0; g < nt; ++g) {
    const int buf = g % kListsT;
    if (!wait_phase(smem_u32(&ms.list_full[buf]), (g / kListsT) & 1, TSITE_LIST_FULL, &ms.wait)) return;
    const int flags = ms.flags[buf];
    mbar_arrive(smem_u32(&ms.list_empty[buf]));
    if (!is_v && (flags & TF_FIRST)) {
      if (!wait_phase(smem_u32(&ms.q_full), item & 1, TSITE_Q_FULL, &ms.wait)) return;
      mbar_arrive_cluster(cluster_addr(smem_u32(&ms.peer_q_full), 0));
      ++item;
    }
#pragma unroll 1
    for (uint32_t c = half; c < 8; c += step) {
      if (is_v && ((flags >> (TF_PARTS + (c >> 1))) & 1) == 0) continue;
      const uint32_t bar = smem_u32(&ms.kv_full[stage0 + st]);
      if (!wait_phase(bar, ph, TSITE_KV_FULL, &ms.wait)) return;
      fence_proxy_async_smem();
      mbar_arrive_cluster(cluster_addr(bar, 0));
      if ((st += step) >= stages) st = half, ph ^= 1;
    }
  }
}

// Three warps issue, Q . K and the halves of P . V, each from its own stages: the wait for
// a stage, the issue and the commits take a warp some 650 cycles a part, its MMAs 256.
// (The halves go to columns of their own, so that their order does not matter; all parts
// of Q . K go into one sum.)  The whole warp walks the tiles, so that
// descriptors are warp-uniform values, and one elected lane issues.  Waits are
// joined over the warp: all lanes go on or none.
template <bool FP8, bool IS_V>
__device__ __forceinline__ void tree_mma_role(int nt, uint32_t sbase, uint32_t tmem, TMisc &ms, uint32_t half) {
  constexpr uint32_t kIdesc = idesc_f16_f32(128, 256, false, IS_V);
  constexpr int kStage0 = IS_V ? kKStages<FP8> : 0;
  // Q, K and P: K-major.  V: MN-major, LBO = distance of the 64-dim blocks, SBO =
  // distance of 8-row groups.
  const uint64_t a_desc = IS_V ? sdesc_sw128(sbase + kOffTP, 16, 1024) : sdesc_sw128(sbase, 16, 1024);
  const uint64_t b_desc = IS_V ? sdesc_sw128(sbase + kOffRing + kStage0 * kPart, 1024, 2048)
                               : sdesc_sw128(sbase + kOffRing, 16, 1024);
  constexpr uint32_t kStages = IS_V ? kVStages<FP8> : kKStages<FP8>, kStep = IS_V ? 2 : 1;
  static_assert(kVStages<FP8> % 2 == 0, "a stage of V is always the same half's");
  uint32_t st = half, ph = 0, item = 0;
  bool ready = false;  // the next stage had landed when it was asked for
  bool empty = true;   // no product has gone into this item's O
  auto wait = [&](uint64_t &bar, uint32_t parity, uint32_t site) -> bool {
    return __all_sync(0xffffffffu, wait_phase(smem_u32(&bar), parity, site, &ms.wait));
  };
#pragma unroll 1
  for (int g = 0; g < nt; ++g) {
    const int buf = g % kListsT;
    if (!wait(ms.list_full[buf], (g / kListsT) & 1, TSITE_LIST_FULL)) return;
    const int flags = ms.flags[buf];
    warp_arrive(smem_u32(&ms.list_empty[buf]));
    const bool first = flags & TF_FIRST, last = flags & TF_LAST, fence = FP8 || !(flags & TF_FULL);
    const int parts = IS_V ? flags >> TF_PARTS : 15, lowest = __ffs(parts) - 1;
    const uint32_t sb = g & 1;
    if (IS_V) {
      if (first && !wait(ms.o_empty, (item & 1) ^ 1, TSITE_O_EMPTY)) return;
    } else {
      if (first && (!wait(ms.q_full, item & 1, TSITE_Q_FULL) || !wait(ms.peer_q_full, item & 1, TSITE_Q_FULL))) return;
      if (!wait(ms.s_empty[sb], ((g >> 1) & 1) ^ 1, TSITE_S_EMPTY)) return;
    }
    if (first) ++item;
    empty = empty || first;
    tc_fence_after();
#pragma unroll 1
    for (uint32_t c = half; c < 8; c += kStep) {
      // (Also of a box whose rows nobody sees: its barriers go through every tile.)
      if (IS_V && !wait(ms.p_full[c >> 1], g & 1, TSITE_P_FULL)) return;
      const bool live = !IS_V || ((parts >> (c >> 1)) & 1) != 0;
      const uint32_t at = st;
      if (live) {
        if (!__all_sync(0xffffffffu, ready) && !wait(ms.kv_full[kStage0 + st], ph, TSITE_KV_FULL)) return;
        if ((st += kStep) >= kStages) st = half, ph ^= 1;
        // The next stage is asked for before this one's products are issued.
        ready = mbar_test(smem_u32(&ms.kv_full[kStage0 + st]), ph);
        if (fence) fence_proxy_async_smem();
      }
      if (IS_V) tc_fence_after();
      const uint64_t a0 = sdesc_add(a_desc, (IS_V ? c >> 1 : c) * 8192);
      const uint64_t b0 = sdesc_add(b_desc, at * kPart);
      const uint32_t d = IS_V ? tmem + 128 * half : tmem + kTmemTS + 128 * sb;
      const bool fresh = IS_V ? empty && (int)(c >> 1) == lowest : c == 0;
      if (elect_lane()) {
        if (live) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            if (ks == 0)
              umma_pair_f16(d, a0, b0, kIdesc, fresh ? 0u : 1u);
            else
              umma_pair_f16_acc(d, sdesc_add(a0, ks * 32), sdesc_add(b0, ks * (IS_V ? 4096 : 32)), kIdesc);
          }
          umma_pair_commit(smem_u32(&ms.kv_empty[kStage0 + at]));
        }
        if (IS_V) {
          umma_pair_commit(smem_u32(&ms.p_empty[c >> 1]));
          if (c >= 6 && last) umma_pair_commit(smem_u32(&ms.o_full[half]));
        } else if (c == 7) {
          umma_pair_commit(smem_u32(&ms.s_full[sb]));
          if (last) umma_pair_commit(smem_u32(&ms.q_empty));
        }
      }
      __syncwarp();
    }
    if (parts != 0) empty = false;
  }
}

// ------------------------------------------------------------------ softmax and epilogue

// The reference of a head lies kLiftT below the largest score of the tile that
// set it, and moves only when a score passes it by kLiftT + kHoldT (the reasons
// and figures stand at paged_attn.cu's kLift): P is 2^15 at most.
constexpr float kLiftT = 10.f, kHoldT = 5.f;
constexpr float kNoRefT = -3e38f;

// This lane's 128 columns of TMEM, times inv (none: zeros), as fp16 (whole) or fp32 to
// the output: 128 bytes of every head at a time, turned in the warp's own rows of P,
// which is free then, so that eight lanes store a head's (`at`: the lane's first).
// (Stores of a head per lane: short lists took 229.6 us, so 211.6.)
__device__ __forceinline__ void take_output(uint32_t cols, uint32_t prow, float inv, bool none, bool whole, uint8_t *at) {
  int l = threadIdx.x & 31;
  asm volatile("" : "+r"(l), "+r"(prow), "+r"(cols));  // nothing of this is kept in registers from tile to tile
  const uint32_t wrow = prow - (l >> 3) * 1024 - (l & 7) * 128;  // of the warp's first head
  const int n = whole ? 4 : 2;                                   // times 16 dims in 128 bytes
#pragma unroll 1
  for (int c = 0; c < 8 / n; ++c) {
#pragma unroll 2
    for (int k = 0; k < n; ++k) {
      float o[16];
      tmem_ld16(cols + 16 * (n * c + k), o);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = none ? 0.f : o[i] * inv;
      if (whole) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 v = __floats2half2_rn(o[8 * i + 2 * e], o[8 * i + 2 * e + 1]);
            y[e] = *reinterpret_cast<const uint32_t *>(&v);
          }
          sts_v4(prow + (((2 * k + i) ^ (l & 7)) << 4), y[0], y[1], y[2], y[3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sts_v4(prow + (((4 * k + i) ^ (l & 7)) << 4), __float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
                 __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3]));
      }
    }
    __syncwarp();
    if (at != nullptr) {
      uint4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int in8 = 4 * (k & 1) + (l >> 3);  // row within eight heads
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[k].x), "=r"(x[k].y), "=r"(x[k].z), "=r"(x[k].w)
                     : "r"(wrow + (k >> 1) * 1024 + in8 * 128 + (((l & 7) ^ in8) << 4)));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4 *>(at + 128 * c + 16 * (l & 7) + k * 4 * kD * (whole ? 2 : 4)) = x[k];
    }
    __syncwarp();
  }
}

// Warp w: TMEM lanes 32 (w & 3) .., that is heads 32 (w & 1) .. and rows 128 of
// the tile's half (w >> 1) & 1, of which it has 64, by w >> 2.  A head's four
// threads are in four warps (a group, w & 1), which vote and meet by themselves.
template <bool FP8>
__device__ __forceinline__ void tree_softmax_role(const TreeAttnParams &p, int nt, int cluster, uint32_t rank,
                                                  uint8_t *smem, uint32_t tmem, TMisc &ms, int tid) {
  const int w = tid >> 5, l = tid & 31;
  const int q = w & 3, hh = w >> 2, half = q >> 1;
  const int h = 32 * (q & 1) + l, box = 2 * half + hh;
  const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
  const uint32_t group = 1 + (q & 1);
  auto tell = [&](uint64_t &bar) {  // one arrival per warp, at rank 0's barrier
    __syncwarp();
    if (l == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&bar), 0));
  };
  bool bad = false, spoiled = false;
  auto wait = [&](uint64_t &bar, uint32_t parity, uint32_t site) {
    bad = bad || !wait_phase(smem_u32(&bar), parity, site, &ms.wait);
    __syncwarp();
  };
  uint32_t n_item = 0;
  float m_ref = kNoRefT, m_lim = kNoRefT, lsum = 0.f;
  uint8_t *prow = smem + kOffTP + box * kPBox + (h >> 3) * 1024 + (h & 7) * 128;
  // The output of an item that has ended: this thread's 128 dims of o (dims 256 hh +
  // 128 half ..) once the last products have gone into them.
  bool pending = false, none = false, whole = false;
  float inv = 0.f;
  int out_tok = -1;
  int slot = 0;
  auto drain = [&](uint32_t tile) {  // ahead of this tile's P
    pending = false;
    wait(ms.o_full[hh], n_item & 1, TSITE_O_FULL);
    wait(ms.p_empty[box], (tile & 1) ^ 1, TSITE_P_EMPTY);
    ++n_item;
    tc_fence_after();
    const int dim0 = 256 * hh + 128 * half, row0 = 32 * (q & 1) + (l >> 3);
    uint8_t *at = nullptr;
    if (out_tok >= 0 && !bad)
      at = whole ? reinterpret_cast<uint8_t *>(p.o + out_tok * p.o_stride + (long long)row0 * kD + dim0)
                 : reinterpret_cast<uint8_t *>(p.ws_o + ((long long)slot * kH + row0) * kD + dim0);
    take_output(tmem + 128 * hh + lanes, smem_u32(prow), inv, none, whole, at);
    tc_fence_before();
    tell(ms.o_empty);
  };
#pragma unroll 1
  for (int g = 0; g < nt; ++g) {
    const int buf = g % kListsT;
    const uint32_t sb = g & 1, s_at = tmem + kTmemTS + 128 * sb + 64 * hh + lanes;
    wait(ms.list_full[buf], (g / kListsT) & 1, TSITE_LIST_FULL);
    const int flags = ms.flags[buf], tok = ms.tok[buf];
    const uint32_t see0 = ms.mask[buf][2 * box], see1 = ms.mask[buf][2 * box + 1];
    if (flags & TF_FIRST) {
      m_ref = m_lim = kNoRefT;
      lsum = 0.f;
      spoiled = false;
    }
    spoiled = spoiled || (flags & TF_SPOILED);
    if (!FP8) warp_arrive(smem_u32(&ms.list_empty[buf]));
    wait(ms.s_full[sb], (g >> 1) & 1, TSITE_S_FULL);
    tc_fence_after();
    float s[64];
    tmem_ld64(s_at, s);
    tmem_wait_ld();
    tc_fence_before();
    tell(ms.s_empty[sb]);
    if (FP8) {
      const float4 *ks = reinterpret_cast<const float4 *>(ms.ksc[buf] + 64 * box);
      const float4 *lv = reinterpret_cast<const float4 *>(ms.lvs[buf] + 64 * box);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float4 k = ks[c], v = lv[c];
        s[4 * c] = fmaf(s[4 * c], k.x, v.x);
        s[4 * c + 1] = fmaf(s[4 * c + 1], k.y, v.y);
        s[4 * c + 2] = fmaf(s[4 * c + 2], k.z, v.z);
        s[4 * c + 3] = fmaf(s[4 * c + 3], k.w, v.w);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 64; ++c) s[c] *= p.scale_log2;
    }
    if ((see0 & see1) != 0xFFFFFFFFu) {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        s[c] = (see0 >> c) & 1u ? s[c] : -INFINITY;
        s[c + 32] = (see1 >> c) & 1u ? s[c + 32] : -INFINITY;
      }
    }
    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int c = 4; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    bool moved = false;
    float alpha = 1.f;
    if (bar_red_or(group, 128, top > m_lim || bad)) {
      // Some head's reference moves: the tile's maximum over a head's four threads.
      ms.red[box][h] = top;
      if (bar_red_or(group, 128, bad)) break;
      const float tmax = fmaxf(fmaxf(ms.red[0][h], ms.red[1][h]), fmaxf(ms.red[2][h], ms.red[3][h]));
      if (tmax > m_lim) {
        // Rounded so that P stays within 2^15 where scores are 16 and more apart.
        const float next = __fsub_ru(tmax, kLiftT);
        alpha = exp2f(m_ref - next);  // 0 while there was none
        m_ref = next;
        m_lim = __fadd_rd(m_ref, kLiftT + kHoldT);
      }
      moved = true;
      lsum *= alpha;
    }
    // This head's 64 weights, rounded once to fp16, V's type, because both operands of a
    // product have one (2^-11 of each at most: outputs are 2.3e-4 to 2.9e-4 from those in 64
    // bits, 2.1e-4 of it their own rounding); the sums add them unrounded, sixteen at a
    // time, so that lse keeps fp32 precision over long rows.
    uint32_t weights[32];
    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float e0 = exp2f(s[2 * i] - m_ref), e1 = exp2f(s[2 * i + 1] - m_ref);
      const __half2 hp = __floats2half2_rn(e0, e1);
      if (FP8) {
        const float2 iv = *reinterpret_cast<const float2 *>(&ms.ivs[buf][64 * box + 2 * i]);
        part[i & 3] = fmaf(e0, iv.x, fmaf(e1, iv.y, part[i & 3]));  // (a V scale of 0: weight, but no value)
      } else {
        part[i & 3] += e0 + e1;
      }
      weights[i] = *reinterpret_cast<const uint32_t *>(&hp);
    }
    lsum += (part[0] + part[1]) + (part[2] + part[3]);
    if (FP8) warp_arrive(smem_u32(&ms.list_empty[buf]));
    if (pending) drain(g);
    if (moved && !(flags & TF_FIRST)) {
      // O under the new reference, once the products so far have gone into it (those
      // of the last box complete last), and before any of this tile does.
      wait(ms.p_empty[3], (g & 1) ^ 1, TSITE_P_EMPTY);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[32];
        tmem_ld32(tmem + 128 * hh + 32 * c + lanes, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= alpha;
        tmem_st32(tmem + 128 * hh + 32 * c + lanes, o);
      }
      tmem_wait_st();
      tc_fence_before();
      bar_sync_id(group, 128);
    }
    wait(ms.p_empty[box], (g & 1) ^ 1, TSITE_P_EMPTY);
    // 16-byte chunk c of the head's 128 bytes at c ^ (h & 7).
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint4 *>(prow + ((c ^ (h & 7)) << 4)) =
          make_uint4(weights[4 * c], weights[4 * c + 1], weights[4 * c + 2], weights[4 * c + 3]);
    fence_proxy_async_smem();
    tc_fence_before();
    tell(ms.p_full[box]);
    if (!(flags & TF_LAST)) continue;

    // End of an item: the sum over a head's four threads.  Its output is taken from
    // TMEM behind the next tile's weights, while the last products run.
    if (moved && (flags & TF_FIRST)) bar_sync_id(group, 128);  // the maxima have been read: nothing since then met
    ms.red[box][h] = lsum;
    if (bar_red_or(group, 128, bad)) break;
    const float sum = (ms.red[0][h] + ms.red[1][h]) + (ms.red[2][h] + ms.red[3][h]);
    // No weight at all: o = 0.  (A sum that is NaN is not that: it stays.)
    none = sum == 0.f;
    inv = spoiled ? __int_as_float(0x7FC00000) : none ? 0.f : 1.f / sum;
    whole = flags & TF_WHOLE;
    out_tok = tok;
    slot = 2 * (2 * cluster + (flags & TF_HEAD ? 1 : 0)) + rank;
    if (box == 0 && tok >= 0) {
      if (!whole)
        p.ws_ml[slot * kH + h] = make_float2(none ? -INFINITY : m_ref, sum);
      else if (p.lse != nullptr)
        p.lse[(long long)tok * kH + h] = none ? -INFINITY : (m_ref + log2f(sum)) * kLn2;
    }
    pending = true;
    bar_sync_id(group, 128);  // the sums have been read
  }
  // All or none: an output is taken in steps that need whole warps.
  if (pending && !bar_red_or(group, 128, bad)) drain(nt);
}

// ------------------------------------------------------------------ kernel

template <bool FP8>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_attn_kernel(const __grid_constant__ TreeAttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  TMisc &ms = *reinterpret_cast<TMisc *>(smem + kOffTMisc);
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&ms.q_full), 1);
    mbar_init(smem_u32(&ms.q_empty), 1);
    mbar_init(smem_u32(&ms.peer_q_full), 1);
    for (int s = 0; s < 7; ++s) {
      // The threads of the warp that loads, or the warps that widen; and the other CTA's report.
      const int widen = s < kKStages<true> ? kWidenKWarps : kWidenVWarps;
      mbar_init(smem_u32(&ms.kv_full[s]), (FP8 ? widen : 32) + (rank == 0 ? 1 : 0));
      mbar_init(smem_u32(&ms.kv_empty[s]), 1);
    }
    for (int s = 0; s < 2 * kCodeSlots; ++s) {
      mbar_init(smem_u32(&ms.code_full[s]), 32);
      mbar_init(smem_u32(&ms.code_empty[s]), s < kCodeSlots ? kWidenKWarps : kWidenVWarps);
    }
    for (int s = 0; s < kListsT; ++s) {
      mbar_init(smem_u32(&ms.list_full[s]), 1);
      // Softmax, the MMA warps, loaders and those that widen V.
      mbar_init(smem_u32(&ms.list_empty[s]), kComputeWarps + 3 + kKLoadWarps<FP8> + kVLoadWarps<FP8> +
                                                 (FP8 ? kWidenVWarps : 0));
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ms.s_full[s]), 1);
      mbar_init(smem_u32(&ms.s_empty[s]), 2 * kComputeWarps);
      mbar_init(smem_u32(&ms.o_full[s]), 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(smem_u32(&ms.p_full[s]), 2 * kComputeWarps / 4);
      mbar_init(smem_u32(&ms.p_empty[s]), 2);
    }
    mbar_init(smem_u32(&ms.o_empty), 2 * kComputeWarps);
    mbar_init(smem_u32(&ms.mma_done), 3);
    ms.wait.timeout_ns = p.timeout_ns;
    ms.wait.err = p.err;
    ms.wait.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_q);
    if (p.grain > 0 && p.seg[1].max_rows > 0) {
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
    }
  }
  if (warp == kQkWarp) tmem_alloc_pair(smem_u32(&ms.tmem_base), kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  grid_launch_dependents();
  grid_dependency_wait();  // the plan, or what the plan is made from
  if (plans_itself(p)) {
    if (warp == kListWarp) plan_by_warp(p, threadIdx.x & 31);
    __syncthreads();
  }
  const int4 head = p.ws_head[0];
  const long long before = (long long)cluster * head.y;
  const int nt = (int)max(0ll, min((long long)head.y, head.x - before));
  if (warp < kComputeWarps) {
    tree_softmax_role<FP8>(p, nt, cluster, rank, smem, tmem, ms, threadIdx.x);
  } else if (warp == kPvWarp0 || warp == kPvWarp1 || warp == kQkWarp) {
    const bool is_v = warp != kQkWarp, lane0 = (threadIdx.x & 31) == 0;
    const uint32_t half = warp == kPvWarp1 ? 1 : 0;
    if (rank == 0) {
      if (is_v)
        tree_mma_role<FP8, true>(nt, sbase, tmem, ms, half);
      else
        tree_mma_role<FP8, false>(nt, sbase, tmem, ms, 0);
      __syncwarp();
      if (elect_lane()) umma_pair_commit(smem_u32(&ms.mma_done));
    } else if (lane0) {
      tree_relay_role<FP8>(nt, ms, is_v, half);
    }
    __syncwarp();
    volatile int never = 0;
    mbar_wait(smem_u32(&ms.mma_done), 0, &never, 3 * p.timeout_ns, p.err, TSITE_DRAIN);
    __syncwarp();
  } else if (warp == kListWarp) {
    tree_list_role<FP8>(p, nt, cluster, rank, ms, threadIdx.x & 31);
  } else if (FP8 && warp >= kWidenV0) {
    tree_widen_role<true>(nt, sbase, ms, threadIdx.x - 32 * kWidenV0);
  } else if (FP8 && warp >= kWidenK0 && warp < kWidenK0 + kWidenKWarps) {
    tree_widen_role<false>(nt, sbase, ms, threadIdx.x - 32 * kWidenK0);
  } else if (warp < kKLoadWarp0 + kKLoadWarps<FP8> ||
             (warp >= kVLoadWarp0<FP8> && warp < kVLoadWarp0<FP8> + kVLoadWarps<FP8>)) {
    const bool is_v = warp >= kVLoadWarp0<FP8>;
    tree_load_role<FP8>(p, nt, rank, sbase, ms, is_v, threadIdx.x - 32 * (is_v ? kVLoadWarp0<FP8> : kKLoadWarp0));
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // neither CTA leaves while the other may still arrive here, or its MMAs read
  tc_fence_after();
  if (warp == kQkWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

// ------------------------------------------------------------------ merge
// A unit is cut where a cluster's tiles end: at most once per cluster.  Block
// (boundary, token, 8 heads): the first boundary inside a unit joins its parts,
// of the cluster it begins in (its second slot) and of those that follow (their
// first).  With M = max m_s and W_s = 2^(m_s - M) l_s:
//   o = sum_s W_s o_s / L,  L = sum_s W_s,  lse = (M + log2 L) ln 2.

constexpr int kMergeHeads = 8;
constexpr int kMergeAhead = 2;

__global__ void __launch_bounds__(32 * kMergeHeads) tree_merge_kernel(const TreeAttnParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int group = blockIdx.x % (kH / kMergeHeads), rest = blockIdx.x / (kH / kMergeHeads);
  const int i = rest & 1, edge = 1 + (rest >> 1), h = group * kMergeHeads + (threadIdx.x >> 5);
  const int4 head = p.ws_head[0];
  const int unit = p.ws_start[edge];  // (anything where there is no such tile)
  const long long at = (long long)edge * head.y;
  if (at >= head.x) return;
  const UnitRec &rec = static_cast<const UnitRec *>(p.ws_unit)[unit];
  const int before = rec.before;
  if (before >= at || at - before > head.y) return;  // no cut here, or not the unit's first
  if (i > rec.two) return;
  const int n = (before + rec.tiles - 1) / head.y - (edge - 1) + 1;  // parts
  auto slot = [&](int k) { return 2ll * (k == 0 ? 2 * (edge - 1) + 1 : 2 * (edge - 1 + k)) + i; };
  float M = -INFINITY, L = 0.f;
  float4 acc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < n; k0 += kMergeAhead) {
    float4 x[kMergeAhead][4];
    float2 ml[kMergeAhead];
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k) {
      const bool have = k0 + k < n;
      const long long sl = slot(have ? k0 + k : 0);
      ml[k] = have ? p.ws_ml[sl * kH + h] : make_float2(-INFINITY, 0.f);
      const float4 *src = reinterpret_cast<const float4 *>(p.ws_o + (sl * kH + h) * kD) + lane;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[k][e] = have ? __ldcs(src + 32 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k) top = fmaxf(top, ml[k].x);
    if (top == -INFINITY) continue;
    const float old = exp2f(M - top);
    M = top;
    L *= old;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = make_float4(acc[e].x * old, acc[e].y * old, acc[e].z * old, acc[e].w * old);
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k) {
      if (ml[k].y == 0.f) continue;  // a part that saw no row
      const float t_ = exp2f(ml[k].x - top) * ml[k].y;
      L += t_;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[e].x = fmaf(t_, x[k][e].x, acc[e].x);
        acc[e].y = fmaf(t_, x[k][e].y, acc[e].y);
        acc[e].z = fmaf(t_, x[k][e].z, acc[e].z);
        acc[e].w = fmaf(t_, x[k][e].w, acc[e].w);
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const long long tok = rec.tok + i;
  __half *o = p.o + tok * p.o_stride + (long long)h * kD;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 a = __floats2half2_rn(acc[e].x * inv, acc[e].y * inv), b = __floats2half2_rn(acc[e].z * inv, acc[e].w * inv);
    *reinterpret_cast<uint2 *>(o + 4 * (lane + 32 * e)) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  }
  if (lane == 0 && p.lse != nullptr) p.lse[tok * kH + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

cudaError_t launch(const void *f, const TreeAttnParams &p, int grid, int threads, size_t smem, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  void *args[] = {const_cast<TreeAttnParams *>(&p)};
  return cudaLaunchKernelExC(&cfg, f, args);
}

}  // namespace

cudaError_t launch_tree_attn(const TreeAttnParams &p, bool e4m3, cudaStream_t s) {
  const int plan_blocks = p.max_units <= kPlanUnits * kPlanBlocks ? (p.max_units + kPlanUnits - 1) / kPlanUnits : kPlanBlocks;
  cudaError_t e = cudaSuccess;
  if (!plans_itself(p)) e = launch((const void *)tree_plan_kernel, p, plan_blocks, kPlanThreads, 0, 1, s);
  if (e == cudaSuccess)
    e = launch(e4m3 ? (const void *)tree_attn_kernel<true> : (const void *)tree_attn_kernel<false>, p, 2 * p.clusters,
               kTreeThreads, kTreeSmem, 2, s);
  if (e == cudaSuccess && p.clusters > 1)
    e = launch((const void *)tree_merge_kernel, p, (p.clusters - 1) * 2 * (kH / kMergeHeads), 32 * kMergeHeads, 0, 1, s);
  return e;
}

cudaError_t prepare_tree_kernels() {
  cudaError_t e = cudaSuccess;
  for (const void *f : {(const void *)tree_attn_kernel<true>, (const void *)tree_attn_kernel<false>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTreeSmem);
  for (const void *f : {(const void *)tree_plan_kernel, (const void *)tree_merge_kernel}) {
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, f);
  }
  return e;
}

}  // namespace ds4a
