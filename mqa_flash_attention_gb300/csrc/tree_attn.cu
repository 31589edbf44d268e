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
// as one MMA of M = 128 (2 x 64 heads) and N = 256 at the full rate (64 cycles of
// 8192 multiply-adds per SM; measured), each SM bringing half of the rows' operand:
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
// slots; a merge joins them.  Lengths are only known on the device: a one-block
// kernel counts the tiles first.
//
// Rows are found through the page tables.  Rows of a tile that neither token
// sees are zero-filled, those that one sees are masked for the other.
#include "attn_params.h"
#include "internal.h"
#include "ptx.cuh"
#include "ptx_async.cuh"
#include "step_params.h"

namespace ds4a {

namespace {

constexpr int kRows = 256;                  // of a tile
constexpr uint32_t kPart = 16384;           // a stage: 64 dims of 128 K rows, or 128 dims of 64 V rows
constexpr int kParts = 16;                  // stages of a tile: 8 of K, 8 of V
constexpr uint32_t kCodePart = kPart / 2;
constexpr uint32_t kOffTP = kQBytes;        // P: 4 boxes [64 heads][64 rows]
constexpr uint32_t kPBox = 8192;
constexpr uint32_t kOffRing = kOffTP + 4 * kPBox;
constexpr uint32_t kRingBytes = 7 * kPart;
constexpr uint32_t kOffTMisc = kOffRing + kRingBytes;
constexpr uint32_t kTmemTS = 256;           // S buffers at columns 256 and 384
constexpr int kListsT = 3;

// fp16 rows: seven stages.  E4M3 rows: codes land in slots of their own and are
// widened into four stages.
template <bool FP8>
constexpr int kStagesT = FP8 ? 4 : 7;
constexpr int kCodeSlots = 6;
static_assert(kStagesT<false> * kPart <= kRingBytes && 4 * kPart + kCodeSlots * kCodePart <= kRingBytes, "stages and code slots share the ring's bytes");
template <bool FP8>
constexpr int kLoadersT = FP8 ? kLoaderThreads - 128 : kLoaderThreads;

constexpr float kLeastLog2ScaleT = -40.f;   // V scales below 2^-40 count as 0: such rows round to 0 in fp16
constexpr unsigned long long kSegBitT = 1, kNoRowT = 2, kNoValue = 4;  // low bits of a list entry

// Of a tile within its item (the cluster's tiles of one unit).
enum : int { TF_FIRST = 1, TF_LAST = 2, TF_WHOLE = 4, TF_GATHERED = 8, TF_SPOILED = 16, TF_HEAD = 32 };

enum : unsigned int {
  TSITE_Q_EMPTY = 0x80, TSITE_KV_EMPTY, TSITE_Q_FULL, TSITE_S_EMPTY, TSITE_KV_FULL, TSITE_P_FULL, TSITE_O_EMPTY,
  TSITE_S_FULL, TSITE_P_EMPTY, TSITE_O_FULL, TSITE_DRAIN, TSITE_CODE_FULL, TSITE_LIST_FULL, TSITE_LIST_EMPTY,
  TSITE_CODE_EMPTY
};

struct TMisc {
  alignas(16) unsigned long long row[kListsT][kRows];  // K address | bits
  alignas(16) float ksc[kListsT][kRows];               // E4M3: scale * log2(e) * K scale
  alignas(16) float lvs[kListsT][kRows];               // E4M3: log2 of the V scale (of 2^-40 at least)
  alignas(16) float ivs[kListsT][kRows];               // E4M3: 2^-lvs
  int2 box[kListsT][kRows / 8];                        // (page, slot) of the runs of a tile that TMA loads
  uint32_t mask[kListsT][kRows / 32];                  // rows that this CTA's token sees
  int flags[kListsT], tok[kListsT];                    // TF_ bits; the token (-1: none)
  alignas(16) float red[4][kH];
  alignas(8) uint64_t q_full, q_empty, peer_q_full;
  uint64_t kv_full[7], kv_empty[7];  // (rank 0's kv_full: of both CTAs)
  uint64_t code_full[kCodeSlots], code_empty[kCodeSlots];
  uint64_t list_full[kListsT], list_empty[kListsT];
  uint64_t s_full[2], s_empty[2], o_full[2];
  uint64_t p_full, p_empty, o_empty, mma_done;
  uint32_t tmem_base;
  int abort_flag;
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

// The rows that a unit's tokens t0 .. t1 see: compressed rows [0, nc), cached raw
// rows [r0, r0 + nr), new rows [d0, d0 + nd).  (Of a tree, what any of its nodes
// could see: their depths are not known here.)
struct UnitRows {
  int nc, r0, nr, d0, nd, n_raw;
  __device__ __forceinline__ int len() const { return nc + nr + nd; }
  __device__ __forceinline__ int tiles() const { return max(1, (len() + kRows - 1) / kRows); }
};

__device__ __forceinline__ UnitRows unit_rows(const TreeAttnParams &p, int4 g, int n, int t0, int t1) {
  const bool chain = p.parent == nullptr;
  const long long pos = max(g.x, 0), raw_pos0 = max(g.z, 0);
  const int n_comp = min(max(g.w, 0), p.seg[1].max_rows);
  UnitRows r;
  r.n_raw = min(max(g.y, 0), p.seg[0].max_rows);
  r.nc = r.r0 = r.nr = r.d0 = r.nd = 0;
  if (!chain && t0 >= kTreeTokens) return r;  // nodes that see nothing
  const long long lo = chain ? pos + t0 : pos, hi = chain ? pos + t1 : pos + min(n, kTreeTokens) - 1;
  r.nc = (int)min((unsigned)n_comp, (unsigned)(hi + 1) / (unsigned)p.ratio);
  r.r0 = (int)min(max(lo - p.window + 1 - raw_pos0, 0ll), (long long)r.n_raw);
  const int r1 = (int)min(max(hi + 1 - raw_pos0, (long long)r.r0), (long long)r.n_raw);
  r.nr = r1 - r.r0;
  const int d1 = min(t1 + 1, p.seg[0].max_rows - r.n_raw);
  r.d0 = chain ? min(max(0, t0 - p.window + 1), d1) : 0;
  r.nd = d1 - r.d0;
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

__global__ void __launch_bounds__(kPlanThreads, 1) tree_plan_kernel(const TreeAttnParams p) {
  __shared__ int warp_sum[32];
  const int tid = threadIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  int units = 0;  // of the sequences before
  for (int b0 = 0; b0 < p.n_seq; b0 += kPlanThreads) {
    const int b = b0 + tid, n = b < p.n_seq ? (tokens_of(p, b).n + 1) / 2 : 0;
    int all;
    const int inc = block_scan(n, warp_sum, all);
    if (b < p.n_seq) p.ws_seq[b] = units + inc - n;
    units = min(units + all, 1 << 30);  // (only ranges that overlap name as many)
  }
  units = min(units, p.max_units);  // more than there is room for
  __syncthreads();
  int tiles = 0;
  for (int u0 = 0; u0 < units; u0 += kPlanThreads) {
    const int u = u0 + tid;
    int4 rec = make_int4(0, 0, 0, 0);
    if (u < units) {
      int lo = 0, hi = p.n_seq;  // the last sequence whose units begin at or before u
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.ws_seq[mid] <= u) lo = mid; else hi = mid;
      }
      const int n = tokens_of(p, lo).n, t0 = 2 * (u - p.ws_seq[lo]);
      rec = make_int4(lo, t0, unit_rows(p, p.geom[lo], n, t0, min(t0 + 1, n - 1)).tiles(), 0);
    }
    int all;
    const int inc = block_scan(rec.z, warp_sum, all);
    if (u < units) {
      rec.w = tiles + inc - rec.z;
      p.ws_unit[u] = rec;
    }
    tiles += all;
  }
  const int per = max(1, (tiles + p.clusters - 1) / p.clusters);
  if (tid == 0) p.ws_head[0] = make_int4(tiles, per, units, 0);
  __syncthreads();
  // The unit of each cluster's first tile.
  for (int u = tid; u < units; u += kPlanThreads) {
    const int4 rec = p.ws_unit[u];
    for (int i = (rec.w + per - 1) / per; (long long)i * per < rec.w + rec.z; ++i) p.ws_start[i] = u;
  }
}

// ------------------------------------------------------------------ loaders

// What token i of the unit sees of the list.
struct View {
  int nc, ra, rb, da, db;
  uint32_t anc[4];
};

template <bool FP8>
__device__ __forceinline__ void tree_load_role(const TreeAttnParams &p, int nt, int cluster, uint32_t rank, uint32_t sbase,
                                               TMisc &ms, int ltid) {
  constexpr int kGroup = kLoadersT<FP8>;
  constexpr int kRowStep = kGroup / 8, kWarps = kGroup / 32;
  constexpr int kMine = (kRows + kGroup - 1) / kGroup;
  constexpr int kSlots = FP8 ? kCodeSlots : kStagesT<false>;
  if (nt <= 0) return;
  volatile int *abrt = &ms.abort_flag;
  const int gtid = (FP8 && ltid >= 32) ? ltid - 128 : ltid, lane = ltid & 31, gwarp = gtid >> 5;
  const int c8 = gtid & 7, rsub = gtid >> 3;
  const bool chain = p.parent == nullptr;
  const long long vdelta0 = p.seg[0].v - p.seg[0].k, vdelta1 = p.seg[1].v - p.seg[1].k;
  const int pad_seg = p.seg[1].max_rows > 0 ? 1 : 0;
  const unsigned long long pad_row = reinterpret_cast<unsigned long long>(p.seg[pad_seg].k) | pad_seg | kNoRowT;
  Ring<kSlots> ring;
  bool ok = true, q_issued = false;
  uint32_t n_item = 0, q_par = 0, filled = 0, last_par = 0;
  int turn = 0;

  // The unit of the tile that is listed next, and what its tokens see.
  int u = p.ws_start[cluster], left = nt;
  int4 rec = p.ws_unit[u];
  int j = cluster * p.ws_head[0].y - rec.w, first_j = j;
  int tok0 = 0, own_tok = 0;
  UnitRows rows;
  View view[2];
  auto enter_unit = [&]() {
    const int4 g = p.geom[rec.x];
    const Span2 s = tokens_of(p, rec.x);
    const int t0 = rec.y, t1 = min(rec.y + 1, s.n - 1);
    tok0 = s.at + t0;
    own_tok = rank == 0 ? tok0 : t1 > t0 ? tok0 + 1 : -1;
    rows = unit_rows(p, g, s.n, t0, t1);
    const long long pos = max(g.x, 0), raw_pos0 = max(g.z, 0);
    const bool dead = !chain && t0 >= kTreeTokens;
    int par[4] = {-1, -1, -1, -1};
    if (!chain && !dead) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (32 * k + lane < min(s.n, kTreeTokens)) par[k] = p.parent[s.at + 32 * k + lane];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      View &v = view[i];
      const int t = i == 0 ? t0 : t1;
      v.nc = v.ra = v.rb = v.da = v.db = 0;
      v.anc[0] = v.anc[1] = v.anc[2] = v.anc[3] = 0;
      if (dead) continue;
      int depth = 0;
      if (chain) {
        depth = t;
        v.da = max(0, t - p.window + 1);
        v.db = t + 1;
      } else {
        // Up to the root; every lane alike.  (Each step goes to an earlier node.)
        for (int at = t;; ++depth) {
          if (depth < p.window) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (at >> 5 == k) v.anc[k] |= 1u << (at & 31);
          }
          const int mine = at < 32 ? par[0] : at < 64 ? par[1] : at < 96 ? par[2] : par[3];
          const int up = __shfl_sync(0xffffffffu, mine, at & 31);
          if (up < 0 || up >= at) break;
          at = up;
        }
      }
      const long long at_pos = pos + depth;
      v.nc = (int)min((unsigned)rows.nc, (unsigned)(at_pos + 1) / (unsigned)p.ratio);
      v.ra = (int)min(max(at_pos - p.window + 1 - raw_pos0, 0ll), (long long)rows.n_raw);
      v.rb = (int)min(max(at_pos + 1 - raw_pos0, 0ll), (long long)rows.n_raw);
    }
  };
  enter_unit();

  // A field of segment sg: a choice of two constants.
  auto of = [&](int sg, auto field) { return sg != 0 ? p.seg[1].*field : p.seg[0].*field; };
  // Tile whose page ids are in flight, then tile whose rows are known.
  int a_row[kMine], a_page[kMine], a_seen[kMine], a_flags = 0, a_own = 0, a_tok0 = 0;
  bool a_full = false, b_full = false, b_tma = false;
  unsigned long long b_at[kMine];
  int b_page[kMine], b_slot[kMine], b_seen[kMine], b_flags = 0, b_own = 0, b_tok0 = 0;
  float b_ks[kMine], b_vs[kMine];

  auto fetch_pages = [&]() {
    const int base = j * kRows, len = rows.len();
    const bool head = left == nt || j == 0;
    if (head) first_j = j;
    const bool last = j == rec.z - 1 || left == 1;
    a_flags = (head ? TF_FIRST : 0) | (last ? TF_LAST : 0) | (last && first_j == 0 && j == rec.z - 1 ? TF_WHOLE : 0) |
              (first_j == 0 ? TF_HEAD : 0);
    a_own = own_tok;
    a_tok0 = tok0;
    a_full = p.run_rows > 0 && base + kRows <= min(view[0].nc, view[1].nc);
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int r = gtid + k * kGroup, x = base + r;
      a_row[k] = a_page[k] = -1;
      a_seen[k] = 0;
      if (r < kRows && x < len) {
        const int sg = x < rows.nc ? 1 : 0;
        int row = x;
        if (sg != 0) {
          a_seen[k] = (x < view[0].nc ? 1 : 0) | (x < view[1].nc ? 2 : 0);
        } else if (x < rows.nc + rows.nr) {
          row = rows.r0 + (x - rows.nc);
          a_seen[k] = (row >= view[0].ra && row < view[0].rb ? 1 : 0) | (row >= view[1].ra && row < view[1].rb ? 2 : 0);
        } else {
          const int d = rows.d0 + (x - rows.nc - rows.nr);
          row = rows.n_raw + d;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = d < 32 ? view[i].anc[0] : d < 64 ? view[i].anc[1] : d < 96 ? view[i].anc[2] : view[i].anc[3];
            const bool seen = chain ? d >= view[i].da && d < view[i].db : ((w >> (d & 31)) & 1u) != 0;
            a_seen[k] |= seen ? 1 << i : 0;
          }
        }
        const int shift = of(sg, &PagedSeg::page_shift), per = of(sg, &PagedSeg::page_rows);
        const int pi = shift >= 0 ? row >> shift : row / per;
        if (a_seen[k] != 0) {
          a_page[k] = of(sg, &PagedSeg::table)[rec.x * of(sg, &PagedSeg::table_stride) + pi];
          a_row[k] = 2 * (row - pi * per) + sg;
        }
      }
    }
    // On to the next tile.
    --left;
    if (left > 0 && ++j == rec.z) {
      j = 0;
      rec = p.ws_unit[++u];
      enter_unit();
    }
  };
  auto find_rows = [&]() {
    b_flags = a_flags;
    b_own = a_own;
    b_tok0 = a_tok0;
    b_full = a_full;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      b_at[k] = pad_row;
      b_page[k] = a_page[k];
      b_slot[k] = a_row[k] >> 1;
      b_seen[k] = 0;
      b_ks[k] = 0.f;
      b_vs[k] = 1.f;
      const int sg = a_row[k] & 1;
      if (a_row[k] >= 0 && (unsigned)a_page[k] < (unsigned)of(sg, &PagedSeg::n_pages)) {
        const int slot = a_row[k] >> 1;
        b_seen[k] = a_seen[k];
        b_at[k] = reinterpret_cast<unsigned long long>(of(sg, &PagedSeg::k) + a_page[k] * of(sg, &PagedSeg::page_stride) +
                                                       slot * of(sg, &PagedSeg::row_stride)) |
                  sg;
        if (FP8) {
          const long long sr = (long long)a_page[k] * of(sg, &PagedSeg::page_rows) + slot;
          b_ks[k] = of(sg, &PagedSeg::k_scale)[sr];
          b_vs[k] = of(sg, &PagedSeg::v_scale)[sr];
        }
      }
    }
    // A V row that one token sees and the other does not must be finite, because
    // its weight of 0 multiplies it all the same: the warp looks these few rows
    // through (new rows, edges of a window).  One that is not finite is left out
    // of the product, and the token that sees it is marked.
    if (!b_full) {
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        unsigned who = __ballot_sync(0xffffffffu, b_seen[k] == 1 || b_seen[k] == 2);
        unsigned bad = 0;
        while (who != 0) {
          constexpr int kAhead = 4;
          uint4 v[kAhead][FP8 ? 1 : 2];
          int l[kAhead];
#pragma unroll
          for (int a = 0; a < kAhead; ++a) {
            l[a] = who != 0 ? __ffs(who) - 1 : -1;
            who &= who - 1;
            const unsigned long long e = __shfl_sync(0xffffffffu, b_at[k], max(l[a], 0));
            const uint8_t *src = reinterpret_cast<const uint8_t *>(e & ~15ull) + ((e & kSegBitT) ? vdelta1 : vdelta0);
#pragma unroll
            for (int w = 0; w < (FP8 ? 1 : 2); ++w)
              v[a][w] = l[a] >= 0 ? reinterpret_cast<const uint4 *>(src)[32 * w + lane] : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int a = 0; a < kAhead; ++a) {
            bool odd = false;
#pragma unroll
            for (int w = 0; w < (FP8 ? 1 : 2); ++w) {
              const uint32_t x[4] = {v[a][w].x, v[a][w].y, v[a][w].z, v[a][w].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (FP8) {
                  // A code of NaN: seven ones.  (Adding 1 to each seven carries into the eighth.)
                  odd = odd || (((x[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
                } else {
                  // An exponent of five ones.
                  odd = odd || (((x[i] & 0x7C007C00u) + 0x04000400u) & 0x80008000u) != 0;
                }
              }
            }
            if (__ballot_sync(0xffffffffu, odd) != 0 && l[a] >= 0) bad |= 1u << l[a];
          }
        }
        if ((bad >> lane) & 1u) b_at[k] |= kNoValue;
        if (__ballot_sync(0xffffffffu, ((bad >> lane) & 1u) != 0 && ((b_seen[k] >> rank) & 1) != 0) != 0)
          b_flags |= TF_SPOILED;
      }
    }
  };
  // The rows of tile g, complete for the whole group; all go on or none.
  // Returns whether TMA loads the tile.
  auto store_list = [&](int g) -> bool {
    const int buf = g % kListsT;
    const bool full = b_full;
    bool absent = false;
    b_tma = false;
    if (ok && !mbar_wait(smem_u32(&ms.list_empty[buf]), ((g / kListsT) & 1) ^ 1, abrt, p.timeout_ns, p.err,
                         TSITE_LIST_EMPTY))
      ok = false;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int r = gtid + k * kGroup;
      if (r < kRows) {  // whole warps
        const unsigned seen = __ballot_sync(0xffffffffu, (b_seen[k] >> rank) & 1);
        if (ok) {
          ms.row[buf][r] = b_at[k];
          if (lane == 0) ms.mask[buf][r >> 5] = seen;
          absent = absent || (b_at[k] & kNoRowT);
          if (full && (r & (p.run_rows - 1)) == 0) ms.box[buf][r >> p.run_shift] = make_int2(b_page[k], b_slot[k]);
        }
      }
    }
    __syncwarp();  // the barrier below is one of whole warps
    const bool odd = bar_red_or(3, kGroup, !ok || (full && absent));
    if (odd) ok = !bar_red_or(3, kGroup, !ok);
    b_tma = full && !odd;
    return b_tma;
  };
  // The rest of it, once its rows are on their way: what the other warps need.
  auto finish_list = [&](int g) {
    const int buf = g % kListsT;
    const bool spoiled = bar_red_or(3, kGroup, (b_flags & TF_SPOILED) != 0);
    if (ok) {
      if (FP8) {
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          const int r = gtid + k * kGroup;
          if (r < kRows) {
            ms.ksc[buf][r] = p.scale_log2 * b_ks[k];
            const float lv = fmaxf(__log2f(b_vs[k]), kLeastLog2ScaleT);
            ms.lvs[buf][r] = lv;
            ms.ivs[buf][r] = exp2f(-lv);
          }
        }
      }
      if (gtid == 0) {
        ms.flags[buf] = (b_flags & ~TF_SPOILED) | (spoiled ? TF_SPOILED : 0) | (b_tma ? 0 : TF_GATHERED);
        ms.tok[buf] = b_own;
      }
    }
    mbar_arrive(smem_u32(&ms.list_full[buf]));
  };
  // One part of tile g into the next stage: parts 0-7 dims 64 part .. of this
  // CTA's K rows, parts 8-15 (nb, kq): dims 256 nb + 128 rank .. of V rows 64 kq ..
  auto emit = [&](int g, int part, bool tma) -> bool {
    const uint32_t slot = FP8 ? sbase + kOffRing + 4 * kPart + ring.st * kCodePart : sbase + kOffRing + ring.st * kPart;
    const uint32_t b_full_bar = smem_u32(FP8 ? &ms.code_full[ring.st] : &ms.kv_full[ring.st]);
    const uint32_t b_empty = smem_u32(FP8 ? &ms.code_empty[ring.st] : &ms.kv_empty[ring.st]);
    const uint32_t ph = ring.ph ^ 1, st_bit = 1u << ring.st;
    ring.advance();
    // Every thread waits for every fill of a stage, whoever loads it: a parity
    // wait is only right for a thread that has seen the phase before.
    if (!(FP8 ? mbar_wait(b_empty, ph, abrt, p.timeout_ns, p.err, TSITE_CODE_EMPTY)
              : mbar_wait(b_empty, ph, abrt, p.timeout_ns, p.err, TSITE_KV_EMPTY)))
      return false;
    const bool is_v = part >= 8;
    const int nb = (part >> 2) & 1, kq = part & 3;
    const int row0 = is_v ? 64 * kq : 128 * (int)rank;           // first row of the part within the tile
    const int dim0 = is_v ? 256 * nb + 128 * (int)rank : 64 * part;
    const int buf = g % kListsT;
    if (tma) {
      // Run i of a part goes to one lane of warp (turn + i) % warps; lane 0 of
      // each warp arrives for all its lanes.
      const int runs = (is_v ? 64 : 128) >> p.run_shift;
      const int first = gwarp - turn, i = (first < 0 ? first + kWarps : first) + lane * kWarps;
      turn = (turn + runs) % kWarps;
      // (fp16: the bytes of both CTAs count at rank 0's barrier; here only the issue does.)
      if (lane == 0) {
        const bool expects = gtid == 0 && (FP8 || rank == 0);
        if (expects) mbar_arrive_expect_tx(b_full_bar, FP8 ? kCodePart : 2 * kPart);
        mbar_arrive_cnt(b_full_bar, expects ? 31 : 32);
      }
      if (i < runs) {
        filled |= st_bit;
        last_par = ph ? last_par & ~st_bit : last_par | st_bit;
        const uint32_t dst = slot + (i << p.run_shift) * (is_v ? (FP8 ? 128u : 256u) : (FP8 ? 64u : 128u));
        const CUtensorMap *m = is_v ? &p.tm_v : &p.tm_k;
        const int2 x = ms.box[buf][(row0 >> p.run_shift) + i];
        if (FP8)
          tma_load_3d(dst, m, b_full_bar, dim0, x.y, x.x);
        else
          tma_load_5d_pair(dst, m, cluster_addr(b_full_bar, 0), 0, 0, dim0 >> 6, x.y >> 3, x.x);
      }
      return true;
    }
    const unsigned long long *list = ms.row[buf] + row0;
    const long long off0 = (is_v ? vdelta0 : 0) + (FP8 ? dim0 : 2 * dim0), off1 = (is_v ? vdelta1 : 0) + (FP8 ? dim0 : 2 * dim0);
    const unsigned long long skip = is_v ? kNoRowT | kNoValue : kNoRowT;
    if (FP8) {
      // 16 codes a copy: 4 copies a row of K, 8 of V; 512 in all.
      for (int i = gtid; i < 512; i += kGroup) {
        const int row = is_v ? i >> 3 : i >> 2, c = is_v ? i & 7 : i & 3;
        const unsigned long long e = list[row];
        cp_async16z(slot + 16 * i, reinterpret_cast<const uint8_t *>(e & ~15ull) + ((e & kSegBitT) ? off1 : off0) + 16 * c,
                    (e & skip) ? 0u : 16u);
      }
    } else if (!is_v) {
#pragma unroll
      for (int it = 0; it < (128 + kRowStep - 1) / kRowStep; ++it) {
        const int row = kRowStep * it + rsub;
        if (row >= 128) break;
        const unsigned long long e = list[row];
        cp_async16z(slot + (row >> 3) * 1024 + (row & 7) * 128 + ((c8 ^ (row & 7)) << 4),
                    reinterpret_cast<const uint8_t *>(e & ~15ull) + ((e & kSegBitT) ? off1 : off0) + 16 * c8,
                    (e & skip) ? 0u : 16u);
      }
    } else {
#pragma unroll
      for (int it = 0; it < (64 + kRowStep - 1) / kRowStep; ++it) {
        const int row = kRowStep * it + rsub;
        if (row >= 64) break;
        const unsigned long long e = list[row];
        const uint32_t dst = slot + (row >> 3) * 2048 + (row & 7) * 128 + ((c8 ^ (row & 7)) << 4), n = (e & skip) ? 0u : 16u;
        const uint8_t *src = reinterpret_cast<const uint8_t *>(e & ~15ull) + ((e & kSegBitT) ? off1 : off0) + 16 * c8;
        cp_async16z(dst, src, n);
        cp_async16z(dst + 1024, src + 128, n);
      }
    }
    cp_async_arrive(b_full_bar);
    return true;
  };
  auto load_q = [&]() {
    if (gtid == 0 && ok) {
      if (!mbar_wait(smem_u32(&ms.q_empty), (n_item & 1) ^ 1, abrt, p.timeout_ns, p.err, TSITE_Q_EMPTY)) {
        ok = false;
      } else {
        mbar_arrive_expect_tx(smem_u32(&ms.q_full), kQBytes);
        tma_load_4d(sbase, &p.tm_q, smem_u32(&ms.q_full), 0, 0, b_own >= 0 ? b_own : b_tok0, 0);
        q_issued = true;
        q_par = n_item & 1;
      }
    }
    ++n_item;
  };

  fetch_pages();
  bool tma = false, tma_v;  // whether TMA loads tile g, and tile g - 1
  for (int g = 0; g <= nt; ++g) {
    tma_v = tma;
    if (g < nt) {
      find_rows();
      if (g + 1 < nt) fetch_pages();
      tma = store_list(g);
      if (b_flags & TF_FIRST) load_q();
      // The list before the last K parts: the ring holds fewer than a tile's eight,
      // and who empties it waits for the list.
      for (int part = 0; part < 4 && ok; ++part) ok = emit(g, part, tma);
      __syncwarp();
      finish_list(g);
      for (int part = 4; part < 8 && ok; ++part) ok = emit(g, part, tma);
    } else {
      __syncwarp();
      ok = !bar_red_or(3, kGroup, !ok);
    }
    if (g > 0)
      for (int part = 8; part < kParts && ok; ++part) ok = emit(g - 1, part, tma_v);
    __syncwarp();
  }
  // No copy may still be landing at exit.  (When every wait succeeded the MMA
  // warp has seen all stages land.)
  cp_async_done();
  volatile int never = 0;
  if (*abrt != 0)
    for (int st = 0; st < kSlots; ++st)
      if (filled & (1u << st))
        mbar_wait(smem_u32(FP8 ? &ms.code_full[st] : &ms.kv_full[st]), (last_par >> st) & 1, &never, 100000000ull,
                  p.err, TSITE_DRAIN);
  if (gtid == 0 && q_issued) mbar_wait(smem_u32(&ms.q_full), q_par, &never, 100000000ull, p.err, TSITE_DRAIN);
}

// Warps 9-12 with E4M3 rows: a slot's codes, 64 a thread, widened exactly into
// the next stage in the layout that the fp16 kernel's copies have.
__device__ __forceinline__ void tree_convert_role(const TreeAttnParams &p, int nt, uint32_t sbase, TMisc &ms, int ct) {
  volatile int *abrt = &ms.abort_flag;
  Ring<kCodeSlots> codes;
  Ring<kStagesT<true>> ring;
  for (long long i = 0; i < (long long)nt * kParts; ++i) {
    // Stages come as K(0), then K(g + 1) and V(g): the first eight, then by turns, the last eight of V.
    const long long eighth = i >> 3, last = 2ll * nt - 1;
    const bool is_v = eighth != 0 && (eighth == last || (eighth & 1) == 0);
    if (!mbar_wait(smem_u32(&ms.code_full[codes.st]), codes.ph, abrt, p.timeout_ns, p.err, TSITE_CODE_FULL)) return;
    const uint32_t src = sbase + kOffRing + 4 * kPart + codes.st * kCodePart, dst = sbase + kOffRing + ring.st * kPart;
    uint4 raw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(raw[k].x), "=r"(raw[k].y), "=r"(raw[k].z), "=r"(raw[k].w)
                   : "r"(src + 16 * (ct + 128 * k)));
    __syncwarp();
    if ((ct & 31) == 0) mbar_arrive(smem_u32(&ms.code_empty[codes.st]));
    if (!mbar_wait(smem_u32(&ms.kv_empty[ring.st]), ring.ph ^ 1, abrt, p.timeout_ns, p.err, TSITE_KV_EMPTY)) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = ct + 128 * k;
      const int row = is_v ? n >> 3 : n >> 2, c = is_v ? n & 7 : n & 3;  // 16 codes: chunks 2c, 2c + 1 of 8 values
      const uint32_t w4[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[2 * e] = e4m3x2_to_f16x2(static_cast<uint16_t>(w4[e] & 0xFFFFu));
        h[2 * e + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w4[e] >> 16));
      }
      const uint32_t drow = dst + (row & 7) * 128 + (is_v ? (row >> 3) * 2048 + (c >> 2) * 1024 : (row >> 3) * 1024);
      const int col = 2 * (c & 3);
      sts_v4(drow + ((col ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
      sts_v4(drow + (((col + 1) ^ (row & 7)) << 4), h[4], h[5], h[6], h[7]);
    }
    mbar_arrive(smem_u32(&ms.kv_full[ring.st]));
    codes.advance();
    ring.advance();
  }
}

// ------------------------------------------------------------------ MMA issue and relay

// The CTA of rank 1 has no MMA to issue: its last warp tells the other CTA what
// has landed here.  Gathered and widened rows are generic-proxy writes: the fence
// makes them visible to the tensor core before the news goes out.
template <bool FP8>
__device__ __forceinline__ void tree_relay_role(const TreeAttnParams &p, int nt, TMisc &ms) {
  volatile int *abrt = &ms.abort_flag;
  Ring<kStagesT<FP8>> ring;
  uint32_t item = 0;
  auto parts = [&](int n) -> bool {
    for (int i = 0; i < n; ++i) {
      if (!mbar_wait(smem_u32(&ms.kv_full[ring.st]), ring.ph, abrt, p.timeout_ns, p.err, TSITE_KV_FULL)) return false;
      fence_proxy_async_smem();
      mbar_arrive_cluster(cluster_addr(smem_u32(&ms.kv_full[ring.st]), 0));
      ring.advance();
    }
    return true;
  };
  if (nt <= 0) return;
  for (int g = 0; g < nt; ++g) {
    const int buf = g % kListsT;
    if (!mbar_wait(smem_u32(&ms.list_full[buf]), (g / kListsT) & 1, abrt, p.timeout_ns, p.err, TSITE_LIST_FULL)) return;
    const int flags = ms.flags[buf];
    mbar_arrive(smem_u32(&ms.list_empty[buf]));
    if (flags & TF_FIRST) {
      if (!mbar_wait(smem_u32(&ms.q_full), item & 1, abrt, p.timeout_ns, p.err, TSITE_Q_FULL)) return;
      mbar_arrive_cluster(cluster_addr(smem_u32(&ms.peer_q_full), 0));
      ++item;
    }
    if (!parts(8)) return;
    if (g > 0 && !parts(8)) return;
  }
  parts(8);
}

// The whole warp walks the tiles, so that descriptors are warp-uniform values, and
// one elected lane issues.  Waits are joined over the warp: all lanes go on or none.
template <bool FP8>
__device__ __forceinline__ void tree_mma_role(const TreeAttnParams &p, int nt, uint32_t sbase, uint32_t tmem, TMisc &ms) {
  volatile int *abrt = &ms.abort_flag;
  constexpr uint32_t kIdescQK = idesc_f16_f32(128, 256, false, false);
  constexpr uint32_t kIdescPV = idesc_f16_f32(128, 256, false, true);
  // Q, K and P: K-major.  V: MN-major, LBO = distance of the 64-dim blocks, SBO =
  // distance of 8-row groups.
  const uint64_t q_desc = sdesc_sw128(sbase, 16, 1024);
  const uint64_t k_desc = sdesc_sw128(sbase + kOffRing, 16, 1024);
  const uint64_t p_desc = sdesc_sw128(sbase + kOffTP, 16, 1024);
  const uint64_t v_desc = sdesc_sw128(sbase + kOffRing, 1024, 2048);
  Ring<kStagesT<FP8>> ring;
  uint32_t q_item = 0, o_item = 0;
  auto wait = [&](uint64_t &bar, uint32_t parity, unsigned int site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity, abrt, p.timeout_ns, p.err, site));
  };
  auto stage_ready = [&](bool gathered) -> bool {
    if (!wait(ms.kv_full[ring.st], ring.ph, TSITE_KV_FULL)) return false;
    if (FP8 || gathered) fence_proxy_async_smem();
    return true;
  };
  auto qk = [&](int g, int flags) -> bool {
    const uint32_t sb = g & 1;
    if (flags & TF_FIRST) {
      if (!wait(ms.q_full, q_item & 1, TSITE_Q_FULL) || !wait(ms.peer_q_full, q_item & 1, TSITE_Q_FULL)) return false;
      ++q_item;
    }
    if (!wait(ms.s_empty[sb], ((g >> 1) & 1) ^ 1, TSITE_S_EMPTY)) return false;
    tc_fence_after();
    const uint32_t d = tmem + kTmemTS + 128 * sb;
    for (int c = 0; c < 8; ++c) {
      if (!stage_ready(flags & TF_GATHERED)) return false;
      const uint64_t a0 = sdesc_add(q_desc, c * kQBoxBytes), b0 = sdesc_add(k_desc, ring.st * kPart);
      if (elect_lane()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          if (ks == 0)
            umma_pair_f16(d, a0, b0, kIdescQK, c != 0 ? 1u : 0u);
          else
            umma_pair_f16_acc(d, sdesc_add(a0, ks * 32), sdesc_add(b0, ks * 32), kIdescQK);
        }
        umma_pair_commit(smem_u32(&ms.kv_empty[ring.st]));
        if (c == 7) umma_pair_commit(smem_u32(&ms.s_full[sb]));
        if (c == 7 && (flags & TF_LAST)) umma_pair_commit(smem_u32(&ms.q_empty));
      }
      __syncwarp();
      ring.advance();
    }
    return true;
  };
  auto pv = [&](int g, int flags) -> bool {
    if (!wait(ms.p_full, g & 1, TSITE_P_FULL)) return false;
    const bool first = flags & TF_FIRST;
    if (first) {
      if (!wait(ms.o_empty, (o_item & 1) ^ 1, TSITE_O_EMPTY)) return false;
      ++o_item;
    }
    tc_fence_after();
    for (int c = 0; c < 8; ++c) {
      const int nb = c >> 2, kq = c & 3;
      if (!stage_ready(flags & TF_GATHERED)) return false;
      const uint64_t a0 = sdesc_add(p_desc, kq * kPBox), b0 = sdesc_add(v_desc, ring.st * kPart);
      const uint32_t d = tmem + 128 * nb;
      if (elect_lane()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          if (ks == 0)
            umma_pair_f16(d, a0, b0, kIdescPV, first && kq == 0 ? 0u : 1u);
          else
            umma_pair_f16_acc(d, sdesc_add(a0, ks * 32), sdesc_add(b0, ks * 4096), kIdescPV);
        }
        umma_pair_commit(smem_u32(&ms.kv_empty[ring.st]));
        if (kq == 3 && (flags & TF_LAST)) umma_pair_commit(smem_u32(&ms.o_full[nb]));
        if (c == 7) umma_pair_commit(smem_u32(&ms.p_empty));
      }
      __syncwarp();
      ring.advance();
    }
    return true;
  };
  bool ok = true;
  int flags = 0;
  for (int g = 0; g <= nt && ok; ++g) {
    const int before = flags;
    if (g < nt) {
      const int buf = g % kListsT;
      ok = wait(ms.list_full[buf], (g / kListsT) & 1, TSITE_LIST_FULL);
      if (!ok) break;
      flags = ms.flags[buf];
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&ms.list_empty[buf]));
      ok = qk(g, flags);
    }
    if (ok && g > 0) ok = pv(g - 1, before);
  }
}

// ------------------------------------------------------------------ softmax and epilogue

// The reference of a head lies kLiftT below the largest score of the tile that
// set it, and moves only when a score passes it by kLiftT + kHoldT (the reasons
// and figures stand at paged_attn.cu's kLift): P is 2^15 at most.
constexpr float kLiftT = 10.f, kHoldT = 5.f;
constexpr float kNoRefT = -3e38f;

__device__ __forceinline__ void stg32(void *at, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Warp w: TMEM lanes 32 (w & 3) .., that is heads 32 (w & 1) .. and rows 128 of
// the tile's half (w >> 1) & 1, of which it has 64, by w >> 2.  A head's four
// threads are in four warps (a group, w & 1), which vote and meet by themselves.
template <bool FP8>
__device__ __forceinline__ void tree_softmax_role(const TreeAttnParams &p, int nt, int cluster, uint32_t rank,
                                                  uint8_t *smem, uint32_t tmem, TMisc &ms, int tid) {
  volatile int *abrt = &ms.abort_flag;
  const int w = tid >> 5, l = tid & 31;
  const int q = w & 3, hh = w >> 2, half = q >> 1;
  const int h = 32 * (q & 1) + l, box = 2 * half + hh;
  const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
  const uint32_t group = 1 + (q & 1);
  const uint32_t r_s_empty[2] = {cluster_addr(smem_u32(&ms.s_empty[0]), 0), cluster_addr(smem_u32(&ms.s_empty[1]), 0)};
  const uint32_t r_p_full = cluster_addr(smem_u32(&ms.p_full), 0), r_o_empty = cluster_addr(smem_u32(&ms.o_empty), 0);
  auto tell = [&](uint32_t bar) {  // one arrival per warp
    __syncwarp();
    if (l == 0) mbar_arrive_cluster(bar);
  };
  bool bad = false, spoiled = false;
  uint32_t n_item = 0;
  float m_ref = kNoRefT, m_lim = kNoRefT, lsum = 0.f;
  uint8_t *prow = smem + kOffTP + box * kPBox + (h >> 3) * 1024 + (h & 7) * 128;
  for (int g = 0; g < nt; ++g) {
    const int buf = g % kListsT;
    const uint32_t sb = g & 1;
    bad = bad || !mbar_wait(smem_u32(&ms.list_full[buf]), (g / kListsT) & 1, abrt, p.timeout_ns, p.err, TSITE_LIST_FULL);
    const int flags = ms.flags[buf], tok = ms.tok[buf];
    const uint32_t see0 = ms.mask[buf][2 * box], see1 = ms.mask[buf][2 * box + 1];
    if (flags & TF_FIRST) {
      m_ref = m_lim = kNoRefT;
      lsum = 0.f;
      spoiled = false;
    }
    spoiled = spoiled || (flags & TF_SPOILED);
    if (!FP8) mbar_arrive(smem_u32(&ms.list_empty[buf]));
    bad = bad || !mbar_wait(smem_u32(&ms.s_full[sb]), (g >> 1) & 1, abrt, p.timeout_ns, p.err, TSITE_S_FULL);
    tc_fence_after();
    float s[64];
    tmem_ld64(tmem + kTmemTS + 128 * sb + 64 * hh + lanes, s);
    tmem_wait_ld();
    tc_fence_before();
    tell(r_s_empty[sb]);
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
    bad = bad || !mbar_wait(smem_u32(&ms.p_empty), (g & 1) ^ 1, abrt, p.timeout_ns, p.err, TSITE_P_EMPTY);
    {
      // This head's 64 weights: 16-byte chunk c of its 128 bytes at c ^ (h & 7).
      // Rounded once to fp16 for the product; the sums add them unrounded, sixteen
      // at a time, so that lse keeps fp32 precision over long rows.
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t w4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = 8 * c + 2 * i;
          const float e0 = exp2f(s[x] - m_ref), e1 = exp2f(s[x + 1] - m_ref);
          if (FP8) {
            const float2 iv = *reinterpret_cast<const float2 *>(&ms.ivs[buf][64 * box + x]);
            const float2 lv = *reinterpret_cast<const float2 *>(&ms.lvs[buf][64 * box + x]);
            part[i] = fmaf(e0, iv.x, fmaf(e1, iv.y, part[i]));
            // A V scale of 0: weight, but no value.
            const __half2 hp = __floats2half2_rn(lv.x <= kLeastLog2ScaleT ? 0.f : e0, lv.y <= kLeastLog2ScaleT ? 0.f : e1);
            w4[i] = *reinterpret_cast<const uint32_t *>(&hp);
          } else {
            part[i] += e0 + e1;
            const __half2 hp = __floats2half2_rn(e0, e1);
            w4[i] = *reinterpret_cast<const uint32_t *>(&hp);
          }
        }
        *reinterpret_cast<uint4 *>(prow + ((c ^ (h & 7)) << 4)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
      }
      lsum += (part[0] + part[1]) + (part[2] + part[3]);
    }
    if (FP8) mbar_arrive(smem_u32(&ms.list_empty[buf]));
    if (moved && !(flags & TF_FIRST)) {
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
    }
    fence_proxy_async_smem();
    tc_fence_before();
    tell(r_p_full);
    if (!(flags & TF_LAST)) continue;

    // End of an item: the sum over a head's four threads, then this thread's 128
    // dims of o (dims 256 hh + 128 half ..) once the last PV has finished them.
    const bool whole = flags & TF_WHOLE;
    ms.red[box][h] = lsum;
    if (bar_red_or(group, 128, bad)) break;
    const float sum = (ms.red[0][h] + ms.red[1][h]) + (ms.red[2][h] + ms.red[3][h]);
    // No weight at all: o = 0.  (A sum that is NaN is not that: it stays.)
    const bool none = sum == 0.f;
    const float inv = spoiled ? __int_as_float(0x7FC00000) : none ? 0.f : 1.f / sum;
    const long long slot = 2ll * (2 * cluster + (flags & TF_HEAD ? 1 : 0)) + rank;
    if (box == 0 && tok >= 0) {
      if (!whole)
        p.ws_ml[slot * kH + h] = make_float2(none ? -INFINITY : m_ref, sum);
      else if (p.lse != nullptr)
        p.lse[(long long)tok * kH + h] = none ? -INFINITY : (m_ref + log2f(sum)) * kLn2;
    }
    bad = bad || !mbar_wait(smem_u32(&ms.o_full[hh]), n_item & 1, abrt, p.timeout_ns, p.err, TSITE_O_FULL);
    tc_fence_after();
    const int dim0 = 256 * hh + 128 * half;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float o[32];
      tmem_ld32(tmem + 128 * hh + 32 * c + lanes, o);
      tmem_wait_ld();
      if (tok < 0) continue;
      if (whole) {
        __half *at = p.o + tok * p.o_stride + (long long)h * kD + dim0 + 32 * c;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const __half2 v = __floats2half2_rn(o[16 * k + 2 * i] * inv, o[16 * k + 2 * i + 1] * inv);
            x[i] = *reinterpret_cast<const uint32_t *>(&v);
          }
          if (p.o_wide) {
            stg32(at + 16 * k, x);
          } else {
            reinterpret_cast<uint4 *>(at + 16 * k)[0] = make_uint4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<uint4 *>(at + 16 * k)[1] = make_uint4(x[4], x[5], x[6], x[7]);
          }
        }
      } else {
        float *at = p.ws_o + (slot * kH + h) * kD + dim0 + 32 * c;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __float_as_uint(o[8 * k + i] * inv);
          stg32(at + 8 * k, x);
        }
      }
    }
    tc_fence_before();
    tell(r_o_empty);
    ++n_item;
    if (bar_red_or(group, 128, bad)) break;  // (and the sums have been read)
  }
}

// ------------------------------------------------------------------ kernel

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_kernel(const __grid_constant__ TreeAttnParams p) {
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
      mbar_init(smem_u32(&ms.kv_full[s]), (FP8 ? 128 : kLoadersT<false>) + (rank == 0 ? 1 : 0));
      mbar_init(smem_u32(&ms.kv_empty[s]), 1);
    }
    for (int s = 0; s < kCodeSlots; ++s) {
      mbar_init(smem_u32(&ms.code_full[s]), kLoadersT<true>);
      mbar_init(smem_u32(&ms.code_empty[s]), 4);
    }
    for (int s = 0; s < kListsT; ++s) {
      mbar_init(smem_u32(&ms.list_full[s]), kLoadersT<FP8>);
      mbar_init(smem_u32(&ms.list_empty[s]), kComputeThreads + 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ms.s_full[s]), 1);
      mbar_init(smem_u32(&ms.s_empty[s]), 2 * kComputeWarps);
      mbar_init(smem_u32(&ms.o_full[s]), 1);
    }
    mbar_init(smem_u32(&ms.p_full), 2 * kComputeWarps);
    mbar_init(smem_u32(&ms.p_empty), 1);
    mbar_init(smem_u32(&ms.o_empty), 2 * kComputeWarps);
    mbar_init(smem_u32(&ms.mma_done), 1);
    ms.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_q);
    if (p.run_rows > 0) {
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
    }
  }
  if (warp == kMmaWarp) tmem_alloc_pair(smem_u32(&ms.tmem_base), kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // both CTAs' barriers and TMEM are ready
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  grid_launch_dependents();
  grid_dependency_wait();  // the plan
  const int4 head = p.ws_head[0];
  const long long before = (long long)cluster * head.y;
  const int nt = (int)max(0ll, min((long long)head.y, head.x - before));
  if (warp < kComputeWarps) {
    tree_softmax_role<FP8>(p, nt, cluster, rank, smem, tmem, ms, threadIdx.x);
  } else if (warp == kMmaWarp) {
    if (rank == 0) {
      tree_mma_role<FP8>(p, nt, sbase, tmem, ms);
      __syncwarp();
      if (elect_lane()) umma_pair_commit(smem_u32(&ms.mma_done));
    } else if ((threadIdx.x & 31) == 0) {
      tree_relay_role<FP8>(p, nt, ms);
    }
    __syncwarp();
    volatile int never = 0;
    mbar_wait(smem_u32(&ms.mma_done), 0, &never, 3 * p.timeout_ns, p.err, TSITE_DRAIN);
    __syncwarp();
  } else {
    const int ltid = threadIdx.x - 32 * kLoaderWarp0;
    if (FP8 && ltid >= 32 && ltid < 160)
      tree_convert_role(p, nt, sbase, ms, ltid - 32);
    else
      tree_load_role<FP8>(p, nt, cluster, rank, sbase, ms, ltid);
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // neither CTA leaves while the other may still arrive here, or its MMAs read
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

// ------------------------------------------------------------------ merge
// A unit is cut where a cluster's tiles end: at most once per cluster.  Block
// (boundary, token, 8 heads): the first boundary inside a unit joins its parts,
// of the cluster it begins in (its second slot) and of those that follow (their
// first).  With M = max m_s and W_s = 2^(m_s - M) l_s:
//   o = sum_s W_s o_s / L,  L = sum_s W_s,  lse = (M + log2 L) ln 2.

constexpr int kMergeHeads = 8;
constexpr int kMergeAhead = 4;

__global__ void __launch_bounds__(32 * kMergeHeads) tree_merge_kernel(const TreeAttnParams p) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int group = blockIdx.x % (kH / kMergeHeads), rest = blockIdx.x / (kH / kMergeHeads);
  const int i = rest & 1, edge = 1 + (rest >> 1), h = group * kMergeHeads + (threadIdx.x >> 5);
  const int4 head = p.ws_head[0];
  const long long at = (long long)edge * head.y;
  if (at >= head.x) return;
  const int4 rec = p.ws_unit[p.ws_start[edge]];
  if (rec.w >= at || at - rec.w > head.y) return;  // no cut here, or not the unit's first
  const Span2 s = tokens_of(p, rec.x);
  const int t = rec.y + i;
  if (t >= s.n) return;
  const int n = (rec.w + rec.z - 1) / head.y - (edge - 1) + 1;  // parts
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
  const long long tok = s.at + t;
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
  cudaError_t e = launch((const void *)tree_plan_kernel, p, 1, kPlanThreads, 0, 1, s);
  if (e == cudaSuccess)
    e = launch(e4m3 ? (const void *)tree_attn_kernel<true> : (const void *)tree_attn_kernel<false>, p, 2 * p.clusters,
               kThreads, kTreeSmem, 2, s);
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
