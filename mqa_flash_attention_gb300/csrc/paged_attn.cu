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
// Work.  A sequence's visible rows, raw then compressed, form one list, cut
// into tiles of 128 rows; row j of the list is found through the page table,
// so pages of any size, tiles that span pages and pages that end inside a tile
// are all alike.  The tiles of all sequences are numbered through and CTA i
// takes ceil(total / CTAs) of them in a row: the load is even whatever the
// lengths.  A CTA's tiles of one sequence are an item.  An item that holds
// the whole sequence writes its output; otherwise it leaves its normalised
// output (fp16) and (m, l) in slot (CTA + sequence) of the workspace (unique,
// since along the tiles either number grows), and the merge kernel joins the
// slots of a sequence.
//
// Per tile, as in attn_kernel.cuh, the rows are on the M side of every MMA:
//   S^T[128 rows][64 heads]  = K_tile[128][512] . Q^T
//   O^T[512 dims][64 heads] += V_tile^T . P^T
// with S^T and O^T in TMEM.  An absent row's K and V are zero-filled in shared
// memory (cp.async with no source bytes), so nothing a page holds beyond the
// rows in use can reach a product, not even as 0 * NaN.
//
// Warps (512 threads, one CTA per SM): 0-7 softmax and epilogue, 8-14 loaders,
// 15 TMEM allocation and MMA issue.  The loaders copy the rows with 16-byte
// cp.async in the 128-byte swizzled layout; in ring order K(0), then K(j+1)
// and V(j) for each tile j, so the next scores are computed while the softmax
// works.  With E4M3 rows, warps 8, 13 and 14 copy codes into the upper half of
// a stage and warps 9-12 widen them in place, exactly.
//
// E4M3 scales.  K's multiplies the scores.  V's scale c_j is folded into the
// exponent: p'_j = 2^(s_j + log2 c_j - m') with m' the running maximum of that
// sum, so the fp16 p' that feeds the MMA has full precision whatever the size
// of the scales; the sum of weights adds p'_j / c_j.
#include "attn_params.h"
#include "internal.h"
#include "paged_params.h"
#include "ptx.cuh"

namespace ds4a {

namespace {

constexpr int kLists = 4;  // row lists in flight
constexpr float kLeastLog2Scale = -40.f;  // V scales below 2^-40 count as 0: such rows round to 0 in fp16

// Wait sites of this kernel.
enum : unsigned int {
  PSITE_Q_EMPTY = 0x60, PSITE_KV_EMPTY, PSITE_Q_FULL, PSITE_S_EMPTY, PSITE_KV_FULL, PSITE_P_FULL, PSITE_O_EMPTY,
  PSITE_S_FULL, PSITE_P_EMPTY, PSITE_O_FULL, PSITE_DRAIN, PSITE_CODE_FULL, PSITE_LIST_FULL, PSITE_LIST_EMPTY
};

struct PMisc {
  alignas(16) unsigned long long row[kLists][kTile];  // K address | segment; 0: no row
  alignas(16) float ksc[kLists][kTile];   // E4M3: scale * log2(e) * K scale
  alignas(16) float lvs[kLists][kTile];   // E4M3: log2 of the V scale (of 2^-40 at least)
  alignas(16) float ivs[kLists][kTile];   // E4M3: 2^-lvs
  alignas(16) float red[4][kH];
  alignas(16) float m_use[kH];
  alignas(16) float alpha[kH];
  alignas(16) float inv_l[kH];
  alignas(8) uint64_t q_full, q_empty;
  uint64_t kv_full[kStages], kv_empty[kStages], code_full[kStages];
  uint64_t list_full[kLists], list_empty[kLists];
  uint64_t s_full[2], s_empty[2];
  uint64_t o_full[4];
  uint64_t p_full, p_empty, o_empty, mma_done;
  unsigned scan[kThreads / 32];
  int first_seq, first_tile;  // where this CTA's tiles start: sequence, tile within it
  int n_tiles;                // tiles of this CTA
  int per_cta;                // tiles of a full CTA
  uint32_t tmem_base;
  int abort_flag;
  int resc_flag[2];
};
constexpr uint32_t kPagedSmem = kOffMisc + ((sizeof(PMisc) + 127) / 128) * 128 + 1024;
static_assert(kPagedSmem <= 232448, "shared memory of one CTA");

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

__device__ __forceinline__ void bar_sync_id(uint32_t id, uint32_t count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
// 16 bytes global -> shared; `bytes` of 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// The rows sequence b's token sees: raw rows [raw_lo, raw_lo + nr), then
// compressed rows [0, nc).  The weights need the compressed ones only.
struct SeqRows {
  int raw_lo, nr, nc;
  __device__ __forceinline__ int tiles() const { return (nr + nc + kTile - 1) / kTile; }
};

template <bool WEIGHTS>
__device__ __forceinline__ SeqRows seq_rows(const PagedAttnParams &p, int b) {
  const int4 g = __ldg(p.geom + b);
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
  s.nc = (int)min((long long)n_comp, ((long long)pos + 1) / p.ratio);
  return s;
}

// A CTA's tiles in order.
template <bool WEIGHTS>
struct Walk {
  int b, j, n;   // sequence, tile within it, its tiles
  SeqRows rows;
  bool first, last;  // of this CTA's tiles of the sequence (an item)
  int left;      // tiles of the CTA from this one on
  __device__ __forceinline__ void start(const PagedAttnParams &p, const PMisc &ms) {
    b = ms.first_seq;
    j = ms.first_tile;
    left = ms.n_tiles;
    if (left <= 0) return;
    rows = seq_rows<WEIGHTS>(p, b);
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
      } while (n == 0);
      j = 0;
      first = true;
    }
    last = j == n - 1 || left == 1;
  }
  // Whole sequence in this item (asked at its last tile): it began here, at tile 0.
  __device__ __forceinline__ bool whole(int first_j) const { return first_j == 0 && j == n - 1; }
};

// Block-wide: where this CTA starts and how many tiles it has; CTA 0 also
// writes each sequence's slots for the merge.
template <bool WEIGHTS>
__device__ __forceinline__ void plan_cta(const PagedAttnParams &p, PMisc &ms) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int mine = 0;
  for (int b = tid; b < p.n_seq; b += kThreads) mine += seq_rows<WEIGHTS>(p, b).tiles();
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) ms.scan[warp] = mine;
  __syncthreads();
  int total = 0;
  for (int i = 0; i < kThreads / 32; ++i) total += ms.scan[i];
  const int G = gridDim.x, per = (total + G - 1) / G;
  const int g0 = min(total, (int)blockIdx.x * per), g1 = min(total, g0 + per);
  if (tid == 0) {
    ms.n_tiles = g1 - g0;
    ms.per_cta = per;
    ms.first_seq = ms.first_tile = 0;
  }
  int carry = 0;
  for (int b0 = 0; b0 < p.n_seq; b0 += kThreads) {
    const int b = b0 + tid;
    const int n = b < p.n_seq ? seq_rows<WEIGHTS>(p, b).tiles() : 0;
    int inc = n;
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    __syncthreads();  // the previous use of scan[] is over
    if (lane == 31) ms.scan[warp] = inc;
    __syncthreads();
    int before = carry;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += ms.scan[i];
      carry += ms.scan[i];
    }
    const int at = before + inc - n;  // tiles before sequence b
    if (n > 0 && at <= g0 && g0 < at + n && g1 > g0) {
      ms.first_seq = b;
      ms.first_tile = g0 - at;
    }
    if (!WEIGHTS && blockIdx.x == 0 && b < p.n_seq) {
      const int c0 = n > 0 ? at / per : 0, c1 = n > 0 ? (at + n - 1) / per : -1;
      p.ws_plan[b] = make_int2(c0 + b, c1 - c0 + 1);
    }
  }
}

// ------------------------------------------------------------------ loaders

template <bool FP8, bool WEIGHTS>
__device__ __forceinline__ void load_role(const PagedAttnParams &p, uint32_t sbase, PMisc &ms, int ltid) {
  constexpr int kGroup = loader_threads<FP8>();
  constexpr int kRowStep = kGroup / 8;
  volatile int *abrt = &ms.abort_flag;
  const int gtid = (FP8 && ltid >= 32) ? ltid - kTile : ltid;  // 0 .. kGroup - 1
  const int c8 = gtid & 7, rsub = gtid >> 3;
  const uint32_t b_q_full = smem_u32(&ms.q_full), b_q_empty = smem_u32(&ms.q_empty);
  const long long vdelta[2] = {p.seg[0].v - p.seg[0].k, p.seg[1].v - p.seg[1].k};
  StageRing ring;
  bool ok = true;
  bool q_issued = false;
  uint32_t n_item = 0, q_par = 0;
  const int nt = ms.n_tiles;

  // The rows of tile `w` into list `g % kLists`.
  auto make_list = [&](const Walk<WEIGHTS> &w, int g) {
    const int buf = g % kLists;
    if (ok && !mbar_wait(smem_u32(&ms.list_empty[buf]), ((g / kLists) & 1) ^ 1, abrt, p.timeout_ns, p.err,
                         PSITE_LIST_EMPTY))
      ok = false;
    if (ok) {
      for (int r = gtid; r < kTile; r += kGroup) {
        const int x = w.j * kTile + r;
        const int sg = x < w.rows.nr ? 0 : 1;
        const int row = sg == 0 ? w.rows.raw_lo + x : x - w.rows.nr;
        unsigned long long at = 0;
        float ksc = 0.f, lvs = 0.f, ivs = 1.f;
        if (x < w.rows.nr + w.rows.nc) {
          const PagedSeg &s = p.seg[sg];
          const int pi = row / s.page_rows, slot = row - pi * s.page_rows;
          const int page = __ldg(s.table + w.b * s.table_stride + pi);
          if ((unsigned)page < (unsigned)s.n_pages) {
            at = reinterpret_cast<unsigned long long>(s.k + page * s.page_stride + slot * s.row_stride) | sg;
            if (FP8) {
              const long long sr = (long long)page * s.page_rows + slot;
              ksc = p.scale_log2 * __ldg(s.k_scale + sr);
              if (!WEIGHTS) {
                lvs = fmaxf(__log2f(__ldg(s.v_scale + sr)), kLeastLog2Scale);
                ivs = exp2f(-lvs);
              }
            }
          }
        }
        ms.row[buf][r] = at;
        if (FP8) {
          ms.ksc[buf][r] = ksc;
          if (!WEIGHTS) {
            ms.lvs[buf][r] = lvs;
            ms.ivs[buf][r] = ivs;
          }
        }
      }
    }
    mbar_arrive(smem_u32(&ms.list_full[buf]));
    ok = !bar_red_or(2, kGroup, !ok);  // the list is complete; all go on or none
  };
  // One part of tile g into the next stage (parts 0-3: K dims 128 part .., 4-7: V).
  auto emit = [&](int g, int part) -> bool {
    if (!mbar_wait(smem_u32(&ms.kv_empty[ring.st]), ring.ph ^ 1, abrt, p.timeout_ns, p.err, PSITE_KV_EMPTY))
      return false;
    const uint32_t stage = sbase + kOffKV + ring.st * kStageBytes;
    const unsigned long long *list = ms.row[g % kLists];
#pragma unroll
    for (int it = 0; it < (kTile + kRowStep - 1) / kRowStep; ++it) {
      const int row = kRowStep * it + rsub;
      if (kTile % kRowStep != 0 && row >= kTile) break;
      const unsigned long long e = list[row];
      const uint32_t n = e != 0 ? 16u : 0u;
      const uint8_t *src = e != 0 ? reinterpret_cast<const uint8_t *>(e & ~15ull) : reinterpret_cast<const uint8_t *>(p.geom);
      if (part >= 4 && e != 0) src += vdelta[e & 1];
      if (FP8) {
        if (e != 0) src += 128 * (part & 3) + 16 * c8;
        cp_async16z(stage + kBoxBytes + row * 128 + 16 * c8, src, n);
      } else {
        if (e != 0) src += 256 * (part & 3) + 16 * c8;
        const uint32_t dst = stage + row * 128 + ((c8 ^ (row & 7)) << 4);
        cp_async16z(dst, src, n);                                // dims 0-63 of the part
        cp_async16z(dst + kBoxBytes, e != 0 ? src + 128 : src, n);  // dims 64-127
      }
    }
    cp_async_arrive(smem_u32(FP8 ? &ms.code_full[ring.st] : &ms.kv_full[ring.st]));
    ring.advance();
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

  Walk<WEIGHTS> w;
  w.start(p, ms);
  if (nt > 0) {
    load_q(w.b);
    make_list(w, 0);
    for (int part = 0; part < 4 && ok; ++part) ok = emit(0, part);
    for (int g = 0; g < nt; ++g) {
      if (g + 1 < nt) {
        w.next(p);
        if (w.first) load_q(w.b);
        make_list(w, g + 1);
        for (int part = 0; part < 4 && ok; ++part) ok = emit(g + 1, part);
      } else {
        ok = !bar_red_or(2, kGroup, !ok);
      }
      if (!WEIGHTS)
        for (int part = 4; part < 8 && ok; ++part) ok = emit(g, part);
    }
  }
  cp_async_done();  // no copy may still be landing at exit
  if (ltid == 0 && q_issued) {
    volatile int never = 0;
    mbar_wait(b_q_full, q_par, &never, 100000000ull, p.err, PSITE_DRAIN);
  }
}

// Warps 9-12 with E4M3 rows: every stage's codes (upper half), one row per
// thread, widened exactly to fp16 in the swizzled layout.  Row r's values
// overwrite only row r's own codes, which its thread has read first.
template <bool WEIGHTS>
__device__ __forceinline__ void convert_role(const PagedAttnParams &p, uint32_t sbase, PMisc &ms, int row) {
  volatile int *abrt = &ms.abort_flag;
  StageRing ring;
  const long long parts = (long long)ms.n_tiles * (WEIGHTS ? 4 : 8);
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
    fence_proxy_async_smem();
    mbar_arrive(smem_u32(&ms.kv_full[ring.st]));
    ring.advance();
  }
}

// ------------------------------------------------------------------ MMA issue

template <bool FP8, bool WEIGHTS>
__device__ __forceinline__ void mma_role_paged(const PagedAttnParams &p, uint32_t sbase, uint32_t tmem, PMisc &ms,
                                               int lane) {
  if (lane == 0) {
    volatile int *abrt = &ms.abort_flag;
    constexpr uint32_t kIdescQK = idesc_f16_f32(128, 64, false, false);
    constexpr uint32_t kIdescPV = idesc_f16_f32(128, 64, true, true);
    const uint64_t k_desc = sdesc_sw128(sbase + kOffKV, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(sbase + kOffKV, kBoxBytes, 1024);
    const uint64_t q_desc = sdesc_sw128(sbase + kOffQ, 16, 1024);
    const uint64_t p_desc = sdesc_sw128(sbase + kOffP, 16, 1024);
    StageRing ring;
    const int nt = ms.n_tiles;
    uint32_t q_item = 0, o_item = 0;
    bool ok = true;
    // Rows copied by cp.async are generic-proxy writes; the fence makes the
    // landed stage visible to the tensor core.
    auto stage_ready = [&]() -> bool {
      if (!mbar_wait(smem_u32(&ms.kv_full[ring.st]), ring.ph, abrt, p.timeout_ns, p.err, PSITE_KV_FULL)) return false;
      if (!FP8) fence_proxy_async_smem();
      tc_fence_after();
      return true;
    };
    auto qk = [&](int g, bool first, bool last) -> bool {
      if (first) {
        if (!mbar_wait(smem_u32(&ms.q_full), q_item & 1, abrt, p.timeout_ns, p.err, PSITE_Q_FULL)) return false;
        ++q_item;
      }
      const uint32_t sb = g & 1;
      if (!mbar_wait(smem_u32(&ms.s_empty[sb]), ((g >> 1) & 1) ^ 1, abrt, p.timeout_ns, p.err, PSITE_S_EMPTY))
        return false;
      tc_fence_after();
      const uint32_t d_s = tmem + kTmemS + 64 * sb;
      for (int c = 0; c < 4; ++c) {
        if (!stage_ready()) return false;
        const uint64_t a0 = sdesc_add(k_desc, ring.st * kStageBytes);
        const uint64_t b0 = sdesc_add(q_desc, 2 * c * kQBoxBytes);
#pragma unroll
        for (int b2 = 0; b2 < 2; ++b2) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t a = sdesc_add(a0, b2 * kBoxBytes + ks * 32);
            const uint64_t b = sdesc_add(b0, b2 * kQBoxBytes + ks * 32);
            if (b2 == 0 && ks == 0)
              umma_f16(d_s, a, b, kIdescQK, c != 0 ? 1u : 0u);
            else
              umma_f16_acc(d_s, a, b, kIdescQK);
          }
        }
        umma_commit(smem_u32(&ms.kv_empty[ring.st]));
        ring.advance();
      }
      umma_commit(smem_u32(&ms.s_full[sb]));
      if (last) umma_commit(smem_u32(&ms.q_empty));
      return true;
    };
    auto pv = [&](int g, bool first, bool last) -> bool {
      if (!mbar_wait(smem_u32(&ms.p_full), g & 1, abrt, p.timeout_ns, p.err, PSITE_P_FULL)) return false;
      if (first) {
        if (!mbar_wait(smem_u32(&ms.o_empty), (o_item & 1) ^ 1, abrt, p.timeout_ns, p.err, PSITE_O_EMPTY))
          return false;
        ++o_item;
      }
      tc_fence_after();
      for (int m = 0; m < 4; ++m) {
        if (!stage_ready()) return false;
        const uint64_t a0 = sdesc_add(v_desc, ring.st * kStageBytes);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint64_t a = sdesc_add(a0, ks * 2048);
          const uint64_t b = sdesc_add(p_desc, ks * 2048);
          if (ks == 0)
            umma_f16(tmem + 64 * m, a, b, kIdescPV, first ? 0u : 1u);
          else
            umma_f16_acc(tmem + 64 * m, a, b, kIdescPV);
        }
        umma_commit(smem_u32(&ms.kv_empty[ring.st]));
        if (last) umma_commit(smem_u32(&ms.o_full[m]));
        ring.advance();
      }
      umma_commit(smem_u32(&ms.p_empty));
      return true;
    };
    Walk<WEIGHTS> w;
    w.start(p, ms);
    if (nt > 0) ok = qk(0, true, w.last);
    for (int g = 0; g < nt && ok; ++g) {
      const bool first = w.first, last = w.last;
      if (g + 1 < nt) {
        w.next(p);
        ok = qk(g + 1, w.first, w.last);
      }
      if (!WEIGHTS) ok = ok && pv(g, first, last);
    }
    umma_commit(smem_u32(&ms.mma_done));
    volatile int never = 0;
    mbar_wait(smem_u32(&ms.mma_done), 0, &never, 100000000ull, p.err, PSITE_DRAIN);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax and epilogue

template <bool FP8>
__device__ __forceinline__ void softmax_role(const PagedAttnParams &p, uint8_t *smem, uint32_t tmem, PMisc &ms,
                                             int tid) {
  volatile int *abrt = &ms.abort_flag;
  const int wq = tid >> 5, l = tid & 31;
  const int q = wq & 3, hh = wq >> 2;  // TMEM lane quarter, head half
  const int r = 32 * q + l;            // row of the tile, or dim of a 128-dim block
  const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
  const uint32_t col0 = 32 * hh;
  const int nt = ms.n_tiles;
  bool bad = false;
  uint32_t n_item = 0;
  float m_ref = -INFINITY;  // reference of head `tid` (threads < 64), log2 units
  float lpart[32];
  int first_j = 0;
  Walk<false> w;
  w.start(p, ms);
  for (int g = 0; g < nt; ++g) {
    if (g > 0) w.next(p);
    if (w.first) {
      first_j = w.j;
      m_ref = -INFINITY;
#pragma unroll
      for (int h = 0; h < 32; ++h) lpart[h] = 0.f;
    }
    const int buf = g % kLists;
    const uint32_t sb = g & 1;
    bad = bad || !mbar_wait(smem_u32(&ms.list_full[buf]), (g / kLists) & 1, abrt, p.timeout_ns, p.err, PSITE_LIST_FULL);
    const bool vis = ms.row[buf][r] != 0;
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
#pragma unroll
    for (int h = 0; h < 32; ++h) s[h] = vis ? fmaf(s[h], sl2, lvs) : -INFINITY;

    ms.red[q][col0 + l] = reduce_heads<true>(s, l);
    if (bar_red_or(1, kComputeThreads, bad)) break;
    if (tid < kH) {
      const float tmax = fmaxf(fmaxf(ms.red[0][tid], ms.red[1][tid]), fmaxf(ms.red[2][tid], ms.red[3][tid]));
      float alpha = 1.f;
      if (m_ref == -INFINITY) {
        m_ref = tmax;
      } else if (tmax > m_ref + kTau) {  // the reference moves only when P would pass 2^8
        alpha = exp2f(m_ref - tmax);
        m_ref = tmax;
      }
      ms.m_use[tid] = m_ref == -INFINITY ? 0.f : m_ref;
      ms.alpha[tid] = alpha;
      if (alpha != 1.f) ms.resc_flag[g & 1] = 1;
    }
    bar_sync_id(1, kComputeThreads);
    const int resc = ms.resc_flag[g & 1];
    if (tid == 0) ms.resc_flag[(g + 1) & 1] = 0;
    bad = bad || !mbar_wait(smem_u32(&ms.p_empty), (g & 1) ^ 1, abrt, p.timeout_ns, p.err, PSITE_P_EMPTY);
    if (resc) {
      float al[32];
      load_row32(ms.alpha + col0, al);
#pragma unroll
      for (int h = 0; h < 32; ++h) lpart[h] *= al[h];
    }
    {
      // P^T row r: heads 32hh .. +31 are 16-byte chunks 4hh .. 4hh+3 of its
      // 128 bytes, chunk c at c ^ (r & 7).  P is rounded once to fp16 for the
      // MMA; the row sums add it unrounded, so lse keeps fp32 precision (the
      // two differ by rounding errors that average out over the rows).
      uint8_t *prow = smem + kOffP + r * 128;
      const bool dead = FP8 && lvs <= kLeastLog2Scale;  // a V scale of 0: weight, but no value
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 m0 = reinterpret_cast<const float4 *>(ms.m_use + col0)[2 * c];
        const float4 m1 = reinterpret_cast<const float4 *>(ms.m_use + col0)[2 * c + 1];
        const float mu[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
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
    if (resc && !w.first) {
      float al[32];
      load_row32(ms.alpha + col0, al);
      tc_fence_after();
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        float o[32];
        tmem_ld32(tmem + 64 * m + col0 + lane_base, o);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 32; ++h) o[h] *= al[h];
        tmem_st32(tmem + 64 * m + col0 + lane_base, o);
      }
      tmem_wait_st();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    mbar_arrive(smem_u32(&ms.p_full));
    if (!w.last) continue;

    // End of an item: row sums, then o block by block as the last PV finishes them.
    const bool whole = w.whole(first_j);
    const long long slot = (long long)blockIdx.x + w.b;
    ms.red[q][col0 + l] = reduce_heads<false>(lpart, l);
    if (bar_red_or(1, kComputeThreads, bad)) break;
    if (tid < kH) {
      const float lsum = ms.red[0][tid] + ms.red[1][tid] + ms.red[2][tid] + ms.red[3][tid];
      ms.inv_l[tid] = lsum > 0.f ? 1.f / lsum : 0.f;
      if (!whole) {
        p.ws_ml[slot * kH + tid] = make_float2(lsum > 0.f ? m_ref : -INFINITY, lsum);
      } else if (p.lse != nullptr) {
        p.lse[(long long)w.b * kH + tid] = lsum > 0.f ? (m_ref + log2f(lsum)) * kLn2 : -INFINITY;
      }
    }
    bar_sync_id(1, kComputeThreads);
    float inv[32];
    load_row32(ms.inv_l + col0, inv);
    const bool odd = l & 1;
    __half *obase = whole ? p.o + w.b * p.o_stride + (long long)col0 * kD + (r & ~1)
                          : p.ws_o + (slot * kH + col0) * kD + (r & ~1);
#pragma unroll 1
    for (int m = 0; m < 4; ++m) {
      bad = bad || !mbar_wait(smem_u32(&ms.o_full[m]), n_item & 1, abrt, p.timeout_ns, p.err, PSITE_O_FULL);
      tc_fence_after();
      float o[32];
      tmem_ld32(tmem + 64 * m + col0 + lane_base, o);
      tmem_wait_ld();
#pragma unroll
      for (int h = 0; h < 32; h += 2) {
        const float a = o[h] * inv[h], c = o[h + 1] * inv[h + 1];
        const float got = __shfl_xor_sync(0xffffffffu, odd ? a : c, 1);
        const __half2 v = odd ? __floats2half2_rn(got, c) : __floats2half2_rn(a, got);
        *reinterpret_cast<__half2 *>(obase + (h + (odd ? 1 : 0)) * kD + 128 * m) = v;
      }
    }
    tc_fence_before();
    mbar_arrive(smem_u32(&ms.o_empty));
    ++n_item;
    if (bar_red_or(1, kComputeThreads, bad)) break;
  }
}

// Weights: row r of a tile is TMEM lane r; each head half adds its 32 heads'
// exponentials in registers and the halves meet in shared memory.
template <bool FP8>
__device__ __forceinline__ void weights_role(const PagedAttnParams &p, uint32_t tmem, PMisc &ms, int tid) {
  volatile int *abrt = &ms.abort_flag;
  const int wq = tid >> 5, l = tid & 31;
  const int q = wq & 3, hh = wq >> 2;
  const int r = 32 * q + l;
  const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
  const uint32_t col0 = 32 * hh;
  const int nt = ms.n_tiles;
  bool bad = false;
  float *part = &ms.red[0][0];  // [2][128] by tile parity (256 floats)
  Walk<true> w;
  w.start(p, ms);
  for (int g = 0; g < nt; ++g) {
    if (g > 0) w.next(p);
    if (w.first) {
      // 2^(s - lse log2 e); a head whose lse is -inf gave no weight to anything.
      bar_sync_id(1, kComputeThreads);
      if (tid < kH) {
        const float v = p.lse_in[(long long)w.b * kH + tid];
        ms.m_use[tid] = v == -INFINITY ? INFINITY : v * kLog2e;
      }
      bar_sync_id(1, kComputeThreads);
    }
    const int buf = g % kLists;
    const uint32_t sb = g & 1;
    const int c = w.j * kTile + r;
    const bool mine = hh == 0 && c < w.rows.nc;
    const float before = mine && p.acc_in != nullptr ? p.acc_in[w.b * p.acc_in_stride + c] : 0.f;
    bad = bad || !mbar_wait(smem_u32(&ms.list_full[buf]), (g / kLists) & 1, abrt, p.timeout_ns, p.err, PSITE_LIST_FULL);
    const bool vis = ms.row[buf][r] != 0;
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
      p.acc_out[w.b * p.acc_out_stride + c] = fmaf(p.decay, before, got);
    }
  }
}

// ------------------------------------------------------------------ kernel

template <bool FP8, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  PMisc &ms = *reinterpret_cast<PMisc *>(smem + kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    ms.resc_flag[0] = ms.resc_flag[1] = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_q);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ms.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  grid_launch_dependents();
  grid_dependency_wait();  // the plan reads the sequences' geometry
  plan_cta<WEIGHTS>(p, ms);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  if (warp < kComputeWarps) {
    if (WEIGHTS)
      weights_role<FP8>(p, tmem, ms, threadIdx.x);
    else
      softmax_role<FP8>(p, smem, tmem, ms, threadIdx.x);
  } else if (warp == kMmaWarp) {
    mma_role_paged<FP8, WEIGHTS>(p, sbase, tmem, ms, lane);
  } else {
    const int ltid = threadIdx.x - 32 * kLoaderWarp0;
    if (FP8 && ltid >= 32 && ltid < 32 + kTile)
      convert_role<WEIGHTS>(p, sbase, ms, ltid - 32);
    else
      load_role<FP8, WEIGHTS>(p, sbase, ms, ltid);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ merge
// One block per (sequence, head): with M = max_s m_s and W_s = 2^(m_s - M) l_s,
//   o = sum_s W_s o_s / L,  L = sum_s W_s,  lse = (M + log2 L) ln 2.
// A sequence one CTA finished alone (one slot) is left alone; one without
// rows (no slot) gets o = 0 and lse = -inf.  Eight threads of 16 bytes cover 64
// dims, the block 512 dims of four slots at a time.

constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedAttnParams p) {
  __shared__ float part[kMergeThreads / 64][kD];
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = blockIdx.x / kH, h = blockIdx.x - b * kH;
  const int tid = threadIdx.x, grp = tid >> 6, v = tid & 63;
  const int2 plan = __ldg(p.ws_plan + b);
  if (plan.y == 1) return;
  const long long base = plan.x;
  float M = -INFINITY;
  for (int s = 0; s < plan.y; ++s) M = fmaxf(M, p.ws_ml[(base + s) * kH + h].x);
  float L = 0.f;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  for (int s = 0; s < plan.y; ++s) {
    const float2 ml = p.ws_ml[(base + s) * kH + h];
    const float wgt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M) * ml.y;
    L += wgt;
    if ((s & 3) == grp) {
      const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p.ws_o + ((base + s) * kH + h) * kD) + v);
      const __half2 *h2 = reinterpret_cast<const __half2 *>(&x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(h2[e]);
        acc[2 * e] = fmaf(wgt, f.x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(wgt, f.y, acc[2 * e + 1]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) part[grp][8 * v + e] = acc[e];
  __syncthreads();
  const float inv = L > 0.f ? 1.f / L : 0.f;
  float2 o = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kMergeThreads / 64; ++i) {
    o.x += part[i][2 * tid];
    o.y += part[i][2 * tid + 1];
  }
  *reinterpret_cast<__half2 *>(p.o + b * p.o_stride + (long long)h * kD + 2 * tid) =
      __floats2half2_rn(o.x * inv, o.y * inv);
  if (p.lse != nullptr && tid == 0)
    p.lse[(long long)b * kH + h] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
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

cudaError_t launch_paged_decode(const PagedAttnParams &p, bool e4m3, int grid, cudaStream_t s) {
  return launch_pdl(e4m3 ? (const void *)paged_attn_kernel<true, false> : (const void *)paged_attn_kernel<false, false>,
                    p, grid, kThreads, kPagedSmem, s);
}

cudaError_t launch_paged_merge(const PagedAttnParams &p, cudaStream_t s) {
  return launch_pdl((const void *)paged_merge_kernel, p, p.n_seq * kH, kMergeThreads, 0, s);
}

cudaError_t launch_paged_weights(const PagedAttnParams &p, bool e4m3, int grid, cudaStream_t s) {
  return launch_pdl(e4m3 ? (const void *)paged_attn_kernel<true, true> : (const void *)paged_attn_kernel<false, true>,
                    p, grid, kThreads, kPagedSmem, s);
}

cudaError_t prepare_paged_kernels() {
  for (const void *f : {(const void *)paged_attn_kernel<false, false>, (const void *)paged_attn_kernel<true, false>,
                        (const void *)paged_attn_kernel<false, true>, (const void *)paged_attn_kernel<true, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPagedSmem);
    if (e != cudaSuccess) return e;
  }
  cudaFuncAttributes a;
  return cudaFuncGetAttributes(&a, (const void *)paged_merge_kernel);
}

}  // namespace ds4a
