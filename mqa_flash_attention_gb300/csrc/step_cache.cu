// The whole-number work around a step with several new tokens per sequence:
// page tables and slots from the rows that sequences have and want, the path of
// drafted tokens that the model agrees with, and the accepted tokens' rows moved
// into place.
#include "internal.h"
#include "ptx.cuh"
#include "step_params.h"

namespace ds4a {

namespace {

// ------------------------------------------------------------------ page tables
// Sequence b holds pages 0 .. held-1 of its table, gives back the first `gone`
// and those from `need` on, and takes max(0, need - held) new ones (all in the
// numbering before the call).  What a page costs is a table entry and an entry
// of the free list; the order (given back by sequence and entry, then taken by
// sequence and entry from the list's end) makes the result one of whole numbers
// that no order of execution changes.  The list's top has to be known before the
// first page is taken, so one CTA adds up and gives back first; taking pages,
// closing the gap of the dropped ones and naming the slots of new rows is a CTA's
// work for each sequence, in a second kernel because there are many.  Bounded by
// two launches and their round trips to L2 (the bytes would take less than 1 us):
// 15.6 us for a call that takes 8 rows' room for each of 64 sequences and one that
// gives it back, 31 us for two of 1,024 sequences of which each takes 500 rows in
// pages of 16.

constexpr int kListThreads = 1024;
constexpr int kListWarps = kListThreads / 32;
constexpr int kByWarps = 128;  // up to here, more than kFewPages / 8 pages are a warp's work
constexpr int kFewPages = 64;  // given back by a sequence: beyond, always a warp's
constexpr int kFillThreads = 128;
constexpr int kFillSlots = 8;  // padding slots of a thread

struct Pages {
  int have, want, held, need, gone;
  __device__ __forceinline__ int grow() const { return max(0, need - held); }
  __device__ __forceinline__ int rows() const { return max(0, want - have); }
};

__device__ __forceinline__ Pages pages_of(const PageTablesParams &p, int b) {
  Pages x;
  const int cap = p.max_pages * p.page_rows;  // at most 2^30
  x.have = min(max(p.have[b], 0), cap);
  x.gone = p.drop == nullptr ? 0 : min(max(p.drop[b], 0), x.have) / p.page_rows;
  // (Wanted rows may pass the table by what the dropped pages make room for.)
  x.want = (int)min((long long)max(p.want[b], 0), (long long)cap + (long long)x.gone * p.page_rows);
  x.held = (x.have + p.page_rows - 1) / p.page_rows;
  x.need = max((int)(((long long)x.want + p.page_rows - 1) / p.page_rows), x.gone);
  return x;
}

// The pages that sequence b gives back, by one lane, eight loads in flight, or by a
// whole warp: f(page, how many came before in this sequence); returns how many.
// A round trip to L2 is what a step costs.  All of n_seq sequences by lanes take
// n / 8 of them, by 32 warps n_seq / 32 * n / 32: lanes are ahead from 128
// sequences on (a call that takes and one that gives back, 1,024 sequences of up to
// 50 pages: 31 us by lanes, 34 by warps; 64 of up to 64 pages: 17.5 and 15.9).
template <class F>
__device__ __forceinline__ int given_back_lane(const PageTablesParams &p, int b, int gone, int need, int held, F f) {
  const int32_t *row = p.table + b * p.table_stride;
  const int n = gone + max(0, held - need);
  int before = 0;
  for (int i0 = 0; i0 < n; i0 += 8) {
    int page[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k;
      page[k] = i < n ? row[i < gone ? i : need + i - gone] : -1;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if ((unsigned)page[k] < (unsigned)p.n_pages) f(page[k], before++);
    }
  }
  return before;
}

template <class F>
__device__ __forceinline__ int given_back_warp(const PageTablesParams &p, int b, int gone, int need, int held,
                                               int lane, F f) {
  const int32_t *row = p.table + b * p.table_stride;
  const int n = gone + max(0, held - need);
  int before = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int page = i < n ? row[i < gone ? i : need + i - gone] : -1;
    const bool valid = (unsigned)page < (unsigned)p.n_pages;
    const unsigned who = __ballot_sync(0xffffffffu, valid);
    if (valid) f(page, before + __popc(who & ((1u << lane) - 1)));
    before += __popc(who);
  }
  return before;
}

// Sum over a warp's lanes up to this one, in 64 bits (new rows of many sequences may
// pass 32).
__device__ __forceinline__ long long scan_lanes(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

__global__ void __launch_bounds__(kListThreads, 1) page_lists_kernel(const PageTablesParams p) {
  __shared__ long long warp_sum[3][kListWarps], at_of[kListThreads];
  __shared__ int3 warp_job[kListThreads];  // gone, need, held; zeros: a lane does it
  __shared__ int back_of[kListThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_launch_dependents();
  grid_dependency_wait();
  const int start = min(max(p.n_free[0], 0), p.n_pages);
  long long top = start, need_all = 0, rows_all = 0;  // before this round
  for (int b0 = 0; b0 < p.n_seq; b0 += kListThreads) {
    const int b = b0 + tid, n_here = min(kListThreads, p.n_seq - b0);
    const bool live = b < p.n_seq;
    Pages x = {0, 0, 0, 0, 0};
    if (live) x = pages_of(p, b);
    // A lane counts what its sequence gives back where that is little; the warps
    // take the other sequences in turn.
    const int n_back = x.gone + max(0, x.held - x.need);
    const bool few = n_back <= (n_here > kByWarps ? kFewPages : kFewPages / 8);
    warp_job[tid] = few ? make_int3(0, 0, 0) : make_int3(x.gone, x.need, x.held);
    back_of[tid] = few ? given_back_lane(p, b, x.gone, x.need, x.held, [](int, int) {}) : 0;
    const bool any_many = __syncthreads_or(!few);
    if (any_many) {
      for (int s = warp; s < n_here; s += kListWarps) {
        const int3 j = warp_job[s];
        const int n = given_back_warp(p, b0 + s, j.x, j.y, j.z, lane, [](int, int) {});
        if (lane == 0 && n > 0) back_of[s] = n;
      }
      __syncthreads();
    }
    const int back = back_of[tid];
    // Sums over the sequences before this one: given back, taken, new rows.
    const long long own[3] = {back, live ? x.grow() : 0, live ? x.rows() : 0};
    long long before[3], all[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      before[k] = scan_lanes(own[k], lane);
      if (lane == 31) warp_sum[k][warp] = before[k];
      before[k] -= own[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const long long v = scan_lanes(warp_sum[k][lane], lane);
      all[k] = __shfl_sync(0xffffffffu, v, 31);
      const long long w = __shfl_sync(0xffffffffu, v, max(warp - 1, 0));
      if (warp > 0) before[k] += w;
    }
    if (live) {
      p.plan[b] = PagePlan{need_all + before[1], rows_all + before[2]};
      p.first[b] = (int)min(rows_all + before[2], (long long)p.n_slots);
    }
    const long long at = top + before[0];
    if (few) {
      given_back_lane(p, b, x.gone, x.need, x.held, [&](int page, int i) {
        if (at + i < p.n_pages) p.free_pages[at + i] = page;
      });
    }
    if (any_many) {
      at_of[tid] = at;
      __syncthreads();
      for (int s = warp; s < n_here; s += kListWarps) {
        const int3 j = warp_job[s];
        const long long at_s = at_of[s];
        given_back_warp(p, b0 + s, j.x, j.y, j.z, lane, [&](int page, int i) {
          if (at_s + i < p.n_pages) p.free_pages[at_s + i] = page;
        });
      }
    }
    top += all[0];
    need_all += all[1];
    rows_all += all[2];
    __syncthreads();  // the sums have been read
  }
  if (tid == 0) {
    // A list that holds every page takes no more (the same page given back twice).
    top = min(top, (long long)p.n_pages);
    p.plan[p.n_seq] = PagePlan{top, rows_all};
    p.first[p.n_seq] = (int)min(rows_all, (long long)p.n_slots);
    p.n_free[0] = (int)max(0ll, top - need_all);
    p.n_short[0] = (int)min(max(0ll, need_all - top), (long long)INT32_MAX);
  }
}

__global__ void __launch_bounds__(kFillThreads) page_fill_kernel(const PageTablesParams p) {
  const int tid = threadIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  const PagePlan total = p.plan[p.n_seq];
  if ((int)blockIdx.x >= p.n_seq) {
    // Slots behind the last new row.
    const long long i0 = (long long)(blockIdx.x - p.n_seq) * kFillThreads * kFillSlots + tid;
#pragma unroll
    for (int u = 0; u < kFillSlots; ++u) {
      const long long i = i0 + u * kFillThreads;
      if (i >= total.rows && i < p.n_slots) p.slots[i] = -1;
    }
    return;
  }
  const int b = blockIdx.x;
  const Pages x = pages_of(p, b);
  const PagePlan at = p.plan[b];
  int32_t *row = p.table + b * p.table_stride;
  // The k-th page taken overall is the k-th from the list's end.
  auto taken = [&](int i) {
    const long long k = total.pages - 1 - (at.pages + i);
    return k >= 0 ? p.free_pages[k] : -1;
  };
  // The kept pages move down by `gone`, a block's width at a time, each read
  // before any entry of its step is written; new ones follow, and what was
  // given back is marked.
  const int kept = min(x.held, x.need) - x.gone, used = max(x.held, x.need - x.gone);
  if (x.gone > 0) {
    for (int i0 = 0; i0 < kept; i0 += kFillThreads) {
      const int i = i0 + tid;
      const int v = i < kept ? row[i + x.gone] : 0;
      __syncthreads();
      if (i < kept) row[i] = v;
      __syncthreads();
    }
  }
  for (int i = kept + tid; i < used; i += kFillThreads) row[i] = i < x.need - x.gone ? taken(i - kept) : -1;
  __syncthreads();
  const int n = x.rows();
  for (int j = tid; j < n; j += kFillThreads) {
    const long long to = at.rows + j;
    if (to >= p.n_slots) break;
    const int r = x.have - x.gone * p.page_rows + j;  // in the new numbering
    const int pi = r / p.page_rows, page = row[pi];
    p.slots[to] = (unsigned)page < (unsigned)p.n_pages ? page * p.page_rows + (r - pi * p.page_rows) : -1;
  }
}

// ------------------------------------------------------------------ acceptance
// A warp per sequence walks from node to node: the next is the lowest child of
// the last one whose token is the one chosen there.  Children come after their
// parent, so up to 128 nodes (four a lane) stay in registers and a step is four
// votes; of longer sequences each step reads on from the last accepted node.
// Bounded by the launch and two round trips: 3.3 us for one tree of 8 nodes, 4.1 us
// for 512 trees of 64 (0.4 MB, 0.06 us).

constexpr int kAcceptWarps = 4;
constexpr int kHeldNodes = 4;  // nodes of a lane

__global__ void __launch_bounds__(32 * kAcceptWarps) tree_accept_kernel(const AcceptParams p) {
  const int lane = threadIdx.x & 31, b = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5);
  grid_launch_dependents();
  grid_dependency_wait();
  if (b >= p.n_seq) return;
  const int t0 = min(max(p.first[b], 0), p.n_tok), n = min(max(p.first[b + 1], t0), p.n_tok) - t0;
  const int32_t *parent = p.parent == nullptr ? nullptr : p.parent + t0;
  const int32_t *token = p.token + t0, *target = p.target + t0;
  int32_t *path = p.path + b * p.path_stride;
  auto parent_of = [&](int t) {
    if (parent == nullptr) return t - 1;
    const int u = parent[t];
    return u >= 0 && u < t ? u : -1;
  };
  int par[kHeldNodes], tok[kHeldNodes], tgt[kHeldNodes];
  const bool held = n <= 32 * kHeldNodes;
  if (held) {
#pragma unroll
    for (int u = 0; u < kHeldNodes; ++u) {
      const int t = 32 * u + lane;
      par[u] = t < n ? parent_of(t) : -2;
      tok[u] = t < n ? token[t] : 0;
      tgt[u] = t < n ? target[t] : 0;
    }
  }
  int at = -1, count = 0;
  int want = p.prev != nullptr ? p.prev[b] : -1;
  bool any = p.prev == nullptr;  // the first root, whatever its token
  while (count < p.width) {
    int next = -1;
    if (held) {
#pragma unroll
      for (int u = 0; u < kHeldNodes; ++u) {
        const unsigned who = __ballot_sync(0xffffffffu, par[u] == at && (any || tok[u] == want));
        if (next < 0 && who != 0) next = 32 * u + __ffs(who) - 1;
      }
    } else {
      for (int c0 = at + 1; c0 < n && next < 0; c0 += 32) {
        const int t = c0 + lane;
        const unsigned who =
            __ballot_sync(0xffffffffu, t < n && parent_of(t) == at && (any || token[t] == want));
        if (who != 0) next = c0 + __ffs(who) - 1;
        if (parent == nullptr) break;  // a chain's only child is the next node
      }
    }
    if (next < 0) break;
    if (held) {
      int v = 0;
#pragma unroll
      for (int u = 0; u < kHeldNodes; ++u)
        if (next >> 5 == u) v = tgt[u];
      want = __shfl_sync(0xffffffffu, v, next & 31);
    } else {
      want = target[next];
    }
    any = false;
    at = next;
    if (lane == 0) path[count] = next;
    ++count;
  }
  for (int i = count + lane; i < p.width; i += 32) path[i] = -1;
  if (lane == 0) {
    p.n_accepted[b] = count;
    p.next[b] = want;
  }
}

// ------------------------------------------------------------------ commit
// Row n_raw + path[i] moves to row n_raw + i.  Along a path (ascending, path[i]
// >= i) no move writes a row that a later one reads, so a thread that owns 16
// bytes of every row may read several rows ahead and writes them in order; a
// block per sequence and pool.  Scales are read by a block's width, then written.
// The rows' bytes take 1 us at most here; what it waits for are round trips, of
// the path, the table and each group of rows.  16 rows ahead: 3.0 us for 32 paths of
// up to 16 fp16 rows in two pools, 4.9 us for 256 of up to 64 E4M3 rows (8 rows: 3.8
// and 10.0 us; 32, which no longer fit the registers: 4.5 and 10.6 us).

constexpr int kMoves = 64;     // moves whose addresses are found at once, one a thread
constexpr int kRowsAhead = 16;

__global__ void __launch_bounds__(kMoves) commit_paged_kernel(const CommitParams p, int pools) {
  __shared__ long long from[kMoves], to[kMoves];  // bytes, -1: no move
  const int tid = threadIdx.x;
  const int b = blockIdx.x / pools, which = blockIdx.x - b * pools;
  grid_launch_dependents();
  grid_dependency_wait();
  const bool e4m3 = p.rows.k_scale != nullptr;
  uint8_t *pool = const_cast<uint8_t *>(which == 0 ? p.rows.k : p.rows.v);
  // One row that serves as K and V may have a scale array for each.
  float *scale0 = const_cast<float *>(which == 0 ? p.rows.k_scale : p.rows.v_scale);
  float *scale1 = pools == 1 && p.rows.v_scale != p.rows.k_scale ? const_cast<float *>(p.rows.v_scale) : nullptr;
  const int n = min(max(p.n_accepted[b], 0), p.width);
  const int base = max(p.geom[b].y, 0);
  const int32_t *path = p.path + b * p.path_stride;
  const int32_t *table = p.rows.table + b * p.rows.table_stride;
  // A row's place: (page, slot), page -1 where there is none.
  auto place = [&](long long r) {
    if (r >= p.rows.max_rows) return make_int2(-1, 0);
    const int pi = (int)r / p.rows.page_rows, page = table[pi];
    return make_int2((unsigned)page < (unsigned)p.rows.n_pages ? page : -1, (int)r - pi * p.rows.page_rows);
  };
  const int chunks = e4m3 ? 32 : 64;  // 16-byte pieces of a row
  for (int i0 = 0; i0 < n; i0 += kMoves) {
    const int i = i0 + tid;
    long long f = -1, t = -1;
    float s0 = 0.f, s1 = 0.f;
    long long st = -1;
    if (i < n) {
      const int u = path[i];
      if (u > i) {
        const int2 src = place((long long)base + u), dst = place((long long)base + i);
        if (src.x >= 0 && dst.x >= 0) {
          f = src.x * p.rows.page_stride + src.y * p.rows.row_stride;
          t = dst.x * p.rows.page_stride + dst.y * p.rows.row_stride;
          if (e4m3) {
            const long long sf = (long long)src.x * p.rows.page_rows + src.y;
            st = (long long)dst.x * p.rows.page_rows + dst.y;
            s0 = scale0[sf];
            if (scale1 != nullptr) s1 = scale1[sf];
          }
        }
      }
    }
    from[tid] = f;
    to[tid] = t;
    __syncthreads();
    if (st >= 0) {
      scale0[st] = s0;
      if (scale1 != nullptr) scale1[st] = s1;
    }
    const int here = min(kMoves, n - i0);
    if (tid < chunks) {
      for (int j0 = 0; j0 < here; j0 += kRowsAhead) {
        uint4 v[kRowsAhead];
#pragma unroll
        for (int k = 0; k < kRowsAhead; ++k)
          if (j0 + k < here && from[j0 + k] >= 0)
            v[k] = *reinterpret_cast<const uint4 *>(pool + from[j0 + k] + 16 * tid);
#pragma unroll
        for (int k = 0; k < kRowsAhead; ++k)
          if (j0 + k < here && from[j0 + k] >= 0) *reinterpret_cast<uint4 *>(pool + to[j0 + k] + 16 * tid) = v[k];
      }
    }
    __syncthreads();  // scales and addresses of the next moves
  }
}

template <class... A>
cudaError_t launch_pdl(void (*f)(A...), unsigned grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, args...);
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesParams &p, cudaStream_t s) {
  const cudaError_t e = launch_pdl(page_lists_kernel, 1, kListThreads, s, p);
  if (e != cudaSuccess) return e;
  const int per = kFillThreads * kFillSlots;
  return launch_pdl(page_fill_kernel, (unsigned)(p.n_seq + ((long long)p.n_slots + per - 1) / per), kFillThreads, s, p);
}

cudaError_t launch_accept(const AcceptParams &p, cudaStream_t s) {
  return launch_pdl(tree_accept_kernel, (unsigned)((p.n_seq + kAcceptWarps - 1) / kAcceptWarps), 32 * kAcceptWarps, s,
                    p);
}

cudaError_t launch_commit(const CommitParams &p, cudaStream_t s) {
  const int pools = p.rows.v != p.rows.k ? 2 : 1;
  return launch_pdl(commit_paged_kernel, (unsigned)(p.n_seq * pools), kMoves, s, p, pools);
}

cudaError_t preload_step_kernels() {
  for (const void *f : {(const void *)page_lists_kernel, (const void *)page_fill_kernel,
                        (const void *)tree_accept_kernel, (const void *)commit_paged_kernel}) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ds4a
