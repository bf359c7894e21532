// Cache-page operators (include/pa_pages.h): bookkeeping of block_table,
// refcount and past on the device, and the copies of page contents.
//
// Bookkeeping (what to copy, which free page goes where) is a chain of short
// dependent steps over a few thousand integers, bound by latency: counts,
// prefix sums and lists that depend on all counts before. Each call's chain
// runs in ONE cluster of kClusterCtas CTAs, whose hardware barrier orders the
// steps (a grid-wide order would need one launch per step). The 256 warps of
// the cluster each own a contiguous range of the pages and of the call's
// sequences; a warp's counts go to every CTA's shared memory, and a warp's
// base is the sum of the counts of the warps before it. Ranks inside a warp's
// range come from ballots. All of it is integer arithmetic in a fixed order,
// so the result does not depend on the order the GPU works in.
//
// Contents are moved by a second kernel (launched early, it waits for the
// first): a warp copies 4 KB of a page at a time, 16 bytes per lane and load,
// eight loads in flight per lane. A copy of a few pairs is one kernel, which
// checks the pairs itself. Bound by HBM, two bytes of traffic per byte copied:
// 768 pages of 73 KB, half filled on average, in 16 layers (920 MB of traffic)
// take 146 us, 6.3 TB/s, 0.93 of a plain copy's rate; a compaction that moves
// 2.3 GB 357 us, 6.5 TB/s. The bookkeeping before it: a fork of 256 sequences 15
// us, a reserve for 512 rows on 131072 pages 17 us, a compaction's plan 7 to 10 us.
// Looking at eight pieces at once to skip those behind the rows to copy gained
// nothing.
#include <climits>
#include <cstdarg>
#include <cstdio>

#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_pages.h"

namespace pa {
namespace pages {
namespace {

namespace cg = cooperative_groups;

constexpr int kClusterCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kClusterCtas * kPlanThreads / 32;  // 256
constexpr int kMaxBlocks = 1 << 22;  // pages, and rows of the table: sums over 256 warps fit int32
// Up to this many tokens the cluster of reserve fills the slots itself; more are
// left to a kernel of their own. GPU time of a step of 512 rows, in the cluster
// and apart: 16 k tokens 23.7 and 24.8 us, 32 k 27.7 and 25.7, 96 k 34.9 and 28.8.
constexpr int64_t kClusterTokens = 24576;
constexpr int kMaxCaches = 128;  // caches of one copy launch (more: several launches)
constexpr int kPieceBytes = 4096;  // bytes one warp copies at a time

struct State {
  int32_t* table;
  int32_t* past;
  int32_t* ref;
  int32_t* err;
  int num_blocks, bs, max_blocks, num_seqs;
};

// Workspace arrays (every call uses a part of them).
struct Scratch {
  int4* pairs;     // [num_blocks] (source, destination, rows, -) of the copies
  int32_t* list;   // [num_blocks] free pages to hand out, lowest first
  int32_t* mark;   // [max(num_blocks, num_seqs)] claims / new page ids
  int32_t* need;   // [num_seqs] pages a sequence lacks (-1: it gets none)
  int32_t* count;  // [1] pairs to copy
};

__host__ __device__ inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t layout(const pa_pages_params& p, char* base, Scratch* s) {
  const size_t nb = (size_t)p.num_blocks, ns = (size_t)p.num_seqs;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += up256(bytes);
    return base ? base + a : nullptr;
  };
  Scratch t;
  t.pairs = reinterpret_cast<int4*>(take((nb > ns ? nb : ns) * sizeof(int4)));
  t.list = reinterpret_cast<int32_t*>(take(nb * 4));
  t.mark = reinterpret_cast<int32_t*>(take((nb > ns ? nb : ns) * 4));
  t.need = reinterpret_cast<int32_t*>(take(ns * 4));
  t.count = reinterpret_cast<int32_t*>(take(4));
  if (s) *s = t;
  return at;
}

// Loads of what another CTA wrote before the last barrier: past L1, in place.
__device__ __forceinline__ int fresh(const int32_t* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ int4 fresh(const int4* p) {
  int4 v;
  asm volatile("ld.global.cg.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
// Programmatic dependent launch: a kernel of this file starts while the one
// before it on the stream still runs, waits here for all of it, and lets the
// next one take its place on the SMs.
__device__ __forceinline__ void chain() {
  asm volatile("griddepcontrol.wait;\n griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Cluster-wide ranks
// ---------------------------------------------------------------------------
struct Plan {
  int lane, warp;  // warp in [0, kPlanWarps) over the cluster
  int thread;      // thread in [0, 32 * kPlanWarps)
};
__device__ __forceinline__ Plan plan_ids() {
  Plan p;
  p.lane = threadIdx.x & 31;
  p.warp = (int)blockIdx.x * (kPlanThreads / 32) + (int)(threadIdx.x >> 5);
  p.thread = (int)blockIdx.x * kPlanThreads + (int)threadIdx.x;
  return p;
}

// Warp w's contiguous share of n things: [w * per, (w + 1) * per).
__device__ __forceinline__ void share(int n, int warp, int* lo, int* hi) {
  const int per = (n + kPlanWarps - 1) / kPlanWarps;
  *lo = (int)min((int64_t)n, (int64_t)warp * per);
  *hi = min(n, *lo + per);
}

// A CTA of the cluster may be stored into only once it has started. A kernel
// says so at its very start and waits for the others in front of its first such
// store, behind loads that take longer; it has to do so, or pass another barrier
// of the cluster, before its first warp_prefix.
__device__ __forceinline__ void cluster_start() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_started() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Exclusive prefix over the cluster's warps of K counts (the same value in
// every lane of a warp) and their totals. `buf` is a shared-memory array of
// its own for each use in a kernel.
template <int K>
__device__ void warp_prefix(const Plan& id, const int (&v)[K], int (&base)[K], int (&total)[K],
                            int (*buf)[kPlanWarps]) {
  cg::cluster_group cl = cg::this_cluster();
  if (id.lane < kClusterCtas) {  // lane r writes this warp's counts into CTA r
    int* peer = cl.map_shared_rank(&buf[0][0], id.lane);
#pragma unroll
    for (int k = 0; k < K; ++k) peer[k * kPlanWarps + id.warp] = v[k];
  }
  cl.sync();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    int b = 0, t = 0;
    for (int w = id.lane; w < kPlanWarps; w += 32) {
      const int x = buf[k][w];
      t += x;
      if (w < id.warp) b += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      b += __shfl_xor_sync(0xffffffffu, b, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    base[k] = b;
    total[k] = t;
  }
}

constexpr int kBatch = 8;  // loads of a lane in flight: every step here waits for memory

// Pages of [lo, hi) that are free (ref == 0; `held` counts the others).
__device__ __forceinline__ int count_pages(const int32_t* ref, int lo, int hi, bool held,
                                           int lane) {
  int n = 0;
  for (int i0 = lo + lane; i0 < hi; i0 += 32 * kBatch) {
    int r[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) r[k] = i0 + 32 * k < hi ? ref[i0 + 32 * k] : 0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) n += i0 + 32 * k < hi && (r[k] != 0) == held ? 1 : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// Calls f(rank, page) for the free (held) pages of [lo, hi) in order, rank
// counting from `base`; stops once rank reaches `most`.
template <typename F>
__device__ __forceinline__ void list_pages(const int32_t* ref, int lo, int hi, bool held, int lane,
                                           int base, int most, F&& f) {
  for (int i0 = lo; i0 < hi && base < most; i0 += 32 * kBatch) {
    int r[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + 32 * k + lane;
      r[k] = i < hi ? ref[i] : 0;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + 32 * k + lane;
      const bool hit = i < hi && (r[k] != 0) == held;
      const unsigned who = __ballot_sync(0xffffffffu, hit);
      const int rank = base + __popc(who & ((1u << lane) - 1u));
      if (hit && rank < most) f(rank, i);
      base += __popc(who);
    }
  }
}

// ---------------------------------------------------------------------------
// copy: which pairs are sound. A destination's mark is the lowest pair that
// names it; a source with a mark is another pair's destination.
// ---------------------------------------------------------------------------
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
copy_plan_kernel(State st, Scratch ws, const int32_t* __restrict__ src,
                 const int32_t* __restrict__ dst, const int32_t* __restrict__ rows, int n) {
  cg::cluster_group cl = cg::this_cluster();
  const Plan id = plan_ids();
  const int nb = st.num_blocks;
  chain();
  auto in_range = [&](int i) {
    return src[i] >= 0 && src[i] < nb && dst[i] >= 0 && dst[i] < nb &&
           (!rows || (rows[i] >= 0 && rows[i] <= st.bs));
  };
  for (int i = id.thread; i < n; i += 32 * kPlanWarps) {
    if (in_range(i) && src[i] != dst[i]) {
      ws.mark[src[i]] = INT_MAX;
      ws.mark[dst[i]] = INT_MAX;
    }
  }
  cl.sync();
  for (int i = id.thread; i < n; i += 32 * kPlanWarps)
    if (in_range(i) && src[i] != dst[i]) atomicMin(&ws.mark[dst[i]], i);
  cl.sync();
  for (int i = id.thread; i < n; i += 32 * kPlanWarps) {
    int4 out = make_int4(0, 0, 0, 0);
    if (!in_range(i)) {
      raise_flag(st.err, PA_DEVERR_PAGE);
    } else if (src[i] != dst[i]) {
      if (fresh(&ws.mark[dst[i]]) == i && fresh(&ws.mark[src[i]]) == INT_MAX)
        out = make_int4(src[i], dst[i], rows ? rows[i] : st.bs, 0);
      else
        raise_flag(st.err, PA_DEVERR_PAGE);
    }
    ws.pairs[i] = out;
  }
  if (id.thread == 0) *ws.count = n;
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
fork_plan_kernel(State st, Scratch ws, const int32_t* __restrict__ parents,
                 const int32_t* __restrict__ children, int n) {
  __shared__ int buf[2][kPlanWarps];
  cg::cluster_group cl = cg::this_cluster();
  const Plan id = plan_ids();
  const int nb = st.num_blocks, ns = st.num_seqs, mb = st.max_blocks;
  chain();
  auto named = [&](int i) {
    return parents[i] >= 0 && parents[i] < ns && children[i] >= 0 && children[i] < ns;
  };
  // a child's mark is the lowest entry that names it; a marked parent is a
  // child of this call
  for (int i = id.thread; i < n; i += 32 * kPlanWarps) {
    if (named(i)) {
      ws.mark[parents[i]] = INT_MAX;
      ws.mark[children[i]] = INT_MAX;
    }
  }
  cl.sync();
  for (int i = id.thread; i < n; i += 32 * kPlanWarps)
    if (named(i)) atomicMin(&ws.mark[children[i]], i);
  cl.sync();

  int lo, hi, plo, phi;
  share(n, id.warp, &lo, &hi);
  share(nb, id.warp, &plo, &phi);
  int v[2] = {0, 0};  // free pages; entries that need one
  for (int i = lo; i < hi; ++i) {  // the warp checks an entry together
    bool page_ok = named(i), ctx_ok = true;
    int need = -1;
    if (page_ok) {
      const int c = children[i], s = parents[i];
      const int ctx = st.past[s], mc = fresh(&ws.mark[c]), ms = fresh(&ws.mark[s]);
      page_ok = mc == i && ms == INT_MAX;
      ctx_ok = ctx >= 0 && (int64_t)ctx <= (int64_t)mb * st.bs;
      if (page_ok && ctx_ok) {
        const int held = (ctx + st.bs - 1) / st.bs;
        const int32_t* prow = st.table + (int64_t)s * mb;
        const int32_t* crow = st.table + (int64_t)c * mb;
        bool ok = true;
        for (int j0 = id.lane; j0 < mb; j0 += 32 * kBatch) {
          int child[kBatch], page[kBatch], refs[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int j = j0 + 32 * k;
            child[k] = j < mb ? crow[j] : -1;
            page[k] = j < held ? prow[j] : -1;
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            refs[k] = page[k] >= 0 && page[k] < nb ? st.ref[page[k]] : j0 + 32 * k < held ? 0 : 1;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) ok = ok && child[k] < 0 && refs[k] > 0;
        }
        page_ok = __all_sync(0xffffffffu, ok);
        need = (ctx % st.bs) != 0 ? 1 : 0;
      }
    }
    if (!page_ok || !ctx_ok) {
      if (id.lane == 0) raise_flag(st.err, page_ok ? PA_DEVERR_CONTEXT : PA_DEVERR_PAGE);
      need = -1;
    }
    if (id.lane == 0) ws.need[i] = need;
    v[1] += need > 0 ? 1 : 0;
  }
  v[0] = count_pages(st.ref, plo, phi, false, id.lane);
  int base[2], total[2];
  warp_prefix<2>(id, v, base, total, buf);
  list_pages(st.ref, plo, phi, false, id.lane, base[0], min(total[0], total[1]),
             [&](int rank, int page) { ws.list[rank] = page; });
  cl.sync();

  int rank = base[1];
  for (int i = lo; i < hi; ++i) {
    const int need = __shfl_sync(0xffffffffu, id.lane == 0 ? ws.need[i] : 0, 0);
    int4 pair = make_int4(0, 0, 0, 0);
    bool take = need >= 0;
    int page = -1;
    if (need > 0) {
      if (rank < total[0]) {
        page = fresh(&ws.list[rank]);
      } else {
        take = false;
        if (id.lane == 0) raise_flag(st.err, PA_DEVERR_POOL);
      }
      ++rank;
    }
    if (take) {
      const int c = children[i], s = parents[i];
      const int ctx = st.past[s], full = ctx / st.bs;
      const int32_t* prow = st.table + (int64_t)s * mb;
      int32_t* crow = st.table + (int64_t)c * mb;
      for (int j0 = id.lane; j0 < full; j0 += 32 * kBatch) {
        int shared[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) shared[k] = j0 + 32 * k < full ? prow[j0 + 32 * k] : 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (j0 + 32 * k < full) {
            crow[j0 + 32 * k] = shared[k];
            atomicAdd(&st.ref[shared[k]], 1);
          }
        }
      }
      if (id.lane == 0) {
        st.past[c] = ctx;
        if (page >= 0) {
          crow[full] = page;
          st.ref[page] = 1;
          pair = make_int4(prow[full], page, ctx % st.bs, 0);
        }
      }
    }
    if (id.lane == 0) ws.pairs[i] = pair;
  }
  if (id.thread == 0) *ws.count = n;
}

// ---------------------------------------------------------------------------
// free: every table entry is taken exactly once (an exchange with -1), so a
// row named twice loses its pages once. A decrement that finds no reference
// is taken back; the end value is max(0, references - entries) in any order.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
free_kernel(State st, const int32_t* __restrict__ seqs, int n) {
  chain();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int s = seqs[i];
    if (s < 0 || s >= st.num_seqs) {
      if (threadIdx.x == 0) raise_flag(st.err, PA_DEVERR_PAGE);
      continue;
    }
    int32_t* row = st.table + (int64_t)s * st.max_blocks;
    for (int j = threadIdx.x; j < st.max_blocks; j += blockDim.x) {
      if (row[j] == -1) continue;
      const int page = atomicExch(&row[j], -1);
      if (page == -1) continue;
      if (page < 0 || page >= st.num_blocks) {
        raise_flag(st.err, PA_DEVERR_PAGE);
      } else if (atomicSub(&st.ref[page], 1) <= 0) {
        atomicAdd(&st.ref[page], 1);
        raise_flag(st.err, PA_DEVERR_PAGE);
      }
    }
    if (threadIdx.x == 0) st.past[s] = 0;
  }
}

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------
// slot_mapping of the tokens me, me + threads, ... once every sequence has its
// pages.
__device__ void fill_slots(const State& st, const Scratch& ws, const int32_t* cum,
                           int64_t num_tokens, int32_t* slot_mapping, int64_t me,
                           int64_t threads) {
  const int ns = st.num_seqs, mb = st.max_blocks, sh = __ffs(st.bs) - 1;
  // Token t belongs to the first sequence whose end exceeds it. A thread looks
  // up kTokens tokens side by side.
  constexpr int kTokens = 4;
  for (int64_t t0 = me; t0 < num_tokens; t0 += threads * kTokens) {
    int seq[kTokens];
    int64_t pos[kTokens];
    bool ok[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      const int64_t t = t0 + k * threads;
      int a = 0, z = ns - 1;
      while (a < z) {
        const int mid = (a + z) >> 1;
        if (t < cum[mid + 1]) z = mid; else a = mid + 1;
      }
      seq[k] = a;
      ok[k] = t < num_tokens && t >= cum[a] && t < cum[a + 1];
      pos[k] = t - cum[a];
    }
    int need[kTokens], past[kTokens], page[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      need[k] = fresh(&ws.need[seq[k]]);
      past[k] = st.past[seq[k]];
    }
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      ok[k] = ok[k] && need[k] >= 0;
      pos[k] += past[k];
      page[k] = ok[k] ? fresh(&st.table[(int64_t)seq[k] * mb + (pos[k] >> sh)]) : 0;
    }
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      const int64_t t = t0 + k * threads;
      if (t < num_tokens)
        slot_mapping[t] = ok[k] ? page[k] * st.bs + (int)(pos[k] & (st.bs - 1)) : -1;
    }
  }
}

constexpr int kStagedSeqs = 4096;

__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
reserve_kernel(State st, Scratch ws, const int32_t* __restrict__ cumseq, int64_t num_tokens,
               int32_t* __restrict__ slot_mapping, bool slots_here) {
  __shared__ int buf[2][kPlanWarps];
  __shared__ int32_t s_cum[kStagedSeqs + 1];  // cumseq for the searches, where it fits
  cluster_start();
  cg::cluster_group cl = cg::this_cluster();
  const Plan id = plan_ids();
  const int nb = st.num_blocks, ns = st.num_seqs, mb = st.max_blocks;
  const int sh = __ffs(st.bs) - 1;
  chain();
  const int32_t* cum = cumseq;
  if (ns <= kStagedSeqs) {
    for (int i = threadIdx.x; i <= ns; i += kPlanThreads) s_cum[i] = cumseq[i];
    cum = s_cum;  // (read behind the cluster's barriers)
  }
  int lo, hi, plo, phi;
  share(ns, id.warp, &lo, &hi);
  share(nb, id.warp, &plo, &phi);
  int v[2] = {0, 0};  // free pages; pages the warp's sequences lack
  for (int b = lo; b < hi; ++b) {
    const int64_t q0 = cumseq[b], q1 = cumseq[b + 1], past = st.past[b];
    int bad = 0, lack = 0;
    if (q0 < 0 || q1 < q0 || q1 > num_tokens) {
      bad = PA_DEVERR_CUMSEQ;
    } else if (q1 > q0) {
      if (past < 0 || past + (q1 - q0) > (int64_t)mb * st.bs) {
        bad = PA_DEVERR_CONTEXT;
      } else {
        const int first = (int)(past >> sh), last = (int)((past + (q1 - q0) - 1) >> sh);
        const int32_t* row = st.table + (int64_t)b * mb;
        bool ok = true;
        for (int j0 = first + id.lane; j0 <= last; j0 += 32 * kBatch) {
          int page[kBatch], refs[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) page[k] = j0 + 32 * k <= last ? row[j0 + 32 * k] : 0;
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            refs[k] = j0 + 32 * k > last || page[k] == -1 ? 1
                      : page[k] >= 0 && page[k] < nb      ? st.ref[page[k]]
                                                          : 0;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            lack += page[k] == -1 ? 1 : 0;
            ok = ok && refs[k] == 1;
          }
        }
        // a page that already holds rows has to be there
        if (id.lane == 0 && (past & (st.bs - 1)) && row[first] == -1) ok = false;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lack += __shfl_xor_sync(0xffffffffu, lack, o);
        if (!__all_sync(0xffffffffu, ok)) bad = PA_DEVERR_PAGE;
      }
    }
    if (bad) lack = 0;
    if (id.lane == 0) {
      if (bad) raise_flag(st.err, bad);
      ws.need[b] = bad ? -1 : lack;
    }
    v[1] = min(v[1] + lack, kMaxBlocks + 1);  // more than any pool has
  }
  v[0] = count_pages(st.ref, plo, phi, false, id.lane);
  int base[2], total[2];
  cluster_started();
  warp_prefix<2>(id, v, base, total, buf);
  list_pages(st.ref, plo, phi, false, id.lane, base[0], min(total[0], total[1]),
             [&](int rank, int page) { ws.list[rank] = page; });
  cl.sync();

  int rank = base[1];
  for (int b = lo; b < hi; ++b) {
    const int lack = __shfl_sync(0xffffffffu, id.lane == 0 ? ws.need[b] : 0, 0);
    if (lack <= 0) continue;
    if ((int64_t)rank + lack > total[0]) {
      if (id.lane == 0) {
        raise_flag(st.err, PA_DEVERR_POOL);
        ws.need[b] = -1;
      }
    } else {
      const int64_t past = st.past[b], q = cumseq[b + 1] - cumseq[b];
      const int first = (int)(past >> sh), last = (int)((past + q - 1) >> sh);
      int32_t* row = st.table + (int64_t)b * mb;
      int at = rank;
      for (int j0 = first; j0 <= last; j0 += 32 * kBatch) {
        int held[kBatch], page[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int j = j0 + 32 * k + id.lane;
          held[k] = j <= last ? row[j] : 0;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const unsigned who = __ballot_sync(0xffffffffu, held[k] == -1);
          page[k] = held[k] == -1 ? fresh(&ws.list[at + __popc(who & ((1u << id.lane) - 1u))]) : -1;
          at += __popc(who);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (page[k] >= 0) {
            row[j0 + 32 * k + id.lane] = page[k];
            st.ref[page[k]] = 1;
          }
        }
      }
    }
    rank = (int)min((int64_t)INT_MAX, (int64_t)rank + lack);
  }
  cl.sync();

  if (slots_here) fill_slots(st, ws, cum, num_tokens, slot_mapping, id.thread, 32 * kPlanWarps);
}

// The slots of a call with many tokens, on the whole GPU behind reserve_kernel.
__global__ void __launch_bounds__(256)
slots_kernel(State st, Scratch ws, const int32_t* __restrict__ cumseq, int64_t num_tokens,
             int32_t* __restrict__ slot_mapping) {
  __shared__ int32_t s_cum[kStagedSeqs + 1];
  chain();
  const int32_t* cum = cumseq;
  if (st.num_seqs <= kStagedSeqs) {
    for (int i = threadIdx.x; i <= st.num_seqs; i += blockDim.x) s_cum[i] = cumseq[i];
    __syncthreads();
    cum = s_cum;
  }
  fill_slots(st, ws, cum, num_tokens, slot_mapping,
             (int64_t)blockIdx.x * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x);
}

// ---------------------------------------------------------------------------
// compact: L held pages; the k-th held page at or above L goes to the k-th
// free page below L. ws.mark becomes every page's new id (-1: not held).
// ---------------------------------------------------------------------------
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
compact_plan_kernel(State st, Scratch ws, int32_t* live_out) {
  __shared__ int buf1[1][kPlanWarps];
  __shared__ int buf2[2][kPlanWarps];
  cluster_start();
  cg::cluster_group cl = cg::this_cluster();
  const Plan id = plan_ids();
  chain();
  int lo, hi;
  share(st.num_blocks, id.warp, &lo, &hi);
  int live[1] = {count_pages(st.ref, lo, hi, true, id.lane)}, before[1], all[1];
  cluster_started();
  warp_prefix<1>(id, live, before, all, buf1);
  const int L = all[0];
  // free pages below L and held pages from L on
  int v[2] = {count_pages(st.ref, lo, min(hi, L), false, id.lane),
              count_pages(st.ref, max(lo, L), hi, true, id.lane)};
  int base[2], total[2];
  warp_prefix<2>(id, v, base, total, buf2);
  for (int i = lo + id.lane; i < hi; i += 32) ws.mark[i] = st.ref[i] != 0 ? i : -1;
  list_pages(st.ref, lo, min(hi, L), false, id.lane, base[0], INT_MAX,
             [&](int rank, int page) { ws.pairs[rank].y = page; });
  list_pages(st.ref, max(lo, L), hi, true, id.lane, base[1], INT_MAX,
             [&](int rank, int page) { ws.pairs[rank].x = page; });
  cl.sync();
  const int m = total[1];
  for (int k = id.thread; k < m; k += 32 * kPlanWarps) {
    const int4 p = fresh(&ws.pairs[k]);
    ws.pairs[k].z = st.bs;
    ws.mark[p.x] = p.y;
    st.ref[p.y] = st.ref[p.x];
    st.ref[p.x] = 0;
  }
  if (id.thread == 0) {
    *ws.count = m;
    if (live_out) *live_out = L;
  }
}

// ---------------------------------------------------------------------------
// Contents
// ---------------------------------------------------------------------------
struct CacheList {
  uint8_t* data[kMaxCaches];
  int64_t page_bytes[kMaxCaches];  // with PA_PAGE_WHOLE
  int32_t first[kMaxCaches + 1];  // pieces of the caches before this one
};

// Where the pairs come from: the plan kernel's list, or (SMALL) the call's own
// arrays of n <= kSmallPairs entries, which every CTA checks for itself by
// comparing each entry with all others (the plan kernel's rules): one launch
// instead of two. Pages of 6 KB in 4 caches, GPU time: 8 pairs 12.4 -> 7.4 us,
// 64 pairs 13.4 -> 11.4 us, 128 pairs 13.4 -> 15.5 us.
constexpr int kSmallPairs = 64;

template <bool SMALL>
__global__ void __launch_bounds__(256, 4)
move_kernel(const __grid_constant__ CacheList cl, int num_caches, State st, const int4* pairs,
            const int32_t* count, const int32_t* new_id, const int32_t* src, const int32_t* dst,
            const int32_t* rows, int n) {
  __shared__ int4 s_pairs[SMALL ? kSmallPairs : 1];
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  chain();
  if (SMALL) {
    const int i = threadIdx.x, nb = st.num_blocks;
    if (i < n) {  // z < 0: out of range; x == y: nothing to copy
      const int r = rows ? rows[i] : st.bs;
      int4 p = make_int4(src[i], dst[i], r, 0);
      if (p.x < 0 || p.x >= nb || p.y < 0 || p.y >= nb || r < 0 || r > st.bs) p.z = -1;
      s_pairs[i] = p;
    }
    __syncthreads();
    bool bad = false, copies = false;
    if (i < n) {
      const int4 p = s_pairs[i];
      copies = p.z >= 0 && p.x != p.y;
      bad = p.z < 0;
      for (int j = 0; j < n; ++j) {
        const int4 q = s_pairs[j];
        if (copies && q.z >= 0 && q.x != q.y && (q.y == p.x || (j < i && q.y == p.y))) bad = true;
      }
      if (bad && blockIdx.x == 0) raise_flag(st.err, PA_DEVERR_PAGE);
    }
    __syncthreads();
    if (i < n && (bad || !copies)) s_pairs[i].z = 0;
    __syncthreads();
  }
  if (!SMALL && new_id) {  // compact: the table follows the pages
    const int64_t entries = (int64_t)st.num_seqs * st.max_blocks;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < entries;
         i += (int64_t)gridDim.x * blockDim.x) {
      const int page = st.table[i];
      if (page == -1) continue;
      const int to = page >= 0 && page < st.num_blocks ? fresh(new_id + page) : -1;
      if (to < 0) raise_flag(st.err, PA_DEVERR_PAGE);
      if (to != page) st.table[i] = to;
    }
  }
  const int pieces = cl.first[num_caches], sh = __ffs(st.bs) - 1;
  const int64_t items = (int64_t)(SMALL ? n : fresh(count)) * pieces;
  for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items;
       it += warps) {
    const int64_t pi = it / pieces;
    const int piece = (int)(it - pi * pieces);
    const int4 p = SMALL ? s_pairs[pi] : fresh(pairs + pi);
    int a = 0, z = num_caches - 1;  // the cache whose pieces hold `piece`
    while (a < z) {
      const int mid = (a + z) >> 1;
      if (piece < cl.first[mid + 1]) z = mid; else a = mid + 1;
    }
    const bool whole = (cl.page_bytes[a] & PA_PAGE_WHOLE) != 0;
    const int64_t pb = cl.page_bytes[a] & ~PA_PAGE_WHOLE;
    const int64_t at = (int64_t)(piece - cl.first[a]) * kPieceBytes;
    // bytes to copy from `at` on
    const int64_t left = (whole ? (p.z > 0 ? pb : 0) : (pb >> sh) * p.z) - at;
    if (left <= 0) continue;
    if (whole) {  // (a page starts on 8 bytes, and there are few of them)
      const int m = (int)(min(left, (int64_t)kPieceBytes) >> 3);
      const uint2* s = reinterpret_cast<const uint2*>(cl.data[a] + p.x * pb + at);
      uint2* d = reinterpret_cast<uint2*>(cl.data[a] + p.y * pb + at);
      for (int k = lane; k < m; k += 32) d[k] = s[k];
      continue;
    }
    const uint4* s = reinterpret_cast<const uint4*>(cl.data[a] + p.x * pb + at);
    uint4* d = reinterpret_cast<uint4*>(cl.data[a] + p.y * pb + at);
    constexpr int kVec = kPieceBytes / 512;  // 16-byte vectors per lane
    uint4 v[kVec];
    if (left >= kPieceBytes) {
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[k] = __ldcs(s + k * 32 + lane);
#pragma unroll
      for (int k = 0; k < kVec; ++k) __stcs(d + k * 32 + lane, v[k]);
    } else {
      const int m = (int)(left >> 4);
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (k * 32 + lane < m) v[k] = __ldcs(s + k * 32 + lane);
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (k * 32 + lane < m) __stcs(d + k * 32 + lane, v[k]);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
pa_status fail(pa_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
pa_status fail(pa_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return record_error(s, buf);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

pa_status check_params(const pa_pages_params* p) {
  if (!p) return fail(PA_ERR_INVALID_ARGUMENT, "params is NULL");
  const int bs = p->block_size;
  if (bs < 16 || (bs & (bs - 1)) != 0)
    return fail(PA_ERR_INVALID_ARGUMENT, "block_size %d must be a power of two >= 16", bs);
  if (p->num_blocks < 1 || p->num_blocks > kMaxBlocks)
    return fail(PA_ERR_INVALID_ARGUMENT, "num_blocks %d must be in 1..%d", p->num_blocks,
                kMaxBlocks);
  if ((int64_t)p->num_blocks * bs > INT32_MAX)
    return fail(PA_ERR_INVALID_ARGUMENT, "num_blocks * block_size exceeds the int32 slot range");
  if (p->max_blocks_per_seq < 1)
    return fail(PA_ERR_INVALID_ARGUMENT, "max_blocks_per_seq must be >= 1");
  if ((int64_t)p->max_blocks_per_seq * bs > INT32_MAX)
    return fail(PA_ERR_INVALID_ARGUMENT, "max_blocks_per_seq * block_size exceeds int32");
  if (p->num_seqs < 1 || p->num_seqs > kMaxBlocks)
    return fail(PA_ERR_INVALID_ARGUMENT, "num_seqs %d must be in 1..%d", p->num_seqs, kMaxBlocks);
  return PA_OK;
}

pa_status check_caches(const pa_pages_params* p, const pa_pages_cache* caches, int32_t n) {
  if (n < 0) return fail(PA_ERR_INVALID_ARGUMENT, "num_caches must be >= 0");
  if (n > 0 && !caches) return fail(PA_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  for (int i = 0; i < n; ++i) {
    if (!caches[i].data || !aligned(caches[i].data, 16))
      return fail(PA_ERR_INVALID_ARGUMENT, "cache %d must be a 16-byte aligned pointer", i);
    const int64_t b = caches[i].page_bytes, bytes = b & ~PA_PAGE_WHOLE;
    if (b > 0 && b != bytes) {
      if (bytes <= 0 || bytes % 8 != 0 || bytes > ((int64_t)1 << 32))
        return fail(PA_ERR_INVALID_ARGUMENT,
                    "cache %d: page_bytes %lld of a tensor of whole pages must be a positive "
                    "multiple of 8, at most 2^32", i, (long long)bytes);
      continue;
    }
    if (b <= 0 || b % (16 * (int64_t)p->block_size) != 0 || b > ((int64_t)1 << 32))
      return fail(PA_ERR_INVALID_ARGUMENT,
                  "cache %d: page_bytes %lld must be a positive multiple of 16 * block_size, "
                  "at most 2^32", i, (long long)b);
  }
  return PA_OK;
}

pa_status check_workspace(const pa_pages_params* p, void* ws, size_t bytes, Scratch* s) {
  const size_t need = layout(*p, nullptr, nullptr);
  if (ws && !aligned(ws, 256))
    return fail(PA_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  if (!ws || bytes < need)
    return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed",
                ws ? bytes : (size_t)0, need);
  layout(*p, static_cast<char*>(ws), s);
  return PA_OK;
}

template <typename... P>
pa_status check_ints(const int32_t* err, const P*... ptrs) {
  for (const void* q : {static_cast<const void*>(ptrs)...}) {
    if (!q) return fail(PA_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
    if (!aligned(q, 4)) return fail(PA_ERR_INVALID_ARGUMENT, "int32 tensors must be 4-byte aligned");
  }
  if (!aligned(err, 4)) return fail(PA_ERR_INVALID_ARGUMENT, "int32 tensors must be 4-byte aligned");
  return PA_OK;
}

pa_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return PA_OK;
  (void)cudaGetLastError();  // not left behind for a later call
  return fail(PA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int sms() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n <= 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      return 148;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

State state(const pa_pages_params& p, int32_t* table, int32_t* past, int32_t* ref, int32_t* err) {
  return State{table, past, ref, err, p.num_blocks, p.block_size, p.max_blocks_per_seq, p.num_seqs};
}

template <typename K, typename... Args>
cudaError_t launch_chained(K kernel, unsigned grid, unsigned block, cudaStream_t stream,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A copy call's own arrays, for the copy of a few pairs.
struct FewPairs {
  const int32_t *src, *dst, *rows;
  int n;
};

// The copies of ws.pairs[0, *ws.count) in every cache, after the plan kernel,
// or those of `few`. `most`: no more pairs than this; new_id: the table rewrite
// of a compaction (in the first launch; without caches a launch of its own).
pa_status launch_move(const State& st, const Scratch& ws, const pa_pages_cache* caches, int32_t n,
                      int64_t most, const int32_t* new_id, const FewPairs* few,
                      cudaStream_t stream) {
  for (int c0 = 0; c0 < n || (new_id && c0 == 0); c0 += kMaxCaches) {
    CacheList cl;
    const int m = n - c0 < kMaxCaches ? n - c0 : kMaxCaches;
    cl.first[0] = 0;
    for (int i = 0; i < m; ++i) {
      cl.data[i] = static_cast<uint8_t*>(caches[c0 + i].data);
      cl.page_bytes[i] = caches[c0 + i].page_bytes;
      cl.first[i + 1] =
          cl.first[i] +
          (int32_t)(((cl.page_bytes[i] & ~PA_PAGE_WHOLE) + kPieceBytes - 1) / kPieceBytes);
    }
    int64_t work = most * cl.first[m];  // warps
    if (new_id && c0 == 0) {
      const int64_t t = (int64_t)st.num_seqs * st.max_blocks / 32 + 1;
      work = work > t ? work : t;
    }
    int64_t blocks = (work + 7) / 8;
    const int64_t cap = (int64_t)sms() * 8;
    if (blocks > cap) blocks = cap;
    if (blocks < 1) blocks = 1;  // (one page: nothing can move)
    const int4* pairs = few ? nullptr : ws.pairs;
    const int32_t* count = few ? nullptr : ws.count;
    const int32_t* ids = c0 == 0 ? new_id : nullptr;
    const FewPairs f = few ? *few : FewPairs{nullptr, nullptr, nullptr, 0};
    const cudaError_t e = launch_chained(few ? move_kernel<true> : move_kernel<false>,
                                         (unsigned)blocks, 256u, stream, cl, m, st, pairs, count,
                                         ids, f.src, f.dst, f.rows, f.n);
    if (e != cudaSuccess) return launched(e, "page copy launch");
  }
  return PA_OK;
}

}  // namespace
}  // namespace pages
}  // namespace pa

using namespace pa;
using namespace pa::pages;

extern "C" {

pa_status pa_pages_validate(const pa_pages_params* p) { return check_params(p); }

size_t pa_pages_workspace_size(const pa_pages_params* p) {
  return check_params(p) == PA_OK ? layout(*p, nullptr, nullptr) : 0;
}

pa_status pa_pages_copy(const pa_pages_params* p, const pa_pages_cache* caches,
                        int32_t num_caches, const int32_t* src, const int32_t* dst,
                        const int32_t* rows, int32_t n, void* workspace, size_t workspace_bytes,
                        int32_t* err_flags, void* stream) {
  Scratch ws;
  pa_status s = check_params(p);
  if (s == PA_OK) s = check_caches(p, caches, num_caches);
  if (s != PA_OK) return s;
  if (n < 0 || n > p->num_blocks)
    return fail(PA_ERR_INVALID_ARGUMENT, "%d pairs: 0..num_blocks are possible", n);
  if (n == 0 || num_caches == 0) return PA_OK;
  if ((s = check_ints(err_flags, src, dst)) != PA_OK) return s;
  if (!aligned(rows, 4)) return fail(PA_ERR_INVALID_ARGUMENT, "int32 tensors must be 4-byte aligned");
  if ((s = check_workspace(p, workspace, workspace_bytes, &ws)) != PA_OK) return s;
  const State st = state(*p, nullptr, nullptr, nullptr, err_flags);
  const cudaStream_t str = reinterpret_cast<cudaStream_t>(stream);
  if (n <= kSmallPairs) {
    const FewPairs few{src, dst, rows, n};
    return launch_move(st, ws, caches, num_caches, n, nullptr, &few, str);
  }
  s = launched(launch_chained(copy_plan_kernel, kClusterCtas, kPlanThreads, str, st, ws, src, dst,
                              rows, n),
               "page copy plan launch");
  if (s != PA_OK) return s;
  return launch_move(st, ws, caches, num_caches, n, nullptr, nullptr, str);
}

pa_status pa_pages_fork(const pa_pages_params* p, const pa_pages_cache* caches,
                        int32_t num_caches, const int32_t* parents, const int32_t* children,
                        int32_t n, int32_t* block_table, int32_t* past, int32_t* refcount,
                        void* workspace, size_t workspace_bytes, int32_t* err_flags,
                        void* stream) {
  Scratch ws;
  pa_status s = check_params(p);
  if (s == PA_OK) s = check_caches(p, caches, num_caches);
  if (s != PA_OK) return s;
  if (n < 0 || n > p->num_seqs)
    return fail(PA_ERR_INVALID_ARGUMENT, "%d forks: 0..num_seqs are possible", n);
  if (n == 0) return PA_OK;
  if ((s = check_ints(err_flags, parents, children, block_table, past, refcount)) != PA_OK)
    return s;
  if ((s = check_workspace(p, workspace, workspace_bytes, &ws)) != PA_OK) return s;
  const State st = state(*p, block_table, past, refcount, err_flags);
  const cudaStream_t str = reinterpret_cast<cudaStream_t>(stream);
  s = launched(launch_chained(fork_plan_kernel, kClusterCtas, kPlanThreads, str, st, ws, parents,
                              children, n),
               "fork launch");
  if (s != PA_OK) return s;
  return launch_move(st, ws, caches, num_caches, n, nullptr, nullptr, str);
}

pa_status pa_pages_free(const pa_pages_params* p, const int32_t* seqs, int32_t n,
                        int32_t* block_table, int32_t* past, int32_t* refcount,
                        int32_t* err_flags, void* stream) {
  pa_status s = check_params(p);
  if (s != PA_OK) return s;
  if (n < 0 || n > p->num_seqs)
    return fail(PA_ERR_INVALID_ARGUMENT, "%d sequences: 0..num_seqs are possible", n);
  if (n == 0) return PA_OK;
  if ((s = check_ints(err_flags, seqs, block_table, past, refcount)) != PA_OK) return s;
  const State st = state(*p, block_table, past, refcount, err_flags);
  const int cap = sms() * 8;
  return launched(launch_chained(free_kernel, (unsigned)(n < cap ? n : cap), 256u,
                                 reinterpret_cast<cudaStream_t>(stream), st, seqs, (int)n),
                  "free launch");
}

pa_status pa_pages_reserve(const pa_pages_params* p, const int32_t* cumseq, int64_t num_tokens,
                           int32_t* block_table, const int32_t* past, int32_t* refcount,
                           int32_t* slot_mapping, void* workspace, size_t workspace_bytes,
                           int32_t* err_flags, void* stream) {
  Scratch ws;
  pa_status s = check_params(p);
  if (s != PA_OK) return s;
  if (num_tokens < 0 || num_tokens > INT32_MAX)
    return fail(PA_ERR_INVALID_ARGUMENT, "num_tokens must be in 0..2^31 - 1");
  if (num_tokens == 0) return PA_OK;
  if ((s = check_ints(err_flags, cumseq, block_table, past, refcount, slot_mapping)) != PA_OK)
    return s;
  if ((s = check_workspace(p, workspace, workspace_bytes, &ws)) != PA_OK) return s;
  const State st = state(*p, block_table, const_cast<int32_t*>(past), refcount, err_flags);
  const cudaStream_t str = reinterpret_cast<cudaStream_t>(stream);
  const bool here = num_tokens <= kClusterTokens;
  s = launched(launch_chained(reserve_kernel, kClusterCtas, kPlanThreads, str, st, ws, cumseq,
                              num_tokens, slot_mapping, here),
               "reserve launch");
  if (s != PA_OK || here) return s;
  int64_t blocks = (num_tokens + 1023) / 1024;
  if (blocks > sms() * 4) blocks = sms() * 4;
  return launched(launch_chained(slots_kernel, (unsigned)blocks, 256u, str, st, ws, cumseq,
                                 num_tokens, slot_mapping),
                  "slots launch");
}

pa_status pa_pages_compact(const pa_pages_params* p, const pa_pages_cache* caches,
                           int32_t num_caches, int32_t* block_table, int32_t* refcount,
                           int32_t* live, void* workspace, size_t workspace_bytes,
                           int32_t* err_flags, void* stream) {
  Scratch ws;
  pa_status s = check_params(p);
  if (s == PA_OK) s = check_caches(p, caches, num_caches);
  if (s != PA_OK) return s;
  if ((s = check_ints(err_flags, block_table, refcount)) != PA_OK) return s;
  if (!aligned(live, 4)) return fail(PA_ERR_INVALID_ARGUMENT, "int32 tensors must be 4-byte aligned");
  if ((s = check_workspace(p, workspace, workspace_bytes, &ws)) != PA_OK) return s;
  const State st = state(*p, block_table, nullptr, refcount, err_flags);
  const cudaStream_t str = reinterpret_cast<cudaStream_t>(stream);
  s = launched(launch_chained(compact_plan_kernel, kClusterCtas, kPlanThreads, str, st, ws, live),
               "compact launch");
  if (s != PA_OK) return s;
  return launch_move(st, ws, caches, num_caches, p->num_blocks / 2, ws.mark, nullptr, str);
}

}  // extern "C"
