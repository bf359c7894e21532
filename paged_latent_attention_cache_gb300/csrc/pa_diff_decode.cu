// Differential attention, decode: one new token per sequence (include/pa_diff.h).
//
// Bound by HBM: each visible key of a kv head is read once (2 hs + vhs
// channels, 512 bytes at 64 / 128) for 2 * (hs + vhs) * 2 multiply-adds per
// head, with up to 8 heads per kv head (more: below). The work is cut for that:
//
// * A tile is 16 keys of one (sequence, kv head, chunk of 8 heads): 16 rows of
//   one page. Up to 8 heads share a tile's bytes. The rows of an mma.sync
//   m16n8k16 are the 8 heads with map 0 (rows 0-7) and map 1 (rows 8-15), so
//   both maps share one product with V; a tcgen05 tile (128 rows) would be
//   filled to an eighth at most and its tensor memory round trip is longer
//   than a tile's work.
// * All tiles of the call, in the order (sequence, kv head and chunk, tile),
//   form one line that is cut into equal parts, one per CTA, whatever the
//   lengths; a part may start and end inside a sequence. Parts are joined by
//   the combine kernel below, as are all results (one code path).
// * Tiles are copied by TMA, the keys of both maps with one box and the values
//   with another (a box per 64 channels where a width is no multiple of 64),
//   into a ring of up to 24 stages. Tile i of a CTA's part goes to warp i % 8, which folds it into
//   running sums of its own and then starts the copy of tile i + stages into
//   the stage it has just read: no barrier inside a part, no producer, and
//   copies run ahead across sequences. A tile is a chain of dependent products
//   and row maxima, so one warp per scheduler cannot keep up with 23 bytes per
//   cycle and SM; a ring per warp leaves room for only four warps (323 us where
//   the shared ring took 246, see below for the case), and one producer warp
//   cannot issue a tile's boxes fast enough (407 us). The stages that no warp
//   reads are the bytes in flight (45 GB/s per SM at 1 us ask for 45 KB).
// * Value rows that no query sees are overwritten with zeros after the copy,
//   scores of such keys with -inf, so what they hold cannot reach a sum.
//
// Measured: 32 sequences of 1024 to 8192 keys, 16 heads over 8 kv heads, bf16
// 128 / 256: 191 us for 1.24 GB, 6.5 TB/s, 0.96 of a plain copy's rate; what is
// left is the start of the first copies and the last parts' joins. Two sequences
// of 300 to 1000 keys, 8 heads, fp16 64 / 128: 11 us, latency only (with the
// write before and the combine behind it 20 us).
//
// With more than 8 heads per kv head every chunk of 8 is a stretch of the line of
// its own and copies the keys again, from L2 at best. The same 32 sequences, 8 kv
// heads: 64 heads 226 us, 128 heads (two chunks) 419; one kv head (floor 23 us): 8
// heads 54 us, 16 69, 32 100, 64 177, 128 (16 chunks) 323, with the combine.
//
// Precision: out = softmax_0 V - lambda softmax_1 V cancels, so errors of the
// two maps weigh more than in a plain softmax. The rotated query and the
// probabilities enter the products as two 16-bit parts each (value and
// remainder, 2^-16 relative in bf16; see Prob). For the scores that is free: a product
// of one map has 8 rows for the heads' values and 8 for their remainders, and
// both sums of a score end up in one lane. For the values it doubles the
// products.
#include <cmath>
#include <type_traits>

#include "pa_diff_common.cuh"
#include "pa_diff_internal.h"

namespace pa {
namespace diff {
namespace {

using tc::ex2;
using tc::grid_dep_launch;
using tc::grid_dep_wait;
using tc::pack2;
using tc::smem_u32;

constexpr int kWarps = 8;
constexpr int kTileKeys = 16;
constexpr int kHeads = 8;        // heads of a chunk
constexpr int kRows = 2 * kHeads;
constexpr int kMaxStages = 24;
constexpr size_t kSmem = 225 * 1024;  // dynamic shared memory of a CTA (one per SM)
constexpr int kThreads = kWarps * 32;
constexpr int kJoin = 64;        // channels joined at a time at the end of a segment
constexpr int kJoinPitch = 72;   // floats of a row there (8 rows x 8 bytes x 4 lanes: no bank twice)
constexpr int kMinTiles = kWarps;  // least part of a CTA

struct Args {
  Geometry g;
  DiffArgs a;
  int grp, chunks, ng;  // heads per kv head, chunks of 8 of them, kvh * chunks
  int vslabs, stage, stages;  // 64-channel value slabs; bytes and number of ring stages
  bool k_whole, v_whole;      // one box per tile (see cache_map)
  int64_t slots;        // partials the workspace holds
  float scale_log2, cap_in, cap_out;
  float* ws_o;          // [slots][16][vhs]
  float2* ws_ml;        // [slots][16] (log2-domain maximum, sum; sum -1: a bad page)
  int64_t* ws_plan;     // [nseq] tiles before the sequence, then total tiles, CTAs in use
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A pair of values as 16-bit parts: hi rounded, lo the rounded remainder.
template <typename T>
__device__ __forceinline__ void split2(float x, float y, uint32_t* hi, uint32_t* lo) {
  const T hx = Half<T>::from_f32(x), hy = Half<T>::from_f32(y);
  *hi = pack2<T>(x, y);
  *lo = pack2<T>(x - Half<T>::to_f32(hx), y - Half<T>::to_f32(hy));
}

// Waits until tile n has landed in its stage. The tiles of a stage go to
// different warps, so a warp may come here before the tile before n in that
// stage was even read, when the barrier's parity still says "complete" for the
// phase before: first the copy of n has to have been started (`last`, set by
// the warp that read the tile before). Bounded like wait_bar.
__device__ __forceinline__ bool wait_tile(uint64_t* full, volatile int* last, int n, uint32_t parity,
                                          volatile int* abort, int32_t* err) {
  if (*last != n) {
    const uint64_t t0 = tc::globaltimer();
    for (uint32_t i = 1; *last != n; ++i) {
      if ((i & 63u) == 0) {
        if (*abort) return false;
        if (tc::globaltimer() - t0 > tc::kWaitLimitNs) {
          *abort = 1;
          raise_flag(err, PA_DEVERR_TIMEOUT);
          return false;
        }
      }
    }
    __threadfence_block();
  }
  return tc::wait_bar(smem_u32(full), parity, abort, err);
}

// Visible keys of decode sequence b: status 0 = [lo, pos]; 1 = not one new
// token (its rows stay); 2 = positions or offsets out of range (zeros).
struct Seq {
  int64_t t, lo, pos;
  int status, err;
};
__device__ __forceinline__ Seq seq_of(const Args& A, int b) {
  const int32_t q0 = A.a.cumseq[b], q1 = A.a.cumseq[b + 1];
  Seq s;
  s.pos = A.a.past[b];
  s.t = q0;
  s.status = s.err = 0;
  if (q1 - q0 != 1) {
    s.status = 1;
    s.err = PA_DEVERR_DECODE_QLEN;
  } else if (q0 < 0 || q0 >= A.a.num_tokens) {
    s.status = 1;
    s.err = PA_DEVERR_CUMSEQ;
  } else if (s.pos < 0 || s.pos >= (int64_t)A.g.max_blocks * A.g.bs) {
    s.status = 2;
    s.err = PA_DEVERR_CONTEXT;
  } else if (A.g.rd > 0 && s.pos >= A.g.cos_rows) {
    s.status = 2;
    s.err = PA_DEVERR_POSITION;
  }
  s.lo = A.g.window >= 0 ? max((int64_t)0, s.pos - A.g.window) : 0;
  return s;
}
__device__ __forceinline__ int tiles_of(const Args& A, int b) {
  const Seq s = seq_of(A, b);
  return s.status ? 0 : (int)(s.pos / kTileKeys - s.lo / kTileKeys) + 1;
}

// One warp: total tiles of the call's line, and (first, before) of the
// sequence that holds its tile x (the tiles of the sequences before it).
__device__ int64_t line_total(const Args& A, int nseq, int lane) {
  int64_t sum = 0;
  for (int i = lane; i < nseq; i += 32) sum += tiles_of(A, A.a.seq_begin + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum * A.ng;
}
// With `plan`, also stores every sequence's prefix.
__device__ void line_find(const Args& A, int nseq, int lane, int64_t x, int* seq, int64_t* before,
                          int64_t* plan) {
  int64_t run = 0;
  bool found = false;
  for (int i0 = 0; i0 < nseq; i0 += 32) {
    const int i = i0 + lane;
    const int64_t n = i < nseq ? (int64_t)tiles_of(A, A.a.seq_begin + i) * A.ng : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int64_t start = run + incl - n;
    if (plan && i < nseq) plan[i] = start;
    const unsigned who = __ballot_sync(0xffffffffu, x >= start && x < start + n);
    if (who && !found) {
      const int src = __ffs(who) - 1;
      *seq = i0 + src;
      *before = __shfl_sync(0xffffffffu, start, src);
      found = true;
      if (!plan) return;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// A place on the line: sequence index, (kv head, chunk), tile, and the
// sequence's range.
struct Cursor {
  int seq, gc, tile, tiles;
  int64_t lo, pos, t;  // the sequence's visible keys and token
};
__device__ __forceinline__ void cursor_load(const Args& A, Cursor& c) {
  const Seq s = seq_of(A, A.a.seq_begin + c.seq);
  c.lo = s.lo;
  c.pos = s.pos;
  c.t = s.t;
  c.tiles = s.status ? 0 : (int)(s.pos / kTileKeys - s.lo / kTileKeys) + 1;
}
// `step` tiles on, over the ends of (kv head, chunk)s and sequences.
__device__ __forceinline__ void cursor_step(const Args& A, Cursor& c, int step, int nseq) {
  c.tile += step;
  while (c.tile >= c.tiles) {
    c.tile -= c.tiles;
    if (++c.gc == A.ng || c.tiles == 0) {
      c.gc = 0;
      if (++c.seq >= nseq) return;
      cursor_load(A, c);
    }
  }
}

// A stage of the ring: 16-row slabs of 64 channels (128-byte swizzle), map 0's,
// map 1's, then the value's. KS >= hs / 16 (4 or 8), VT >= vhs / 8 fix the
// register arrays.
constexpr int kSlab = kTileKeys * 128;

template <typename T, int KS, int VT>
__global__ void __launch_bounds__(kThreads, 1)
diff_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ Args A) {
  constexpr int KSL = KS / 4;  // slabs of a map
  extern __shared__ uint8_t smem_raw[];
  __shared__ Cursor s_first, s_cur;
  __shared__ int s_count;
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ int s_bad[kWarps];
  __shared__ int s_abort;
  __shared__ uint64_t s_full[kMaxStages];
  __shared__ int s_stage_bad[kMaxStages];  // the tile in the stage has no valid page
  __shared__ int s_last[kMaxStages];       // the last tile copied into it
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  const Geometry& g = A.g;
  const DiffArgs& a = A.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nseq = a.seq_end - a.seq_begin;
  const int hs = g.hs, vhs = g.vhs, nvt = vhs >> 3, stages = A.stages;
  const int sh = __ffs(g.bs) - 1;
  const bool early = (g.flags & PA_FLAG_AFTER_WRITE) != 0;
  bool waited = !early;
  if (!early) grid_dep_wait();
  grid_dep_launch();

  // ---- this CTA's part of the line
  if (warp == 0) {
    int64_t* plan = blockIdx.x == 0 ? A.ws_plan : nullptr;
    Cursor c;
    int64_t total, n = 0, incl = 0;
    if (nseq <= 32) {  // one round of loads, the rest in registers
      c.tiles = 0;
      if (lane < nseq) {
        c.seq = lane;
        cursor_load(A, c);
      }
      n = incl = (int64_t)c.tiles * A.ng;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
      if (plan && lane < nseq) plan[lane] = incl - n;
    } else {
      total = line_total(A, nseq, lane);
    }
    const int64_t ctas = min((int64_t)gridDim.x, max((int64_t)1, total / kMinTiles));
    if (plan && lane == 0) {
      plan[nseq] = total;
      plan[nseq + 1] = ctas;
    }
    const bool some = blockIdx.x < ctas && total > 0;
    const int64_t x0 = some ? (int64_t)blockIdx.x * total / ctas : 0;
    const int64_t x1 = some ? ((int64_t)blockIdx.x + 1) * total / ctas : 0;
    int64_t before = incl - n;
    bool mine = x0 >= before && x0 < incl;  // the lane whose sequence holds tile x0
    if (nseq > 32) {
      if (some || plan) line_find(A, nseq, lane, x0, &c.seq, &before, plan);
      if (some) cursor_load(A, c);
      mine = lane == 0;
    }
    if (some && mine) {
      const int64_t off = x0 - before;
      c.gc = (int)(off / c.tiles);
      c.tile = (int)(off - (int64_t)c.gc * c.tiles);
      s_first = c;
    }
    if (lane == 0) s_count = (int)(x1 - x0);
  }
  if (warp == 1 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      tc::mbar_init(smem_u32(&s_full[s]), 1);
      s_last[s] = -1;
    }
    s_abort = 0;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&kmap);
    tc::prefetch_tmap(&vmap);
  }
  __syncthreads();
  const int count = s_count;  // tiles of this CTA
  if (count == 0) {
    if (!waited) grid_dep_wait();
    return;
  }
  const Cursor first = s_first;

  const uint32_t ring = smem_u32(smem);
  uint4* q_s = reinterpret_cast<uint4*>(smem + (size_t)stages * A.stage);
  float* join = reinterpret_cast<float*>(q_s + 2 * KS * 32);

  // ---- copies: the warp's tiles below `stages` now, tile i + stages after i.
  // The cursor stands at the next one, whose page id is loaded a tile ahead.
  Cursor lc = first;
  int next_tile = warp < stages ? warp : warp + stages;
  auto page_of = [&]() {
    if (lc.seq >= nseq) return -1;  // (the lengths changed under the kernel)
    const int key0 = (int)(lc.lo / kTileKeys + lc.tile) * kTileKeys;
    return a.block_table[(int64_t)(a.seq_begin + lc.seq) * g.max_blocks + (key0 >> sh)];
  };
  int next_page = 0;
  if (next_tile < count) {
    cursor_step(A, lc, next_tile, nseq);
    next_page = page_of();
  }
  auto issue = [&](int stage) {
    if (next_tile >= count) return;
    const int key0 = (int)(lc.lo / kTileKeys + lc.tile) * kTileKeys;
    if (!waited && (!(g.flags & PA_FLAG_OWN_SLOTS) || key0 + kTileKeys > lc.pos)) {
      grid_dep_wait();  // from here on rows the write phase may store are read
      waited = true;
    }
    const int gk = lc.gc / A.chunks;
    const bool ok = next_page >= 0 && next_page < g.num_blocks;
    // (no such page: a row out of range, which the copy fills with zeros)
    const int row = ok ? next_page * g.bs + (key0 & (g.bs - 1)) : g.num_blocks * g.bs;
    if (elect_one()) {
      if (!ok) raise_flag(a.err_flags, PA_DEVERR_BLOCK);
      s_stage_bad[stage] = ok ? 0 : 1;
      __threadfence_block();
      *(volatile int*)&s_last[stage] = next_tile;
      const uint32_t bar = smem_u32(&s_full[stage]);
      const uint32_t dst = ring + stage * A.stage, vdst = dst + 2 * KSL * kSlab;
      tc::mbar_expect_tx(bar, (uint32_t)A.stage);
      if (A.k_whole) {
        tma_load_4d(dst, &kmap, 0, gk, row, 0, bar);
      } else {
#pragma unroll
        for (int i = 0; i < 2 * KSL; ++i)
          tma_load_4d(dst + i * kSlab, &kmap, (i % KSL) * 64, 2 * gk + i / KSL, row, 0, bar);
      }
      if (A.v_whole) {
        tma_load_4d(vdst, &vmap, 0, gk, row, 0, bar);
      } else {
        for (int k = 0; k < A.vslabs; ++k)
          tma_load_4d(vdst + k * kSlab, &vmap, k * 64, gk, row, 0, bar);
      }
    }
    __syncwarp();
    // tiles below `stages` come one after another, later ones in step with
    // the warp's own
    const int step = next_tile + kWarps < stages || next_tile >= stages
                         ? kWarps
                         : warp + stages - next_tile;
    next_tile += step;
    if (next_tile < count) {
      cursor_step(A, lc, step, nseq);
      next_page = page_of();
    }
  };
  for (int t = warp; t < stages; t += kWarps) issue(t);

  // ---- the (sequence, kv head, chunk)s of the part, one after another
  int n = warp;      // this warp's next tile of the CTA, its stage and parity
  int st = warp % stages;
  uint32_t par = (uint32_t)(warp / stages) & 1u;
  int at = 0;        // tiles of the CTA before the current segment
  bool ok = true;
  // ldmatrix addresses within a slab: keys (scores): lanes 0-7 keys 0-7 chunk
  // 0, 8-15 keys 0-7 chunk 1, 16-23 keys 8-15 chunk 0, 24-31 keys 8-15 chunk 1;
  // values (transposed): lanes 8-15 are keys 8-15 of chunk 0
  const uint32_t k_row = (lane & 7) + ((lane >> 4) << 3), k_hc = (lane >> 3) & 1;
  const uint32_t v_row = (lane & 7) + (((lane >> 3) & 1) << 3), v_hc = lane >> 4;
  const uint32_t k_off = k_row * 128 + ((k_hc ^ (k_row & 7)) << 4);
  const uint32_t v_off = v_row * 128 + ((v_hc ^ (v_row & 7)) << 4);
  Cursor cur = first;
  while (at < count) {
    const int seg = min(cur.tiles - cur.tile, count - at);  // tiles of this segment
    if (seg <= 0 || cur.seq >= nseq) break;  // (the lengths changed under the kernel)
    const int gk = cur.gc / A.chunks;
    const int h0 = gk * A.grp + (cur.gc - gk * A.chunks) * kHeads;
    const int nh = min(kHeads, A.grp - (cur.gc - gk * A.chunks) * kHeads);
    // the query rows, rotated, as A fragments of each map: rows 0-7 the heads'
    // values, rows 8-15 the remainders; [map][k step][lane] of four registers
    {
      for (int i = tid; i < kRows * KS * 2; i += kWarps * 32) {
        const int m = i & 1, hh = (i >> 1) & 7, d0 = (i >> 4) * 8;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (hh < nh && d0 < hs) {
          const T* row = (const T*)a.query + ((cur.t * g.H + h0 + hh) * 2 + m) * (int64_t)hs;
          unpack8<T>(*reinterpret_cast<const uint4*>(row + d0), x);
          if (g.rd > 0 && d0 >= g.ro && d0 < g.ro + g.rd) {
            const int half = g.rd >> 1;
            const int dp = g.interleaved ? d0 : d0 - g.ro < half ? d0 + half : d0 - half;
            float xp[8];
            unpack8<T>(*reinterpret_cast<const uint4*>(row + dp), xp);
            rope8<T>(x, xp, d0, g.ro, g.rd, g.interleaved, (const T*)a.cos_cache + cur.pos * half,
                     (const T*)a.sin_cache + cur.pos * half);
          }
        }
        uint32_t* f = reinterpret_cast<uint32_t*>(q_s + (m * KS + (d0 >> 4)) * 32 + hh * 4) +
                      (d0 & 8 ? 2 : 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) split2<T>(x[2 * e], x[2 * e + 1], f + 4 * e, f + 4 * e + 1);
      }
      __syncthreads();
    }

    float o[VT][4];
#pragma unroll
    for (int i = 0; i < VT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool bad = false;
    for (; n < at + seg; n += kWarps) {
      if (ok)
        ok = __all_sync(0xffffffffu,
                        wait_tile(&s_full[st], &s_last[st], n, par, &s_abort, a.err_flags));
      if (!ok) {
        bad = true;
        continue;
      }
      bad |= s_stage_bad[st] != 0;
      const uint32_t kb = ring + st * A.stage + k_off;
      const uint32_t vb0 = ring + st * A.stage + 2 * KSL * kSlab;
      const uint32_t vb = vb0 + v_off;

      // scores of both maps, two halves of 8 keys each
      float s[2][2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][j][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 q = q_s[(i * KS + ks) * 32 + lane];
          uint32_t k[4];
          ldsm4(k, (kb ^ ((ks & 3) << 5)) + (i * KSL + (ks >> 2)) * kSlab);
          mma<T>(s[i][0], q.x, q.y, q.z, q.w, k[0], k[1]);
          mma<T>(s[i][1], q.x, q.y, q.z, q.w, k[2], k[3]);
        }
      }
      // v[map][8-key half][key of the pair], log2 domain
      float v[2][2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) v[i][j][e] = s[i][j][e] + s[i][j][2 + e];
      if (A.cap_out > 0.f) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) v[i][j][e] = A.cap_out * tc::tanh_ex2(v[i][j][e] * A.cap_in);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) v[i][j][e] *= A.scale_log2;
      }
      const int64_t key0 = (cur.lo / kTileKeys + cur.tile + (n - at)) * kTileKeys;
      if (key0 < cur.lo || key0 + kTileKeys - 1 > cur.pos) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int64_t key = key0 + j * 8 + (lane & 3) * 2 + e;
            if (key < cur.lo || key > cur.pos) v[0][j][e] = v[1][j][e] = -INFINITY;
          }
        // zero the value rows of those keys: 16-byte pieces, a row after another
        for (int i = lane; i < kTileKeys * A.vslabs * 8; i += 32) {
          const int r = (i >> 3) & 15;
          if (key0 + r < cur.lo || key0 + r > cur.pos)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             vb0 + (i >> 7) * kSlab + r * 128 + (i & 7) * 16),
                         "r"(0)
                         : "memory");
        }
        tc::fence_proxy_async();  // before the stage's next copy
        __syncwarp();
      }
      // running maxima (each head's row is held by four lanes)
      float f[2] = {1.f, 1.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float t = fmaxf(fmaxf(v[i][0][0], v[i][0][1]), fmaxf(v[i][1][0], v[i][1][1]));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        if (t > mx[i] + Prob<T>::lazy || mx[i] == -INFINITY) {
          f[i] = mx[i] == -INFINITY ? 0.f : ex2(mx[i] - t);
          mx[i] = t;
          l[i] *= f[i];
        }
      }
      if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
        for (int c = 0; c < VT; ++c) {
          o[c][0] *= f[0];
          o[c][1] *= f[0];
          o[c][2] *= f[1];
          o[c][3] *= f[1];
        }
      }
      // probabilities as A fragments: rows 0-7 map 0, rows 8-15 map 1
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mu = (mx[i] == -INFINITY ? 0.f : mx[i]) - Prob<T>::shift;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p0 = ex2(v[i][j][0] - mu), p1 = ex2(v[i][j][1] - mu);
          l[i] += p0 + p1;
          split2<T>(p0, p1, &ph[j * 2 + i], &pl[j * 2 + i]);
        }
      }
      // o += P V: the 16 keys are one k step; four 8-channel tiles at a
      // time, so that the two products of a tile are not back to back
#pragma unroll
      for (int c = 0; c < VT; c += 4) {
        if (c < nvt) {
          uint32_t w[4], x[4];
          ldsm4_t(w, (vb ^ ((c & 4) << 4)) + (c >> 3) * kSlab);
          ldsm4_t(x, (vb ^ (((c & 4) + 2) << 4)) + (c >> 3) * kSlab);
          mma<T>(o[c], ph[0], ph[1], ph[2], ph[3], w[0], w[1]);
          mma<T>(o[c + 1], ph[0], ph[1], ph[2], ph[3], w[2], w[3]);
          mma<T>(o[c + 2], ph[0], ph[1], ph[2], ph[3], x[0], x[1]);
          mma<T>(o[c + 3], ph[0], ph[1], ph[2], ph[3], x[2], x[3]);
          mma<T>(o[c], pl[0], pl[1], pl[2], pl[3], w[0], w[1]);
          mma<T>(o[c + 1], pl[0], pl[1], pl[2], pl[3], w[2], w[3]);
          mma<T>(o[c + 2], pl[0], pl[1], pl[2], pl[3], x[0], x[1]);
          mma<T>(o[c + 3], pl[0], pl[1], pl[2], pl[3], x[2], x[3]);
        }
      }
      __syncwarp();
      issue(st);
      for (st += kWarps; st >= stages; st -= stages) par ^= 1;
    }

    // ---- the warps' results, joined in the order of the warps
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if ((lane & 3) == 0) {
        s_m[warp][i * 8 + (lane >> 2)] = mx[i];
        s_l[warp][i * 8 + (lane >> 2)] = l[i];
      }
    }
    if (lane == 0) s_bad[warp] = bad ? 1 : 0;
    __syncthreads();
    const int64_t pair = (int64_t)cur.seq * A.ng + cur.gc;
    const int64_t slot = (int64_t)blockIdx.x + pair;
    float w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 8 + (lane >> 2);
      float M = s_m[0][r];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) M = fmaxf(M, s_m[k][r]);
      w[i] = mx[i] == -INFINITY ? 0.f : ex2(mx[i] - M);
      if (warp == kWarps - 1 && (lane & 3) == 0) {
        float L = 0.f;
        bool any = false;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          L += s_m[k][r] == -INFINITY ? 0.f : ex2(s_m[k][r] - M) * s_l[k][r];
          any |= s_bad[k] != 0;
        }
        A.ws_ml[slot * kRows + r] = make_float2(M, any ? -1.f : L);
      }
    }
    // 64 channels at a time: every warp leaves its rows in shared memory, thread
    // (row, four channels) adds them up. (Warp after warp adding to one buffer
    // took 17000 cycles a segment at 128 / 256, this 6000.)
#pragma unroll
    for (int cc = 0; cc < VT / 8; ++cc) {
      if (cc * 8 < nvt) {
        if (cc > 0) __syncthreads();  // (behind the reads of the chunk before)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float* row = join + (warp * kRows + i * 8 + (lane >> 2)) * kJoinPitch + (lane & 3) * 2;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float2*>(row + c * 8) =
                make_float2(o[cc * 8 + c][2 * i] * w[i], o[cc * 8 + c][2 * i + 1] * w[i]);
        }
        __syncthreads();
        const int r = tid >> 4, c = (tid & 15) * 4;
        if ((r & 7) < nh && cc * kJoin + c < vhs) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kWarps; ++k) {
            const float4 y =
                *reinterpret_cast<const float4*>(join + (k * kRows + r) * kJoinPitch + c);
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
          }
          *reinterpret_cast<float4*>(A.ws_o + (slot * kRows + r) * (int64_t)vhs + cc * kJoin + c) = x;
        }
      }
    }
    // one thread moves on to the next segment, so that all warps agree on it
    at += seg;
    if (tid == 0 && at < count) {
      cursor_step(A, cur, seg, nseq);
      s_cur = cur;
    }
    __syncthreads();
    if (at < count) cur = s_cur;
  }
  if (!waited) grid_dep_wait();
  // after a wait that gave up, or a part left early because the lengths changed,
  // copies may still be in flight
  __syncthreads();
  if ((s_abort || at < count) && tid < stages && s_last[tid] >= 0)
    tc::drain_wait(smem_u32(&s_full[tid]), (uint32_t)(s_last[tid] / stages) & 1u, a.err_flags);
}

// Joins the parts of each (sequence, head), takes the difference of the two
// maps and the norm. One CTA per (sequence, kv head, chunk), one warp per
// head, lane = channels lane, lane + 32, ...; parts of one head lie in
// consecutive slots. Latency bound: one round trip for the plan, one per four
// parts.
template <typename T>
__global__ void __launch_bounds__(kHeads * 32) diff_combine_kernel(const __grid_constant__ Args A) {
  const Geometry& g = A.g;
  const DiffArgs& a = A.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nseq = a.seq_end - a.seq_begin;
  const int x = blockIdx.x, gc = blockIdx.y;
  const int gk = gc / A.chunks, first = (gc - gk * A.chunks) * kHeads;
  const int hs = g.hs, vhs = g.vhs;
  // weights and the sequence: older than the attention kernel
  float d0 = 0.f, d1 = 0.f;
  const float* lv = a.lambda_vectors;
  for (int d = lane; d < hs; d += 32) {
    d0 = fmaf(lv[d], lv[hs + d], d0);
    d1 = fmaf(lv[2 * hs + d], lv[3 * hs + d], d1);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    d0 += __shfl_xor_sync(0xffffffffu, d0, o);
    d1 += __shfl_xor_sync(0xffffffffu, d1, o);
  }
  const float lam = expf(d0) - expf(d1) + a.lambda_init;
  float nw[8];
#pragma unroll
  for (int c = 0; c < 8; ++c)
    nw[c] = c * 32 + lane < vhs ? Half<T>::to_f32(((const T*)a.norm_weight)[c * 32 + lane]) : 0.f;
  const Seq s = seq_of(A, a.seq_begin + x);
  grid_dep_wait();
  if (s.status && gc == 0 && threadIdx.x == 0) raise_flag(a.err_flags, s.err);
  if (s.status == 1 || first + warp >= A.grp) return;
  const int h = gk * A.grp + first + warp;
  T* out = (T*)a.out + (s.t * g.H + h) * (int64_t)vhs;
  if (s.status) {
    for (int c = lane; c < vhs; c += 32) out[c] = Half<T>::from_f32(0.f);
    return;
  }
  const int64_t total = A.ws_plan[nseq], ctas = A.ws_plan[nseq + 1];
  const int64_t tiles = s.pos / kTileKeys - s.lo / kTileKeys + 1;
  const int64_t t0 = A.ws_plan[x] + gc * tiles, t1 = t0 + tiles - 1;
  // the CTA of line tile t: the last whose part starts at or before it
  const int64_t c0 = ((t0 + 1) * ctas - 1) / total, c1 = ((t1 + 1) * ctas - 1) / total;
  const int64_t slot0 = c0 + (int64_t)x * A.ng + gc;
  // (within the workspace even if the lengths changed under the kernels)
  const int parts = (int)max((int64_t)0, min(c1 - c0 + 1, A.slots - slot0));
  float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f}, o[2][8] = {};
  bool bad = false;
  for (int p0 = 0; p0 < parts; p0 += 4) {
    float2 ml[2][4];
    float v[2][4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ml[i][k] = make_float2(-INFINITY, 0.f);
        if (p0 + k < parts) {
          const int64_t row = (slot0 + p0 + k) * kRows + i * 8 + warp;
          ml[i][k] = A.ws_ml[row];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c * 32 + lane < vhs) v[i][k][c] = A.ws_o[row * vhs + c * 32 + lane];
        }
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float m = ml[i][k].x;
        bad |= ml[i][k].y < 0.f;
        if (!(ml[i][k].y <= 0.f)) {  // (a sum that is not a number counts)
          if (m > M[i]) {
            const float f = ex2(M[i] - m);
            L[i] *= f;
#pragma unroll
            for (int c = 0; c < 8; ++c) o[i][c] *= f;
            M[i] = m;
          }
          const float w = ex2(m - M[i]);
          L[i] += w * ml[i][k].y;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c * 32 + lane < vhs) o[i][c] = fmaf(w, v[i][k][c], o[i][c]);
        }
      }
  }
  const float i0 = 1.f / L[0], i1 = lam / L[1];
  float r[8], ss = 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    r[c] = c * 32 + lane < vhs ? o[0][c] * i0 - o[1][c] * i1 : 0.f;
    ss = fmaf(r[c], r[c], ss);
  }
#pragma unroll
  for (int q = 16; q > 0; q >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, q);
  const float inv = (1.f - a.lambda_init) / sqrtf(ss / (float)vhs + a.norm_eps);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int ch = c * 32 + lane;
    if (ch < vhs)
      out[ch] = Half<T>::from_f32(bad ? 0.f : r[c] * inv * nw[c]);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct Plan {
  int vslabs, stage, stages, ks, vt;
  size_t smem;
};

Plan plan_of(const Geometry& g) {
  Plan p;
  p.ks = g.hs <= 64 ? 4 : 8;
  p.vt = g.vhs <= 128 ? 16 : 32;
  p.vslabs = (g.vhs + 63) / 64;
  p.stage = kSlab * (p.ks / 2 + p.vslabs);
  const size_t fixed = 1024 + (size_t)p.ks * 32 * 16 * 2 +
                       (size_t)kWarps * kRows * kJoinPitch * 4;
  const int s = (int)((kSmem - fixed) / (size_t)p.stage);
  p.stages = s > kMaxStages ? kMaxStages : s;
  p.smem = fixed + (size_t)p.stages * p.stage;
  return p;
}

struct Layout {
  int ctas, chunks, ng;
  int64_t slots;
  size_t o, ml, bytes;
};
Layout layout_of(const Geometry& g, const Plan& p, int64_t nseq) {
  Layout l;
  l.chunks = (g.H / g.kvh + kHeads - 1) / kHeads;
  l.ng = g.kvh * l.chunks;
  l.ctas = g.num_sms;
  l.slots = l.ctas + nseq * l.ng;
  l.o = ((size_t)l.slots * kRows * g.vhs * 4 + 255) & ~(size_t)255;
  l.ml = ((size_t)l.slots * kRows * 8 + 255) & ~(size_t)255;
  l.bytes = l.o + l.ml + (size_t)(nseq + 2) * 8;
  return l;
}

// A cache of `heads` rows of `width` channels per slot, as (channel, head, slot,
// slab), in boxes of 16 slots. With `whole` (a width that is a multiple of 64)
// the channels are cut into slabs of 64 (the fourth dimension, 128 bytes apart)
// and one box holds a row's slabs one after another; otherwise a box holds one
// slab and the channel dimension ends at the width (zeros behind it).
cudaError_t cache_map(CUtensorMap* map, bool bf16, const void* base, int width, int heads,
                      int64_t slots, bool whole) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t wb = (cuuint64_t)width * 2;
  const cuuint32_t slabs = whole ? (cuuint32_t)(width / 64) : 1u;
  const cuuint64_t dims[4] = {whole ? 64u : (cuuint64_t)width, (cuuint64_t)heads,
                              (cuuint64_t)slots, slabs};
  const cuuint64_t str[3] = {wb, wb * heads, 128};
  const cuuint32_t box[4] = {64, 1, kTileKeys, slabs}, estr[4] = {1, 1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(base), dims, str, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <typename T, int KS, int VT>
cudaError_t launch(const Args& A, const Plan& p, int ctas, cudaStream_t stream) {
  static std::atomic<bool> configured[64];
  auto kern = diff_decode_kernel<T, KS, VT>;
  cudaError_t e = once_per_device(configured, A.g.device, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const int64_t slots = (int64_t)A.g.num_blocks * A.g.bs;
  CUtensorMap kmap, vmap;
  if (e == cudaSuccess)  // (both maps of a kv head are one row of 2 hs channels)
    e = A.k_whole ? cache_map(&kmap, bf16, A.a.key_cache, 2 * A.g.hs, A.g.kvh, slots, true)
                  : cache_map(&kmap, bf16, A.a.key_cache, A.g.hs, 2 * A.g.kvh, slots, false);
  if (e == cudaSuccess)
    e = cache_map(&vmap, bf16, A.a.value_cache, A.g.vhs, A.g.kvh, slots, A.v_whole);
  if (e == cudaSuccess)
    e = tc::launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), p.smem, stream, kmap, vmap, A);
  if (e != cudaSuccess) return e;
  return tc::launch_pdl(diff_combine_kernel<T>,
                        dim3((unsigned)(A.a.seq_end - A.a.seq_begin), (unsigned)A.ng),
                        dim3(kHeads * 32), 0, stream, A);
}

}  // namespace

size_t decode_workspace(const Geometry& g, int64_t nseq) {
  return layout_of(g, plan_of(g), nseq).bytes;
}

cudaError_t launch_decode(const Geometry& g, const DiffArgs& a) {
  const Plan p = plan_of(g);
  const Layout l = layout_of(g, p, a.seq_end - a.seq_begin);
  Args A{};
  A.g = g;
  A.a = a;
  A.grp = g.H / g.kvh;
  A.chunks = l.chunks;
  A.ng = l.ng;
  A.vslabs = p.vslabs;
  A.k_whole = g.hs % 64 == 0;
  A.v_whole = g.vhs % 64 == 0;
  A.stage = p.stage;
  A.stages = p.stages;
  A.slots = l.slots;
  A.scale_log2 = g.scale * tc::kLog2e;
  A.cap_in = g.softcap > 0.f ? g.scale / g.softcap : 0.f;
  A.cap_out = g.softcap > 0.f ? g.softcap * tc::kLog2e : 0.f;
  char* w = static_cast<char*>(a.workspace);
  A.ws_o = reinterpret_cast<float*>(w);
  A.ws_ml = reinterpret_cast<float2*>(w + l.o);
  A.ws_plan = reinterpret_cast<int64_t*>(w + l.o + l.ml);
  auto go = [&](auto* typed) -> cudaError_t {
    using T = std::remove_pointer_t<decltype(typed)>;
    if (p.ks == 4 && p.vt == 16) return launch<T, 4, 16>(A, p, l.ctas, a.stream);
    if (p.ks == 4) return launch<T, 4, 32>(A, p, l.ctas, a.stream);
    if (p.vt == 16) return launch<T, 8, 16>(A, p, l.ctas, a.stream);
    return launch<T, 8, 32>(A, p, l.ctas, a.stream);
  };
  return g.dtype == PA_DTYPE_BF16 ? go((__nv_bfloat16*)nullptr) : go((__half*)nullptr);
}

}  // namespace diff
}  // namespace pa
