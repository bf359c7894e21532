// Attention over 8-bit caches, prefill: any number of new tokens per sequence
// (include/pa_quant.h), on the tensor cores (tcgen05, TMEM).
//
// A work unit is QT tiles of up to 128 query rows of one kv head: tpc consecutive
// tokens of one sequence x the kv head's grp heads each. Its visible keys are cut
// into tiles of N. Where a batch has too few units for the GPU, several CTAs share
// a unit's tiles and quant_join_kernel adds up their parts.
//
// Inside a CTA:
//   warp 25      copies a tile's codes (TMA through the block table), C tiles ahead
//   warp 26      a tile's scales: pages two tiles ahead, scales one
//   warps 16-23  write codes as fp16 (exactly) in the layout the products read, four
//                warps keys and four values, into rings of R key and R value tiles. Both
//                query tiles use what is converted once.
//   warp 24      S = Q K^T (N columns of TMEM per buffer), O += P V (A = P from TMEM,
//                written over its S). Two buffers per query tile: scores run two key tiles
//                ahead, so that a softmax does not wait for them.
//   warps 0-15   softmax, two threads per row, each with half of a tile's keys and of the
//                output's channels (QT 1: warps 0-7). Per tile the two tell each other
//                whether a maximum rises by more than kLazy, which is rare (pair_any).
// TMEM columns: O, 128 for each of two query tiles or 256 for one | 2 QT buffers of N |
// QT 1: the queries' second addends.
//
// Scales cost next to nothing: a page's rows come 16 at a time, so 16 columns of S
// have one key scale, which joins the factor of the exponent's multiply-add, and one
// value scale 2^e, whose e joins its addend (see kShift in pa_quant_read.cuh). The sum of
// the 16 probabilities is multiplied by 2^-e again.
//
// Measured: some 4096 tokens each behind 4096 and 2096, 32 heads over 8 of 128 / 128, 775 us in bf16
// and 937 in fp16 (queries in two addends); the products alone take 360 at the card's
// bf16 rate. What bounds it is the way of one tile through a softmax, some 2000 cycles, and
// the instructions along it: 13 per warp of scores, issue slots 67 % in use. Without the products
// it takes 721 us, without exponentials and conversion 713, without either 657. One thread per row (64 exponentials each) took 790,
// tiles of 128 keys with one buffer per query tile no less.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "pa_diff_common.cuh"
#include "pa_quant_plan.h"
#include "pa_quant_read.cuh"

namespace pa {
namespace quant {
namespace {

using namespace pa::tc;

constexpr int kConvWarp = 16, kMmaWarp = 24, kCopyWarp = 25, kScaleWarp = 26, kThreads = 28 * 32;
constexpr int kSlab = kRows * 128;  // bytes of a 64-channel slab of 128 query rows
constexpr int N = 64;               // keys of a tile
constexpr int kMaxRing = 4, kAhead = 8;  // tiles converted ahead; tiles whose scales are kept

struct Bars {
  uint64_t q_full, k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t s_full[4], p_full[4], sc_full[kAhead], pv_done[2], drain;
  uint64_t c_full[4], c_empty[4];  // codes: two of keys, two of values
  uint32_t tmem_base;
  int bad, abort, any_odd;
  // keys with a NaN value that some rows of the unit see and others do not: position
  // pos + 1 + i (after the first token) in the first eight words, lo + i (before the
  // last one's window) behind
  uint32_t odd[16];
};
constexpr int kNumBars = 1 + 4 * kMaxRing + 8 + kAhead + 3 + 8;

struct PreP {
  ReadP R;
  float* ws_o;   // [planned * splits][QT * 128][vhs]
  float2* ws_ml; // [planned * splits][QT * 128] maximum (log2 domain; NaN: an invalid page), sum
  int64_t num_slots;
  int box;       // rows of a copy: min(bs, N)
  int tpc;       // tokens of a query tile
  int few;       // sequences of no more tokens are another kernel's
  int planned, splits;  // units x kv heads that are split, CTAs of each (see prefill_part)
  int slabs, vslabs, klpr, vlpr;  // 64-channel slabs, lanes for a row's 8-byte pieces
};

// wait_bar in less code (that of a CTA's roles together has to fit the instruction
// caches) and fewer instructions. IDLE: for roles that run ahead, which sleep between two looks.
template <bool IDLE>
__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t par, volatile int* abort,
                                           int32_t* err) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_try_wait(bar, par); ++i) {
    if (IDLE) __nanosleep(256);
    if (i & 63) continue;
    if (*abort) return false;
    const uint64_t t = globaltimer();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitLimitNs) {
      *abort = 1;
      raise_flag(err, PA_DEVERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

struct Unit {
  int64_t t, pos, lo, lo_hi, pos_hi, last0;  // see resolve()
  int b, ntok, begin, n;                     // sequence, tokens, first tile, tiles
  int status;                                // 0 run, 1 nothing, 2 told already
};

// Unit `unit` of the batch, by a warp: the sequences' units in order, the last
// ones (with the most keys) first. first..: what is filled in for all lanes.
template <int QT>
__device__ Unit resolve(const PreP& A, int unit, int split, int splits, int lane) {
  const ReadP& P = A.R;
  const int per = QT * A.tpc;
  auto units_of = [&](int i, int* q0, int* q) {
    *q0 = *q = 0;
    if (i < P.nseq) {
      *q0 = P.cumseq[P.seq_begin + i];
      *q = (int)((uint32_t)P.cumseq[P.seq_begin + i + 1] - (uint32_t)*q0);  // (of any offsets)
      if (*q <= A.few) *q = 0;
    }
    return *q > 0 ? (*q - 1) / per + 1 : 0;
  };
  Unit u{};
  u.status = 1;
  int total = 0, q0, q;
  for (int base = 0; base < P.nseq; base += 32) total += units_of(base + lane, &q0, &q);
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (unit >= total) return u;
  unit = total - 1 - unit;
  int run = 0;
  for (int base = 0; base < P.nseq; base += 32) {
    const int cnt = units_of(base + lane, &q0, &q);
    int incl = cnt;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int start = run + incl - cnt;
    const unsigned who = __ballot_sync(0xffffffffu, unit >= start && unit < start + cnt);
    if (who) {
      const int src = __ffs(who) - 1;
      const int at = __shfl_sync(0xffffffffu, unit - start, src) * per;
      q0 = __shfl_sync(0xffffffffu, q0, src);
      q = __shfl_sync(0xffffffffu, q, src);
      u.b = P.seq_begin + base + src;
      const int64_t past = P.past[u.b];
      u.t = (int64_t)q0 + at;
      u.ntok = min(per, q - at);
      u.pos = past + at;
      u.pos_hi = P.cross ? past - 1 : u.pos + u.ntok - 1;  // the last key that any row sees
      u.last0 = P.cross ? past - 1 : u.pos;                // that all rows see, from below
      u.lo = P.window >= 0 ? max((int64_t)0, u.pos - P.window) : 0;
      u.lo_hi = P.window >= 0 ? max((int64_t)0, u.pos_hi - P.window) : 0;
      u.status = 0;
      if (past < 0 || u.pos_hi >= (int64_t)P.max_blocks * P.bs)
        u.status = PA_DEVERR_CONTEXT;
      else if (u.t < 0 || u.t + u.ntok > P.num_tokens)
        u.status = PA_DEVERR_CUMSEQ;
      else if (P.rd > 0 && u.pos_hi >= P.cos_rows)
        u.status = PA_DEVERR_POSITION;
      if (u.status == 0 && u.pos_hi >= u.lo) {
        const int first = (int)(u.lo / N), all = (int)(u.pos_hi / N) + 1 - first;
        const int s0 = (int)((int64_t)all * split / splits);
        u.begin = first + s0;
        u.n = (int)((int64_t)all * (split + 1) / splits) - s0;
      }
      return u;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  return u;
}

__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(bar));
}
__device__ __forceinline__ uint64_t pack_f32(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpack_f32(uint64_t v, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
// Registers of a warpgroup's threads, out of what the block was launched with:
// 72 for each of seven warpgroups, 4 x kSoftRegs + 2 x kConvRegs + kMmaRegs = 504.
constexpr int kSoftRegs = 80, kConvRegs = 64, kMmaRegs = 56;
static_assert(4 * kSoftRegs + 2 * kConvRegs + kMmaRegs <= 7 * 72, "registers");
// Two warps that share 32 rows of a query tile.
__device__ __forceinline__ void pair_sync(int pair) {
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");
}
__device__ __forceinline__ bool pair_any(int pair, bool x) {
  uint32_t any;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, %2, 64, p;\n"
      " selp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"((uint32_t)x), "r"(pair + 1)
      : "memory");
  return any;
}
// Floats as integers of the same order.
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) {
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}
// 2^-e of a whole number e held as a float.
__device__ __forceinline__ float inverse_pow2(float e) {
  return __int_as_float((127 << 23) - (__float_as_int(e + 12582912.f) << 23));
}
template <int R>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
// The query rows of a tile (token, head), normalized and rotated, as fp16 in
// swizzled slabs; mult: what takes the factor of the lane's row back, times the scale. Rows behind
// the last are zeros. By the tile's eight warps, 16 rows each: rows of the warp's quad from
// 16 part on. mult: of the 32 rows, by way of s_row. Rows in two addends (two_addends): the
// second one into rest_s, laid out the same, and from there into TMEM where rest_t names
// columns.
template <typename T>
__device__ __noinline__ void load_query(const PreP& A, const Unit& u, int g, int tile, int rows,
                                        int warp, int part, int pair, int lane, uint8_t* q_s,
                                        uint8_t* rest_s, uint32_t rest_t, float* s_row, float* mult) {
  const ReadP& P = A.R;
  int lpr = 2;
  while (lpr * 8 < P.hs) lpr <<= 1;
  const int d0 = (lane & (lpr - 1)) * 8, step = 32 / lpr, half = P.rd >> 1;
  auto place = [&](int row) {
    return reinterpret_cast<uint4*>(q_s + (d0 >> 6) * kSlab + row * 128 +
                                    ((((d0 >> 3) & 7) ^ (row & 7)) << 4));
  };
  constexpr bool kRest = std::is_same<T, __half>::value;
  // all rows on their way, to the places where they are changed
#pragma unroll 4
  for (int r0 = 16 * part; r0 < 16 * part + 16; r0 += step) {
    const int row = warp * 32 + r0 + lane / lpr;
    const bool live = row < rows;
    const int tok = live ? row / P.grp : 0, h = live ? row - tok * P.grp : 0;
    const T* src = reinterpret_cast<const T*>(P.query) +
                   ((u.t + tile * A.tpc + tok) * P.H + g * P.grp + h) * P.hs + d0;
    if (d0 < P.hs)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(place(row))),
                   "l"(live ? src : reinterpret_cast<const T*>(P.query)), "r"(live ? 16 : 0)
                   : "memory");
  }
  const int mine = warp * 32 + 16 * part + lane;
  if (P.rd > 0 && lane < 16 && mine < rows) {  // and the rows' angles
    const int64_t at = (u.pos + tile * A.tpc + mine / P.grp) * half;
    for (int c = 0; c < half; c += 64) {
      asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const T*>(P.cos_cache) + at + c));
      asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const T*>(P.sin_cache) + at + c));
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
  for (int r0 = 16 * part; r0 < 16 * part + 16; r0 += step) {
    const int row = warp * 32 + r0 + lane / lpr;
    const bool live = row < rows;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (d0 < P.hs) unpack8<T>(*place(row), x);
    norm_rotate8<T>(x, live, d0, P.hs, lpr, reinterpret_cast<const T*>(P.q_norm), P.eps, P.ro, P.rd,
                    P.interleaved, reinterpret_cast<const T*>(P.cos_cache),
                    reinterpret_cast<const T*>(P.sin_cache),
                    u.pos + tile * A.tpc + (live ? row / P.grp : 0));
    uint4 hx;
    uint4 rest;
    const float back = scaled_row8(x, &hx, &rest, lpr);
    if (d0 < P.hs) {
      *place(row) = hx;
      if (kRest && P.two) *(place(row) + ((rest_s - q_s) >> 4)) = rest;
    }
    if ((lane & (lpr - 1)) == 0) s_row[row] = back;
  }
  __syncwarp();
  pair_sync(pair);
  if (kRest && rest_t) {  // (channels behind hs are not multiplied)
    const int row = warp * 32 + lane;
    for (int c = part; c < A.slabs; c += 2) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(rest_s + c * kSlab + row * 128 + ((i ^ (row & 7)) << 4));
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
      tmem_st32(rest_t + c * 32, w);
    }
    tmem_wait_st();
    tc_fence_before();
  }
  *mult = s_row[warp * 32 + lane] * (P.cap_in > 0.f ? P.cap_in : P.scale_log2);
}

// mma_ss and mma_ts with descriptors of a common upper word.
__device__ __forceinline__ void mma_ss_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                          uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n"
      " mov.b64 y, {%2, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                          uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts64(uint32_t a, uint2 v) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(v.x), "r"(v.y) : "memory");
}
// A masked score. (As an instruction of its own: the compiler turned a branch around 64
// selections into selections that every tile goes through.)
__device__ __forceinline__ void hide_unless(uint32_t seen, uint32_t& x) {
  asm volatile("{\n .reg .pred p;\n setp.eq.u32 p, %1, 0;\n @p mov.b32 %0, 0xff800000;\n}\n"
               : "+r"(x)
               : "r"(seen));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

// CAP: 0 no softcap, 1 one, 2 a wide one (capped).
template <int QT, int R, int C, int CAP, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
quant_prefill_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PreP A) {
  constexpr int kSegs = N / 16;
  constexpr int kColS = 256;      // first column of the S buffers
  constexpr int kKBox = N * 128;  // bytes of a 64-channel slab of N keys
  const ReadP& P = A.R;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit s_unit;
  __shared__ Bars bars_s;
  __shared__ float2 s_scale[kAhead][kSegs];  // key scale, exponent e of the value's
  __shared__ int s_row[QT * kRows];  // rows' factors, maxima, sums, in turn
  __shared__ int s_fail[QT * 4];  // 1 + the tile at which a pair's warps give up
  __shared__ int2 s_in[kAhead];  // segments with a key, a value scale (or nothing to see), a bit each
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  Bars* bars = &bars_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q_bytes = A.slabs * kSlab, k_bytes = A.slabs * kKBox, v_bytes = A.vslabs * kKBox;
  uint8_t* q_s = smem;
  // (the queries' second addends: behind the first ones, or in TMEM behind the scores, by
  // way of the keys' ring, which is as large as they are)
  uint8_t* k_s = q_s + (QT == 2 && TWO ? 2 : 1) * QT * q_bytes;
  constexpr int kColRest = kColS + 2 * N;
  uint8_t* v_s = k_s + R * k_bytes;
  uint8_t* codes = v_s + R * v_bytes;  // C key tiles, C value tiles
  const int g = prefill_part(blockIdx.x, A.planned, A.splits).at % P.kvh;

  if (!P.early) grid_dep_wait();
  if (warp == 0) {
    const PrefillPart part = prefill_part(blockIdx.x, A.planned, A.splits);
    const int split = part.split;
    Unit u = resolve<QT>(A, part.at / P.kvh, split, part.splits, lane);
    if (u.status > 1) {  // invalid positions: told, and zeros
      if (lane == 0 && g == 0 && split == 0) raise_flag(P.err_flags, u.status);
      const int64_t t0 = max((int64_t)0, u.t), t1 = min(u.t + u.ntok, P.num_tokens);
      if (split == 0)
        for (int64_t t = t0; t < t1; ++t) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(P.out) + (t * P.H + g * P.grp) * P.vhs / 2;
          for (int i = lane; i < P.grp * P.vhs / 2; i += 32) dst[i] = 0;
        }
      u.status = 2;
    }
    if (lane == 0) s_unit = u;
  } else if (warp == 1) {
    uint64_t* all = &bars->q_full;
    for (int i = lane; i < kNumBars; i += 32) {
      uint64_t* at = all + i;
      uint32_t count = 1;
      if (at == &bars->q_full) count = QT * 8;
      if ((at >= bars->k_full && at < bars->k_full + kMaxRing) ||
          (at >= bars->v_full && at < bars->v_full + kMaxRing))
        count = 4;
      if (at >= bars->c_empty && at < bars->c_empty + 4) count = 4;
      if (at >= bars->p_full && at < bars->p_full + 4) count = 8;
      mbar_init(smem_u32(at), count);
    }
    if (lane < 16) bars->odd[lane] = 0;
    if (lane < QT * 4) s_fail[lane] = 0;
    if (lane == 0) bars->bad = bars->abort = bars->any_odd = 0;
    fence_barrier_init();
  } else if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  } else if (warp == kScaleWarp && blockIdx.x == 0) {  // offsets have to rise, within the tokens
    bool bad = false;
    for (int i = lane; i < P.nseq; i += 32) {
      const int c0 = P.cumseq[P.seq_begin + i], c1 = P.cumseq[P.seq_begin + i + 1];
      bad |= c0 < 0 || c0 > c1 || c1 > P.num_tokens;
    }
    if (bad) raise_flag(P.err_flags, PA_DEVERR_CUMSEQ);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort = &bars->abort;
  const Unit& U = s_unit;
  const bool run = U.status == 0;
  const int n = run ? U.n : 0;
  auto wait = [&](uint64_t* bar, uint32_t par) {
    return wait_short<false>(smem_u32(bar), par, abort, P.err_flags);
  };
  auto wait_idle = [&](uint64_t* bar, uint32_t par) {
    return wait_short<true>(smem_u32(bar), par, abort, P.err_flags);
  };
  const int qt = QT == 2 ? (warp >> 2) & 1 : 0;  // (softmax warps)
  const int half = QT == 2 ? warp >> 3 : warp >> 2;  // of a tile's keys, and of the channels
  const int quad = warp & 3, row = quad * 32 + lane;
  const int tok0 = qt * A.tpc, ntok = run ? max(0, min(A.tpc, U.ntok - tok0)) : 0;
  const int rows = ntok * P.grp;
  const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
  const bool soft = warp < QT * 8;
  const int pair = qt * 4 + quad;
  int* row_at = &s_row[qt * kRows + row];
  float m = -INFINITY, l = 0.f;
  bool ok = true;

  // (each role with its registers, and nothing common behind them but the end)
  if (warp < kConvWarp) {
    more_registers<kSoftRegs>();
    if (n > 0 && soft) {
      // =================== softmax ===================
      uint8_t* q_t = q_s + qt * q_bytes;
      float mult;
      float* s_back = reinterpret_cast<float*>(&s_row[qt * kRows]);
      if (P.bf16) load_query<__nv_bfloat16>(A, U, g, qt, rows, quad, half, pair, lane, q_t, q_t, 0, s_back,
                                            &mult);
      else load_query<__half>(A, U, g, qt, rows, quad, half, pair, lane, q_t,
                              QT == 2 ? q_t + QT * q_bytes : k_s,
                              QT == 1 && TWO ? lane_addr + kColRest : 0, s_back, &mult);
      fence_proxy_async();
      arrive_warp(&bars->q_full, lane);
      pair_sync(pair);
      if (half == 0) *row_at = ordered(-INFINITY);
      // keys counted from the first tile's first one
      const int64_t key0 = (int64_t)U.begin * N, pos_r = U.pos + tok0 + row / P.grp;
      const int last_r = (int)((P.cross ? U.pos_hi : min(pos_r, U.pos_hi)) - key0);
      const int lo_r = (int)((P.window >= 0 ? max((int64_t)0, pos_r - P.window) : 0) - key0);
      const int last0 = (int)(U.last0 - key0);
      const int lo_hi = (int)(U.lo_hi - key0);
      const uint32_t o_addr = lane_addr + (QT == 2 ? qt * 128 : 0);
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const int buf = qt + QT * (k & 1);
        const uint32_t par = (k >> 1) & 1;
        const uint32_t cols = lane_addr + kColS + buf * N;
        const int j0 = k * N;
        const bool edge = j0 < lo_hi || j0 + N - 1 > last0;
        // (S comes behind the conversion of its keys, and that behind the tile's scales)
        ok = __all_sync(0xffffffffu, ok && wait(&bars->s_full[buf], par));
        tc_fence_after();
        uint32_t x[32];
        tmem_ld32_nowait(cols + half * 32, x);
        const float2 sc[2] = {s_scale[k % kAhead][2 * half], s_scale[k % kAhead][2 * half + 1]};
        tmem_wait_ld();
        reg_fence(x);
        if (edge) {  // bits of the columns that the row sees
          const int j1 = j0 + half * 32;
          const int a = min(32, max(0, lo_r - j1)), b = max(-1, min(31, last_r - j1)) + 1;
          const uint32_t seen = (b < 32 ? (1u << b) - 1 : ~0u) & (a < 32 ? ~0u << a : 0u);
#pragma unroll
          for (int e = 0; e < 32; ++e) hide_unless(seen & (1u << e), x[e]);
        }
        // (a masked score, -inf, times 0 would be NaN)
        auto factor_of = [&](const float2& c) { return fmaxf(c.x * mult, 1e-37f); };
        auto at = [&](int i) { return __uint_as_float(x[i]); };
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v0 = max3(at(16 * i), at(16 * i + 1), at(16 * i + 2));
          float v1 = max3(at(16 * i + 3), at(16 * i + 4), at(16 * i + 5));
#pragma unroll
          for (int e = 6; e < 14; e += 4) {
            v0 = max3(v0, at(16 * i + e), at(16 * i + e + 1));
            v1 = max3(v1, at(16 * i + e + 2), at(16 * i + e + 3));
          }
          v0 = max3(fmaxf(v0, v1), at(16 * i + 14), at(16 * i + 15));
          const float f = factor_of(sc[i]);
          if (CAP) v0 = v0 == -INFINITY ? v0 : capped<CAP == 2>(P, v0 * f);
          top = fmaxf(top, fmaf(v0, CAP ? 1.f : f, sc[i].y));
        }
        // The row's maximum goes by both halves. (Both warps have read their scores behind
        // this, and P may go over them. A wait that ran out is told there: neither warp
        // may wait for the other alone.)
        float factor = 1.f;
        if (!ok && lane == 0) s_fail[pair] = k + 1;
        tc_fence_before();
        const bool rise = pair_any(pair, top > m + kLazy || !ok);
        tc_fence_after();
        if (rise) {
          atomicMax(row_at, ordered(top));
          pair_sync(pair);
          // (the other may be a tile ahead, and give up there)
          const int fail = *const_cast<volatile int*>(&s_fail[pair]);
          ok = fail == 0 || fail > k + 1;
          if (!ok) break;
          const float both = unordered(*const_cast<volatile int*>(row_at));
          if (both > m + kLazy) {
            factor = ex2(m - both);  // (from -inf: 0)
            m = both;
            l *= factor;
          }
        }
        const float nm = kShift - (m == -INFINITY ? 0.f : m);
        // in passes over the registers, so that the exponentials issue back to back
        float v[32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = factor_of(sc[h]);
          const float fe = CAP ? 1.f : f, add = nm + sc[h].y;
          const uint64_t f2 = pack_f32(fe, fe), a2 = pack_f32(add, add);
#pragma unroll
          for (int e = 16 * h; e < 16 * h + 16; e += 2) {
            float a = at(e), b = at(e + 1);
            if (CAP) {
              a = a == -INFINITY ? a : capped<CAP == 2>(P, a * f);
              b = b == -INFINITY ? b : capped<CAP == 2>(P, b * f);
            }
            uint64_t y;
            asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(pack_f32(a, b)), "l"(f2), "l"(a2));
            unpack_f32(y, &v[e], &v[e + 1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = ex2(v[e]);
        uint32_t p[16];
        uint64_t sum[4];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          p[e] = pack2<__half>(v[2 * e], v[2 * e + 1]);
          const uint64_t p2 = pack_f32(v[2 * e], v[2 * e + 1]);
          const int q = (e >> 3) * 2 + (e & 1);  // two sums for each scale
          if ((e & 7) < 2) sum[q] = p2;
          else asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[q]) : "l"(p2));
        }
        tmem_st16(cols + half * 16, p);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[2 * h]) : "l"(sum[2 * h + 1]));
          float a, b;
          unpack_f32(sum[2 * h], &a, &b);
          l = fmaf(a + b, inverse_pow2(sc[h].y), l);
        }
        if (k > 0 && __any_sync(0xffffffffu, factor != 1.f)) {
          ok = __all_sync(0xffffffffu, wait(&bars->pv_done[qt], (k - 1) & 1));
          tc_fence_after();
#pragma unroll 1
          for (int c = half * 32; c < P.vhs && ok; c += 64) {  // (columns behind vhs are nobody's)
            uint32_t o[32];
            tmem_ld32_nowait(o_addr + c, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
            tmem_st32(o_addr + c, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        if (ok) arrive_warp(&bars->p_full[buf], lane);
      }
      grid_dep_launch();
      if (ok) ok = __all_sync(0xffffffffu, wait(&bars->drain, 0));
      tc_fence_after();
      // both halves' sums
      if (!ok && lane == 0) s_fail[pair] = 1;
      __syncwarp();
      pair_sync(pair);
      if (half == 1) *row_at = __float_as_int(l);
      pair_sync(pair);
      if (half == 0) {
        l += __int_as_float(*row_at);
        *row_at = __float_as_int(l);
      }
      __syncwarp();
      pair_sync(pair);
      l = __int_as_float(*const_cast<volatile int*>(row_at));
      ok = *const_cast<volatile int*>(&s_fail[pair]) == 0;
    }
    if (P.early) grid_dep_wait();
    // =================== outputs ===================
    if (run && soft && ok && !*abort && quad * 32 < rows) {
      const bool live = row < rows, bad = bars->bad != 0;
      const int tok = live ? row / P.grp : 0, h = g * P.grp + row - tok * P.grp;
      const int64_t pos_r = U.pos + tok0 + tok;
      if (bars->any_odd) {
        const int64_t back = P.window >= 0 ? P.window : pos_r;
#pragma unroll 1
        for (int i = 0; i < 512; ++i)
          if (bars->odd[i >> 5] >> (i & 31) & 1u) {
            const int64_t j = i < 256 ? U.pos + 1 + i : U.lo + (i - 256);
            if (j <= pos_r && j >= pos_r - back) l = NAN;
          }
      }
      if (bad && lane == 0 && half == 0) raise_flag(P.err_flags, PA_DEVERR_BLOCK);
      const uint32_t o_addr = lane_addr + (QT == 2 ? qt * 128 : 0);
      // (as part.splits == 1; kept from before the loop it cost the loop 1.5 %)
      if (A.splits == 1 || (int)blockIdx.x >= A.planned * A.splits) {
        float sum = l;
        if (P.head_sink && live) sum += ex2(to_f32(P, P.head_sink, h) * kLog2e - m + kShift);
        // (the sum is NaN where a NaN was seen)
        const bool none = bad || n == 0 || (m == -INFINITY && l == 0.f);
        const float inv = 1.f / sum;
        __half* dst = reinterpret_cast<__half*>(P.out) + ((U.t + tok0 + tok) * P.H + h) * P.vhs;
#pragma unroll 1
        for (int c = half * 16; c < P.vhs; c += 32) {
          uint32_t r[16], w[8];
          if (n > 0) tmem_ld16(o_addr + c, r);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = none ? 0u : pack_out(P, __uint_as_float(r[2 * e]) * inv,
                                        __uint_as_float(r[2 * e + 1]) * inv);
          if (live) {
            reinterpret_cast<uint4*>(dst + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      } else if (n > 0) {
        const int64_t at = (int64_t)blockIdx.x * (QT * kRows) + qt * kRows + row;
        float* dst = A.ws_o + at * P.vhs;
#pragma unroll 1
        for (int c = half * 16; c < P.vhs; c += 32) {
          uint32_t r[16];
          tmem_ld16(o_addr + c, r);
          if (live)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(dst + c + e) = make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
        }
        if (live && half == 0) A.ws_ml[at] = make_float2(bad ? NAN : m, l);
      }
    }
  } else if (warp < kMmaWarp) {
    fewer_registers<kConvRegs>();
    if (n > 0) {
      // =================== codes to fp16 ===================
      const int64_t lo = U.lo, hi = U.pos_hi, all_lo = U.lo_hi, all_hi = U.last0, pos = U.pos;
      constexpr int kRowsW = N / 4;  // of a tile per warp
      const int w = warp & 3, h = (warp - kConvWarp) >> 2;  // four warps for keys, four for values
      const int pitch = h ? P.vhs : P.hs;  // bytes of a row of codes
      const int lpr = h ? A.vlpr : A.klpr;   // lanes (a power of two) for its 8-byte pieces
      const int lr = lane / lpr, c = lane & (lpr - 1), rows = 32 / lpr;  // (rows at a time)
      const bool mine = c * 8 < pitch;
      const uint32_t src = smem_u32(codes) + (h ? C * N * P.hs : 0) +
                           (w * kRowsW + lr) * pitch + c * 8;
      const uint32_t dst = smem_u32(h ? v_s : k_s) + (c >> 3) * kKBox + (w * kRowsW + lr) * 128;
      // What the conversion must not see: rows of pages without a scale count as zeros;
      // values that no row of the unit sees become zeros (0 times NaN is NaN), and a NaN
      // that only some see as well: those are marked, and the rows that see them answer
      // NaN. in: a bit per segment.
      auto scrub = [&](uint32_t code, int64_t j0, int in) {
#pragma unroll 1
        for (int r = 0; r < kRowsW; r += rows) {
          const int at = w * kRowsW + r + lr;
          const int64_t j = j0 + at;
          if (!mine) continue;
          const uint2 v = lds64(code + src + r * pitch);
          if (!(in >> (at >> 4) & 1) || (h && (j < lo || j > hi))) {
            sts64(code + src + r * pitch, make_uint2(0, 0));
          } else if (h && (j < all_lo || j > all_hi) && (nan_codes(v.x) | nan_codes(v.y))) {
            const int bit = j > all_hi ? (int)(j - pos) - 1 : 256 + (int)(j - lo);
            atomicOr(&bars->odd[bit >> 5], 1u << (bit & 31));
            bars->any_odd = 1;
            sts64(code + src + r * pitch, make_uint2(0, 0));
          }
        }
      };
      // The warp's rows in fp16, eight channels a lane at a time: eight lanes write eight
      // different chunks of a row (chunk ch of row q stands at ch ^ (q & 7)). Loads go
      // ahead of the stores, which they may not pass.
      constexpr int kBatch = 4;
      uint32_t from[kBatch], to[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        from[i] = src + i * rows * pitch;
        to[i] = i * rows * 128 + (((c ^ lr ^ (i * rows)) & 7) << 4);
      }
      auto convert = [&](uint32_t code, uint32_t slot) {  // from, to
#pragma unroll 1
        for (int r0 = 0; r0 < kRowsW; r0 += kBatch * rows) {
          uint2 v[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (mine && r0 + i * rows < kRowsW) v[i] = lds64(from[i] + code + r0 * pitch);
          const uint32_t base = slot + dst + r0 * 128, turn = (r0 & 7) << 4;
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (mine && r0 + i * rows < kRowsW)
              {
                uint32_t o[4];
                codes4(v[i].x, &o[0], &o[1]);
                codes4(v[i].y, &o[2], &o[3]);
                sts128((base + to[i]) ^ turn, o[0], o[1], o[2], o[3]);
              }
        }
      };
      uint64_t* empty = h ? bars->v_empty : bars->k_empty;
      uint64_t* full = h ? bars->v_full : bars->k_full;
      // (the ring is not the keys' before the query has gone through it)
      const bool go = QT == 2 || !TWO || h || wait_idle(&bars->q_full, 0);
#pragma unroll 1
      for (int k = 0; k < n && __all_sync(0xffffffffu, go); ++k) {
        if (!__all_sync(0xffffffffu, wait_idle(&bars->sc_full[k % kAhead], (k / kAhead) & 1) &&
                                         wait_idle(&bars->c_full[2 * h + k % C], (k / C) & 1) &&
                                         (k < R || wait_idle(&empty[k % R], ((k / R) & 1) ^ 1))))
          break;
        const int2 in = s_in[k % kAhead];
        const int64_t j0 = (int64_t)(U.begin + k) * N;
        if ((in.x & in.y) != (1 << kSegs) - 1 || (h && (j0 < all_lo || j0 + N - 1 > all_hi)))
          scrub((k % C) * N * pitch, j0, h ? in.y : in.x);
        convert((k % C) * N * pitch, (k % R) * (h ? v_bytes : k_bytes));
        fence_proxy_async();
        arrive_warp(&full[k % R], lane);
        if (lane == 0) mbar_arrive(smem_u32(&bars->c_empty[2 * h + k % C]));
      }
    }
    if (P.early) grid_dep_wait();
  } else {
    fewer_registers<kMmaRegs>();
    if (n > 0 && warp == kMmaWarp) {
      // =================== products ===================
      if (diff::elect_one()) {
        constexpr uint32_t id_qk = idesc_f16(false, kRows, N, false);
        const uint32_t id_pv = idesc_f16(false, kRows, P.vhs, true);
        const int steps = P.hs >> 4;
        const uint32_t k_base = smem_u32(k_s), v_base = smem_u32(v_s), q_base = smem_u32(q_s);
        // Descriptors by their lower words (the upper ones stay as they are), with offsets
        // fixed at compile time in a slab: an MMA takes its thread 15 to 60 cycles to issue
        // so, and 75 to 100 with offsets worked out step by step.
        const uint64_t qk_proto = sdesc(q_base, 16, 1024), v_proto = sdesc(v_base, kKBox, 1024);
        const uint32_t qk_hi = (uint32_t)(qk_proto >> 32), v_hi = (uint32_t)(v_proto >> 32);
        const uint32_t q_lo = (uint32_t)qk_proto, v_lo = (uint32_t)v_proto;
        const uint32_t k_lo = (uint32_t)sdesc(k_base, 16, 1024);
        const uint32_t q_step = q_bytes >> 4, k_step = k_bytes >> 4, v_step = v_bytes >> 4;
        auto qk = [&](uint32_t slot, int buf, int tile) {
          tc_fence_after();
          uint32_t qd = q_lo + tile * q_step, kd = k_lo + slot * k_step, add = 0;
          const uint32_t d = tmem + kColS + buf * N;
          int left = steps;
#pragma unroll 1
          for (; left >= 4; left -= 4, qd += kSlab >> 4, kd += kKBox >> 4, add = 1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_ss_lo(d, qd + 2 * i, kd + 2 * i, qk_hi, id_qk, i > 0 ? 1u : add);
#pragma unroll 1
          for (; left > 0; --left, qd += 2, kd += 2, add = 1) mma_ss_lo(d, qd, kd, qk_hi, id_qk, add);
          if (TWO) {
            qd = q_lo + (QT + tile) * q_step;
            kd = k_lo + slot * k_step;
#pragma unroll 1
            for (int s = 0; s < steps; s += 4, qd += kSlab >> 4, kd += kKBox >> 4)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (s + i >= steps) break;
                if (QT == 2) mma_ss_lo(d, qd + 2 * i, kd + 2 * i, qk_hi, id_qk, 1);
                else mma_ts_lo(d, tmem + kColRest + (s + i) * 8, kd + 2 * i, qk_hi, id_qk, 1);
              }
          }
          tc_commit(smem_u32(&bars->s_full[buf]));
        };
        auto pv = [&](uint32_t slot, int buf, int tile, uint32_t add) {
          tc_fence_after();
          const uint32_t vd = v_lo + slot * v_step;
          const uint32_t p = tmem + kColS + buf * N, d = tmem + (QT == 2 ? tile * 128 : 0);
#pragma unroll
          for (int i = 0; i < kSegs; ++i)
            mma_ts_lo(d, p + i * 8, vd + i * 128, v_hi, id_pv, i > 0 ? 1u : add);
          tc_commit(smem_u32(&bars->pv_done[tile]));
        };
        // Scores run two key tiles ahead: those of tile k + 2 take the buffer of tile k's P,
        // behind its product.
        bool go = wait(&bars->q_full, 0);
#pragma unroll 1
        for (int k = 0; k < 2 && k < n && go; ++k) {
          go = wait(&bars->k_full[k], 0);
          if (!go) break;
#pragma unroll
          for (int t = 0; t < QT; ++t) qk(k, t + QT * k, t);
          tc_commit(smem_u32(&bars->k_empty[k]));
        }
        uint32_t v_slot = 0, v_turn = 0, k_slot = 2 % R, k_turn = (2 / R) & 1, p_turn = 0;
#pragma unroll 1
        for (int k = 0; k < n && go; ++k) {
          const int b0 = QT * (k & 1);
          const bool more = k + 2 < n;
          go = wait(&bars->v_full[v_slot], v_turn) &&
               (!more || wait(&bars->k_full[k_slot], k_turn));
#pragma unroll
          for (int t = 0; t < QT; ++t) {
            go = go && wait(&bars->p_full[b0 + t], p_turn);
            if (!go) break;
            pv(v_slot, b0 + t, t, k > 0 ? 1u : 0u);
            if (more) qk(k_slot, b0 + t, t);
          }
          if (!go) break;
          tc_commit(smem_u32(&bars->v_empty[v_slot]));
          if (more) tc_commit(smem_u32(&bars->k_empty[k_slot]));
          if (++v_slot == R) {
            v_slot = 0;
            v_turn ^= 1;
          }
          if (++k_slot == R) {
            k_slot = 0;
            k_turn ^= 1;
          }
          p_turn ^= k & 1;
        }
        tc_commit(smem_u32(&bars->drain));
        drain_wait(smem_u32(&bars->drain), 0, P.err_flags);
      }
      __syncwarp();
    } else if (n > 0 && warp == kCopyWarp) {
      // =================== copies of codes ===================
      const int64_t lo = U.lo, hi = U.pos_hi;
      const int32_t* table = P.block_table + (int64_t)U.b * P.max_blocks;
      const int nbox = N / A.box;
      // cache row of box `lane`: behind the last one (zeros arrive) where there is
      // nothing to see or no page
      auto look_up = [&](int k) {
        const int64_t key = (int64_t)(U.begin + k) * N + lane * A.box;
        if (k >= n || lane >= nbox || key > hi || key + A.box - 1 < lo) return (int)A.num_slots;
        const int32_t page = table[key >> P.sh];
        return page >= 0 && page < P.num_blocks ? (page << P.sh) + (int)(key & (P.bs - 1))
                                                : (int)A.num_slots;
      };
      int row = look_up(0);
      if (P.early) grid_dep_wait();
      int issued = 0;
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const int next = look_up(k + 1);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int width = h ? P.vhs : P.hs;
          const uint32_t dst = smem_u32(codes) + (h ? C * N * P.hs : 0) + (k % C) * N * width +
                               lane * A.box * width;
          const uint32_t bar = smem_u32(&bars->c_full[2 * h + k % C]);
          if (!__all_sync(0xffffffffu,
                          k < C || wait_idle(&bars->c_empty[2 * h + k % C], ((k / C) & 1) ^ 1)))
            break;
          if (lane == 0) mbar_expect_tx(bar, N * width);
          __syncwarp();
          if (lane < nbox) tma_load_3d(dst, h ? &vmap : &kmap, 0, g, row, bar);
          ++issued;
        }
        if (*abort) break;
        row = next;
      }
      if (*abort && lane == 0) {  // copies may be in flight
        for (int i = max(0, issued - 2 * C); i < issued; ++i) {
          const int k = i >> 1;
          drain_wait(smem_u32(&bars->c_full[2 * (i & 1) + k % C]), (k / C) & 1, P.err_flags);
        }
      }
      __syncwarp();
    } else if (n > 0 && warp == kScaleWarp) {
      // =================== scales ===================
      const int64_t lo = U.lo, hi = U.pos_hi;
      const int32_t* table = P.block_table + (int64_t)U.b * P.max_blocks;
      // page of segment `lane` of a tile: -1 invalid, -2 nothing to see there
      auto look_up = [&](int k) {
        const int64_t key = (int64_t)(U.begin + k) * N + lane * 16;
        if (k >= n || lane >= kSegs || key > hi || key + 15 < lo) return -2;
        const int32_t page = table[key >> P.sh];
        return page >= 0 && page < P.num_blocks ? page : -1;
      };
      auto scale_at = [&](int page) {
        return page >= 0 ? P.scales[(int64_t)page * P.kvh + g] : make_float2(0.f, 0.f);
      };
      int pg0 = look_up(0), pg1 = look_up(1);
      if (P.early) grid_dep_wait();
      float2 sc0 = scale_at(pg0);
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const int pg2 = look_up(k + 2);
        const float2 sc1 = scale_at(pg1);
        const int ke = scale_exponent(sc0.x), ve = scale_exponent(sc0.y);
        const bool kin = pg0 >= 0 && ke != kNone, vin = pg0 >= 0 && ve != kNone;
        if (pg0 == -1) bars->bad = 1;
        // Place k % kAhead held the scales of tile k - kAhead. Once this tile's place in the
        // ring is free, S of tile k - R is done; it came behind P V of tile k - R - 2, and
        // that behind the softmax of a tile and its values.
        static_assert(kAhead >= R + 2, "scales");
        if (!__all_sync(0xffffffffu,
                        k < R || wait_idle(&bars->k_empty[k % R], ((k / R) & 1) ^ 1)))
          break;
        const unsigned kb = __ballot_sync(0xffffffffu, kin || pg0 < 0);
        const unsigned vb = __ballot_sync(0xffffffffu, vin || pg0 < 0);
        constexpr unsigned kAll = (1u << kSegs) - 1;
        if (lane < kSegs)
          s_scale[k % kAhead][lane] = make_float2(kin ? sc0.x : 1.f, vin ? ve : kLeast);
        if (lane == 0) s_in[k % kAhead] = make_int2(kb & kAll, vb & kAll);
        arrive_warp(&bars->sc_full[k % kAhead], lane);
        pg0 = pg1;
        pg1 = pg2;
        sc0 = sc1;
      }
    }
    if (P.early) grid_dep_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds up the parts of a unit: four channels of a row a thread, eight rows a CTA.
template <int QT>
__global__ void __launch_bounds__(256) quant_join_kernel(const __grid_constant__ PreP A) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ Unit s_unit;
  const ReadP& P = A.R;
  const int unit = blockIdx.x / P.kvh, g = blockIdx.x - unit * P.kvh;
  if (threadIdx.x < 32) {
    const Unit u = resolve<QT>(A, unit, 0, 1, threadIdx.x);
    if (threadIdx.x == 0) s_unit = u;
  }
  __syncthreads();
  const Unit& U = s_unit;
  if (U.status != 0) return;
  const int quads = P.vhs >> 2, rows = U.ntok * P.grp;
  for (int i = blockIdx.y * 256 + threadIdx.x; i < rows * quads; i += gridDim.y * 256) {
    const int r = i / quads, c = (i - r * quads) * 4;
    const int tok = r / P.grp, h = g * P.grp + r - tok * P.grp;
    const int tile = tok / A.tpc, row = (tok - tile * A.tpc) * P.grp + r - tok * P.grp;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    bool bad = false;
    // (loads of four parts at once: one part after the other was latency and nothing else)
    for (int s0 = 0; s0 < A.splits; s0 += 4) {
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = s0 + i;
        const bool part = s < A.splits &&
                          (int64_t)U.n * s / A.splits != (int64_t)U.n * (s + 1) / A.splits;  // has tiles
        const int64_t at =
            ((int64_t)blockIdx.x * A.splits + s) * (QT * kRows) + tile * kRows + row;
        ml[i] = part ? A.ws_ml[at] : make_float2(-INFINITY, 0.f);
        v[i] = part ? *reinterpret_cast<const float4*>(A.ws_o + at * P.vhs + c)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bad |= isnan(ml[i].x);
        const float t = fmaxf(m, ml[i].x), base = t == -INFINITY ? 0.f : t;
        const float fa = ex2(m - base), fb = ex2(ml[i].x - base);
        m = t;
        l = l * fa + ml[i].y * fb;
        o = make_float4(o.x * fa + v[i].x * fb, o.y * fa + v[i].y * fb, o.z * fa + v[i].z * fb,
                        o.w * fa + v[i].w * fb);
      }
    }
    float sum = l;
    if (P.head_sink) sum += ex2(to_f32(P, P.head_sink, h) * kLog2e - m + kShift);
    const bool none = bad || (m == -INFINITY && l == 0.f);
    const float inv = 1.f / sum;
    const uint32_t w0 = none ? 0u : pack_out(P, o.x * inv, o.y * inv);
    const uint32_t w1 = none ? 0u : pack_out(P, o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(P.out) + ((U.t + tok) * P.H + h) * P.vhs + c) =
        make_uint2(w0, w1);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr size_t kMaxShared = 225 * 1024;  // (beside 2 KB of the kernel's own)
size_t shared_bytes(const Geometry& g, const PreP& A, int qt, int ring, int codes) {
  return 1024 + (size_t)qt * (qt == 2 && A.R.two ? 2 : 1) * A.slabs * kSlab +
         (size_t)ring * (A.slabs + A.vslabs) * N * 128 + (size_t)codes * N * (g.hs + g.vhs);
}

template <int QT, int R, int C, int CAP, bool TWO>
cudaError_t launch_one(const Geometry& g, const QuantArgs& a, const PreP& A,
                       const PrefillGrid& grid) {
  static std::atomic<bool> configured[64];
  auto kern = quant_prefill_kernel<QT, R, C, CAP, TWO>;
  const size_t smem = shared_bytes(g, A, QT, R, C);
  cudaError_t e = once_per_device(configured, g.device, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap kmap, vmap;
  if ((e = codes_map(&kmap, a.key_cache, g, g.hs, 0, A.box)) != cudaSuccess) return e;
  if ((e = codes_map(&vmap, a.value_cache, g, g.vhs, 0, A.box)) != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)grid.launched()), dim3(kThreads), smem, a.stream, kmap, vmap,
                 A);
  if (e != cudaSuccess || A.splits == 1) return e;
  return launch_pdl(quant_join_kernel<QT>,
                    dim3((unsigned)grid.planned, QT * kRows * (g.vhs / 4) / 256), dim3(256), 0,
                    a.stream, A);
}

template <int QT, int R, int C>
cudaError_t launch(const Geometry& g, const QuantArgs& a, const PreP& A, const PrefillGrid& grid) {
  auto of = [&](auto cap) {
    return A.R.two ? launch_one<QT, R, C, cap(), true>(g, a, A, grid)
                   : launch_one<QT, R, C, cap(), false>(g, a, A, grid);
  };
  if (A.R.cap_in <= 0.f) return of(std::integral_constant<int, 0>());
  return A.R.cap_wide ? of(std::integral_constant<int, 2>()) : of(std::integral_constant<int, 1>());
}

// One query tile where two accumulators do not fit in TMEM, or two queries beside
// the rings in shared memory.
int query_tiles(const Geometry& g, int two) {
  return g.vhs <= 128 && g.hs <= (two ? 128 : 192) ? 2 : 1;
}

}  // namespace

size_t prefill_workspace(const Geometry& g, int64_t nseq) {
  const size_t rows = (size_t)g.num_sms * query_tiles(g, 0) * kRows;  // (at most)
  return std::max(rows * g.vhs * sizeof(float) + rows * sizeof(float2), rows_workspace(g, nseq));
}

cudaError_t launch_prefill(const Geometry& g, const QuantArgs& a) {
  const int64_t nseq = a.seq_end - a.seq_begin;
  const int64_t tokens = range_tokens(a.num_tokens, a.num_seqs, nseq);
  const ReadChoice choice = choose_kernels(tokens, nseq, g.H / g.kvh);
  if (choice.rows) {
    const cudaError_t e = launch_rows(g, a, false, choice.few);
    if (e != cudaSuccess || !choice.many) return e;
  }
  PreP A{};
  A.R = read_params(g, a);
  const int qt = query_tiles(g, A.R.two);
  A.tpc = kRows / A.R.grp;
  A.slabs = (g.hs + 63) / 64;
  A.vslabs = (g.vhs + 63) / 64;
  auto lanes = [](int width) {
    int l = 2;
    while (l * 8 < width) l *= 2;
    return l;
  };
  A.klpr = lanes(g.hs);
  A.vlpr = lanes(g.vhs);
  A.box = std::min(g.bs, N);
  A.num_slots = (int64_t)g.num_blocks * g.bs;
  A.ws_o = static_cast<float*>(a.workspace);
  A.ws_ml = reinterpret_cast<float2*>(A.ws_o + (size_t)g.num_sms * qt * kRows * g.vhs);
  const PrefillGrid grid =
      prefill_grid(a.num_tokens, tokens, A.R.nseq, choice.few, g.kvh, qt * A.tpc,
                   ((int64_t)g.max_blocks * g.bs + N - 1) / N, g.num_sms);
  if (grid.planned == 0) return cudaSuccess;
  if (grid.launched() > INT32_MAX) return cudaErrorInvalidConfiguration;
  A.few = choice.few;
  if (choice.rows) A.R.early = 0;  // (behind the other kernel, not behind the write)
  A.planned = (int)grid.planned;
  A.splits = grid.splits;
  // four tiles converted ahead where they fit
  if (qt == 1) return launch<1, 2, 1>(g, a, A, grid);
  return shared_bytes(g, A, 2, 4, 2) <= kMaxShared ? launch<2, 4, 2>(g, a, A, grid)
                                                   : launch<2, 2, 2>(g, a, A, grid);
}

}  // namespace quant
}  // namespace pa
