// Attention over 8-bit caches, prefill: any number of new tokens per sequence
// (include/pa_quant.h), on the tensor cores (tcgen05, TMEM).
//
// A work unit is QT tiles of up to 128 query rows of one kv head: tpc consecutive
// tokens of one sequence x the kv head's grp heads each. Its visible keys are cut
// into tiles of N. Where a batch has too few units for the GPU, several CTAs share
// a unit's tiles and quant_join_kernel adds up their parts.
//
// Inside a CTA:
//   warps 8-11  bring a tile's codes into registers, a tile ahead, and write them as
//               fp16 (exactly) in the layout the products read: rings of two key and
//               two value tiles. Both query tiles use what is converted once. Their
//               pages are looked up two tiles ahead, the scales one.
//   warp 12     S = Q K^T (N columns of TMEM per buffer), O += P V (A = P from TMEM,
//               written over its S). QT 2: a buffer per query tile, whose softmax runs
//               while the other's products do; QT 1: two buffers in turn.
//   warps 0-7   softmax, a thread per row, warps 0-3 for query tile 0 (or the only
//               one), 4-7 for tile 1.
// TMEM columns: O, 128 for each of two query tiles or 256 for one | two buffers of N.
//
// Scales cost next to nothing: a page's rows come 16 at a time, so 16 columns of S
// have one key scale, which joins the factor of the exponent's multiply-add, and one
// value scale 2^e, whose e joins its addend (see kShift in pa_quant_read.cuh). The sum of
// the 16 probabilities is multiplied by 2^-e again.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "pa_diff_common.cuh"
#include "pa_quant_read.cuh"

namespace pa {
namespace quant {
namespace {

using namespace pa::tc;

constexpr int kConvWarp = 8, kMmaWarp = 12, kThreads = 13 * 32;
constexpr int kSlab = kRows * 128;  // bytes of a 64-channel slab of 128 query rows
constexpr int kPasses = 8;          // 16-byte pieces of a tile per converting thread, at most
constexpr int kAhead = 4;           // tiles whose scales are kept

struct Bars {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2];
  uint64_t sc_full[kAhead], pv_done, drain;
  uint32_t tmem_base;
  int bad, abort, any_odd;
  // keys with a NaN value that some rows of the unit see and others do not: position
  // pos + 1 + i (after the first token) in the first eight words, lo + i (before the
  // last one's window) behind
  uint32_t odd[16];
};
constexpr int kNumBars = 1 + 5 * 2 + 2 + kAhead + 2;

struct PreP {
  ReadP R;
  float* ws_o;   // [units * kvh * splits][QT * 128][vhs]
  float2* ws_ml; // [units * kvh * splits][QT * 128] maximum (log2 domain; NaN: an invalid page), sum
  int tpc;       // tokens of a query tile
  int splits;    // CTAs per unit
  int slabs, vslabs, klpr, vlpr;  // 64-channel slabs, lanes per row of codes
};

struct Unit {
  int64_t t, pos, lo, lo_hi, pos_hi, last0;  // see resolve()
  int b, ntok, begin, n;                     // sequence, tokens, first tile, tiles
  int status;                                // 0 run, 1 nothing, 2 told already
};

// Unit `unit` of the batch, by a warp: the sequences' units in order, the last
// ones (with the most keys) first. first..: what is filled in for all lanes.
template <int QT, int N>
__device__ Unit resolve(const PreP& A, int unit, int split, int lane) {
  const ReadP& P = A.R;
  const int per = QT * A.tpc;
  auto units_of = [&](int i, int* q0, int* q) {
    *q0 = *q = 0;
    if (i < P.nseq) {
      *q0 = P.cumseq[P.seq_begin + i];
      *q = P.cumseq[P.seq_begin + i + 1] - *q0;
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
        const int s0 = (int)((int64_t)all * split / A.splits);
        u.begin = first + s0;
        u.n = (int)((int64_t)all * (split + 1) / A.splits) - s0;
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
// Without waiting; tmem_wait_ld() and fence16() before the registers are read.
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// The query rows of a tile (token, head), normalized and rotated, as fp16 in
// swizzled slabs; mult: what takes a row's factor back, times the scale. Rows behind
// the last are zeros. By the tile's four warps.
template <typename T>
__device__ __forceinline__ void load_query(const PreP& A, const Unit& u, int g, int tile, int rows,
                                           int warp, int lane, uint8_t* q_s, float* mult) {
  const ReadP& P = A.R;
  int lpr = 2;
  while (lpr * 8 < P.hs) lpr <<= 1;
  const int d0 = (lane & (lpr - 1)) * 8, step = 32 / lpr;
#pragma unroll 4
  for (int r0 = 0; r0 < 32; r0 += step) {
    const int row = warp * 32 + r0 + lane / lpr;
    const bool live = row < rows;
    const int tok = live ? row / P.grp : 0, h = row - tok * P.grp;
    const int64_t tt = tile * A.tpc + tok;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (live && d0 < P.hs)
      unpack8<T>(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(P.query) +
                                                 ((u.t + tt) * P.H + g * P.grp + h) * P.hs + d0),
                 x);
    norm_rotate8<T>(x, live, d0, P.hs, lpr, reinterpret_cast<const T*>(P.q_norm), P.eps, P.ro, P.rd,
                    P.interleaved, reinterpret_cast<const T*>(P.cos_cache),
                    reinterpret_cast<const T*>(P.sin_cache), u.pos + tt);
    uint4 hx;
    const float back = scaled_row8(x, &hx, lpr);
    if (d0 < P.hs)
      *reinterpret_cast<uint4*>(q_s + (d0 >> 6) * kSlab + row * 128 +
                                ((((d0 >> 3) & 7) ^ (row & 7)) << 4)) = hx;
    if (d0 == 0) mult[row] = back * (P.cap_in > 0.f ? P.cap_in : P.scale_log2);
  }
}

// Four codes' NaNs as 0x80 in their bytes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

template <int QT, int N, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
quant_prefill_kernel(const __grid_constant__ PreP A) {
  constexpr int kSegs = N / 16;
  constexpr int kColS = 256;      // first column of the S buffers
  constexpr int kKBox = N * 128;  // bytes of a 64-channel slab of N keys
  const ReadP& P = A.R;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit s_unit;
  __shared__ Bars bars_s;
  __shared__ float s_mult[QT * kRows];
  __shared__ float2 s_scale[kAhead][kSegs];  // key scale, exponent of the value's
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  Bars* bars = &bars_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q_bytes = A.slabs * kSlab, k_bytes = A.slabs * kKBox, v_bytes = A.vslabs * kKBox;
  uint8_t* q_s = smem;
  uint8_t* k_s = q_s + QT * q_bytes;
  uint8_t* v_s = k_s + 2 * k_bytes;
  const int split = blockIdx.x % A.splits, rest = blockIdx.x / A.splits;
  const int g = rest % P.kvh, unit = rest / P.kvh;

  if (!P.early) grid_dep_wait();
  if (warp == 0) {
    Unit u = resolve<QT, N>(A, unit, split, lane);
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
      if (at == &bars->q_full) count = QT * 4;
      if ((at >= bars->k_full && at < bars->k_full + 2) || (at >= bars->v_full && at < bars->v_full + 2))
        count = 4;
      if (at >= bars->p_full && at < bars->p_full + 2) count = 4;
      mbar_init(smem_u32(at), count);
    }
    if (lane < 16) bars->odd[lane] = 0;
    if (lane == 0) bars->bad = bars->abort = bars->any_odd = 0;
    fence_barrier_init();
  } else if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
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
    return wait_bar(smem_u32(bar), par, abort, P.err_flags);
  };
  const int qt = QT == 2 ? warp >> 2 : 0;  // (softmax warps)
  const int quad = warp & 3, row = quad * 32 + lane;
  const int tok0 = qt * A.tpc, ntok = run ? max(0, min(A.tpc, U.ntok - tok0)) : 0;
  const int rows = ntok * P.grp;
  const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
  const bool soft = warp < (QT == 2 ? 8 : 4);
  float m = -INFINITY, l = 0.f;
  bool ok = true;

  if (run && n > 0) {
    if (soft) {
      // =================== softmax ===================
      uint8_t* q_t = q_s + qt * q_bytes;
      if (P.bf16) load_query<__nv_bfloat16>(A, U, g, qt, rows, quad, lane, q_t, s_mult + qt * kRows);
      else load_query<__half>(A, U, g, qt, rows, quad, lane, q_t, s_mult + qt * kRows);
      fence_proxy_async();
      arrive_warp(&bars->q_full, lane);
      const int64_t pos_r = U.pos + tok0 + row / P.grp;
      const int64_t last_r = P.cross ? U.pos_hi : min(pos_r, U.pos_hi);
      const int64_t lo_r = P.window >= 0 ? max((int64_t)0, pos_r - P.window) : 0;
      const float mult = s_mult[qt * kRows + row];
      const int64_t last0 = U.last0, lo_hi = U.lo_hi;
      const uint32_t o_addr = lane_addr + (QT == 2 ? qt * 128 : 0);
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const int buf = QT == 2 ? qt : k & 1;
        const uint32_t par = QT == 2 ? k & 1 : (k >> 1) & 1;
        const uint32_t cols = lane_addr + kColS + buf * N;
        const int64_t j0 = (int64_t)(U.begin + k) * N;
        const bool edge = j0 < lo_hi || j0 + N - 1 > last0;
        ok = __all_sync(0xffffffffu, wait(&bars->s_full[buf], par) &&
                                         wait(&bars->sc_full[k % kAhead], (k / kAhead) & 1));
        if (!ok) break;
        tc_fence_after();
        const float2* scale = s_scale[k % kAhead];
        const int c0 = (int)max((int64_t)0, min((int64_t)N, lo_r - j0));       // seen columns
        const int c1 = (int)max((int64_t)-1, min((int64_t)(N - 1), last_r - j0));
        uint32_t pk[N / 2];
        float lsum, top;
        // The exponentials use the running maximum as it stands; the tile's own is taken
        // beside them, and only where it passes that by more than 2^kLazy the tile is
        // computed again.
        auto tile = [&]() {
          const float nm = kShift - (m == -INFINITY ? 0.f : m);
          lsum = 0.f;
          top = -INFINITY;
          uint32_t s[2][16];
          tmem_ld16_nowait(cols, s[0]);
#pragma unroll
          for (int i = 0; i < kSegs; ++i) {
            tmem_wait_ld();
            uint32_t(&x)[16] = s[i & 1];
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              asm volatile("" : "+r"(x[e]), "+r"(x[e + 1]), "+r"(x[e + 2]), "+r"(x[e + 3]),
                           "+r"(x[e + 4]), "+r"(x[e + 5]), "+r"(x[e + 6]), "+r"(x[e + 7]));
            if (i + 1 < kSegs) tmem_ld16_nowait(cols + (i + 1) * 16, s[(i + 1) & 1]);
            const float2 sc = scale[i];
            const float f = fmaxf(sc.x * mult, 1e-37f);  // (a masked score, -inf, times 0 would be NaN)
            if (CAP) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                x[e] = __float_as_uint(capped(P, __uint_as_float(x[e]) * f));
            }
            if (edge) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (i * 16 + e < c0 || i * 16 + e > c1) x[e] = __float_as_uint(-INFINITY);
            }
            float v0 = __uint_as_float(x[0]), v1 = __uint_as_float(x[1]);
#pragma unroll
            for (int e = 2; e < 14; e += 4) {
              v0 = fmaxf(v0, fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
              v1 = fmaxf(v1, fmaxf(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])));
            }
            v0 = fmaxf(fmaxf(v0, v1), fmaxf(__uint_as_float(x[14]), __uint_as_float(x[15])));
            top = fmaxf(top, CAP ? v0 + sc.y : fmaf(v0, f, sc.y));
            const float fe = CAP ? 1.f : f, add = nm + sc.y;
            const uint64_t f2 = pack_f32(fe, fe), a2 = pack_f32(add, add);
            uint64_t sum = pack_f32(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              uint64_t y;
              asm("fma.rn.f32x2 %0, %1, %2, %3;"
                  : "=l"(y)
                  : "l"(pack_f32(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]))), "l"(f2),
                    "l"(a2));
              float a, b;
              unpack_f32(y, &a, &b);
              a = ex2(a);
              b = ex2(b);
              const uint64_t p2 = pack_f32(a, b);
              asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(p2));
              pk[i * 8 + e] = pack2<__half>(a, b);
            }
            float a, b;
            unpack_f32(sum, &a, &b);
            lsum = fmaf(a + b, ex2(-sc.y), lsum);
          }
        };
        tile();
        if (__any_sync(0xffffffffu, top > m + kLazy)) {
          float factor = 1.f;
          if (top > m + kLazy) {
            factor = ex2(m - top);  // (from -inf: 0)
            m = top;
            l *= factor;
          }
          if (k > 0 && __any_sync(0xffffffffu, factor != 1.f)) {
            if (QT == 1)  // (with two tiles S comes behind the last product)
              ok = __all_sync(0xffffffffu, wait(&bars->pv_done, (k - 1) & 1));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < P.vhs; c += 16) {
              uint32_t r[16];
              tmem_ld16(o_addr + c, r);
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * factor);
              tmem_st16(o_addr + c, r);
            }
          }
          tile();
        }
        l += lsum;
#pragma unroll
        for (int c = 0; c < N / 2; c += 16) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pk[c + e];
          tmem_st16(cols + c, w);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&bars->p_full[buf], lane);
      }
      grid_dep_launch();
      if (ok) ok = __all_sync(0xffffffffu, wait(&bars->drain, 0));
      tc_fence_after();
    } else if (warp >= kConvWarp && warp < kMmaWarp) {
      // =================== codes to fp16 ===================
      const int ct = tid - kConvWarp * 32;
      const int64_t lo = U.lo, hi = U.pos_hi, all_lo = U.lo_hi, all_hi = U.last0, pos = U.pos;
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
      struct Rows {  // of a cache: this thread's pieces of a tile
        const uint8_t* base;
        int64_t step;  // bytes of a row of all heads
        int pieces, piece, row, rows, passes;
      };
      auto rows_of = [&](const uint8_t* cache, int width, int lpr) {
        Rows r;
        r.step = (int64_t)P.kvh * width;
        r.pieces = width >> 4;
        r.piece = ct & (lpr - 1);
        r.row = ct / lpr;
        r.rows = 128 / lpr;
        r.passes = N / r.rows;
        r.base = cache + (int64_t)g * width + r.piece * 16;
        return r;
      };
      const Rows KR = rows_of(P.key_cache, P.hs, A.klpr), VR = rows_of(P.value_cache, P.vhs, A.vlpr);
      // (a warp's rows of a pass lie in one segment)
      auto load = [&](const Rows& R, int k, int pages, uint4 (&c)[kPasses]) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          c[i] = make_uint4(0, 0, 0, 0);
          if (i < R.passes) {
            const int r = i * R.rows + R.row;
            const int page = __shfl_sync(0xffffffffu, pages, r >> 4);
            const int64_t key = (int64_t)(U.begin + k) * N + r;
            if (page >= 0 && R.piece < R.pieces)
              c[i] = *reinterpret_cast<const uint4*>(
                  R.base + (((int64_t)page << P.sh) + (key & (P.bs - 1))) * R.step);
          }
        }
      };
      auto store = [&](const Rows& R, uint8_t* dst, const uint4 (&c)[kPasses], int in) {
        const int flip = (R.piece >> 2) & 1;  // (eight lanes write eight different chunks)
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          if (i < R.passes) {
            const int r = i * R.rows + R.row;
            const bool there = __shfl_sync(0xffffffffu, in, r >> 4) != 0;
            if (R.piece < R.pieces) {
              uint4 w = c[i];
              if (!there) w = make_uint4(0, 0, 0, 0);
              const uint4 a = make_uint4(codes2(w.x), codes2(w.x >> 16), codes2(w.y), codes2(w.y >> 16));
              const uint4 b = make_uint4(codes2(w.z), codes2(w.z >> 16), codes2(w.w), codes2(w.w >> 16));
              uint8_t* at = dst + (R.piece >> 2) * kKBox + r * 128;
              const int c0 = (R.piece & 3) * 2, x = r & 7;
              *reinterpret_cast<uint4*>(at + (((c0 + flip) ^ x) << 4)) = flip ? b : a;
              *reinterpret_cast<uint4*>(at + (((c0 + 1 - flip) ^ x) << 4)) = flip ? a : b;
            }
          }
        }
      };
      // Values that no row sees become zeros (0 times NaN is NaN), and a NaN that only
      // some see as well: those are marked, and the rows that see them answer NaN.
      auto mask = [&](int k, uint4 (&c)[kPasses]) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          if (i >= VR.passes) continue;
          const int64_t j = (int64_t)(U.begin + k) * N + i * VR.rows + VR.row;
          if (j < lo || j > hi) {
            c[i] = make_uint4(0, 0, 0, 0);
          } else if (j < all_lo || j > all_hi) {
            if (nan_codes(c[i].x) | nan_codes(c[i].y) | nan_codes(c[i].z) | nan_codes(c[i].w)) {
              c[i] = make_uint4(0, 0, 0, 0);
              const int bit = j > all_hi ? (int)(j - pos) - 1 : 256 + (int)(j - lo);
              atomicOr(&bars->odd[bit >> 5], 1u << (bit & 31));
              bars->any_odd = 1;
            }
          }
        }
      };
      int pg0 = look_up(0), pg1 = look_up(1);
      if (P.early) grid_dep_wait();
      float2 sc0 = scale_at(pg0);
      uint4 kc[kPasses], vc[kPasses];
      load(KR, 0, pg0, kc);
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        load(VR, k, pg0, vc);
        const int pg2 = look_up(k + 2);
        const float2 sc1 = scale_at(pg1);
        const int ke = scale_exponent(sc0.x), ve = scale_exponent(sc0.y);
        const int kin = pg0 >= 0 && ke != kNone, vin = pg0 >= 0 && ve != kNone;
        if (pg0 == -1) bars->bad = 1;
        const uint32_t par = ((k >> 1) & 1) ^ 1;
        if (!__all_sync(0xffffffffu, k < 2 || wait(&bars->k_empty[k & 1], par))) break;
        if (warp == kConvWarp) {  // (the tile four before is done with: see kAhead)
          if (lane < kSegs) s_scale[k % kAhead][lane] = make_float2(kin ? sc0.x : 1.f, vin ? ve : kLeast);
          arrive_warp(&bars->sc_full[k % kAhead], lane);
        }
        store(KR, k_s + (k & 1) * k_bytes, kc, kin);
        fence_proxy_async();
        arrive_warp(&bars->k_full[k & 1], lane);
        if (k + 1 < n) load(KR, k + 1, pg1, kc);
        const int64_t j0 = (int64_t)(U.begin + k) * N;
        if (j0 < all_lo || j0 + N - 1 > all_hi) mask(k, vc);
        if (!__all_sync(0xffffffffu, k < 2 || wait(&bars->v_empty[k & 1], par))) break;
        store(VR, v_s + (k & 1) * v_bytes, vc, vin);
        fence_proxy_async();
        arrive_warp(&bars->v_full[k & 1], lane);
        pg0 = pg1;
        pg1 = pg2;
        sc0 = sc1;
      }
    } else if (warp == kMmaWarp) {
      // =================== products ===================
      if (diff::elect_one()) {
        constexpr uint32_t id_qk = idesc_f16(false, kRows, N, false);
        const uint32_t id_pv = idesc_f16(false, kRows, P.vhs, true);
        const int steps = P.hs >> 4;
        const uint32_t k_base = smem_u32(k_s), v_base = smem_u32(v_s), q_base = smem_u32(q_s);
        auto qk = [&](int k, int buf, int tile) {
          tc_fence_after();
          const uint64_t kd = sdesc(k_base + (k & 1) * k_bytes, 16, 1024);
          const uint64_t qd = sdesc(q_base + tile * q_bytes, 16, 1024);
#pragma unroll 4
          for (int i = 0; i < steps; ++i) {
            const uint32_t in = (uint32_t)(i & 3) * 2;
            mma_ss(tmem + kColS + buf * N, qd + (uint32_t)(i >> 2) * (kSlab >> 4) + in,
                   kd + (uint32_t)(i >> 2) * (kKBox >> 4) + in, id_qk, i > 0 ? 1u : 0u);
          }
          tc_commit(smem_u32(&bars->s_full[buf]));
        };
        auto pv = [&](int k, int buf, int tile) {
          tc_fence_after();
          const uint64_t vd = sdesc(v_base + (k & 1) * v_bytes, kKBox, 1024);
#pragma unroll
          for (int i = 0; i < kSegs; ++i)
            mma_ts(tmem + (QT == 2 ? tile * 128 : 0), tmem + kColS + buf * N + i * 8,
                   vd + (uint64_t)(i * 128), id_pv, (k > 0 || i > 0) ? 1u : 0u);
        };
        auto full = [&](uint64_t* bar, int k) { return wait(&bar[k & 1], (k >> 1) & 1); };
        bool go = wait(&bars->q_full, 0);
        if (QT == 2) {
          go = go && full(bars->k_full, 0);
          if (go) {
            qk(0, 0, 0);
            qk(0, 1, 1);
            tc_commit(smem_u32(&bars->k_empty[0]));
          }
          for (int k = 0; k < n && go; ++k) {
            for (int t = 0; t < 2 && go; ++t) {
              go = wait(&bars->p_full[t], k & 1) && (t == 1 || full(bars->v_full, k));
              if (!go) break;
              pv(k, t, t);
              if (k + 1 < n) {
                go = t == 1 || full(bars->k_full, k + 1);
                if (go) qk(k + 1, t, t);
              }
            }
            if (go) {
              tc_commit(smem_u32(&bars->v_empty[k & 1]));
              tc_commit(smem_u32(&bars->k_empty[(k + 1) & 1]));
            }
          }
        } else {
          for (int k = 0; k < 2 && k < n && go; ++k) {
            go = full(bars->k_full, k);
            if (go) qk(k, k, 0);
            if (go) tc_commit(smem_u32(&bars->k_empty[k]));
          }
          for (int k = 0; k < n && go; ++k) {
            go = full(bars->p_full, k) && full(bars->v_full, k);
            if (!go) break;
            pv(k, k & 1, 0);
            tc_commit(smem_u32(&bars->pv_done));
            tc_commit(smem_u32(&bars->v_empty[k & 1]));
            if (k + 2 < n) {
              go = full(bars->k_full, k + 2);
              if (go) qk(k + 2, k & 1, 0);
              if (go) tc_commit(smem_u32(&bars->k_empty[k & 1]));
            }
          }
        }
        tc_commit(smem_u32(&bars->drain));
        drain_wait(smem_u32(&bars->drain), 0, P.err_flags);
      }
      __syncwarp();
    }
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
    if (bad && lane == 0) raise_flag(P.err_flags, PA_DEVERR_BLOCK);
    const uint32_t o_addr = lane_addr + (QT == 2 ? qt * 128 : 0);
    if (A.splits == 1) {
      float sum = l;
      if (P.head_sink && live) sum += ex2(to_f32(P, P.head_sink, h) * kLog2e - m + kShift);
      // (the sum is NaN where a NaN was seen)
      const bool none = bad || n == 0 || (m == -INFINITY && l == 0.f);
      const float inv = 1.f / sum;
      __half* dst = reinterpret_cast<__half*>(P.out) + ((U.t + tok0 + tok) * P.H + h) * P.vhs;
#pragma unroll 1
      for (int c = 0; c < P.vhs; c += 16) {
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
      for (int c = 0; c < P.vhs; c += 16) {
        uint32_t r[16];
        tmem_ld16(o_addr + c, r);
        if (live)
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4*>(dst + c + e) = make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
      }
      if (live) A.ws_ml[at] = make_float2(bad ? NAN : m, l);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds up the parts of a unit: four channels of a row a thread, eight rows a CTA.
template <int QT, int N>
__global__ void __launch_bounds__(256) quant_join_kernel(const __grid_constant__ PreP A) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ Unit s_unit;
  const ReadP& P = A.R;
  const int unit = blockIdx.x / P.kvh, g = blockIdx.x - unit * P.kvh;
  if (threadIdx.x < 32) {
    PreP whole = A;
    whole.splits = 1;
    const Unit u = resolve<QT, N>(whole, unit, 0, threadIdx.x);
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
    for (int s = 0; s < A.splits; ++s) {
      if ((int64_t)U.n * s / A.splits == (int64_t)U.n * (s + 1) / A.splits) continue;  // no tiles
      const int64_t at =
          ((int64_t)blockIdx.x * A.splits + s) * (QT * kRows) + tile * kRows + row;
      const float2 ml = A.ws_ml[at];
      const float4 v = *reinterpret_cast<const float4*>(A.ws_o + at * P.vhs + c);
      bad |= isnan(ml.x);
      const float t = fmaxf(m, ml.x), base = t == -INFINITY ? 0.f : t;
      const float fa = ex2(m - base), fb = ex2(ml.x - base);
      m = t;
      l = l * fa + ml.y * fb;
      o = make_float4(o.x * fa + v.x * fb, o.y * fa + v.y * fb, o.z * fa + v.z * fb,
                      o.w * fa + v.w * fb);
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
template <int QT, int N, bool CAP>
cudaError_t launch(const Geometry& g, const QuantArgs& a, const PreP& A, int64_t ctas) {
  static std::atomic<bool> configured[64];
  auto kern = quant_prefill_kernel<QT, N, CAP>;
  const size_t smem = 1024 + (size_t)QT * A.slabs * kSlab + 2 * (size_t)(A.slabs + A.vslabs) * N * 128;
  cudaError_t e = once_per_device(configured, g.device, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024);
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)(ctas * A.splits)), dim3(kThreads), smem, a.stream, A);
  if (e != cudaSuccess || A.splits == 1) return e;
  return launch_pdl(quant_join_kernel<QT, N>, dim3((unsigned)ctas, 8), dim3(256), 0, a.stream, A);
}

// One query tile where two accumulators do not fit in TMEM, or two queries beside
// the rings in shared memory.
int query_tiles(const Geometry& g) { return g.vhs <= 128 && g.hs <= 192 ? 2 : 1; }

}  // namespace

size_t prefill_workspace(const Geometry& g, int64_t, int64_t) {
  const size_t rows = (size_t)g.num_sms * query_tiles(g) * kRows;
  return rows * g.vhs * sizeof(float) + rows * sizeof(float2);
}

cudaError_t launch_prefill(const Geometry& g, const QuantArgs& a) {
  PreP A{};
  A.R = read_params(g, a);
  const int qt = query_tiles(g), n = g.hs > 128 || g.vhs > 128 ? 64 : 128;
  A.tpc = kRows / A.R.grp;
  A.slabs = (g.hs + 63) / 64;
  A.vslabs = (g.vhs + 63) / 64;
  auto lanes = [](int width) {
    int l = 2;
    while (l * 16 < width) l *= 2;
    return l;
  };
  A.klpr = lanes(g.hs);
  A.vlpr = lanes(g.vhs);
  A.ws_o = static_cast<float*>(a.workspace);
  A.ws_ml = reinterpret_cast<float2*>(A.ws_o + (size_t)g.num_sms * qt * kRows * g.vhs);
  // (a sequence with tokens has at most one unit that is not full)
  const int64_t units = a.num_tokens / (qt * A.tpc) + std::min((int64_t)A.R.nseq, a.num_tokens);
  const int64_t ctas = units * g.kvh;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  // parts of four tiles at least, as long as there are SMs
  const int64_t tiles = ((int64_t)g.max_blocks * g.bs + n - 1) / n;
  A.splits = (int)std::max<int64_t>(1, std::min<int64_t>(g.num_sms / ctas, tiles / 4));
  const bool cap = g.softcap > 0.f;
  if (qt == 2 && n == 128)
    return cap ? launch<2, 128, true>(g, a, A, ctas) : launch<2, 128, false>(g, a, A, ctas);
  if (qt == 2) return cap ? launch<2, 64, true>(g, a, A, ctas) : launch<2, 64, false>(g, a, A, ctas);
  return cap ? launch<1, 64, true>(g, a, A, ctas) : launch<1, 64, false>(g, a, A, ctas);
}

}  // namespace quant
}  // namespace pa
