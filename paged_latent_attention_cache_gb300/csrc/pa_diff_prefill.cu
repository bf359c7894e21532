// Differential attention, prefill: any number of new tokens per sequence
// (include/pa_diff.h), on the tensor cores (tcgen05, TMEM, TMA).
//
// A work unit is up to 128 query rows of one kv head: tpc consecutive tokens
// of one sequence x the kv head's grp heads. Its two softmax maps run on the
// two CTAs of a cluster, CTA r with map r: the accumulator of one map is 128 x
// vhs f32, half of a TMEM at vhs 256, so both maps of a unit do not fit one SM
// together with their scores, and each map streams keys of its own anyway.
// The CTAs run apart until the end, where they exchange halves of their
// normalized outputs through distributed shared memory: CTA r takes the
// difference of value channels [r vg / 2, (r + 1) vg / 2), the sums of squares
// of the norm are exchanged the same way, and each writes its channels once.
// Nothing but the output leaves the chip.
//
// Inside a CTA, per tile of 128 keys:
//   warps 8-10 TMA through the block table: a ring of key tiles, and one of value
//             half tiles (64 keys), which are freed at other times: a key tile
//             by QK^T, a value half by its half of PV. One ring of whole stages
//             held keys until PV and left two stages at 128 / 256. All slabs of
//             a tile come by one 4-D box where the width is a multiple of 64: a
//             copy costs its thread some 190 cycles, and one warp with a copy
//             per slab was the slowest part of the kernel (2500 cycles a tile).
//   warp 11   QK^T (S: 128 x 128 f32 in TMEM), PV (A = P from TMEM, O: 128 x vg)
//   warps 0-7 softmax, two threads per row, 64 columns each. S is read into
//             registers once, P is written over it. TMEM columns: O vg <= 256 |
//             two buffers of 128 for S and P (three where vg <= 128): QK^T of the
//             next tile runs while the softmax works on this one.
//
// Precision: out = softmax_0 V - lambda softmax_1 V cancels, so errors of the
// two maps weigh more than in a plain softmax. The rotated query and the
// probabilities enter the products as two 16-bit parts each (value and
// remainder), as in decode (see Prob): P's parts side by side in the 64 columns that a
// thread's scores had, the query's remainders in slabs of their own. The result
// is then as exact as its own rounding. With both rounded to the dtype its error
// was twice that (bf16 3.4e-3 instead of 1.7e-3 relative), and either of the two
// roundings alone still makes it one and a half times; without the second parts
// 128 / 256 took 732 us instead of 1140, 64 / 128 586 instead of 765.
//
// Bound: per tile and map the MMAs take 2 * 128 * 128 * (hs + vhs) / 4096 cycles
// (3100 at 128 / 256, 1536 at 64 / 128) with both parts, and the exponentials
// 16384 / 32 = 512 beside 1000 for maxima, sums, parts and packing. Measured, 2 x
// 4096 new tokens over 0 and 4096 cached ones, 16 heads over 4 kv heads, bf16:
// 128 / 256 1140 us, 1.8 PFLOP/s of products (0.93 of a library product's rate,
// 0.47 counting the formula's own): a tile takes 3150 cycles, a unit some 24000
// outside its tiles (lookup and query, the exchange, the norm). 64 / 128 765 us,
// 2240 cycles a tile, bound by the softmax warps' instructions; two groups of
// them on alternate tiles took 731, but 36 instead of 34 us for short prompts (2 x
// 250 tokens, 8 heads), which are a chain of latencies, and were not kept.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "pa_diff_common.cuh"
#include "pa_diff_internal.h"
#include "pa_tc_cluster.cuh"

namespace pa {
namespace diff {
namespace {

using namespace pa::tc;

constexpr int kN = 128;             // keys of a tile
constexpr int kSoftWarps = 8;
constexpr int kSoft = kSoftWarps * 32;
constexpr int kProdWarp = 8, kMmaWarp = 11;  // warps 8, 9, 10: keys, value halves 0 and 1
constexpr int kPreThreads = 384;
constexpr int kBox = kN * 128;      // bytes of a 64-channel slab of 128 rows
constexpr int kMaxK = 4, kMaxV = 16;  // slots of the rings
constexpr int kVKeys = 64;            // keys of a value slot
constexpr int kVBox = kVKeys * 128;   // bytes of its 64-channel slab
constexpr size_t kSmemMax = 225 * 1024;

struct PreBars {
  uint64_t k_full[kMaxK], k_empty[kMaxK], v_full[kMaxV], v_empty[kMaxV];
  uint64_t s_full[3], p_full[3], pv_done[2];
  uint64_t q_full, drain, x_full[4];  // (x_full: a quadrant of 32 rows each)
  uint64_t v_land[2][2];  // [half][tile parity] values whose unseen rows are zeroed before v_full
  uint64_t q_tma;  // (set up by the warp that uses it first)
  uint32_t tmem_base;
  int bad, abort;
  // keys with a value that is not finite: position pos + i (after the unit's
  // first token) in the first four words, lo + i (before its last window) behind
  uint32_t odd[8];
  int any_odd;
};

constexpr int kNumBars = 2 * kMaxK + 2 * kMaxV + 8 + 6 + 4;  // all but q_tma
static_assert(offsetof(PreBars, q_tma) == kNumBars * 8, "barriers in one row");

// Division by a number that the host knows, of dividends below 2^31, by a
// product: n d' >> s with d' = ceil(2^s / d), s = 31 + ceil(log2 d) (Granlund and
// Montgomery, 1994), for the short code that a CTA's start wants (unit_warp).
struct Divisor {
  uint32_t mul, shift;
};
__device__ __forceinline__ int divide(int n, const Divisor& d) {
  return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift);
}

struct PreArgs {
  Params P;           // what the shared helpers read
  Divisor by_kvh, by_tpc, by_grp;
  int hs;
  int lo0, lo1;       // k steps of QK^T that the rotation reaches: those take q's remainder too
  int bufs;           // buffers of S and P
  int nk, nv, v_bytes, v_rows;  // slots of the rings; bytes of a value slot, rows of its boxes
  bool k_whole, v_whole;        // widths that are multiples of 64: see cache_map
  const float* lambda_vectors;
  const void* norm_weight;
  float lambda_init, norm_eps;
};

// Not 0 if a 16-byte piece of values holds an infinity or NaN: x - x is +0 else.
template <typename T>
__device__ __forceinline__ uint32_t minus_itself(uint32_t v) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("sub.bf16x2 %0, %0, %0;" : "+r"(v));
  else
    asm("sub.f16x2 %0, %0, %0;" : "+r"(v));
  return v;
}
template <typename T>
__device__ __forceinline__ uint32_t not_finite(const uint4& v) {
  return minus_itself<T>(v.x) | minus_itself<T>(v.y) | minus_itself<T>(v.z) |
         minus_itself<T>(v.w);
}
// One arrival for the whole warp (256 threads on one barrier queue up there).
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
// `bytes` of this CTA's shared memory into the peer's, counted on its barrier.
__device__ __forceinline__ void bulk_copy_peer(uint32_t dst, uint32_t src, uint32_t bytes,
                                               uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(dst), "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_peer(uint32_t raddr, float a) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(raddr), "f"(a) : "memory");
}

template <typename T>
__device__ __forceinline__ void unpack_half2(uint32_t v, float* a, float* b) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    *a = __uint_as_float(v << 16);
    *b = __uint_as_float(v & 0xffff0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
    *a = f.x;
    *b = f.y;
  }
}

// Eight values as 16-bit parts: rounded, and the rounded remainder.
template <typename T>
__device__ __forceinline__ void split8(const float (&x)[8], uint4* hi, uint4* lo) {
  float h[8], d[8];
  *hi = pack8<T>(x);
  unpack8<T>(*hi, h);
#pragma unroll
  for (int e = 0; e < 8; ++e) d[e] = x[e] - h[e];
  *lo = pack8<T>(d);
}

// The rotation of one query row in place in its swizzled slabs (16-byte chunk
// c of row r at c ^ (r & 7)), by two threads (`part` 0 and 1), in f32; what
// rounding takes away goes to the same place of the slabs `q_lo`. The table entries of a half-split row are loaded (`load`) before the
// query has landed; 8-channel groups g = part, part + 2, .. of the first half.
template <typename T>
struct RowAngles {
  uint4 c[4], s[4];
  __device__ __forceinline__ void load(const Params& P, int part, int64_t pos) {
    const int half = P.rd >> 1;
    const T* crow = reinterpret_cast<const T*>(P.cos_cache) + pos * half;
    const T* srow = reinterpret_cast<const T*>(P.sin_cache) + pos * half;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = (2 * i + part) * 8;
      if (d < half) {
        c[i] = *reinterpret_cast<const uint4*>(crow + d);
        s[i] = *reinterpret_cast<const uint4*>(srow + d);
      }
    }
  }
};
__device__ __forceinline__ uint4* q_chunk(uint8_t* q_s, int row, int d0) {
  return reinterpret_cast<uint4*>(q_s + (d0 >> 6) * kBox + row * 128 +
                                  ((((d0 >> 3) & 7) ^ (row & 7)) << 4));
}
template <typename T>
__device__ __forceinline__ void rotate_row(uint8_t* q_s, uint8_t* q_lo, int row, int part,
                                           const Params& P,
                                           int64_t pos, RowAngles<T>& A) {
  const int half = P.rd >> 1;
  if (part == 0) {  // the other half of a k step that the rotation ends in
    if (P.ro & 8) *q_chunk(q_lo, row, P.ro - 8) = make_uint4(0, 0, 0, 0);
    if ((P.ro + P.rd) & 8) *q_chunk(q_lo, row, P.ro + P.rd) = make_uint4(0, 0, 0, 0);
  }
  if (P.interleaved) {
    const T* crow = reinterpret_cast<const T*>(P.cos_cache) + pos * half;
    const T* srow = reinterpret_cast<const T*>(P.sin_cache) + pos * half;
#pragma unroll 1
    for (int d0 = P.ro + part * 8; d0 < P.ro + P.rd; d0 += 16) {
      float a[8], none[8];
      unpack8<T>(*q_chunk(q_s, row, d0), a);
      rope8<T>(a, none, d0, P.ro, P.rd, 1, crow, srow);
      split8<T>(a, q_chunk(q_s, row, d0), q_chunk(q_lo, row, d0));
    }
    return;
  }
#pragma unroll 1
  for (int d = part * 8; d < half; d += 16) {
    float x[8], y[8], c[8], sn[8], u[8], v[8];
    unpack8<T>(*q_chunk(q_s, row, P.ro + d), x);
    unpack8<T>(*q_chunk(q_s, row, P.ro + half + d), y);
    unpack8<T>(A.c[0], c);
    unpack8<T>(A.s[0], sn);
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // as rope8
      u[e] = fmaf(x[e], c[e], -y[e] * sn[e]);
      v[e] = fmaf(y[e], c[e], x[e] * sn[e]);
    }
    split8<T>(u, q_chunk(q_s, row, P.ro + d), q_chunk(q_lo, row, P.ro + d));
    split8<T>(v, q_chunk(q_s, row, P.ro + half + d), q_chunk(q_lo, row, P.ro + half + d));
#pragma unroll
    for (int i = 0; i < 3; ++i) {  // (a loop, with the next entries in place)
      A.c[i] = A.c[i + 1];
      A.s[i] = A.s[i + 1];
    }
  }
}

// Largest of 32 scores (three-operand maxima).
__device__ __forceinline__ float max32(const uint32_t (&x)[32]) {
  float v[2] = {__uint_as_float(x[0]), __uint_as_float(x[1])};
#pragma unroll
  for (int e = 2; e < 30; e += 4) {
    v[0] = fmaxf(v[0], fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
    v[1] = fmaxf(v[1], fmaxf(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])));
  }
  return fmaxf(fmaxf(v[0], v[1]), fmaxf(__uint_as_float(x[30]), __uint_as_float(x[31])));
}

// 2^(v sl + nm) of 32 raw scores of a row (CAP: of their softcapped ones) as
// 16-bit parts, rounded and remainder; returns the sum of the unrounded values.
// In passes over the registers, so that the 32 exponentials issue back to back,
// multiply-adds, sums and remainders on pairs.
template <typename T, bool CAP>
__device__ __forceinline__ float exp_row(const uint32_t (&r)[32], uint32_t (&hi)[16], uint32_t (&lo)[16],
                                         const Params& P, float nm) {
  auto score = [&](int e) {
    const float v = __uint_as_float(r[e]);
    return !CAP || v == -INFINITY ? v : P.cap_out * tanh_ex2(v * P.cap_in);
  };
  uint64_t x[16];
  const float sl = CAP ? 1.f : P.scale_log2;
  const uint64_t sl2 = pack_f32(sl, sl), nm2 = pack_f32(nm, nm);
#pragma unroll
  for (int e = 0; e < 16; ++e)
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(x[e])
        : "l"(pack_f32(score(2 * e), score(2 * e + 1))), "l"(sl2), "l"(nm2));
  float p[32];
#pragma unroll
  for (int e = 0; e < 16; ++e) unpack_f32(x[e], &p[2 * e], &p[2 * e + 1]);
#pragma unroll
  for (int e = 0; e < 32; ++e) p[e] = ex2(p[e]);
  const uint64_t minus = pack_f32(-1.f, -1.f);
  uint64_t sum[2] = {pack_f32(0.f, 0.f), pack_f32(0.f, 0.f)};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint64_t v = pack_f32(p[2 * e], p[2 * e + 1]);
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[e & 1]) : "l"(v));
    hi[e] = pack2<T>(p[2 * e], p[2 * e + 1]);
    float h0, h1, d0, d1;
    unpack_half2<T>(hi[e], &h0, &h1);
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pack_f32(h0, h1)), "l"(minus), "l"(v));
    unpack_f32(d, &d0, &d1);
    lo[e] = pack2<T>(d0, d1);
  }
  float a, b, c, d;
  unpack_f32(sum[0], &a, &b);
  unpack_f32(sum[1], &c, &d);
  return (a + b) + (c + d);
}

// prefill_group_warp for up to 32 sequences: one round of loads, the rest in
// registers, instead of a chain of three. Short code: it is fetched cold in
// every CTA (with divisions and the scan unrolled it took 2700 cycles).
__device__ __forceinline__ Work unit_warp(const PreArgs& A, int unit, int lane) {
  const Params& P = A.P;
  const int nseq = P.pf_end - P.pf_begin;
  if (nseq > 32) return prefill_group_warp(P, unit, P.tpc);
  int q0 = 0, q1 = 0, past = 0;
  if (lane < nseq) {
    q0 = P.cumseq[P.pf_begin + lane];
    q1 = P.cumseq[P.pf_begin + lane + 1];
    past = P.past[P.pf_begin + lane];
  }
  const int cnt = q1 > q0 ? divide(q1 - q0 - 1, A.by_tpc) + 1 : 0;
  int incl = cnt;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  Work w;
  w.status = 1;
  w.splits = 1;
  w.ntok = 0;
  w.decode = 0;
  const int u = __shfl_sync(0xffffffffu, incl, 31) - 1 - unit;  // the last tokens first
  const unsigned who = __ballot_sync(0xffffffffu, u >= 0 && u >= incl - cnt && u < incl);
  if (who) {
    const int src = __ffs(who) - 1;
    const int g = __shfl_sync(0xffffffffu, u - (incl - cnt), src);
    const int first = __shfl_sync(0xffffffffu, q0, src);
    const int len = __shfl_sync(0xffffffffu, q1 - q0, src);
    w.past = __shfl_sync(0xffffffffu, past, src);
    w.b = P.pf_begin + src;
    w.t = first + (int64_t)g * P.tpc;
    w.ntok = min(P.tpc, len - g * P.tpc);
    w.pos = w.past + (int64_t)g * P.tpc;
    w.status = 0;
  }
  return w;
}

// Zeroes the rows of a value slot (keys j0 .. j0 + 63) that no row of the unit
// sees, by one warp, 8 lanes a row, four rows at a time. A key that some rows see and others do not
// has probability 0 in the latter, and 0 times infinity or NaN is NaN: such
// values are zeroed as well, and the key is marked, so that the rows that see it
// answer NaN in the end.
template <typename T>
__device__ __forceinline__ void zero_values(uint8_t* slot, PreBars* bars, int vslabs, int64_t j0,
                                            int64_t lo, int64_t lo_hi, int64_t pos, int64_t pos_hi,
                                            int lane) {
  // rows from r_lo to r_hi that some row does not see, in them [s_lo, s_hi) that
  // any does
  const int r_lo = j0 < lo_hi ? 0 : (int)max((int64_t)0, pos + 1 - j0);
  const int r_hi = j0 + kVKeys - 1 > pos ? kVKeys : (int)min((int64_t)kVKeys, lo_hi - j0);
  const int s_lo = (int)max((int64_t)r_lo, min((int64_t)kVKeys, lo - j0));
  const int s_hi = (int)max((int64_t)0, min((int64_t)r_hi, pos_hi + 1 - j0));
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint8_t* mine = slot + (lane >> 3) * 128 + (lane & 7) * 16;
  uint32_t odd = 0;
#pragma unroll 1
  for (int c = 0; c < vslabs; ++c) {  // 16 rows at a time, without branches
#pragma unroll 1
    for (int r = r_lo & ~3; r < r_hi; r += 16) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int q = r + 4 * k + (lane >> 3);
        uint4* at = reinterpret_cast<uint4*>(mine + c * kVBox + (r + 4 * k) * 128);
        const bool seen = q >= s_lo && q < s_hi;
        v[k] = zero;
        if (seen) v[k] = *at;
        if (!seen && q >= r_lo && q < r_hi) *at = zero;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) odd |= not_finite<T>(v[k]);
    }
  }
  if (!__any_sync(0xffffffffu, odd != 0)) return;
#pragma unroll 1
  for (int r = s_lo + (lane >> 3); r < s_hi; r += 4) {
    const int64_t j = j0 + r;
    if (j <= pos && j >= lo_hi) continue;  // all rows see it
#pragma unroll 1
    for (int c = 0; c < vslabs; ++c) {
      uint4* at = reinterpret_cast<uint4*>(slot + c * kVBox + r * 128 + (lane & 7) * 16);
      if (not_finite<T>(*at)) {
        *at = zero;
        const int bit = j > pos ? (int)(j - pos) : 128 + (int)(j - lo);
        atomicOr(&bars->odd[bit >> 5], 1u << (bit & 31));
        bars->any_odd = 1;
      }
    }
  }
}

template <typename T, bool CAP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPreThreads, 1)
diff_prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ CUtensorMap qmap, const __grid_constant__ PreArgs A) {
  const Params& P = A.P;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Work work;
  __shared__ PreBars bars_s;
  __shared__ float s_max[2][kRows];
  __shared__ int s_again[2][2][4];  // [tile parity][half][quadrant]
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* q_s = smem;
  uint8_t* q_lo = smem + P.q_bytes;        // the query's remainders (with a rotation)
  uint8_t* k_s = q_lo + (P.rd > 0 ? P.q_bytes : 0);  // key slots: slabs of kN rows
  uint8_t* v_s = k_s + A.nk * P.k_bytes;   // value slots: slabs of kVKeys rows
  // in the query's place, once the last QK^T is done: the halves' sums,
  // [CTA * 2 + half] sums of squares (the peer's too), and the norm's weights
  float (*s_sum)[kRows] = reinterpret_cast<float (*)[kRows]>(q_s);
  float (*s_ss)[kRows] = s_sum + 2;
  uint4* s_norm = reinterpret_cast<uint4*>(s_ss + 4);  // the norm's weights
  PreBars* bars = &bars_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slabs = P.slabs, vslabs = P.vslabs, vg = P.vg;
  const int kvh = P.kvh, grp = P.grp, vhs = P.vhs;
  const int map = (int)cluster_rank();
  const int pair = blockIdx.x >> 1;
  const int unit = divide(pair, A.by_kvh), gk = pair - unit * kvh;

  if (warp == 0) {
    if (lane == 0) {
      mbar_init(smem_u32(&bars->q_tma), 1);
      fence_barrier_init();
    }
    if (!P.early) grid_dep_wait();
    Work w = unit_warp(A, unit, lane);
    if (w.status == 0) {
      const int64_t pos_hi = w.pos + w.ntok - 1;
      const bool bad_ctx = w.past < 0 || pos_hi >= (int64_t)P.max_blocks * P.bs || w.t < 0 ||
                           w.t + w.ntok > P.num_tokens;
      const bool bad_pos = P.rd > 0 && pos_hi >= P.cos_rows;
      const int64_t lo_key = P.window >= 0 ? max((int64_t)0, w.pos - P.window) : 0;
      w.t_begin = lo_key / kN;
      w.t_end = pos_hi / kN + 1;
      if (bad_ctx || bad_pos) {
        if (lane == 0 && gk == 0 && map == 0)
          raise_flag(P.err_flags, bad_ctx ? PA_DEVERR_CONTEXT : PA_DEVERR_POSITION);
        const int nt = w.t < 0 ? 0 : (int)max((int64_t)0, min((int64_t)w.ntok, P.num_tokens - w.t));
        if (map == 0)
          for (int i = lane; i < nt * grp * vhs; i += 32) {
            const int tt = i / (grp * vhs), rem = i - tt * grp * vhs;
            reinterpret_cast<T*>(P.out)[((w.t + tt) * P.H + gk * grp) * (int64_t)vhs + rem] =
                Half<T>::from_f32(0.f);
          }
        w.status = 2;
      }
    }
    if (lane == 0) work = w;
    __syncwarp();
    if (w.status == 0 && elect_one()) {  // the query, ahead of everything else
      const uint32_t qb = smem_u32(&bars->q_tma);
      mbar_expect_tx(qb, (uint32_t)(slabs * grp * P.tpc * 128));
      for (int slab = 0; slab < slabs; ++slab)
        tma_load_4d(smem_u32(q_s) + slab * kBox, &qmap, slab * 64, map, gk * grp, (int)w.t, qb);
    }
  } else if (warp == 1) {
    // a lane per barrier
    uint64_t* all = bars->k_full;
    for (int i = lane; i < kNumBars; i += 32) {
      uint32_t count = 1;
      if ((all + i >= bars->p_full && all + i < bars->p_full + 3) || all + i == &bars->q_full)
        count = kSoftWarps;
      mbar_init(smem_u32(all + i), count);
    }
    if (lane == 0) {
      bars->bad = 0;
      bars->abort = 0;
      bars->any_odd = 0;
    }
    if (lane < 8) bars->odd[lane] = 0;
    fence_barrier_init();
  } else if (warp == kProdWarp && lane == 0) {
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    prefetch_tmap(&qmap);
  } else if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp != 0 && !P.early) grid_dep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t col_s = vg;  // buffers of kN columns: S, then P in its place
  const int bufs = A.bufs;
  volatile int* abort = &bars->abort;
  const Work W = work;
  const bool run = W.status == 0;
  const int ntok = W.ntok, rows = run ? ntok * grp : 0;
  const int n = run ? (int)max((int64_t)0, W.t_end - W.t_begin) : 0;

  // what the softmax threads carry to the epilogue
  const int half = warp >> 2, row = (warp & 3) * 32 + lane;
  const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const bool live = warp < kSoftWarps && (warp & 3) * 32 < rows;
  float coef = 0.f;
  bool ok = true;

  if (run) {
    const int64_t pos = W.pos, t_begin = W.t_begin;
    const int64_t pos_hi = pos + ntok - 1;
    const int64_t lo = P.window >= 0 ? max((int64_t)0, pos - P.window) : 0;
    const int64_t lo_hi = P.window >= 0 ? max((int64_t)0, pos_hi - P.window) : 0;

    if (warp < kSoftWarps) {
      // =================== softmax ===================
      const int64_t pos_r = row < rows ? pos + divide(row, A.by_grp) : -1;
      const int64_t lo_r = P.window >= 0 ? max((int64_t)0, pos_r - P.window) : 0;
      RowAngles<T> ang;
      if (row < rows && P.rd > 0 && !P.interleaved) ang.load(P, half, pos_r);
      float lam = 0.f;
      if (map == 1) {
        float d0 = 0.f, d1 = 0.f;
        const float* lv = A.lambda_vectors;
        for (int d = lane; d < A.hs; d += 32) {
          d0 = fmaf(lv[d], lv[A.hs + d], d0);
          d1 = fmaf(lv[2 * A.hs + d], lv[3 * A.hs + d], d1);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          d0 += __shfl_xor_sync(0xffffffffu, d0, o);
          d1 += __shfl_xor_sync(0xffffffffu, d1, o);
        }
        lam = expf(d0) - expf(d1) + A.lambda_init;
      }
      ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->q_tma), 0, abort, P.err_flags));
      if (ok && row < rows && P.rd > 0) rotate_row<T>(q_s, q_lo, row, half, P, pos_r, ang);
      fence_proxy_async();
      arrive_warp(&bars->q_full, lane);

      float m_used = -INFINITY, l = 0.f;
      const float sl = CAP ? 1.f : P.scale_log2;
      auto score = [&](float v) {  // log2-domain score of a raw one
        return !CAP ? v * sl : v == -INFINITY ? -INFINITY : P.cap_out * tanh_ex2(v * P.cap_in);
      };
      // Scales columns [c0, c1) of this row of O, once the PV before tile k has
      // added to it.
      auto rescale_o = [&](int k, float factor, int c0, int c1) {
        const bool w = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->pv_done[(k - 1) & 1]),
                                                        ((k - 1) >> 1) & 1, abort, P.err_flags));
        if (w) {
          tc_fence_after();
#pragma unroll 1
          for (int c = c0; c < c1; c += 16) {
            uint32_t r[16];
            tmem_ld16(lane_addr + c, r);
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * factor);
            tmem_st16(lane_addr + c, r);
          }
        }
        return w;
      };
      // Every warp goes through all n tiles and meets its partner of the
      // quadrant in each; after a wait that gave up (ok false) it does nothing
      // else.
      int buf = 0;
      uint32_t spar = 0;
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const int pb = k & 1;
        const uint32_t cols = lane_addr + col_s + buf * kN + half * 64;  // this thread's
        const int64_t j0 = (t_begin + k) * kN;
        const bool edge = j0 < lo_hi || j0 + kN - 1 > pos;
        if (ok)
          ok = __all_sync(0xffffffffu,
                          wait_bar(smem_u32(&bars->s_full[buf]), spar, abort, P.err_flags));
        uint64_t* p_full = &bars->p_full[buf];
        if (++buf == bufs) {
          buf = 0;
          spar ^= 1;
        }
        uint32_t s[2][32];
        if (live && ok) {
          tc_fence_after();
          tmem_ld32_nowait(cols, s[0]);
          tmem_ld32_nowait(cols + 32, s[1]);
          tmem_wait_ld();
          reg_fence(s[0]);
          reg_fence(s[1]);
          tc_fence_before();
        }
        // The exponentials use the running maximum as it stands; the tile's own
        // maximum is taken beside them, and only if it passes the running one by
        // more than 2^lazy (or there is none yet) do the two warps of the quadrant
        // exchange maxima and compute the tile again (waiting for the exchange
        // first was 1 % slower).
        float vmax = -INFINITY, lsum = 0.f;
        auto exps = [&]() {
          const float nm = Prob<T>::shift - (m_used == -INFINITY ? 0.f : m_used);
          uint32_t hi[16], lo[16];
          lsum = exp_row<T, CAP>(s[0], hi, lo, P, nm);
          tmem_st16(cols, hi);
          tmem_st16(cols + 32, lo);
          lsum += exp_row<T, CAP>(s[1], hi, lo, P, nm);
          tmem_st16(cols + 16, hi);
          tmem_st16(cols + 48, lo);
        };
        bool again = false;
        if (live && ok) {
          if (edge) {
            const int c0 = (int)min((int64_t)kN, max((int64_t)0, lo_r - j0)) - half * 64;
            const int c1 = (int)max((int64_t)-1, min((int64_t)(kN - 1), pos_r - j0)) - half * 64;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c * 32 + e < c0 || c * 32 + e > c1) s[c][e] = __float_as_uint(-INFINITY);
          }
          if (k > 0) exps();
          vmax = fmaxf(max32(s[0]), max32(s[1]));
          again = __any_sync(0xffffffffu,
                             row < rows && (m_used == -INFINITY ||
                                            score(vmax) > m_used + Prob<T>::lazy));
        }
        if (live) {
          if (lane == 0) s_again[pb][half][warp & 3] = again ? 1 : 0;
          named_sync(1 + (warp & 3), 64);
          if (s_again[pb][0][warp & 3] | s_again[pb][1][warp & 3]) {
            s_max[half][row] = vmax;
            named_sync(1 + (warp & 3), 64);
            if (ok) {
              const float mt = score(fmaxf(s_max[0][row], s_max[1][row]));
              float factor = 1.f;
              bool rescale = false;
              if (m_used == -INFINITY) {
                m_used = mt;  // (nothing but zeros was added before a first visible key)
              } else if (mt > m_used + Prob<T>::lazy) {
                factor = ex2(m_used - mt);
                m_used = mt;
                l *= factor;
                rescale = true;
              }
              tmem_wait_st();  // nothing else orders two stores to the same columns
              exps();
              // (k >= 1) each half scales half of O
              if (__any_sync(0xffffffffu, rescale))
                ok = rescale_o(k, factor, half * (vg >> 1), (half + 1) * (vg >> 1));
            }
          }
          l += lsum;
          tmem_wait_st();
          tc_fence_before();
        }
        if (ok) arrive_warp(p_full, lane);
      }
      grid_dep_launch();
      uint4 nw = make_uint4(0, 0, 0, 0);
      if (tid * 8 < vhs) nw = reinterpret_cast<const uint4*>(A.norm_weight)[tid];
      named_sync(9, kSoft);
      // All products, by a barrier with one phase. (pv_done has a phase for every
      // second tile: with three buffers the scores of the last tile may be there
      // before PV of tile n - 3 is, and a wait for tile n - 1's phase would return
      // at once, as one for the phase before it does.)
      if (ok && n > 0)
        ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&bars->drain), 0, abort, P.err_flags));
      ok = __all_sync(0xffffffffu, ok && !*abort);  // (a role that gave up comes here too)
      tc_fence_after();
      if (live) {
        s_sum[half][row] = l;
      }
      if (tid * 8 < vhs) s_norm[tid] = nw;
      named_sync(9, kSoft);
      const float lt = s_sum[0][row] + s_sum[1][row];
      coef = lt > 0.f ? (map == 0 ? 1.f : lam) / lt : 0.f;
      if (bars->any_odd) {
        // (from the unit's record again: nothing of this is kept over the tiles)
        const int64_t p0 = work.pos, last = p0 + divide(row, A.by_grp);
        const int64_t back = P.window >= 0 ? P.window : last;
#pragma unroll 1
        for (int i = 0; i < 256; ++i)
          if (bars->odd[i >> 5] >> (i & 31) & 1u) {
            const int64_t j = i < 128 ? p0 + i : max((int64_t)0, p0 - back) + (i - 128);
            if (j <= last && j >= last - back) coef = NAN;
          }
      }
    } else if (warp < kMmaWarp) {
      // =================== TMA producers ===================
      const bool keys = warp == kProdWarp;
      int dirty_from = 0;
      if (P.early && P.own_slots) dirty_from = (int)max((int64_t)0, W.past / kN - t_begin);
      bool waited = !P.early;
      const int32_t* bt = P.block_table + (int64_t)W.b * P.max_blocks;
      const int sh = __ffs(P.bs) - 1;
      // keys: a tile per slot; values: this warp's half tile, every second of the line
      const int slots = keys ? A.nk : A.nv, step = keys ? 1 : 2, h = keys ? 0 : warp - kProdWarp - 1;
      uint64_t* full = keys ? bars->k_full : bars->v_full;
      uint64_t* empty = keys ? bars->k_empty : bars->v_empty;
      const uint32_t bytes = keys ? (uint32_t)P.k_bytes : (uint32_t)A.v_bytes;
      const uint32_t base = keys ? smem_u32(k_s) : smem_u32(v_s);
      const uint32_t slab_bytes = keys ? kBox : kVBox;
      const int box = keys ? P.box_rows : A.v_rows, nbox = (keys ? kN : kVKeys) / box;
      const CUtensorMap* tm = keys ? &kmap : &vmap;
      const int head = keys ? 2 * gk + map : gk, nslab = keys ? slabs : vslabs;
      const bool whole = keys ? A.k_whole : A.v_whole;
      int slot = h, issued = 0;
      uint32_t par = 1;
      // Value slots at an end of the keys land on a barrier of their own; this
      // warp zeroes what not all rows see, one tile later (the next copy is on
      // its way then), and only then says that they are full.
      uint64_t* land = bars->v_land[h];
      uint32_t land_par = 0;  // a bit per barrier
      int held = -1, held_slot = 0;
      auto release = [&]() {
        if (held < 0) return;
        const uint32_t bar = smem_u32(&land[held & 1]), p = land_par >> (held & 1) & 1u;
        if (__all_sync(0xffffffffu, wait_bar(bar, p, abort, P.err_flags))) {
          zero_values<T>(v_s + held_slot * A.v_bytes, bars, vslabs,
                         (t_begin + held) * kN + h * kVKeys, lo, lo_hi, pos, pos_hi, lane);
          fence_proxy_async();
        } else if (lane == 0) {
          drain_wait(bar, p, P.err_flags);
        }
        land_par ^= 1u << (held & 1);
        arrive_warp(&full[held_slot], lane);
        held = -1;
      };
      for (int k = 0; k < n; ++k) {
        if (!waited && k >= dirty_from) {
          grid_dep_wait();
          waited = true;
        }
        // cache row of box `lane` (out of range where no row of the unit sees
        // it, or its page is invalid: TMA fills zeros)
        int y = (int)P.num_slots;
        const int64_t key0 = (t_begin + k) * kN + h * kVKeys + (int64_t)lane * box;
        if (lane < nbox && key0 <= pos_hi && key0 + box - 1 >= lo) {
          const int32_t phys = bt[key0 >> sh];
          if (phys >= 0 && phys < P.num_blocks) {
            y = (int)((int64_t)phys * P.bs + (key0 & (int64_t)(P.bs - 1)));
          } else {
            bars->bad = 1;
            raise_flag(P.err_flags, PA_DEVERR_BLOCK);
          }
        }
        if (issued * step + h >= slots) {
          release();  // (the wait may be for the product behind these values)
          bool w = true;
          if (lane == 0) w = wait_bar(smem_u32(&empty[slot]), par, abort, P.err_flags);
          if (!__shfl_sync(0xffffffffu, w ? 1 : 0, 0)) break;
        }
        const int64_t h0 = (t_begin + k) * kN + h * kVKeys;
        const bool ends = !keys && (h0 < lo_hi || h0 + kVKeys - 1 > pos);
        const uint32_t bar = smem_u32(ends ? &land[k & 1] : &full[slot]), dst0 = base + slot * bytes;
        const int y0 = __shfl_sync(0xffffffffu, y, 0);
        if (elect_one()) mbar_expect_tx(bar, bytes);
        __syncwarp();
        if (nbox == 1) {
          if (elect_one()) {
            if (whole) {
              tma_load_4d(dst0, tm, 0, head, y0, 0, bar);
            } else {
              for (int c = 0; c < nslab; ++c)
                tma_load_4d(dst0 + c * slab_bytes, tm, c * 64, head, y0, 0, bar);
            }
          }
        } else if (lane < nbox) {  // a lane per box
          const uint32_t dst = dst0 + lane * box * 128;
          for (int c = 0; c < nslab; ++c)
            tma_load_4d(dst + c * slab_bytes, tm, whole ? 0 : c * 64, head, y, whole ? c : 0, bar);
        }
        __syncwarp();
        release();
        if (ends) {
          held = k;
          held_slot = slot;
        }
        ++issued;
        slot += step;
        if (slot >= slots) {
          slot -= slots;
          par ^= 1;
        }
        __syncwarp();
      }
      release();
      if (!waited) grid_dep_wait();
      if (*abort && lane == 0) {  // copies may be in flight: wait for each slot's last
        if (keys) drain_wait(smem_u32(&bars->q_tma), 0, P.err_flags);
        for (int i = max(0, issued - (slots + step - 1) / step); i < issued; ++i)
          drain_wait(smem_u32(&full[(i * step + h) % slots]), ((i * step + h) / slots) & 1,
                     P.err_flags);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // =================== MMA issuer ===================
      if (elect_one()) {
        constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
        constexpr uint32_t id_qk = idesc_f16(kBf16, kRows, kN, false);
        const uint32_t id_pv = idesc_f16(kBf16, kRows, vg, true);
        const int nk = P.hs >> 4;
        const uint64_t q_desc = sdesc(smem_u32(q_s), 16, 1024);
        const uint32_t k_base = smem_u32(k_s), v_base = smem_u32(v_s);
        int sk = 0, sv = 0;  // next slots, and their parities
        uint32_t kpar = 0, vpar = 0;
        auto wait = [&](uint64_t* bar, uint32_t par) {
          return wait_bar(smem_u32(bar), par, abort, P.err_flags);
        };
        const uint64_t lo_desc = sdesc(smem_u32(q_lo), 16, 1024);
        int sb = 0;  // the next buffer of S
        auto qk = [&]() {
          if (!wait(&bars->k_full[sk], kpar)) return false;
          tc_fence_after();
          const uint64_t kd = sdesc(k_base + sk * P.k_bytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if (kk < nk) {
              const uint32_t o = (uint32_t)(kk >> 2) * (kBox >> 4) + (uint32_t)(kk & 3) * 2;
              mma_ss(tmem + col_s + sb * kN, q_desc + o, kd + o, id_qk, kk > 0 ? 1u : 0u);
            }
          }
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if (kk >= A.lo0 && kk < A.lo1) {
              const uint32_t o = (uint32_t)(kk >> 2) * (kBox >> 4) + (uint32_t)(kk & 3) * 2;
              mma_ss(tmem + col_s + sb * kN, lo_desc + o, kd + o, id_qk, 1u);
            }
          }
          tc_commit(smem_u32(&bars->s_full[sb]));
          if (++sb == bufs) sb = 0;
          tc_commit(smem_u32(&bars->k_empty[sk]));
          if (++sk == A.nk) {
            sk = 0;
            kpar ^= 1;
          }
          return true;
        };
        auto pv = [&](int k, int pbuf, int hp) {
          if (!wait(&bars->v_full[sv], vpar)) return false;
          tc_fence_after();
          const uint64_t vd = sdesc(v_base + sv * A.v_bytes, kVBox, 1024);
          const uint32_t pa = tmem + col_s + pbuf * kN + hp * 64;
#pragma unroll
          for (int kk = 0; kk < kVKeys / 16; ++kk)
            mma_ts(tmem, pa + kk * 8, vd + (uint64_t)(kk * 128), id_pv,
                   (k > 0 || hp || kk > 0) ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < kVKeys / 16; ++kk)  // the remainders
            mma_ts(tmem, pa + 32 + kk * 8, vd + (uint64_t)(kk * 128), id_pv, 1u);
          tc_commit(smem_u32(&bars->v_empty[sv]));
          if (++sv == A.nv) {
            sv = 0;
            vpar ^= 1;
          }
          return true;
        };
        // QK^T runs `bufs` - 1 tiles ahead of PV. Its buffer held P of the tile whose
        // PV was issued last, and products run in the order of their issue.
        int pbuf = 0;
        uint32_t ppar = 0;
        bool go = wait(&bars->q_full, 0) && qk();
        if (bufs == 3 && n > 1) go = go && qk();
        for (int k = 0; k < n && go; ++k) {
          if (k + bufs - 1 < n) go = qk();
          go = go && wait(&bars->p_full[pbuf], ppar) && pv(k, pbuf, 0) && pv(k, pbuf, 1);
          if (go) tc_commit(smem_u32(&bars->pv_done[k & 1]));
          if (++pbuf == bufs) {
            pbuf = 0;
            ppar ^= 1;
          }
        }
        tc_commit(smem_u32(&bars->drain));
        drain_wait(smem_u32(&bars->drain), 0, P.err_flags);
      }
      __syncwarp();
    }
  } else {
    if (P.early) grid_dep_wait();
    grid_dep_launch();
  }

  // =================== epilogue ===================
  // CTA r finishes channels [r vg / 2, (r + 1) vg / 2). The cluster barriers are
  // met by every thread of both CTAs, whatever the unit's state. The outputs
  // travel a quadrant of 32 rows at a time. Everything is a loop: code that a CTA
  // runs only once is fetched cold (short prompts 33.5 -> 32.5 us).
  const int cols = vg >> 2;        // columns a thread hands over, and columns it finishes
  const int xquad = 32 * vg * 2;   // half the channels of a quadrant's rows, f32
  uint8_t* x_out = k_s;            // in the rings, which nobody uses any more
  uint8_t* x_in = k_s + 4 * xquad;
  const int quad = warp & 3;
  const bool fin = live && ok && n > 0;
  // 16-byte chunk ch of row r stands at ch ^ (r & 7)
  auto chunk = [&](uint8_t* at, int pitch, int ch) {
    return at + row * pitch + ((ch ^ (row & 7)) << 4);
  };
  cluster_arrive();  // this CTA's rings are free
  if (fin) {
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
      uint32_t r[16];
      tmem_ld16(lane_addr + (1 - map) * (vg >> 1) + half * cols + c, r);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4*>(chunk(x_out, vg * 2, ((half * cols + c) >> 2) + e)) =
            make_float4(__uint_as_float(r[4 * e]) * coef, __uint_as_float(r[4 * e + 1]) * coef,
                        __uint_as_float(r[4 * e + 2]) * coef, __uint_as_float(r[4 * e + 3]) * coef);
    }
    fence_proxy_async();
  }
  if (live) named_sync(1 + quad, 64);
  cluster_wait();  // the peer's are
  if (live) {
    uint64_t* full = &bars->x_full[quad];
    if (half == 0 && elect_one()) {
      mbar_expect_tx(smem_u32(full), (uint32_t)xquad);
      if (ok)
        bulk_copy_peer(map_peer(smem_u32(x_in + quad * xquad), 1 - map),
                       smem_u32(x_out + quad * xquad), (uint32_t)xquad,
                       map_peer(smem_u32(full), 1 - map));
    }
    __syncwarp();
    if (ok)
      ok = __all_sync(0xffffffffu, wait_bar(smem_u32(full), 0, abort, P.err_flags));
    else if (half == 0 && lane == 0)  // the peer may write into this CTA until then
      drain_wait(smem_u32(full), 0, P.err_flags);
    __syncwarp();
  }
  if (fin && ok) {  // the difference, in place of the peer's part
    float ss = 0.f;
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
      uint32_t r[16];
      tmem_ld16(lane_addr + map * (vg >> 1) + half * cols + c, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float4* at = reinterpret_cast<float4*>(chunk(x_in, vg * 2, ((half * cols + c) >> 2) + e));
        const float4 p = *at;
        float d[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float own = __uint_as_float(r[4 * e + i]) * coef;
          d[i] = map == 0 ? own - d[i] : d[i] - own;
          ss = fmaf(d[i], d[i], ss);
        }
        *at = make_float4(d[0], d[1], d[2], d[3]);
      }
    }
    s_ss[map * 2 + half][row] = ss;
    st_peer(map_peer(smem_u32(&s_ss[map * 2 + half][row]), 1 - map), ss);
  }
  cluster_sync_all();
  // the finished 16-bit channels go through shared memory, so that a warp
  // writes whole rows: 2 rows of 256 bytes at vg 256
  const int pitch = vg <= 128 ? 128 : 256;
  const int first = map * (vg >> 1);  // this CTA's channels
  if (fin && ok) {
    const float ss = (s_ss[0][row] + s_ss[1][row]) + (s_ss[2][row] + s_ss[3][row]);
    const bool bad = bars->bad != 0;
    const float inv = (1.f - A.lambda_init) / sqrtf(ss / (float)vhs + A.norm_eps);
#pragma unroll 1
    for (int c = 0; c < cols; c += 8) {
      const int ch = half * cols + c;
      if (first + ch < vhs) {
        float w[8], o[8];
        unpack8<T>(s_norm[(first + ch) >> 3], w);
        const float4 p = *reinterpret_cast<const float4*>(chunk(x_in, vg * 2, ch >> 2));
        const float4 q = *reinterpret_cast<const float4*>(chunk(x_in, vg * 2, (ch >> 2) + 1));
        const float x[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = bad ? 0.f : x[e] * inv * w[e];
        *reinterpret_cast<uint4*>(chunk(x_out, pitch, ch >> 3)) = pack8<T>(o);
      }
    }
  }
  if (run && warp < kSoftWarps) {
    named_sync(9, kSoft);
    // 16 lanes a row
    const int nc = max(0, min(vg >> 1, vhs - first)) >> 3, c = lane & 15;
    if (ok && !*abort && c < nc) {
      T* base = reinterpret_cast<T*>(P.out) + (W.t * P.H + gk * grp) * (int64_t)vhs + first + c * 8;
      for (int q = warp * 2 + (lane >> 4); q < rows; q += kSoftWarps * 2) {
        const int tok = divide(q, A.by_grp);
        *reinterpret_cast<uint4*>(base + ((int64_t)tok * P.H + (q - tok * grp)) * vhs) =
            *reinterpret_cast<const uint4*>(x_out + q * pitch + ((c ^ (q & 7)) << 4));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
cudaError_t encode(CUtensorMap* map, bool bf16, const void* base, int rank, const cuuint64_t* dims,
                   const cuuint64_t* str, const cuuint32_t* box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             (cuuint32_t)rank, const_cast<void*>(base), dims, str, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// A cache of `heads` rows of `width` channels per slot, as (channel, head, slot,
// slab). A width that is a multiple of 64 is cut into slabs of 64 channels (the
// fourth dimension, 128 bytes apart), so that one box of `rows` slots holds all
// of them, slab after slab; otherwise the channels stay one dimension, which
// ends at the width (zeros behind it), and a box holds one slab.
// `all`: boxes of all slabs (else of one).
cudaError_t cache_map(CUtensorMap* map, bool bf16, const void* base, int width, int heads,
                      cuuint64_t slots, int rows, bool all) {
  const bool whole = width % 64 == 0;
  const cuuint64_t wb = (cuuint64_t)width * 2;
  const cuuint64_t dims[4] = {whole ? 64u : (cuuint64_t)width, (cuuint64_t)heads, slots,
                              whole ? (cuuint64_t)(width / 64) : 1u};
  const cuuint64_t str[3] = {wb, wb * heads, 128};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)rows,
                             whole && all ? (cuuint32_t)(width / 64) : 1u};
  return encode(map, bf16, base, 4, dims, str, box);
}

template <typename T, bool CAP>
cudaError_t launch(const Geometry& g, const DiffArgs& a, const PreArgs& A, int64_t units) {
  static std::atomic<bool> configured[64];
  auto kern = diff_prefill_kernel<T, CAP>;
  cudaError_t e = once_per_device(configured, g.device, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  });
  if (e != cudaSuccess) return e;
  const Params& P = A.P;
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const cuuint64_t slots = (cuuint64_t)g.num_blocks * g.bs, hb = (cuuint64_t)g.hs * 2;
  CUtensorMap kmap, vmap, qmap;
  e = cache_map(&kmap, bf16, a.key_cache, g.hs, 2 * g.kvh, slots, P.box_rows, P.box_rows == kN);
  if (e == cudaSuccess)
    e = cache_map(&vmap, bf16, a.value_cache, g.vhs, g.kvh, slots, A.v_rows, A.v_rows == kVKeys);
  if (e != cudaSuccess) return e;
  {  // query [T][H][2][hs]: boxes of 64 channels x one map x grp heads x tpc tokens
    const cuuint64_t dims[4] = {(cuuint64_t)g.hs, 2, (cuuint64_t)g.H, (cuuint64_t)a.num_tokens};
    const cuuint64_t str[3] = {hb, 2 * hb, 2 * hb * g.H};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)P.grp, (cuuint32_t)P.tpc};
    if ((e = encode(&qmap, bf16, a.query, 4, dims, str, box)) != cudaSuccess) return e;
  }
  const size_t smem =
      1024 + (size_t)P.q_bytes * (P.rd > 0 ? 2 : 1) + (size_t)A.nk * P.k_bytes +
      (size_t)A.nv * A.v_bytes;
  return launch_pdl(kern, dim3((unsigned)(units * g.kvh * 2)), dim3(kPreThreads), smem, a.stream,
                    kmap, vmap, qmap, A);
}

}  // namespace

static Divisor divisor(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return {(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

cudaError_t launch_prefill(const Geometry& g, const DiffArgs& a) {
  PreArgs A{};
  Params& P = A.P;
  const int grp = g.H / g.kvh;
  P.out = a.out;
  P.cos_cache = a.cos_cache;
  P.sin_cache = a.sin_cache;
  P.cumseq = a.cumseq;
  P.past = a.past;
  P.block_table = a.block_table;
  P.err_flags = a.err_flags;
  P.num_tokens = a.num_tokens;
  P.num_slots = (int64_t)g.num_blocks * g.bs;
  P.num_seqs = a.num_seqs;
  P.pf_begin = P.seq_begin = a.seq_begin;
  P.pf_end = P.seq_end = a.seq_end;
  P.H = g.H;
  P.hs = g.hs;
  P.vhs = g.vhs;
  P.ro = g.ro;
  P.rd = g.rd;
  P.interleaved = g.interleaved;
  P.cos_rows = g.cos_rows;
  P.bs = g.bs;
  P.num_blocks = g.num_blocks;
  P.max_blocks = g.max_blocks;
  P.scale_log2 = g.scale * kLog2e;
  P.cap_in = g.softcap > 0.f ? g.scale / g.softcap : 0.f;
  P.cap_out = g.softcap * kLog2e;
  P.window = g.window;
  P.box_rows = g.bs < kN ? g.bs : kN;
  P.early = (g.flags & PA_FLAG_AFTER_WRITE) ? 1 : 0;
  P.own_slots = (g.flags & PA_FLAG_OWN_SLOTS) ? 1 : 0;
  P.kvh = g.kvh;
  P.grp = grp;
  P.tpc = kRows / grp;
  A.by_kvh = divisor((uint32_t)g.kvh);
  A.by_tpc = divisor((uint32_t)P.tpc);
  A.by_grp = divisor((uint32_t)grp);
  P.slabs = (g.hs + 63) / 64;
  P.vslabs = (g.vhs + 63) / 64;
  P.vg = 64 * P.vslabs;
  P.q_bytes = P.slabs * kBox;
  P.k_bytes = P.slabs * kBox;
  A.v_rows = g.bs < kVKeys ? g.bs : kVKeys;
  A.v_bytes = P.vslabs * kVBox;
  // four key tiles (two of 32 KB), the rest for values: at least three halves
  A.nk = P.slabs == 1 ? 4 : 2;
  A.nv = (int)((kSmemMax - 1024 - 2 * P.q_bytes - (size_t)A.nk * P.k_bytes) / A.v_bytes);
  if (A.nv > kMaxV) A.nv = kMaxV;
  A.lo0 = g.rd > 0 ? g.ro / 16 : 0;
  A.lo1 = g.rd > 0 ? (g.ro + g.rd + 15) / 16 : 0;
  A.bufs = P.vg <= 128 ? 3 : 2;
  A.k_whole = g.hs % 64 == 0;
  A.v_whole = g.vhs % 64 == 0;
  A.hs = g.hs;
  A.lambda_vectors = a.lambda_vectors;
  A.norm_weight = a.norm_weight;
  A.lambda_init = a.lambda_init;
  A.norm_eps = a.norm_eps;
  // (a sequence with tokens has at most one unit that is not full)
  const int64_t units =
      a.num_tokens / P.tpc + std::min((int64_t)(a.seq_end - a.seq_begin), a.num_tokens);
  if (units * g.kvh * 2 > INT32_MAX) return cudaErrorInvalidConfiguration;
  const bool cap = g.softcap > 0.f;
  auto go = [&](auto* typed) {
    using T = std::remove_pointer_t<decltype(typed)>;
    return cap ? launch<T, true>(g, a, A, units) : launch<T, false>(g, a, A, units);
  };
  return g.dtype == PA_DTYPE_BF16 ? go((__nv_bfloat16*)nullptr) : go((__half*)nullptr);
}

}  // namespace diff
}  // namespace pa
