// Attention over 8-bit caches, decode: one new token per sequence
// (include/pa_quant.h), bound by HBM.
//
// The line. A unit is a sequence, a kv head and up to 8 NB of its query heads; its
// visible keys are cut into tiles of 16. All tiles of all units form one line,
// which is cut into equal parts, one per CTA, whatever the lengths. A CTA's part
// of a unit is a segment: its warps take the segment's tiles in turn, each with a
// softmax of its own, and join at the segment's end. A unit that lies in several
// parts is joined by quant_combine_kernel.
//
// Loads. Every lane copies (cp.async, 16 bytes) just the codes that it will
// multiply itself into a ring of its own, D tiles ahead and past the ends of
// segments, so there is no barrier between copies and products, and a tile's
// pages are looked up a batch of 32 tiles before. Key rows and value rows of a
// tile are read whole: 8 lanes of 16 bytes for 128 channels.
//
// Products. mma.sync m16n8k16, keys (then value channels) as the 16 rows and the
// heads as the 8 columns: with rows of heads, as the usual order has it, a group of
// eight or fewer would fill half of a product. The order of the 16 keys and of the
// channels inside the products is chosen so that what a lane has copied is what its
// registers of A hold: lane (g, t) = (lane / 4, lane % 4) owns
//   of key slot g and g + 8 (keys kappa = 4 (g / 2) + g % 2, and + 2): pieces of 16
//     channels t, t + 4, ..; a word of 4 codes is one k step's A registers
//   of the values of keys 4 t .. 4 t + 3: piece g (and g + 8); a byte of each of two
//     words is a register.
// E4M3 is exact in fp16; P^T becomes the B operand by movmatrix.
#include <algorithm>
#include <type_traits>

#include "pa_quant_read.cuh"

namespace pa {
namespace quant {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kTile = 16;
constexpr size_t kSmemMax = 225 * 1024;

struct DecP {
  ReadP R;
  float4* ws_o;     // [2 CTAs][8 VP NB][32] accumulators as the lanes hold them
  float2* ws_ml;    // [2 CTAs][8 NB] maximum (log2 domain), sum
  int64_t* ws_plan; // [nseq + 1] tiles before each sequence, then the tiles of a part
  int units;        // per sequence
  int chunks;       // units per kv head
  int min_part;
};

struct Span {  // the tiles that a sequence's token sees
  int64_t lo, last, t;  // first and last key, token
  int tiles, first;     // (first tile)
  int err;              // PA_DEVERR_* that keeps it from being read, or 0
  bool rows;            // it has a row of out
};
__device__ __forceinline__ Span span_of(const ReadP& P, int b) {
  const int64_t c0 = P.cumseq[P.seq_begin + b], c1 = P.cumseq[P.seq_begin + b + 1];
  const int64_t past = P.past[P.seq_begin + b];
  Span s;
  s.t = c0;
  s.last = P.cross ? past - 1 : past;
  s.lo = P.window >= 0 ? max((int64_t)0, s.last - P.window) : 0;
  s.rows = c1 - c0 == 1 && c0 >= 0 && c0 < P.num_tokens;
  s.err = c1 - c0 != 1                                                ? PA_DEVERR_DECODE_QLEN
          : !s.rows                                                   ? PA_DEVERR_CUMSEQ
          : past < 0 || s.last >= (int64_t)P.max_blocks * P.bs        ? PA_DEVERR_CONTEXT
          : P.rd > 0 && s.last >= P.cos_rows                          ? PA_DEVERR_POSITION
                                                                      : 0;
  s.first = (int)(s.lo / kTile);
  s.tiles = s.err || s.last < s.lo ? 0 : (int)(s.last / kTile) - s.first + 1;
  return s;
}

// A walk over the line: the segment that starts at tile x of the line, its unit,
// and the line's end for this CTA.
struct Walk {
  int64_t x, end, start;  // (start: of sequence b)
  int b, tiles, first;
  int unit, from, len;    // the segment: unit, first tile (in the cache), tiles
  __device__ __forceinline__ bool valid() const { return x < end; }
  __device__ __forceinline__ void segment() {
    if (!valid()) return;
    const uint64_t off = (uint64_t)(x - start);
    unit = off >> 32 ? (int)(off / (uint32_t)tiles) : (int)((uint32_t)off / (uint32_t)tiles);
    const int in = (int)(off - (uint64_t)unit * tiles);
    from = first + in;
    len = (int)min((int64_t)(tiles - in), end - x);
  }
  __device__ __forceinline__ void next(const DecP& A) {
    x += len;
    if (!valid()) return;
    if (x == start + (int64_t)tiles * A.units) {
      start = x;
      do {
        const Span s = span_of(A.R, ++b);
        tiles = s.tiles;
        first = s.first;
      } while (tiles == 0);
    }
    segment();
  }
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// 16 bytes into shared memory; zeros where there is nothing to read.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Accumulators i0..i0 + 3 of a head block (see the products): eight channels of two
// heads, times inv, to out. `row`: the unit's first row of out.
template <typename F>
__device__ __forceinline__ void store_heads(const ReadP& P, int64_t row, int nh, int h, int gq,
                                            int i0, bool zero, const float (&inv)[2], F&& acc) {
  const int ch = 16 * (gq + (i0 & ~7)) + 2 * (i0 & 7);
  if (ch >= P.vhs) return;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (h + e >= nh) continue;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = zero ? 0 : pack_out(P, acc(k, e) * inv[e], acc(k, e + 2) * inv[e]);
    *reinterpret_cast<uint4*>(reinterpret_cast<__half*>(P.out) + (row + h + e) * P.vhs + ch) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// What the sink of head h0 + h adds to a sum with maximum m.
__device__ __forceinline__ float sink_part(const ReadP& P, int h0, int h, int nh, float m) {
  return P.head_sink && h < nh ? ex2(to_f32(P, P.head_sink, h0 + h) * kLog2e - m + kShift) : 0.f;
}

// Shared memory of a CTA behind the rings: the query and the joining buffers.
template <int KP, int VP, int NB>
struct Shape {
  static constexpr int kStage = (2 * KP + 4 * VP) * 512;  // bytes of a warp's tile
  static constexpr int kRow = KP * 64 + 8;                // halves of a query row
  static constexpr int kAcc = 8 * VP * NB;                // float4 accumulators of a lane
  static constexpr int kQ = 8 * NB * kRow * 2;
  static constexpr int kJoin = (kWarps / 2) * (kAcc * 512 + NB * 128);
  static constexpr int kLeft = (int)kSmemMax - kQ - kJoin - 8 * NB * 4 - 1024;
  static constexpr int kFit = kLeft / (kWarps * (kStage + 8));
  static constexpr int D = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kWarps * D * (kStage + 8) + kQ + kJoin + 8 * NB * 4;
  static_assert(D >= 2, "ring");
};

template <int KP, int VP, int NB>
__global__ void __launch_bounds__(kThreads, 1)
quant_decode_kernel(const __grid_constant__ DecP A) {
  using S = Shape<KP, VP, NB>;
  constexpr int D = S::D;
  const ReadP& P = A.R;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* ring = smem;
  float2* meta = reinterpret_cast<float2*>(smem + kWarps * D * S::kStage);  // [warp][D]
  __half* s_q = reinterpret_cast<__half*>(reinterpret_cast<uint8_t*>(meta) + kWarps * D * 8);
  float4* join_o = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(s_q) + S::kQ);
  float2* join_ml = reinterpret_cast<float2*>(join_o + (kWarps / 2) * S::kAcc * 32);
  float* s_mult = reinterpret_cast<float*>(join_ml + (kWarps / 2) * NB * 16);
  __shared__ int64_t s_scan[kWarps];
  __shared__ int64_t s_hit[2];  // sequence of this CTA's first tile, tiles before it
  __shared__ int s_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;

  if (!P.early) grid_dep_wait();

  // ---- the plan: tiles before each sequence (a prefix sum, 256 sequences a round)
  int64_t carry = 0, my_start = 0;
  int mine = 0;
  if (tid == 0) s_hit[0] = -1;
  auto round = [&](int base) {  // start of sequence base + tid, and the carry behind the round
    const int b = base + tid;
    mine = b < P.nseq ? span_of(P, b).tiles : 0;
    int64_t v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = v;
    __syncthreads();
    int64_t before = carry;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_scan[w];
      carry += s_scan[w];
    }
    my_start = before + v - mine;
    if (blockIdx.x == 0 && b < P.nseq) A.ws_plan[b] = my_start;
  };
  for (int base = 0; base < P.nseq; base += kThreads) round(base);
  const int64_t total = carry * A.units;
  const int64_t part = max((int64_t)A.min_part, (total + gridDim.x - 1) / gridDim.x);
  if (blockIdx.x == 0 && tid == 0) A.ws_plan[P.nseq] = part;
  Walk W;
  W.x = min(total, blockIdx.x * part);
  W.end = min(total, W.x + part);
  for (int base = 0; base < P.nseq && W.x < W.end; base += kThreads) {
    if (P.nseq > kThreads) {
      if (base == 0) carry = 0;
      round(base);
    }
    if (mine > 0 && my_start * A.units <= W.x && W.x < (my_start + mine) * A.units) {
      s_hit[0] = base + tid;
      s_hit[1] = my_start;
    }
  }
  __syncthreads();
  if (W.valid()) {
    W.b = (int)s_hit[0];
    W.start = s_hit[1] * A.units;
    const Span s = span_of(P, W.b);
    W.tiles = s.tiles;
    W.first = s.first;
    W.segment();
  }
  if (P.early) grid_dep_wait();

  // ---- this warp's copies: a walk of its own ahead of the products
  Walk C = W;
  int ct = 0;        // next tile of its segment (counting the warp's own)
  int page0 = 0, page1 = 0;     // of this batch's and the next batch's tiles, a lane each
  float2 sc0 = make_float2(0.f, 0.f), sc1 = sc0;
  const int64_t krow = (int64_t)P.kvh * P.hs, vrow = (int64_t)P.kvh * P.vhs;
  const int npk = P.hs >> 4, npv = P.vhs >> 4;
  auto own_tiles = [&](const Walk& w) {
    return w.len > warp ? (w.len - warp + kWarps - 1) / kWarps : 0;
  };
  auto look_up = [&](int k) {  // the page of the warp's tile k + lane
    const int64_t key = (int64_t)(C.from + warp + (k + lane) * kWarps) * kTile;
    return k + lane < own_tiles(C)
               ? P.block_table[(int64_t)(P.seq_begin + C.b) * P.max_blocks + (key >> P.sh)]
               : 0;
  };
  auto scale_at = [&](int page) {
    return page >= 0 && page < P.num_blocks
               ? P.scales[(int64_t)page * P.kvh + C.unit / A.chunks]
               : make_float2(0.f, 0.f);
  };
  auto enter = [&]() {  // the first segment from here on with a tile of this warp
    while (C.valid() && own_tiles(C) == 0) C.next(A);
    ct = 0;
    if (C.valid()) {
      page0 = look_up(0);
      sc0 = scale_at(page0);
    }
  };
  int put = 0;
  const int kappa = 4 * (gq >> 1) + (gq & 1);
  uint8_t* my_ring = ring + warp * D * S::kStage + lane * 16;
  auto produce = [&]() {
    if (C.valid()) {
      const int k = ct & 31;
      if (k == 8) page1 = look_up((ct & ~31) + 32);
      if (k == 16) sc1 = scale_at(page1);
      const int page = __shfl_sync(0xffffffffu, page0, k);
      const float ks = __shfl_sync(0xffffffffu, sc0.x, k), vs = __shfl_sync(0xffffffffu, sc0.y, k);
      const bool good = page >= 0 && page < P.num_blocks;
      const int ke = scale_exponent(ks), ve = scale_exponent(vs);
      const bool kin = good && ke != kNone, vin = good && ve != kNone;
      const int tile = C.from + warp + ct * kWarps;
      const int64_t row = (good ? (int64_t)page << P.sh : 0) + ((tile * kTile) & (P.bs - 1));
      const int g = C.unit / A.chunks;
      const uint32_t dst = smem_u32(my_ring + put * S::kStage);
      const uint8_t* kr = P.key_cache + (row + kappa) * krow + g * P.hs;
      const uint8_t* vr = P.value_cache + (row + 4 * tq) * vrow + g * P.vhs;
#pragma unroll
      for (int i = 0; i < KP; ++i) {
        const int piece = tq + 4 * i;
        const bool in = kin && piece < npk;
        const uint8_t* src = piece < npk ? kr + piece * 16 : kr;
        copy16(dst + (2 * i) * 512, src, in);
        copy16(dst + (2 * i + 1) * 512, src + 2 * krow, in);
      }
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        const int piece = gq + 8 * i;
        if (piece < npv) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            copy16(dst + (2 * KP + 4 * i + j) * 512, vr + j * vrow + piece * 16, vin);
        }
      }
      if (lane == 0)
        meta[warp * D + put] = make_float2(good ? (kin ? ks : 1.f) : NAN, vin ? (float)ve : kLeast);
      if (++ct == own_tiles(C)) {
        C.next(A);
        enter();
      } else if ((ct & 31) == 0) {
        page0 = page1;
        sc0 = sc1;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++put == D) put = 0;
  };
  enter();
#pragma unroll 1
  for (int i = 0; i < D; ++i) produce();
  int get = 0;

  // ---- segments
#pragma unroll 1
  while (W.valid()) {
    const int g = W.unit / A.chunks, h0 = (W.unit - g * A.chunks) * 8 * NB;
    const int nh = min(8 * NB, P.grp - h0);
    const Span sp = span_of(P, W.b);
    const int64_t qrow = sp.t * P.H + g * P.grp + h0;
    __syncthreads();
    if (tid == 0) s_bad = 0;
    for (int r = warp; r < 8 * NB; r += kWarps) {
      float x[8], back = 0.f;
      uint4 h = make_uint4(0, 0, 0, 0);
      if (r < nh) {
        if (P.bf16) query_row8<__nv_bfloat16>(P, qrow + r, sp.last, x);
        else query_row8<__half>(P, qrow + r, sp.last, x);
        back = scaled_row8(x, &h);
      }
      if (lane * 8 < KP * 64) *reinterpret_cast<uint4*>(s_q + r * S::kRow + lane * 8) = h;
      if (lane == 0) s_mult[r] = back * (P.cap_in > 0.f ? P.cap_in : P.scale_log2);
    }
    __syncthreads();
    constexpr bool kKeep = KP * NB <= 4;  // the query's fragments in registers
    uint32_t bq[kKeep ? NB : 1][kKeep ? KP : 1][8];
    auto q_frag = [&](int nb, int i, uint32_t (&f)[8]) {
      const uint4* src =
          reinterpret_cast<const uint4*>(s_q + (nb * 8 + gq) * S::kRow + 16 * (tq + 4 * i));
      const uint4 u = src[0], v = src[1];
      f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
      f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
    };
    if constexpr (kKeep) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < KP; ++i) q_frag(nb, i, bq[nb][i]);
    }
    float mult[NB][2], m[NB][2], l[NB][2];
    float acc[8 * VP][NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mult[nb][e] = s_mult[nb * 8 + 2 * tq + e];
        m[nb][e] = -INFINITY;
        l[nb][e] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < 8 * VP; ++i)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][nb][e] = 0.f;

    bool bad = false;
#pragma unroll 1
    for (int tile = W.from + warp; tile < W.from + W.len; tile += kWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
      __syncwarp();
      const uint4* at = reinterpret_cast<const uint4*>(my_ring + get * S::kStage);
      const float2 mt = meta[warp * D + get];
      if (++get == D) get = 0;
      const float ks = mt.x, ev = mt.y;
      bad |= isnan(ks);
      float c[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[nb][e] = 0.f;
#pragma unroll
      for (int i = 0; i < KP; ++i) {
        const uint4 r0 = at[(2 * i) * 32], r1 = at[(2 * i + 1) * 32];
        const uint32_t a[4] = {r0.x, r0.y, r0.z, r0.w}, b[4] = {r1.x, r1.y, r1.z, r1.w};
        uint32_t f[NB][8];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if constexpr (kKeep) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[nb][e] = bq[nb][i][e];
          } else {
            q_frag(nb, i, f[nb]);
          }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t a0 = codes2(a[s]), a2 = codes2(a[s] >> 16);
          const uint32_t a1 = codes2(b[s]), a3 = codes2(b[s] >> 16);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma(c[nb], a0, a1, a2, a3, f[nb][2 * s], f[nb][2 * s + 1]);
        }
      }
      // scores of keys kappa (c[0], c[1]) and kappa + 2 for heads 2 t and 2 t + 1
      const int64_t j0 = (int64_t)tile * kTile;
      const bool edge = j0 < sp.lo || j0 + kTile - 1 > sp.last;
      bool rise = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = ks * mult[nb][e & 1];
          float y = P.cap_in > 0.f ? capped(P, c[nb][e] * f) + ev : fmaf(c[nb][e], f, ev);
          if (edge) {
            const int64_t j = j0 + kappa + (e & 2);
            if (j < sp.lo || j > sp.last) y = -INFINITY;
          }
          c[nb][e] = y;
          rise |= y > m[nb][e & 1] + kLazy;
        }
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = fmaxf(c[nb][e], c[nb][e + 2]);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            if (t > m[nb][e]) {
              const float f = ex2(m[nb][e] - t);  // (from -inf: 0)
              m[nb][e] = t;
              l[nb][e] *= f;
#pragma unroll
              for (int i = 0; i < 8 * VP; ++i) {
                acc[i][nb][e] *= f;
                acc[i][nb][e + 2] *= f;
              }
            }
          }
      }
      uint32_t pb[NB][2];
      const float out_of = ex2(-ev);  // (a whole number: exact)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mm = m[nb][e & 1];
          p[e] = ex2(c[nb][e] - (mm == -INFINITY ? 0.f : mm) + kShift);
        }
        l[nb][0] = fmaf(p[0] + p[2], out_of, l[nb][0]);
        l[nb][1] = fmaf(p[1] + p[3], out_of, l[nb][1]);
        pb[nb][0] = transposed(tc::pack2<__half>(p[0], p[1]));
        pb[nb][1] = transposed(tc::pack2<__half>(p[2], p[3]));
      }
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = at[(2 * KP + 4 * i + j) * 32];
          if (edge && (j0 + 4 * tq + j < sp.lo || j0 + 4 * tq + j > sp.last))
            v[j] = make_uint4(0, 0, 0, 0);  // (0 times NaN is NaN)
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t w0 = word(v[0], s), w1 = word(v[1], s), w2 = word(v[2], s), w3 = word(v[3], s);
          const uint32_t x01 = __byte_perm(w0, w1, 0x5140), y01 = __byte_perm(w0, w1, 0x7362);
          const uint32_t x23 = __byte_perm(w2, w3, 0x5140), y23 = __byte_perm(w2, w3, 0x7362);
          uint32_t a0 = codes2(x01), a1 = codes2(x01 >> 16), a2 = codes2(x23), a3 = codes2(x23 >> 16);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma(acc[i * 8 + 2 * s][nb], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
          a0 = codes2(y01), a1 = codes2(y01 >> 16), a2 = codes2(y23), a3 = codes2(y23 >> 16);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma(acc[i * 8 + 2 * s + 1][nb], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
        }
      }
      __syncwarp();  // (meta is read)
      produce();
    }
    // a warp's sums over its key lanes
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], o);
    if (bad && lane == 0) s_bad = 1;
    // joined by halves: warps [n, 2 n) hand over to warps [0, n)
#pragma unroll 1
    for (int n = kWarps / 2; n > 0; n >>= 1) {
      if (n < kWarps / 2) __syncthreads();  // the buffers are read
      if (warp >= n && warp < 2 * n) {
#pragma unroll
        for (int i = 0; i < 8 * VP; ++i)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            join_o[((warp - n) * S::kAcc + i * NB + nb) * 32 + lane] =
                make_float4(acc[i][nb][0], acc[i][nb][1], acc[i][nb][2], acc[i][nb][3]);
        if (gq == 0) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              join_ml[(warp - n) * NB * 8 + nb * 8 + 2 * tq + e] = make_float2(m[nb][e], l[nb][e]);
        }
      }
      __syncthreads();
      if (warp < n) {
        float fa[NB][2], fb[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 o = join_ml[warp * NB * 8 + nb * 8 + 2 * tq + e];
            const float t = fmaxf(m[nb][e], o.x), base = t == -INFINITY ? 0.f : t;
            fa[nb][e] = ex2(m[nb][e] - base);
            fb[nb][e] = ex2(o.x - base);
            m[nb][e] = t;
            l[nb][e] = l[nb][e] * fa[nb][e] + o.y * fb[nb][e];
          }
#pragma unroll
        for (int i = 0; i < 8 * VP; ++i)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float4 o = join_o[(warp * S::kAcc + i * NB + nb) * 32 + lane];
            acc[i][nb][0] = acc[i][nb][0] * fa[nb][0] + o.x * fb[nb][0];
            acc[i][nb][1] = acc[i][nb][1] * fa[nb][1] + o.y * fb[nb][1];
            acc[i][nb][2] = acc[i][nb][2] * fa[nb][0] + o.z * fb[nb][0];
            acc[i][nb][3] = acc[i][nb][3] * fa[nb][1] + o.w * fb[nb][1];
          }
      }
    }
    if (warp == 0) {
      const bool any_bad = s_bad != 0;
      if (any_bad && lane == 0) raise_flag(P.err_flags, PA_DEVERR_BLOCK);
      if (W.len == W.tiles) {  // the whole unit
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float inv[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            inv[e] = 1.f / (l[nb][e] + sink_part(P, g * P.grp + h0, nb * 8 + 2 * tq + e, nh, m[nb][e]));
#pragma unroll
          for (int i = 0; i < 8 * VP; i += 4)
            store_heads(P, qrow, nh, nb * 8 + 2 * tq, gq, i, any_bad, inv,
                        [&](int k, int e) { return acc[i + k][nb][e]; });
        }
      } else {
        // the first part that starts in this CTA, or one behind another's end
        const int64_t slot = 2 * (int64_t)blockIdx.x + (W.x > blockIdx.x * part ? 1 : 0);
#pragma unroll
        for (int i = 0; i < 8 * VP; ++i)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            A.ws_o[(slot * S::kAcc + i * NB + nb) * 32 + lane] =
                make_float4(acc[i][nb][0], acc[i][nb][1], acc[i][nb][2], acc[i][nb][3]);
        if (gq == 0) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              A.ws_ml[slot * 8 * NB + nb * 8 + 2 * tq + e] =
                  make_float2(any_bad ? NAN : m[nb][e], l[nb][e]);
        }
      }
    }
    W.next(A);
  }
  grid_dep_launch();
  // sequences without tiles: told, and zeros
  for (int b = blockIdx.x; b < P.nseq; b += gridDim.x) {
    const Span s = span_of(P, b);
    if (s.err && tid == 0) raise_flag(P.err_flags, s.err);
    if (s.tiles == 0 && s.rows) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(P.out) + s.t * P.H * P.vhs / 2;
      for (int i = tid; i < P.H * P.vhs / 2; i += kThreads) dst[i] = 0;
    }
  }
}

// Joins the parts of a unit: a warp for four accumulators of a head block.
template <int VP, int NB>
__global__ void __launch_bounds__(64 * VP * NB)
quant_combine_kernel(const __grid_constant__ DecP A) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kAcc = 8 * VP * NB, kRound = 4;
  const ReadP& P = A.R;
  const int b = blockIdx.x / A.units, u = blockIdx.x - b * A.units;
  const int64_t part = A.ws_plan[P.nseq], before = A.ws_plan[b];
  const Span sp = span_of(P, b);
  if (sp.tiles == 0) return;
  const int64_t start = before * A.units + (int64_t)u * sp.tiles, end = start + sp.tiles;
  const int64_t c0 = start / part, c1 = (end - 1) / part;
  if (c0 == c1) return;
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const int task = threadIdx.x >> 5, nb = task % NB, i0 = task / NB * 4;
  const int g = u / A.chunks, h0 = (u - g * A.chunks) * 8 * NB, nh = min(8 * NB, P.grp - h0);
  const int h = nb * 8 + 2 * tq;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
  bool bad = false;
  for (int64_t c = c0; c <= c1; c += kRound) {
    float4 o[kRound][4];
    float4 ml[kRound];  // maximum and sum of heads h and h + 1
#pragma unroll
    for (int r = 0; r < kRound; ++r) {
      if (c + r > c1) continue;
      const int64_t slot = 2 * (c + r) + (c + r == c0 && start > c0 * part ? 1 : 0);
      ml[r] = *reinterpret_cast<const float4*>(A.ws_ml + slot * 8 * NB + h);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[r][k] = A.ws_o[(slot * kAcc + (i0 + k) * NB + nb) * 32 + lane];
    }
#pragma unroll
    for (int r = 0; r < kRound; ++r) {
      if (c + r > c1) continue;
      const float pm[2] = {ml[r].x, ml[r].z}, pl[2] = {ml[r].y, ml[r].w};
      float fa[2], fb[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        bad |= isnan(pm[e]);
        const float t = fmaxf(m[e], pm[e]), base = t == -INFINITY ? 0.f : t;
        fa[e] = ex2(m[e] - base);
        fb[e] = ex2(pm[e] - base);
        m[e] = t;
        l[e] = l[e] * fa[e] + pl[e] * fb[e];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[k][0] = acc[k][0] * fa[0] + o[r][k].x * fb[0];
        acc[k][1] = acc[k][1] * fa[1] + o[r][k].y * fb[1];
        acc[k][2] = acc[k][2] * fa[0] + o[r][k].z * fb[0];
        acc[k][3] = acc[k][3] * fa[1] + o[r][k].w * fb[1];
      }
    }
  }
  float inv[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) inv[e] = 1.f / (l[e] + sink_part(P, g * P.grp + h0, h + e, nh, m[e]));
  store_heads(P, sp.t * P.H + g * P.grp + h0, nh, h, gq, i0, bad, inv,
              [&](int k, int e) { return acc[k][e]; });
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct Plan {
  int kp, vp, nb, chunks;
  size_t o, ml, plan;  // bytes of the workspace's parts
};
Plan plan_of(const Geometry& g, int64_t nseq) {
  Plan p;
  p.kp = (g.hs + 63) / 64;
  p.vp = (g.vhs + 127) / 128;
  const int grp = g.H / g.kvh;
  p.nb = grp > 8 ? 2 : 1;
  p.chunks = (grp + 8 * p.nb - 1) / (8 * p.nb);
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  const size_t slots = 2 * (size_t)g.num_sms;
  p.o = up(slots * 8 * p.vp * p.nb * 512);
  p.ml = up(slots * 8 * p.nb * sizeof(float2));
  p.plan = up((size_t)(nseq + 1) * sizeof(int64_t));
  return p;
}

template <int KP, int VP, int NB>
cudaError_t launch(const Geometry& g, const QuantArgs& a, const DecP& A) {
  using S = Shape<KP, VP, NB>;
  static std::atomic<bool> configured[64];
  auto kern = quant_decode_kernel<KP, VP, NB>;
  cudaError_t e = once_per_device(configured, g.device, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  });
  if (e != cudaSuccess) return e;
  e = tc::launch_pdl(kern, dim3((unsigned)g.num_sms), dim3(kThreads), S::kSmem, a.stream, A);
  if (e != cudaSuccess) return e;
  return tc::launch_pdl(quant_combine_kernel<VP, NB>, dim3((unsigned)(A.R.nseq * A.units)),
                        dim3(64 * VP * NB), 0, a.stream, A);
}

}  // namespace

size_t decode_workspace(const Geometry& g, int64_t nseq) {
  const Plan p = plan_of(g, nseq);
  return p.o + p.ml + p.plan;
}

cudaError_t launch_decode(const Geometry& g, const QuantArgs& a) {
  DecP A{};
  A.R = read_params(g, a);
  const Plan p = plan_of(g, A.R.nseq);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  A.ws_o = reinterpret_cast<float4*>(ws);
  A.ws_ml = reinterpret_cast<float2*>(ws + p.o);
  A.ws_plan = reinterpret_cast<int64_t*>(ws + p.o + p.ml);
  A.chunks = p.chunks;
  A.units = g.kvh * p.chunks;
  A.min_part = 2 * kWarps;
  if ((int64_t)A.R.nseq * A.units > INT32_MAX) return cudaErrorInvalidConfiguration;
  auto nb = [&](auto kp, auto vp) {
    return p.nb == 1 ? launch<kp(), vp(), 1>(g, a, A) : launch<kp(), vp(), 2>(g, a, A);
  };
  auto vp = [&](auto kp) {
    return p.vp == 1 ? nb(kp, std::integral_constant<int, 1>()) : nb(kp, std::integral_constant<int, 2>());
  };
  switch (p.kp) {
    case 1: return vp(std::integral_constant<int, 1>());
    case 2: return vp(std::integral_constant<int, 2>());
    case 3: return vp(std::integral_constant<int, 3>());
    default: return vp(std::integral_constant<int, 4>());
  }
}

}  // namespace quant
}  // namespace pa
