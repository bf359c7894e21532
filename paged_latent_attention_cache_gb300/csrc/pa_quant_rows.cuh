// Attention over 8-bit caches for few query rows (include/pa_quant.h): decode, one new
// token per sequence, and prefill of a few tokens each. Bound by HBM where there is much to
// read: 32 sequences of 8192 to 65536 keys, 32 heads over 8 of 128 / 128, 422 us, 5.7 TB/s;
// of 1024 to 8192 66 us, 4.6 TB/s, some 15 us of which are the plan, the first copies and
// the joining of parts; 32 of 90 to 1500, 16 heads of 64, 29 us, 1.8 TB/s.
//
// The line. A unit is a sequence, a kv head and up to 8 NB of its query rows (token x
// head of the group); its visible keys are cut into tiles of 16 TH. All tiles of all units
// form one line, every unit's behind `extra` that stand for the time that the unit takes
// by itself. The line is cut into equal parts, one per CTA, whatever the lengths. A
// CTA's part of a unit is a segment: its warps take the segment's tiles in turn, each
// with a softmax of its own, and join at the segment's end. A unit that lies in several
// parts is joined by quant_combine_kernel.
//
// Loads. Each warp has a ring of its own, D tiles deep and kept full past the ends of
// segments: 16 rows of 128 codes per TMA box, one lane issues them once the warp has read
// the tile that was there, so a warp waits for nothing but its own copies. A tile's pages
// are looked up a batch of 32 tiles before. (cp.async, 16 bytes a lane, stopped at 4.6
// TB/s with 8, 12 and 16 warps an SM alike.)
//
// Products. mma.sync m16n8k16, keys (then value channels) as the 16 rows and the query
// rows as the 8 columns: the other way round a group of eight or fewer would fill half
// of a product. The order of the 16 keys and of the channels inside the products is
// chosen so that 16 bytes that a lane loads are registers of A as they are, without bank
// conflicts in the boxes' 128-byte swizzle: lane (g, t) = (lane / 4, lane % 4) takes
//   of key slot g and g + 8 (keys kappa = g / 2 + 4 (g % 2), and + 8): pieces of 16
//     channels t, t + 4, ..; a word of 4 codes is one k step's A registers
//   of the values of keys t, t + 4, t + 8, t + 12: piece g / 2 + 4 (g % 2) (and + 8); a
//     byte of each of two words is a register.
// E4M3 is exact in fp16; P^T becomes the B operand by movmatrix.
//
// (A header, so that pa_quant_decode.cu and pa_quant_decode_two.cu, the queries in one
// and in two addends, compile side by side.)
#pragma once

#include <type_traits>

#include "pa_diff_common.cuh"
#include "pa_quant_read.cuh"

namespace pa {
namespace quant {
namespace rows {

constexpr int kWarps = 4, kThreads = kWarps * 32;

struct DecP {
  ReadP R;
  float4* ws_o;      // [2 CTAs][8 VP NB][32] accumulators as the lanes hold them
  float2* ws_ml;     // [2 CTAs][8 NB] maximum (log2 domain), sum
  int64_t* ws_line;  // [nseq + 1] length of the line before each sequence, then that of a part
  int32_t* ws_units; // [nseq + 1] units before each sequence, then all
  int decode;        // one token per sequence, others are told
  int few;           // otherwise: sequences of more tokens are another kernel's
  int rows;          // 8 NB
  int tile;          // keys: 16 TH
  int box;           // rows of a copy: min(bs, tile)
  int min_part;
  int extra;         // what a unit counts on the line beside its tiles
};

struct Span {  // a sequence's tokens and the tiles that they see
  int64_t pos, hi, lo, t;  // position of the first token, last and first key, first token
  int q, tiles, first;     // tokens, tiles, first tile
  int chunks;              // units per kv head
  int err;                 // PA_DEVERR_* that keeps it from being read, or 0
  bool rows;               // it has rows of out
};
__device__ __forceinline__ Span span_of(const DecP& A, int b) {
  const ReadP& P = A.R;
  const int64_t c0 = P.cumseq[P.seq_begin + b], c1 = P.cumseq[P.seq_begin + b + 1];
  const int64_t past = P.past[P.seq_begin + b], q = c1 - c0;
  Span s;
  s.t = c0;
  s.q = (int)max((int64_t)0, q);
  s.pos = past;
  s.hi = P.cross ? past - 1 : past + q - 1;
  s.lo = P.window >= 0 ? max((int64_t)0, past - P.window) : 0;
  const bool mine = A.decode || q <= A.few;
  s.rows = mine && q > 0 && c0 >= 0 && c1 <= P.num_tokens && (q == 1 || !A.decode);
  s.err = !mine                                                  ? 0
          : A.decode && q != 1                                     ? PA_DEVERR_DECODE_QLEN
          : q < 0 || (q > 0 && !s.rows)                          ? PA_DEVERR_CUMSEQ
          : q > 0 && (past < 0 || s.hi >= (int64_t)P.max_blocks * P.bs) ? PA_DEVERR_CONTEXT
          : q > 0 && P.rd > 0 && s.hi >= P.cos_rows              ? PA_DEVERR_POSITION
                                                                 : 0;
  s.first = (int)(s.lo / A.tile);
  s.tiles = !mine || s.err || q <= 0 || s.hi < s.lo ? 0 : (int)(s.hi / A.tile) - s.first + 1;
  s.chunks = s.tiles ? (s.q * P.grp + A.rows - 1) / A.rows : 0;
  return s;
}

// A walk over the line: the segment that starts at tile x of the line, its unit,
// and the line's end for this CTA.
struct Walk {
  int64_t x, end, start;  // (start: of sequence b)
  int b, tiles, first, chunks;
  int g, chunk;           // the segment's unit
  int step;               // its length on the line
  int from, len;          // first tile (in the cache), tiles (0: the part ended before them)
  int lo, hi;             // keys that any of its tokens sees
  __device__ __forceinline__ bool valid() const { return x < end; }
  __device__ __forceinline__ void enter(const DecP& A, int seq, int64_t at) {
    const Span s = span_of(A, seq);
    b = seq;
    start = at;
    tiles = s.tiles;
    first = s.first;
    chunks = s.chunks;
    lo = (int)s.lo;
    hi = (int)s.hi;
  }
  __device__ __forceinline__ void segment(const DecP& A) {
    const uint64_t off = (uint64_t)(x - start);
    const uint32_t all = tiles + A.extra;
    const int unit = off >> 32 ? (int)(off / all) : (int)((uint32_t)off / all);
    const int in = (int)(off - (uint64_t)unit * all);
    g = unit / chunks;
    chunk = unit - g * chunks;
    step = (int)min((int64_t)(all - in), end - x);
    const int t0 = max(0, in - A.extra);
    from = first + t0;
    len = max(0, in + step - A.extra) - t0;
  }
  __device__ __forceinline__ void next(const DecP& A) {
    x += step;
    if (!valid()) return;
    if (x == start + (int64_t)(tiles + A.extra) * A.R.kvh * chunks) {
      int seq = b;
      do enter(A, ++seq, x);
      while (tiles == 0);
    }
    segment(A);
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
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Accumulators i0..i0 + 3 of a block of query rows (see the products): eight channels
// of rows r and r + 1 of the unit, times inv, to out. piece: the lane's (of 16 channels).
template <typename F>
__device__ __forceinline__ void store_rows(const ReadP& P, const Span& sp, int g, int r0, int nr,
                                           int r, int piece, int i0, bool zero, const float (&inv)[2],
                                           F&& acc) {
  const int ch = 16 * (piece + (i0 & ~7)) + 2 * (i0 & 7);
  if (ch >= P.vhs) return;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (r + e >= nr) continue;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = zero ? 0 : pack_out(P, acc(k, e) * inv[e], acc(k, e + 2) * inv[e]);
    const int tok = (r0 + r + e) / P.grp, h = g * P.grp + (r0 + r + e) - tok * P.grp;
    *reinterpret_cast<uint4*>(reinterpret_cast<__half*>(P.out) +
                              ((sp.t + tok) * P.H + h) * P.vhs + ch) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 1 / sum of row r of a unit, whose maximum is m, with its head's sink. (A row that
// saw nothing, m -inf and sum 0, answers zeros: 0 times 1.)
__device__ __forceinline__ float inverse(const ReadP& P, int g, int r0, int r, int nr, float m,
                                         float sum) {
  if (m == -INFINITY && sum == 0.f) return 1.f;
  if (P.head_sink && r < nr)
    sum += ex2(to_f32(P, P.head_sink, g * P.grp + (r0 + r) % P.grp) * kLog2e - m + kShift);
  return 1.f / sum;
}

// CTAs per SM and the shared memory of one: rings, query, joining buffers. Twelve
// warps an SM where the registers allow it: with eight (one CTA of 255 registers a
// thread) 32 sequences of 1024 to 8192 keys (32 heads over 8, 128 / 128) took 104 us where
// twelve took 90. With values above 128 channels and 16 rows a unit a thread's 255 registers do not
// hold everything, and up to 96 bytes of it go by local memory; 32 sequences of 1024 to 8192 keys:
// 64 heads over 4 of 128 / 256 70 us in bf16, 78 in fp16 (3.2, 2.9 TB/s; with 128 / 128 none spill but
// fp16's 8 rows, 8 bytes), five tokens each of 32 heads over 8 192 and 214.
template <int KP, int VP, int NB, int TH, bool LO>
struct Shape {
  static constexpr int kCtas = TH == 2 && NB == 1 ? 3 : 2;
  static constexpr int kBox = TH * 16 * 128;              // a tile's keys of 128 codes
  static constexpr int kKeys = (KP + 1) / 2 * kBox;       // of a warp's tile
  static constexpr int kStage = kKeys + VP * kBox;
  static constexpr int kRow = KP * 64 + 8;                // halves of a query row
  static constexpr int kAcc = 8 * VP * NB;                // float4 accumulators of a lane
  static constexpr int kQ = 8 * NB * kRow * 2 * (LO ? 2 : 1);
  static constexpr int kJoin = (kWarps / 2) * (kAcc * 512 + NB * 64);
  static constexpr int kBoth = kQ > kJoin ? kQ : kJoin;   // one after the other
  static constexpr int kLeft = 228 * 1024 / kCtas - 1024 - 320 - 1024 - kBoth;
  static constexpr int kFit = kLeft / (kWarps * (kStage + 24));
  static constexpr int D = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = 1024 + kWarps * D * (kStage + 24) + kBoth;
  static_assert(D >= 2, "ring");
};

// LO: the query in two addends (two_addends in pa_quant_read.cuh)
template <int KP, int VP, int NB, int TH, bool LO>
__global__ void __launch_bounds__(kThreads, Shape<KP, VP, NB, TH, LO>::kCtas)
quant_rows_kernel(const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ DecP A) {
  using S = Shape<KP, VP, NB, TH, LO>;
  constexpr int D = S::D, R = 8 * NB, kTile = 16 * TH;
  const ReadP& P = A.R;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kWarps * D * S::kStage);  // [warp][D]
  float4* meta = reinterpret_cast<float4*>(full + kWarps * D);                  // [warp][D]
  __half* s_q = reinterpret_cast<__half*>(meta + kWarps * D);
  float4* join_o = reinterpret_cast<float4*>(s_q);
  float2* join_ml = reinterpret_cast<float2*>(join_o + (kWarps / 2) * S::kAcc * 32);
  __shared__ float s_mult[R];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int s_scan_u[kWarps];
  __shared__ int64_t s_hit[2];  // sequence of this CTA's first tile, tiles before it
  __shared__ int s_bad, s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;

  const int piece = (gq >> 1) + 4 * (gq & 1);  // of values; kappa as well
  volatile int* abort = &s_abort;
  uint64_t* my_full = full + warp * D;
  if (lane < D) tc::mbar_init(smem_u32(my_full + lane), 1);
  tc::fence_barrier_init();
  if (tid == 0) s_abort = 0;
  if (!P.early) grid_dep_wait();

  // ---- the plan: tiles and units before each sequence (prefix sums, 128 sequences a
  // round)
  int64_t carry = 0, my_start = 0, mine = 0;
  int carry_u = 0;
  auto round = [&](int base) {  // start of sequence base + tid, and the carry behind the round
    const int b = base + tid;
    int units = 0;
    mine = 0;
    if (b < P.nseq) {
      const Span s = span_of(A, b);
      units = s.chunks * P.kvh;
      mine = (int64_t)(s.tiles + A.extra) * units;
    }
    int64_t v = mine;
    int w = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      const int z = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) {
        v += y;
        w += z;
      }
    }
    __syncthreads();
    if (lane == 31) {
      s_scan[warp] = v;
      s_scan_u[warp] = w;
    }
    __syncthreads();
    int64_t before = carry;
    int before_u = carry_u;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) {
        before += s_scan[i];
        before_u += s_scan_u[i];
      }
      carry += s_scan[i];
      carry_u += s_scan_u[i];
    }
    my_start = before + v - mine;
    if (blockIdx.x == 0 && b < P.nseq) {
      A.ws_line[b] = my_start;
      A.ws_units[b] = before_u + w - units;
    }
  };
#pragma unroll 1
  for (int base = 0; base < P.nseq; base += kThreads) round(base);
  const int64_t total = carry;
  const int64_t part = max((int64_t)A.min_part, (total + gridDim.x - 1) / gridDim.x);
  if (blockIdx.x == 0 && tid == 0) {
    A.ws_line[P.nseq] = part;
    A.ws_units[P.nseq] = carry_u;
  }
  Walk W;
  W.x = min(total, blockIdx.x * part);
  W.end = min(total, W.x + part);
#pragma unroll 1
  for (int base = 0; base < P.nseq && W.x < W.end; base += kThreads) {
    if (P.nseq > kThreads) {
      if (base == 0) carry = carry_u = 0;
      round(base);
    }
    if (mine > 0 && my_start <= W.x && W.x < my_start + mine) {
      s_hit[0] = base + tid;
      s_hit[1] = my_start;
    }
  }
  __syncthreads();
  if (W.valid()) {
    W.enter(A, (int)s_hit[0], s_hit[1]);
    W.segment(A);
  }
  if (P.early) grid_dep_wait();

  // ---- this warp's copies: a walk of its own ahead of the products
  Walk C = W;
  int ct = 0, own = 0;          // next tile of its segment (counting the warp's own), all of them
  int page0 = 0, page1 = 0;     // of this batch's and the next batch's tiles, a lane each
  float2 sc0 = make_float2(0.f, 0.f), sc1 = sc0;
  const int kappa = piece;
  uint8_t* my_ring = ring + warp * D * S::kStage;
  const int none = P.num_blocks << P.sh;  // (zeros arrive from behind the last slot)
  // A lane of a batch: half lane % nbox of the warp's tile lane / nbox (a tile lies in a
  // page, or in two of 16 rows).
  const int nbox = TH == 2 ? kTile / A.box : 1, batch = 32 / nbox;
  auto look_up = [&](int k) {  // its page behind the warp's tile k; -1 invalid, -2 not needed
    const int t = k + (nbox == 2 ? lane >> 1 : lane);
    const int64_t key = (int64_t)(C.from + warp + t * kWarps) * kTile + (nbox == 2 ? (lane & 1) * 16 : 0);
    if (t >= own || key > C.hi || key + A.box - 1 < C.lo) return -2;
    const int page = P.block_table[(int64_t)(P.seq_begin + C.b) * P.max_blocks + (key >> P.sh)];
    return page >= 0 && page < P.num_blocks ? page : -1;
  };
  auto scale_at = [&](int page) {
    return page >= 0 ? P.scales[(int64_t)page * P.kvh + C.g] : make_float2(0.f, 0.f);
  };
  auto begin = [&]() {  // the first segment from here on with a tile of this warp
    own = 0;
    while (C.valid()) {
      own = C.len > warp ? (C.len - warp + kWarps - 1) / kWarps : 0;
      if (own) break;
      C.next(A);
    }
    ct = 0;
    if (C.valid()) {
      page0 = look_up(0);
      sc0 = scale_at(page0);
    }
  };
  int put = 0, issued = 0, taken = 0;
  auto produce = [&]() {
    if (C.valid()) {
      const int k = ct & (batch - 1);
      if (k == batch / 4) page1 = look_up((ct & ~(batch - 1)) + batch);
      if (k == batch / 2) sc1 = scale_at(page1);
      const int tile = C.from + warp + ct * kWarps;
      const uint32_t dst = smem_u32(my_ring + put * S::kStage), bar = smem_u32(my_full + put);
      float4 mt;
#pragma unroll
      for (int h = 0; h < TH; ++h) {
        if (h < nbox) {
          const int from = k * nbox + h;
          const int page = __shfl_sync(0xffffffffu, page0, from);
          const float ks = __shfl_sync(0xffffffffu, sc0.x, from);
          const float vs = __shfl_sync(0xffffffffu, sc0.y, from);
          const int ve = scale_exponent(vs);
          const bool kin = page >= 0 && scale_exponent(ks) != kNone, vin = page >= 0 && ve != kNone;
          const int row = (page << P.sh) + ((tile * kTile + h * 16) & (P.bs - 1));
          (h ? mt.z : mt.x) = page != -1 ? (kin ? ks : 1.f) : NAN;
          (h ? mt.w : mt.y) = vin ? (float)ve : kLeast;
          if (diff::elect_one()) {
            if (h == 0) tc::mbar_expect_tx(bar, S::kStage);
#pragma unroll
            for (int i = 0; i < (KP + 1) / 2; ++i)
              tc::tma_load_3d(dst + i * S::kBox + h * 2048, &kmap, i * 128, C.g, kin ? row : none, bar);
#pragma unroll
            for (int i = 0; i < VP; ++i)
              tc::tma_load_3d(dst + S::kKeys + i * S::kBox + h * 2048, &vmap, i * 128, C.g,
                              vin ? row : none, bar);
          }
        } else {
          mt.z = mt.x;
          mt.w = mt.y;
        }
      }
      if (lane == 0) meta[warp * D + put] = mt;
      __syncwarp();
      ++issued;
      if (++ct == own) {
        C.next(A);
        begin();
      } else if ((ct & (batch - 1)) == 0) {
        page0 = page1;
        sc0 = sc1;
      }
    }
    if (++put == D) put = 0;
  };
  begin();
#pragma unroll 1
  for (int i = 0; i < D; ++i) produce();
  int get = 0;
  uint32_t turn = 0;

  // ---- segments
#pragma unroll 1
  while (W.valid()) {
    if (W.len == 0) {
      W.next(A);
      continue;
    }
    const int r0 = W.chunk * R;
    const Span sp = span_of(A, W.b);
    const int nr = min(R, sp.q * P.grp - r0);
    __syncthreads();
    if (tid == 0) s_bad = 0;
    for (int r = warp; r < R; r += kWarps) {
      float x[8], back = 0.f;
      uint4 h = make_uint4(0, 0, 0, 0), rest = h;
      if (r < nr) {
        const int tok = (r0 + r) / P.grp, head = W.g * P.grp + (r0 + r) - tok * P.grp;
        const int64_t i = (sp.t + tok) * P.H + head;
        if (P.bf16) query_row8<__nv_bfloat16>(P, i, sp.pos + tok, x);
        else query_row8<__half>(P, i, sp.pos + tok, x);
        back = scaled_row8(x, &h, &rest);
      }
      if (lane * 8 < KP * 64) {
        *reinterpret_cast<uint4*>(s_q + r * S::kRow + lane * 8) = h;
        if (LO) *reinterpret_cast<uint4*>(s_q + (R + r) * S::kRow + lane * 8) = rest;
      }
      if (lane == 0) s_mult[r] = back * (P.cap_in > 0.f ? P.cap_in : P.scale_log2);
    }
    __syncthreads();
    constexpr bool kKeep = KP * NB <= 4;  // the query's fragments in registers
    uint32_t bq[kKeep ? NB : 1][kKeep ? KP : 1][8];
    auto q_frag = [&](int nb, int i, uint32_t (&f)[8]) {
      const uint32_t at = smem_u32(s_q + (nb * 8 + gq) * S::kRow + 16 * (tq + 4 * i));  // nb >= NB: rest
      const uint4 u = lds128(at), v = lds128(at + 16);
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
    // keys that all rows of the unit see, counted from the segment's first
    const int64_t key0 = (int64_t)W.from * kTile;
    const int tok_lo = r0 / P.grp, tok_hi = (r0 + nr - 1) / P.grp;
    const int all_hi = (int)((P.cross ? sp.hi : sp.pos + tok_lo) - key0);
    const int all_lo = (int)((P.window >= 0 ? max((int64_t)0, sp.pos + tok_hi - P.window) : 0) - key0);

    bool bad = false;
#pragma unroll 1
    for (int tile = warp; tile < W.len; tile += kWarps) {
      if (!__all_sync(0xffffffffu,
                      tc::wait_bar(smem_u32(my_full + get), turn, abort, P.err_flags)))
        break;  // (told; the warp's part stays as it is, and nothing more is copied)
      const uint32_t keys = smem_u32(my_ring) + get * S::kStage, values = keys + S::kKeys;
      const uint4 mw = lds128(smem_u32(meta + warp * D + get));
      const float ks[2] = {__uint_as_float(mw.x), __uint_as_float(mw.z)};
      const float ev[2] = {__uint_as_float(mw.y), __uint_as_float(mw.w)};
      ++taken;
      if (++get == D) {
        get = 0;
        turn ^= 1;
      }
      auto value = [&](int i, int h, int j) {  // of key 16 h + t + 4 j
        return values + i * S::kBox + h * 2048 + (tq + 4 * j) * 128 +
               ((piece ^ (tq + 4 * (j & 1))) << 4);
      };
      float c[TH][NB][4];
#pragma unroll
      for (int h = 0; h < TH; ++h) {
        bad |= isnan(ks[h]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[h][nb][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < KP; ++i) {
        const uint32_t at = keys + (i >> 1) * S::kBox + kappa * 128 +
                            (((tq + 4 * (i & 1)) ^ (kappa & 7)) << 4);
        uint4 u0[TH], u1[TH];
#pragma unroll
        for (int h = 0; h < TH; ++h) {
          u0[h] = lds128(at + h * 2048);
          u1[h] = lds128(at + h * 2048 + 8 * 128);
        }
        uint32_t f[NB][8], fr[LO ? NB : 1][8];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if constexpr (LO) q_frag(NB + nb, i, fr[nb]);
          if constexpr (kKeep) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[nb][e] = bq[nb][i][e];
          } else {
            q_frag(nb, i, f[nb]);
          }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int h = 0; h < TH; ++h) {
            uint32_t a0, a1, a2, a3;
            codes4(word(u0[h], s), &a0, &a2);
            codes4(word(u1[h], s), &a1, &a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              mma(c[h][nb], a0, a1, a2, a3, f[nb][2 * s], f[nb][2 * s + 1]);
              if constexpr (LO) mma(c[h][nb], a0, a1, a2, a3, fr[nb][2 * s], fr[nb][2 * s + 1]);
            }
          }
      }
      // scores of keys 16 h + kappa (c[0], c[1]) and + 8 for rows 2 t and 2 t + 1
      const int j0 = tile * kTile;
      auto scale_scores = [&](auto cap, auto wide) {
#pragma unroll
        for (int h = 0; h < TH; ++h)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float f = ks[h] * mult[nb][e & 1];
              c[h][nb][e] = cap() ? capped<wide()>(P, c[h][nb][e] * f) + ev[h]
                                  : fmaf(c[h][nb][e], f, ev[h]);
            }
      };
      if (P.cap_in <= 0.f) scale_scores(std::false_type(), std::false_type());
      else if (!P.cap_wide) scale_scores(std::true_type(), std::false_type());
      else scale_scores(std::true_type(), std::true_type());
      if (j0 < all_lo || j0 + kTile - 1 > all_hi) {
        // an end of what the rows see: unseen values become zeros (0 times NaN is NaN),
        // and a NaN among values that only some rows see goes over to their scores
        const int hi = (int)(sp.hi - key0), lo = (int)(sp.lo - key0);
        uint32_t odd = 0;
#pragma unroll 1
        for (int j = 0; j < 4 * TH; ++j) {
          const int key = tq + 4 * j;
          const bool unseen = j0 + key < lo || j0 + key > hi;
#pragma unroll
          for (int i = 0; i < VP; ++i) {
            const uint32_t at = value(i, j >> 2, j & 3);
            const uint4 v = lds128(at);
            const bool nan = nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w);
            if (unseen || nan) sts128(at, 0, 0, 0, 0);
            if (nan && !unseen) odd |= 1u << key;
          }
        }
        tc::fence_proxy_async();  // (a copy is the next to write there)
        odd = __reduce_or_sync(0xffffffffu, odd);
#pragma unroll
        for (int h = 0; h < TH; ++h)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = 16 * h + kappa + 4 * (e & 2);
              const int tok = (r0 + nb * 8 + 2 * tq + (e & 1)) / P.grp;
              const int64_t pos = sp.pos + tok - key0;
              if (odd >> key & 1u) c[h][nb][e] = NAN;
              if (j0 + key > (P.cross ? (int64_t)hi : pos) ||
                  (P.window >= 0 && pos - (j0 + key) > P.window))
                c[h][nb][e] = -INFINITY;
            }
      }
      float top[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[nb][e] = fmaxf(c[0][nb][e], c[0][nb][e + 2]);
          if (TH == 2) top[nb][e] = fmaxf(top[nb][e], fmaxf(c[TH - 1][nb][e], c[TH - 1][nb][e + 2]));
        }
      bool rise = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) rise |= top[nb][e] > m[nb][e] + kLazy;
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = top[nb][e];
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
      uint32_t pb[TH][NB][2];
#pragma unroll
      for (int h = 0; h < TH; ++h) {
        const float out_of = pow2(-(int)ev[h]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mm = m[nb][e & 1];
            p[e] = ex2(c[h][nb][e] - ((mm == -INFINITY ? 0.f : mm) - kShift));
          }
          l[nb][0] = fmaf(p[0] + p[2], out_of, l[nb][0]);
          l[nb][1] = fmaf(p[1] + p[3], out_of, l[nb][1]);
          pb[h][nb][0] = transposed(tc::pack2<__half>(p[0], p[1]));
          pb[h][nb][1] = transposed(tc::pack2<__half>(p[2], p[3]));
        }
      }
#pragma unroll
      for (int i = 0; i < VP; ++i)
#pragma unroll
        for (int h = 0; h < TH; ++h) {
          uint4 v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = lds128(value(i, h, j));
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint32_t w0 = word(v[0], s), w1 = word(v[1], s), w2 = word(v[2], s), w3 = word(v[3], s);
            uint32_t a0, a1, a2, a3;
            codes4(__byte_perm(w0, w1, 0x5140), &a0, &a1);
            codes4(__byte_perm(w2, w3, 0x5140), &a2, &a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma(acc[i * 8 + 2 * s][nb], a0, a1, a2, a3, pb[h][nb][0], pb[h][nb][1]);
            codes4(__byte_perm(w0, w1, 0x7362), &a0, &a1);
            codes4(__byte_perm(w2, w3, 0x7362), &a2, &a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma(acc[i * 8 + 2 * s + 1][nb], a0, a1, a2, a3, pb[h][nb][0], pb[h][nb][1]);
          }
        }
      __syncwarp();  // (the tile is read)
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
      __syncthreads();  // the query, or the buffers, are read
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
              join_ml[(warp - n) * R + nb * 8 + 2 * tq + e] = make_float2(m[nb][e], l[nb][e]);
        }
      }
      __syncthreads();
      if (warp < n) {
        float fa[NB][2], fb[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 o = join_ml[warp * R + nb * 8 + 2 * tq + e];
            const float t = fmaxf(m[nb][e], o.x), base = t == -INFINITY ? 0.f : t;
            fa[nb][e] = ex2(m[nb][e] - base);
            fb[nb][e] = ex2(o.x - base);
            // (a row of NaN scores keeps maximum -inf: its sum has to stay NaN)
            l[nb][e] = l[nb][e] * fa[nb][e] + o.y * fb[nb][e];
            m[nb][e] = t;
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
      const bool any_bad = s_bad != 0 || *abort;
      if (s_bad && lane == 0) raise_flag(P.err_flags, PA_DEVERR_BLOCK);
      if (W.len == W.tiles) {  // the whole unit
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float inv[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            inv[e] = inverse(P, W.g, r0, nb * 8 + 2 * tq + e, nr, m[nb][e], l[nb][e]);
#pragma unroll
          for (int i = 0; i < 8 * VP; i += 4)
            store_rows(P, sp, W.g, r0, nr, nb * 8 + 2 * tq, piece, i, any_bad, inv,
                       [&](int k, int e) { return acc[i + k][nb][e]; });
        }
      } else {
        // the first segment of this CTA's part, or one behind another's end
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
              A.ws_ml[slot * R + nb * 8 + 2 * tq + e] =
                  make_float2(any_bad ? NAN : m[nb][e], l[nb][e]);
        }
      }
    }
    W.next(A);
  }
  if (*abort && lane == 0)  // copies may be in flight
    for (int i = taken; i < issued; ++i)
      tc::drain_wait(smem_u32(my_full + i % D), (i / D) & 1, P.err_flags);
  __syncwarp();
  grid_dep_launch();
  // sequences without tiles: told, and zeros
  for (int b = blockIdx.x; b < P.nseq; b += gridDim.x) {
    const Span s = span_of(A, b);
    if (s.err && tid == 0) raise_flag(P.err_flags, s.err);
    if (s.tiles == 0 && s.rows) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(P.out) + s.t * P.H * P.vhs / 2;
      const int64_t n = (int64_t)s.q * P.H * P.vhs / 2;
      for (int64_t i = tid; i < n; i += kThreads) dst[i] = 0;
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <int KP, int VP, int NB, int TH, bool LO>
cudaError_t launch_one(const Geometry& g, const QuantArgs& a, const DecP& A) {
  using S = Shape<KP, VP, NB, TH, LO>;
  static std::atomic<bool> configured[64];
  auto kern = quant_rows_kernel<KP, VP, NB, TH, LO>;
  cudaError_t e = once_per_device(configured, g.device, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap kmap, vmap;
  if ((e = codes_map(&kmap, a.key_cache, g, g.hs, 128, A.box)) != cudaSuccess) return e;
  if ((e = codes_map(&vmap, a.value_cache, g, g.vhs, 128, A.box)) != cudaSuccess) return e;
  return tc::launch_pdl(kern, dim3((unsigned)(g.num_sms * S::kCtas)), dim3(kThreads), S::kSmem,
                        a.stream, kmap, vmap, A);
}

// The kernel for head sizes up to 64 kp and 128 vp and 8 nb rows a unit; tiles of 32 keys
// where a ring of them fits (the long sequences above 422 us, with tiles of 16 and two CTAs an SM
// 441; 32 of 90 to 1500 keys, 16 heads of 64, 29 and 39), or else of 16.
template <bool LO>
cudaError_t launch_rows_kernel(const Geometry& g, const QuantArgs& a, const DecP& A, int kp, int vp,
                               int nb) {
  auto of = [&](auto KP, auto VP) {
    constexpr int TH = KP() <= 2 && VP() == 1 ? 2 : 1;
    return nb == 1 ? launch_one<KP(), VP(), 1, TH, LO>(g, a, A)
                   : launch_one<KP(), VP(), 2, TH, LO>(g, a, A);
  };
  auto keys = [&](auto KP) {
    return vp == 1 ? of(KP, std::integral_constant<int, 1>()) : of(KP, std::integral_constant<int, 2>());
  };
  switch (kp) {
    case 1: return keys(std::integral_constant<int, 1>());
    case 2: return keys(std::integral_constant<int, 2>());
    case 3: return keys(std::integral_constant<int, 3>());
    default: return keys(std::integral_constant<int, 4>());
  }
}
extern template cudaError_t launch_rows_kernel<true>(const Geometry&, const QuantArgs&, const DecP&,
                                                     int, int, int);

}  // namespace rows
}  // namespace quant
}  // namespace pa
