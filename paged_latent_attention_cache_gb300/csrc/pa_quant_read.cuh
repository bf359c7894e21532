// What the read kernels over 8-bit caches share: parameters, the range of keys
// that a sequence's tokens see, warp products.
#pragma once

#include "pa_quant_common.cuh"
#include "pa_quant_internal.h"
#include "pa_tc_common.cuh"

namespace pa {
namespace quant {

using tc::ex2;
using tc::grid_dep_launch;
using tc::grid_dep_wait;
using tc::kLog2e;
using tc::smem_u32;
using tc::tanh_ex2;

// A probability times the scale of its value enters the product with the codes
// as fp16 2^(y - M + kShift): y = log2e s + e, s the score and 2^e the value's scale, M
// the row's running maximum of y, which may lag behind by kLazy (the power is
// below 2^(kShift + kLazy) = 2^15 then, fp16 ends at 2^16). So no value is scaled on
// its own, and what fp16 cuts off (2^-25) is 2^-33 of the row's largest product. The
// softmax's sum takes the scale out again, page by page, in f32: y - M >= -96 for
// the keys that carry the sum, scales being 2^-48..2^48.
constexpr float kLazy = 7.f, kShift = 8.f;

struct ReadP {
  const void* query;
  const uint8_t* key_cache;
  const uint8_t* value_cache;
  const float2* scales;
  const void* cos_cache;
  const void* sin_cache;
  const void* q_norm;
  const void* head_sink;
  const int32_t* cumseq;
  const int32_t* past;
  const int32_t* block_table;
  void* out;
  int32_t* err_flags;
  int64_t num_tokens;
  int seq_begin, nseq;
  int H, kvh, grp, hs, vhs, ro, rd, interleaved, cos_rows, bs, sh, num_blocks, max_blocks;
  int window, cross, bf16, early;
  int two;           // query rows as two fp16 addends (see scaled_row8)
  float scale_log2;  // scale * log2(e)
  float cap_in;      // scale / softcap, 0 without softcap
  float cap_out;     // softcap * log2(e)
  int cap_wide;      // softcap above kWideCap
  float eps;
};

// Whether query rows enter the products as two fp16 addends: where norm or rotation
// leave more than fp16 holds (a row as it came is exact) and the output is fp16 too. One
// rounding of the row moves a score by some 2^-12 of the scores' spread, more than all
// other roundings of an fp16 output together: over 5000 keys of N(0, 1) at 64 channels
// the output is 5.2e-4 off with it and 2.8e-4 without, 2.1e-4 of which its own rounding
// is. A bf16 output is rounded eight times as coarsely.
inline bool two_addends(const Geometry& g, const QuantArgs& a) {
  return g.dtype != PA_DTYPE_BF16 && (g.rd > 0 || a.q_norm);
}

// From 2^60 on a softcap moves no score by a place of its f32 value (by s^2 / (3 softcap^2) of
// it, scores below 2^48), and its reciprocal times the scales would leave f32's range.
// Above kWideCap its tanh goes by capped<true> (1e-7 of 128 is 1.3e-5 of a score, a twentieth of
// an fp16 output's rounding; up to it long prefill takes 1242 us, above 1905).
constexpr float kWideCap = 128.f;
inline float softcap_of(const Geometry& g) { return g.softcap < 0x1p60f ? g.softcap : 0.f; }

inline ReadP read_params(const Geometry& g, const QuantArgs& a) {
  ReadP P{};
  P.query = a.query;
  P.key_cache = a.key_cache;
  P.value_cache = a.value_cache;
  P.scales = a.scales;
  P.cos_cache = a.cos_cache;
  P.sin_cache = a.sin_cache;
  P.q_norm = a.q_norm;
  P.head_sink = a.head_sink;
  P.cumseq = a.cumseq;
  P.past = a.past;
  P.block_table = a.block_table;
  P.out = a.out;
  P.err_flags = a.err_flags;
  P.num_tokens = a.num_tokens;
  P.seq_begin = a.seq_begin;
  P.nseq = a.seq_end - a.seq_begin;
  P.H = g.H;
  P.kvh = g.kvh;
  P.grp = g.H / g.kvh;
  P.hs = g.hs;
  P.vhs = g.vhs;
  P.ro = g.ro;
  P.rd = g.rd;
  P.interleaved = g.interleaved;
  P.cos_rows = g.cos_rows;
  P.bs = g.bs;
  while ((1 << P.sh) < g.bs) ++P.sh;
  P.num_blocks = g.num_blocks;
  P.max_blocks = g.max_blocks;
  P.window = g.window;
  P.cross = a.cross;
  P.bf16 = g.dtype == PA_DTYPE_BF16;
  P.early = (g.flags & PA_FLAG_AFTER_WRITE) ? 1 : 0;
  P.two = two_addends(g, a);
  P.scale_log2 = g.scale * kLog2e;
  const float softcap = softcap_of(g);
  P.cap_in = softcap > 0.f ? g.scale / softcap : 0.f;
  P.cap_out = softcap * kLog2e;
  P.cap_wide = softcap > kWideCap;
  P.eps = g.rms_eps;
  return P;
}

// A cache as (channel, kv head, slot); boxes of `rows` slots of one head: all of its
// channels, or `swizzled` of them (128, swizzled; zeros behind the head's last).
inline cudaError_t codes_map(CUtensorMap* map, const void* base, const Geometry& g, int width,
                             int swizzled, int rows) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)g.kvh,
                              (cuuint64_t)g.num_blocks * g.bs};
  const cuuint64_t str[2] = {(cuuint64_t)width, (cuuint64_t)width * g.kvh};
  const cuuint32_t box[3] = {(cuuint32_t)(swizzled ? swizzled : width), 1, (cuuint32_t)rows};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, str, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// log2e times the softcapped score whose ratio to softcap is x. tanh_ex2 is some 1e-7 off
// whatever x is, and a softcap far above the scores magnifies that to more than they are: with
// WIDE, tanh's series below 1/4 (the next term is 1382 / 155925 x^10 < 9e-9 of the result).
template <bool WIDE>
__device__ __forceinline__ float capped(const ReadP& P, float x) {
  if (!WIDE) return P.cap_out * tanh_ex2(x);
  const float t = x * x;
  const float r = fmaf(fmaf(fmaf(62.f / 2835.f, t, -17.f / 315.f), t, 2.f / 15.f), t, -1.f / 3.f);
  return P.cap_out * (fabsf(x) < 0.25f ? fmaf(x * t, r, x) : tanh_ex2(x));
}

// Eight channels of a query row as fp16, the row times a power of two that
// brings its largest channel to [2^14, 2^15) (a row: `lpr` lanes, eight channels
// each), and what that rounding left, as fp16 again. Returns what takes the factor
// back. (A row of zeros, or one that is not finite, keeps factor 1.)
__device__ __forceinline__ float scaled_row8(const float (&x)[8], uint4* h, uint4* rest,
                                             int lpr = 32) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
  for (int o = lpr >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  int e = (int)(__float_as_uint(m) >> 23) - 127;  // m in [2^e, 2^(e + 1))
  if (m == 0.f || e == 128) e = 14;
  e = max(-112, e);  // (the factor ends at 2^126)
  const float f = pow2(14 - e);
  uint32_t w[4], v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i] * f, b = x[2 * i + 1] * f;
    w[i] = tc::pack2<__half>(a, b);
    const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    // (nothing is left of an infinity: its scores are decided)
    v[i] = tc::pack2<__half>(isinf(r.x) ? 0.f : a - r.x, isinf(r.y) ? 0.f : b - r.y);
  }
  *h = make_uint4(w[0], w[1], w[2], w[3]);
  *rest = make_uint4(v[0], v[1], v[2], v[3]);
  return pow2(e - 14);
}

// Channels [8 lane, 8 lane + 8) of the query row i (token * H + head) in f32, after
// norm and rotation (T: the dtype). The whole warp.
template <typename T>
__device__ __forceinline__ void query_row8(const ReadP& P, int64_t i, int64_t pos, float (&x)[8]) {
  const int d0 = (threadIdx.x & 31) * 8;
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.f;
  if (d0 < P.hs)
    unpack8<T>(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(P.query) + i * P.hs + d0),
               x);
  norm_rotate8<T>(x, true, d0, P.hs, 32, reinterpret_cast<const T*>(P.q_norm), P.eps, P.ro, P.rd,
                  P.interleaved, reinterpret_cast<const T*>(P.cos_cache),
                  reinterpret_cast<const T*>(P.sin_cache), pos);
}

__device__ __forceinline__ float to_f32(const ReadP& P, const void* p, int64_t i) {
  return P.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i])
                : __half2float(reinterpret_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ uint32_t pack_out(const ReadP& P, float a, float b) {
  return P.bf16 ? tc::pack2<__nv_bfloat16>(a, b) : tc::pack2<__half>(a, b);
}

// Shared memory by its address (pointers into an aligned region become generic loads,
// which take several times as long).
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Four codes' NaNs as 0x80 in their bytes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Four codes as two words of fp16.
__device__ __forceinline__ void codes4(uint32_t four, uint32_t* lo, uint32_t* hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
      " cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(*lo), "=r"(*hi)
      : "r"(four));
}

}  // namespace quant
}  // namespace pa
