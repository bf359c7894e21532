// Device helpers shared by the kernels over 8-bit caches.
#pragma once

#include <cuda_fp8.h>

#include "pa_common.cuh"

namespace pa {
namespace quant {

constexpr int kLeast = -48, kMost = 48;  // exponents of the scales

// The exponent of a scale, or kNone where a page has none.
constexpr int kNone = -127;
__device__ __forceinline__ int scale_exponent(float s) {
  const uint32_t u = __float_as_uint(s);
  const int e = (int)(u >> 23) - 127;  // (a negative number or NaN: out of range)
  return (u & 0x807fffffu) == 0 && e >= kLeast && e <= kMost ? e : kNone;
}
__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// The least e in range with amax <= 448 * 2^e (amax finite, >= 0): amax = m 2^k
// with 1 <= m < 2, and 448 = 1.75 * 2^8.
__device__ __forceinline__ int needed_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(kLeast, min(kMost, e));
}

// Two values as E4M3 codes (low byte first), saturated, ties to even.
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Two codes (low byte first) as f32.
__device__ __forceinline__ float2 decode2(uint32_t two) {
  return __half22float2(
      __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3)));
}
// Four codes times a power of two f <= 1, rounded to codes again.
__device__ __forceinline__ uint32_t shrink4(uint32_t w, float f) {
  const float2 a = decode2(w), b = decode2(w >> 16);
  return encode2(a.x * f, a.y * f) | encode2(b.x * f, b.y * f) << 16;
}

// The sequence b with cumseq[b] <= t < cumseq[b + 1], by a warp: 32 offsets
// at a time. Returns -1 (in all lanes) where there is none.
__device__ __forceinline__ int find_sequence(const int32_t* cumseq, int num_seqs, int64_t t,
                                             int lane) {
  int lo = 0, hi = num_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
    const unsigned in = __ballot_sync(0xffffffffu, at < hi && (at == lo || cumseq[at] <= t));
    lo += (31 - __clz(in)) * step;
    hi = min(hi, lo + step);
  }
  return cumseq[lo] <= t && t < cumseq[lo + 1] ? lo : -1;
}

// Eight channels [d0, d0 + 8) of a row, held by lane d0 / 8 of a group of `lpr`
// lanes (a power of two), after RMSNorm with weight w (if given) and the rotation
// at position pos, in f32. Every lane of the warp comes here; a lane with d0 >=
// hs holds zeros, as do those of a group without a row (`row` false).
template <typename T>
__device__ __forceinline__ void norm_rotate8(float (&x)[8], bool row, int d0, int hs, int lpr,
                                             const T* __restrict__ w, float eps, int ro, int rd,
                                             int interleaved, const T* __restrict__ cos_cache,
                                             const T* __restrict__ sin_cache, int64_t pos) {
  const int lane = threadIdx.x & 31;
  if (w) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    for (int o = lpr >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = 1.0f / sqrtf(ss / (float)hs + eps);
    if (d0 < hs) {
      float v[8];
      unpack8<T>(*reinterpret_cast<const uint4*>(w + d0), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * r * v[e];
    }
  }
  if (rd > 0) {
    const bool rot = row && d0 >= ro && d0 < ro + rd;
    const int half = rd >> 1;
    const int src = !rot || interleaved ? lane
                    : d0 - ro < half    ? lane + (half >> 3)
                                        : lane - (half >> 3);
    float xp[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) xp[e] = __shfl_sync(0xffffffffu, x[e], src & 31);
    if (rot)
      rope8<T>(x, xp, d0, ro, rd, interleaved, cos_cache + pos * half, sin_cache + pos * half);
  }
}

}  // namespace quant
}  // namespace pa
