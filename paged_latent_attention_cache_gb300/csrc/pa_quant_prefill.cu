// Attention over 8-bit caches (include/pa_quant.h): a warp per (token, head) (prefill).
#include <algorithm>

#include "pa_quant_common.cuh"
#include "pa_quant_internal.h"

namespace pa {
namespace quant {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct PlainArgs {
  QuantArgs a;
  int H, kvh, hs, vhs, ro, rd, interleaved, cos_rows, bs, num_blocks, max_blocks, window, decode;
  float scale, softcap, eps;
};

template <typename T>
__global__ void __launch_bounds__(256) quant_plain_kernel(const __grid_constant__ PlainArgs P) {
  asm volatile("griddepcontrol.wait;\n griddepcontrol.launch_dependents;" ::: "memory");
  const QuantArgs& a = P.a;
  const int lane = threadIdx.x & 31, sh = __ffs(P.bs) - 1;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  __shared__ float s_q[8][256];
  float* sq = s_q[threadIdx.x >> 5];
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
       i < a.num_tokens * P.H; i += warps) {
    const int64_t t = i / P.H;
    const int h = (int)(i - t * P.H), g = h / (P.H / P.kvh);
    const int b = find_sequence(a.cumseq, a.num_seqs, t, lane);
    if (b < 0) {
      if (lane == 0) raise_flag(a.err_flags, PA_DEVERR_CUMSEQ);
      continue;
    }
    if (b < a.seq_begin || b >= a.seq_end) continue;
    const int64_t c0 = a.cumseq[b], c1 = a.cumseq[b + 1], past = a.past[b];
    if (P.decode && c1 - c0 != 1) {
      if (lane == 0) raise_flag(a.err_flags, PA_DEVERR_DECODE_QLEN);
      continue;
    }
    T* out = reinterpret_cast<T*>(a.out) + i * P.vhs;
    const int64_t pos = past + (t - c0);
    const int64_t last = a.cross ? past - 1 : pos;
    const int64_t top = a.cross ? past - 1 : past + (c1 - c0) - 1;
    bool bad = false;
    if (past < 0 || top >= (int64_t)P.max_blocks * P.bs) {
      if (lane == 0) raise_flag(a.err_flags, PA_DEVERR_CONTEXT);
      bad = true;
    } else if (P.rd > 0 && top >= P.cos_rows) {
      if (lane == 0) raise_flag(a.err_flags, PA_DEVERR_POSITION);
      bad = true;
    }
    const int64_t lo = P.window >= 0 ? max((int64_t)0, last - P.window) : 0;
    float o[8], l = 0.f, m = -INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.f;
    if (!bad) {
      float x[8];
      const T* q = reinterpret_cast<const T*>(a.query) + i * P.hs + lane * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
      if (lane * 8 < P.hs) unpack8<T>(*reinterpret_cast<const uint4*>(q), x);
      norm_rotate8<T>(x, true, lane * 8, P.hs, 32, reinterpret_cast<const T*>(a.q_norm), P.eps, P.ro,
                      P.rd, P.interleaved, reinterpret_cast<const T*>(a.cos_cache),
                      reinterpret_cast<const T*>(a.sin_cache), pos);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) sq[lane * 8 + e] = x[e];
      __syncwarp();
      for (int64_t j = lo; j <= last; ++j) {
        const int32_t page = a.block_table[(int64_t)b * P.max_blocks + (j >> sh)];
        if (page < 0 || page >= P.num_blocks) {
          if (lane == 0) raise_flag(a.err_flags, PA_DEVERR_BLOCK);
          bad = true;
          break;
        }
        const int64_t row = ((int64_t)page * P.bs + (j & (P.bs - 1))) * P.kvh + g;
        const float2 sc = a.scales[(int64_t)page * P.kvh + g];
        const float ks = scale_exponent(sc.x) == kNone ? 0.f : sc.x;
        const float vs = scale_exponent(sc.y) == kNone ? 0.f : sc.y;
        float s = 0.f;
        for (int d = lane; d < P.hs; d += 32)
          s = fmaf(sq[d], decode2(a.key_cache[row * P.hs + d]).x, s);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        s *= ks * P.scale;
        if (P.softcap > 0.f) s = P.softcap * tanhf(s / P.softcap);
        const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = e * 32 + lane;
          if (d < P.vhs) o[e] = o[e] * f + p * vs * decode2(a.value_cache[row * P.vhs + d]).x;
        }
      }
      if (a.head_sink && m != -INFINITY) {
        const float z = Half<T>::to_f32(reinterpret_cast<const T*>(a.head_sink)[h]);
        l += expf(z - m);
      }
    }
    const float inv = bad || m == -INFINITY ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e * 32 + lane < P.vhs)
        out[e * 32 + lane] = Half<T>::from_f32(bad || m == -INFINITY ? 0.f : o[e] * inv);
  }
}

cudaError_t launch_plain(const Geometry& g, const QuantArgs& a, int decode) {
  const PlainArgs P{a, g.H, g.kvh, g.hs, g.vhs, g.ro, g.rd, g.interleaved, g.cos_rows, g.bs,
                    g.num_blocks, g.max_blocks, g.window, decode, g.scale, g.softcap, g.rms_eps};
  const int64_t blocks = std::min((a.num_tokens * g.H + 7) / 8, (int64_t)g.num_sms * 8);
  if (g.dtype == PA_DTYPE_BF16)
    quant_plain_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, a.stream>>>(P);
  else
    quant_plain_kernel<__half><<<(unsigned)blocks, 256, 0, a.stream>>>(P);
  return cudaGetLastError();
}

}  // namespace

size_t prefill_workspace(const Geometry&, int64_t, int64_t) { return 0; }
cudaError_t launch_prefill(const Geometry& g, const QuantArgs& a) { return launch_plain(g, a, 0); }

}  // namespace quant
}  // namespace pa
