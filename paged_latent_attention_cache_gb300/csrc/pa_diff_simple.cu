// Differential attention, the plain kernel: one CTA per (token, head) with
// both maps. A tile of 128 keys at a time: thread k computes the two scores
// of key k (the query in shared memory as f32), the CTA updates each map's
// running maximum and sum, and thread c adds the tile's values to channels
// c and c + 128 of both outputs. Right for every geometry; bound by its
// uncoalesced key reads.
#include <type_traits>

#include "pa_common.cuh"
#include "pa_diff_internal.h"

namespace pa {
namespace diff {
namespace {

constexpr int kTile = 128;

__device__ __forceinline__ float block_reduce(float v, bool is_max, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = is_max ? fmaxf(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = red[0];
  for (int i = 1; i < kTile / 32; ++i) r = is_max ? fmaxf(r, red[i]) : r + red[i];
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kTile)
diff_simple_kernel(Geometry g, DiffArgs a) {
  __shared__ float q[2][128], p[2][kTile], red[kTile / 32];
  __shared__ int32_t s_bad;
  const int tid = threadIdx.x, h = blockIdx.x % g.H;
  const int64_t unit = blockIdx.x / g.H;
  const int hs = g.hs, vhs = g.vhs, gk = h / (g.H / g.kvh);
  int64_t t = unit, pos = 0;
  int32_t b = 0;
  if (!locate_token(t, a.cumseq, a.past, a.num_seqs, tid == 0 ? a.err_flags : nullptr, &b, &pos))
    return;
  if (b < a.seq_begin || b >= a.seq_end) return;
  T* out = (T*)a.out + (t * g.H + h) * (int64_t)vhs;
  const bool bad_ctx = a.past[b] < 0 || pos >= (int64_t)g.max_blocks * g.bs;
  const bool bad_pos = g.rd > 0 && pos >= g.cos_rows;
  if (bad_ctx || bad_pos) {
    if (tid == 0) raise_flag(a.err_flags, bad_ctx ? PA_DEVERR_CONTEXT : PA_DEVERR_POSITION);
    for (int c = tid; c < vhs; c += kTile) out[c] = Half<T>::from_f32(0.f);
    return;
  }
  // the query's maps, rotated
  const T* qr = (const T*)a.query + (t * g.H + h) * 2 * (int64_t)hs;
  for (int i = tid; i < 2 * (hs / 8); i += kTile) {
    const int m = i / (hs / 8), d0 = (i % (hs / 8)) * 8;
    const T* row = qr + m * hs;
    float x[8], xp[8];
    unpack8<T>(*reinterpret_cast<const uint4*>(row + d0), x);
    if (g.rd > 0 && d0 >= g.ro && d0 < g.ro + g.rd) {
      const int half = g.rd >> 1;
      const int dp = g.interleaved ? d0 : d0 - g.ro < half ? d0 + half : d0 - half;
      unpack8<T>(*reinterpret_cast<const uint4*>(row + dp), xp);
      rope8<T>(x, xp, d0, g.ro, g.rd, g.interleaved, (const T*)a.cos_cache + pos * half,
               (const T*)a.sin_cache + pos * half);
    }
    for (int e = 0; e < 8; ++e) q[m][d0 + e] = x[e];
  }
  if (tid == 0) s_bad = 0;
  __syncthreads();
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][2] = {};
  const int64_t lo = g.window >= 0 ? max((int64_t)0, pos - g.window) : 0;
  for (int64_t j0 = lo / kTile * kTile; j0 <= pos; j0 += kTile) {
    const int64_t j = j0 + tid;
    const bool seen = j >= lo && j <= pos;
    float s[2] = {-INFINITY, -INFINITY};
    if (seen) {
      const int32_t page = a.block_table[(int64_t)b * g.max_blocks + j / g.bs];
      if (page < 0 || page >= g.num_blocks) {
        s_bad = 1;
        raise_flag(a.err_flags, PA_DEVERR_BLOCK);
      } else {
        const int64_t row = (int64_t)page * g.bs + j % g.bs;
        for (int i = 0; i < 2; ++i) {
          const T* k = (const T*)a.key_cache + ((row * g.kvh + gk) * 2 + i) * hs;
          float dot = 0.f;
          for (int d = 0; d < hs; d += 8) {
            float x[8];
            unpack8<T>(*reinterpret_cast<const uint4*>(k + d), x);
            for (int e = 0; e < 8; ++e) dot = fmaf(q[i][d + e], x[e], dot);
          }
          s[i] = dot * g.scale;
          if (g.softcap > 0.f) s[i] = g.softcap * tanhf(s[i] / g.softcap);
        }
      }
    }
    for (int i = 0; i < 2; ++i) {
      const float mt = fmaxf(m[i], block_reduce(s[i], true, red));
      const float f = m[i] == -INFINITY ? 0.f : expf(m[i] - mt);
      const float e = s[i] == -INFINITY ? 0.f : expf(s[i] - mt);
      p[i][tid] = e;
      l[i] = l[i] * f + block_reduce(e, false, red);
      m[i] = mt;
      o[i][0] *= f;
      o[i][1] *= f;
    }
    __syncthreads();
    for (int k = 0; k < kTile; ++k) {
      const int64_t jk = j0 + k;
      if (jk < lo || jk > pos) continue;
      const int32_t page = a.block_table[(int64_t)b * g.max_blocks + jk / g.bs];
      if (page < 0 || page >= g.num_blocks) continue;
      const T* v = (const T*)a.value_cache +
                   (((int64_t)page * g.bs + jk % g.bs) * g.kvh + gk) * (int64_t)vhs;
      for (int c = 0; c < 2; ++c) {
        if (tid + c * kTile < vhs) {
          const float x = Half<T>::to_f32(v[tid + c * kTile]);
          o[0][c] = fmaf(p[0][k], x, o[0][c]);
          o[1][c] = fmaf(p[1][k], x, o[1][c]);
        }
      }
    }
    __syncthreads();
  }
  float d1 = 0.f, d2 = 0.f;
  const float* lv = a.lambda_vectors;
  for (int d = tid; d < hs; d += kTile) {
    d1 = fmaf(lv[d], lv[hs + d], d1);
    d2 = fmaf(lv[2 * hs + d], lv[3 * hs + d], d2);
  }
  const float lam = expf(block_reduce(d1, false, red)) - expf(block_reduce(d2, false, red)) +
                    a.lambda_init;
  float r[2], ss = 0.f;
  for (int c = 0; c < 2; ++c) {
    r[c] = o[0][c] / l[0] - lam * (o[1][c] / l[1]);
    if (tid + c * kTile < vhs) ss = fmaf(r[c], r[c], ss);
  }
  ss = block_reduce(ss, false, red);
  const float inv = (1.f - a.lambda_init) / sqrtf(ss / (float)vhs + a.norm_eps);
  const bool bad = s_bad != 0;
  for (int c = 0; c < 2; ++c) {
    const int ch = tid + c * kTile;
    if (ch < vhs)
      out[ch] = Half<T>::from_f32(bad ? 0.f : r[c] * inv * Half<T>::to_f32(((const T*)a.norm_weight)[ch]));
  }
}

}  // namespace

cudaError_t launch_simple(const Geometry& g, const DiffArgs& a) {
  const dim3 grid((unsigned)(a.num_tokens * g.H));
  if (g.dtype == PA_DTYPE_BF16) diff_simple_kernel<__nv_bfloat16><<<grid, kTile, 0, a.stream>>>(g, a);
  else diff_simple_kernel<__half><<<grid, kTile, 0, a.stream>>>(g, a);
  return cudaGetLastError();
}

}  // namespace diff
}  // namespace pa
