// Attention over 8-bit caches for few query rows: the plan, the kernel of pa_quant_rows.cuh,
// and the one that joins its parts.
#include <algorithm>

#include "pa_quant_plan.h"
#include "pa_quant_rows.cuh"

namespace pa {
namespace quant {
namespace {

using namespace rows;

// Joins the parts of a unit: a warp for four accumulators of a block of rows and every
// kSlices-th part, then the slices. Bound by latency: 4 to 7 us. (A warp for all parts: two
// sequences of up to 131072 keys took 2.6 us longer.)
constexpr int kSlices = 4;
template <int VP, int NB>
__global__ void __launch_bounds__(64 * VP * NB * kSlices)
quant_combine_kernel(const __grid_constant__ DecP A) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kTasks = 2 * VP * NB, kAcc = 8 * VP * NB, R = 8 * NB;
  const ReadP& P = A.R;
  __shared__ float4 s_acc[kSlices - 1][kTasks][4][32];
  __shared__ float4 s_ml[kSlices - 1][kTasks][32];
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const int task = (threadIdx.x >> 5) % kTasks, slice = (threadIdx.x >> 5) / kTasks;
  // (in decode every sequence that is read has as many units)
  const int per = P.kvh * ((P.grp + R - 1) / R);
  const int b = A.decode ? blockIdx.x / per : find_sequence(A.ws_units, P.nseq, blockIdx.x, lane);
  if (b < 0 || b >= P.nseq) return;
  const int u = blockIdx.x - (A.decode ? b * per : A.ws_units[b]);
  const int64_t part = A.ws_line[P.nseq], before = A.ws_line[b];
  const Span sp = span_of(A, b);
  if (sp.tiles == 0 || u < 0 || u >= P.kvh * sp.chunks) return;  // (offsets that do not rise)
  const int64_t start = before + (int64_t)u * (sp.tiles + A.extra), end = start + A.extra + sp.tiles;
  const int64_t c0 = (start + A.extra) / part, c1 = (end - 1) / part;
  if (c0 == c1) return;
  const int nb = task % NB, i0 = task / NB * 4;
  const int g = u / sp.chunks, r0 = (u - g * sp.chunks) * R, nr = min(R, sp.q * P.grp - r0);
  const int h = nb * 8 + 2 * tq;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
  bool bad = false;
  auto add = [&](const float4& ml, const float4 (&o)[4]) {  // maxima and sums of rows h, h + 1
    const float pm[2] = {ml.x, ml.z}, pl[2] = {ml.y, ml.w};
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
      acc[k][0] = acc[k][0] * fa[0] + o[k].x * fb[0];
      acc[k][1] = acc[k][1] * fa[1] + o[k].y * fb[1];
      acc[k][2] = acc[k][2] * fa[0] + o[k].z * fb[0];
      acc[k][3] = acc[k][3] * fa[1] + o[k].w * fb[1];
    }
  };
#pragma unroll 2
  for (int64_t c = c0 + slice; c <= c1; c += kSlices) {
    const int64_t slot = 2 * c + (c == c0 && start > c0 * part ? 1 : 0);
    const float4 ml = *reinterpret_cast<const float4*>(A.ws_ml + slot * R + h);
    float4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = A.ws_o[(slot * kAcc + (i0 + k) * NB + nb) * 32 + lane];
    add(ml, o);
  }
  if (slice > 0) {
    s_ml[slice - 1][task][lane] = make_float4(bad ? NAN : m[0], l[0], bad ? NAN : m[1], l[1]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      s_acc[slice - 1][task][k][lane] = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
  }
  __syncthreads();
  if (slice > 0) return;
#pragma unroll 1
  for (int s = 0; s < min((int64_t)(kSlices - 1), c1 - c0); ++s) {
    float4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = s_acc[s][task][k][lane];
    add(s_ml[s][task][lane], o);
  }
  float inv[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) inv[e] = inverse(P, g, r0, h + e, nr, m[e], l[e]);
  store_rows(P, sp, g, r0, nr, h, (gq >> 1) + 4 * (gq & 1), i0, bad, inv,
             [&](int k, int e) { return acc[k][e]; });
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// What a unit counts on the line beside its tiles: its query's rows, the joining of its
// warps and its results take a CTA as long as some 20 tiles, with 16 rows 40. Without it,
// parts with many short units were the last ones by far. Measured with 0, 12, 20, 40 (us).
// 8 rows: 32 sequences of 90 to 1500 keys, 16 heads of 64, 50.2, 32.1, 29.3, 29.8; of 256 to
// 1024 keys, 8 kv heads of 128 with 4 query heads each, 24.3, 18.8, 19.1, 21.5; of 1024 to 8192,
// 71.0, 67.5, 66.4, 67.2. 16 rows: two sequences of 60000 to 131072 keys, 4 kv heads with 16 each,
// 66.7, 62.7, 61.2, 59.1; drafts of 3 to 7 tokens over 2000 to 16000, 113, 101, 97.5, 93.9.
// Tiles of 16 keys (head sizes above 128) cost about as much each, their channels being more:
// 0, 12, 20, 40, 80 at 256 / 256, 32 heads over 8: 90 to 1500 keys 71.3, 39.9, 37.6, 37.0, 39.9;
// 1024 to 8192 117, 110, 108, 109, 115; 64 over 4 (16 rows) 61.5, 32.2, 33.6, 36.5, 45.1 and
// 91.3, 79.3, 78.0, 74.6, 85.1. (Furthest off: 16 heads of 128 / 256 over 90 to 1500, 54.4 and with 40 48.5.)
constexpr int kExtra = 20;

struct Plan {
  int kp, vp, nb, th, ctas;
  size_t o, ml, line, units;  // bytes of the workspace's parts
};
Plan plan_of(const Geometry& g, int64_t nseq, int64_t rows) {
  Plan p;
  p.kp = (g.hs + 63) / 64;
  p.vp = (g.vhs + 127) / 128;
  p.nb = rows > 8 ? 2 : 1;
  p.th = p.kp <= 2 && p.vp == 1 ? 2 : 1;
  p.ctas = p.th == 2 && p.nb == 1 ? 3 : 2;  // (as Shape has it)
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  const size_t slots = 2 * (size_t)g.num_sms * p.ctas;
  p.o = up(slots * 8 * p.vp * p.nb * 512);
  p.ml = up(slots * 8 * p.nb * sizeof(float2));
  p.line = up((size_t)(nseq + 1) * sizeof(int64_t));
  p.units = up((size_t)(nseq + 1) * sizeof(int32_t));
  return p;
}

}  // namespace

// (of any number of rows)
size_t rows_workspace(const Geometry& g, int64_t nseq) {
  const Plan p = plan_of(g, nseq, 8), q = plan_of(g, nseq, 16);
  return std::max(p.o + p.ml, q.o + q.ml) + p.line + p.units;
}

cudaError_t launch_rows(const Geometry& g, const QuantArgs& a, bool decode, int32_t few) {
  DecP A{};
  A.R = read_params(g, a);
  const int64_t nseq = A.R.nseq, tokens = decode ? nseq : a.num_tokens;  // (at most)
  // rows of a sequence: all have as many in decode; otherwise the mean says whether a
  // unit takes 8 or 16
  const int64_t mean = decode ? nseq : range_tokens(a.num_tokens, a.num_seqs, nseq);
  const int64_t rows = (mean * A.R.grp + nseq - 1) / nseq;
  const Plan p = plan_of(g, nseq, rows);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  A.ws_o = reinterpret_cast<float4*>(ws);
  A.ws_ml = reinterpret_cast<float2*>(ws + p.o);
  A.ws_line = reinterpret_cast<int64_t*>(ws + p.o + p.ml);
  A.ws_units = reinterpret_cast<int32_t*>(ws + p.o + p.ml + p.line);
  A.decode = decode;
  A.few = few;
  A.rows = 8 * p.nb;
  A.tile = 16 * p.th;
  A.box = std::min(g.bs, A.tile);
  A.extra = kExtra * p.nb;
  A.min_part = 2 * kWarps;
  const int64_t units =
      decode ? nseq * g.kvh * ((A.R.grp + A.rows - 1) / A.rows)
             : g.kvh * (tokens * A.R.grp / A.rows + nseq);  // at most
  if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e = A.R.two ? launch_rows_kernel<true>(g, a, A, p.kp, p.vp, p.nb)
                                : launch_rows_kernel<false>(g, a, A, p.kp, p.vp, p.nb);
  if (e != cudaSuccess) return e;
  auto combine = [&](auto kern) {
    return tc::launch_pdl(kern, dim3((unsigned)units), dim3(64 * p.vp * p.nb * kSlices), 0, a.stream, A);
  };
  if (p.vp == 1) return p.nb == 1 ? combine(quant_combine_kernel<1, 1>) : combine(quant_combine_kernel<1, 2>);
  return p.nb == 1 ? combine(quant_combine_kernel<2, 1>) : combine(quant_combine_kernel<2, 2>);
}

}  // namespace quant
}  // namespace pa
