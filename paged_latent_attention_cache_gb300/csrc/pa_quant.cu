// Caches in 8 bits (include/pa_quant.h): entry points, write phase, reading back.
#include <math.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <type_traits>

#include "pa_quant_common.cuh"
#include "pa_quant_internal.h"
#include "pa_quant_plan.h"

namespace pa {

// (pa_api.cu) the SEPARATE layout's parameter checks
pa_status resolve_separate(const pa_separate_params* p, Geometry* g);

namespace quant {
namespace {

constexpr int kMaxBlock = 4096;  // rows of a page

// ---------------------------------------------------------------------------
// Write phase. A CTA takes a run (the tokens of one sequence in one page) and
// a kv head: the largest magnitudes of its rows give the scales, the codes
// follow, and where a scale has grown the page's other rows are brought to it.
// No other CTA touches that head of the page, so nothing is atomic and the
// result does not depend on an order.
//
// Runs are numbered without a scan over the batch: sequence b gets numbers from
// first(b) = 2 b + cumseq[b] / bs on. It has at most (q - 1) / bs + 2 runs, and
// first(b + 1) - first(b) >= q / bs + 2. So a CTA finds its sequence by a search
// over cumseq, an offset per thread at a time.
//
// Bound by instructions for prompts, some 225 per eight channels (14740 new tokens of 8 kv
// heads of 128 / 128, 94 MB: 39.5 us, 2.4 TB/s), and by its chain of loads for single tokens
// (32 of them 4.4 us). All rows of a run are on their way to shared memory (cp.async) before its
// slots are looked at; each thread copies just what it will read, so no barrier stands between.
// The rotated keys stay there in f32 for their encoding. With a load per row where it was used
// those tokens took 66 us, with keys rotated twice 52. Threads and shared memory: write_plan.
// ---------------------------------------------------------------------------
struct WriteArgs {
  const void* key;
  const void* value;
  const void* cos_cache;
  const void* sin_cache;
  const void* k_norm;
  const int32_t* slot_mapping;
  const int32_t* cumseq;
  const int32_t* past;
  uint8_t* key_cache;
  uint8_t* value_cache;
  float2* scales;
  int32_t* err_flags;
  int64_t num_tokens, num_slots;
  int num_seqs, kvh, hs, vhs, ro, rd, interleaved, cos_rows, bs;
  float eps;
  int lpr;  // lanes per row: a power of two >= max(hs, vhs) / 8
  int cap;  // rows that shared memory holds at once
};

__device__ __forceinline__ uint32_t smem_address(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 load16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void store16(uint32_t a, const float* x) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3])
               : "memory");
}
// The larger magnitudes of two pairs (NaN loses), and of the two of a pair.
template <typename T>
__device__ __forceinline__ uint32_t max_pairs(uint32_t a, uint32_t b) {
  a &= 0x7fff7fffu;
  b &= 0x7fff7fffu;
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  else
    asm("max.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}
template <typename T>
__device__ __forceinline__ float max_pair(uint32_t a) {
  const T* h = reinterpret_cast<const T*>(&a);
  return fmaxf(Half<T>::to_f32(h[0]), Half<T>::to_f32(h[1]));
}
__device__ __forceinline__ float finite_max8(const float (&x)[8], float m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = fabsf(x[e]);
    if (a < INFINITY) m = fmaxf(m, a);
  }
  return m;
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  return make_uint2(encode2(x[0] * inv, x[1] * inv) | encode2(x[2] * inv, x[3] * inv) << 16,
                    encode2(x[4] * inv, x[5] * inv) | encode2(x[6] * inv, x[7] * inv) << 16);
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS)
quant_write_kernel(const __grid_constant__ WriteArgs A) {
  asm volatile("griddepcontrol.wait;\n griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(16) uint8_t s_rows[];  // [cap] keys (then the first half of their f32 words), the others, values; s_new
  uint8_t* s_new = s_rows + (size_t)A.cap * (2 * A.hs + A.vhs) * 2;  // [bs] rows that the call writes
  __shared__ int s_first;
  __shared__ float s_max[2][THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.y, bs = A.bs, sh = __ffs(bs) - 1;
  const int run = blockIdx.x;
  const bool tells = g == 0;  // one CTA of a run reports its errors
  auto first = [&](int b) { return 2 * (int64_t)b + (A.cumseq[b] >> sh); };
  if (run == 0 && tells) {  // offsets have to rise from 0 to the number of tokens
    bool bad = false;
    for (int b = tid; b < A.num_seqs; b += THREADS) bad |= A.cumseq[b] > A.cumseq[b + 1];
    if (tid == 0) bad |= A.cumseq[0] != 0 || A.cumseq[A.num_seqs] != A.num_tokens;
    if (bad) raise_flag(A.err_flags, PA_DEVERR_CUMSEQ);
  }
  int lo = 0, hi = A.num_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + THREADS - 1) / THREADS, at = lo + tid * step;
    const int n = __syncthreads_count(at < hi && (at == lo || first(at) <= run));
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  const int64_t c0 = A.cumseq[lo], c1 = A.cumseq[lo + 1], p0 = A.past[lo];
  const int64_t q = c1 - c0;
  const int64_t i = run - first(lo);  // the sequence's i-th run
  if (i < 0 || q <= 0 || c0 < 0 || c1 > A.num_tokens) return;
  if (p0 < 0) {
    if (tells && tid == 0 && i == 0) raise_flag(A.err_flags, PA_DEVERR_CONTEXT);
    return;
  }
  const int64_t begin = max(p0, ((p0 >> sh) + i) << sh), end = min(p0 + q, ((p0 >> sh) + i + 1) << sh);
  if (begin >= end) return;
  const int n = (int)(end - begin), row0 = (int)(begin & (bs - 1));
  const int64_t t0 = c0 + (begin - p0);

  const int lpr = A.lpr, rows_at_once = THREADS / lpr, mine = tid / lpr;
  const int d0 = (tid & (lpr - 1)) * 8;
  const int64_t kstep = (int64_t)A.kvh * A.hs, vstep = (int64_t)A.kvh * A.vhs;
  const T* key = reinterpret_cast<const T*>(A.key) + t0 * kstep + (int64_t)g * A.hs + d0;
  const T* value = reinterpret_cast<const T*>(A.value) + t0 * vstep + (int64_t)g * A.vhs + d0;
  const uint32_t k_at = smem_address(s_rows) + d0 * 2, k_more = A.cap * A.hs * 2;
  const uint32_t v_at = k_at + 2 * k_more;
  auto fetch = [&](int j0) {  // rows j0 .. j0 + cap
    for (int j = j0 + mine; j < min(n, j0 + A.cap); j += rows_at_once) {
      if (d0 < A.hs) copy16(k_at + (j - j0) * A.hs * 2, key + j * kstep);
      if (d0 < A.vhs) copy16(v_at + (j - j0) * A.vhs * 2, value + j * vstep);
      if (A.rd > 0 && begin + j < A.cos_rows && d0 * 8 < A.rd >> 1) {
        // (64 angles a line; lanes 0, 1, ..)
        const int64_t a = (begin + j) * (A.rd >> 1) + d0 * 8;
        asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const T*>(A.cos_cache) + a));
        asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const T*>(A.sin_cache) + a));
      }
    }
  };
  fetch(0);

  // rows that the call writes: tokens with a slot of the page that the run's
  // first one names
  for (int r = tid; r < bs; r += THREADS) s_new[r] = 0;
  if (tid == 0) s_first = n;
  __syncthreads();
  int err = 0;
  for (int j = tid; j < n; j += THREADS) {
    const int32_t slot = A.slot_mapping[t0 + j];
    if (slot == -1) continue;
    if (slot < 0 || slot >= A.num_slots || (slot & (bs - 1)) != row0 + j) {
      err |= PA_DEVERR_SLOT;
    } else if (A.rd > 0 && begin + j >= A.cos_rows) {
      err |= PA_DEVERR_POSITION;
    } else {
      atomicMin(&s_first, j);
      s_new[row0 + j] = 1;
    }
  }
  __syncthreads();
  const int first_j = s_first;
  if (first_j < n) {
    const int32_t page_of = A.slot_mapping[t0 + first_j] >> sh;
    for (int j = tid; j < n; j += THREADS)
      if (s_new[row0 + j] && A.slot_mapping[t0 + j] >> sh != page_of) {
        s_new[row0 + j] = 0;
        err |= PA_DEVERR_SLOT;
      }
  }
  if (err && tells) raise_flag(A.err_flags, err);
  if (first_j >= n) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  const int64_t page = A.slot_mapping[t0 + first_j] >> sh;
  __syncthreads();

  float2* scale = A.scales + page * A.kvh + g;
  const float2 was = s_new[0] ? make_float2(0.f, 0.f) : *scale;
  // Largest magnitudes of rows j0 .. j0 + cap; the keys rotated.
  float km = 0.f, vm = 0.f;
  auto transform = [&](int j0, bool finite) {
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
    for (int j1 = 0; j1 < A.cap && j0 + j1 < n; j1 += rows_at_once) {
      const int j = j0 + j1 + mine;
      const bool row = j < n && s_new[row0 + j];
      const uint32_t k = k_at + (j1 + mine) * A.hs * 2;
      float x[8];
      uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
      if (row && d0 < A.hs) kw = load16(k);
      if (row && d0 < A.vhs) vw = load16(v_at + (j1 + mine) * A.vhs * 2);
      unpack8<T>(kw, x);
      norm_rotate8<T>(x, row, d0, A.hs, lpr, reinterpret_cast<const T*>(A.k_norm), A.eps, A.ro, A.rd,
                      A.interleaved, reinterpret_cast<const T*>(A.cos_cache),
                      reinterpret_cast<const T*>(A.sin_cache), begin + j);
      if (row && d0 < A.hs) {
        store16(k, x);
        store16(k + k_more, x + 4);
      }
      if (finite) {
        float v[8];
        unpack8<T>(vw, v);
        km = finite_max8(x, km);
        vm = finite_max8(v, vm);
      } else {  // (NaN loses a comparison, an infinity shows)
#pragma unroll
        for (int e = 0; e < 8; ++e) km = fmaxf(km, fabsf(x[e]));
        vm = fmaxf(vm, max_pair<T>(max_pairs<T>(max_pairs<T>(vw.x, vw.y), max_pairs<T>(vw.z, vw.w))));
      }
    }
  };
  auto transform_all = [&](bool finite, bool again) {
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += A.cap) {
      if (j0 > 0 || again) fetch(j0);
      transform(j0, finite);
    }
  };
  transform_all(false, false);
  if (__syncthreads_or(km == INFINITY || vm == INFINITY)) {  // the largest finite ones then
    km = vm = 0.f;
    transform_all(true, true);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
    vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
  }
  if (lane == 0) {
    s_max[0][warp] = km;
    s_max[1][warp] = vm;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    km = fmaxf(km, s_max[0][w]);
    vm = fmaxf(vm, s_max[1][w]);
  }
  const int ko = scale_exponent(was.x), vo = scale_exponent(was.y);
  const int ke = max(ko, needed_exponent(km)), ve = max(vo, needed_exponent(vm));
  uint8_t* kpage = A.key_cache + page * bs * kstep + (int64_t)g * A.hs;
  uint8_t* vpage = A.value_cache + page * bs * vstep + (int64_t)g * A.vhs;
  const float kinv = pow2(-ke), vinv = pow2(-ve);
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += A.cap) {
    if (n > A.cap) {  // (else they are still there)
      fetch(j0);
      transform(j0, true);
    }
#pragma unroll 2
    for (int j1 = 0; j1 < A.cap && j0 + j1 < n; j1 += rows_at_once) {
      const int j = j0 + j1 + mine;
      if (j >= n || !s_new[row0 + j]) continue;
      float x[8];
      if (d0 < A.hs) {
        const uint32_t k = k_at + (j1 + mine) * A.hs * 2;
        const uint4 a = load16(k), b = load16(k + k_more);
        x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y);
        x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
        x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y);
        x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
        *reinterpret_cast<uint2*>(kpage + (row0 + j) * kstep + d0) = encode8(x, kinv);
      }
      if (d0 < A.vhs) {
        unpack8<T>(load16(v_at + (j1 + mine) * A.vhs * 2), x);
        *reinterpret_cast<uint2*>(vpage + (row0 + j) * vstep + d0) = encode8(x, vinv);
      }
    }
  }
  auto shrink = [&](uint8_t* at, int64_t step, int width, float f) {
    const int pieces = width >> 4;
    for (int i = tid; i < bs * pieces; i += THREADS) {
      const int r = i / pieces;
      if (s_new[r]) continue;
      uint4* p = reinterpret_cast<uint4*>(at + r * step + (i - r * pieces) * 16);
      const uint4 w = *p;
      *p = make_uint4(shrink4(w.x, f), shrink4(w.y, f), shrink4(w.z, f), shrink4(w.w, f));
    }
  };
  if (ko != kNone && ko < ke) shrink(kpage, kstep, A.hs, pow2(max(-126, ko - ke)));
  if (vo != kNone && vo < ve) shrink(vpage, vstep, A.vhs, pow2(max(-126, vo - ve)));
  __syncthreads();  // (all have read the old scale)
  if (tid == 0) *scale = make_float2(pow2(ke), pow2(ve));
}

// ---------------------------------------------------------------------------
// Reading back: a warp for a few tokens in a row, 16 codes a lane: one search and one
// look into the table serve several tokens. Bound by HBM: 16 sequences of 1024 to 8192
// rows of 8 heads of 128 / 128 (475 MB) 88 us, 5.4 TB/s; a warp per token took 94.
// ---------------------------------------------------------------------------
struct RestoreArgs {
  const uint8_t* key_cache;
  const uint8_t* value_cache;
  const float2* scales;
  const int32_t* cumseq;
  const int32_t* past;
  const int32_t* block_table;
  void* key;
  void* value;
  int32_t* err_flags;
  int64_t num_tokens;
  int num_seqs, kvh, hs, vhs, bs, num_blocks, max_blocks;
};

template <typename T>
__device__ __forceinline__ T saturated(float x);
template <>
__device__ __forceinline__ __half saturated<__half>(float x) {
  return __float2half_rn(x > 65504.f ? 65504.f : x < -65504.f ? -65504.f : x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 saturated<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);  // (448 * 2^48 is far below its end)
}

template <typename T>
__device__ __forceinline__ void restore16(const uint4& c, float scale, T* dst) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  T h[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = decode2(w[i]), b = decode2(w[i] >> 16);
    h[4 * i] = saturated<T>(a.x * scale);
    h[4 * i + 1] = saturated<T>(a.y * scale);
    h[4 * i + 2] = saturated<T>(b.x * scale);
    h[4 * i + 3] = saturated<T>(b.y * scale);
  }
  reinterpret_cast<uint4*>(dst)[0] = reinterpret_cast<const uint4*>(h)[0];
  reinterpret_cast<uint4*>(dst)[1] = reinterpret_cast<const uint4*>(h)[1];
}

template <typename T>
__global__ void __launch_bounds__(256)
quant_restore_kernel(const __grid_constant__ RestoreArgs A) {
  asm volatile("griddepcontrol.wait;\n griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, sh = __ffs(A.bs) - 1;
  const int kp = A.hs >> 4, vp = A.vhs >> 4;
  const int kn = A.key ? A.kvh * kp : 0, vn = A.value ? A.kvh * vp : 0;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  if (blockIdx.x == 0 && threadIdx.x == 0 &&
      (A.cumseq[0] != 0 || A.cumseq[A.num_seqs] != A.num_tokens))
    raise_flag(A.err_flags, PA_DEVERR_CUMSEQ);
  // tokens [first, last) of this warp: the search and the table's entries serve several
  const int64_t each = (A.num_tokens + warps - 1) / warps;
  const int64_t first = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * each;
  const int64_t last = min(A.num_tokens, first + each);
  int b = -1;
  int64_t c0 = 0, c1 = 0, past = 0, block = -1;
  int32_t page = -1;
  for (int64_t t = first; t < last; ++t) {
    if (t >= c1 || b < 0) {
      b = find_sequence(A.cumseq, A.num_seqs, t, lane);
      if (b < 0) {
        if (lane == 0) raise_flag(A.err_flags, PA_DEVERR_CUMSEQ);
        continue;
      }
      c0 = A.cumseq[b];
      c1 = A.cumseq[b + 1];
      past = A.past[b];
      block = -1;
    }
    const int64_t pos = past + (t - c0);
    if (pos < 0 || pos >= (int64_t)A.max_blocks * A.bs) {
      if (lane == 0) raise_flag(A.err_flags, PA_DEVERR_CONTEXT);
      page = -1;
      block = -1;
    } else if (pos >> sh != block) {
      block = pos >> sh;
      page = A.block_table[(int64_t)b * A.max_blocks + block];
      if (page < 0 || page >= A.num_blocks) {
        if (lane == 0) raise_flag(A.err_flags, PA_DEVERR_BLOCK);
        page = -1;
      }
    }
    const int64_t row = (int64_t)page * A.bs + (pos & (A.bs - 1));
#pragma unroll 4
    for (int i = lane; i < kn + vn; i += 32) {
      const bool is_key = i < kn;
      const int at = is_key ? i : i - kn, per = is_key ? kp : vp;
      T* dst = (is_key ? reinterpret_cast<T*>(A.key) + t * (A.kvh * A.hs)
                       : reinterpret_cast<T*>(A.value) + t * (A.kvh * A.vhs)) + at * 16;
      uint4 c = make_uint4(0, 0, 0, 0);
      float s = 0.f;
      if (page >= 0) {
        const uint8_t* src = is_key ? A.key_cache + row * (A.kvh * A.hs)
                                    : A.value_cache + row * (A.kvh * A.vhs);
        c = *reinterpret_cast<const uint4*>(src + at * 16);
        const float2 two = A.scales[(int64_t)page * A.kvh + at / per];
        s = is_key ? two.x : two.y;
        if (scale_exponent(s) == kNone) {  // (zeros, whatever the codes: 0 times NaN is NaN)
          c = make_uint4(0, 0, 0, 0);
          s = 0.f;
        }
      }
      restore16<T>(c, s, dst);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
pa_status fail(pa_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
pa_status fail(pa_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return record_error(s, buf);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

pa_status resolve(const pa_quant_params* p, Geometry* g) {
  if (!p) return fail(PA_ERR_INVALID_ARGUMENT, "params is NULL");
  if (p->flags & ~(PA_FLAG_AFTER_WRITE | PA_FLAG_OWN_SLOTS))
    return fail(PA_ERR_INVALID_ARGUMENT, "unknown flag bits 0x%x", p->flags);
  if (p->cross != 0 && p->cross != 1) return fail(PA_ERR_INVALID_ARGUMENT, "cross must be 0 or 1");
  if (p->cross && (p->rotary_dim != 0 || p->local_window_size >= 0))
    return fail(PA_ERR_INVALID_ARGUMENT,
                "cross attention has no positions: rotary_dim must be 0 and local_window_size < 0");
  pa_separate_params q = {};
  q.dtype = p->dtype;
  q.num_heads = p->num_heads;
  q.kv_num_heads = p->kv_num_heads;
  q.head_size = p->head_size;
  q.rotary_offset = p->rotary_offset;
  q.rotary_dim = p->rotary_dim;
  q.rotary_interleaved = p->rotary_interleaved;
  q.cos_rows = p->cos_rows;
  q.block_size = p->block_size;
  q.num_blocks = p->num_blocks;
  q.max_blocks_per_seq = p->max_blocks_per_seq;
  q.scale = p->scale;
  q.softcap = p->softcap;
  q.local_window_size = p->local_window_size;
  q.rms_eps = p->rms_eps;
  q.flags = p->flags;
  const pa_status s = resolve_separate(&q, g);
  if (s != PA_OK) return s;
  if (p->v_head_size < 0) return fail(PA_ERR_INVALID_ARGUMENT, "v_head_size must be >= 0");
  g->vhs = p->v_head_size == 0 ? g->hs : p->v_head_size;
  if (g->H > 65535)
    return fail(PA_ERR_NOT_IMPLEMENTED, "num_heads %d exceeds the supported maximum 65535", g->H);
  if (g->hs > 256 || g->vhs > 256 || g->vhs % 16 != 0 || g->H / g->kvh > 128)
    return fail(PA_ERR_NOT_IMPLEMENTED,
                "8-bit caches: head_size and v_head_size multiples of 16 up to 256 and at most "
                "128 heads per kv head (got %d, %d, %d)", g->hs, g->vhs, g->H / g->kvh);
  if (g->bs > kMaxBlock)
    return fail(PA_ERR_NOT_IMPLEMENTED, "block_size %d exceeds the supported maximum %d", g->bs,
                kMaxBlock);
  return PA_OK;
}

pa_status check_tokens(int64_t num_tokens, int32_t num_seqs, const Geometry& g) {
  if (num_tokens < 0 || num_seqs < 0)
    return fail(PA_ERR_INVALID_ARGUMENT, "num_tokens and num_seqs must be >= 0");
  if (num_seqs > 1 << 28) return fail(PA_ERR_INVALID_ARGUMENT, "num_seqs must be <= 2^28");
  if (num_tokens * (int64_t)g.H >= ((int64_t)1 << 30) || num_tokens > INT32_MAX)
    return fail(PA_ERR_INVALID_ARGUMENT, "num_tokens * num_heads must be < 2^30");
  return PA_OK;
}

template <typename K, typename A>
pa_status launch(K kernel, dim3 grid, int threads, size_t smem, void* stream, const A& args,
                 const char* what) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
  if (e == cudaSuccess) return PA_OK;
  (void)cudaGetLastError();  // not left behind for a later call
  return fail(PA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The checks of a read call; g: the geometry, a.cross is filled in.
pa_status check_read(Phase ph, const pa_quant_params* p, QuantArgs* args, Geometry* geometry) {
  QuantArgs& a = *args;
  Geometry& g = *geometry;
  pa_status s = resolve(p, &g);
  if (s == PA_OK) s = check_tokens(a.num_tokens, a.num_seqs, g);
  if (s != PA_OK) return s;
  if (a.seq_begin < 0 || a.seq_end < a.seq_begin || a.seq_end > a.num_seqs)
    return fail(PA_ERR_INVALID_ARGUMENT, "sequence range [%d, %d) outside [0, %d)", a.seq_begin,
                a.seq_end, a.num_seqs);
  if (a.num_tokens == 0 || a.seq_end == a.seq_begin) return PA_OK;
  if (ph == Phase::kDecode && (int64_t)(a.seq_end - a.seq_begin) > a.num_tokens)
    return fail(PA_ERR_INVALID_ARGUMENT,
                "decode over %d sequences needs at least that many tokens (have %lld)",
                a.seq_end - a.seq_begin, (long long)a.num_tokens);
  if (!a.query || !a.key_cache || !a.value_cache || !a.scales || !a.cumseq || !a.past ||
      !a.block_table || !a.out)
    return fail(PA_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (g.rd > 0 && (!a.cos_cache || !a.sin_cache))
    return fail(PA_ERR_INVALID_ARGUMENT, "cos_cache/sin_cache are required when rotary_dim > 0");
  if (!aligned(a.query, 16) || !aligned(a.out, 16) || !aligned(a.q_norm, 16) ||
      !aligned(a.head_sink, 2) ||
      (g.rd > 0 && (!aligned(a.cos_cache, 16) || !aligned(a.sin_cache, 16))))
    return fail(PA_ERR_INVALID_ARGUMENT,
                "half-precision tensors must be 16-byte aligned (head_sink 2-byte)");
  if (!aligned(a.key_cache, 16) || !aligned(a.value_cache, 16) || !aligned(a.scales, 8))
    return fail(PA_ERR_INVALID_ARGUMENT, "caches must be 16-byte and scales 8-byte aligned");
  if (!aligned(a.cumseq, 4) || !aligned(a.past, 4) || !aligned(a.block_table, 4) ||
      !aligned(a.err_flags, 4))
    return fail(PA_ERR_INVALID_ARGUMENT, "int32 tensors must be 4-byte aligned");
  if (a.workspace && !aligned(a.workspace, 256))
    return fail(PA_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  const int64_t nseq = a.seq_end - a.seq_begin;
  const size_t need = ph == Phase::kDecode ? rows_workspace(g, nseq) : prefill_workspace(g, nseq);
  if (need > 0 && (!a.workspace || a.workspace_bytes < need))
    return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed",
                a.workspace ? a.workspace_bytes : (size_t)0, need);
  a.cross = p->cross;
  return PA_OK;
}

pa_status launch_read(Phase ph, const Geometry& g, const QuantArgs& a) {
  if (a.num_tokens == 0 || a.seq_end == a.seq_begin) return PA_OK;
  const cudaError_t e = ph == Phase::kDecode ? launch_rows(g, a, true, kAnyTokens) : launch_prefill(g, a);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();  // not left behind for a later call
    return fail(PA_ERR_CUDA, "attention over an 8-bit cache: %s", cudaGetErrorString(e));
  }
  return PA_OK;
}

pa_status read(Phase ph, const pa_quant_params* p, QuantArgs a) {
  Geometry g;
  const pa_status s = check_read(ph, p, &a, &g);
  return s == PA_OK ? launch_read(ph, g, a) : s;
}

}  // namespace
}  // namespace quant
}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_quant_validate(const pa_quant_params* p) {
  Geometry g;
  return quant::resolve(p, &g);
}

pa_status pa_quant_write(const pa_quant_params* p, const void* key, const void* value,
                         int64_t num_tokens, const void* cos_cache, const void* sin_cache,
                         const void* k_norm_weight, const int32_t* slot_mapping,
                         const int32_t* cumseq, const int32_t* past, int32_t num_seqs,
                         void* key_cache, void* value_cache, float* scales, int32_t* err_flags,
                         void* stream) {
  using quant::aligned;
  using quant::fail;
  Geometry g;
  pa_status s = quant::resolve(p, &g);
  if (s == PA_OK) s = quant::check_tokens(num_tokens, num_seqs, g);
  if (s != PA_OK) return s;
  if (num_tokens == 0) return PA_OK;
  if (num_seqs < 1) return fail(PA_ERR_INVALID_ARGUMENT, "tokens given but num_seqs is 0");
  if (!key || !value || !slot_mapping || !cumseq || !past || !key_cache || !value_cache || !scales)
    return fail(PA_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (g.rd > 0 && (!cos_cache || !sin_cache))
    return fail(PA_ERR_INVALID_ARGUMENT, "cos_cache/sin_cache are required when rotary_dim > 0");
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_norm_weight, 16) ||
      (g.rd > 0 && (!aligned(cos_cache, 16) || !aligned(sin_cache, 16))))
    return fail(PA_ERR_INVALID_ARGUMENT, "half-precision tensors must be 16-byte aligned");
  if (!aligned(key_cache, 16) || !aligned(value_cache, 16) || !aligned(scales, 8))
    return fail(PA_ERR_INVALID_ARGUMENT, "caches must be 16-byte and scales 8-byte aligned");
  if (!aligned(slot_mapping, 4) || !aligned(cumseq, 4) || !aligned(past, 4) ||
      !aligned(err_flags, 4))
    return fail(PA_ERR_INVALID_ARGUMENT, "int32 tensors must be 4-byte aligned");
  int lpr = 2;
  while (lpr * 8 < g.hs || lpr * 8 < g.vhs) lpr *= 2;
  const int row_bytes = (2 * g.hs + g.vhs) * 2;
  const quant::WritePlan plan =
      quant::write_plan(num_tokens, num_seqs, g.kvh, g.bs, lpr, row_bytes, g.num_sms);
  const size_t smem = (size_t)plan.cap * row_bytes + g.bs;
  const quant::WriteArgs A{key, value, cos_cache, sin_cache, k_norm_weight, slot_mapping, cumseq,
                           past, (uint8_t*)key_cache, (uint8_t*)value_cache, (float2*)scales,
                           err_flags, num_tokens, (int64_t)g.num_blocks * g.bs, num_seqs, g.kvh,
                           g.hs, g.vhs, g.ro, g.rd, g.interleaved, g.cos_rows, g.bs, g.rms_eps,
                           lpr, plan.cap};
  const dim3 grid((unsigned)plan.runs, (unsigned)g.kvh);
  auto go = [&](auto* typed, auto th) {
    auto kern = quant::quant_write_kernel<std::remove_pointer_t<decltype(typed)>, th()>;
    static std::atomic<bool> configured[64];
    const cudaError_t e = once_per_device(configured, g.device, [&] {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  quant::kRowBytes + quant::kMaxBlock);
    });
    if (e != cudaSuccess) {
      (void)cudaGetLastError();  // not left behind for a later call
      return fail(PA_ERR_CUDA, "8-bit write launch: %s", cudaGetErrorString(e));
    }
    return quant::launch(kern, grid, th(), smem, stream, A, "8-bit write launch");
  };
  auto typed = [&](auto* t) {
    switch (plan.threads) {
      case 128: return go(t, std::integral_constant<int, 128>());
      case 256: return go(t, std::integral_constant<int, 256>());
      default: return go(t, std::integral_constant<int, 512>());
    }
  };
  return g.dtype == PA_DTYPE_BF16 ? typed((__nv_bfloat16*)nullptr) : typed((__half*)nullptr);
}

pa_status pa_quant_restore(const pa_quant_params* p, const void* key_cache,
                           const void* value_cache, const float* scales, const int32_t* cumseq,
                           const int32_t* past, const int32_t* block_table, int32_t num_seqs,
                           int64_t num_tokens, void* key, void* value, int32_t* err_flags,
                           void* stream) {
  using quant::aligned;
  using quant::fail;
  Geometry g;
  pa_status s = quant::resolve(p, &g);
  if (s == PA_OK) s = quant::check_tokens(num_tokens, num_seqs, g);
  if (s != PA_OK) return s;
  if (num_tokens == 0 || (!key && !value)) return PA_OK;
  if (num_seqs < 1) return fail(PA_ERR_INVALID_ARGUMENT, "tokens given but num_seqs is 0");
  if (!key_cache || !value_cache || !scales || !cumseq || !past || !block_table)
    return fail(PA_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (!aligned(key, 16) || !aligned(value, 16))
    return fail(PA_ERR_INVALID_ARGUMENT, "half-precision tensors must be 16-byte aligned");
  if (!aligned(key_cache, 16) || !aligned(value_cache, 16) || !aligned(scales, 8))
    return fail(PA_ERR_INVALID_ARGUMENT, "caches must be 16-byte and scales 8-byte aligned");
  if (!aligned(cumseq, 4) || !aligned(past, 4) || !aligned(block_table, 4) ||
      !aligned(err_flags, 4))
    return fail(PA_ERR_INVALID_ARGUMENT, "int32 tensors must be 4-byte aligned");
  const quant::RestoreArgs A{(const uint8_t*)key_cache, (const uint8_t*)value_cache,
                             (const float2*)scales, cumseq, past, block_table, key, value,
                             err_flags, num_tokens, num_seqs, g.kvh, g.hs, g.vhs, g.bs,
                             g.num_blocks, g.max_blocks};
  int64_t blocks = (num_tokens + 7) / 8;
  const int64_t cap = (int64_t)g.num_sms * 8;
  if (blocks > cap) blocks = cap;
  const dim3 grid((unsigned)blocks);
  return g.dtype == PA_DTYPE_BF16
             ? quant::launch(quant::quant_restore_kernel<__nv_bfloat16>, grid, 256, 0, stream, A,
                             "8-bit restore launch")
             : quant::launch(quant::quant_restore_kernel<__half>, grid, 256, 0, stream, A,
                             "8-bit restore launch");
}

pa_status pa_quant_decode(const pa_quant_params* p, const void* query, int64_t num_tokens,
                          const void* key_cache, const void* value_cache, const float* scales,
                          const void* cos_cache, const void* sin_cache, const void* q_norm_weight,
                          const void* head_sink, const int32_t* cumseq, const int32_t* past,
                          const int32_t* block_table, int32_t num_seqs, int32_t seq_begin,
                          int32_t seq_end, void* workspace, size_t workspace_bytes, void* out,
                          int32_t* err_flags, void* stream) {
  return quant::read(Phase::kDecode, p,
                     quant::QuantArgs{query, num_tokens, (const uint8_t*)key_cache,
                                      (const uint8_t*)value_cache, (const float2*)scales,
                                      cos_cache, sin_cache, q_norm_weight, head_sink, cumseq, past,
                                      block_table, num_seqs, seq_begin, seq_end, workspace,
                                      workspace_bytes, out, err_flags, (cudaStream_t)stream, 0});
}

pa_status pa_quant_prefill(const pa_quant_params* p, const void* query, int64_t num_tokens,
                           const void* key_cache, const void* value_cache, const float* scales,
                           const void* cos_cache, const void* sin_cache,
                           const void* q_norm_weight, const void* head_sink,
                           const int32_t* cumseq, const int32_t* past, const int32_t* block_table,
                           int32_t num_seqs, int32_t seq_begin, int32_t seq_end, void* workspace,
                           size_t workspace_bytes, void* out, int32_t* err_flags, void* stream) {
  return quant::read(Phase::kPrefill, p,
                     quant::QuantArgs{query, num_tokens, (const uint8_t*)key_cache,
                                      (const uint8_t*)value_cache, (const float2*)scales,
                                      cos_cache, sin_cache, q_norm_weight, head_sink, cumseq, past,
                                      block_table, num_seqs, seq_begin, seq_end, workspace,
                                      workspace_bytes, out, err_flags, (cudaStream_t)stream, 0});
}

pa_status pa_quant_mixed(const pa_quant_params* p, const void* query, const void* key,
                         const void* value, int64_t num_tokens, const void* cos_cache,
                         const void* sin_cache, const void* q_norm_weight,
                         const void* k_norm_weight, const void* head_sink,
                         const int32_t* slot_mapping, const int32_t* cumseq, const int32_t* past,
                         const int32_t* block_table, int32_t num_seqs, int32_t num_decode_seqs,
                         void* key_cache, void* value_cache, float* scales, void* workspace,
                         size_t workspace_bytes, void* out, int32_t* err_flags, void* stream) {
  using quant::fail;
  if (!p) return fail(PA_ERR_INVALID_ARGUMENT, "params is NULL");
  if (p->cross)
    return fail(PA_ERR_INVALID_ARGUMENT, "cross attention writes and reads in calls of their own");
  if (num_decode_seqs < 0 || num_decode_seqs > num_seqs)
    return fail(PA_ERR_INVALID_ARGUMENT, "num_decode_seqs %d outside [0, %d]", num_decode_seqs,
                num_seqs);
  // what the reads would refuse is refused before the write is enqueued
  quant::QuantArgs a{query, num_tokens, (const uint8_t*)key_cache, (const uint8_t*)value_cache,
                     (const float2*)scales, cos_cache, sin_cache, q_norm_weight, head_sink, cumseq,
                     past, block_table, num_seqs, 0, num_decode_seqs, workspace, workspace_bytes,
                     out, err_flags, (cudaStream_t)stream, 0};
  quant::QuantArgs b = a;
  b.seq_begin = num_decode_seqs;
  b.seq_end = num_seqs;
  Geometry g;
  pa_status s = quant::check_read(Phase::kDecode, p, &a, &g);
  if (s == PA_OK) s = quant::check_read(Phase::kPrefill, p, &b, &g);
  if (s == PA_OK)
    s = pa_quant_write(p, key, value, num_tokens, cos_cache, sin_cache, k_norm_weight, slot_mapping,
                       cumseq, past, num_seqs, key_cache, value_cache, scales, err_flags, stream);
  if (s != PA_OK) return s;
  g.flags |= PA_FLAG_AFTER_WRITE;
  if ((s = quant::launch_read(Phase::kDecode, g, a)) != PA_OK) return s;
  if (num_decode_seqs > 0) g.flags &= ~PA_FLAG_AFTER_WRITE;
  return quant::launch_read(Phase::kPrefill, g, b);
}

size_t pa_quant_workspace_size(const pa_quant_params* p, int32_t num_seqs, int64_t num_tokens) {
  Geometry g;
  if (quant::resolve(p, &g) != PA_OK || num_seqs <= 0 || num_tokens <= 0) return 0;
  return quant::prefill_workspace(g, num_seqs);  // (decode's is part of it)
}

}  // extern "C"
