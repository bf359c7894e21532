// Differential attention (include/pa_diff.h): entry points and write phase.
#include <math.h>

#include <cstdarg>
#include <cstdio>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_diff_internal.h"

namespace pa {

// (pa_api.cu) the SEPARATE layout's parameter checks
pa_status resolve_separate(const pa_separate_params* p, Geometry* g);

namespace diff {
namespace {

// ---------------------------------------------------------------------------
// Write phase: one thread per (token, 8-channel group) of the token's
// kvH * (2 hs + vhs) channels, keys first; 16-byte loads and stores, every
// byte once (a rotary group also reads its partner group, from L1).
// ---------------------------------------------------------------------------
// Largest batch whose offsets are staged in shared memory (the search for a
// token's sequence is then no chain of global loads).
constexpr int kStagedSeqs = 8191;

template <typename T>
__global__ void __launch_bounds__(256)
diff_write_kernel(const T* __restrict__ key, const T* __restrict__ value,
                  const T* __restrict__ cos_cache, const T* __restrict__ sin_cache,
                  const int32_t* __restrict__ slot_mapping, const int32_t* __restrict__ cumseq,
                  const int32_t* __restrict__ past, int32_t num_seqs, T* __restrict__ key_cache,
                  T* __restrict__ value_cache, int64_t num_tokens, int kvh, int hs, int vhs,
                  int ro, int rd, int interleaved, int cos_rows, int64_t num_slots,
                  int32_t* err_flags, int step_t, int step_c) {
  // This kernel takes its place while the one before it ends; once that is
  // complete, a read kernel behind this one may start its prologue (it waits for
  // this grid before it reads the cache).
  asm volatile("griddepcontrol.wait;\n griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ int32_t s_cum[];  // cumseq[0..num_seqs] when staged
  const int32_t* cum = cumseq;
  if (num_seqs <= kStagedSeqs) {
    for (int i = threadIdx.x; i <= num_seqs; i += blockDim.x) s_cum[i] = cumseq[i];
    __syncthreads();
    cum = s_cum;
  }
  const int kg = kvh * 2 * (hs >> 3), vg = kvh * (vhs >> 3), groups = kg + vg;
  // (t, c) is one division away from the thread's number (below 2^31); a step is
  // the grid's threads, step_t tokens and step_c groups
  const int first_item = (int)(blockIdx.x * blockDim.x + threadIdx.x);
  int64_t t = first_item / groups;
  int c = first_item - (int)t * groups;
  for (; t < num_tokens; t += step_t, c += step_c) {
    if (c >= groups) {
      c -= groups;
      if (++t >= num_tokens) break;
    }
    const bool is_key = c < kg;
    const bool first = c == 0;  // one thread per token reports its errors
    const int32_t slot = slot_mapping[t];
    const T* src = is_key ? key + t * kg * 8 + c * 8 : value + t * vg * 8 + (int64_t)(c - kg) * 8;
    uint4 v = *reinterpret_cast<const uint4*>(src);
    const int d0 = is_key ? (c * 8) % hs : 0;  // channel within the map
    const bool rot = is_key && rd > 0 && d0 >= ro && d0 < ro + rd;
    uint4 vp = v;
    if (rot && !interleaved) {
      const int half = rd >> 1;
      vp = *reinterpret_cast<const uint4*>(src + (d0 - ro < half ? half : -half));
    }
    if (slot < 0 || (int64_t)slot >= num_slots) {
      if (slot != -1 && first) raise_flag(err_flags, PA_DEVERR_SLOT);
      continue;
    }
    int32_t b;
    int64_t pos;
    if (!locate_token(t, cum, past, num_seqs, first ? err_flags : nullptr, &b, &pos)) continue;
    if (rd > 0 && (pos < 0 || pos >= cos_rows)) {  // the token's row is skipped
      if (first) raise_flag(err_flags, pos < 0 ? PA_DEVERR_CONTEXT : PA_DEVERR_POSITION);
      continue;
    }
    if (rot) {
      float x[8], xp[8];
      unpack8<T>(v, x);
      unpack8<T>(vp, xp);
      rope8<T>(x, xp, d0, ro, rd, interleaved, cos_cache + pos * (rd >> 1),
               sin_cache + pos * (rd >> 1));
      v = pack8<T>(x);
    }
    T* dst = is_key ? key_cache + (int64_t)slot * kg * 8 + c * 8
                    : value_cache + (int64_t)slot * vg * 8 + (int64_t)(c - kg) * 8;
    *reinterpret_cast<uint4*>(dst) = v;
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

pa_status resolve(const pa_diff_params* p, Geometry* g) {
  if (!p) return fail(PA_ERR_INVALID_ARGUMENT, "params is NULL");
  if (p->flags & ~(PA_FLAG_AFTER_WRITE | PA_FLAG_OWN_SLOTS))
    return fail(PA_ERR_INVALID_ARGUMENT, "unknown flag bits 0x%x", p->flags);
  if (!(isfinite(p->norm_eps) && p->norm_eps >= 0.f))
    return fail(PA_ERR_INVALID_ARGUMENT, "norm_eps must be finite and >= 0");
  if (!isfinite(p->lambda_init)) return fail(PA_ERR_INVALID_ARGUMENT, "lambda_init must be finite");
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
  q.flags = p->flags;
  const pa_status s = resolve_separate(&q, g);
  if (s != PA_OK) return s;
  if (p->v_head_size < 0) return fail(PA_ERR_INVALID_ARGUMENT, "v_head_size must be >= 0");
  g->vhs = p->v_head_size == 0 ? 2 * g->hs : p->v_head_size;
  g->rms_eps = p->norm_eps;
  if (g->H > 65535)
    return fail(PA_ERR_NOT_IMPLEMENTED, "num_heads %d exceeds the supported maximum 65535", g->H);
  if (g->hs > 128 || g->vhs > 256 || g->vhs % 8 != 0 || g->H / g->kvh > 128)
    return fail(PA_ERR_NOT_IMPLEMENTED,
                "differential attention: head_size <= 128, v_head_size a multiple of 8 <= 256 "
                "and at most 128 heads per kv head (got %d, %d, %d)", g->hs, g->vhs,
                g->H / g->kvh);
  return PA_OK;
}

pa_status check_tokens(int64_t num_tokens, int32_t num_seqs, const Geometry& g) {
  if (num_tokens < 0 || num_seqs < 0)
    return fail(PA_ERR_INVALID_ARGUMENT, "num_tokens and num_seqs must be >= 0");
  if (num_tokens * (int64_t)g.H >= ((int64_t)1 << 30) || num_tokens > INT32_MAX)
    return fail(PA_ERR_INVALID_ARGUMENT, "num_tokens * num_heads must be < 2^30");
  return PA_OK;
}

pa_status read(Phase ph, const pa_diff_params* p, DiffArgs a) {
  Geometry g;
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
  if (!a.query || !a.key_cache || !a.value_cache || !a.lambda_vectors || !a.norm_weight ||
      !a.cumseq || !a.past || !a.block_table || !a.out)
    return fail(PA_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (g.rd > 0 && (!a.cos_cache || !a.sin_cache))
    return fail(PA_ERR_INVALID_ARGUMENT, "cos_cache/sin_cache are required when rotary_dim > 0");
  if (!aligned(a.query, 16) || !aligned(a.key_cache, 16) || !aligned(a.value_cache, 16) ||
      !aligned(a.norm_weight, 16) || !aligned(a.out, 16) ||
      (g.rd > 0 && (!aligned(a.cos_cache, 16) || !aligned(a.sin_cache, 16))))
    return fail(PA_ERR_INVALID_ARGUMENT, "half-precision tensors must be 16-byte aligned");
  if (!aligned(a.lambda_vectors, 4) || !aligned(a.cumseq, 4) || !aligned(a.past, 4) ||
      !aligned(a.block_table, 4) || !aligned(a.err_flags, 4))
    return fail(PA_ERR_INVALID_ARGUMENT,
                "int32 tensors and lambda_vectors must be 4-byte aligned");
  if (a.workspace && !aligned(a.workspace, 256))
    return fail(PA_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  a.lambda_init = p->lambda_init;
  a.norm_eps = p->norm_eps;
  if (ph == Phase::kDecode) {
    const size_t need = decode_workspace(g, a.seq_end - a.seq_begin);
    if (!a.workspace || a.workspace_bytes < need)
      return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed",
                  a.workspace ? a.workspace_bytes : (size_t)0, need);
  }
  const cudaError_t e = ph == Phase::kDecode ? launch_decode(g, a) : launch_prefill(g, a);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();  // not left behind for a later call
    return fail(PA_ERR_CUDA, "differential attention launch: %s", cudaGetErrorString(e));
  }
  return PA_OK;
}

}  // namespace
}  // namespace diff
}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_diff_validate(const pa_diff_params* p) {
  Geometry g;
  return diff::resolve(p, &g);
}

pa_status pa_diff_write(const pa_diff_params* p, const void* key, const void* value,
                        int64_t num_tokens, const void* cos_cache, const void* sin_cache,
                        const int32_t* slot_mapping, const int32_t* cumseq, const int32_t* past,
                        int32_t num_seqs, void* key_cache, void* value_cache, int32_t* err_flags,
                        void* stream) {
  using diff::aligned;
  using diff::fail;
  Geometry g;
  pa_status s = diff::resolve(p, &g);
  if (s == PA_OK) s = diff::check_tokens(num_tokens, num_seqs, g);
  if (s != PA_OK) return s;
  if (num_tokens == 0) return PA_OK;
  if (num_seqs < 1) return fail(PA_ERR_INVALID_ARGUMENT, "tokens given but num_seqs is 0");
  if (!key || !value || !slot_mapping || !cumseq || !past || !key_cache || !value_cache)
    return fail(PA_ERR_INVALID_ARGUMENT, "a required pointer is NULL");
  if (g.rd > 0 && (!cos_cache || !sin_cache))
    return fail(PA_ERR_INVALID_ARGUMENT, "cos_cache/sin_cache are required when rotary_dim > 0");
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(key_cache, 16) ||
      !aligned(value_cache, 16) ||
      (g.rd > 0 && (!aligned(cos_cache, 16) || !aligned(sin_cache, 16))))
    return fail(PA_ERR_INVALID_ARGUMENT, "half-precision tensors must be 16-byte aligned");
  if (!aligned(slot_mapping, 4) || !aligned(cumseq, 4) || !aligned(past, 4) ||
      !aligned(err_flags, 4))
    return fail(PA_ERR_INVALID_ARGUMENT, "int32 tensors must be 4-byte aligned");
  const int64_t groups = (int64_t)g.kvh * ((2 * g.hs + g.vhs) >> 3);
  int64_t blocks = (num_tokens * groups + 255) / 256;
  const int64_t cap = (int64_t)g.num_sms * 16;
  if (blocks > cap) blocks = cap;
  const int step_t = (int)(blocks * 256 / groups), step_c = (int)(blocks * 256 % groups);
  const size_t smem =
      num_seqs <= diff::kStagedSeqs ? (size_t)(num_seqs + 1) * sizeof(int32_t) : 0;
  auto go = [&](auto* typed) {
    using T = std::remove_pointer_t<decltype(typed)>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(
        &cfg, diff::diff_write_kernel<T>, (const T*)key, (const T*)value, (const T*)cos_cache,
        (const T*)sin_cache, slot_mapping, cumseq, past, num_seqs, (T*)key_cache,
        (T*)value_cache, num_tokens, g.kvh, g.hs, g.vhs, g.ro, g.rd, g.interleaved, g.cos_rows,
        (int64_t)g.num_blocks * g.bs, err_flags, step_t, step_c);
  };
  const cudaError_t e =
      g.dtype == PA_DTYPE_BF16 ? go((__nv_bfloat16*)nullptr) : go((__half*)nullptr);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();  // not left behind for a later call
    return fail(PA_ERR_CUDA, "differential write launch: %s", cudaGetErrorString(e));
  }
  return PA_OK;
}

pa_status pa_diff_decode(const pa_diff_params* p, const void* query, int64_t num_tokens,
                         const void* key_cache, const void* value_cache, const void* cos_cache,
                         const void* sin_cache, const float* lambda_vectors,
                         const void* norm_weight, const int32_t* cumseq, const int32_t* past,
                         const int32_t* block_table, int32_t num_seqs, int32_t seq_begin,
                         int32_t seq_end, void* workspace, size_t workspace_bytes, void* out,
                         int32_t* err_flags, void* stream) {
  return diff::read(Phase::kDecode, p,
                    diff::DiffArgs{query, num_tokens, key_cache, value_cache, cos_cache,
                                   sin_cache, lambda_vectors, norm_weight, cumseq, past,
                                   block_table, num_seqs, seq_begin, seq_end, workspace,
                                   workspace_bytes, out, err_flags, (cudaStream_t)stream, 0.f,
                                   0.f});
}

pa_status pa_diff_prefill(const pa_diff_params* p, const void* query, int64_t num_tokens,
                          const void* key_cache, const void* value_cache, const void* cos_cache,
                          const void* sin_cache, const float* lambda_vectors,
                          const void* norm_weight, const int32_t* cumseq, const int32_t* past,
                          const int32_t* block_table, int32_t num_seqs, int32_t seq_begin,
                          int32_t seq_end, void* workspace, size_t workspace_bytes, void* out,
                          int32_t* err_flags, void* stream) {
  return diff::read(Phase::kPrefill, p,
                    diff::DiffArgs{query, num_tokens, key_cache, value_cache, cos_cache,
                                   sin_cache, lambda_vectors, norm_weight, cumseq, past,
                                   block_table, num_seqs, seq_begin, seq_end, workspace,
                                   workspace_bytes, out, err_flags, (cudaStream_t)stream, 0.f,
                                   0.f});
}

size_t pa_diff_workspace_size(const pa_diff_params* p, int32_t num_seqs, int64_t num_tokens) {
  Geometry g;
  if (diff::resolve(p, &g) != PA_OK || num_seqs <= 0 || num_tokens <= 0) return 0;
  return diff::decode_workspace(g, num_seqs);
}

}  // extern "C"
