/*
 * pa_diff.h — C ABI of differential attention over paged caches.
 *
 * A third attention mode beside the LATENT and SEPARATE layouts of
 * pa_latent.h: every head has two query and key maps and one value, and
 * attends with the difference of the two softmax maps. For token t at
 * position pos of its sequence, head h, kv head g = h / (H / kvH):
 *
 *   q_i   = RoPE(query[t, h, i]),  K_i,j = key_cache[row j, g, i]      i = 0, 1
 *   s_i,j = scale * q_i . K_i,j, then softcap * tanh(s / softcap) if softcap > 0
 *           over the keys j = 0..pos (with a window: pos - j <= window)
 *   o     = sum_j (softmax(s_0)_j - lambda * softmax(s_1)_j) V_j[g]
 *   out[t, h] = (1 - lambda_init) * norm_weight * o / sqrt(mean(o^2) + norm_eps)
 *
 * with the learned scalar of the layer
 *
 *   lambda = exp(v[0] . v[1]) - exp(v[2] . v[3]) + lambda_init,
 *   v = lambda_vectors float32 [4, hs].
 *
 * Layouts (H heads, kvH kv heads, hs channels per map, vhs per value):
 *   query [T, H, 2, hs]   key [T, kvH, 2, hs]   value [T, kvH, vhs]
 *   key_cache [num_blocks, bs, kvH, 2, hs]   value_cache [num_blocks, bs, kvH, vhs]
 *   out [T, H, vhs]   norm_weight [vhs]   (all in the query dtype)
 * Index tensors, paging, the write and read phases, streams, graphs, status
 * codes, err_flags and ownership are those of pa_latent.h; the pages can be
 * kept by the operators of pa_pages.h.
 *
 * Arithmetic: products accumulate in f32; softmax, lambda, the difference
 * and the norm are f32; out is rounded once. Operands of the products: keys
 * and values as they are; the rotated query and the probabilities as two
 * 16-bit parts each (value and remainder), so that the difference of the two
 * maps is as exact as its own rounding. In fp16 a probability is off by 2^-34
 * of the row's largest at most: where the largest has a value near zero (an
 * attention sink), that holds for others down to about 2^-22 of it.
 */
#ifndef PA_DIFF_H
#define PA_DIFF_H

#include "pa_latent.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pa_diff_params {
  int32_t dtype;              /* pa_dtype of every half-precision tensor             */
  int32_t num_heads;          /* H heads (2 H query maps), at most 65535             */
  int32_t kv_num_heads;       /* kvH >= 1, dividing H; H / kvH <= 128                */
  int32_t head_size;          /* hs, channels per map: multiple of 16, 16..128       */
  int32_t v_head_size;        /* vhs: multiple of 8, 8..256; 0 means 2 * hs          */
  int32_t rotary_offset;      /* as pa_latent_params, within each map                */
  int32_t rotary_dim;
  int32_t rotary_interleaved;
  int32_t cos_rows;
  int32_t block_size;
  int32_t num_blocks;
  int32_t max_blocks_per_seq;
  float scale;                /* 0 selects 1/sqrt(hs)                                */
  float softcap;
  int32_t local_window_size;
  float lambda_init;          /* finite                                              */
  float norm_eps;             /* finite, >= 0                                        */
  int32_t flags;              /* PA_FLAG_AFTER_WRITE / PA_FLAG_OWN_SLOTS             */
} pa_diff_params;

pa_status pa_diff_validate(const pa_diff_params* p);

/* Write phase: for every token t with slot_mapping[t] >= 0 and kv head g,
 *   key_cache[slot, g, i] = RoPE(key[t, g, i]), rounded to the dtype;
 *   value_cache[slot, g]  = value[t, g].
 * Arguments and errors as pa_separate_write. */
pa_status pa_diff_write(const pa_diff_params* p, const void* key, const void* value,
                        int64_t num_tokens, const void* cos_cache, const void* sin_cache,
                        const int32_t* slot_mapping, const int32_t* cumseq, const int32_t* past,
                        int32_t num_seqs, void* key_cache, void* value_cache, int32_t* err_flags,
                        void* stream);

/* Read phase for sequences [seq_begin, seq_end): decode takes one new token
 * per sequence, prefill any number. lambda_vectors is 4-byte, the other
 * tensors 16-byte aligned. The rest as pa_latent_decode / pa_latent_prefill:
 * the workspace is pa_diff_workspace_size bytes, rows of a sequence with
 * invalid positions or pages are zeros (in prefill those of the tokens that
 * meet one, and of tokens up to 128 / (H / kvH) beside them), those of a
 * decode sequence with another number of new tokens stay as they were.
 * What a token does not see (later tokens, rows before its window or behind
 * its sequence, pages of others) may hold infinities or NaN; one in what it
 * sees may make all of its row NaN. */
pa_status pa_diff_decode(const pa_diff_params* p, const void* query, int64_t num_tokens,
                         const void* key_cache, const void* value_cache, const void* cos_cache,
                         const void* sin_cache, const float* lambda_vectors,
                         const void* norm_weight, const int32_t* cumseq, const int32_t* past,
                         const int32_t* block_table, int32_t num_seqs, int32_t seq_begin,
                         int32_t seq_end, void* workspace, size_t workspace_bytes, void* out,
                         int32_t* err_flags, void* stream);
pa_status pa_diff_prefill(const pa_diff_params* p, const void* query, int64_t num_tokens,
                          const void* key_cache, const void* value_cache, const void* cos_cache,
                          const void* sin_cache, const float* lambda_vectors,
                          const void* norm_weight, const int32_t* cumseq, const int32_t* past,
                          const int32_t* block_table, int32_t num_seqs, int32_t seq_begin,
                          int32_t seq_end, void* workspace, size_t workspace_bytes, void* out,
                          int32_t* err_flags, void* stream);

/* Workspace bytes a decode or prefill call over at most num_seqs sequences
 * and num_tokens tokens needs on the current device; 0 for invalid
 * parameters. */
size_t pa_diff_workspace_size(const pa_diff_params* p, int32_t num_seqs, int64_t num_tokens);

#ifdef __cplusplus
}
#endif

#endif /* PA_DIFF_H */
