/*
 * pa_quant.h — C ABI of grouped-query and cross attention over paged caches
 * held in 8 bits.
 *
 * The 8-bit form of the SEPARATE mode of pa_latent.h: keys and values are
 * E4M3 codes ("e4m3fn", one byte per channel), and every page has a scale for
 * each kv head and cache, a power of two. A channel's value is code * scale.
 *
 *   key_cache   uint8   [num_blocks, bs, kvH, hs]    codes
 *   value_cache uint8   [num_blocks, bs, kvH, vhs]   codes
 *   scales      float32 [num_blocks, kvH, 2]         of keys and of values
 *
 * A scale is 2^e with e in -48..48, or 0 where its page has none yet (any
 * other value counts as 0). The rows of a page without one are zeros, whatever
 * their codes. A page's scales belong to the page: pa_pages.h carries them along
 * as a tensor of PA_PAGE_WHOLE.
 *
 * Write: for page p and kv head g, x = the rows of the call in that page (keys:
 * after RMSNorm and RoPE, in f32; values as they are), and of either cache
 *
 *   need  = the least 2^e, -48 <= e <= 48, with |x| <= 448 * 2^e for every
 *           finite x (2^48 where that is not enough)
 *   old   = scales[p, g], or 0 if the call writes row 0 of the page
 *   scale = max(old, need)
 *   codes of the call's rows      = e4m3(x / scale)
 *   codes of the page's other rows = e4m3(code * old / scale)  if 0 < old < scale
 *
 * with e4m3 rounding to nearest even, saturated to +-448; NaN stays NaN, an
 * infinity becomes +-448. So a page is filled from its row 0 on by as many
 * calls as it takes, and its scale grows with what is appended.
 *
 * Read: as in the SEPARATE mode, s_j = scale * q . K_j over the keys a token
 * sees, softcap, softmax with an optional sink logit, sum_j p_j V_j. With
 * `cross` 0, those are the keys at positions 0..pos (with a window: pos - j <=
 * window). With `cross` 1 a token sees all past[b] cached rows and nothing of
 * its own: attention to an encoder's states, which pa_quant_write has stored
 * once (past[b] is their number then, the tokens have no position). A token
 * that sees no key answers zeros.
 *
 * Layouts (H heads, kvH kv heads, hs and vhs channels per key and value):
 *   query [T, H, hs]   key [T, kvH, hs]   value [T, kvH, vhs]   out [T, H, vhs]
 * Index tensors, paging, streams, graphs, status codes, err_flags, alignment
 * and ownership are those of pa_latent.h (scales: 8-byte aligned).
 *
 * Arithmetic: products accumulate in f32, softmax is f32, out is rounded once.
 * Operands of the products are fp16 whatever the dtype: codes exactly, the
 * query times a power of two that brings its row's largest channel to 2^14
 * (11 bits of each channel, none lost down to 2^-28 of the largest; with fp16
 * out and rotation or norm, which leave more than 11 bits, two addends: 22),
 * probabilities times the values' scales relative to the row's largest such
 * product (11 bits, down to 2^-22 of it; 2^-33 of it at worst below).
 */
#ifndef PA_QUANT_H
#define PA_QUANT_H

#include "pa_latent.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pa_quant_params {
  int32_t dtype;              /* pa_dtype of every half-precision tensor             */
  int32_t num_heads;          /* H query heads, at most 65535                        */
  int32_t kv_num_heads;       /* kvH >= 1, dividing H; H / kvH <= 128                */
  int32_t head_size;          /* hs: multiple of 16, 16..256                         */
  int32_t v_head_size;        /* vhs: multiple of 16, 16..256; 0 means hs            */
  int32_t rotary_offset;      /* as pa_latent_params; no rotation with cross         */
  int32_t rotary_dim;
  int32_t rotary_interleaved;
  int32_t cos_rows;
  int32_t block_size;         /* bs: power of two, 16..4096                          */
  int32_t num_blocks;
  int32_t max_blocks_per_seq;
  float scale;                /* 0 selects 1/sqrt(hs)                                */
  float softcap;
  int32_t local_window_size;  /* < 0 with cross                                      */
  float rms_eps;              /* RMSNorm epsilon (used when a norm weight is given)  */
  int32_t cross;              /* 1: tokens see the cached rows and none of their own */
  int32_t flags;              /* PA_FLAG_AFTER_WRITE / PA_FLAG_OWN_SLOTS             */
} pa_quant_params;

/* PA_FLAG_OWN_SLOTS is accepted and changes nothing here: every read waits for
 * the write before its first cache row. (A write may change all rows and the scale
 * of a page that it appends to, so rows below past[b] are not untouched by it.) */

pa_status pa_quant_validate(const pa_quant_params* p);

/* Write phase, as defined above. Arguments and errors as pa_separate_write,
 * and: slot_mapping[t] is a row of the same number in its page as token t's
 * position has (slot % bs == position % bs), and the tokens of one sequence
 * whose positions lie in one page share a page; a token that breaks either
 * sets PA_DEVERR_SLOT and is skipped. A page is named by tokens of one
 * sequence and one page of positions only, in a call. (An encoder's states are written as a sequence's tokens from past 0.) */
pa_status pa_quant_write(const pa_quant_params* p, const void* key, const void* value,
                         int64_t num_tokens, const void* cos_cache, const void* sin_cache,
                         const void* k_norm_weight, const int32_t* slot_mapping,
                         const int32_t* cumseq, const int32_t* past, int32_t num_seqs,
                         void* key_cache, void* value_cache, float* scales, int32_t* err_flags,
                         void* stream);

/* Reads rows back: for every token t of sequence b, the cached row at position
 * past[b] + t - cumseq[b], code * scale rounded to the dtype (saturated to its
 * largest value).
 *   key [num_tokens, kvH*hs], value [num_tokens, kvH*vhs]   output, either may
 *   be NULL
 * Rows of a position outside the table or of an invalid page are zeros
 * (PA_DEVERR_CONTEXT, PA_DEVERR_BLOCK); rows behind cumseq[num_seqs] stay as
 * they were (PA_DEVERR_CUMSEQ). */
pa_status pa_quant_restore(const pa_quant_params* p, const void* key_cache,
                           const void* value_cache, const float* scales, const int32_t* cumseq,
                           const int32_t* past, const int32_t* block_table, int32_t num_seqs,
                           int64_t num_tokens, void* key, void* value, int32_t* err_flags,
                           void* stream);

/* Read phase for sequences [seq_begin, seq_end): decode takes one new token
 * per sequence, prefill any number. Arguments, errors and the rows written as
 * pa_separate_decode / pa_separate_prefill; both need a workspace of
 * pa_quant_workspace_size bytes. Rows of a sequence with invalid positions are
 * zeros, as are the rows of tokens that meet an invalid page (in prefill also of
 * tokens up to 256 / (H / kvH) beside them). What a token does not see (later
 * tokens, rows before its window or behind its sequence, pages of others) may
 * hold NaN codes and any scales; a NaN in what it sees may make all of its row
 * NaN. */
pa_status pa_quant_decode(const pa_quant_params* p, const void* query, int64_t num_tokens,
                          const void* key_cache, const void* value_cache, const float* scales,
                          const void* cos_cache, const void* sin_cache, const void* q_norm_weight,
                          const void* head_sink, const int32_t* cumseq, const int32_t* past,
                          const int32_t* block_table, int32_t num_seqs, int32_t seq_begin,
                          int32_t seq_end, void* workspace, size_t workspace_bytes, void* out,
                          int32_t* err_flags, void* stream);
pa_status pa_quant_prefill(const pa_quant_params* p, const void* query, int64_t num_tokens,
                           const void* key_cache, const void* value_cache, const float* scales,
                           const void* cos_cache, const void* sin_cache,
                           const void* q_norm_weight, const void* head_sink,
                           const int32_t* cumseq, const int32_t* past, const int32_t* block_table,
                           int32_t num_seqs, int32_t seq_begin, int32_t seq_end, void* workspace,
                           size_t workspace_bytes, void* out, int32_t* err_flags, void* stream);

/* One step of a serving batch in one call: pa_quant_write over all tokens, then
 * pa_quant_decode over sequences [0, num_decode_seqs) and pa_quant_prefill over the
 * rest, with the flags of a read that follows the write. Not with cross. */
pa_status pa_quant_mixed(const pa_quant_params* p, const void* query, const void* key,
                         const void* value, int64_t num_tokens, const void* cos_cache,
                         const void* sin_cache, const void* q_norm_weight,
                         const void* k_norm_weight, const void* head_sink,
                         const int32_t* slot_mapping, const int32_t* cumseq, const int32_t* past,
                         const int32_t* block_table, int32_t num_seqs, int32_t num_decode_seqs,
                         void* key_cache, void* value_cache, float* scales, void* workspace,
                         size_t workspace_bytes, void* out, int32_t* err_flags, void* stream);

/* Workspace bytes a decode or prefill call over at most num_seqs sequences
 * and num_tokens tokens needs on the current device; 0 for invalid
 * parameters. */
size_t pa_quant_workspace_size(const pa_quant_params* p, int32_t num_seqs, int64_t num_tokens);

#ifdef __cplusplus
}
#endif

#endif /* PA_QUANT_H */
