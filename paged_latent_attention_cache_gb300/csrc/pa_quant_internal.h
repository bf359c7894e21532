// Internal interface of the kernels over 8-bit caches: pa_quant.cu (entry
// points, write phase, reading back) and its read kernels. The public interface
// is include/pa_quant.h.
#pragma once

#include "pa_internal.h"
#include "pa_quant.h"

namespace pa {
namespace quant {

// Arguments of one read call.
struct QuantArgs {
  const void* query;
  int64_t num_tokens;
  const uint8_t* key_cache;
  const uint8_t* value_cache;
  const float2* scales;
  const void* cos_cache;
  const void* sin_cache;
  const void* q_norm;     // optional
  const void* head_sink;  // optional
  const int32_t* cumseq;
  const int32_t* past;
  const int32_t* block_table;
  int32_t num_seqs, seq_begin, seq_end;
  void* workspace;
  size_t workspace_bytes;
  void* out;
  int32_t* err_flags;
  cudaStream_t stream;
  int cross;
};

// Few query rows per sequence (pa_quant_decode.cu): decode, and prefill of a few
// tokens (sequences of at most `few`); workspace bytes for nseq sequences
size_t rows_workspace(const Geometry& g, int64_t nseq);
cudaError_t launch_rows(const Geometry& g, const QuantArgs& a, bool decode, int32_t few);
// prefill (pa_quant_prefill.cu), which hands few rows to launch_rows; workspace bytes
size_t prefill_workspace(const Geometry& g, int64_t nseq);
cudaError_t launch_prefill(const Geometry& g, const QuantArgs& a);

}  // namespace quant
}  // namespace pa
