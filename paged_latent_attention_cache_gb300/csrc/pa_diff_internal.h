// Internal interface of the differential-attention kernels: pa_diff.cu
// (entry points, write phase) and its read kernels. The public interface is
// include/pa_diff.h.
#pragma once

#include "pa_diff.h"
#include "pa_internal.h"

namespace pa {
namespace diff {

// Arguments of one read call. In Geometry, H and kvh count heads (not maps),
// hs is the width of one map and vhs the value's.
struct DiffArgs {
  const void* query;
  int64_t num_tokens;
  const void* key_cache;
  const void* value_cache;
  const void* cos_cache;
  const void* sin_cache;
  const float* lambda_vectors;
  const void* norm_weight;
  const int32_t* cumseq;
  const int32_t* past;
  const int32_t* block_table;
  int32_t num_seqs, seq_begin, seq_end;
  void* workspace;
  size_t workspace_bytes;
  void* out;
  int32_t* err_flags;
  cudaStream_t stream;
  float lambda_init, norm_eps;
};

// decode (pa_diff_decode.cu); workspace bytes for nseq sequences
size_t decode_workspace(const Geometry& g, int64_t nseq);
cudaError_t launch_decode(const Geometry& g, const DiffArgs& a);
// prefill (pa_diff_prefill.cu); needs no workspace
cudaError_t launch_prefill(const Geometry& g, const DiffArgs& a);

}  // namespace diff
}  // namespace pa
