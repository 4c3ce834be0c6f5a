// pa_ops.h - internal launch interface of the operators around the cache: the
// rotary cache write, attention with score modifiers, the commit of a drafted
// tree and the eviction.  Not installed; not part of the public ABI.
#pragma once

#include "pa_kernels.h"

namespace pa {

struct RopeArgs {
  void* q_out;
  int64_t q_out_stride;
  const void* q;
  int64_t q_stride;
  int num_heads;
  const float* inv_freq;
  const int64_t* positions;
  int rotary_dim;
  int interleaved;
  float rope_scale;
  ReshapeArgs w;  // the cache write: k, v, caches, slots, quantisation
};

cudaError_t launch_rope_and_cache(const RopeArgs& a, cudaStream_t stream);

// A pa_status: PA_ERR_WORKSPACE before anything is enqueued, or that of the launches.
int launch_attend(AttendParams p, void* workspace, size_t workspace_bytes, cudaStream_t stream);
// (size_t)-1 when the device cannot be asked
size_t attend_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                              int max_blocks_per_seq, int max_q_len, int kv_dtype, bool accumulate);

struct CommitArgs {
  void* k_cache;
  void* v_cache;
  int64_t num_blocks;
  int row_bytes;
  const int32_t* block_tables;
  int max_blocks_per_seq;
  const int32_t* seq_lens;
  const int32_t* q_starts;
  const int32_t* path;
  const int32_t* path_lens;
  int max_path;
  int32_t* new_lens;
  int num_seqs, num_kv_heads, block_size, block_shift;
  unsigned int* err;
};
cudaError_t launch_commit_tree(const CommitArgs& a, cudaStream_t stream);

struct EvictArgs {
  void* k_cache;
  void* v_cache;
  int64_t num_blocks;
  int row_bytes;
  const float* mass;
  int64_t mass_stride_seq, mass_stride_head;
  const int32_t* block_tables;
  int max_blocks_per_seq;
  const int32_t* seq_lens;
  const int32_t* dst_tables;
  int max_dst_blocks;
  int32_t* kept;
  float* mass_out;
  int32_t* new_lens;
  int num_seqs, num_kv_heads, block_size, block_shift;
  int budget, recent, sinks;
  unsigned int* err;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace pa
