// Declarations shared by the translation units behind include/q4kv_extend.h.
#pragma once

#include "q4kv_internal.cuh"
#include "q4kv_extend.h"

namespace q4kv {

struct RotaryAppendArgs {
  PoolView pool;
  q4kv_rotary rot;
  const void *k, *v;
  int in_dtype;
  int32_t batch, max_new;
  const int32_t* n_new;
  int64_t seq_stride, token_stride;
  const void* q;      // NULL = no queries
  void* q_out;
  int32_t n_q_heads;  // 0 when q is NULL
  int64_t q_seq_stride, q_token_stride, o_seq_stride, o_token_stride;
  const int32_t* tables;
  int32_t max_blocks;
  const int32_t* seq_lens;
  const int32_t* positions;  // NULL = seq_lens[b] + i on every axis
};
cudaError_t launch_append_rotary(const RotaryAppendArgs& a, cudaStream_t stream);

struct GatherArgs {
  PoolView pool;
  const int32_t* tables;
  int32_t max_blocks, batch;
  const int32_t* starts;   // NULL = 0
  const int32_t* offsets;
  int64_t n_rows;
  void *k_out, *v_out;
  int64_t out_stride;
  int out_dtype;
  int unrotate_k;
};
cudaError_t launch_gather(const GatherArgs& a, cudaStream_t stream);

struct ExtendArgs {
  PoolView pool;
  q4kv_extend_plan plan;
  const void* q;
  int q_dtype;
  int64_t q_seq_stride, q_token_stride;
  const int32_t* tables;
  const int32_t* seq_lens;
  const int32_t* n_new;    // NULL = max_new
  float scale;
  void* out;
  int out_dtype;
  int64_t o_seq_stride, o_token_stride;
  float* ws_o;   // [splits][batch * max_new * n_q_heads][D]
  float2* ws_ml; // [splits][batch * max_new * n_q_heads] (reference maximum, sum)
};
cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t stream);

// How the chunk kernel cuts its work: a CTA takes `rows` query rows (token,
// head of the group) of one KV head; it walks their keys in tiles of `tile`
// tokens, in `streams` interleaved partial results.
struct ExtendShape {
  int rows, tile, streams;
};
inline ExtendShape extend_shape(int d, int64_t group_rows) {
  if (d == 256) return {128, 64, 1};
  return group_rows > 128 ? ExtendShape{256, 128, 1} : ExtendShape{128, 128, 2};
}

// Single-token attention over seq_lens[b] + 1 tokens by the decode kernel (api.cu).
q4kv_status one_token_attention(const q4kv_pool* pool, const q4kv_decode_plan* plan, const void* q, int32_t q_dtype,
                                const int32_t* block_tables, const int32_t* seq_lens, float softmax_scale, void* out,
                                int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream);

// Host argument checks shared with api.cu.
q4kv_status check_pool(const q4kv_pool* p);
q4kv_status check_append(const q4kv_pool* pool, const void* k, const void* v, int32_t in_dtype, int32_t batch,
                         int32_t max_new, const int32_t* n_new, int64_t seq_stride, int64_t token_stride,
                         const int32_t* tables, int32_t max_blocks, const int32_t* seq_lens, int64_t* rows);

}  // namespace q4kv
