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
  unsigned tries;  // of one wait of a block, after which it gives up
};
constexpr unsigned kTries = 1u << 24;   // seconds
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

}  // namespace q4kv
