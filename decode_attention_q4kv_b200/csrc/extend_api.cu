// Host side of include/q4kv_extend.h: argument checks, launch plans and
// dispatch.  Every check happens before anything is enqueued.
#include <math.h>
#include <string.h>

#include "extend_internal.cuh"

using namespace q4kv;

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
inline q4kv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? Q4KV_OK : Q4KV_ERR_CUDA; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// A [batch][max_new] array of rows of `row` elements of `size` bytes.
bool rows_ok(const void* p, int64_t seq_stride, int64_t token_stride, int64_t row, int size) {
  return p != nullptr && aligned(p, 16) && seq_stride >= 0 && token_stride >= row && (seq_stride * size) % 16 == 0 &&
         (token_stride * size) % 16 == 0;
}

// No two rows of such an array share memory (token_stride >= row).  Sequence
// after sequence and token after token are seen at once; other interleavings
// row by row: rows b and i apart by less than a row's length in one axis come
// back by a whole number of steps of the other.
bool rows_apart(int64_t seq_stride, int64_t token_stride, int64_t row, int64_t batch, int64_t max_new) {
  if (batch <= 1 || seq_stride >= (max_new - 1) * token_stride + row) return true;
  if (seq_stride >= row && token_stride >= (batch - 1) * seq_stride + row) return true;
  if (seq_stride < row) return false;
  for (int64_t b = 1; b < batch; ++b) {
    const int64_t at = b * seq_stride, i = at / token_stride;   // neighbours of sequence b's first row
    if (i < max_new && at - i * token_stride < row) return false;
    if (i + 1 < max_new && (i + 1) * token_stride - at < row) return false;
  }
  return true;
}

// The checks every call makes of its pool (q4kv_block_image_stride makes them
// and computes a size on the host).
q4kv_status check_pool(const q4kv_pool* pool) {
  size_t stride;
  return q4kv_block_image_stride(pool, &stride);
}
bool has_blocks(const q4kv_pool* pool) { return pool->n_q4_blocks + pool->n_q8_blocks + pool->n_q2_blocks > 0; }

}  // namespace

extern "C" {

q4kv_status q4kv_append_rotary(const q4kv_pool* pool, const q4kv_rotary* rotary, const void* k, const void* v,
                               int32_t in_dtype, int32_t batch, int32_t max_new, const int32_t* n_new,
                               int64_t seq_stride, int64_t token_stride, const void* q, int32_t n_q_heads,
                               int64_t q_seq_stride, int64_t q_token_stride, void* q_out, int64_t q_out_seq_stride,
                               int64_t q_out_token_stride, const int32_t* tables, int32_t max_blocks,
                               const int32_t* seq_lens, const int32_t* positions, void* stream) {
  const q4kv_status st = check_pool(pool);
  if (st != Q4KV_OK) return st;
  if (batch < 0 || max_new < 0 || (in_dtype != Q4KV_F16 && in_dtype != Q4KV_BF16)) return Q4KV_ERR_INVALID_ARG;
  const bool rows = batch > 0 && max_new > 0;
  if (rows) {
    const int64_t row = static_cast<int64_t>(pool->n_kv_heads) * pool->head_dim;
    if (!rows_ok(k, seq_stride, token_stride, row, 2) || !rows_ok(v, seq_stride, token_stride, row, 2) || !has_blocks(pool) ||
        tables == nullptr || !aligned(tables, 4) || max_blocks < 1 || seq_lens == nullptr || !aligned(seq_lens, 4) ||
        (n_new != nullptr && !aligned(n_new, 4)))
      return Q4KV_ERR_INVALID_ARG;
  }
  if (rotary == nullptr || (rotary->interleaved != 0 && rotary->interleaved != 1) || rotary->n_axes < 1 ||
      rotary->n_axes > Q4KV_MAX_AXES || rotary->max_positions < 1 || rotary->rot_dim < 32 || rotary->rot_dim % 32 != 0 ||
      rotary->rot_dim > pool->head_dim || rotary->table == nullptr || !aligned(rotary->table, 16))
    return Q4KV_ERR_INVALID_ARG;
  for (int f = 0; f < rotary->rot_dim / 2; ++f)
    if (rotary->axis[f] >= rotary->n_axes) return Q4KV_ERR_INVALID_ARG;
  if (positions != nullptr && !aligned(positions, 4)) return Q4KV_ERR_INVALID_ARG;
  RotaryAppendArgs a;
  a.q = nullptr;
  a.q_out = nullptr;
  a.n_q_heads = 0;
  a.q_seq_stride = a.q_token_stride = a.o_seq_stride = a.o_token_stride = 0;
  if (q != nullptr) {
    if (n_q_heads < 1) return Q4KV_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(n_q_heads) * pool->head_dim;
    if (!rows_ok(q, q_seq_stride, q_token_stride, row, 2) ||
        !rows_ok(q_out, q_out_seq_stride, q_out_token_stride, row, 2))
      return Q4KV_ERR_INVALID_ARG;
    if (!rows_apart(q_out_seq_stride, q_out_token_stride, row, batch, max_new)) return Q4KV_ERR_INVALID_ARG;
    if (q == q_out && (q_seq_stride != q_out_seq_stride || q_token_stride != q_out_token_stride))
      return Q4KV_ERR_INVALID_ARG;
    a.q = q;
    a.q_out = q_out;
    a.n_q_heads = n_q_heads;
    a.q_seq_stride = q_seq_stride;
    a.q_token_stride = q_token_stride;
    a.o_seq_stride = q_out_seq_stride;
    a.o_token_stride = q_out_token_stride;
  }
  if (!rows) return Q4KV_OK;
  a.pool = view_of(*pool);
  a.rot = *rotary;
  a.k = k;
  a.v = v;
  a.in_dtype = in_dtype;
  a.batch = batch;
  a.max_new = max_new;
  a.n_new = n_new;
  a.seq_stride = seq_stride;
  a.token_stride = token_stride;
  a.tables = tables;
  a.max_blocks = max_blocks;
  a.seq_lens = seq_lens;
  a.positions = positions;
  return from_cuda(launch_append_rotary(a, as_stream(stream)));
}

q4kv_status q4kv_gather_tokens(const q4kv_pool* pool, const int32_t* tables, int32_t max_blocks, int32_t batch,
                               const int32_t* starts, const int32_t* offsets, int64_t n_rows, void* k_out, void* v_out,
                               int64_t out_stride, int32_t out_dtype, int32_t unrotate_k, void* stream) {
  const q4kv_status st = check_pool(pool);
  if (st != Q4KV_OK) return st;
  if ((out_dtype != Q4KV_F32 && out_dtype != Q4KV_F16 && out_dtype != Q4KV_BF16) || batch < 0 || n_rows < 0 ||
      n_rows > 0x7fffffff || (unrotate_k != 0 && unrotate_k != 1))
    return Q4KV_ERR_INVALID_ARG;
  const int size = out_dtype == Q4KV_F32 ? 4 : 2;
  if (out_stride < static_cast<int64_t>(pool->n_kv_heads) * pool->head_dim || (out_stride * size) % 16 != 0)
    return Q4KV_ERR_INVALID_ARG;
  if (n_rows == 0 || batch == 0) return Q4KV_OK;
  if (tables == nullptr || !aligned(tables, 4) || max_blocks < 1 || offsets == nullptr || !aligned(offsets, 4) ||
      (starts != nullptr && !aligned(starts, 4)) || k_out == nullptr || v_out == nullptr || !aligned(k_out, 16) ||
      !aligned(v_out, 16))
    return Q4KV_ERR_INVALID_ARG;
  // keys' and values' rows may lie between one another, not on one another
  const uintptr_t row = static_cast<uintptr_t>(pool->n_kv_heads) * pool->head_dim * size, step = static_cast<uintptr_t>(out_stride) * size;
  const uintptr_t ka = reinterpret_cast<uintptr_t>(k_out), va = reinterpret_cast<uintptr_t>(v_out);
  const uintptr_t apart = ka < va ? va - ka : ka - va;
  if (apart < static_cast<uintptr_t>(n_rows - 1) * step + row && (apart % step < row || step - apart % step < row))
    return Q4KV_ERR_INVALID_ARG;
  GatherArgs a;
  a.pool = view_of(*pool);
  a.tables = tables;
  a.max_blocks = max_blocks;
  a.batch = batch;
  a.starts = starts;
  a.offsets = offsets;
  a.n_rows = n_rows;
  a.k_out = k_out;
  a.v_out = v_out;
  a.out_stride = out_stride;
  a.out_dtype = out_dtype;
  a.unrotate_k = unrotate_k;
  return from_cuda(launch_gather(a, as_stream(stream)));
}

// One new token per sequence is what the decode kernel does; it reads the codes
// without turning them into fp16 tiles.
static bool one_token(int32_t max_new, int32_t window, int g, int32_t head_dim) {
  return max_new == 1 && window == 0 && g <= 8 && g * head_dim <= 1024;
}

constexpr int64_t kMaxTokens = 32768;

// decode_splits < 0 lets the decode planner choose from num_sms.
static q4kv_status make_plan(int32_t batch, int32_t max_new, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                             int32_t max_blocks, int32_t window, int32_t n_splits, int32_t decode_splits,
                             int32_t num_sms, q4kv_extend_plan* plan) {
  if (plan == nullptr || batch < 0 || max_new < 0 || n_q_heads < 1 || n_kv_heads < 1 || max_blocks < 1 || window < 0 ||
      n_splits < 0 || num_sms < 0 || n_q_heads % n_kv_heads != 0 || batch > 65535 || n_kv_heads > 65535)
    return Q4KV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_blocks) * kBlockTokens > 0x7fffffff ||
      static_cast<int64_t>(batch) * max_new * n_q_heads > 0x7fffffff)
    return Q4KV_ERR_INVALID_ARG;
  if (head_dim != 128 && head_dim != 256) return Q4KV_ERR_UNSUPPORTED;
  const int g = n_q_heads / n_kv_heads;
  if (g > 64) return Q4KV_ERR_UNSUPPORTED;
  if (num_sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return Q4KV_ERR_CUDA;
  }
  const int64_t group_rows = static_cast<int64_t>(max_new) * g;
  const ExtendShape sh = extend_shape(head_dim, group_rows);
  // the most keys a row tile can see, in steps of the streams together
  int64_t ctx = static_cast<int64_t>(max_blocks) * kBlockTokens;
  if (window > 0) ctx = min(ctx, static_cast<int64_t>(window) + (sh.rows + g - 1) / g + sh.tile);
  const int64_t step = static_cast<int64_t>(sh.tile) * sh.streams;
  const int64_t steps = (ctx + step - 1) / step;
  // An accumulator takes at most kMaxTokens tokens: the tensor cores cut off what they
  // add up in binary32, so a sum of one sign falls short by 6e-9 of itself for every token.
  // (Values of mean 4 over 524288 tokens in one accumulator came out 3.2e-3 too small,
  // over 131072 8.1e-4, over 32768 2.0e-4; a rounding to fp16 is 4.9e-4 at most.)
  const int64_t smin = (steps * sh.tile + kMaxTokens - 1) / kMaxTokens;
  int64_t s = n_splits;
  if (s == 0) {
    // Time in SM cycles: CTAs (one per SM at a time), each with its key tiles and
    // what starting and ending it costs, and the partial results written and
    // read again.  The figures are fitted to times measured with forced split
    // counts: 4200 cycles a step of 128 tokens x 256 rows, 5000 of 256 x 128 (4300 of 256 x 32),
    // 2400 of 64 x 128 (heads of 256), 27000 a CTA, 3300 bytes a cycle.
    // Sequences of one length run in waves; of several, a CTA that ends early
    // makes room for the next (three quarters of the work, and half of the last
    // CTA's as a tail).  Which it will be is not known here, so a batch is
    // planned for the mean of both.
    const double step_cycles = head_dim == 256 ? 2400.0 : sh.rows == 256 ? 4200.0 : group_rows <= 32 ? 4300.0 : 5000.0;
    const double partial_cycles = static_cast<double>(batch) * max_new * n_q_heads * head_dim * 8.0 / 3300.0 * sh.streams;
    const int64_t items = max(int64_t{1}, static_cast<int64_t>(batch) * n_kv_heads * ((group_rows + sh.rows - 1) / sh.rows));
    double best = 1e300;
    s = smin;
    for (int64_t cand = smin; cand <= max(smin, min(steps, int64_t{4} * num_sms)); ++cand) {
      const int64_t per = (steps + cand - 1) / cand;
      if ((steps + per - 1) / per != cand) continue;
      const double one = per * step_cycles + 27000.0;
      double cost = static_cast<double>((items * cand + num_sms - 1) / num_sms) * one;
      if (batch > 1) {
        const double part = static_cast<double>(items * cand) / num_sms * (0.75 * per * step_cycles + 27000.0) + 0.5 * one;
        cost = 0.5 * (cost + max(part, one));
      }
      if (cand * sh.streams > 1) cost += cand * partial_cycles + 6000.0;
      if (cost < best - 1e-9) {
        best = cost;
        s = cand;
      }
    }
  }
  s = max(smin, min(s, steps));
  const int64_t per = (steps + s - 1) / s;
  s = (steps + per - 1) / per;
  memset(plan, 0, sizeof(*plan));
  plan->batch = batch;
  plan->max_new = max_new;
  plan->n_q_heads = n_q_heads;
  plan->n_kv_heads = n_kv_heads;
  plan->head_dim = head_dim;
  plan->max_blocks_per_seq = max_blocks;
  plan->window = window;
  plan->n_splits = static_cast<int32_t>(s);
  const int64_t partials = s * sh.streams;
  if (partials > 1) {
    const size_t rows = static_cast<size_t>(batch) * max_new * n_q_heads * partials;
    plan->workspace_bytes = round_up(rows * head_dim * sizeof(float), 256) + round_up(rows * sizeof(float2), 256);
  }
  if (one_token(max_new, window, g, head_dim)) {
    q4kv_decode_plan d;
    const q4kv_status st = q4kv_decode_plan_make(batch, n_q_heads, n_kv_heads, head_dim, max_blocks,
                                                 decode_splits < 0 ? 0 : decode_splits, num_sms, &d);
    if (st != Q4KV_OK) return st;
    plan->decode_splits = d.n_splits;
    plan->workspace_bytes = max(plan->workspace_bytes, d.workspace_bytes);
  } else if (decode_splits > 0) {
    return Q4KV_ERR_INVALID_ARG;
  }
  return Q4KV_OK;
}

q4kv_status q4kv_extend_plan_make(int32_t batch, int32_t max_new, int32_t n_q_heads, int32_t n_kv_heads,
                                  int32_t head_dim, int32_t max_blocks_per_seq, int32_t window, int32_t n_splits,
                                  int32_t num_sms, q4kv_extend_plan* plan) {
  return make_plan(batch, max_new, n_q_heads, n_kv_heads, head_dim, max_blocks_per_seq, window, n_splits, -1, num_sms,
                   plan);
}

// tries: of one wait of the chunk kernel (the decode kernel takes no such limit).
static q4kv_status extend_attention(const q4kv_pool* pool, const q4kv_extend_plan* plan, const void* q, int32_t q_dtype,
                                    int64_t q_seq_stride, int64_t q_token_stride, const int32_t* block_tables,
                                    const int32_t* seq_lens, const int32_t* n_new, float softmax_scale, void* out,
                                    int32_t out_dtype, int64_t out_seq_stride, int64_t out_token_stride, void* workspace,
                                    size_t workspace_bytes, unsigned tries, void* stream) {
  q4kv_status st = check_pool(pool);
  if (st != Q4KV_OK) return st;
  if (plan == nullptr) return Q4KV_ERR_INVALID_ARG;
  // the plan must be one q4kv_extend_plan_make would produce for this pool
  q4kv_extend_plan ref;
  if (plan->n_splits < 1) return Q4KV_ERR_INVALID_ARG;
  st = make_plan(plan->batch, plan->max_new, plan->n_q_heads, plan->n_kv_heads, plan->head_dim,
                 plan->max_blocks_per_seq, plan->window, plan->n_splits, plan->decode_splits, 1, &ref);
  if (st != Q4KV_OK) return st;
  if (plan->head_dim != pool->head_dim || plan->n_kv_heads != pool->n_kv_heads || ref.n_splits != plan->n_splits ||
      ref.decode_splits != plan->decode_splits || ref.workspace_bytes != plan->workspace_bytes)
    return Q4KV_ERR_INVALID_ARG;
  if ((q_dtype != Q4KV_F16 && q_dtype != Q4KV_BF16) ||
      (out_dtype != Q4KV_F32 && out_dtype != Q4KV_F16 && out_dtype != Q4KV_BF16) || !isfinite(softmax_scale))
    return Q4KV_ERR_INVALID_ARG;
  if (plan->batch == 0 || plan->max_new == 0) return Q4KV_OK;
  const int64_t row = static_cast<int64_t>(plan->n_q_heads) * plan->head_dim;
  if (!rows_ok(q, q_seq_stride, q_token_stride, row, 2) ||
      !rows_ok(out, out_seq_stride, out_token_stride, row, out_dtype == Q4KV_F32 ? 4 : 2))
    return Q4KV_ERR_INVALID_ARG;
  if (!rows_apart(out_seq_stride, out_token_stride, row, plan->batch, plan->max_new)) return Q4KV_ERR_INVALID_ARG;
  if (block_tables == nullptr || !aligned(block_tables, 4) || seq_lens == nullptr || !aligned(seq_lens, 4) ||
      (n_new != nullptr && !aligned(n_new, 4)))
    return Q4KV_ERR_INVALID_ARG;
  if (!has_blocks(pool)) return Q4KV_ERR_INVALID_ARG;
  if (plan->workspace_bytes > 0 &&
      (workspace == nullptr || workspace_bytes < plan->workspace_bytes || !aligned(workspace, 256)))
    return Q4KV_ERR_WORKSPACE;
  const float scale = softmax_scale > 0.0f ? softmax_scale : 1.0f / sqrtf(static_cast<float>(plan->head_dim));
  // (the decode kernel wants aligned tables and numbers rows of codes in 32 bits)
  const int64_t widest = max(pool->n_q4_blocks, max(pool->n_q8_blocks, pool->n_q2_blocks));
  if (tries == kTries && plan->decode_splits > 0 && n_new == nullptr && (plan->batch == 1 || (q_seq_stride == row && out_seq_stride == row)) &&
      aligned(block_tables, 16) && widest * pool->n_kv_heads * kBlockTokens < (int64_t{1} << 31)) {
    q4kv_decode_plan d;
    st = q4kv_decode_plan_make(plan->batch, plan->n_q_heads, plan->n_kv_heads, plan->head_dim, plan->max_blocks_per_seq,
                               plan->decode_splits, 1, &d);
    if (st != Q4KV_OK) return st;
    DecodeArgs a = {};
    a.pool = view_of(*pool);
    a.plan = d;
    a.q = q;
    a.q_dtype = q_dtype;
    a.tables = block_tables;
    a.seq_lens = seq_lens;
    a.add_const = 1;                       // the sequence with its new token
    a.scale = scale;
    a.out = out;
    a.out_dtype = out_dtype;
    a.ws_o = static_cast<float*>(workspace);
    if (d.workspace_bytes > 0) {
      const size_t partials = static_cast<size_t>(d.batch) * d.n_q_heads * d.n_splits;
      a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + round_up(partials * d.head_dim * sizeof(float), 256));
    }
    return from_cuda(launch_decode(a, as_stream(stream)));
  }
  ExtendArgs a;
  a.pool = view_of(*pool);
  a.plan = *plan;
  a.q = q;
  a.q_dtype = q_dtype;
  a.q_seq_stride = q_seq_stride;
  a.q_token_stride = q_token_stride;
  a.tables = block_tables;
  a.seq_lens = seq_lens;
  a.n_new = n_new;
  a.scale = scale;
  a.out = out;
  a.out_dtype = out_dtype;
  a.o_seq_stride = out_seq_stride;
  a.o_token_stride = out_token_stride;
  a.tries = tries;
  a.ws_o = static_cast<float*>(workspace);
  const size_t partial_rows = static_cast<size_t>(plan->batch) * plan->max_new * plan->n_q_heads * plan->n_splits *
                              extend_shape(plan->head_dim, static_cast<int64_t>(plan->max_new) *
                                                               (plan->n_q_heads / plan->n_kv_heads)).streams;
  a.ws_ml = plan->workspace_bytes > 0
                ? reinterpret_cast<float2*>(static_cast<char*>(workspace) +
                                            round_up(partial_rows * plan->head_dim * sizeof(float), 256))
                : nullptr;
  return from_cuda(launch_extend(a, as_stream(stream)));
}

q4kv_status q4kv_extend_attention(const q4kv_pool* pool, const q4kv_extend_plan* plan, const void* q, int32_t q_dtype,
                                  int64_t q_seq_stride, int64_t q_token_stride, const int32_t* block_tables,
                                  const int32_t* seq_lens, const int32_t* n_new, float softmax_scale, void* out,
                                  int32_t out_dtype, int64_t out_seq_stride, int64_t out_token_stride, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return extend_attention(pool, plan, q, q_dtype, q_seq_stride, q_token_stride, block_tables, seq_lens, n_new,
                          softmax_scale, out, out_dtype, out_seq_stride, out_token_stride, workspace, workspace_bytes,
                          kTries, stream);
}

q4kv_status q4kv_selftest_extend_wait(const q4kv_pool* pool, const q4kv_extend_plan* plan, const void* q,
                                      int32_t q_dtype, int64_t q_seq_stride, int64_t q_token_stride,
                                      const int32_t* block_tables, const int32_t* seq_lens, const int32_t* n_new,
                                      float softmax_scale, void* out, int32_t out_dtype, int64_t out_seq_stride,
                                      int64_t out_token_stride, void* workspace, size_t workspace_bytes, int32_t tries,
                                      void* stream) {
  if (tries < 0 || static_cast<unsigned>(tries) >= kTries) return Q4KV_ERR_INVALID_ARG;
  return extend_attention(pool, plan, q, q_dtype, q_seq_stride, q_token_stride, block_tables, seq_lens, n_new,
                          softmax_scale, out, out_dtype, out_seq_stride, out_token_stride, workspace, workspace_bytes,
                          static_cast<unsigned>(tries), stream);
}

}  // extern "C"
