/*
 * q4kv_extend.h -- growing a cached prompt by a chunk of tokens: rotary
 * positions and quantisation in one write, attention of the chunk over the
 * paged cache, and reading token ranges back.  Part of libq4kv.so; pools,
 * formats, status codes, error bits and conventions are those of q4kv.h.
 *
 * [AMBP] sec. 2.1 item 4 (a prompt that extends a cached prefix, an EXTEND
 * match, grows the cache instead of being prefilled again) is the path these
 * serve: q4kv_append_rotary writes the chunk, q4kv_extend_attention attends
 * from it, q4kv_gather_tokens hands cached tokens on.
 */
#ifndef Q4KV_EXTEND_H
#define Q4KV_EXTEND_H

#include "q4kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Q4KV_MAX_AXES 4
#define Q4KV_MAX_PAIRS 128

/* A further bit of pool->error_word. */
#define Q4KV_DEVERR_POSITION 64u /* a rotary position outside [0, max_positions) */

/*
 * Rotary positions.  The first rot_dim channels of a head form rot_dim / 2
 * pairs (a, b): channels (f, f + rot_dim/2), or (2f, 2f + 1) when interleaved.
 * Pair f is turned by the angle whose (cos, sin) is table[p][f], p being the
 * token's position on axis[f] (time, height, width, ...; one axis for text):
 *   a' = fl(fl(a c) - fl(b s)),  b' = fl(fl(b c) + fl(a s))
 * in binary32, rounded once (to nearest even) to the input's 16-bit type.
 * The channels from rot_dim on pass unchanged.
 */
typedef struct {
  int32_t rot_dim;       /* a multiple of 32, 32 <= rot_dim <= head_dim */
  int32_t interleaved;   /* 0 or 1 */
  int32_t n_axes;        /* 1 .. Q4KV_MAX_AXES */
  int32_t max_positions; /* rows of table, >= 1 */
  const float *table;    /* device [max_positions][rot_dim/2][2], 16-byte aligned */
  uint8_t axis[Q4KV_MAX_PAIRS]; /* axis of each pair, < n_axes; entries from rot_dim/2 on are ignored */
} q4kv_rotary;

/*
 * Rotate the new tokens' keys (and queries) by their positions and quantise
 * keys and values into the pool as they are written, in one launch.  The pool
 * receives exactly the bytes q4kv_append_tokens would write for the rotated
 * 16-bit keys.
 *   k, v, in_dtype, batch, max_new, n_new, seq_stride, token_stride, tables,
 *   max_blocks, seq_lens   as for q4kv_append_tokens
 *   q            device, in_dtype, or NULL (then q_out is ignored): the
 *                [n_q_heads][D] row of token i of sequence b at element
 *                b*q_seq_stride + i*q_token_stride
 *   q_out        the rotated queries, same type, its own strides; may be q
 *                itself with equal strides, and overlap it in no other way
 *   positions    device int32 [n_axes][batch][max_new], or NULL: token i of
 *                sequence b is at seq_lens[b] + i on every axis
 * q, q_out and the strides keep the alignment rules of k and v; no two rows of
 * q_out may share memory.  q_out rows of tokens at or past n_new[b] are written
 * as 0.  A token whose position lies
 * outside the table raises Q4KV_DEVERR_POSITION; it is not cached and its
 * q_out row is 0, as for a length or block id out of range.
 */
q4kv_status q4kv_append_rotary(const q4kv_pool *pool, const q4kv_rotary *rotary, const void *k, const void *v,
                               int32_t in_dtype, int32_t batch, int32_t max_new, const int32_t *n_new,
                               int64_t seq_stride, int64_t token_stride, const void *q, int32_t n_q_heads,
                               int64_t q_seq_stride, int64_t q_token_stride, void *q_out, int64_t q_out_seq_stride,
                               int64_t q_out_token_stride, const int32_t *tables, int32_t max_blocks,
                               const int32_t *seq_lens, const int32_t *positions, void *stream);

/*
 * Read token ranges back through the block tables, packed.
 *   tables       device int32 [batch][max_blocks]
 *   starts       device int32 [batch], first token read of each sequence;
 *                NULL = 0
 *   offsets      device int32 [batch + 1], non-decreasing: rows
 *                offsets[b] .. offsets[b+1] - 1 are the tokens of sequence b
 *                from starts[b] on
 *   n_rows       rows of k_out and v_out; rows outside [offsets[0],
 *                offsets[batch]) are left as they were
 *   k_out, v_out device [n_rows][Hkv][D] of out_dtype (F32, F16 or BF16),
 *                16-byte aligned, rows out_stride elements apart
 *                (out_stride >= Hkv*D, a multiple of 16 bytes); no row of one
 *                may share memory with a row of the other
 * Values as for q4kv_dequantize (x = fl(code*s + z), rounded once; keys
 * un-rotated when unrotate_k is 1 and the pool stores them rotated; remapped
 * slots read K = -1e4, V = 0).  A token outside its table, or in a block whose
 * id is out of range, reads 0 and raises Q4KV_DEVERR_SEQ_LEN or
 * Q4KV_DEVERR_BLOCK_ID.
 */
q4kv_status q4kv_gather_tokens(const q4kv_pool *pool, const int32_t *tables, int32_t max_blocks, int32_t batch,
                               const int32_t *starts, const int32_t *offsets, int64_t n_rows, void *k_out, void *v_out,
                               int64_t out_stride, int32_t out_dtype, int32_t unrotate_k, void *stream);

/*
 * Launch plan of one chunk shape: batch sequences of up to max_new new tokens
 * each over tables of max_blocks_per_seq blocks.  The keys that a tile of query
 * rows sees are cut into n_splits equal ranges whose partial results are merged
 * by log-sum-exp.
 */
typedef struct {
  int32_t batch;
  int32_t max_new;
  int32_t n_q_heads;
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t max_blocks_per_seq;
  int32_t window;           /* 0 = none */
  int32_t n_splits;
  int32_t decode_splits;    /* splits of the single-token kernel; 0 where it does not apply */
  int32_t reserved;         /* 0 */
  size_t workspace_bytes;   /* device scratch a call needs (may be 0) */
} q4kv_extend_plan;

/*
 * Fill `plan`.  n_splits > 0 forces that split count, clamped to the context and
 * to what keeps a partial result at 32768 tokens or less (the tensor cores' sums fall
 * short by up to 2^-12 of themselves over so many, and by more over more);
 * 0 lets the library choose from num_sms (0 = those of the current device).
 * Supported: head_dim 128 or 256, 1 <= n_q_heads / n_kv_heads <= 64.
 */
q4kv_status q4kv_extend_plan_make(int32_t batch, int32_t max_new, int32_t n_q_heads, int32_t n_kv_heads,
                                  int32_t head_dim, int32_t max_blocks_per_seq, int32_t window, int32_t n_splits,
                                  int32_t num_sms, q4kv_extend_plan *plan);

/*
 * Attention of each sequence's new tokens over its cache, which already holds
 * them (q4kv_append_tokens or q4kv_append_rotary ran before).
 *   q            device, q_dtype Q4KV_F16 or Q4KV_BF16: the [n_q_heads][D] row
 *                of token i of sequence b at element b*q_seq_stride +
 *                i*q_token_stride; 16-byte aligned, strides multiples of 16
 *                bytes, q_token_stride >= n_q_heads*D
 *   seq_lens     device int32 [batch], lengths BEFORE the new tokens
 *   n_new        device int32 [batch], 0 <= n_new[b] <= max_new; NULL =
 *                max_new for every sequence
 *   block_tables device int32 [batch][max_blocks_per_seq]
 *   out          as q, of out_dtype (F32, F16 or BF16), its own strides; no
 *                two of its rows may share memory, nor may it overlap q
 *   softmax_scale <= 0 selects 1/sqrt(D); the scaled queries and the logits
 *                have to be finite in binary32
 *   workspace    as for q4kv_decode_attention
 * Token i of sequence b sees the positions t <= seq_lens[b] + i and, with
 * plan->window > 0, t > seq_lens[b] + i - window.  Remapped slots have logit
 * -1e4 and value 0 as in q4kv_decode_attention; a token that sees remapped
 * slots only returns 0.  Rows at or past n_new[b] are written as 0.  Keys and
 * values are rounded to fp16 for the tensor cores, by at most 2^-11 of their size
 * (2^-25 where they are below 2^-14).  Where the rounded scale carries a finite
 * group past the largest fp16 value, it is lowered by one step, which moves the
 * group's values by at most 2^-10 of its range.  A token with a key or value
 * that is not finite in fp16 even so reaches no row that does not see it; the
 * rows that do become NaN, as does a row whose query is not finite.
 * One new token per sequence (max_new == 1, no window, n_new NULL, rows next to
 * each other) takes the kernel of q4kv_decode_attention, with its accuracy;
 * there a length of -1 is an empty sequence (row 0, no error bit), and queries, keys
 * and values have to be finite.
 * A sequence longer than its table raises Q4KV_DEVERR_SEQ_LEN, a block id out
 * of range Q4KV_DEVERR_BLOCK_ID; the affected rows are written as 0.
 */
q4kv_status q4kv_extend_attention(const q4kv_pool *pool, const q4kv_extend_plan *plan, const void *q, int32_t q_dtype,
                                  int64_t q_seq_stride, int64_t q_token_stride, const int32_t *block_tables,
                                  const int32_t *seq_lens, const int32_t *n_new, float softmax_scale, void *out,
                                  int32_t out_dtype, int64_t out_seq_stride, int64_t out_token_stride, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * Diagnostic: q4kv_extend_attention by the chunk kernel with `tries` (0 <= tries
 * < 2^24, the kernel's own limit) tries of each wait inside it before the block
 * gives up.  Where one gives up, the block's rows are written as 0 and
 * Q4KV_DEVERR_TIMEOUT is raised; with 0 every block counts as having given up.
 */
q4kv_status q4kv_selftest_extend_wait(const q4kv_pool *pool, const q4kv_extend_plan *plan, const void *q,
                                      int32_t q_dtype, int64_t q_seq_stride, int64_t q_token_stride,
                                      const int32_t *block_tables, const int32_t *seq_lens, const int32_t *n_new,
                                      float softmax_scale, void *out, int32_t out_dtype, int64_t out_seq_stride,
                                      int64_t out_token_stride, void *workspace, size_t workspace_bytes, int32_t tries,
                                      void *stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4KV_EXTEND_H */
