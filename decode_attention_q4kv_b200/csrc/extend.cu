// Attention of a chunk of new tokens over the paged quantised cache.
//
// One warp per query row: a lane holds D/32 consecutive channels; keys and
// values are decoded as they are read, the softmax keeps a running maximum and
// sum in binary32.
#include <math.h>

#include "extend_internal.cuh"

namespace q4kv {
namespace {

template <int D>
__device__ __forceinline__ void load_row(const PoolView& P, bool key, int blk, int h, int slot, int lane,
                                         float (&x)[D / 32]) {
  constexpr int E = D / 32;
  const int bits = P.bits_of(blk);
  const int64_t phys = bits == 4 ? blk : (bits == 8 ? blk - P.n_q4 : blk - P.n_q4 - P.n_q8);
  const int64_t row = (phys * P.n_kv_heads + h) * kBlockTokens + slot;
  const uint8_t* codes = bits == 4 ? (key ? P.k_codes4 : P.v_codes4)
                                   : (bits == 8 ? (key ? P.k_codes8 : P.v_codes8) : (key ? P.k_codes2 : P.v_codes2));
  const __half2* params = bits == 4 ? (key ? P.k_params4 : P.v_params4)
                                    : (bits == 8 ? (key ? P.k_params8 : P.v_params8) : (key ? P.k_params2 : P.v_params2));
  codes += row * (D * bits / 8);
  float s = 1.0f, z = 0.0f;
  if (!P.fp8) {
    const __half2 p = params[row * (D / kGroup) + lane * E / kGroup];
    s = __low2float(p);
    z = __high2float(p);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lane * E + e;
    if (P.fp8) {
      __nv_fp8_e4m3 f;
      f.__x = codes[c];
      x[e] = static_cast<float>(f);
    } else {
      const int v = bits == 8 ? codes[c] : bits == 4 ? (codes[c / 2] >> (4 * (c & 1))) & 15 : (codes[c / 4] >> (2 * (c & 3))) & 3;
      x[e] = __fmaf_rn(static_cast<float>(v), s, z);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(256) extend_simple_kernel(const __grid_constant__ ExtendArgs a, int64_t n_rows) {
  constexpr int E = D / 32;
  const PoolView& P = a.pool;
  const int lane = threadIdx.x & 31;
  const int hq = a.plan.n_q_heads, g = hq / P.n_kv_heads, T = a.plan.max_new, mb = a.plan.max_blocks_per_seq;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (row >= n_rows) return;
  const int h = static_cast<int>(row % hq), i = static_cast<int>(row / hq % T), b = static_cast<int>(row / hq / T);
  const int len = a.seq_lens[b], nn = a.n_new == nullptr ? T : min(a.n_new[b], T);
  bool ok = i < nn;
  if (ok && (len < 0 || static_cast<int64_t>(len) + nn > static_cast<int64_t>(mb) * kBlockTokens)) {
    if (lane == 0) raise_error(P.error_word, Q4KV_DEVERR_SEQ_LEN);
    ok = false;
  }
  float acc[E] = {}, m = -INFINITY, l = 0.0f;
  if (ok) {
    float q[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t at = b * a.q_seq_stride + i * a.q_token_stride + static_cast<int64_t>(h) * D + lane * E + e;
      q[e] = a.q_dtype == Q4KV_F16 ? __half2float(static_cast<const __half*>(a.q)[at])
                                   : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at]);
    }
    if (P.k_rotated) {
#pragma unroll
      for (int st = 1; st < E; st <<= 1)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((e & st) == 0) {
            const float x = q[e], y = q[e + st];
            q[e] = x + y;
            q[e + st] = x - y;
          }
#pragma unroll
      for (int st = 1; st < 32; st <<= 1)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float o = __shfl_xor_sync(0xffffffffu, q[e], st);
          q[e] = lane & st ? o - q[e] : q[e] + o;
        }
#pragma unroll
      for (int e = 0; e < E; ++e) q[e] *= rotation_constant(D);
    }
    const int end = len + i;
    for (int t = a.plan.window > 0 ? max(0, end - a.plan.window + 1) : 0; t <= end; ++t) {
      const int blk = a.tables[static_cast<int64_t>(b) * mb + t / kBlockTokens];
      if (blk < 0 || blk >= P.n_blocks()) {
        if (lane == 0) raise_error(P.error_word, Q4KV_DEVERR_BLOCK_ID);
        ok = false;
        break;
      }
      const int slot = t % kBlockTokens;
      const bool gone = (P.mask[static_cast<int64_t>(blk) * kMaskWords + slot / 32] >> (slot % 32)) & 1u;
      float s = Q4KV_SENTINEL_LOGIT, x[E] = {};
      if (!gone) {
        load_row<D>(P, true, blk, h / g, slot, lane, x);
        s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += q[e] * x[e];
#pragma unroll
        for (int st = 1; st < 32; st <<= 1) s += __shfl_xor_sync(0xffffffffu, s, st);
        s *= a.scale;
        load_row<D>(P, false, blk, h / g, slot, lane, x);
      }
      const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn);
      l = l * c + p;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * c + (gone ? 0.0f : p * x[e]);
      m = mn;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t at = b * a.o_seq_stride + i * a.o_token_stride + static_cast<int64_t>(h) * D + lane * E + e;
    const float y = ok ? acc[e] / l : 0.0f;
    if (a.out_dtype == Q4KV_F32) static_cast<float*>(a.out)[at] = y;
    else if (a.out_dtype == Q4KV_F16) static_cast<__half*>(a.out)[at] = __float2half_rn(y);
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
  }
}

}  // namespace

cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.plan.batch) * a.plan.max_new * a.plan.n_q_heads;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (a.plan.head_dim == 128) extend_simple_kernel<128><<<grid, 256, 0, stream>>>(a, rows);
  else extend_simple_kernel<256><<<grid, 256, 0, stream>>>(a, rows);
  return cudaGetLastError();
}

}  // namespace q4kv
