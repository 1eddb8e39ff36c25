// Rotary positions and quantisation of a chunk of new tokens in one launch.
//
// Pair (a, b) of a head, frequency f, at position p on the pair's axis, with
// (c, s) = table[p][f]:
//   a' = fl(fl(a c) - fl(b s)),  b' = fl(fl(b c) + fl(a s)),
// one IEEE binary32 operation each, rounded once to the 16-bit input type.
// The rotated key then takes the encoder's steps (encode.cuh), so the pool
// receives the bytes an append of the rotated 16-bit row writes.
//
// A warp item is one new token and `per` consecutive groups of VPW heads: the
// key/value groups first, then the query groups.  A lane holds 16 channels of
// one head, as in the encoder; its channels, and so its pairs' angles, are the
// same in every group, so the (cos, sin) row is read once per item.  With
// pairs (f, f + rot/2) the partner channels sit in another lane of the same
// head and come as 8 shuffles of the raw 16-bit words.
//
// Bound by latency: each item looks up its length, block, positions and angles
// before it can turn a row.  A half-pair lane holds 16 (cos, sin), 32 registers
// beside the encoder's; an interleaved one 8.  So interleaved pairs ask for 3
// blocks of 256 threads per SM and half pairs for 2 (at 3 they spill 356 and 564
// bytes with heads of 128).  Measured, L2 flushed before each call, us at 2 / at 3 blocks:
//   4 x 2048 tokens, 32/8 heads of 128, fp16     half 65.6 / 73.7   interleaved 59.4 / 56.3
//   the same on three axes                       half 73.8 / 82.9   interleaved 67.6 / 63.6
//   1 x 8191 tokens, 16/8 heads of 256, bf16     half 82.5 / 92.7   interleaved 77.8 / 73.7
//   4 x 512 tokens, 32/8 heads of 128, fp16      half 26.7 / 35.7   interleaved 22.7 / 26.6
// (of interleaved pairs the last goes the other way).
// 8-bit, 2-bit and raw-key blocks and bf16 take the same within 3 %, E4M3 59.5.
// 1 x 8191 moves 220 MB at 2.7 TB/s (34 us at the copy bandwidth; issue 43 %, 22 % of
// the warps resident).  Keys and values loaded before the look-ups: 132 us (155 registers).
#include "encode.cuh"
#include "extend_internal.cuh"

namespace q4kv {
namespace {

__device__ __forceinline__ uint32_t pack2(__half, float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(__half, uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 unpack2(__nv_bfloat16, uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// A lane's share of the rotation: its pairs' (cos, +-sin).
struct Turn {
  float2 cs[kEPL];
  int partner;      // lane that holds the partner channels
  bool on;          // the lane's channels are rotated
};

template <typename InT, bool INTER>
__device__ __forceinline__ void turn_words(uint32_t (&w)[8], const Turn& t) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = unpack2(InT(), w[i]);
      const float c = t.cs[i].x, s = t.cs[i].y;
      const float a = __fsub_rn(__fmul_rn(x.x, c), __fmul_rn(x.y, s));
      const float b = __fadd_rn(__fmul_rn(x.y, c), __fmul_rn(x.x, s));
      if (t.on) w[i] = pack2(InT(), a, b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t o = __shfl_sync(0xffffffffu, w[i], t.partner);
      const float2 x = unpack2(InT(), w[i]), y = unpack2(InT(), o);
      // the sign of the sine is the lane's: -s for a', +s for b'
      const float lo = __fadd_rn(__fmul_rn(x.x, t.cs[2 * i].x), __fmul_rn(y.x, t.cs[2 * i].y));
      const float hi = __fadd_rn(__fmul_rn(x.y, t.cs[2 * i + 1].x), __fmul_rn(y.y, t.cs[2 * i + 1].y));
      if (t.on) w[i] = pack2(InT(), lo, hi);
    }
  }
}

// FIXED: nothing writes the row during the launch.  (Queries may be rotated in place.)
template <bool FIXED>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[8]) {
  const uint4* u = static_cast<const uint4*>(p);
  const uint4 a = FIXED ? __ldg(u) : u[0], b = FIXED ? __ldg(u + 1) : u[1];
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

template <int D, typename InT, bool ROT, bool INTER>
__global__ void __launch_bounds__(256, INTER ? 3 : 2) append_rotary_kernel(const __grid_constant__ RotaryAppendArgs a, int per) {
  using S = Shape<D>;
  griddep_wait();
  griddep_launch_dependents();
  const PoolView& pool = a.pool;
  const int lane = threadIdx.x & 31;
  const int r = lane / S::LPV, j = lane % S::LPV;
  const int hkv = pool.n_kv_heads, hq = a.n_q_heads;
  const int kv_groups = (hkv + S::VPW - 1) / S::VPW, groups = kv_groups + (hq + S::VPW - 1) / S::VPW;
  const int parts = (groups + per - 1) / per;
  const int64_t n_items = static_cast<int64_t>(a.batch) * a.max_new * parts;
  const int64_t n_warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;

  // the lane's pairs: first frequency, sign, partner lane, axes (2 bits each)
  constexpr int kPairs = INTER ? kEPL / 2 : kEPL;
  const int half = a.rot.rot_dim / 2;
  Turn t;
  t.on = j * kEPL < a.rot.rot_dim;
  const bool second = !INTER && j * kEPL >= half;
  t.partner = !t.on || INTER ? lane : (second ? lane - half / kEPL : lane + half / kEPL);
  const int f0 = !t.on ? 0 : (INTER ? j * (kEPL / 2) : (second ? j * kEPL - half : j * kEPL));
  uint32_t axes = 0;
#pragma unroll
  for (int e = 0; e < kPairs; ++e) axes |= static_cast<uint32_t>(a.rot.axis[f0 + e] & 3) << (2 * e);

  for (int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; item < n_items;
       item += n_warps) {
    const int part = static_cast<int>(item % parts);
    const int64_t bi = item / parts;
    const int i = static_cast<int>(bi % a.max_new);
    const int b = static_cast<int>(bi / a.max_new);
    const bool real = a.n_new == nullptr || i < __ldg(a.n_new + b);
    const int len = __ldg(a.seq_lens + b);
    const int64_t p = static_cast<int64_t>(len) + i;
    bool ok = real;
    uint32_t err = 0;
    int32_t blk = -1;
    if (len < 0 || p >= static_cast<int64_t>(a.max_blocks) * kBlockTokens) {
      ok = false;
      err = Q4KV_DEVERR_SEQ_LEN;
    } else {
      blk = __ldg(a.tables + static_cast<int64_t>(b) * a.max_blocks + p / kBlockTokens);
      if (blk < 0 || blk >= pool.n_blocks()) {
        ok = false;
        err = Q4KV_DEVERR_BLOCK_ID;
      }
    }
    int pos[Q4KV_MAX_AXES];
#pragma unroll
    for (int x = 0; x < Q4KV_MAX_AXES; ++x) {
      pos[x] = 0;
      if (x < a.rot.n_axes && real) {
        const int64_t q = a.positions == nullptr
                              ? p
                              : __ldg(a.positions + (static_cast<int64_t>(x) * a.batch + b) * a.max_new + i);
        if (q < 0 || q >= a.rot.max_positions) {
          ok = false;
          err |= Q4KV_DEVERR_POSITION;
        } else {
          pos[x] = static_cast<int>(q);
        }
      }
    }
    if (!ok) {                                   // warp-uniform
      if (real && lane == 0 && part == 0) raise_error(pool.error_word, err);
    } else if (t.on) {
      const float2* tab = reinterpret_cast<const float2*>(a.rot.table);
      if (a.rot.n_axes == 1) {
        const float4* row = reinterpret_cast<const float4*>(tab + static_cast<int64_t>(pos[0]) * half + f0);
#pragma unroll
        for (int e = 0; e < kPairs / 2; ++e) {
          const float4 x = __ldg(row + e);
          t.cs[2 * e] = make_float2(x.x, x.y);
          t.cs[2 * e + 1] = make_float2(x.z, x.w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          const uint32_t x = (axes >> (2 * e)) & 3u;
          const int pe = x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3];
          t.cs[e] = __ldg(tab + static_cast<int64_t>(pe) * half + f0 + e);
        }
      }
      if (!INTER && !second) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) t.cs[e].y = -t.cs[e].y;
      }
    }

    const int g0 = part * per, g1 = min(groups, (part + 1) * per);
    // queries: a group's row is on its way while the one before is turned
    const int q0 = max(g0, kv_groups);
    if (q0 < g1) {
      const InT* src = static_cast<const InT*>(a.q) + b * a.q_seq_stride + i * a.q_token_stride + j * kEPL;
      InT* dst = static_cast<InT*>(a.q_out) + b * a.o_seq_stride + i * a.o_token_stride + j * kEPL;
      // (lanes past the last head load and store nothing)
      auto head = [&](int g) { return (g - kv_groups) * S::VPW + r; };
      uint32_t w[8] = {}, next[8] = {};
      if (ok && head(q0) < hq) load_words<false>(src + static_cast<int64_t>(head(q0)) * D, next);
#pragma unroll 1
      for (int gi = q0; gi < g1; ++gi) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = next[e];
        if (ok && gi + 1 < g1 && head(gi + 1) < hq) load_words<false>(src + static_cast<int64_t>(head(gi + 1)) * D, next);
        if (ok) turn_words<InT, INTER>(w, t);
        if (head(gi) < hq) {
          uint4* o = reinterpret_cast<uint4*>(dst + static_cast<int64_t>(head(gi)) * D);
          o[0] = make_uint4(w[0], w[1], w[2], w[3]);
          o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    }
    if (!ok) continue;
    for (int gi = g0; gi < min(g1, kv_groups); ++gi) {
      const int slot = static_cast<int>(p % kBlockTokens);
      const int h = gi * S::VPW + r;
      const bool valid = h < hkv;
      const int hs = valid ? h : hkv - 1;
      const int64_t src = b * a.seq_stride + i * a.token_stride + static_cast<int64_t>(hs) * D + j * kEPL;
      uint32_t wk[8], wv[8];
      load_words<true>(static_cast<const InT*>(a.k) + src, wk);
      load_words<true>(static_cast<const InT*>(a.v) + src, wv);
      turn_words<InT, INTER>(wk, t);
      float2 xk[8], xv[8];
      unpack16<InT>(make_uint4(wk[0], wk[1], wk[2], wk[3]), make_uint4(wk[4], wk[5], wk[6], wk[7]), xk);
      unpack16<InT>(make_uint4(wv[0], wv[1], wv[2], wv[3]), make_uint4(wv[4], wv[5], wv[6], wv[7]), xv);
      const int bits = pool.bits_of(blk);
      const bool is8 = bits == 8;
      const int64_t phys = bits == 4 ? blk : (is8 ? blk - pool.n_q4 : blk - pool.n_q4 - pool.n_q8);
      const int64_t row = (phys * hkv + hs) * kBlockTokens + slot;   // (block, head, slot)
      if (pool.fp8) {
        if (valid) {
          store_fp8(xk, pool.k_codes8 + row * D + j * kEPL);
          store_fp8(xv, pool.v_codes8 + row * D + j * kEPL);
        }
      } else {
        if (ROT) rotate_pairs<D>(xk, j);
        constexpr float ks = ROT ? kRotScale<D> : 1.0f;
        if (is8)
          encode_kv<8>(xk, ks, xv, j, valid, pool.k_codes8 + row * D, pool.k_params8 + row * S::NG,
                       pool.v_codes8 + row * D, pool.v_params8 + row * S::NG);
        else if (bits == 2)
          encode_kv<2>(xk, ks, xv, j, valid, pool.k_codes2 + row * (D / 4), pool.k_params2 + row * S::NG,
                       pool.v_codes2 + row * (D / 4), pool.v_params2 + row * S::NG);
        else
          encode_kv<4>(xk, ks, xv, j, valid, pool.k_codes4 + row * (D / 2), pool.k_params4 + row * S::NG,
                       pool.v_codes4 + row * (D / 2), pool.v_params4 + row * S::NG);
      }
      if (lane == 0 && gi == 0)
        atomicAnd(pool.mask + static_cast<int64_t>(blk) * kMaskWords + slot / 32, ~(1u << (slot % 32)));
    }
  }
}

}  // namespace

cudaError_t launch_append_rotary(const RotaryAppendArgs& a, cudaStream_t stream) {
  const int d = a.pool.head_dim;
  const int vpw = d == 128 ? Shape<128>::VPW : Shape<256>::VPW;
  const int groups = (a.pool.n_kv_heads + vpw - 1) / vpw + (a.n_q_heads + vpw - 1) / vpw;
  const int64_t tokens = static_cast<int64_t>(a.batch) * a.max_new;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 148;
  int per = 1;
  while (per < groups && tokens * ((groups + per - 1) / per) > static_cast<int64_t>(sms) * 32) ++per;
  const int64_t items = tokens * ((groups + per - 1) / per);
  int64_t g = (items + 7) / 8;                   // 8 warps per CTA
  if (g > static_cast<int64_t>(sms) * 8) g = static_cast<int64_t>(sms) * 8;
  const dim3 grid(static_cast<unsigned>(g)), block(256);
#define Q4KV_AR(DD, T, R, I) return launch_pdl(append_rotary_kernel<DD, T, R, I>, grid, block, 0, stream, a, per)
#define Q4KV_ARI(DD, T)                                    \
  if (a.pool.k_rotated && a.rot.interleaved) Q4KV_AR(DD, T, true, true);   \
  if (a.pool.k_rotated) Q4KV_AR(DD, T, true, false);       \
  if (a.rot.interleaved) Q4KV_AR(DD, T, false, true);      \
  Q4KV_AR(DD, T, false, false)
  if (d == 128 && a.in_dtype == Q4KV_F16) { Q4KV_ARI(128, __half); }
  if (d == 128) { Q4KV_ARI(128, __nv_bfloat16); }
  if (a.in_dtype == Q4KV_F16) { Q4KV_ARI(256, __half); }
  Q4KV_ARI(256, __nv_bfloat16);
#undef Q4KV_ARI
#undef Q4KV_AR
}

}  // namespace q4kv
