// Reading token ranges back through the block tables, packed.
//
// Row n of the output is token starts[b] + n - offsets[b] of the sequence b
// with offsets[b] <= n < offsets[b + 1]; x = fl(code s + z), keys optionally
// through c H x, rounded once.
//
// A warp takes VPW consecutive rows and `per` heads of them: where its rows lie
// is looked up once, then it walks the heads.  A lane holds 16 channels of one
// row as 8 pairs (p, p + 8), as the encoder does, so that the rotation's
// butterflies are packed binary32 operations.  Codes become floats two at a time
// through fp16 (0x64xx is 1024 + xx: a mask, an or and a subtraction, exact);
// integer conversions would go through the special-function unit at a quarter
// of the rate.
//
// Bound by memory: 10 x 32768 tokens of 8 heads of 128, a quarter of the blocks
// 8-bit, to fp16 with the keys un-rotated take 350 us, 5.1 TB/s of the 1.8 GB that
// have to move (0.80 of the copy bandwidth; 322 us, 0.87, in a short run).  In short
// runs it was 483 us with one head per look-up and integer conversions, 404 us
// without the codes of the next head on their way, 348 us at 3 blocks per SM instead of 4.
#include "encode.cuh"
#include "extend_internal.cuh"

namespace q4kv {
namespace {

__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ __half2 code_half2(uint32_t v, uint32_t mask, float scale) {
  // the masked field of each half, times `scale`, exactly
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(mask), "r"(0x64006400u));
  if (scale == 1.0f) return __hsub2(as_half2(d), __float2half2_rn(1024.0f));
  return __hfma2(as_half2(d), __float2half2_rn(scale), __float2half2_rn(-1024.0f * scale));
}

// The lane's packed codes of one row, W words.
template <int BITS>
struct Codes {
  uint32_t w[BITS / 2];
};
template <int BITS>
__device__ __forceinline__ Codes<BITS> load_codes(const uint8_t* row, int j) {
  Codes<BITS> c;
  if (BITS == 2) {
    c.w[0] = __ldg(reinterpret_cast<const uint32_t*>(row) + j);
  } else if (BITS == 4) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(row) + j);
    c.w[0] = u.x;
    c.w[1 % (BITS / 2)] = u.y;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(row) + j);
    c.w[0] = u.x;
    c.w[1 % (BITS / 2)] = u.y;
    c.w[2 % (BITS / 2)] = u.z;
    c.w[3 % (BITS / 2)] = u.w;
  }
  return c;
}

// fl(code s + z) of channel pairs (p, p + 8).
template <int BITS>
__device__ __forceinline__ void to_values(const Codes<BITS>& c, __half2 sz, float2 (&x)[8]) {
  const float s = __low2float(sz), z = __high2float(sz);
  const float2 s2 = make_float2(s, s), z2 = make_float2(z, z);
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    __half2 h;
    if (BITS == 4) {
      // codes 0-3 (or 4-7) of the first 8 channels in one half, of the last 8 in the other
      const uint32_t v = __byte_perm(c.w[0], c.w[1 % (BITS / 2)], p < 4 ? 0x5410 : 0x7632) >> (8 * ((p & 3) >> 1));
      h = code_half2(v, p & 1 ? 0x00F000F0u : 0x000F000Fu, p & 1 ? 0.0625f : 1.0f);
    } else if (BITS == 2) {
      const uint32_t v = c.w[0] >> (p < 4 ? 0 : 8);
      h = code_half2(v, 0x00030003u << (2 * (p & 3)), 1.0f / static_cast<float>(1 << (2 * (p & 3))));
    } else {
      const uint32_t b = p & 3;
      const uint32_t v = __byte_perm(c.w[(p >> 2) % (BITS / 2)], c.w[(2 + (p >> 2)) % (BITS / 2)], b | b << 4 | (4 + b) << 8 | (4 + b) << 12);
      h = code_half2(v, 0x00FF00FFu, 1.0f);
    }
    x[p] = __ffma2_rn(__half22float2(h), s2, z2);
  }
}
__device__ __forceinline__ void fp8_values(const Codes<8>& c, float2 (&x)[8]) {
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const uint32_t b = p & 3;
    const uint32_t v = __byte_perm(c.w[p >> 2], c.w[2 + (p >> 2)], b | (4 + b) << 4);
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xFFFFu), __NV_E4M3);
    x[p] = __half22float2(*reinterpret_cast<const __half2*>(&h));
  }
}

template <typename OutT>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack_out<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack_out<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename OutT>
__device__ __forceinline__ void store_pairs(OutT* dst, const float2 (&x)[8]) {
  uint4* d = reinterpret_cast<uint4*>(dst);
  d[0] = make_uint4(pack_out<OutT>(x[0].x, x[1].x), pack_out<OutT>(x[2].x, x[3].x), pack_out<OutT>(x[4].x, x[5].x),
                    pack_out<OutT>(x[6].x, x[7].x));
  d[1] = make_uint4(pack_out<OutT>(x[0].y, x[1].y), pack_out<OutT>(x[2].y, x[3].y), pack_out<OutT>(x[4].y, x[5].y),
                    pack_out<OutT>(x[6].y, x[7].y));
}
template <>
__device__ __forceinline__ void store_pairs<float>(float* dst, const float2 (&x)[8]) {
  float4* d = reinterpret_cast<float4*>(dst);
  d[0] = make_float4(x[0].x, x[1].x, x[2].x, x[3].x);
  d[1] = make_float4(x[4].x, x[5].x, x[6].x, x[7].x);
  d[2] = make_float4(x[0].y, x[1].y, x[2].y, x[3].y);
  d[3] = make_float4(x[4].y, x[5].y, x[6].y, x[7].y);
}

// Heads h0 .. h1 - 1 of the lane's row: decode, un-rotate, store.  The codes of
// the next head are on their way while one is worked on.
template <int D, typename OutT, int BITS, bool FP8>
__device__ __forceinline__ void heads(const PoolView& pool, int64_t phys, int slot, int j, int h0, int h1, bool ok, bool masked,
                                      bool turn, bool write, OutT* kd, OutT* vd) {
  constexpr int NG = D / kGroup;
  constexpr int64_t kHeadCodes = static_cast<int64_t>(kBlockTokens) * (D / 8 * BITS), kHeadParams = kBlockTokens * NG;
  const int64_t row = (phys * pool.n_kv_heads + h0) * kBlockTokens + slot;
  const uint8_t* kc = (BITS == 4 ? pool.k_codes4 : BITS == 8 ? pool.k_codes8 : pool.k_codes2) + row * (D / 8 * BITS);
  const uint8_t* vc = (BITS == 4 ? pool.v_codes4 : BITS == 8 ? pool.v_codes8 : pool.v_codes2) + row * (D / 8 * BITS);
  const __half2* kp = (BITS == 4 ? pool.k_params4 : BITS == 8 ? pool.k_params8 : pool.k_params2) + row * NG + (j >> 2);
  const __half2* vp = (BITS == 4 ? pool.v_params4 : BITS == 8 ? pool.v_params8 : pool.v_params2) + row * NG + (j >> 2);
  Codes<BITS> nk = {}, nv = {};
  __half2 nsk = {}, nsv = {};
  auto fetch = [&]() {
    nk = load_codes<BITS>(kc, j);
    nv = load_codes<BITS>(vc, j);
    kc += kHeadCodes;
    vc += kHeadCodes;
    if (!FP8) {
      nsk = __ldg(kp);
      nsv = __ldg(vp);
      kp += kHeadParams;
      vp += kHeadParams;
    }
  };
  if (ok) fetch();
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const Codes<BITS> ck = nk, cv = nv;
    const __half2 sk = nsk, sv = nsv;
    if (ok && h + 1 < h1) fetch();
    float2 x[8];
    if (FP8) fp8_values(*reinterpret_cast<const Codes<8>*>(&ck), x);
    else to_values<BITS>(ck, sk, x);
    if (turn) {
      rotate_pairs<D>(x, j);
      if (kRotScale<D> != 1.0f) {
#pragma unroll
        for (int p = 0; p < 8; ++p) x[p] = make_float2(x[p].x * kRotScale<D>, x[p].y * kRotScale<D>);
      }
    }
    if (masked || !ok) {
      const float s = masked ? Q4KV_SENTINEL_LOGIT : 0.0f;
#pragma unroll
      for (int p = 0; p < 8; ++p) x[p] = make_float2(s, s);
    }
    if (write) store_pairs<OutT>(kd, x);
    if (FP8) fp8_values(*reinterpret_cast<const Codes<8>*>(&cv), x);
    else to_values<BITS>(cv, sv, x);
    if (masked || !ok) {
#pragma unroll
      for (int p = 0; p < 8; ++p) x[p] = make_float2(0.0f, 0.0f);
    }
    if (write) store_pairs<OutT>(vd, x);
    kd += D;
    vd += D;
  }
}

template <int D, typename OutT>
__global__ void __launch_bounds__(256, 4) gather_kernel(const __grid_constant__ GatherArgs a, int64_t n_items, int per) {
  using S = Shape<D>;
  griddep_wait();
  griddep_launch_dependents();
  const PoolView& pool = a.pool;
  const int lane = threadIdx.x & 31;
  const int r = lane / S::LPV, j = lane % S::LPV;
  const int hkv = pool.n_kv_heads, parts = (hkv + per - 1) / per;
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (item >= n_items) return;
  const int part = static_cast<int>(item % parts);
  const int64_t n = item / parts * S::VPW + r;
  // the sequence of row n: the last b with offsets[b] <= n
  const bool inside = n < a.n_rows && n >= __ldg(a.offsets) && n < __ldg(a.offsets + a.batch);
  int b = 0;
  if (inside) {
    int hi = a.batch;                            // offsets[b] <= n < offsets[hi]
    while (hi - b > 1) {
      const int mid = (b + hi) / 2;
      if (__ldg(a.offsets + mid) <= n) b = mid;
      else hi = mid;
    }
  }
  __syncwarp();
  bool ok = inside, masked = false;
  int bits = 4, slot = 0;
  int64_t phys = 0;
  if (inside) {
    const int64_t p = (a.starts == nullptr ? 0 : static_cast<int64_t>(__ldg(a.starts + b))) + n - __ldg(a.offsets + b);
    if (p < 0 || p >= static_cast<int64_t>(a.max_blocks) * kBlockTokens) {
      raise_error(pool.error_word, Q4KV_DEVERR_SEQ_LEN);
      ok = false;
    } else {
      const int32_t blk = __ldg(a.tables + static_cast<int64_t>(b) * a.max_blocks + p / kBlockTokens);
      if (blk < 0 || blk >= pool.n_blocks()) {
        raise_error(pool.error_word, Q4KV_DEVERR_BLOCK_ID);
        ok = false;
      } else {
        bits = pool.bits_of(blk);
        slot = static_cast<int>(p % kBlockTokens);
        phys = bits == 4 ? blk : (bits == 8 ? blk - pool.n_q4 : blk - pool.n_q4 - pool.n_q8);
        masked = (__ldg(pool.mask + static_cast<int64_t>(blk) * kMaskWords + slot / 32) >> (slot % 32)) & 1u;
      }
    }
  }
  __syncwarp();
  const bool turn = a.unrotate_k && pool.k_rotated;
  const int64_t at = n * a.out_stride + j * kEPL;
  const int h1 = min(hkv, (part + 1) * per);
  // The widths of a warp's rows differ only where a block ends among them.  Rows of
  // 2-bit blocks take that way too: three walks over the heads, of which one loads.
  const bool all4 = __all_sync(0xffffffffu, bits == 4), all8 = __all_sync(0xffffffffu, bits == 8);
  const int h0 = part * per;
  OutT* kd = static_cast<OutT*>(a.k_out) + at + static_cast<int64_t>(h0) * D;
  OutT* vd = static_cast<OutT*>(a.v_out) + at + static_cast<int64_t>(h0) * D;
  if (pool.fp8) {
    heads<D, OutT, 8, true>(pool, phys, slot, j, h0, h1, ok, masked, false, inside, kd, vd);
  } else if (all4) {
    heads<D, OutT, 4, false>(pool, phys, slot, j, h0, h1, ok, masked, turn, inside, kd, vd);
  } else if (all8) {
    heads<D, OutT, 8, false>(pool, phys, slot, j, h0, h1, ok, masked, turn, inside, kd, vd);
  } else {                                       // every lane takes part in each (the rotation shuffles)
    heads<D, OutT, 4, false>(pool, phys, slot, j, h0, h1, ok && bits == 4, masked, turn, inside && bits == 4, kd, vd);
    heads<D, OutT, 8, false>(pool, phys, slot, j, h0, h1, ok && bits == 8, masked, turn, inside && bits == 8, kd, vd);
    heads<D, OutT, 2, false>(pool, phys, slot, j, h0, h1, ok && bits == 2, masked, turn, inside && bits == 2, kd, vd);
  }
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, cudaStream_t stream) {
  const int d = a.pool.head_dim;
  const int vpw = d == 128 ? Shape<128>::VPW : Shape<256>::VPW;
  const int64_t groups = (a.n_rows + vpw - 1) / vpw;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 148;
  // heads of a warp: one while the warps do not fill the GPU, all of them (so
  // that the look-up is shared) when there are enough rows
  int per = 1;
  while (per < a.pool.n_kv_heads && groups * ((a.pool.n_kv_heads + per - 1) / per) > static_cast<int64_t>(sms) * 64) ++per;
  const int64_t items = groups * ((a.pool.n_kv_heads + per - 1) / per);
  const int64_t g = (items + 7) / 8;
  if (g > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(g)), block(256);
#define Q4KV_G(DD, T) return launch_pdl(gather_kernel<DD, T>, grid, block, 0, stream, a, items, per)
  if (d == 128 && a.out_dtype == Q4KV_F32) Q4KV_G(128, float);
  if (d == 128 && a.out_dtype == Q4KV_F16) Q4KV_G(128, __half);
  if (d == 128) Q4KV_G(128, __nv_bfloat16);
  if (a.out_dtype == Q4KV_F32) Q4KV_G(256, float);
  if (a.out_dtype == Q4KV_F16) Q4KV_G(256, __half);
  Q4KV_G(256, __nv_bfloat16);
#undef Q4KV_G
}

}  // namespace q4kv
