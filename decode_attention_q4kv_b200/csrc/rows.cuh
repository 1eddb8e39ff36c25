// Decoding of one (token, head) row of the paged format, shared by the
// dequantise and card kernels (quantize.cu) and the read-back kernel
// (gather.cu).  A lane holds 16 consecutive channels of one row, as in the
// encoder (encode.cuh).
#pragma once
#include "encode.cuh"

namespace q4kv {
namespace {

// Scalar butterflies for the decoder's optional un-rotation (channels 16j ..
// 16j+15 of the lane in order); same stage order and operations as above.
template <int D>
__device__ __forceinline__ void fwht_vector(float (&x)[kEPL], int j) {
#pragma unroll
  for (int h = 1; h < kEPL; h <<= 1) {
#pragma unroll
    for (int i = 0; i < kEPL; ++i) {
      if ((i & h) == 0) {
        const float a = x[i], b = x[i + h];
        x[i] = __fadd_rn(a, b);
        x[i + h] = __fsub_rn(a, b);
      }
    }
  }
#pragma unroll
  for (int h = kEPL; h < D; h <<= 1) {
    const int lane_bit = h / kEPL;
    const bool upper = (j & lane_bit) != 0;
#pragma unroll
    for (int i = 0; i < kEPL; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, x[i], lane_bit);
      x[i] = upper ? __fsub_rn(other, x[i]) : __fadd_rn(x[i], other);
    }
  }
}

template <int D>
__device__ __forceinline__ void rotate_vector(float (&x)[kEPL], int j) {
  fwht_vector<D>(x, j);
  const float c = rotation_constant(D);
#pragma unroll
  for (int i = 0; i < kEPL; ++i) x[i] = __fmul_rn(x[i], c);
}

// ---------------------------------------------------------------------------
// dequantisation
// ---------------------------------------------------------------------------

template <int BITS>
__device__ __forceinline__ void decode_lane(const uint8_t* __restrict__ codes,
                                            const __half2* __restrict__ params, int j,
                                            float (&x)[kEPL]) {
  const __half2 p = params[j >> 2];
  const float s = __low2float(p);
  const float z = __high2float(p);
  uint32_t w[4];
  if (BITS == 2) {
    w[0] = *reinterpret_cast<const uint32_t*>(codes + j * 4);
#pragma unroll
    for (int i = 0; i < kEPL; ++i) x[i] = __fmaf_rn(static_cast<float>((w[0] >> (2 * i)) & 3u), s, z);
  } else if (BITS == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(codes + j * 8);
    w[0] = u.x;
    w[1] = u.y;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = __fmaf_rn(static_cast<float>((w[0] >> (4 * i)) & 15u), s, z);
      x[8 + i] = __fmaf_rn(static_cast<float>((w[1] >> (4 * i)) & 15u), s, z);
    }
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(codes + j * 16);
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
#pragma unroll
    for (int i = 0; i < kEPL; ++i)
      x[i] = __fmaf_rn(static_cast<float>((w[i / 4] >> (8 * (i % 4))) & 255u), s, z);
  }
}

// The lane's 16 E4M3 bytes as binary32 (every E4M3 value is exact in fp16).
__device__ __forceinline__ void decode_fp8_lane(const uint8_t* __restrict__ codes, int j, float (&x)[kEPL]) {
  const uint4 u = *reinterpret_cast<const uint4*>(codes + j * kEPL);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename OutT>
__device__ __forceinline__ void store16(OutT* dst, const float (&x)[kEPL]);
template <>
__device__ __forceinline__ void store16<float>(float* dst, const float (&x)[kEPL]) {
  float4* d = reinterpret_cast<float4*>(dst);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
template <>
__device__ __forceinline__ void store16<__half>(__half* dst, const float (&x)[kEPL]) {
  __align__(16) __half h[kEPL];
#pragma unroll
  for (int i = 0; i < kEPL; ++i) h[i] = __float2half_rn(x[i]);
  uint4* d = reinterpret_cast<uint4*>(dst);
  d[0] = reinterpret_cast<const uint4*>(h)[0];
  d[1] = reinterpret_cast<const uint4*>(h)[1];
}

template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* dst, const float (&x)[kEPL]) {
  __align__(16) __nv_bfloat16 h[kEPL];
#pragma unroll
  for (int i = 0; i < kEPL; ++i) h[i] = __float2bfloat16_rn(x[i]);
  uint4* d = reinterpret_cast<uint4*>(dst);
  d[0] = reinterpret_cast<const uint4*>(h)[0];
  d[1] = reinterpret_cast<const uint4*>(h)[1];
}

}  // namespace
}  // namespace q4kv
