// Reading token ranges back through the block tables, packed.
//
// Row n of the output is token starts[b] + n - offsets[b] of the sequence b
// with offsets[b] <= n < offsets[b + 1]; x = fl(code s + z), keys optionally
// through c H x, rounded once.  A warp takes VPW consecutive rows of one head
// (a lane holds 16 channels of one row, as in the encoder), the warps of a CTA
// take the heads of the same rows, so the rows written by a CTA are contiguous.
#include "extend_internal.cuh"
#include "rows.cuh"

namespace q4kv {
namespace {

template <int D, typename OutT>
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ GatherArgs a, int64_t n_items) {
  using S = Shape<D>;
  griddep_wait();
  griddep_launch_dependents();
  const PoolView& pool = a.pool;
  const int lane = threadIdx.x & 31;
  const int r = lane / S::LPV, j = lane % S::LPV;
  const int hkv = pool.n_kv_heads;
  const int64_t n_warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  const int first = __ldg(a.offsets);

  for (int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; item < n_items;
       item += n_warps) {
    const int h = static_cast<int>(item % hkv);
    const int64_t n = item / hkv * S::VPW + r;
    // the sequence of row n: the last b with offsets[b] <= n
    int lo = 0, hi = a.batch;                    // offsets[lo] <= n < offsets[hi], once both ends hold
    const bool inside = n < a.n_rows && n >= first && n < __ldg(a.offsets + a.batch);
    while (inside && hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__ldg(a.offsets + mid) <= n) lo = mid;
      else hi = mid;
    }
    __syncwarp();
    bool ok = inside;
    int64_t row = 0;
    int bits = 4;
    bool masked = false;
    if (inside) {
      const int64_t p = (a.starts == nullptr ? 0 : static_cast<int64_t>(__ldg(a.starts + lo))) + n - __ldg(a.offsets + lo);
      if (p < 0 || p >= static_cast<int64_t>(a.max_blocks) * kBlockTokens) {
        raise_error(pool.error_word, Q4KV_DEVERR_SEQ_LEN);
        ok = false;
      } else {
        const int32_t blk = __ldg(a.tables + static_cast<int64_t>(lo) * a.max_blocks + p / kBlockTokens);
        if (blk < 0 || blk >= pool.n_blocks()) {
          raise_error(pool.error_word, Q4KV_DEVERR_BLOCK_ID);
          ok = false;
        } else {
          bits = pool.bits_of(blk);
          const int slot = static_cast<int>(p % kBlockTokens);
          const int64_t phys = bits == 4 ? blk : (bits == 8 ? blk - pool.n_q4 : blk - pool.n_q4 - pool.n_q8);
          row = (phys * hkv + h) * kBlockTokens + slot;
          masked = (pool.mask[static_cast<int64_t>(blk) * kMaskWords + slot / 32] >> (slot % 32)) & 1u;
        }
      }
    }
    float x[kEPL], y[kEPL];
#pragma unroll
    for (int i = 0; i < kEPL; ++i) x[i] = y[i] = 0.0f;
    if (ok) {
      if (pool.fp8) {
        decode_fp8_lane(pool.k_codes8 + row * D, j, x);
        decode_fp8_lane(pool.v_codes8 + row * D, j, y);
      } else if (bits == 8) {
        decode_lane<8>(pool.k_codes8 + row * D, pool.k_params8 + row * S::NG, j, x);
        decode_lane<8>(pool.v_codes8 + row * D, pool.v_params8 + row * S::NG, j, y);
      } else if (bits == 2) {
        decode_lane<2>(pool.k_codes2 + row * (D / 4), pool.k_params2 + row * S::NG, j, x);
        decode_lane<2>(pool.v_codes2 + row * (D / 4), pool.v_params2 + row * S::NG, j, y);
      } else {
        decode_lane<4>(pool.k_codes4 + row * (D / 2), pool.k_params4 + row * S::NG, j, x);
        decode_lane<4>(pool.v_codes4 + row * (D / 2), pool.v_params4 + row * S::NG, j, y);
      }
    }
    __syncwarp();
    if (a.unrotate_k && pool.k_rotated) rotate_vector<D>(x, j);
    if (masked) {
#pragma unroll
      for (int i = 0; i < kEPL; ++i) {
        x[i] = Q4KV_SENTINEL_LOGIT;
        y[i] = 0.0f;
      }
    }
    if (inside) {
      const int64_t at = n * a.out_stride + static_cast<int64_t>(h) * D + j * kEPL;
      store16<OutT>(static_cast<OutT*>(a.k_out) + at, x);
      store16<OutT>(static_cast<OutT*>(a.v_out) + at, y);
    }
  }
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, cudaStream_t stream) {
  const int d = a.pool.head_dim;
  const int vpw = d == 128 ? Shape<128>::VPW : Shape<256>::VPW;
  const int64_t items = (a.n_rows + vpw - 1) / vpw * a.pool.n_kv_heads;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 148;
  int64_t g = (items + 7) / 8;
  if (g > static_cast<int64_t>(sms) * 64) g = static_cast<int64_t>(sms) * 64;
  const dim3 grid(static_cast<unsigned>(g)), block(256);
#define Q4KV_G(DD, T) return launch_pdl(gather_kernel<DD, T>, grid, block, 0, stream, a, items)
  if (d == 128 && a.out_dtype == Q4KV_F32) Q4KV_G(128, float);
  if (d == 128 && a.out_dtype == Q4KV_F16) Q4KV_G(128, __half);
  if (d == 128) Q4KV_G(128, __nv_bfloat16);
  if (a.out_dtype == Q4KV_F32) Q4KV_G(256, float);
  if (a.out_dtype == Q4KV_F16) Q4KV_G(256, __half);
  Q4KV_G(256, __nv_bfloat16);
#undef Q4KV_G
}

}  // namespace q4kv
