// Attention of a chunk of new tokens over the paged quantised cache.
//
// For the rows (token i, head of the group) of one KV head:
//   o = sum_t p_t V_t / sum_t p_t,  p_t = 2^(s_t - m),  s_t = log2(e) scale <q, K_t>
// over the positions t the token sees.  A CTA holds 128 or 256 rows; it walks
// their keys in tiles, S = Q K^T and O += P V on the tensor cores (fp16
// operands, fp32 accumulators in tensor memory).
//
// Warp roles (28 warps, the last two idle):
//   softmax  four groups of four warps, one row per thread: maximum, weights, sum
//            of 64 columns at a time (a step).  Two groups share the rows of one
//            accumulator and take its steps by turns, each with a logit buffer of
//            its own: while the weights of one step are made, the logits of the
//            next are loaded, and the products around them run.  The weights go
//            back into the tensor memory that held the logits, and are the A
//            operand of the second product.
//   decode   four warps turn the keys' codes into fp16, four the values', in the
//            layout the tensor cores read (rows of 128 bytes, 128-byte swizzle);
//            remapped slots and slots past the end become zeros
//   product  one thread issues the matrix products
//   feed     one thread copies each tile's packed codes, scales and mask into a
//            ring in shared memory (bulk copies)
//
// Within 8 channels the decoded order is 0 4 1 5 2 6 3 7 (what one mask and one
// subtraction per pair of codes leave); q is stored in the same order and the
// output's columns are put back when they are written.
//
// Roundings: K and V to fp16 (one fused multiply-add code * s + z), q (with scale
// and log2(e) in it) to fp16 after a power-of-two scaling per row, the weights to
// fp16 (scaled by 2^6, so that weights down to 2^-30 of the largest survive).  Each
// is at most 2^-11 of what is rounded, or half a step of fp16's smallest numbers:
// 2^-25 for K and V below 2^-14, 2^-31 of its row's largest channel for q, 2^-30 of
// the row's largest weight for the weights.  Maxima, sums and accumulators are
// binary32; the tensor cores cut off what they add up, up to 2^-12 of a sum over
// the most tokens that a plan gives an accumulator.  The running maximum is only
// moved when it grows by more than 2^8: until then weights above 1 are harmless (at
// most 2^14 in fp16), and the accumulator is not rescaled.
// For N(0, 1) inputs the output is off by 4e-4 of its size, 2e-4 of it the fp16
// output's own rounding; codes are 4 bits, so the cache itself is off by percents.
//
// Bound by the softmax warps: a step of 128 tokens x 256 rows takes ~4200 cycles,
// the products of it ~2050, and the CTA has 27000 cycles of start and end (the plan's
// fit; what they consist of was not taken apart).  One chunk of 512 tokens, 32/8 heads
// of 128, on 8192: 107 us, 0.39 of the measured bf16 rate; issue 61 %, tensor pipe
// 41 %, exponentials' unit 44 %, no pipe full.  2048 tokens on 32768 (a quarter of the
// blocks 8-bit): 1157 us for a call by itself, 1374 in runs of minutes under the power
// cap (0.58 and 0.49).  Of 1165 us of an earlier state of the kernel, without the looks for
// what is not finite, 770 were left without the softmax, 1028 without
// decoding, 1039 without the exponentials, 1145 with a sixteenth of the products.
// Four softmax warps a row tile and parity hide the latency of tensor-memory loads
// (~300 cycles while products run); polynomial exponentials on the FMA pipe, sleeping
// waits, more decode warps and other register shares gained nothing.
#include <math.h>

#include "encode.cuh"
#include "extend_internal.cuh"
#include "tcgen05.cuh"

namespace q4kv {
namespace {

constexpr int kDecodeWarp0 = 16, kMmaWarp = 24, kFeedWarp = 25;
constexpr int kThreads = 28 * 32;
// Registers: 72 a thread at launch (asked for with __maxnreg__; the launch looks, for
// shares above what the block has would wait forever), shared out anew by role.
constexpr int kRegs = 72, kOtherRegs = 56;
constexpr float kNone = -3.0e38f; // reference maximum of a row that has seen nothing: below every logit
constexpr int kCols = 64;        // logit columns of a softmax step
constexpr int kSlots = 4;        // decoded tiles
constexpr uint32_t kTile = 32768;// bytes of a decoded tile
constexpr uint32_t kSBase = 256; // tensor-memory columns: accumulators from 0, logits from here
constexpr int kMaxRaw = 7;
constexpr float kShift = 6.0f;   // weights are stored times 2^6
constexpr float kLazy = 8.0f;    // growth of the maximum (log2) that moves it
constexpr float kLog2e = 1.4426950408889634f;

// MODE 0: D = 128, two row tiles of 128, two softmax groups each.
// MODE 1: D = 128, one row tile; the two pairs of softmax groups take alternate
//         key tiles with their own accumulators (two partial results).
// MODE 2: D = 256, one row tile, two softmax groups.
// MODE 3: MODE 1 for up to 32 rows: the tile holds each four times, and each copy
//         takes 16 of a step's 64 columns (its weights of the others are 0), so
//         that all four warps of a group have work; the copies are added up at
//         the end.  MODE 1 / MODE 3, us, 32/8 heads: 16 x 5 tokens on up to 32768
//         282 / 247, a quarter 8-bit 412 / 367, E4M3 488 / 446; 64 x 1 on 8192 386 / 335;
//         8 x 8 on 8192 62.5 / 58.4; 1 x 4 on 32768 44 / 41; 4 x 30, 8/8 heads, on 16384
//         64.5 / 58.4.  Heads of 256 have no such shape: up to 32 rows leave three of
//         the four warps of a group without work there.
template <int MODE>
struct Geo {
  static constexpr bool ALT = MODE == 1 || MODE == 3;  // alternate key tiles
  static constexpr int COPIES = MODE == 3 ? 4 : 1;     // of a row in the tile
  // Registers of a softmax and of a decoding thread.  With 16 columns a thread the
  // softmax needs fewer, and a lane can decode its four tokens at once
  // (the calls above with the shares and lanes of the other shapes: 267, 397, 451,
  // 360, 60.4, 42 and 62.3 us).
  static constexpr int kSoftRegs = MODE == 3 ? 64 : 88, kDecodeRegs = MODE == 3 ? 96 : 48, kAtOnce = MODE == 3 ? 4 : 1;
  static_assert(16 * kSoftRegs + 8 * kDecodeRegs + 4 * kOtherRegs <= 28 * kRegs, "register shares");
  static constexpr int D = MODE == 2 ? 256 : 128;
  static constexpr int BN = MODE == 2 ? 64 : 128;      // tokens of a key tile
  static constexpr int STEPS = BN / kCols;             // softmax steps of a key tile
  static constexpr int QT = MODE == 0 ? 2 : 1;         // row tiles
  static constexpr int STREAMS = ALT ? 2 : 1;    // partial results of a row
  static constexpr int R = 128 * QT;
  static constexpr uint32_t kQ = QT * 128 * D * 2;
  static constexpr uint32_t kRawAt = kQ + kSlots * kTile;
  static constexpr uint32_t kRawRing = ALT ? 65600 : 32800;   // 4 or 2 packed tiles of 8-bit codes, 7 or 3 of 4-bit ones
  static constexpr uint32_t kMiscAt = kRawAt + kRawRing;
};

struct Misc {
  // Copy n (keys and values in turn) completes raw_full[n % (2 * entries)] and
  // frees kv_empty[n % (2 * kSlots)]: keys and values are decoded by different
  // warps, and with twice as many barriers as places each barrier belongs to
  // one of the two.  A parity wait tells only two phases apart, so a warp may
  // wait on a barrier only after it has seen the phase before; on a barrier
  // shared by both kinds the phase before would be the other warps' business.
  uint64_t raw_full[2 * kMaxRaw], raw_empty[kMaxRaw], kv_full[kSlots], kv_empty[2 * kSlots], spare;
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2];   // by accumulator and logit buffer
  uint64_t turn[2][4];     // by accumulator and quarter of its rows: the reference after a step is known
  uint32_t tmem;
  int abort;
  int issued;              // tiles that the feed has sent for
  // What is in a ring entry: 16 times the index of the tile's block among those of
  // its code width, plus the width; 0 = a block id out of range or no tile yet.  One
  // word, so that a decoder whose wait gave up still finds a block of this pool.
  // (2^28 blocks of one width would be terabytes.)
  uint32_t raw_what[kMaxRaw];
  // Remapped slots of key tile j and whether its block id is out of range, at
  // j % 8, from the key decoders to the softmax.  (A decoder that writes for tile
  // j + 8 has seen the keys of tile j + 5 used up.  Their products were issued after
  // those of tile j + 3's values, which wait for that tile's weights, so the softmax
  // is past tile j.)
  alignas(16) uint32_t gone[8][4];
  int bad[8];
  int odd_first, odd_last; // tokens of this CTA whose value is not finite lie between these
  float reference[256];    // per row: the reference maximum after the last step that settled
  int8_t exponent[256];    // per row: q was scaled by 2^(6 - exponent)
};
template <int MODE>
constexpr uint32_t smem_bytes() { return Geo<MODE>::kMiscAt + sizeof(Misc); }
static_assert(Geo<0>::kMiscAt % 16 == 0 && Geo<1>::kMiscAt % 16 == 0 && Geo<2>::kMiscAt % 16 == 0, "alignment");
static_assert(smem_bytes<0>() <= 232448 && smem_bytes<1>() <= 232448 && smem_bytes<2>() <= 232448 && smem_bytes<3>() <= 232448, "shared memory");

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// One try of a wait, the hardware's own suspension only.
__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// Bounded wait.  When it runs out, abort is set and this and every later wait of
// the block returns at once: the roles walk their loops to the end (every access
// stays inside its buffers whatever they hold), the block waits for what is still
// in flight, the rows are written as 0 and the error bit is raised.  No sleep
// between tries: every wait here is short and on the critical path of the next role.
struct Gate {
  Misc* ms;
  unsigned tries;          // of one wait
};
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, Gate g) {
  if (phase_done(bar, parity)) return;
  for (unsigned i = 1; i < g.tries; ++i) {
    if (phase_done(bar, parity)) return;
    if ((i & 1023u) == 0 && *reinterpret_cast<volatile int*>(&g.ms->abort) != 0) return;
  }
  *reinterpret_cast<volatile int*>(&g.ms->abort) = 1;
}
__device__ __forceinline__ void warp_wait(uint64_t* bar, uint32_t parity, Gate g) {
  wait(bar, parity, g);
  __syncwarp();
}

__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[32]) { tmem_ld32(addr, r); }
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[8]) { tmem_ld8(addr, r); }

// A decoding lane's place: its first token in the tile and its 32-channel
// unit; its four tokens lie step() apart.
struct Lane {
  int t, u;
  static constexpr __host__ __device__ int step(int d) { return d == 128 ? 32 : 16; }
};

// (a & b) | c
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// 8 codes as 4 half pairs in the order above: fp16(code * s + z), one rounding.
// 0x64xx is 1024 + xx in fp16: a mask and an or give codes exactly, less 1024.
__device__ __forceinline__ void codes4(uint32_t w, __half2 s, __half2 z, uint32_t* o) {
  const __half2 k1024 = __float2half2_rn(1024.0f), k16 = __float2half2_rn(0.0625f), k64 = __float2half2_rn(-64.0f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = w >> (8 * i);
    const __half2 lo = __hsub2(u2h(and_or(v, 0x000F000Fu, 0x64006400u)), k1024);
    const __half2 hi = __hfma2(u2h(and_or(v, 0x00F000F0u, 0x64006400u)), k16, k64);   // (1024 + 16 code) / 16 - 64
    o[2 * i] = h2u(__hfma2(lo, s, z));
    o[2 * i + 1] = h2u(__hfma2(hi, s, z));
  }
}
__device__ __forceinline__ void codes8(uint32_t w0, uint32_t w1, __half2 s, __half2 z, uint32_t* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = __byte_perm(w0, w1, static_cast<uint32_t>(i | i << 4 | (4 + i) << 8 | (4 + i) << 12));
    o[i] = h2u(__hfma2(__hsub2(u2h(and_or(v, 0x00FF00FFu, 0x64006400u)), __float2half2_rn(1024.0f)), s, z));
  }
}
__device__ __forceinline__ void codes2(uint32_t w16, __half2 s, __half2 z, uint32_t* o) {   // codes 0-3, codes 4-7 in halves
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = 1.0f / static_cast<float>(1 << (2 * i));
    const __half2 h = __hfma2(u2h(and_or(w16, 0x00030003u << (2 * i), 0x64006400u)), __float2half2_rn(f),
                              __float2half2_rn(-1024.0f * f));
    o[i] = h2u(__hfma2(h, s, z));
  }
}
__device__ __forceinline__ void codes_fp8(uint32_t w0, uint32_t w1, bool live, uint32_t* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = __byte_perm(w0, w1, static_cast<uint32_t>(i | (4 + i) << 4));
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xFFFFu), __NV_E4M3);
    o[i] = live ? h2u(*reinterpret_cast<const __half2*>(&h)) : 0u;
  }
}

// Scale and zero of a group whose largest code decodes to a finite fp16 value.
// A scale rounded up may carry a finite group past fp16 (the error of 15 s is at
// most half a step of s times 15, and one step less of s takes back twice that);
// what is still not finite then makes the token odd.
template <int MAX>
__device__ __forceinline__ bool finite_group(uint32_t sz) {
  const __half2 q = u2h(sz);
  return __hle(__habs(__hfma(__low2half(q), __int2half_rn(MAX), __high2half(q))), __ushort_as_half(0x7BFFu));
}
template <int MAX>
__device__ __forceinline__ bool tame_group(uint32_t& sz) {
  if (finite_group<MAX>(sz)) return true;
  if ((sz & 0x7FFFu) != 0) --sz;
  return finite_group<MAX>(sz);
}
constexpr uint32_t kNanGroup = 0x7FFF7FFFu;   // every code of it is NaN
// Some byte is an E4M3 NaN.
__device__ __forceinline__ bool fp8_nan(uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; }

// Whether token t is live and its value not finite.  (This and mend_groups are
// calls, rarely made, kept out of the loops' code; they use 30 and 15 registers,
// fewer than any role's share.)
template <int D>
__device__ __noinline__ bool odd_token(const PoolView& P, const int32_t* table, int h, int t) {
  const int blk = __ldg(table + t / kBlockTokens), slot = t % kBlockTokens;
  if (blk < 0 || blk >= P.n_blocks()) return false;
  if ((__ldg(P.mask + static_cast<int64_t>(blk) * kMaskWords + slot / 32) >> (slot % 32)) & 1u) return false;
  const int bits = P.bits_of(blk);
  const int64_t phys = bits == 4 ? blk : (bits == 8 ? blk - P.n_q4 : blk - P.n_q4 - P.n_q8);
  const int64_t row = (phys * P.n_kv_heads + h) * kBlockTokens + slot;
  bool odd = false;
  if (P.fp8) {
    for (int i = 0; i < D / 4; ++i) odd |= fp8_nan(__ldg(reinterpret_cast<const uint32_t*>(P.v_codes8 + row * D) + i));
    return odd;
  }
  const __half2* params = (bits == 4 ? P.v_params4 : (bits == 8 ? P.v_params8 : P.v_params2)) + row * (D / kGroup);
  for (int i = 0; i < D / kGroup; ++i) {
    uint32_t sz = h2u(__ldg(params + i));
    odd |= !(bits == 4 ? tame_group<15>(sz) : (bits == 8 ? tame_group<255>(sz) : tame_group<3>(sz)));
  }
  return odd;
}

// The lane's four tokens of a tile, 32 channels each.  The loads come first so
// that their latencies overlap.  A token that does not count takes scale and
// zero 0 (whatever its own are), so its values are 0.  With `check` 8-bit codes
// are looked at for what is not finite, as below.  BITS 0: E4M3 bytes.
template <int D, int BITS, int AT_ONCE>
__device__ __forceinline__ void decode_tile(const uint8_t* raw, const uint8_t* params, const Lane& ln, uint32_t live,
                                            uint8_t* dst, bool check, bool key, int t0, Misc* ms) {
  constexpr int W = BITS == 0 ? 8 : BITS;              // words of 32 codes
  constexpr int TS = Lane::step(D);
  constexpr int ROW = D / 8 * W;                       // bytes of a token
  const uint8_t* src = raw + ln.t * ROW + ln.u * 4 * W;
#pragma unroll AT_ONCE
  for (int it = 0; it < 4; ++it) {
    const uint8_t* p = src + it * TS * ROW;
    uint32_t w[W], sz = 0;
    if (W == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x;
      w[1] = x.y;
    } else {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[q];
        w[4 * q] = x.x;
        w[4 * q + 1] = x.y;
        w[(4 * q + 2) % W] = x.z;
        w[(4 * q + 3) % W] = x.w;
      }
    }
    if (BITS != 0) sz = *reinterpret_cast<const uint32_t*>(params + ((ln.t + it * TS) * (D / kGroup) + (ln.u >> 1)) * 4);
    bool on = (live >> it) & 1u;
    if ((BITS == 0 || BITS == 8) && check && on) {
      if (BITS == 0) {
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) odd |= (w[i] & 0x7F7F7F7Fu) + 0x01010101u;
        on = (odd & 0x80808080u) == 0;
      } else {
        on = tame_group<255>(sz);
        if (!on && key) {
          on = true;
          sz = kNanGroup;
        }
      }
      if (!on) {
        atomicMin(&ms->odd_first, t0 + ln.t + it * TS);
        atomicMax(&ms->odd_last, t0 + ln.t + it * TS);
      }
    }
    const __half2 q = u2h(on ? sz : 0u);
    const __half2 s = __low2half2(q), z = __high2half2(q);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t o[4];
      if (BITS == 0) codes_fp8(w[(2 * c) % W], w[(2 * c + 1) % W], on, o);
      else if (BITS == 8) codes8(w[(2 * c) % W], w[(2 * c + 1) % W], s, z, o);
      else if (BITS == 4) codes4(w[c % W], s, z, o);
      else codes2(__byte_perm(w[(c >> 1) % W], 0, c & 1 ? 0x4342 : 0x4140), s, z, o);
      // (the lane's tokens are the same modulo 8)
      *reinterpret_cast<uint4*>(dst + it * (TS / 8) * 1024 + (((4 * (ln.u & 1) + c) ^ (ln.t & 7)) << 4)) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// A value that is not finite takes 0 as well: a product with it would reach the
// rows that do not see its token, too (a weight of 0 times it is NaN).  Its
// place is noted, and the rows that do see it become NaN at the end.  A key's
// logits are replaced where they are not seen, so a key that is not finite only has
// to be NaN, for infinities of one sign would give the logit -Inf, and the weight 0.
// (E4M3 has no infinities.)
//
// Whether one of the warp's tokens needs it is found out with one look at their
// scales, two groups a lane.  Scales in shared memory are put right there, 8-bit
// ones are left to decode_tile.  (Without any look 64 x 1 tokens on 8192 take 322 us
// instead of 335, 16 x 5 on up to 32768 237 instead of 247, 4 x 509 on 16384 840
// instead of 854, 5 x 256 with heads of 256 308 instead of 328, E4M3 of heads of 256
// 172 instead of 178.  Beside every token's decoding the look at values alone cost 8 to
// 13 %, in a warp of its own, which delays the decoders, 1 to 16 %.)
template <int D, int MAX>
__device__ __noinline__ void mend_groups(uint2* at, uint2 sz, bool key, bool live, int t, Misc* ms) {
  const bool fx = tame_group<MAX>(sz.x), fy = tame_group<MAX>(sz.y);
  const uint32_t odd = key ? kNanGroup : 0u;
  *at = make_uint2(fx ? sz.x : odd, fy ? sz.y : odd);
  if (!key && live && !(fx && fy)) {
    atomicMin(&ms->odd_first, t);
    atomicMax(&ms->odd_last, t);
  }
}
template <int D, int MAX>
__device__ __forceinline__ bool odd_groups(uint8_t* params, const uint8_t* mask, bool key, int dw, int lane, int t0, int end, Misc* ms) {
  const int t = D == 128 ? dw * 8 + (lane & 7) + 32 * (lane >> 3) : dw * 4 + ((lane >> 1) & 3) + 16 * (lane >> 3);
  uint2* at = reinterpret_cast<uint2*>(params + t * (D / kGroup) * 4) + (D == 128 ? 0 : lane & 1);
  const uint2 sz = *at;
  const bool odd = !(finite_group<MAX>(sz.x) && finite_group<MAX>(sz.y));
  if (!__any_sync(0xffffffffu, odd)) return false;
  if (MAX != 255) {
    const int slot = (t0 & 64) * (D / 256) + t;            // within the 128 slots of the mask
    if (odd) mend_groups<D, MAX>(at, sz, key, t0 + t < end && !((mask[slot >> 3] >> (slot & 7)) & 1u), t0 + t, ms);
    __syncwarp();
  }
  return true;
}

// Output columns 8k .. 8k+7 back in channel order.
__device__ __forceinline__ void channel_order(const uint32_t (&r)[32], float f, float (&y)[32]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[8 * k + i] = __uint_as_float(r[8 * k + 2 * i]) * f;
      y[8 * k + 4 + i] = __uint_as_float(r[8 * k + 2 * i + 1]) * f;
    }
}
__device__ __forceinline__ uint32_t pack16(int dtype, float x, float y) {
  if (dtype == Q4KV_F16) return h2u(__floats2half2_rn(x, y));
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The part of the work one CTA has; every thread computes the same.
struct Item {
  int b, h, split;
  int g, T;
  int len, nn;         // cached tokens, new tokens
  int r0, r1, rv;      // rows of the tile, end of the rows there are, end of the rows of real tokens
  int t0, n;           // first token of the first key tile, key tiles
  bool bad;
};
template <int MODE>
__device__ __forceinline__ Item item_of(const ExtendArgs& a) {
  using G = Geo<MODE>;
  Item w;
  const int S = a.plan.n_splits;
  w.T = a.plan.max_new;
  w.g = a.plan.n_q_heads / a.pool.n_kv_heads;
  w.h = blockIdx.y;
  w.b = blockIdx.z;
  // later row tiles see more keys and start first
  const int tile = static_cast<int>((gridDim.x - 1 - blockIdx.x) / S);
  w.split = static_cast<int>((gridDim.x - 1 - blockIdx.x) % S);
  w.len = __ldg(a.seq_lens + w.b);
  w.nn = a.n_new == nullptr ? w.T : max(0, min(__ldg(a.n_new + w.b), w.T));
  w.bad = w.len < 0 || static_cast<int64_t>(w.len) + w.nn > static_cast<int64_t>(a.plan.max_blocks_per_seq) * kBlockTokens;
  w.r0 = tile * G::R;
  w.r1 = min(w.r0 + G::R, w.T * w.g);
  w.rv = min(w.r1, w.nn * w.g);
  w.t0 = w.n = 0;
  if (w.bad || w.rv <= w.r0) return w;
  const int end = w.len + (w.rv - 1) / w.g + 1;
  const int begin = a.plan.window > 0 ? max(0, w.len + w.r0 / w.g - a.plan.window + 1) : 0;
  const int first = begin / G::BN, tiles = (end + G::BN - 1) / G::BN - first;
  const int steps = (tiles + G::STREAMS - 1) / G::STREAMS, per = (steps + S - 1) / S;
  const int j0 = min(tiles, w.split * per * G::STREAMS), j1 = min(tiles, (w.split + 1) * per * G::STREAMS);
  w.t0 = (first + j0) * G::BN;
  w.n = j1 - j0;
  return w;
}

template <int MODE, bool FP8>
__global__ void __maxnreg__(kRegs) extend_kernel(const __grid_constant__ ExtendArgs a, uint32_t raw_stride,
                                                 int n_raw) {
  using G = Geo<MODE>;
  constexpr int D = G::D, BN = G::BN;
  extern __shared__ __align__(1024) uint8_t sm[];
  griddep_wait();
  griddep_launch_dependents();
  const PoolView& P = a.pool;
  Misc* ms = reinterpret_cast<Misc*>(sm + G::kMiscAt);
  const Gate gate{ms, a.tries};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Item w = item_of<MODE>(a);
  const int hq = a.plan.n_q_heads, S = a.plan.n_splits, mb = a.plan.max_blocks_per_seq;
  const int partials = S * G::STREAMS;
  const int64_t all_rows = static_cast<int64_t>(a.plan.batch) * w.T * hq;

  if (w.bad && w.nn > 0 && tid == 0) raise_error(P.error_word, Q4KV_DEVERR_SEQ_LEN);
  if (partials == 1) {   // rows of no real token are 0 (the merge sees to them otherwise)
    const int z0 = w.bad ? w.r0 : max(w.r0, w.rv);
    const int size = a.out_dtype == Q4KV_F32 ? 4 : 2, pieces = D * size / 16;
    for (int x = tid; x < (w.r1 - z0) * pieces; x += kThreads) {
      const int r = z0 + x / pieces;
      uint8_t* row = static_cast<uint8_t*>(a.out) + (w.b * a.o_seq_stride + (r / w.g) * a.o_token_stride +
                                                     static_cast<int64_t>(w.h * w.g + r % w.g) * D) * size;
      reinterpret_cast<uint4*>(row)[x % pieces] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (w.bad || w.rv <= w.r0) return;
  if (w.n == 0) {        // no keys in this split
    for (int x = tid; x < (w.rv - w.r0) * G::STREAMS; x += kThreads) {
      const int r = w.r0 + x / G::STREAMS;
      const int64_t row = (static_cast<int64_t>(w.b) * w.T + r / w.g) * hq + w.h * w.g + r % w.g;
      a.ws_ml[(w.split * G::STREAMS + x % G::STREAMS) * all_rows + row] = make_float2(-INFINITY, 0.0f);
    }
    return;
  }

  // Softmax warps (of a group) with real rows, per accumulator; MODE 0 drops its second row tile
  // when no row is in it.  Steps of 64 columns of each accumulator.
  const int warps0 = G::COPIES == 4 ? 4 : min(4, (w.rv - w.r0 + 31) / 32);
  const int warps1 = MODE == 2 ? 0 : G::ALT ? warps0 : max(0, min(4, (w.rv - w.r0 - 128 + 31) / 32));
  const int groups = warps1 > 0 ? 2 : 1;
  const int steps0 = (G::ALT ? (w.n + 1) / 2 : w.n) * G::STEPS, steps1 = (G::ALT ? w.n / 2 : w.n) * G::STEPS;

  if (tid == 0) {
    for (int i = 0; i < 2 * n_raw; ++i) mbar_init(&ms->raw_full[i], 1);
    for (int i = 0; i < n_raw; ++i) {
      mbar_init(&ms->raw_empty[i], 4);
      ms->raw_what[i] = 0;
    }
    for (int i = 0; i < kSlots; ++i) mbar_init(&ms->kv_full[i], 4);
    for (int i = 0; i < 2 * kSlots; ++i) mbar_init(&ms->kv_empty[i], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ms->s_full[i >> 1][i & 1], 1);
      mbar_init(&ms->p_full[i >> 1][i & 1], i < 2 ? warps0 : max(1, warps1));
      mbar_init(&ms->o_done[i >> 1][i & 1], 1);
    }
    mbar_init(&ms->spare, 1);
    for (int i = 0; i < 8; ++i) mbar_init(&ms->turn[i >> 2][i & 3], 1);
    ms->abort = a.tries == 0;
    ms->odd_first = 0x7fffffff;
    ms->odd_last = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(&ms->tmem, 512);

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  const int end = w.len + w.nn;                            // tokens of the sequence
  const int32_t* table = a.tables + static_cast<int64_t>(w.b) * mb;
  // of a softmax warp: its accumulator and its parity of steps
  const int group = MODE == 2 ? warp >> 3 : (warp >> 3) & 1, side = (warp >> 2) & 1;

  if (warp < kDecodeWarp0) {
    // Q: rotate, times log2(e) scale, scale each row by a power of two, round to
    // fp16.  What is left to do to the products is then a power of two, which is
    // exact, so that logits and the reference maximum differ by what they differ by,
    // however large both are.  Rows of no real token are left as they are: no other
    // row depends on them.
    using Sh = Shape<D>;
    constexpr int kPasses = G::R / Sh::VPW / 16;           // of a warp
    const int rl = lane / Sh::LPV, j = lane % Sh::LPV;
    auto in_tile = [](int row) { return G::COPIES == 4 ? row & 31 : row; };
    // (a warp's passes lie 16 apart; the next one's row is on its way meanwhile)
    auto load = [&](int p, uint4 (&in)[2]) {
      const int rr = w.r0 + in_tile((p * 16 + warp) * Sh::VPW) + rl;
      in[0] = in[1] = make_uint4(0u, 0u, 0u, 0u);
      if (p < kPasses && rr < w.rv) {
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __half*>(a.q) + w.b * a.q_seq_stride + (rr / w.g) * a.q_token_stride +
            static_cast<int64_t>(w.h * w.g + rr % w.g) * D + j * kEPL);
        in[0] = __ldg(src);
        in[1] = __ldg(src + 1);
      }
    };
    uint4 in[2], next[2];
    load(0, next);
    const float qs = a.scale * kLog2e * (P.k_rotated ? kRotScale<D> : 1.0f);
#pragma unroll 1
    for (int p = 0; p < kPasses; ++p) {
      const int row = (p * 16 + warp) * Sh::VPW + rl;
      if (G::COPIES == 1 && w.r0 + (p * 16 + warp) * Sh::VPW >= w.rv) break;   // (the whole warp)
      in[0] = next[0];
      in[1] = next[1];
      load(p + 1, next);
      __syncwarp();
      float2 x[8];
      if (a.q_dtype == Q4KV_F16) unpack16<__half>(in[0], in[1], x);
      else unpack16<__nv_bfloat16>(in[0], in[1], x);
      if (P.k_rotated) rotate_pairs<D>(x, j);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = make_float2(x[i].x * qs, x[i].y * qs);
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max3(m, fabsf(x[i].x), fabsf(x[i].y));
#pragma unroll
      for (int st = 1; st < Sh::LPV; st <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, st));
      // the row's largest magnitude comes to lie in [64, 128); a row with an infinity
      // is NaN (one with a NaN is by itself), so that its logits cannot all be -Inf
      const int e = m == 0.0f ? 0 : min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -100), 127);
      const float f = m == INFINITY ? NAN : __uint_as_float(static_cast<uint32_t>(127 + 6 - e) << 23);
      if (j == 0) ms->exponent[row] = static_cast<int8_t>(e);
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] = h2u(__floats2half2_rn(x[i].x * f, x[i + 4].x * f));
        o[4 + i] = h2u(__floats2half2_rn(x[i].y * f, x[i + 4].y * f));
      }
      const int lr = row & 127;
      uint8_t* base = sm + (row >> 7) * (128 * D * 2) + (j >> 2) * (128 * 128) + (lr >> 3) * 1024 + (lr & 7) * 128;
      const int c = (2 * j) & 7;
      *reinterpret_cast<uint4*>(base + ((c ^ (lr & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(base + (((c + 1) ^ (lr & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    fence_async_shared();
  }
  // those that use Q wait for it
  if (warp <= kMmaWarp && (warp < kDecodeWarp0 || warp == kMmaWarp)) asm volatile("bar.sync 1, %0;" ::"n"(17 * 32) : "memory");

  struct {
    float m, l;
    bool poison, any;
  } result = {kNone, 0.0f, false, false};
  if (warp >= kMmaWarp) {
    regs_down<kOtherRegs>();
    if (warp == kFeedWarp) {
      // ---- feed ----------------------------------------------------------------
      if (elect_one()) {
        int e = -1, f = -1;
        uint32_t lap = 0;                                  // parity of n / n_raw
        int n = 0;
        for (; n < 2 * w.n; ++n) {
          const int t = w.t0 + (n >> 1) * BN;
          const int blk = __ldg(table + t / kBlockTokens);
          if (++e == n_raw) e = 0, lap ^= 1;
          if (++f == 2 * n_raw) f = 0;
          wait(&ms->raw_empty[e], lap ^ 1, gate);
          if (*reinterpret_cast<volatile int*>(&ms->abort) != 0) break;
          uint64_t* full = &ms->raw_full[f];
          uint8_t* dst = sm + G::kRawAt + e * raw_stride;
          if (blk < 0 || blk >= P.n_blocks()) {
            raise_error(P.error_word, Q4KV_DEVERR_BLOCK_ID);
            ms->raw_what[e] = 0;
            mbar_arrive(full);
          } else {
            const int bits = P.bits_of(blk);
            const int64_t phys = bits == 4 ? blk : (bits == 8 ? blk - P.n_q4 : blk - P.n_q4 - P.n_q8);
            const int64_t row = (phys * P.n_kv_heads + w.h) * kBlockTokens + t % kBlockTokens;
            const bool key = (n & 1) == 0;
            const uint8_t* codes = bits == 4 ? (key ? P.k_codes4 : P.v_codes4)
                                             : (bits == 8 ? (key ? P.k_codes8 : P.v_codes8) : (key ? P.k_codes2 : P.v_codes2));
            const __half2* params = bits == 4 ? (key ? P.k_params4 : P.v_params4)
                                              : (bits == 8 ? (key ? P.k_params8 : P.v_params8) : (key ? P.k_params2 : P.v_params2));
            // (the scales of 8-bit codes stay in global memory: the ring has no room for them)
            const uint32_t cb = BN * D / 8 * bits, pb = bits == 8 ? 0 : BN * (D / kGroup) * 4;
            ms->raw_what[e] = static_cast<uint32_t>(phys) << 4 | static_cast<uint32_t>(bits);
            mbar_arrive_tx(full, cb + pb + 16);
            bulk_g2s(dst, codes + row * (D / 8 * bits), cb, full);
            if (pb > 0) bulk_g2s(dst + raw_stride - 16 - BN * (D / kGroup) * 4, params + row * (D / kGroup), pb, full);
            bulk_g2s(dst + raw_stride - 16, P.mask + static_cast<int64_t>(blk) * kMaskWords + (t % kBlockTokens) / 128 * 4, 16, full);
          }
        }
        ms->issued = n;
      }
    } else if (warp == kMmaWarp) {
      // ---- product -------------------------------------------------------------
      if (elect_one()) {
        constexpr uint32_t kQk = mma_f16_desc(128, BN, false), kPv = mma_f16_desc(128, D, true);
        const uint64_t q0 = smem_operand(smem_u32(sm), 16, 1024), k0 = smem_operand(smem_u32(sm) + G::kQ, 16, 1024),
                       v0 = smem_operand(smem_u32(sm) + G::kQ, BN * 128, 1024);
        // O += P V of step v of accumulator s
        auto pv = [&](int s, int v) {
          const int j = G::ALT ? 2 * (v / G::STEPS) + s : v / G::STEPS, h = v % G::STEPS, n = 2 * j + 1;
          if (h == 0 && (MODE != 0 || s == 0)) wait(&ms->kv_full[n % kSlots], (n / kSlots) & 1, gate);   // first use
          wait(&ms->p_full[s][v & 1], (v >> 1) & 1, gate);
          tc_fence_after();
          const uint32_t p = tmem + kSBase + s * (2 * kCols) + (v & 1) * kCols;
          const uint64_t vd = v0 + (((n % kSlots) * kTile + h * (kCols * 128)) >> 4);
#pragma unroll
          for (int k = 0; k < kCols / 16; ++k) mma_ts(tmem + s * 128, p + k * 8, vd + k * (2048 >> 4), kPv, v > 0 || k > 0);
          mma_commit(&ms->o_done[s][v & 1]);
          if (h == G::STEPS - 1 && (MODE != 0 || s == groups - 1)) mma_commit(&ms->kv_empty[n % (2 * kSlots)]);
        };
        // S = Q K^T of accumulator s's tile i.  (The products that read the
        // weights in these buffers were issued before; products of one thread
        // run in order.)
        auto qk = [&](int s, int i) {
          const int j = G::ALT ? 2 * i + s : i, n = 2 * j;
          if (MODE != 0 || s == 0) {
            wait(&ms->kv_full[n % kSlots], (n / kSlots) & 1, gate);
            tc_fence_after();
          }
          const uint64_t qd = q0 + (MODE == 0 ? s * (128 * D * 2 >> 4) : 0), kd = k0 + ((n % kSlots) * kTile >> 4);
          const uint32_t logits = tmem + kSBase + s * (2 * kCols) + (G::STEPS == 1 ? (i & 1) * kCols : 0);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(logits, qd + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4), kd + (((k >> 2) * (BN * 128) + (k & 3) * 32) >> 4), kQk,
                   k > 0);
          if (G::STEPS == 1) {
            mma_commit(&ms->s_full[s][i & 1]);
          } else {
            mma_commit(&ms->s_full[s][0]);
            mma_commit(&ms->s_full[s][1]);
          }
          if (MODE != 0 || s == groups - 1) mma_commit(&ms->kv_empty[n % (2 * kSlots)]);
        };
        // logits of a tile of 128 tokens fill both buffers; of 64, one of two
        constexpr int kAhead = G::STEPS == 1 ? 2 : 1;
        for (int i = 0; i < steps0 / G::STEPS + kAhead; ++i)
          for (int s = 0; s < groups; ++s) {
            const int tiles = (s == 0 ? steps0 : steps1) / G::STEPS;
            if (i >= kAhead && i - kAhead < tiles)
              for (int h = 0; h < G::STEPS; ++h) pv(s, (i - kAhead) * G::STEPS + h);
            if (i < tiles) qk(s, i);
          }
      }
    }
    __syncwarp();
  } else if (warp >= kDecodeWarp0) {
    if (G::kDecodeRegs > kRegs) regs_up<G::kDecodeRegs>();
    else regs_down<G::kDecodeRegs>();
    // ---- decode ----------------------------------------------------------------
    const int dw = warp & 3, kind = (warp - kDecodeWarp0) >> 2;
    // a warp takes 8 tokens x 128 channels or 4 x 256 at a time, a lane 32
    // channels of one token; the tokens are skewed over the lanes so that both
    // the reads of codes and the swizzled writes are free of bank conflicts
    Lane ln;
    ln.u = D == 128 ? lane & 3 : lane & 7;
    ln.t = D == 128 ? dw * 8 + ((((lane >> 2) & 1) + 2 * (ln.u >> 1) + 2 * (lane >> 3)) & 7)
                    : dw * 4 + (((ln.u >> 1) + (lane >> 3)) & 3);
    const uint32_t dst0 = (ln.u >> 1) * (BN * 128) + (ln.t >> 3) * 1024 + (ln.t & 7) * 128;
    int e = kind, f = kind;                                // n % n_raw, n % (2 n_raw)
    uint32_t lap = 0;                                      // parity of n / (2 n_raw)
    for (int n = kind; n < 2 * w.n; n += 2) {
      warp_wait(&ms->raw_full[f], lap, gate);
      const uint32_t what = __shfl_sync(0xffffffffu, ms->raw_what[e], 0);   // (one branch for the warp, even where a wait gave up)
      const int bits = what & 15u;
      uint8_t* raw = sm + G::kRawAt + e * raw_stride;
      uint8_t* params = raw + raw_stride - 16 - BN * (D / kGroup) * 4;
      const int t0 = w.t0 + (n >> 1) * BN;
      // which of the lane's four tokens count
      uint32_t live = 0;
      {
        const uint4 m = *reinterpret_cast<const uint4*>(raw + raw_stride - 16);
        const bool upper = D == 256 && (t0 & 64) != 0;
        const uint32_t m0 = upper ? m.z : m.x, m1 = upper ? m.w : m.y;
        const uint32_t word[4] = {m0, D == 128 ? m1 : m0, D == 128 ? m.z : m1, D == 128 ? m.w : m1};
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int bit = D == 128 ? ln.t : ln.t + 16 * (it & 1);
          if (t0 + ln.t + it * Lane::step(D) < end && !((word[it] >> bit) & 1u)) live |= 1u << it;
        }
      }
      if (bits == 0) live = 0;
      if (kind == 0 && dw == 0 && lane < 4) {
        const int j = (n >> 1) & 7;
        const uint32_t* mask = reinterpret_cast<const uint32_t*>(raw + raw_stride - 16);
        ms->gone[j][lane] = bits == 0 ? 0u : mask[D == 256 && (t0 & 64) != 0 ? (lane & 1) + 2 : lane];
        if (lane == 0) ms->bad[j] = bits == 0;
      }
      const int before = n - kSlots;                       // the tile that was in the slot
      if (before >= 0) warp_wait(&ms->kv_empty[before % (2 * kSlots)], (before / (2 * kSlots)) & 1, gate);
      uint8_t* dst = sm + G::kQ + (n % kSlots) * kTile + dst0;
      const bool key = kind == 0;
      if (FP8) decode_tile<D, 0, G::kAtOnce>(raw, params, ln, live, dst, !key, key, t0, ms);
      else if (bits == 8) {
        uint8_t* global = reinterpret_cast<uint8_t*>(key ? P.k_params8 : P.v_params8) +
                          ((static_cast<int64_t>(what >> 4) * P.n_kv_heads + w.h) * kBlockTokens + t0 % kBlockTokens) *
                              (D / kGroup * 4);
        const bool odd = odd_groups<D, 255>(global, nullptr, key, dw, lane, t0, end, ms);
        decode_tile<D, 8, G::kAtOnce>(raw, global, ln, live, dst, odd, key, t0, ms);
      } else if (bits == 2) {
        odd_groups<D, 3>(params, raw + raw_stride - 16, key, dw, lane, t0, end, ms);
        decode_tile<D, 2, G::kAtOnce>(raw, params, ln, live, dst, false, key, t0, ms);
      } else {                                             // (or no block: nothing is live)
        odd_groups<D, 15>(params, raw + raw_stride - 16, key, dw, lane, t0, end, ms);
        decode_tile<D, 4, G::kAtOnce>(raw, params, ln, live, dst, false, key, t0, ms);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms->raw_empty[e]);
        mbar_arrive(&ms->kv_full[n % kSlots]);
      }
      if ((e += 2) >= n_raw) e -= n_raw;
      if ((f += 2) >= 2 * n_raw) f -= 2 * n_raw, lap ^= 1;
    }
  } else {
    if (G::kSoftRegs > kRegs) regs_up<G::kSoftRegs>();
    else regs_down<G::kSoftRegs>();
    if (group < 2 && (warp & 3) < (group == 0 ? warps0 : warps1)) {
      // ---- softmax -------------------------------------------------------------
      const int local = (MODE == 0 ? group * 128 : 0) + (G::COPIES == 4 ? 0 : (warp & 3) * 32) + lane;
      constexpr int kShare = kCols / G::COPIES;            // of a step's columns
      const int col0 = G::COPIES == 4 ? (warp & 3) * kShare : 0;
      const int r = w.r0 + local;
      const bool real = r < w.rv;
      const int pos = w.len + min(r, w.rv - 1) / w.g;      // the row's position
      // 2^exponent: from products to logits (rows behind the last real one take its place)
      const float rs = __uint_as_float(static_cast<uint32_t>(127 - 6 + ms->exponent[min(r, w.rv - 1) - w.r0]) << 23);
      // positions of the warp's first and last row: a step that all of them see
      // whole needs no mask
      const int pos_first = w.len + (w.r0 + local - lane) / w.g, pos_last = w.len + min(w.r0 + local - lane + 31, w.rv - 1) / w.g;
      const float sent = Q4KV_SENTINEL_LOGIT * kLog2e / rs;   // a remapped slot's logit before scaling
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t o_at = tmem + lanes + group * 128;
      const int steps = group == 0 ? steps0 : steps1;
      // first token of step k
      auto token = [&](int k) {
        return w.t0 + (G::ALT ? (2 * (k / G::STEPS) + group) * BN + k % G::STEPS * kCols : k * kCols);
      };
      float m = kNone, l = 0.0f;
      bool poison = false;
      const float2 rs2 = make_float2(rs, rs);
      uint64_t* turn = &ms->turn[group][warp & 3];
      float* reference = &ms->reference[group * 128 + (warp & 3) * 32 + lane];
      const uint32_t s_at = tmem + lanes + kSBase + group * (2 * kCols) + side * kCols;

#pragma unroll 1
      for (int k = side; k < steps; k += 2) {
        const int t0 = token(k);
        const int hi = pos - t0 - col0;                    // last column the row sees
        const int lo = a.plan.window > 0 ? pos - a.plan.window + 1 - t0 - col0 : 0;
        constexpr int kHalf = kShare / 2;
        uint32_t x[2][kHalf];
        warp_wait(&ms->s_full[group][side], (k >> 1) & 1, gate);
        tc_fence_after();
        tmem_load(s_at + col0, x[0]);
        tmem_load(s_at + col0 + kHalf, x[1]);
        // (the key decoders wrote this before the tile that the logits come from)
        const int j = G::ALT ? 2 * (k / G::STEPS) + group : k / G::STEPS;
        uint2 gone;
        if (G::COPIES == 4) {
          const uint32_t g = reinterpret_cast<const uint16_t*>(&ms->gone[j & 7][2 * (k % G::STEPS)])[warp & 3];
          gone = make_uint2(g & 0xFFu, g >> 8);
        } else {
          gone = *reinterpret_cast<const uint2*>(&ms->gone[j & 7][2 * (k % G::STEPS)]);
        }
        const bool bad = ms->bad[j & 7] != 0;
        const bool edge = pos_first - t0 < kCols - 1 || (a.plan.window != 0 && pos_last - a.plan.window >= t0);
        tmem_wait_ld(x[0]);
        tmem_wait_ld(x[1]);
        if (bad && hi + col0 >= 0 && lo + col0 < kCols) poison = true;
        if ((gone.x | gone.y) != 0) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) {
            if ((gone.x >> i) & 1u) x[0][i] = __float_as_uint(sent);
            if ((gone.y >> i) & 1u) x[1][i] = __float_as_uint(sent);
          }
        }
        if (edge) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int h1 = hi - kHalf * c, l1 = lo - kHalf * c;
            uint32_t seen = h1 >= 31 ? 0xffffffffu : (h1 < 0 ? 0u : (2u << h1) - 1u);
            seen &= l1 <= 0 ? 0xffffffffu : (l1 > 31 ? 0u : 0xffffffffu << l1);
#pragma unroll
            for (int i = 0; i < kHalf; ++i)
              if (!((seen >> i) & 1u)) x[c][i] = __float_as_uint(-INFINITY);
          }
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = fmaxf(__uint_as_float(x[q & 1][q >> 1]), __uint_as_float(x[q & 1][(q >> 1) + 2]));
#pragma unroll
        for (int i = 4; i < kHalf; i += 4)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mx[q] = max3(mx[q], __uint_as_float(x[q & 1][i + (q >> 1)]), __uint_as_float(x[q & 1][i + 2 + (q >> 1)]));
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * rs;
        // the reference after the step before, which the other group settles
        float ref = kNone;
        if (k > 0) {
          warp_wait(turn, (k - 1) & 1, gate);
          ref = *reinterpret_cast<volatile float*>(reference);
        }
        if (__any_sync(0xffffffffu, real && top > ref + kLazy)) {
          // Move it: it stays a whole number, so everything scaled by it scales
          // by a power of two.
          const float to = fmaxf(ceilf(fmaxf(ref, top)), kNone);
          if (k > 0) {
            const float f = __int_as_float((static_cast<int>(fmaxf(ref - to, -127.0f)) + 127) << 23);
            warp_wait(&ms->o_done[group][side ^ 1], ((k - 1) >> 1) & 1, gate);
            tc_fence_after();
#pragma unroll 1
            for (int e = 0; e < D / 8; ++e) {
              uint32_t o[8];
              tmem_ld8(o_at + 8 * e, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st8(o_at + 8 * e, o);
            }
          }
          ref = to;
        }
        if (k == 0 || ref != m) *reinterpret_cast<volatile float*>(reference) = ref;
        __syncwarp();
        if (lane == 0) mbar_arrive(turn);
        l *= exp2_fast(m - ref);                           // (the group's sum goes by the reference it last saw)
        m = ref;
        const float2 off2 = make_float2(kShift - m, kShift - m);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < kShare / 8; ++c) {
          uint32_t p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = 4 * c + i;
            const float2 e = __ffma2_rn(make_float2(__uint_as_float(x[2 * at / kHalf][2 * at % kHalf]), __uint_as_float(x[2 * at / kHalf][2 * at % kHalf + 1])),
                                        rs2, off2);
            const float2 q = make_float2(exp2_fast(e.x), exp2_fast(e.y));
            sum[i & 1] = __fadd2_rn(sum[i & 1], q);
            p[i] = h2u(__floats2half2_rn(q.x, q.y));
          }
          tmem_st4(s_at + col0 / 2 + 4 * c, p);
        }
        if (G::COPIES == 4) {
          const uint32_t zero[8] = {};
#pragma unroll
          for (int q = 1; q < 4; ++q) tmem_st8(s_at + 8 * (((warp & 3) + q) & 3), zero);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms->p_full[group][side]);
      }
      // The last product: the group that made its weights has seen the product
      // two before it, as a wait on that barrier has to.
      if (steps > 0 && ((steps - 1) & 1) == side) warp_wait(&ms->o_done[group][(steps - 1) & 1], ((steps - 1) >> 1) & 1, gate);
      result.m = m;
      result.l = l;
      result.poison = poison;
      result.any = steps > 0;
    }
  }
  tc_fence_before();
  __syncthreads();         // every product is done: the places of the tiles, packed and decoded, are free
  // Or somebody's wait gave up (no role waits any more, so all threads see the
  // same): the copies and products in flight are waited for here, where no role
  // can give up behind them.  A place was filled again only after its copy had been
  // seen to land, so only the last n_raw copies can be on their way.
  if (*reinterpret_cast<volatile int*>(&ms->abort) != 0) {
    if (warp == kFeedWarp && elect_one())
      for (int c = max(0, ms->issued - n_raw); c < ms->issued; ++c) mbar_wait(&ms->raw_full[c % (2 * n_raw)], (c / (2 * n_raw)) & 1);
    if (warp == kMmaWarp && elect_one()) {
      mma_commit(&ms->spare);
      mbar_wait(&ms->spare, 0);
    }
    __syncthreads();
  }
  tc_fence_after();
  // what the groups of the same rows have, in the packed tiles' place
  float4* told = reinterpret_cast<float4*>(sm + G::kRawAt);
  const int place = (group * 2 + side) * 128 + (warp & 3) * 32 + lane;
  const bool mine_real = warp < kDecodeWarp0 && group < 2 && (warp & 3) < (group == 0 ? warps0 : warps1);
  if (mine_real) told[place] = make_float4(result.m, result.l, result.poison ? 1.0f : 0.0f, 0.0f);
  __syncthreads();

  // ---- result ------------------------------------------------------------------
  // The rows go through shared memory, 16 bytes a lane and swizzled by the row,
  // and every warp then writes whole rows.
  const bool wide = partials > 1 || a.out_dtype == Q4KV_F32;
  const int pieces = wide ? D / 4 : D / 8;                 // 16-byte pieces of a row
  const int64_t part = static_cast<int64_t>(w.split) * G::STREAMS * all_rows;
  uint8_t* stage = sm + G::kQ;
  if (mine_real) {
    const bool ok = ms->abort == 0;
    const float4 other = told[place ^ 128];
    const float top = fmaxf(result.m, other.x);            // (references only grow: the last one)
    result.l = result.l * exp2_fast(result.m - top) + other.y * exp2_fast(other.x - top);
    result.m = top;
    result.poison = result.poison || other.z != 0.0f;
    const int r = w.r0 + (MODE == 0 ? group * 128 : 0) + (G::COPIES == 4 ? 0 : (warp & 3) * 32) + lane;
    float copy = 1.0f;       // this copy's accumulator goes by its own reference
    if (G::COPIES == 4) {
      float l = 0.0f, m = kNone;
#pragma unroll
      for (int q = 0; q < 8; ++q) m = fmaxf(m, told[(group * 2 + (q & 1)) * 128 + (q >> 1) * 32 + lane].x);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 one = told[(group * 2 + (q & 1)) * 128 + (q >> 1) * 32 + lane];
        l += one.y * exp2_fast(one.x - m);
      }
      copy = exp2_fast(result.m - m);
      result.m = m;
      result.l = l;
    }
    if (ms->odd_last >= 0) {
      const int pos = w.len + min(r, w.rv - 1) / w.g;
      const int seen = a.plan.window > 0 ? max(0, pos - a.plan.window + 1) : 0;
      for (int t = max(ms->odd_first, seen); t <= min(ms->odd_last, pos); ++t)
        if (odd_token<D>(P, table, w.h, t)) result.l = NAN;
    }
    // (a sum that is NaN: a query or a seen token is not finite; then so is the row)
    const bool fine = ok && !result.poison && !(result.l <= 0.0f);
    if (partials > 1 && r < w.rv && side == 0 && (G::COPIES == 1 || (warp & 3) == 0))
      a.ws_ml[part + (G::ALT ? group : 0) * all_rows + (static_cast<int64_t>(w.b) * w.T + r / w.g) * hq + w.h * w.g + r % w.g] =
          make_float2(!ok ? 0.0f : !(result.l <= 0.0f) ? result.m : -INFINITY, ok && !result.poison ? result.l : -1.0f);
    if (result.any) {
      const uint32_t o_at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + group * 128;
      const float f = partials > 1 ? copy : (fine ? 1.0f / result.l : 0.0f);
      uint8_t* mine = stage + (group * 128 + (warp & 3) * 32 + lane) * (pieces * 16);
#pragma unroll 1
      for (int c = side * (D / 64); c < (side + 1) * (D / 64); ++c) {
        uint32_t x[32];
        float y[32];
        tmem_ld32(o_at + 32 * c, x);
        tmem_wait_ld(x);
        channel_order(x, f, y);
        if (partials == 1 && !fine) {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = 0.0f;
        }
        if (wide) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(mine + ((8 * c + e) ^ (lane & 7)) * 16) = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(mine + ((4 * c + e) ^ (lane & 7)) * 16) =
                make_uint4(pack16(a.out_dtype, y[8 * e], y[8 * e + 1]), pack16(a.out_dtype, y[8 * e + 2], y[8 * e + 3]),
                           pack16(a.out_dtype, y[8 * e + 4], y[8 * e + 5]), pack16(a.out_dtype, y[8 * e + 6], y[8 * e + 7]));
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  {
    const int rows = w.rv - w.r0;
    for (int x = warp; x < (G::ALT && steps1 > 0 ? 2 : 1) * rows; x += kThreads / 32) {
      const int s = G::ALT && x >= rows ? 1 : 0, q = x - s * rows, r = w.r0 + q;
      const int i = r / w.g, head = w.h * w.g + r % w.g;
      uint8_t* dst;
      if (partials > 1) dst = reinterpret_cast<uint8_t*>(a.ws_o + (part + s * all_rows + (static_cast<int64_t>(w.b) * w.T + i) * hq + head) * D);
      else dst = static_cast<uint8_t*>(a.out) + (w.b * a.o_seq_stride + i * a.o_token_stride + static_cast<int64_t>(head) * D) * (wide ? 4 : 2);
      const uint8_t* src = stage + (G::ALT ? s * 128 + q : q) * (pieces * 16);
      for (int e = lane; e < pieces; e += 32) {
        uint4 v = *reinterpret_cast<const uint4*>(src + (e ^ (q & 7)) * 16);
        if (G::COPIES == 4) {
          float4 y = *reinterpret_cast<const float4*>(&v);
#pragma unroll
          for (int c = 1; c < 4; ++c) {
            const float4 o = *reinterpret_cast<const float4*>(src + c * 32 * (pieces * 16) + (e ^ (q & 7)) * 16);
            y = make_float4(y.x + o.x, y.y + o.y, y.z + o.z, y.w + o.w);
          }
          v = *reinterpret_cast<const uint4*>(&y);
        }
        reinterpret_cast<uint4*>(dst)[e] = v;
      }
    }
  }
  if (tid == 0 && ms->abort != 0) raise_error(P.error_word, Q4KV_DEVERR_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// Merge of a row's partial results; a warp per row.
template <int D>
__global__ void __launch_bounds__(256) extend_merge_kernel(const __grid_constant__ ExtendArgs a, int partials, int64_t rows) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int hq = a.plan.n_q_heads, T = a.plan.max_new;
  const int head = static_cast<int>(row % hq), i = static_cast<int>(row / hq % T), b = static_cast<int>(row / hq / T);
  const int len = __ldg(a.seq_lens + b), nn = a.n_new == nullptr ? T : max(0, min(__ldg(a.n_new + b), T));
  const bool real = i < nn && len >= 0 && static_cast<int64_t>(len) + nn <= static_cast<int64_t>(a.plan.max_blocks_per_seq) * kBlockTokens;
  constexpr int E = D / 32;
  float acc[E] = {}, L = 0.0f, M = -INFINITY;
  bool poison = false;
  if (real) {
    for (int p = lane; p < partials; p += 32) {
      const float2 v = a.ws_ml[p * rows + row];
      M = fmaxf(M, v.x);
      poison |= v.y < 0.0f;
    }
#pragma unroll
    for (int st = 1; st < 32; st <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, st));
    poison = __any_sync(0xffffffffu, poison);
    if (!poison && M != -INFINITY) {
      // four partial results at a time, their loads together
      for (int p0 = 0; p0 < partials; p0 += 4) {
        float2 v[4];
        float4 x[4][E / 4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (p0 + q < partials) {
            const int64_t part = (p0 + q) * rows + row;
            v[q] = a.ws_ml[part];
#pragma unroll
            for (int e = 0; e < E / 4; ++e) x[q][e] = *reinterpret_cast<const float4*>(a.ws_o + part * D + lane * E + 4 * e);
          }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (p0 + q < partials && v[q].x != -INFINITY) {   // (one that saw no keys has written no accumulator)
            const float f = exp2f(v[q].x - M);
            L = fmaf(v[q].y, f, L);
#pragma unroll
            for (int e = 0; e < E / 4; ++e) {
              acc[4 * e] = fmaf(x[q][e].x, f, acc[4 * e]);
              acc[4 * e + 1] = fmaf(x[q][e].y, f, acc[4 * e + 1]);
              acc[4 * e + 2] = fmaf(x[q][e].z, f, acc[4 * e + 2]);
              acc[4 * e + 3] = fmaf(x[q][e].w, f, acc[4 * e + 3]);
            }
          }
      }
    }
  }
  const float f = L <= 0.0f ? 0.0f : 1.0f / L;
  const int64_t at = b * a.o_seq_stride + i * a.o_token_stride + static_cast<int64_t>(head) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    const float y[4] = {acc[e] * f, acc[e + 1] * f, acc[e + 2] * f, acc[e + 3] * f};
    if (a.out_dtype == Q4KV_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + e) = make_float4(y[0], y[1], y[2], y[3]);
    } else if (a.out_dtype == Q4KV_F16) {
      *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at + e) =
          make_uint2(h2u(__floats2half2_rn(y[0], y[1])), h2u(__floats2half2_rn(y[2], y[3])));
    } else {
      const __nv_bfloat162 u = __floats2bfloat162_rn(y[0], y[1]), v = __floats2bfloat162_rn(y[2], y[3]);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at + e) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
    }
  }
}

template <int MODE, bool FP8>
cudaError_t launch_mode(const ExtendArgs& a, cudaStream_t stream) {
  using G = Geo<MODE>;
  const q4kv_extend_plan& p = a.plan;
  const int64_t group_rows = static_cast<int64_t>(p.max_new) * (p.n_q_heads / p.n_kv_heads);
  const int64_t x = (group_rows + G::R - 1) / G::R * p.n_splits;
  if (x > 0x7fffffff) return cudaErrorInvalidValue;
  // packed codes, scales (except for 8-bit codes) and mask
  const uint32_t stride = a.pool.n_q8 > 0 ? G::BN * G::D + 16 : G::BN * G::D / 2 + G::BN * (G::D / kGroup) * 4 + 16;
  const int n_raw = min(kMaxRaw, static_cast<int>(G::kRawRing / stride));
  constexpr uint32_t kSmem = smem_bytes<MODE>();
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, extend_kernel<MODE, FP8>);
  if (e != cudaSuccess) return e;
  if (attr.numRegs != kRegs) return cudaErrorInvalidKernelImage;   // the register shares would not add up
  e = cudaFuncSetAttribute(extend_kernel<MODE, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(extend_kernel<MODE, FP8>, dim3(static_cast<unsigned>(x), p.n_kv_heads, p.batch), dim3(kThreads), kSmem, stream, a,
                 stride, n_raw);
  if (e != cudaSuccess) return e;
  const int partials = p.n_splits * G::STREAMS;
  if (partials == 1) return cudaSuccess;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.max_new * p.n_q_heads;
  return launch_pdl(extend_merge_kernel<G::D>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, stream, a, partials,
                    rows);
}

}  // namespace

cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t stream) {
  const q4kv_extend_plan& p = a.plan;
  const int64_t group_rows = static_cast<int64_t>(p.max_new) * (p.n_q_heads / p.n_kv_heads);
  const ExtendShape sh = extend_shape(p.head_dim, group_rows);
  if (a.pool.fp8) {
    if (p.head_dim == 256) return launch_mode<2, true>(a, stream);
    if (sh.rows == 256) return launch_mode<0, true>(a, stream);
    return group_rows <= 32 ? launch_mode<3, true>(a, stream) : launch_mode<1, true>(a, stream);
  }
  if (p.head_dim == 256) return launch_mode<2, false>(a, stream);
  if (sh.rows == 256) return launch_mode<0, false>(a, stream);
  return group_rows <= 32 ? launch_mode<3, false>(a, stream) : launch_mode<1, false>(a, stream);
}

}  // namespace q4kv
