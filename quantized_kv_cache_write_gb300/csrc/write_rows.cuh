// Device helpers of the kernels that write head rows into a slot pool: widening, the int8 and
// E4M3 quantisers of one row, and the slot of a token.
#pragma once

#include "qkv_internal.cuh"

namespace qkv {
namespace {

struct HeadVec {
  float x[8];
};

// Eight consecutive 16-bit activations (bf16, or IEEE half when F16), loaded raw (streaming:
// the new tokens are consumed once) and widened exactly to fp32.
__device__ __forceinline__ uint4 load_raw8(const uint16_t* src) {
  uint4 raw;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w)
               : "l"(src));
  return raw;
}

template <bool F16>
__device__ __forceinline__ HeadVec widen8(const uint4& raw) {
  HeadVec h;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      h.x[2 * i] = f.x;
      h.x[2 * i + 1] = f.y;
    } else {
      h.x[2 * i] = bf16lo(w[i]);
      h.x[2 * i + 1] = bf16hi(w[i]);
    }
  }
  return h;
}

// int8 codes without a division per value. With r = fl(1 / s), the exact products
// x fl(r (1 -+ 2^-20)) lie below and above the IEEE quotient fl(x / s): the roundings of r and
// of r (1 -+ 2^-20) each move a value by at most 2^-24 of itself, so both products differ from
// x / s by more than 2^-22 of it, on opposite sides, and fl(x / s) by at most 2^-24. Rounding to
// an integer is monotonic, so where both products round to the same integer, fl(x / s) rounds to
// it as well; otherwise (x / s within about 2^-20 of a half-integer, a few values in 10^4) the
// division decides. This holds while r is a finite normal float: scales in [2^-100, 2^100];
// other scales always divide. (E4M3 keeps its division: a bracket there takes two conversions
// per pair instead of one, which measured slower than the divisions.)
constexpr float kBracket = 9.5367431640625e-07f;  // 2^-20
__device__ __forceinline__ bool bracket_ok(float s) { return s >= 7.8886090522101181e-31f && s <= 1.2676506002282294e30f; }
__device__ __forceinline__ float bracket_lo(float s) { return __fmul_rn(__frcp_rn(s), 1.0f - kBracket); }
__device__ __forceinline__ float bracket_hi(float s) { return __fmul_rn(__frcp_rn(s), 1.0f + kBracket); }
// RN(y + 1.5 2^23) holds rint(y), ties to even, in its low mantissa bits for |y| < 2^22; its low
// byte is the code's two's complement byte
constexpr float kRintMagic = 12582912.0f;

// Maximum over the W consecutive lanes that hold a row (the whole warp takes part).
template <int W = 32>
__device__ __forceinline__ float warp_max(float a) {
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
  return a;
}

// Whether a token's slot is written: false when it is skipped (-1) or out of range (flagged by
// lane 0 of the warp that `flags`, one per token).
__device__ __forceinline__ bool slot_ok(int64_t slot, int64_t num_slots, uint32_t* dev_status, int lane, bool flags) {
  if (slot == -1) return false;
  if (slot < -1 || slot >= num_slots) {
    if (lane == 0 && flags && dev_status != nullptr) atomicOr(dev_status, QKV_DEV_BAD_SLOT);
    return false;
  }
  return true;
}

// The slot of token t in a paged pool: -1 when its position is -1 (skipped); -2 (flagged, then
// skipped) for a position outside [-1, max_blocks * block_size), a sequence outside
// [0, num_seqs) or an unallocated block (id < 0); a slot past the pool is flagged by the caller.
__device__ __forceinline__ int64_t paged_slot(const WritePaging& pg, int64_t t, int64_t num_slots) {
  const int seq = __ldg(pg.token_seq + t), pos = __ldg(pg.token_pos + t);  // both loads in flight
  if (pos == -1) return -1;
  if (pos < -1 || static_cast<int64_t>(pos) >= static_cast<int64_t>(pg.max_blocks) * pg.block_size || seq < 0 ||
      seq >= pg.num_seqs)
    return -2;
  const int b = pos / pg.block_size;
  const int blk = __ldg(pg.block_table + static_cast<int64_t>(seq) * pg.max_blocks + b);
  if (blk < 0) return -2;
  return static_cast<int64_t>(blk) * pg.block_size + (pos - b * pg.block_size);
}

// int8 codes (four to a word) and the scale of one head row. W lanes hold the row; the whole warp takes part.
template <int W>
__device__ __forceinline__ float int8_codes(const HeadVec& hv, uint32_t (&word)[2]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(hv.x[i]));
  a = warp_max<W>(a);
  const float scale = __fdiv_rn(a, 127.0f);
  word[0] = word[1] = 0u;
  if (scale > 0.f) {
    // |x| <= amax and scale = fl(amax / 127) keep |x / scale| below 127.5, so the clamp never
    // acts on a finite value (a NaN value fails the bracket test and takes the clamped division)
    const bool br = bracket_ok(scale);
    const float rlo = bracket_lo(scale), rhi = bracket_hi(scale);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float lo = __fmaf_rn(hv.x[i], rlo, kRintMagic), hi = __fmaf_rn(hv.x[i], rhi, kRintMagic);
      c[i] = (br && lo == hi) ? __float_as_uint(lo)
                              : static_cast<uint32_t>(max(-127, min(127, __float2int_rn(__fdiv_rn(hv.x[i], scale)))));
    }
    // low bytes of c[4w .. 4w + 3] into word w, c[4w] lowest: two byte permutes per pair, one
    // to join the pairs
#pragma unroll
    for (int w = 0; w < 2; ++w)
      word[w] = __byte_perm(__byte_perm(c[4 * w], c[4 * w + 1], 0x0040), __byte_perm(c[4 * w + 2], c[4 * w + 3], 0x0040),
                            0x5410);
  }
  return scale;
}

// int8 codes and scale of one head row into record `rec` of `cache` (and `scale_out`, side layout).
// W lanes hold the row, `lane` counts them; the whole warp takes part, rows that are not stored too.
template <bool kInline, int W = 32>
__device__ __forceinline__ void store_int8_row(const HeadVec& hv, int lane, bool act, int head_dim, int64_t rec,
                                               uint8_t* __restrict__ cache, float* __restrict__ scale_out,
                                               bool stored = true) {
  uint32_t word[2];
  const float scale = int8_codes<W>(hv, word);
  if (!stored) return;
  if (kInline) {
    uint8_t* base = cache + rec * (head_dim + 4);  // head_dim codes, then the fp32 scale
    uint32_t* dst = reinterpret_cast<uint32_t*>(base + lane * 8);  // records are 4 B aligned
    if (act) {
      dst[0] = word[0];
      dst[1] = word[1];
    }
    if (lane == 0) *reinterpret_cast<float*>(base + head_dim) = scale;
  } else {
    if (act) *reinterpret_cast<uint2*>(cache + rec * head_dim + lane * 8) = make_uint2(word[0], word[1]);
    if (lane == 0) scale_out[rec] = scale;
  }
}

// E4M3 codes of eight values, four to a word.
__device__ __forceinline__ uint2 e4m3_codes(const HeadVec& hv, float s) {
  uint32_t p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 y = make_float2(__fdiv_rn(hv.x[2 * j], s), __fdiv_rn(hv.x[2 * j + 1], s));
    // .x lands in the low byte; round to nearest even, saturate to +-448, sign kept.
    p[j] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
  }
  // code pairs 2w, 2w + 1 into word w (low halves), one byte permute each
  return make_uint2(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410));
}

// E4M3 codes of one head row (lanes that own dims only) into record `rec` of `cache`.
__device__ __forceinline__ void store_e4m3_row(const HeadVec& hv, int lane, int head_dim, int64_t rec, float s,
                                               uint8_t* __restrict__ cache) {
  *reinterpret_cast<uint2*>(cache + rec * head_dim + lane * 8) = e4m3_codes(hv, s);
}

}  // namespace
}  // namespace qkv
