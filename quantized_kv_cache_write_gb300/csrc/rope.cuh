// Device helpers of the kernels that rotate head rows by position: the rotation of a pair, and the angles of
// tokens whose positions have several axes.
#pragma once

#include "write_rows.cuh"

namespace qkv {
namespace {

// Four consecutive 16-bit values; q through the ordinary path, as it may be rotated in place.
template <bool RW>
__device__ __forceinline__ uint2 load_raw4(const uint16_t* src) {
  uint2 raw;
  if (RW)
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n" : "=r"(raw.x), "=r"(raw.y) : "l"(src) : "memory");
  else
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n" : "=r"(raw.x), "=r"(raw.y) : "l"(src));
  return raw;
}
template <bool F16>
__device__ __forceinline__ uint2 round4(const float* x) {
  return F16 ? make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3])) : make_uint2(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]));
}
// (a, b) of a pair by its cosine and sine, every product and sum rounded. Scalar: packed pairs of products and
// sums are fused by the compiler, with one rounding less (seen as changed bytes).
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = a;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(x, s));
}

// A token's positions by axis (axes that the call does not have: 0).
struct TokenAxes {
  int pos[kMaxAxes];
  __device__ __forceinline__ void load(const RopeAxes& a, int64_t t, int64_t num_tokens) {
#pragma unroll
    for (int i = 0; i < kMaxAxes; ++i) pos[i] = i < a.num_axes ? __ldg(a.axis_pos + i * num_tokens + t) : 0;
  }
  __device__ __forceinline__ bool valid(const RopeAxes& a, int64_t num_positions) const {
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kMaxAxes; ++i) ok &= pos[i] >= 0 && (i >= a.num_axes || pos[i] < num_positions);
    return ok;
  }
  __device__ __forceinline__ int of(uint32_t axis) const {
    const int lo = axis & 1 ? pos[1] : pos[0], hi = axis & 1 ? pos[3] : pos[2];
    return axis & 2 ? hi : lo;
  }
};
// Cosines (at `half` further on: sines) of N pairs from `pair` on, a multiple of N, by their axes: a vector where
// they agree, which is the rule where the axes take runs of pairs.
template <int N>
__device__ __forceinline__ void axis_angles(const RopeAxes& a, const TokenAxes& t, const float* cos_sin, int rot, int pair,
                                            float (&c)[N], float (&s)[N]) {
  const uint32_t axes = a.pair_axis[pair >> 4] >> (2 * (pair & 15)) & (N == 4 ? 0xffu : 0xfu);
  const uint32_t first = axes & 3u;
  if (axes == first * (N == 4 ? 0x55u : 0x5u)) {
    const float* at = cos_sin + static_cast<int64_t>(t.of(first)) * rot + pair;
    if (N == 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(at)), y = __ldg(reinterpret_cast<const float4*>(at + (rot >> 1)));
      c[0] = x.x, c[1] = x.y, c[N - 2] = x.z, c[N - 1] = x.w;
      s[0] = y.x, s[1] = y.y, s[N - 2] = y.z, s[N - 1] = y.w;
    } else {
      const float2 x = __ldg(reinterpret_cast<const float2*>(at)), y = __ldg(reinterpret_cast<const float2*>(at + (rot >> 1)));
      c[0] = x.x, c[1] = x.y, s[0] = y.x, s[1] = y.y;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float* at = cos_sin + static_cast<int64_t>(t.of(axes >> (2 * i) & 3u)) * rot + pair + i;
    c[i] = __ldg(at), s[i] = __ldg(at + (rot >> 1));
  }
}
// The angles of a lane's two runs of four dims, from d0 and d1 on. Half-split pairs: the runs are partners, one
// angle per dim of the first; adjacent pairs: two of each run. Dims past the rotated ones get none.
template <bool PAIRS>
__device__ __forceinline__ void axes_angles(const RopeAxes& a, const TokenAxes& t, const float* cos_sin, int rot, int d0, int d1,
                                            float4& cs, float4& sn) {
  if (PAIRS) {
    float c[2], s[2];
    if (d0 < rot) axis_angles<2>(a, t, cos_sin, rot, d0 >> 1, c, s), cs.x = c[0], cs.y = c[1], sn.x = s[0], sn.y = s[1];
    if (d1 < rot) axis_angles<2>(a, t, cos_sin, rot, d1 >> 1, c, s), cs.z = c[0], cs.w = c[1], sn.z = s[0], sn.w = s[1];
  } else if (d0 < rot) {
    float c[4], s[4];
    axis_angles<4>(a, t, cos_sin, rot, d0, c, s);
    cs = make_float4(c[0], c[1], c[2], c[3]), sn = make_float4(s[0], s[1], s[2], s[3]);
  }
}

}  // namespace
}  // namespace qkv
