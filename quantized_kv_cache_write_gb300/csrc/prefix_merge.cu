// Join of the partial results of a shared-prefix attention call, one (row, query head) pair at a time:
//   lse = log sum_s exp(lse_s),  o = v_scale sum_s exp(lse_s - lse) o_s   (v_scale: E4M3's layer scale),
// over the parts of the prefix and of the row's own keys, rounded once to the output's 16-bit type.
// Rows that see nothing get o = 0, lse = -inf; padding rows are left as they were.
// The partials come out of L2 (they were written just before). With many parts four warps share a
// pair: each takes every fourth part, and shared memory joins them.
#include "prefix_umma.cuh"

namespace qkv {
namespace prefix {
namespace {

constexpr int kMergeWarps = 4;

// WP: warps per pair (1 or 4).
template <int HD, int WP>
__global__ void __launch_bounds__(32 * kMergeWarps) prefix_merge_kernel(const PrefixArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = WP == 1 ? 0 : warp;
  const int64_t unit = WP == 1 ? static_cast<int64_t>(blockIdx.x) * kMergeWarps + warp : blockIdx.x;  // pair
  const int64_t stride = a.rows * a.num_q_heads;
  if (unit >= stride) return;
  const int64_t row = unit / a.num_q_heads;
  const int state = row_state(a, row, lane == 0 && sub == 0 && unit == row * a.num_q_heads);
  // the parts of the prefix that this pair's tile was cut into, then those of its own keys
  int pre = a.prefix_parts;
  if (a.umma_cg > 0) {
    const int G = a.num_q_heads / a.num_kv_heads, head = static_cast<int>(unit - row * a.num_q_heads), h = head / G;
    const uint32_t pair = static_cast<uint32_t>(row) * G + (head - h * G);
    const uint32_t first = (static_cast<uint32_t>(h) * a.umma_ptiles + pair / a.umma_pairs) * a.umma_blocks;
    pre = static_cast<int>(team_of(a, first + a.umma_blocks - 1) - team_of(a, first)) + 1;
  }
  await_previous();
  if (state == kPadRow) return;
  const int skip = a.prefix_parts - pre;  // part numbers that this pair does not have
  const int parts = state == kEmptyRow ? 0 : pre + a.own_parts;
  auto at = [&](int s) -> int64_t { return (s < pre ? s : s + skip) * stride; };
  const float* lp = a.lse_part + unit;
  const float* op = a.o_part + unit * HD;
  float m = -INFINITY;
  bool nan = false;
  for (int s = lane; s < parts; s += 32) {
    const float v = __ldcg(lp + at(s));
    nan |= v != v;
    m = fmaxf(m, v);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  nan = __any_sync(0xffffffffu, nan);
  constexpr int kVec = HD / 128;
  float4 acc[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  const bool any = m != -INFINITY || nan;
  const float ref = m == -INFINITY ? 0.f : m;
  if (any) {
    // this warp's parts are sub + WP i; lane i holds the weight of the i-th of 32
    for (int s0 = sub; s0 < parts; s0 += 32 * WP) {
      const int mine_at = s0 + WP * lane;
      const float v = mine_at < parts ? __ldcg(lp + at(mine_at)) : -INFINITY;
      // a part without keys wrote no values: -1. One with keys counts though its weight is 0: its values may be NaN
      const float mine = v == -INFINITY ? -1.f : expf(v - ref);
      const int n = min(32, (parts - s0 + WP - 1) / WP);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float got = __shfl_sync(0xffffffffu, mine, i);
        const bool there = !(got < 0.f);
        const float w = there ? got : 0.f;
        sum += w;
        const float4* src = reinterpret_cast<const float4*>(op + at(s0 + WP * i) * HD);
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (there) x = __ldcg(src + lane + 32 * v);
          acc[v].x += w * x.x, acc[v].y += w * x.y, acc[v].z += w * x.z, acc[v].w += w * x.w;
        }
      }
    }
  }
  if (WP > 1) {
    __shared__ float4 sAcc[kMergeWarps][HD / 4];
    __shared__ float sSum[kMergeWarps];
#pragma unroll
    for (int v = 0; v < kVec; ++v) sAcc[warp][lane + 32 * v] = acc[v];
    if (lane == 0) sSum[warp] = sum;
    __syncthreads();
    if (warp >= kVec) return;
    sum = (sSum[0] + sSum[1]) + (sSum[2] + sSum[3]);
    const int col = lane + 32 * warp;
    float4 t = sAcc[0][col];
#pragma unroll
    for (int w = 1; w < kMergeWarps; ++w) {
      const float4 x = sAcc[w][col];
      t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
    }
    acc[0] = t;
  }
  const float f = any ? (a.merge_scale / sum) : 0.f;
#pragma unroll
  for (int v = 0; v < (WP > 1 ? 1 : kVec); ++v)
    *reinterpret_cast<uint2*>(a.out + unit * HD + 4 * (lane + 32 * (WP > 1 ? warp : v))) =
        make_uint2(round2(a.q_f16, acc[v].x * f, acc[v].y * f), round2(a.q_f16, acc[v].z * f, acc[v].w * f));
  if (lane == 0 && (WP == 1 || warp == 0) && a.lse != nullptr) a.lse[unit] = any ? ref + logf(sum) : -INFINITY;
}

// Four warps share a pair where there are at least so many parts and not enough pairs to fill the GPU with one
// warp each. us for the call, one warp | four: int8, 16 heads of 256, 8192 own keys: 16 pairs of 32 parts 20.5 | 15.0,
// 128 of 32 26.2 | 19.7, 512 of 16 51 | 48, 2048 of 16 161 | 158, 4096 of 10 276 | 278; one row of 65536, 16 of 128 parts
// 49 | 27. e4m3, 64 heads of 128, 4096 own keys: 256 pairs of 8 parts 15.1 | 13.8, 2048 of 8 67.7 | 67.1, 4096 of 5 108 |
// 111; behind 32768 shared keys 512 of 23 39.8 | 35.5, 2048 of 12 57.5 | 57.7, 4096 of 12 82.3 | 85.7. bf16, 16 heads of
// 256 behind 20000: 128 of 86 49.5 | 31.8, 2048 of 13 95.2 | 94.6.
constexpr int kSharedParts = 8;
constexpr int64_t kSharedPairs = 2048;

template <int HD>
cudaError_t launch_merge(const PrefixArgs& a, cudaStream_t stream) {
  const int64_t pairs = a.rows * a.num_q_heads;
  const bool overlaps = a.prefix_parts + a.own_parts > 0;
  if (a.prefix_parts + a.own_parts >= kSharedParts && pairs <= kSharedPairs)
    return launch_after(prefix_merge_kernel<HD, 4>, static_cast<unsigned>(pairs), 32 * kMergeWarps, 0, overlaps, stream, a);
  return launch_after(prefix_merge_kernel<HD, 1>, static_cast<unsigned>((pairs + kMergeWarps - 1) / kMergeWarps),
                      32 * kMergeWarps, 0, overlaps, stream, a);
}

}  // namespace
}  // namespace prefix

cudaError_t launch_prefix_merge(const PrefixArgs& a, cudaStream_t stream) {
  return a.head_dim == 256 ? prefix::launch_merge<256>(a, stream) : prefix::launch_merge<128>(a, stream);
}

}  // namespace qkv
