// Join of the partial results of a shared-prefix attention call: one (row, query head) per warp,
//   lse = log sum_s exp(lse_s),  o = v_scale_post sum_s exp(lse_s - lse) o_s,
// over the parts of the prefix and of the row's own keys, rounded once to the output's 16-bit type.
// Rows that see nothing get o = 0, lse = -inf; padding rows are left as they were.
// The partials come out of L2 (they were written just before).
#include "prefix_umma.cuh"

namespace qkv {
namespace prefix {
namespace {

template <int HD>
__global__ void __launch_bounds__(128) prefix_merge_kernel(const PrefixArgs a, float v_scale_post) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);  // (row, head)
  const int64_t stride = a.rows * a.num_q_heads;
  if (unit >= stride) return;
  const int64_t row = unit / a.num_q_heads;
  const int state = row_state(a, row, lane == 0 && unit == row * a.num_q_heads);
  if (state == kPadRow) return;
  // the parts of the prefix that this pair's tile was cut into, then those of its own keys
  int pre = a.prefix_parts;
  if (a.umma_cg > 0) {
    const int G = a.num_q_heads / a.num_kv_heads, head = static_cast<int>(unit - row * a.num_q_heads), h = head / G;
    const int64_t nb = (a.prefix_len + a.umma_keys - 1) / a.umma_keys, total = a.umma_tiles * nb;
    const int64_t tile = static_cast<int64_t>(h) * a.umma_ptiles + (row * G + (head - h * G)) / a.umma_pairs;
    pre = static_cast<int>(team_of((tile + 1) * nb - 1, total, a.umma_teams) - team_of(tile * nb, total, a.umma_teams)) + 1;
  }
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
    for (int s0 = 0; s0 < parts; s0 += 32) {
      const float mine = s0 + lane < parts ? expf(__ldcg(lp + at(s0 + lane)) - ref) : 0.f;
      const int n = min(32, parts - s0);
#pragma unroll 4
      for (int s = 0; s < n; ++s) {
        const float w = __shfl_sync(0xffffffffu, mine, s);
        if (w == 0.f) continue;  // a part without keys wrote no values
        sum += w;
        const float4* src = reinterpret_cast<const float4*>(op + at(s0 + s) * HD);
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          const float4 x = __ldcg(src + lane + 32 * v);
          acc[v].x += w * x.x, acc[v].y += w * x.y, acc[v].z += w * x.z, acc[v].w += w * x.w;
        }
      }
    }
  }
  const float f = any ? v_scale_post / sum : 0.f;
#pragma unroll
  for (int v = 0; v < kVec; ++v)
    *reinterpret_cast<uint2*>(a.out + unit * HD + 4 * (lane + 32 * v)) =
        make_uint2(round2(a.q_f16, acc[v].x * f, acc[v].y * f), round2(a.q_f16, acc[v].z * f, acc[v].w * f));
  if (lane == 0 && a.lse != nullptr) a.lse[unit] = any ? ref + logf(sum) : -INFINITY;
}

}  // namespace
}  // namespace prefix

cudaError_t launch_prefix_merge(const PrefixArgs& a, float v_scale_post, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>((a.rows * a.num_q_heads + 3) / 4);
  if (a.head_dim == 256)
    prefix::prefix_merge_kernel<256><<<blocks, 128, 0, stream>>>(a, v_scale_post);
  else
    prefix::prefix_merge_kernel<128><<<blocks, 128, 0, stream>>>(a, v_scale_post);
  return cudaGetLastError();
}

}  // namespace qkv
