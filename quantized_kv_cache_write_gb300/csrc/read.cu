// The pool read back: K and V rows of given tokens, dequantised into contiguous tensors; K optionally turned back
// to before its rotation.
//
// A record's value is code * scale (fp32, one rounding; 16-bit pools: the value itself), and, turned back by its
// token's angle, for a pair (a, b):
//   a' = fl(fl(a c) + fl(b s)),   b' = fl(fl(b c) - fl(a s)),
// rounded once to the output's type. A 16-bit pool's values into its own type are copied as they are.
//
// The lanes hold a row as in append.cuh: head_dim / 8 lanes, two runs of four dims that are rotation partners. A
// warp takes kRows rows per lane group of one token, K heads first, then V heads.
#include "rope.cuh"

namespace qkv {
namespace {

constexpr int kReadThreads = 128;

// Four values of a record from dim d on, as fp32 (int8, E4M3: before their scale), and raw.
template <int FMT>
__device__ __forceinline__ uint2 record4(const uint8_t* rec, int d) {
  if (FMT == QKV_BF16 || FMT == QKV_F16) return load_raw4<false>(reinterpret_cast<const uint16_t*>(rec) + d);
  uint32_t w;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];\n" : "=r"(w) : "l"(rec + d));
  return make_uint2(w, 0);
}
template <int FMT>
__device__ __forceinline__ void widen4(const uint2& raw, float* x) {
  if (FMT == QKV_BF16) {
    x[0] = bf16lo(raw.x), x[1] = bf16hi(raw.x), x[2] = bf16lo(raw.y), x[3] = bf16hi(raw.y);
  } else if (FMT == QKV_INT8_SIDE || FMT == QKV_INT8_INLINE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(raw.x >> (8 * i)));
  } else {
    const uint32_t lo = FMT == QKV_F16 ? raw.x : e4m3pair_to_f16x2(raw.x), hi = FMT == QKV_F16 ? raw.y : e4m3pair_to_f16x2(raw.x >> 16);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&lo)), g = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[0] = f.x, x[1] = f.y, x[2] = g.x, x[3] = g.y;
  }
}

// TURN: 0 K as it is stored; 1 turned back, half-split pairs; 2 turned back, adjacent pairs.
template <int FMT, int HD, int TURN, int kRows>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadArgs a) {
  constexpr int W = HD / 8, kPerWarp = 32 / W;
  constexpr bool kInt8 = FMT == QKV_INT8_SIDE || FMT == QKV_INT8_INLINE, k16 = FMT == QKV_BF16 || FMT == QKV_F16;
  constexpr int kRecord = FMT == QKV_INT8_INLINE ? HD + 4 : k16 ? 2 * HD : HD;
  const int lane = threadIdx.x & 31, j = lane & (W - 1), sub = lane / W;
  const int hk = a.k_out != nullptr ? a.num_kv_heads : 0, rows = hk + (a.v_out != nullptr ? a.num_kv_heads : 0);
  const uint32_t units = static_cast<uint32_t>((rows + kRows * kPerWarp - 1) / (kRows * kPerWarp));
  const uint64_t wid = (static_cast<uint64_t>(blockIdx.x) * kReadThreads + threadIdx.x) >> 5;
  const uint64_t total = static_cast<uint64_t>(a.num_tokens) * units;
  if (wid >= total) return;  // warp-uniform
  const int64_t t = total <= 0xFFFFFFFFull ? static_cast<uint32_t>(wid) / units : static_cast<int64_t>(wid / units);
  const int u = static_cast<int>(wid - static_cast<uint64_t>(t) * units);
  const int r0 = u * kRows * kPerWarp + sub;
  TokenAxes ax;
  if (TURN) ax.load(a.axes, t, a.num_tokens);
  const int64_t slot = a.slot_mapping != nullptr ? __ldg(a.slot_mapping + t) : paged_slot(a.paging, t, a.num_slots);
  if (slot < 0 || slot >= a.num_slots) {
    if (slot != -1 && u == 0 && lane == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_INDEX);
    return;
  }
  if (TURN != 0 && !ax.valid(a.axes, a.num_positions)) {  // no angle: the token is skipped whole
    if (ax.pos[0] != -1 && u == 0 && lane == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_INDEX);
    return;
  }
  const int rot = a.rotary_dim, half = rot >> 1;
  int d0 = 4 * j, d1 = HD / 2 + 4 * j;
  if (TURN == 1) {
    if (8 * j < rot) d1 = half + 4 * j;
    else d0 = rot + 4 * (j - rot / 8), d1 = d0 + (HD - rot) / 2;
  }
  uint2 lo[kRows], hi[kRows];
  float scale[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + kPerWarp * i;
    lo[i] = hi[i] = make_uint2(0, 0);
    scale[i] = 0.f;
    if (r < rows) {
      const bool is_k = r < hk;
      const int64_t rec = slot * a.num_kv_heads + (is_k ? r : r - hk);
      const uint8_t* src = (is_k ? a.k_cache : a.v_cache) + rec * kRecord;
      lo[i] = record4<FMT>(src, d0), hi[i] = record4<FMT>(src, d1);
      if (FMT == QKV_INT8_INLINE) scale[i] = __ldg(reinterpret_cast<const float*>(src + HD));
      if (FMT == QKV_INT8_SIDE) scale[i] = __ldg((is_k ? a.k_scale : a.v_scale) + rec);
      if (FMT == QKV_E4M3) scale[i] = is_k ? a.k_scale_layer : a.v_scale_layer;
    }
  }
  float4 cs = make_float4(0.f, 0.f, 0.f, 0.f), sn = cs;
  if (TURN != 0 && u * kRows * kPerWarp < hk) axes_angles<TURN == 2>(a.axes, ax, a.cos_sin, rot, d0, d1, cs, sn);
  const bool turns0 = d0 < rot, turns1 = d1 < rot;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + kPerWarp * i;
    if (r >= rows) break;
    const bool is_k = r < hk;
    float x[8];
    widen4<FMT>(lo[i], x), widen4<FMT>(hi[i], x + 4);
    if (!k16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __fmul_rn(x[k], scale[i]);
    }
    if (TURN == 1 && is_k && turns0) {
      rotate(x[0], x[4], cs.x, -sn.x), rotate(x[1], x[5], cs.y, -sn.y);
      rotate(x[2], x[6], cs.z, -sn.z), rotate(x[3], x[7], cs.w, -sn.w);
    } else if (TURN == 2 && is_k) {
      if (turns0) rotate(x[0], x[1], cs.x, -sn.x), rotate(x[2], x[3], cs.y, -sn.y);
      if (turns1) rotate(x[4], x[5], cs.z, -sn.z), rotate(x[6], x[7], cs.w, -sn.w);
    }
    const int64_t at = t * a.out_stride + static_cast<int64_t>(is_k ? r : r - hk) * HD;
    void* out = is_k ? a.k_out : a.v_out;
    if (a.out_type == QKV_OUT_F32) {
      float* dst = static_cast<float*>(out) + at;
      *reinterpret_cast<float4*>(dst + d0) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(dst + d1) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      uint16_t* dst = static_cast<uint16_t*>(out) + at;
      uint2 p = a.out_type == QKV_OUT_F16 ? round4<true>(x) : round4<false>(x);
      uint2 q = a.out_type == QKV_OUT_F16 ? round4<true>(x + 4) : round4<false>(x + 4);
      const bool same = k16 && (FMT == QKV_F16) == (a.out_type == QKV_OUT_F16);
      if (same && !(TURN != 0 && is_k)) p = lo[i], q = hi[i];
      *reinterpret_cast<uint2*>(dst + d0) = p;
      *reinterpret_cast<uint2*>(dst + d1) = q;
    }
  }
}

// Rows per lane group: as in append.cuh, one while the launch does not fill the GPU.
constexpr int64_t kSmallWarps = 8192;

template <int FMT, int HD, int TURN>
cudaError_t launch(const ReadArgs& a, cudaStream_t stream) {
  constexpr int kPerWarp = 256 / HD;
  const int rows = a.num_kv_heads * ((a.k_out != nullptr ? 1 : 0) + (a.v_out != nullptr ? 1 : 0));
  const int64_t single = a.num_tokens * ((rows + kPerWarp - 1) / kPerWarp);
  auto blocks = [](int64_t warps) { return static_cast<unsigned>((warps * 32 + kReadThreads - 1) / kReadThreads); };
  if (single <= kSmallWarps)
    read_kernel<FMT, HD, TURN, 1><<<blocks(single), kReadThreads, 0, stream>>>(a);
  else
    read_kernel<FMT, HD, TURN, 4><<<blocks(a.num_tokens * ((rows + 4 * kPerWarp - 1) / (4 * kPerWarp))), kReadThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int FMT, int HD>
cudaError_t launch(const ReadArgs& a, cudaStream_t stream) {
  if (a.cos_sin == nullptr || a.k_out == nullptr) return launch<FMT, HD, 0>(a, stream);
  return a.interleaved ? launch<FMT, HD, 2>(a, stream) : launch<FMT, HD, 1>(a, stream);
}
template <int FMT>
cudaError_t launch(const ReadArgs& a, cudaStream_t stream) {
  return a.head_dim == 256 ? launch<FMT, 256>(a, stream) : launch<FMT, 128>(a, stream);
}

}  // namespace

cudaError_t launch_read(const ReadArgs& a, qkv_format fmt, cudaStream_t stream) {
  switch (fmt) {
    case QKV_BF16: return launch<QKV_BF16>(a, stream);
    case QKV_F16: return launch<QKV_F16>(a, stream);
    case QKV_INT8_SIDE: return launch<QKV_INT8_SIDE>(a, stream);
    case QKV_INT8_INLINE: return launch<QKV_INT8_INLINE>(a, stream);
    case QKV_E4M3: return launch<QKV_E4M3>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qkv
