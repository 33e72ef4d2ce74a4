// The pool read back: K and V rows of given tokens, dequantised into contiguous tensors; K optionally turned back
// to before its rotation.
//
// A record's value is code * scale (fp32, one rounding; 16-bit pools: the value itself), and, turned back by its
// token's angle, for a pair (a, b):
//   a' = fl(fl(a c) + fl(b s)),   b' = fl(fl(b c) - fl(a s)),
// rounded once to the output's type. A 16-bit pool's values into its own type are copied as they are.
//
// Rows are numbered through all tokens (a token's K heads, then its V heads); a warp takes kRows of them per lane group,
// of whatever tokens, so that the slots' lookups and then the rows' loads of all of them are in flight together.
// As they are stored, a lane takes 16 consecutive bytes of a row; turned back, the lanes hold a row as in append.cuh:
// head_dim / 8 of them, two runs of four dims that are rotation partners.
//
// Bound by memory: a record in and 2 or 4 B out per value. Measured: 131072 tokens of an int8 side pool, one head of 256, to
// bf16 45 us (4.5 TB/s); with 4 B loads and a warp per row 58. 65536 such tokens turned back, with 64 MB of angles, 58
// us, 2.3 times the bytes' time (angles asked for with the rows: the same, and bf16 in 8 heads of 128 56 -> 62): a lane's 4 B
// loads, and two dependent loads (positions, angles) per row before its stores.
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

// The row numbered flat: its token, its number among the token's rows, and its slot (-1: no row, or a skipped one).
struct Row {
  int64_t token, slot;
  int r;
};
template <bool TURN>
__device__ __forceinline__ Row find_row(const ReadArgs& a, uint64_t flat, uint64_t total, int rows, bool flags) {
  Row x;
  // numbered in 32 bits where they fit
  x.token = total <= 0xFFFFFFFFull ? static_cast<uint32_t>(flat) / static_cast<uint32_t>(rows) : static_cast<int64_t>(flat / rows);
  x.r = static_cast<int>(flat - static_cast<uint64_t>(x.token) * rows);
  x.slot = -1;
  if (flat >= total) return x;
  x.slot = a.slot_mapping != nullptr ? __ldg(a.slot_mapping + x.token) : paged_slot(a.paging, x.token, a.num_slots);
  bool bad = x.slot < -1 || x.slot >= a.num_slots;
  if (TURN) {
    TokenAxes ax;
    ax.load(a.axes, x.token, a.num_tokens);
    if (!ax.valid(a.axes, a.num_positions)) {  // no angle: the token is skipped whole
      bad |= ax.pos[0] != -1 && x.slot != -1;
      x.slot = -1;
    }
  }
  if (bad) {
    x.slot = -1;
    if (x.r == 0 && flags && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_INDEX);
  }
  return x;
}

// 32 bytes: one store where the outputs are aligned to them (`wide`): 32768 int8 tokens to bf16 10.4 us, 11.7 with two.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// K and V as they are stored.
template <int FMT, int HD, int kRows>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadArgs a, const bool wide) {
  constexpr bool k16 = FMT == QKV_BF16 || FMT == QKV_F16;
  constexpr int RB = k16 ? 2 * HD : HD, W = RB / 16, kPerWarp = 32 / W, N = k16 ? 8 : 16;  // N: values of a lane
  constexpr int kRecord = FMT == QKV_INT8_INLINE ? HD + 4 : RB;
  const int lane = threadIdx.x & 31, j = lane & (W - 1), sub = lane / W;
  const int hk = a.k_out != nullptr ? a.num_kv_heads : 0, rows = hk + (a.v_out != nullptr ? a.num_kv_heads : 0);
  const uint64_t first = ((static_cast<uint64_t>(blockIdx.x) * kReadThreads + threadIdx.x) >> 5) * kRows * kPerWarp;
  const uint64_t total = static_cast<uint64_t>(a.num_tokens) * rows;
  Row row[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) row[i] = find_row<false>(a, first + kPerWarp * i + sub, total, rows, j == 0);
  uint4 raw[kRows];
  float scale[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    scale[i] = 0.f;
    if (row[i].slot >= 0) {
      const bool is_k = row[i].r < hk;
      const int64_t rec = row[i].slot * a.num_kv_heads + (is_k ? row[i].r : row[i].r - hk);
      const uint8_t* src = (is_k ? a.k_cache : a.v_cache) + rec * kRecord;
      if (FMT == QKV_INT8_INLINE) {  // records sit on 4 B boundaries
        const uint32_t* w = reinterpret_cast<const uint32_t*>(src + 16 * j);
        raw[i] = make_uint4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
        scale[i] = __ldg(reinterpret_cast<const float*>(src + HD));
      } else {
        raw[i] = load_raw8(reinterpret_cast<const uint16_t*>(src + 16 * j));
        if (FMT == QKV_INT8_SIDE) scale[i] = __ldg((is_k ? a.k_scale : a.v_scale) + rec);
        if (FMT == QKV_E4M3) scale[i] = is_k ? a.k_scale_layer : a.v_scale_layer;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (row[i].slot < 0) continue;
    const bool is_k = row[i].r < hk;
    const int64_t at = row[i].token * a.out_stride + static_cast<int64_t>(is_k ? row[i].r : row[i].r - hk) * HD + N * j;
    void* out = is_k ? a.k_out : a.v_out;
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float x[N];
#pragma unroll
    for (int k = 0; k < N / 4; ++k) widen4<FMT>(k16 ? make_uint2(w[2 * k % 4], w[(2 * k + 1) % 4]) : make_uint2(w[k % 4], 0), x + 4 * k);
    if (!k16) {
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = __fmul_rn(x[k], scale[i]);
    }
    if (a.out_type == QKV_OUT_F32) {
#pragma unroll
      for (int k = 0; k < N; k += 8) {
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(x[k + e]);
        store32(static_cast<float*>(out) + at + k, o, wide);
      }
    } else if (k16 && (FMT == QKV_F16) == (a.out_type == QKV_OUT_F16)) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = raw[i];
    } else {
      uint32_t o[N / 2];
#pragma unroll
      for (int k = 0; k < N / 2; ++k) o[k] = a.out_type == QKV_OUT_F16 ? pack_half2(x[2 * k], x[2 * k + 1]) : pack_bf162(x[2 * k], x[2 * k + 1]);
      if constexpr (N == 16) store32(static_cast<uint16_t*>(out) + at, o, wide);
      else *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// K turned back, V as it is stored. PAIRS: adjacent pairs.
template <int FMT, int HD, bool PAIRS, int kRows>
__global__ void __launch_bounds__(kReadThreads) read_turned_kernel(const ReadArgs a) {
  constexpr int W = HD / 8, kPerWarp = 32 / W;
  constexpr bool k16 = FMT == QKV_BF16 || FMT == QKV_F16;
  constexpr int kRecord = FMT == QKV_INT8_INLINE ? HD + 4 : k16 ? 2 * HD : HD;
  const int lane = threadIdx.x & 31, j = lane & (W - 1), sub = lane / W;
  const int hk = a.k_out != nullptr ? a.num_kv_heads : 0, rows = hk + (a.v_out != nullptr ? a.num_kv_heads : 0);
  const uint64_t first = ((static_cast<uint64_t>(blockIdx.x) * kReadThreads + threadIdx.x) >> 5) * kRows * kPerWarp;
  const uint64_t total = static_cast<uint64_t>(a.num_tokens) * rows;
  const int rot = a.rotary_dim, half = rot >> 1;
  int d0 = 4 * j, d1 = HD / 2 + 4 * j;
  if (!PAIRS) {
    if (8 * j < rot) d1 = half + 4 * j;
    else d0 = rot + 4 * (j - rot / 8), d1 = d0 + (HD - rot) / 2;
  }
  const bool turns0 = d0 < rot, turns1 = d1 < rot;
  Row row[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) row[i] = find_row<true>(a, first + kPerWarp * i + sub, total, rows, j == 0);
  uint2 lo[kRows], hi[kRows];
  float scale[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    lo[i] = hi[i] = make_uint2(0, 0);
    scale[i] = 0.f;
    if (row[i].slot >= 0) {
      const bool is_k = row[i].r < hk;
      const int64_t rec = row[i].slot * a.num_kv_heads + (is_k ? row[i].r : row[i].r - hk);
      const uint8_t* src = (is_k ? a.k_cache : a.v_cache) + rec * kRecord;
      lo[i] = record4<FMT>(src, d0), hi[i] = record4<FMT>(src, d1);
      if (FMT == QKV_INT8_INLINE) scale[i] = __ldg(reinterpret_cast<const float*>(src + HD));
      if (FMT == QKV_INT8_SIDE) scale[i] = __ldg((is_k ? a.k_scale : a.v_scale) + rec);
      if (FMT == QKV_E4M3) scale[i] = is_k ? a.k_scale_layer : a.v_scale_layer;
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (row[i].slot < 0) continue;
    const bool is_k = row[i].r < hk;
    float x[8];
    widen4<FMT>(lo[i], x), widen4<FMT>(hi[i], x + 4);
    if (!k16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __fmul_rn(x[k], scale[i]);
    }
    float4 cs = make_float4(0.f, 0.f, 0.f, 0.f), sn = cs;
    if (is_k) {
      TokenAxes ax;
      ax.load(a.axes, row[i].token, a.num_tokens);
      axes_angles<PAIRS>(a.axes, ax, a.cos_sin, rot, d0, d1, cs, sn);
    }
    if (!PAIRS && is_k && turns0) {
      rotate(x[0], x[4], cs.x, -sn.x), rotate(x[1], x[5], cs.y, -sn.y);
      rotate(x[2], x[6], cs.z, -sn.z), rotate(x[3], x[7], cs.w, -sn.w);
    } else if (PAIRS && is_k) {
      if (turns0) rotate(x[0], x[1], cs.x, -sn.x), rotate(x[2], x[3], cs.y, -sn.y);
      if (turns1) rotate(x[4], x[5], cs.z, -sn.z), rotate(x[6], x[7], cs.w, -sn.w);
    }
    const int64_t at = row[i].token * a.out_stride + static_cast<int64_t>(is_k ? row[i].r : row[i].r - hk) * HD;
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
      if (same && !(is_k && turns0)) p = lo[i];  // not turned: the bits as they are, a NaN's payload too
      if (same && !(is_k && turns1)) q = hi[i];
      *reinterpret_cast<uint2*>(dst + d0) = p;
      *reinterpret_cast<uint2*>(dst + d1) = q;
    }
  }
}

// Rows per lane group: one while the launch does not fill the GPU, four above. Tokens read to bf16, in us with one | four,
// replayed from a graph (warps with one): int8 side, one head of 256: 1024 (1024) 2.6 | 4.2, 16384 (16384) 6.1 | 6.7, 32768
// (32768) 9.9 | 10.4; turned back: 16384 (32768) 14.3 | 14.3, 32768 (65536) 26.1 | 25.1; bf16, 8 heads of 128: 2048 (16384)
// 5.2 | 5.4, 8192 (65536) 15.1 | 14.2, 32768 73 | 60.
constexpr int64_t kSmallReadWarps = 32768;

template <int FMT, int HD>
cudaError_t launch(const ReadArgs& a, cudaStream_t stream) {
  const int64_t rows = a.num_tokens * a.num_kv_heads * ((a.k_out != nullptr ? 1 : 0) + (a.v_out != nullptr ? 1 : 0));
  const bool turned = a.cos_sin != nullptr && a.k_out != nullptr;
  const int lanes = turned ? HD / 8 : FMT == QKV_BF16 || FMT == QKV_F16 ? HD / 8 : HD / 16;  // of a row
  const int64_t single = (rows * lanes + 31) / 32;
  const bool one = single <= kSmallReadWarps;
  const unsigned grid = static_cast<unsigned>(((one ? single : (single + 3) / 4) * 32 + kReadThreads - 1) / kReadThreads);
  if (!turned) {
    auto off = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    const int64_t row_bytes = a.out_stride * (a.out_type == QKV_OUT_F32 ? 4 : 2);
    const bool wide = ((off(a.k_out) | off(a.v_out) | static_cast<uintptr_t>(row_bytes)) & 31) == 0;
    if (one) read_kernel<FMT, HD, 1><<<grid, kReadThreads, 0, stream>>>(a, wide);
    else read_kernel<FMT, HD, 4><<<grid, kReadThreads, 0, stream>>>(a, wide);
  } else if (a.interleaved) {
    if (one) read_turned_kernel<FMT, HD, true, 1><<<grid, kReadThreads, 0, stream>>>(a);
    else read_turned_kernel<FMT, HD, true, 4><<<grid, kReadThreads, 0, stream>>>(a);
  } else {
    if (one) read_turned_kernel<FMT, HD, false, 1><<<grid, kReadThreads, 0, stream>>>(a);
    else read_turned_kernel<FMT, HD, false, 4><<<grid, kReadThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
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
