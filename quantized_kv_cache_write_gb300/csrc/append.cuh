// Append of a step's tokens to the cache: the position rotation of q and K and the store of K and V
// in the pool's format, in one pass over the packed projection's output.
//
// For the pair (a, b) of head dims with angle theta (its cos and sin from the table):
//   a' = fl(fl(a c) - fl(b s)),   b' = fl(fl(b c) + fl(a s)),
// three fp32 roundings and no fused multiply-add, so that the value that is quantised -- and with it
// every stored byte -- is the one a plain fp32 program gives. q' is rounded once to q's type; K' goes
// through the writes' own quantisers (write_rows.cuh), V unrotated.
//
// A row (one head of q, K or V) is held by head_dim / 8 lanes, two runs of four dims each: dims 4j of
// the rotated part's first half and of its second, which are partners, so that a lane rotates what it
// holds with four cosines and four sines and no exchange (adjacent pairs, and dims past the rotated
// part: four dims of each half of what is left). A warp takes kRows rows of one token for each of its
// lane groups, so the token's cos and sin are loaded once into registers for all of them; the row
// loads are issued before the position's dependent loads return.
//
// Bound by memory: 2 B in and 2 B out per q value, 2 B in and a record out per K and V value. Measured:
// 8192 tokens x 18 heads of 256 into an int8 pool 32.5 us (4.8 TB/s), 16384 x 48 heads of 128 into a
// bf16 pool 74 us (5.5 TB/s); with 16 B per lane and partners exchanged by shuffles 37.6 and 92 us
// (twice the cosines and sines per lane, twice the widening). Issue slots are 60 % busy there and warps
// wait for the rows' loads.
//
// AXES: a pair's angle is that of one of up to four positions of the token (time, height, width of an image's or a
// video's patches), by the pair's axis. The four pairs of a lane are loaded as a vector where they share an axis.
#pragma once

#include "rope.cuh"

namespace qkv {
namespace {

constexpr int kAppendThreads = 128;  // 8192 tokens x 18 heads of 256, int8: 32.5 us, 35.7 with 256

// FMT: the pool's format. F16: IEEE-half activations. HD: head dim. PAIRS: adjacent pairs. AXES: several positions.
template <int FMT, bool F16, int HD, bool PAIRS, bool AXES, int kRows>
__global__ void __launch_bounds__(kAppendThreads) append_rope_kernel(const AppendArgs a) {
  constexpr int W = HD / 8, kPerWarp = 32 / W;  // lanes per row, rows of a warp at a time
  constexpr bool kInt8 = FMT == QKV_INT8_SIDE || FMT == QKV_INT8_INLINE;
  const int lane = threadIdx.x & 31, j = lane & (W - 1), sub = lane / W;
  const int rows = a.num_q_heads + 2 * a.num_kv_heads;
  const uint32_t units = static_cast<uint32_t>((rows + kRows * kPerWarp - 1) / (kRows * kPerWarp));
  const uint64_t wid = (static_cast<uint64_t>(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
  const uint64_t total = static_cast<uint64_t>(a.num_tokens) * units;
  if (wid >= total) return;  // warp-uniform
  int64_t t;
  int u;
  if (total <= 0xFFFFFFFFull) {
    const uint32_t t32 = static_cast<uint32_t>(wid) / units;
    t = t32;
    u = static_cast<int>(static_cast<uint32_t>(wid) - t32 * units);
  } else {
    t = static_cast<int64_t>(wid / units);
    u = static_cast<int>(wid - static_cast<uint64_t>(t) * units);
  }
  int pos;
  TokenAxes ax;
  if (AXES) ax.load(a.axes, t, a.num_tokens);
  else pos = __ldg(a.token_pos + t);
  const int r0 = u * kRows * kPerWarp + sub;  // this lane group's rows: r0 + kPerWarp i
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;

  // the lane's two runs of four dims
  const int rot = a.rotary_dim, half = rot >> 1;
  int d0, d1;
  if (PAIRS) d0 = 4 * j, d1 = HD / 2 + 4 * j;
  else if (8 * j < rot) d0 = 4 * j, d1 = half + 4 * j;
  else d0 = rot + 4 * (j - rot / 8), d1 = d0 + (HD - rot) / 2;

  uint4 raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + kPerWarp * i;
    uint2 lo = make_uint2(0, 0), hi = lo;
    if (r < hq) {
      const uint16_t* src = a.q + t * a.q_stride + static_cast<int64_t>(r) * HD;
      if (a.q != nullptr) lo = load_raw4<true>(src + d0), hi = load_raw4<true>(src + d1);
    } else if (r < rows) {
      const uint16_t* src = (r < hq + hkv ? a.k + static_cast<int64_t>(r - hq) * HD : a.v + static_cast<int64_t>(r - hq - hkv) * HD) + t * a.kv_stride;
      lo = load_raw4<false>(src + d0), hi = load_raw4<false>(src + d1);
    }
    raw[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }

  // the token's slot (the warps that hold K or V rows) and angles
  const bool flags = u == hq / (kRows * kPerWarp);  // the warp of the first K row flags
  if (AXES ? !ax.valid(a.axes, a.num_positions) : pos < 0 || static_cast<int64_t>(pos) >= a.num_positions) {
    if ((AXES ? ax.pos[0] : pos) != -1 && flags && lane == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_SLOT);
    return;  // no angle: the token is skipped whole
  }
  bool store = false;
  int64_t slot = -1;
  if ((u + 1) * kRows * kPerWarp > hq) {
    slot = a.slot_mapping != nullptr ? __ldg(a.slot_mapping + t) : paged_slot(a.paging, t, a.num_slots);
    store = slot_ok(slot, a.num_slots, a.dev_status, lane, flags);
  }
  const bool turns0 = d0 < rot, turns1 = d1 < rot;  // one without the other: adjacent pairs
  float4 cs = make_float4(0.f, 0.f, 0.f, 0.f), sn = cs;
  const float* angle = AXES ? nullptr : a.cos_sin + static_cast<int64_t>(pos) * rot;
  if (AXES) {
    axes_angles<PAIRS>(a.axes, ax, a.cos_sin, rot, d0, d1, cs, sn);
  } else if (PAIRS) {
    auto angles = [&](int d, float& c0, float& c1, float& s0, float& s1) {
      const float2 c = __ldg(reinterpret_cast<const float2*>(angle + d / 2)), s = __ldg(reinterpret_cast<const float2*>(angle + half + d / 2));
      c0 = c.x, c1 = c.y, s0 = s.x, s1 = s.y;
    };
    if (turns0) angles(d0, cs.x, cs.y, sn.x, sn.y);
    if (turns1) angles(d1, cs.z, cs.w, sn.z, sn.w);
  } else if (turns0) {
    cs = __ldg(reinterpret_cast<const float4*>(angle + d0)), sn = __ldg(reinterpret_cast<const float4*>(angle + half + d0));
  }

#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + kPerWarp * i;
    HeadVec x = widen8<F16>(raw[i]);
    if (r < hq + hkv) {
      if (PAIRS) {
        if (turns0) rotate(x.x[0], x.x[1], cs.x, sn.x), rotate(x.x[2], x.x[3], cs.y, sn.y);
        if (turns1) rotate(x.x[4], x.x[5], cs.z, sn.z), rotate(x.x[6], x.x[7], cs.w, sn.w);
      } else if (turns0) {
        rotate(x.x[0], x.x[4], cs.x, sn.x), rotate(x.x[1], x.x[5], cs.y, sn.y);
        rotate(x.x[2], x.x[6], cs.z, sn.z), rotate(x.x[3], x.x[7], cs.w, sn.w);
      }
    }
    // a warp whose rows are all query rows is done here; the others go on together
    if (r < hq && a.q != nullptr) {
      uint16_t* dst = a.q_out + t * a.q_out_stride + static_cast<int64_t>(r) * HD;
      *reinterpret_cast<uint2*>(dst + d0) = round4<F16>(x.x);
      *reinterpret_cast<uint2*>(dst + d1) = round4<F16>(x.x + 4);
    }
    const int first = u * kRows * kPerWarp + kPerWarp * i;
    if (first + kPerWarp <= hq || first >= rows) continue;
    const bool is_k = r < hq + hkv;
    const bool mine = store && r >= hq && r < rows;
    const int64_t rec = slot * hkv + (is_k ? r - hq : r - hq - hkv);
    uint8_t* cache = is_k ? a.k_cache : a.v_cache;
    if (kInt8 || FMT == QKV_E4M3) {
      uint32_t word[2];
      float scale = 0.f;
      if (FMT == QKV_E4M3) {
        const uint2 codes = e4m3_codes(x, is_k ? a.k_scale_layer : a.v_scale_layer);
        word[0] = codes.x, word[1] = codes.y;
      } else {
        scale = int8_codes<W>(x, word);
      }
      if (!mine) continue;
      uint8_t* dst = cache + rec * (FMT == QKV_INT8_INLINE ? HD + 4 : HD);
      *reinterpret_cast<uint32_t*>(dst + d0) = word[0];
      *reinterpret_cast<uint32_t*>(dst + d1) = word[1];
      if (FMT == QKV_INT8_INLINE && j == 0) *reinterpret_cast<float*>(dst + HD) = scale;
      if (FMT == QKV_INT8_SIDE && j == 0) (is_k ? a.k_scale : a.v_scale)[rec] = scale;
    } else if (mine) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(cache) + rec * HD;
      *reinterpret_cast<uint2*>(dst + d0) = is_k ? round4<F16>(x.x) : make_uint2(raw[i].x, raw[i].y);
      *reinterpret_cast<uint2*>(dst + d1) = is_k ? round4<F16>(x.x + 4) : make_uint2(raw[i].z, raw[i].w);
    }
  }
}

// Rows per lane group: one while the launch is too small to fill the GPU (each row's loads then start in a warp of
// their own), four above. Tokens x (16 + 2 heads of 256), int8, in us with one | four: 64: 3.0 | 3.7, 256 (4608
// warps with one): 3.4 | 3.9, 512 (9216): 4.3 | 4.2, 8192: 42 | 32.
constexpr int64_t kSmallWarps = 8192;

template <int FMT, bool F16, int HD, bool PAIRS, bool AXES>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  constexpr int kPerWarp = 256 / HD;
  const int rows = a.num_q_heads + 2 * a.num_kv_heads;
  const int64_t single = a.num_tokens * ((rows + kPerWarp - 1) / kPerWarp);
  if (single <= kSmallWarps) {
    append_rope_kernel<FMT, F16, HD, PAIRS, AXES, 1>
        <<<static_cast<unsigned>((single * 32 + kAppendThreads - 1) / kAppendThreads), kAppendThreads, 0, stream>>>(a);
  } else {
    const int64_t warps = a.num_tokens * ((rows + 4 * kPerWarp - 1) / (4 * kPerWarp));
    append_rope_kernel<FMT, F16, HD, PAIRS, AXES, 4>
        <<<static_cast<unsigned>((warps * 32 + kAppendThreads - 1) / kAppendThreads), kAppendThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

template <int FMT, bool F16, bool AXES>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  if (a.head_dim == 256) return a.interleaved ? launch<FMT, F16, 256, true, AXES>(a, stream) : launch<FMT, F16, 256, false, AXES>(a, stream);
  return a.interleaved ? launch<FMT, F16, 128, true, AXES>(a, stream) : launch<FMT, F16, 128, false, AXES>(a, stream);
}

template <bool AXES>
cudaError_t launch(const AppendArgs& a, qkv_format fmt, bool f16, cudaStream_t stream) {
  switch (fmt) {
    case QKV_BF16: return launch<QKV_BF16, false, AXES>(a, stream);
    case QKV_F16: return launch<QKV_F16, true, AXES>(a, stream);
    case QKV_INT8_SIDE: return f16 ? launch<QKV_INT8_SIDE, true, AXES>(a, stream) : launch<QKV_INT8_SIDE, false, AXES>(a, stream);
    case QKV_INT8_INLINE: return f16 ? launch<QKV_INT8_INLINE, true, AXES>(a, stream) : launch<QKV_INT8_INLINE, false, AXES>(a, stream);
    case QKV_E4M3: return f16 ? launch<QKV_E4M3, true, AXES>(a, stream) : launch<QKV_E4M3, false, AXES>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace qkv
