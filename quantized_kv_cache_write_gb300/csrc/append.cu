// Append of a step's tokens to the cache: the position rotation of q and K and the store of K and V
// in the pool's format, in one pass over the packed projection's output.
//
// For the pair (a, b) of head dims with angle theta (its cos and sin from the table):
//   a' = fl(fl(a c) - fl(b s)),   b' = fl(fl(b c) + fl(a s)),
// three fp32 roundings and no fused multiply-add, so that the value that is quantised -- and with it
// every stored byte -- is the one a plain fp32 program gives. q' is rounded once to q's type; K' goes
// through the writes' own quantisers (write_rows.cuh), V unrotated.
//
// A row (one head of q, K or V) is held by head_dim / 8 lanes, eight dims each: 16 B loads, and pairs
// (i, i + rotary_dim / 2) meet by one shuffle of the raw 16-bit words. A warp takes kRows rows of one
// token for each of its lane groups, so the token's cos and sin are loaded once into registers for
// all of them; the row loads are issued before the position's dependent loads return.
// Bound by memory: 2 B in and 2 B out per q value, 2 B in and a record out per K and V value.
#include "write_rows.cuh"

namespace qkv {
namespace {

constexpr int kAppendThreads = 256;

// As load_raw8, but through the ordinary path: q may be rotated in place.
__device__ __forceinline__ uint4 load_raw8_rw(const uint16_t* src) {
  uint4 raw;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w)
               : "l"(src)
               : "memory");
  return raw;
}

template <bool F16>
__device__ __forceinline__ uint4 round8(const HeadVec& h) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = F16 ? pack_half2(h.x[2 * i], h.x[2 * i + 1]) : pack_bf162(h.x[2 * i], h.x[2 * i + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// FMT: the pool's format. F16: IEEE-half activations. HD: head dim. PAIRS: adjacent pairs.
template <int FMT, bool F16, int HD, bool PAIRS, int kRows>
__global__ void __launch_bounds__(kAppendThreads) append_rope_kernel(const AppendArgs a) {
  constexpr int W = HD / 8, kPerWarp = 32 / W;  // lanes per row, rows of a warp at a time
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
  const int pos = __ldg(a.token_pos + t);
  const int r0 = u * kRows * kPerWarp + sub;  // this lane group's rows: r0 + kPerWarp i
  const int hq = a.num_q_heads, hkv = a.num_kv_heads;

  uint4 raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + kPerWarp * i;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (r < hq) {
      if (a.q != nullptr) raw[i] = load_raw8_rw(a.q + t * a.q_stride + static_cast<int64_t>(r) * HD + 8 * j);
    } else if (r < hq + hkv) {
      raw[i] = load_raw8(a.k + t * a.kv_stride + static_cast<int64_t>(r - hq) * HD + 8 * j);
    } else if (r < rows) {
      raw[i] = load_raw8(a.v + t * a.kv_stride + static_cast<int64_t>(r - hq - hkv) * HD + 8 * j);
    }
  }

  // the token's slot (the warps that hold K or V rows) and angles
  const bool flags = u == hq / (kRows * kPerWarp);  // the warp of the first K row flags
  if (pos < 0 || static_cast<int64_t>(pos) >= a.num_positions) {
    if (pos != -1 && flags && lane == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_SLOT);
    return;  // no angle: the token is skipped whole
  }
  bool store = false;
  int64_t slot = -1;
  if ((u + 1) * kRows * kPerWarp > hq) {
    slot = a.slot_mapping != nullptr ? __ldg(a.slot_mapping + t) : paged_slot(a.paging, t, a.num_slots);
    store = slot_ok(slot, a.num_slots, a.dev_status, lane, flags);
  }
  const int half = a.rotary_dim >> 1, hl = half >> 3;  // dims and lanes of half the rotated part
  const bool turns = j < 2 * hl;
  const int mate = PAIRS ? j : (j < hl ? j + hl : j - hl);  // lane with the partner dims (rotated lanes)
  constexpr int kAngles = PAIRS ? 4 : 8;
  float cs[kAngles], sn[kAngles];
  if (turns) {
    const float* p = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim + kAngles * (PAIRS ? j : (j < hl ? j : j - hl));
#pragma unroll
    for (int i = 0; i < kAngles; i += 4) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(p + i));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(p + half + i));
      cs[i] = c4.x, cs[i + 1] = c4.y, cs[i + 2] = c4.z, cs[i + 3] = c4.w;
      sn[i] = s4.x, sn[i + 1] = s4.y, sn[i + 2] = s4.z, sn[i + 3] = s4.w;
    }
    if (!PAIRS && j < hl) {  // a' = a c + b (-s): the same roundings
#pragma unroll
      for (int i = 0; i < kAngles; ++i) sn[i] = -sn[i];
    }
  }

#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = r0 + kPerWarp * i;
    HeadVec x = widen8<F16>(raw[i]);
    if (PAIRS) {
      if (turns && r < hq + hkv) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float p = x.x[2 * d], q = x.x[2 * d + 1];
          x.x[2 * d] = __fsub_rn(__fmul_rn(p, cs[d % kAngles]), __fmul_rn(q, sn[d % kAngles]));
          x.x[2 * d + 1] = __fadd_rn(__fmul_rn(q, cs[d % kAngles]), __fmul_rn(p, sn[d % kAngles]));
        }
      }
    } else {
      const int from = (lane & ~(W - 1)) | (turns ? mate : j);
      uint4 other;
      other.x = __shfl_sync(0xffffffffu, raw[i].x, from);
      other.y = __shfl_sync(0xffffffffu, raw[i].y, from);
      other.z = __shfl_sync(0xffffffffu, raw[i].z, from);
      other.w = __shfl_sync(0xffffffffu, raw[i].w, from);
      if (turns && r < hq + hkv) {
        const HeadVec y = widen8<F16>(other);
#pragma unroll
        for (int d = 0; d < 8; ++d)
          x.x[d] = __fadd_rn(__fmul_rn(x.x[d], cs[d % kAngles]), __fmul_rn(y.x[d], sn[d % kAngles]));
      }
    }
    // a warp whose rows are all query rows is done here; the others go on together
    if (r < hq && a.q != nullptr)
      *reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + static_cast<int64_t>(r) * HD + 8 * j) = round8<F16>(x);
    const int first = u * kRows * kPerWarp + kPerWarp * i;
    if (first + kPerWarp <= hq || first >= rows) continue;
    const bool is_k = r < hq + hkv;
    const bool mine = store && r >= hq && r < rows;
    const int64_t rec = slot * hkv + (is_k ? r - hq : r - hq - hkv);
    uint8_t* cache = is_k ? a.k_cache : a.v_cache;
    if (FMT == QKV_INT8_SIDE)
      store_int8_row<false, W>(x, j, true, HD, rec, cache, is_k ? a.k_scale : a.v_scale, mine);
    else if (FMT == QKV_INT8_INLINE)
      store_int8_row<true, W>(x, j, true, HD, rec, cache, nullptr, mine);
    else if (mine) {
      if (FMT == QKV_E4M3)
        store_e4m3_row(x, j, HD, rec, is_k ? a.k_scale_layer : a.v_scale_layer, cache);
      else
        *reinterpret_cast<uint4*>(cache + (rec * HD + 8 * j) * 2) = is_k ? round8<F16>(x) : raw[i];
    }
  }
}

// Rows per lane group: one while the launch is too small to fill the GPU (each row's loads then
// start in a warp of their own), four above.
constexpr int64_t kSmallWarps = 8192;

template <int FMT, bool F16, int HD, bool PAIRS>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  constexpr int kPerWarp = 256 / HD;
  const int rows = a.num_q_heads + 2 * a.num_kv_heads;
  const int64_t single = a.num_tokens * ((rows + kPerWarp - 1) / kPerWarp);
  if (single <= kSmallWarps) {
    append_rope_kernel<FMT, F16, HD, PAIRS, 1>
        <<<static_cast<unsigned>((single * 32 + kAppendThreads - 1) / kAppendThreads), kAppendThreads, 0, stream>>>(a);
  } else {
    const int64_t warps = a.num_tokens * ((rows + 4 * kPerWarp - 1) / (4 * kPerWarp));
    append_rope_kernel<FMT, F16, HD, PAIRS, 4>
        <<<static_cast<unsigned>((warps * 32 + kAppendThreads - 1) / kAppendThreads), kAppendThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

template <int FMT, bool F16>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  if (a.head_dim == 256) return a.interleaved ? launch<FMT, F16, 256, true>(a, stream) : launch<FMT, F16, 256, false>(a, stream);
  return a.interleaved ? launch<FMT, F16, 128, true>(a, stream) : launch<FMT, F16, 128, false>(a, stream);
}

}  // namespace

cudaError_t launch_append_rope(const AppendArgs& a, qkv_format fmt, bool f16, cudaStream_t stream) {
  switch (fmt) {
    case QKV_BF16: return launch<QKV_BF16, false>(a, stream);
    case QKV_F16: return launch<QKV_F16, true>(a, stream);
    case QKV_INT8_SIDE: return f16 ? launch<QKV_INT8_SIDE, true>(a, stream) : launch<QKV_INT8_SIDE, false>(a, stream);
    case QKV_INT8_INLINE: return f16 ? launch<QKV_INT8_INLINE, true>(a, stream) : launch<QKV_INT8_INLINE, false>(a, stream);
    case QKV_E4M3: return f16 ? launch<QKV_E4M3, true>(a, stream) : launch<QKV_E4M3, false>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qkv
