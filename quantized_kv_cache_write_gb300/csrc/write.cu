// Quantize-on-write kernels: int8 per-(token, head) absmax/127 (side or inline scale
// layout) and FP8 E4M3 with calibrated per-layer scales, plus the amax/448 calibration
// reduction. New tokens are bf16, or IEEE half for the FP16-activation contract of
// "[Model][SM70][FP8] Add calibrated E4M3 QSA KV cache" §Purpose (exact widening either way).
//
// Pages: "int8 per-(token,head) KV cache for the Qwen3.8-Flash-Next QSA path" §The finding
// worth upstreaming (per-(token,head) scale, 260 B inline record vs side tensor);
// "Qwen3.8 Flash Next NVFP4 QSA FP8 E4M3 KV Scales" §Calibration (stored = e4m3fn(x/scale),
// scale = max envelope / 448).
//
// One warp owns one (token, head) row of K or V, or both rows when the write is large: 32 lanes
// x 8 values = a 256-wide head vector, read as one coalesced line (head_dim 128: lanes 16..31
// idle); the absmax is a 5-step shuffle reduction; the codes leave as one coalesced line.
// Every code is the one the IEEE quotient fl(x / scale) rounds to (round-to-nearest-even), so
// the stored bytes equal a plain fp32 reference bit for bit; int8 takes the division itself
// only where a bracket of two multiplications cannot decide (see bracket_lo / bracket_hi).
#include <atomic>

#include "write_rows.cuh"

namespace qkv {
namespace {

constexpr int kWriteThreads = 256;

// Large writes pair a token head's K and V rows in one warp (two row loads in flight per
// lane, one slot load for both); small ones give each row its own warp, twice the warps to
// spread a latency-bound launch over. Measured on one GB300 (int8 side / E4M3): 262144 tokens
// 143 -> 117 / 113 -> 91 us paired; 2048 tokens 7-9 / 7 us either way.
constexpr int64_t kPairedMinUnits = 16384;  // (token, head) units from which rows are paired

// The (token t, head h) of a unit. 32-bit division whenever the index fits, which it does at
// any realistic size (64-bit division is several times longer).
__device__ __forceinline__ void decode_unit(int64_t unit, int num_heads, int64_t& t, int& h) {
  if (unit <= 0xFFFFFFFFll) {
    const uint32_t t32 = static_cast<uint32_t>(unit) / static_cast<uint32_t>(num_heads);
    t = t32;
    h = static_cast<int>(static_cast<uint32_t>(unit) - t32 * static_cast<uint32_t>(num_heads));
  } else {
    t = unit / num_heads;
    h = static_cast<int>(unit - t * num_heads);
  }
}

// The warp's rows: one row (K or V: kv) of a (token, head) unit, or both rows of a unit when
// paired. Every row and the slot are loaded before any is used, so the loads are in flight
// together (a skipped token's rows are still in bounds: t < num_tokens). Returns false for a
// warp past the end, a skipped token or a bad slot; the result is warp-uniform.
template <bool kPaired, bool kPaged>
__device__ __forceinline__ bool warp_rows(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int head_dim,
                                          int64_t num_tokens, int num_heads, int64_t token_stride,
                                          const int64_t* __restrict__ slot_mapping, const WritePaging& pg,
                                          int64_t num_slots, uint32_t* dev_status, int lane, bool act,
                                          uint4 (&raw)[2], int& kv, int64_t& rec) {
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * kWriteThreads + threadIdx.x) >> 5;
  const int64_t unit = kPaired ? wid : wid >> 1;
  if (unit >= num_tokens * num_heads) return false;
  kv = kPaired ? 0 : static_cast<int>(wid & 1);
  int64_t t;
  int h;
  decode_unit(unit, num_heads, t, h);
  const int64_t off = t * token_stride + static_cast<int64_t>(h) * head_dim + lane * 8;
  raw[0] = act ? load_raw8((kv ? v : k) + off) : make_uint4(0, 0, 0, 0);
  if (kPaired) raw[1] = act ? load_raw8(v + off) : make_uint4(0, 0, 0, 0);
  const int64_t slot = kPaged ? paged_slot(pg, t, num_slots) : slot_mapping[t];
  if (!slot_ok(slot, num_slots, dev_status, lane, kv == 0 && h == 0)) return false;
  rec = slot * num_heads + h;
  return true;
}

template <bool kInline, bool F16, bool kPaired, bool kPaged>
__global__ void __launch_bounds__(kWriteThreads)
    write_int8_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int head_dim,
                      int64_t num_tokens, int num_heads, int64_t token_stride,
                      const int64_t* __restrict__ slot_mapping, const WritePaging pg, uint8_t* __restrict__ k_cache,
                      uint8_t* __restrict__ v_cache, float* __restrict__ k_scale,
                      float* __restrict__ v_scale, int64_t num_slots, uint32_t* dev_status) {
  const int lane = threadIdx.x & 31;
  const bool act = 8 * lane < head_dim;  // lane owns head dims 8 lane .. 8 lane + 7 (128: lanes 0..15)
  uint4 raw[2];
  int kv;
  int64_t rec;
  if (!warp_rows<kPaired, kPaged>(k, v, head_dim, num_tokens, num_heads, token_stride, slot_mapping, pg, num_slots,
                                  dev_status, lane, act, raw, kv, rec))
    return;
  store_int8_row<kInline>(widen8<F16>(raw[0]), lane, act, head_dim, rec, kv ? v_cache : k_cache,
                          kv ? v_scale : k_scale);
  if (kPaired) store_int8_row<kInline>(widen8<F16>(raw[1]), lane, act, head_dim, rec, v_cache, v_scale);
}

template <bool F16, bool kPaired, bool kPaged>
__global__ void __launch_bounds__(kWriteThreads)
    write_e4m3_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int head_dim,
                      int64_t num_tokens, int num_heads, int64_t token_stride,
                      const int64_t* __restrict__ slot_mapping, const WritePaging pg, uint8_t* __restrict__ k_cache,
                      uint8_t* __restrict__ v_cache, float k_scale, float v_scale, int64_t num_slots,
                      uint32_t* dev_status) {
  const int lane = threadIdx.x & 31;
  const bool act = 8 * lane < head_dim;  // head_dim 128: lanes 16..31 own no dims (no shuffles follow)
  uint4 raw[2];
  int kv;
  int64_t rec;
  if (!warp_rows<kPaired, kPaged>(k, v, head_dim, num_tokens, num_heads, token_stride, slot_mapping, pg, num_slots,
                                  dev_status, lane, act, raw, kv, rec) ||
      !act)
    return;
  store_e4m3_row(widen8<F16>(raw[0]), lane, head_dim, rec, kv ? v_scale : k_scale, kv ? v_cache : k_cache);
  if (kPaired) store_e4m3_row(widen8<F16>(raw[1]), lane, head_dim, rec, v_scale, v_cache);
}

// max |x| over n bf16 values, as fp32 bits (non-negative floats order like their bits). A
// grid-stride loop with four 16 B loads in flight per thread.
__device__ __forceinline__ uint32_t absmax8(uint32_t m, const uint4& r) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, max((w[j] & 0x7FFFu) << 16, w[j] & 0x7FFF0000u));
  return m;
}

__global__ void __launch_bounds__(256)
    absmax_bf16_kernel(const uint16_t* __restrict__ x, int64_t n, uint32_t* __restrict__ amax_bits) {
  uint32_t m = 0;
  const int64_t nvec = n / 8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const uint4* xv = reinterpret_cast<const uint4*>(x);
  int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (; i + 3 * stride < nvec; i += 4 * stride) {
    uint4 r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) r[u] = __ldg(xv + i + u * stride);
#pragma unroll
    for (int u = 0; u < 4; ++u) m = absmax8(m, r[u]);
  }
  for (; i < nvec; i += stride) m = absmax8(m, __ldg(xv + i));
  for (int64_t j = nvec * 8 + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; j < n; j += stride)
    m = max(m, static_cast<uint32_t>(x[j] & 0x7FFFu) << 16);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  __shared__ uint32_t red[8];
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) m = max(m, red[w]);
    atomicMax(amax_bits, m);
  }
}

__global__ void e4m3_scale_kernel(const uint32_t* __restrict__ amax_bits, float* __restrict__ scale_out) {
  scale_out[0] = __fdiv_rn(__uint_as_float(amax_bits[0]), 448.0f);
}

bool write_paired(int64_t num_tokens, int num_heads) { return num_tokens * num_heads >= kPairedMinUnits; }

unsigned write_blocks(int64_t num_tokens, int num_heads) {
  const int64_t warps = num_tokens * num_heads * (write_paired(num_tokens, num_heads) ? 1 : 2);
  return static_cast<unsigned>((warps * 32 + kWriteThreads - 1) / kWriteThreads);
}

template <bool kInline, bool F16, bool kPaired, bool kPaged>
void launch_int8(unsigned blocks, const uint16_t* k, const uint16_t* v, int head_dim, int64_t num_tokens,
                 int num_heads, int64_t token_stride, const int64_t* slot_mapping, const WritePaging& pg,
                 uint8_t* kc, uint8_t* vc, float* ks, float* vs, int64_t num_slots, uint32_t* dev_status,
                 cudaStream_t stream) {
  write_int8_kernel<kInline, F16, kPaired, kPaged><<<blocks, kWriteThreads, 0, stream>>>(
      k, v, head_dim, num_tokens, num_heads, token_stride, slot_mapping, pg, kc, vc, ks, vs, num_slots, dev_status);
}

template <bool kInline, bool F16>
void launch_int8(bool paired, bool paged, unsigned blocks, const uint16_t* k, const uint16_t* v, int head_dim,
                 int64_t num_tokens, int num_heads, int64_t token_stride, const int64_t* slot_mapping,
                 const WritePaging& pg, uint8_t* kc, uint8_t* vc, float* ks, float* vs, int64_t num_slots,
                 uint32_t* dev_status, cudaStream_t stream) {
  auto kern = paired ? (paged ? launch_int8<kInline, F16, true, true> : launch_int8<kInline, F16, true, false>)
                     : (paged ? launch_int8<kInline, F16, false, true> : launch_int8<kInline, F16, false, false>);
  kern(blocks, k, v, head_dim, num_tokens, num_heads, token_stride, slot_mapping, pg, kc, vc, ks, vs, num_slots,
       dev_status, stream);
}

template <bool F16, bool kPaired, bool kPaged>
void launch_e4m3(unsigned blocks, const uint16_t* k, const uint16_t* v, int head_dim, int64_t num_tokens,
                 int num_heads, int64_t token_stride, const int64_t* slot_mapping, const WritePaging& pg,
                 uint8_t* kc, uint8_t* vc, float ks, float vs, int64_t num_slots, uint32_t* dev_status,
                 cudaStream_t stream) {
  write_e4m3_kernel<F16, kPaired, kPaged><<<blocks, kWriteThreads, 0, stream>>>(
      k, v, head_dim, num_tokens, num_heads, token_stride, slot_mapping, pg, kc, vc, ks, vs, num_slots, dev_status);
}

}  // namespace

cudaError_t launch_write_int8(const void* k, const void* v, bool f16, int head_dim, int64_t num_tokens, int num_heads,
                              int64_t token_stride, const int64_t* slot_mapping, const WritePaging* paging,
                              bool inline_layout, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                              int64_t num_slots, uint32_t* dev_status, cudaStream_t stream) {
  const unsigned blocks = write_blocks(num_tokens, num_heads);
  const bool pr = write_paired(num_tokens, num_heads), pgd = paging != nullptr;
  const WritePaging pg = pgd ? *paging : WritePaging{nullptr, nullptr, nullptr, 0, 0, 1};
  auto kk = static_cast<const uint16_t*>(k);
  auto vv = static_cast<const uint16_t*>(v);
  auto kc = static_cast<uint8_t*>(k_cache);
  auto vc = static_cast<uint8_t*>(v_cache);
  float* ks = inline_layout ? nullptr : k_scale;
  float* vs = inline_layout ? nullptr : v_scale;
  auto kern = inline_layout ? (f16 ? launch_int8<true, true> : launch_int8<true, false>)
                            : (f16 ? launch_int8<false, true> : launch_int8<false, false>);
  kern(pr, pgd, blocks, kk, vv, head_dim, num_tokens, num_heads, token_stride, slot_mapping, pg, kc, vc, ks, vs,
       num_slots, dev_status, stream);
  return cudaGetLastError();
}

cudaError_t launch_write_e4m3(const void* k, const void* v, bool f16, int head_dim, int64_t num_tokens, int num_heads,
                              int64_t token_stride, const int64_t* slot_mapping, const WritePaging* paging,
                              void* k_cache, void* v_cache, float k_scale, float v_scale, int64_t num_slots,
                              uint32_t* dev_status, cudaStream_t stream) {
  const bool pr = write_paired(num_tokens, num_heads), pgd = paging != nullptr;
  const WritePaging pg = pgd ? *paging : WritePaging{nullptr, nullptr, nullptr, 0, 0, 1};
  auto kern = f16 ? (pr ? (pgd ? launch_e4m3<true, true, true> : launch_e4m3<true, true, false>)
                        : (pgd ? launch_e4m3<true, false, true> : launch_e4m3<true, false, false>))
                  : (pr ? (pgd ? launch_e4m3<false, true, true> : launch_e4m3<false, true, false>)
                        : (pgd ? launch_e4m3<false, false, true> : launch_e4m3<false, false, false>));
  kern(write_blocks(num_tokens, num_heads), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), head_dim,
       num_tokens, num_heads, token_stride, slot_mapping, pg, static_cast<uint8_t*>(k_cache),
       static_cast<uint8_t*>(v_cache), k_scale, v_scale, num_slots, dev_status, stream);
  return cudaGetLastError();
}

cudaError_t launch_e4m3_calibrate(const void* x, int64_t n, uint32_t* amax_bits, float* scale_out,
                                  cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(amax_bits, 0, sizeof(uint32_t), stream);
  if (e != cudaSuccess) return e;
  if (n > 0) {
    // one wave of 256-thread blocks (8 per SM); each thread then keeps four loads in flight
    static std::atomic<int> sm_count[64] = {};
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int sms = sm_count[dev].load(std::memory_order_relaxed);
    if (sms == 0) {
      e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
      sm_count[dev].store(sms, std::memory_order_relaxed);
    }
    int64_t want = (n / 8 + 255) / 256;
    const int64_t cap = static_cast<int64_t>(sms) * 8;
    const unsigned blocks = static_cast<unsigned>(want < 1 ? 1 : (want > cap ? cap : want));
    absmax_bf16_kernel<<<blocks, 256, 0, stream>>>(static_cast<const uint16_t*>(x), n, amax_bits);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  e4m3_scale_kernel<<<1, 1, 0, stream>>>(amax_bits, scale_out);
  return cudaGetLastError();
}

}  // namespace qkv
