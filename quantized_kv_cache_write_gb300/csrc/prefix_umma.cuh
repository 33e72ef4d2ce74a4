// The shared prefix of qkv_prefix_attn on the fifth-generation tensor cores: S = Q K^T and O += P V by
// tcgen05.mma with accumulators in tensor memory, for batches with many (row, query head) pairs.
//
// The pairs of all rows (row-major) are the M of both products. A team of CG SMs (a cluster; the
// MMAs span both SMs of a pair) takes NT tiles of 128 CG pairs: two tiles for 128-wide heads, so that one
// tile's softmax runs under the other's MMAs; one for 256-wide heads, whose O takes half of tensor
// memory, with S double-buffered instead. The (tile, KV head) x key-block units of the call are cut
// into equal contiguous ranges, one per team, one CTA per SM; a range covers part of one tile's keys or
// the end of one and the start of the next, and every such segment leaves a partial result that the
// merge joins. A pair's SMs each hold their own 128 pairs' Q, S, P and O, and half of K (by keys)
// and V (by dims): each converts half of the pool's values, and shared memory is read and written half as
// often per MMA as with one SM.
//
// Warps: sixteen for the softmax (four threads per pair, a quarter of a block's columns each), two groups of four
// producers, one for the records, one for the scales, one for the MMAs (of the team's first SM). Slots
// (rows of 128 B, 128 B swizzle) pass from the producers to the MMA warp in the order
// K_0 K_1 V_0 K_2 V_1 ..., one group every second one; K is K-major, V MN-major, and both are stored alike, one
// 128 B row per key and 64 dims.
//   records: block list -> record numbers of a block's keys, into a ring, eight blocks ahead.
//   producers: 16 B loads into registers, converted to fp16 (codes are exact) and stored to the slot once it is
//     free; then the registers take the group's next slot. 16-bit pools are copied straight into the slot
//     (cp.async).
//   scales: K and V scales, the mask of the block's keys and the largest V scale into a small ring.
//   MMA: one warp, of which an elected lane issues. P is the A operand in tensor memory, in the columns of the S it was made from.
//   softmax: y = S ks fac (log2 units). Reference R = M + E - kShift: M follows the row's maximum lazily
//     (raised when a logit passes it by 2^kRaise), E is a power-of-two bound on the V scales, so p vs 2^-R
//     stays below fp16's range; l and O both carry 2^-R, and a raise of R rescales both. The thread's columns
//     stay in registers from the one load of S on; the row's four threads vote whether any column passes the
//     reference by too much; then p replaces the columns, and each thread's part of P goes over its own part of S.
//     A raise rescales O last, after P is stored, when those registers are free. Measured, 256 rows x 16 heads
//     behind 65536 int8 keys, us for the call: 235; 253 with the maxima exchanged in every block instead of the
//     vote; 269 with O rescaled before P besides. 64 rows x 64 heads behind 32768 e4m3 keys, thousands of cycles:
//     142; 165 with the maxima exchanged; 265 with O rescaled before P besides.
// Arithmetic as in prefix_attn.cuh: exact codes, logits and sums in fp32, p rounded once.
//
// The roles' loops are kept rolled: five of them run at once on each scheduler, and fully unrolled they
// outgrow the instruction cache (measured: 5.3 stalled warps per issue on instruction fetch, 256 rows x 16
// heads behind 65536 int8 keys 549 us against 394 us).
//
// Every wait is bounded: a wait that runs out sets QKV_DEV_TIMEOUT, the CTA drains its MMAs, frees its
// tensor memory and returns.
#pragma once

#include <cstdlib>

#include "masked_tiles.cuh"

namespace qkv {
namespace prefix {

constexpr int kTileM = 128;  // pairs of a tile on one SM
constexpr int kProdWarps = 4;  // of a group; two groups
constexpr int kParts = 4;      // threads of a pair: each takes a part of a block's columns
constexpr uint64_t kWaitNs = 2000000000;  // after which a wait is declared lost
constexpr int kScRing = 4, kRecRing = 8;
// keys of a block: 128; 64 where one SM holds 256-wide heads alone
constexpr int umma_block_keys(int head_dim, int cg) { return head_dim == 256 && cg == 1 ? 64 : 128; }

template <int FMT, int HD, int NT, int CG, bool MASK = false>
struct Umma {
  using F = Fmt<FMT>;
  static constexpr int KB = umma_block_keys(HD, CG);
  static constexpr int kSoftWarps = 4 * kParts, kRecWarp = kSoftWarps + 2 * kProdWarps, kScWarp = kRecWarp + 1, kMmaWarp = kScWarp + 1;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  // The softmax's window: a logit may pass its reference by 2^kRaise, and p there is 2^kShift (int8: times a V
  // scale over its bound, which sits up to 2^kHeadroom above the largest seen). fp16 operands stay below 2^15, and
  // a p below fp16's normal range is off by at most 2^-25 2^-kShift, int8 2^(1 + kHeadroom) of that: 2^-28 of the
  // largest V. bf16 operands have fp32's range.
  static constexpr float kRaise = F::kBf16 ? 16.f : F::kInt8 ? 10.f : 12.f, kShift = F::kBf16 ? 0.f : 15.f - kRaise;
  static constexpr int kHeadroom = 1;
  static constexpr int kKRows = KB / CG, kVDims = HD / CG;  // this SM's part of a block
  static constexpr uint32_t kSlotBytes = uint32_t(KB) * HD * 2 / CG;
  static constexpr uint32_t kQTile = kTileM * HD * 2;
  static constexpr int kSlots = kSlotBytes == 16384 ? 8 : NT * HD >= 256 ? 4 : 5;
  static constexpr uint32_t kQ = 0, kRing = NT * kQTile, kSc = kRing + kSlots * kSlotBytes;
  // per block: K scales, V scales, key mask (4 words), largest V scale
  static constexpr uint32_t kScVs = 4 * KB, kScMask = 8 * KB, kScVmax = kScMask + 16, kScStage = kScVmax + 16;
  static constexpr uint32_t kRec = kSc + kScRing * kScStage;       // record numbers of a block's keys
  static constexpr uint32_t kRow = kRec + kRecRing * 4 * KB;       // per row: its threads' maxima (sums), two phases
  // MASK: each pair's range, nearest position and slope; each softmax warp's positions that all its rows see; blocks whose
  // values that are not finite were left out (a bit for each block modulo 32)
  static constexpr uint32_t kTab = kRow + 2 * kParts * 4 * kTileM, kAll = kTab + (MASK ? NT * kTileM * 16 : 0);
  static constexpr uint32_t kSeg = kAll + (MASK ? NT * kSoftWarps * 8 : 0);  // the published segments
  static constexpr uint32_t kOdd = kSeg + (MASK ? 4 * kSegWords * kSegRing : 0);
  // each softmax warp's place for a tile's output on its way out: 32 rows of 64 B, of 32 B where there is no room for those
  static constexpr uint32_t kOut = kOdd + (MASK ? 16 : 0);
  static constexpr uint32_t kOutRow = kOut + kSoftWarps * 32 * 64 + 2048 <= 232448 ? 64 : 32;
  static constexpr uint32_t kSegFull = kOut + (MASK ? kSoftWarps * 32 * kOutRow : 0), kSegEmpty = kSegFull + (MASK ? 8 * kSegRing : 0);
  static constexpr uint32_t kBar = kSegEmpty + (MASK ? 8 * kSegRing : 0);
  static constexpr uint32_t kFull = kBar, kEmpty = kFull + 8 * kSlots, kSFull = kEmpty + 8 * kSlots, kPFull = kSFull + 16,
                            kPvDone = kPFull + 16, kScFull = kPvDone + 16, kScEmpty = kScFull + 8 * kScRing,
                            kRecFull = kScEmpty + 8 * kScRing, kRecEmpty = kRecFull + 8 * kRecRing,
                            kQFull = kRecEmpty + 8 * kRecRing,
                            kDrain = kQFull + 8, kTmemSlot = kDrain + 8, kFlag = kTmemSlot + 4, kSmem = kFlag + 4 + 1024;
  static_assert(kSmem <= 232448, "one CTA per SM");
  // tensor memory columns: O of each tile, then two S buffers
  static constexpr uint32_t kO = 0, kS = NT * HD;
  static_assert(kS + 2 * KB <= 512, "tensor memory");
  // instruction descriptors (kind::f16, fp32 accumulator): A / B type at bits 7 and 10 (0 fp16, 1 bf16),
  // B MN-major at bit 16, N / 8 at bit 17, M / 16 at bit 24
  static constexpr uint32_t kType = F::kBf16 ? (1u << 7) | (1u << 10) : 0u;
  static constexpr uint32_t kM = uint32_t(kTileM * CG / 16) << 24;
  static constexpr uint32_t kIdS = (1u << 4) | kType | (uint32_t(KB / 8) << 17) | kM;
  static constexpr uint32_t kIdO = (1u << 4) | kType | (1u << 16) | (uint32_t(HD / 8) << 17) | kM;
};

// 128 B-swizzled shared-memory matrix descriptor: address, leading and stride byte offsets, version 1.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t((sbo >> 4) & 0x3FFFu) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// The MMAs' issuing warp runs its loop with all lanes, so that descriptors stay in uniform registers; one
// elected lane (`lead`) issues. acc: add to D, else overwrite it.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
#define QKV_PREFIX_MMA(GROUP, A, AC)                                                                                    \
  asm volatile(                                                                                                         \
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"                                         \
      " @q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], " A ", %2, %3, p;\n}\n" ::"r"(d), AC(a), "l"(b), "r"(id),   \
      "r"(acc), "r"(lead)                                                                                               \
      : "memory")
template <int CG>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t lead) {
  if (CG == 2) QKV_PREFIX_MMA("2", "%1", "l");
  else QKV_PREFIX_MMA("1", "%1", "l");
}
template <int CG>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t lead) {
  if (CG == 2) QKV_PREFIX_MMA("2", "[%1]", "r");
  else QKV_PREFIX_MMA("1", "[%1]", "r");
}
#undef QKV_PREFIX_MMA
// Arrive on this barrier (of both SMs of a pair) when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void commit_to(uint32_t mbar) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(mbar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(mbar) : "memory");
}
template <int CG>
__device__ __forceinline__ void team_tmem_alloc(uint32_t smem_dst) {
  if (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_dst), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  } else {
    tmem_alloc(smem_dst, 512);
    tmem_relinquish_alloc_permit();
  }
}
template <int CG>
__device__ __forceinline__ void team_tmem_dealloc(uint32_t taddr) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(512u) : "memory");
  else
    tmem_dealloc(taddr, 512);
}
// Every thread of the team.
template <int CG>
__device__ __forceinline__ void team_sync() {
  if (CG == 2) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  } else {
    __syncthreads();
  }
}
__device__ __forceinline__ void bar_init(uint32_t mbar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(mbar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t mbar) {
  asm volatile("{\n .reg .b64 st;\n mbarrier.arrive.shared::cta.b64 st, [%0];\n}\n" ::"r"(mbar) : "memory");
}
// Arrive on the barrier at this offset in the team's first SM. What it hands over lies in this SM's own
// shared or tensor memory and is read there by the MMAs, so the proxy (or tensor-memory) fence before it is
// the order that is needed; a release at cluster scope would wait for the thread's global loads too (measured:
// about 750 cycles an arrival, twice per block and producer).
template <int CG>
__device__ __forceinline__ void lead_arrive(uint32_t mbar) {
  if (CG == 2)
    asm volatile(
        "{\n .reg .b32 ra;\n mapa.shared::cluster.u32 ra, %0, 0;\n"
        " mbarrier.arrive.shared::cluster.b64 _, [ra];\n}\n" ::"r"(mbar)
        : "memory");
  else
    bar_arrive(mbar);
}
// One poll: the hardware may suspend the thread until the phase is over, for up to a millisecond here.
__device__ __forceinline__ bool bar_try(uint32_t mbar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(mbar), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0u;
}
// Whether the phase of the given parity is over, without waiting for it.
__device__ __forceinline__ bool bar_test(uint32_t mbar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(mbar), "r"(parity)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t));
  return t;
}
// Wait for the phase of the given parity; false when the time ran out or (where it `stops` a wait)
// the CTA's stop flag is up.
__device__ __forceinline__ bool bar_wait(uint32_t mbar, uint32_t parity, uint32_t flag, bool stops = true) {
  if (bar_try(mbar, parity)) return true;
  const uint64_t start = now_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (bar_try(mbar, parity)) return true;
    if (stops && lds32(flag) != 0u) return false;
    if (now_ns() - start > kWaitNs) break;
  }
  sts32(flag, 1u);
  return false;
}
// One instruction instead of two on the integer pipe, the busiest of the softmax (NaN operands drop out, as with fmaxf):
// 256 rows x 16 heads behind 65536 int8 keys 234 -> 231 us.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
template <typename T>
__device__ __forceinline__ void swap_places(T& a, T& b) {
  const T x = a;
  a = b, b = x;
}
// N columns times their scales; N columns whose key is missing to -inf.
template <int N>
__device__ __forceinline__ void scale_by(float (&v)[N], const float4* src) {
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    const float4 f = src[k];
    f2scale(v + 4 * k, f2pack(f.x, f.y));
    f2scale(v + 4 * k + 2, f2pack(f.z, f.w));
  }
}
template <int N>
__device__ __forceinline__ void scale_by(float (&v)[N], uint32_t at) {
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    const uint4 f = lds128(at + 16 * k);
    f2scale(v + 4 * k, f2pack(__uint_as_float(f.x), __uint_as_float(f.y)));
    f2scale(v + 4 * k + 2, f2pack(__uint_as_float(f.z), __uint_as_float(f.w)));
  }
}
template <int N>
__device__ __forceinline__ void mask_by(float (&v)[N], uint32_t mask) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (!((mask >> k) & 1)) v[k] = -INFINITY;
}
// 16 bytes, or zeros; issued here, however late they are used.
__device__ __forceinline__ uint4 load_if(const uint4* p, bool there) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
      " @p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(static_cast<uint32_t>(there)));
  return v;
}
// 16 or 32 columns of this thread's tensor-memory lane; 8 or 16 packed ones
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[32]) { tmem_ld32(taddr, v); }
__device__ __forceinline__ void tmem_loaded(float (&v)[32]) { tmem_wait_ld(v); }
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&v)[16]) { tmem_st_x16(taddr, v); }
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_loaded(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])::"memory");
}
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The team whose range holds unit x.
__device__ __forceinline__ uint32_t team_of(const PrefixArgs& a, uint32_t x) {
  const uint32_t cut = a.umma_extra * (a.umma_share + 1);
  return x < cut ? x / (a.umma_share + 1) : a.umma_extra + (x - cut) / a.umma_share;
}

// A team's next segment: the part of its unit range that lies in one (KV head, pair tile).
struct Segment {
  uint32_t u, end;  // units still to do
  uint32_t team;
  int tile, b0, b1, part;
  __device__ __forceinline__ bool next(const PrefixArgs& a) {
    if (u >= end) return false;
    const uint32_t nb = a.umma_blocks, t = u / nb, t0 = t * nb;
    tile = static_cast<int>(t);
    b0 = static_cast<int>(u - t0);
    b1 = static_cast<int>(min(end - t0, nb));
    part = b0 > 0 ? static_cast<int>(team - team_of(a, t0)) : 0;  // a tile's first units: its first part
    u = t0 + b1;
    return true;
  }
};
template <int CG>
__device__ __forceinline__ Segment first_segment(const PrefixArgs& a) {
  Segment s;
  s.team = blockIdx.x / CG;
  s.u = s.team * a.umma_share + min(s.team, a.umma_extra);
  s.end = s.u + a.umma_share + (s.team < a.umma_extra ? 1 : 0);
  return s;
}

// Positions of the prefix to records of the pool.
// MASK: positions from `lo` on only.
template <bool MASK>
struct Records {
  const int32_t* blocks;
  int64_t num_slots;
  int bsz, shift, len, H, h, lo = 0;
  bool pow2;
  __device__ __forceinline__ bool in(int p) const { return p < len && (!MASK || p >= lo); }
  __device__ __forceinline__ void init(const PrefixArgs& a, int head) {
    blocks = a.prefix_blocks, num_slots = a.num_slots, bsz = a.block_size, len = a.prefix_len, H = a.num_kv_heads, h = head;
    pow2 = (bsz & (bsz - 1)) == 0, shift = __ffs(bsz) - 1;
  }
  __device__ __forceinline__ void of_tile(const PrefixArgs& a, const MaskedTile& t) {
    lo = t.lo, len = t.hi;
    blocks = a.block_table + static_cast<int64_t>(t.hi > 0 ? t.seq : 0) * a.max_blocks;  // no keys: no sequence either
  }
  __device__ __forceinline__ int block_of(int p) const { return pow2 ? p >> shift : p / bsz; }
  // block id of position p, -1 past the prefix
  __device__ __forceinline__ int lookup(int p) const { return in(p) ? __ldg(blocks + block_of(p)) : -1; }
  // record of position p in block blk, -1: none
  __device__ __forceinline__ int record(int p, int blk) const {
    const int64_t slot = static_cast<int64_t>(blk) * bsz + (p - block_of(p) * bsz);
    return (in(p) && blk >= 0 && slot < num_slots) ? static_cast<int>(slot) * H + h : -1;
  }
};

// A 16-bit value (its bits) that is not finite.
template <bool BF16>
__device__ __forceinline__ bool odd16(uint32_t x) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
  return (x & kExp) == kExp;
}
// Two 16-bit values with those that are not finite set to 0.
template <bool BF16>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  return w & ((odd16<BF16>(w) ? 0u : 0x0000ffffu) | (odd16<BF16>(w >> 16) ? 0u : 0xffff0000u));
}

// E4M3 codes with the NaNs set to 0; not 0: there were any.
__device__ __forceinline__ uint32_t drop_odd_e4m3(uint4& v) {
  const uint32_t a = __vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu), b = __vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu);
  const uint32_t c = __vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu), d = __vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  v.x &= ~a, v.y &= ~b, v.z &= ~c, v.w &= ~d;
  return a | b | c | d;
}

// One operand's part of a block as the producers move it: ROWS keys of kBytes bytes each, from byte
// `off` of the record on. Each warp of a group takes a quarter of the rows; a row is kLpr lanes of 16 B. In the slot,
// 64 dims of one key are a 128 B row, swizzled; columns of 64 dims are ROWS rows apart.
template <int FMT, int HD, int ROWS, int DIMS>
struct Operand {
  using F = Fmt<FMT>;
  static constexpr int kBytes = F::kBytes ? DIMS : 2 * DIMS, kLpr = kBytes / 16;
  static constexpr int kPerInstr = 32 / kLpr, kWarpRows = ROWS / kProdWarps, kInstr = kWarpRows / kPerInstr;
  static constexpr uint32_t kCol = ROWS * 128;
  static constexpr int kGlobalRow = F::kInline ? HD + 4 : F::kBytes ? HD : 2 * HD;
  static_assert(kLpr <= 32 && kWarpRows <= 32 && kInstr >= 1, "rows of at most 512 B");

  // 16-bit pools: the whole part by cp.async; missing keys are zero-filled
  static __device__ __forceinline__ void copy(uint32_t slot, const uint8_t* cache, int pw, int lane, uint32_t rec, int off) {
    const int ch = lane % kLpr;
#pragma unroll 4
    for (int u = 0; u < kInstr; ++u) {
      const int lr = kPerInstr * u + lane / kLpr;
      const int rk = static_cast<int>(lds32(rec + 4 * lr));
      const int row = kWarpRows * pw + lr;
      cp_async16(slot + (ch >> 3) * kCol + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                 cache + static_cast<uint64_t>(static_cast<uint32_t>(max(rk, 0))) * kGlobalRow + off + 16 * ch, rk >= 0 ? 16 : 0);
    }
  }
  // The lane's own copied chunks with the values that are not finite set to 0; whether there were any.
  template <bool BF16>
  static __device__ __forceinline__ bool drop_odd(uint32_t slot, int pw, int lane) {
    const int ch = lane % kLpr;
    bool any = false;
#pragma unroll 4
    for (int u = 0; u < kInstr; ++u) {
      const int row = kWarpRows * pw + kPerInstr * u + lane / kLpr;
      const uint32_t at = slot + (ch >> 3) * kCol + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
      const uint4 v = lds128(at);
      const uint4 w = make_uint4(finite2<BF16>(v.x), finite2<BF16>(v.y), finite2<BF16>(v.z), finite2<BF16>(v.w));
      if ((v.x ^ w.x) | (v.y ^ w.y) | (v.z ^ w.z) | (v.w ^ w.w)) sts128(at, w), any = true;
    }
    return any;
  }
};

// Bytes pools: a slot's rows of one operand as a lane sees them. K's and V's parts differ only in these
// numbers, so one copy of the code serves both.
struct Rows {
  const uint8_t* src;  // the lane's 16 B of record 0
  uint32_t rec;        // the ring entry's offset of the lane's first row
  uint32_t at, first;  // the lane's place in a slot: column and row, and its first chunk (16 B)
  uint32_t odd;        // whether that is the odd chunk of the pair: the eight lanes of a store phase fill eight
  int per;             // keys per instruction
};
template <typename OP>
__device__ __forceinline__ Rows rows_of(const uint8_t* src, int pw, int lane, int first_row) {
  constexpr int L = OP::kLpr;
  const int ch = lane % L;  // the lane's 16 dims: two chunks of the key's 128 B row
  Rows r;
  r.src = src + 16 * ch;
  r.rec = 4 * (first_row + OP::kWarpRows * pw + lane / L);
  r.odd = L > 4 && (ch & 4) ? 1 : 0;
  r.at = (ch >> 2) * OP::kCol + (OP::kWarpRows * pw + lane / L) * 128;  // the warp's first row is a multiple of 8
  r.first = ((2 * (ch & 3) + r.odd) ^ (lane / L)) << 4;
  r.per = OP::kPerInstr;
  return r;
}
// N instructions' 16 B (a missing key's: zeros) into registers.
template <int FMT, int HD, int N>
__device__ __forceinline__ void load_rows(uint4 (&raw)[N], const Rows& r, uint32_t ring) {
  using F = Fmt<FMT>;
  constexpr int kGlobalRow = F::kInline ? HD + 4 : HD;
  int rk[N];
#pragma unroll
  for (int u = 0; u < N; ++u) rk[u] = static_cast<int>(lds32(ring + r.rec + 4 * r.per * u));
#pragma unroll
  for (int u = 0; u < N; ++u) {
    raw[u] = make_uint4(0, 0, 0, 0);
    if (rk[u] >= 0) {
      const uint8_t* p = r.src + static_cast<uint64_t>(static_cast<uint32_t>(rk[u])) * kGlobalRow;
      if (F::kInline) {  // records sit on 4 B boundaries
        const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
        raw[u] = make_uint4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
      } else {
        raw[u] = __ldg(reinterpret_cast<const uint4*>(p));
      }
    }
  }
}
// The codes to fp16 and into the slot.
template <int FMT, int N>
__device__ __forceinline__ void convert_rows(uint32_t slot, const Rows& r, const uint4 (&raw)[N]) {
  using F = Fmt<FMT>;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (F::kInt8) {
        o[2 * k] = i8pair_to_f16x2(w[k]);
        o[2 * k + 1] = i8pair_to_f16x2(w[k] >> 8);
      } else {
        o[2 * k] = e4m3pair_to_f16x2(w[k]);
        o[2 * k + 1] = e4m3pair_to_f16x2(w[k] >> 16);
      }
    }
    const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
    const uint32_t row = r.per * u;  // row & 7: these bits and the lane's, which are disjoint
    const uint32_t a0 = slot + r.at + row * 128 + (r.first ^ ((row & 7) << 4));
    sts128(a0, r.odd ? hi : lo);
    sts128(a0 ^ 16, r.odd ? lo : hi);
  }
}

// Slots of a segment of B blocks in ring order: K_0 K_1 V_0 K_2 V_1 ... K_B-1 V_B-2 V_B-1.
__device__ __forceinline__ uint32_t k_slot(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t v_slot(int j, int B) { return j == B - 1 ? 2 * B - 1 : 2 * j + 2; }

// Scores of N columns in log2 units from their logits: x fac, capped and less the distance bias. The columns' positions are
// base + k; `row` addresses the pair's nearest position and its slope. Where the warp's logits are all small against the cap,
// as they nearly always are, tanh is its polynomial, two columns at a time; the bias is linear where no row of the warp has
// its nearest position inside the columns. 2048 rows x 32 heads of 128 behind 20000 bf16 keys, us: 1036 without either; with
// the cap 1831 while each column chose for itself.
template <int N>
__device__ __forceinline__ void adjust_scores(float (&x)[N], float fac, float cap, bool bias, uint32_t row, int base) {
  if (cap > 0.f) {
    const uint64_t fac2 = f2pack(fac, fac);
    const float up = cap * kLog2e;
    float big = 0.f;
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      f2unpack(f2mul(f2pack(x[k], x[k + 1]), fac2), x[k], x[k + 1]);
      big = max3(big, fabsf(x[k]), fabsf(x[k + 1]));
    }
    if (__all_sync(0xffffffffu, big < kTanhSmall)) {
      uint64_t c[6];
#pragma unroll
      for (int i = 0; i < 6; ++i) c[i] = f2pack(up * kTanh[i], up * kTanh[i]);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        const uint64_t z = f2pack(x[k], x[k + 1]), z2 = f2mul(z, z);
        uint64_t s = c[5];
#pragma unroll
        for (int i = 4; i >= 0; --i) s = f2fma(z2, s, c[i]);
        f2unpack(f2mul(z, s), x[k], x[k + 1]);
      }
    } else {
      // column by column, the large ones first: both forms of all columns at once would spill
      uint32_t small = 0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (fabsf(x[k]) < kTanhSmall) small |= 1u << k;
        else x[k] = tanh_exp(x[k]);
      }
      asm volatile("" : "+r"(small));
      // the polynomial step by step as above, so that a score does not depend on the rows that share its warp
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float z2 = x[k] * x[k];
        float s = up * kTanh[5];
#pragma unroll
        for (int i = 4; i >= 0; --i) s = fmaf(z2, s, up * kTanh[i]);
        x[k] *= (small >> k) & 1 ? s : up;
      }
    }
    fac = 1.f;
  }
  if (bias) {
    const uint64_t fac2 = f2pack(fac, fac);
    const uint2 v = lds64(row);
    const int at = base - static_cast<int>(v.x);
    const float from = static_cast<float>(at), slope = __uint_as_float(v.y);
    if (__all_sync(0xffffffffu, at >= 0 || at + N <= 1)) {
      const float s = at >= 0 ? slope : -slope;
      const uint64_t s2 = f2pack(s, s), from2 = f2pack(s * from, s * from), two = f2pack(2.f, 2.f);
      uint64_t k2 = f2pack(0.f, 1.f);
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        f2unpack(f2fma(f2pack(x[k], x[k + 1]), fac2, f2fma(s2, k2, from2)), x[k], x[k + 1]);
        k2 = f2add(k2, two);
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = fmaf(slope, fabsf(from + static_cast<float>(k)), x[k] * fac);
    }
  }
}

// Record of both SMs (each has half of the dims, and all rows) that block j holds values that were left out. It is there
// before the block's hand-over, which the product and its readers wait for.
template <int CG>
__device__ __forceinline__ void note_odd(uint32_t odd, int j) {
#pragma unroll
  for (int i = 0; i < CG; ++i)
    asm volatile("{\n .reg .b32 ra;\n mapa.shared::cluster.u32 ra, %0, %1;\n red.relaxed.cluster.shared::cluster.or.b32 [ra], %2;\n}\n" ::"r"(odd), "r"(i),
                 "r"(1u << (j & 31))
                 : "memory");
  asm volatile("fence.acq_rel.cluster;\n" ::: "memory");
}

// The values that are not finite which the producers of a masked segment left out of blocks that some rows do not see whole,
// added to the thread's part of O (HD / kParts dims from d0 on) where its row sees their keys. Nearly always there are
// none.
struct Odd {
  const MaskedTile* tile;
  int b0, b1;       // the segment's blocks
  uint32_t bits;    // address of the record of such blocks
  uint32_t range;   // and of the pair's range
};
template <int FMT, int HD, int KB>
__device__ __forceinline__ void add_odd(const PrefixArgs& a, const Odd& odd, int h, uint32_t to, int d0, bool in) {
  using F = Fmt<FMT>;
  const uint32_t bits = lds32(odd.bits);
  if (__builtin_expect(!__any_sync(0xffffffffu, bits != 0u), 1)) return;
  const uint2 lim = lds64(odd.range);
  const int lo = static_cast<int>(lim.x), hi = in ? static_cast<int>(lim.y) : 0;
  const MaskedTile tile = *odd.tile;
  Records<true> rc;
  rc.init(a, h);
  rc.of_tile(a, tile);
  for (int j = odd.b0; j < odd.b1; ++j) {
    const int p0 = j * KB;
    if (!((bits >> (j & 31)) & 1) || (p0 >= tile.all_lo && p0 + KB <= tile.all_hi)) continue;
    for (int c = 0; c < HD / kParts; c += 16) {
      float o[16];
      tmem_load(to + c, o);
      tmem_loaded(o);
      for (int p = max(p0, tile.lo); p < min(p0 + KB, tile.hi); ++p) {
        const int rec = rc.record(p, rc.lookup(p));
        if (rec < 0 || p < lo || p >= hi) continue;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(rec)) * HD + d0 + c + k;
          if (FMT == QKV_E4M3) {
            if ((__ldg(a.v_cache + at) & 0x7f) == 0x7f) o[k] = NAN;
          } else {
            const uint32_t v = __ldg(reinterpret_cast<const uint16_t*>(a.v_cache) + at);
            if (odd16<F::kBf16>(v)) o[k] += F::kBf16 ? __uint_as_float(v << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
          }
        }
      }
      __syncwarp();
      uint32_t w[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k]);
      tmem_st_x16(to + c, w);
      tmem_wait_st();
    }
  }
}

// The segments of the prefix, or the published ones of the masked rows, alike for the roles.
template <bool MASK, typename U, int CG>
struct Segments;
template <typename U, int CG>
struct Segments<false, U, CG> : Segment {
  __device__ __forceinline__ void begin(const PrefixArgs& a, uint32_t) { static_cast<Segment&>(*this) = first_segment<CG>(a); }
  __device__ __forceinline__ int head(const PrefixArgs& a) const { return tile / a.umma_ptiles; }
  __device__ __forceinline__ void done() const {}
};
template <typename U, int CG>
struct Segments<true, U, CG> {
  uint32_t sb, count;
  int b0, b1;
  bool lost;  // the wait for a segment ran out
  __device__ __forceinline__ void begin(const PrefixArgs&, uint32_t base) { sb = base, count = 0, lost = false; }
  __device__ __forceinline__ uint32_t at(uint32_t n) const { return sb + U::kSeg + 4 * kSegWords * (n % kSegRing); }
  __device__ __forceinline__ int word(SegWord w) const { return static_cast<int>(lds32(at(count - 1) + 4 * w)); }
  __device__ __forceinline__ int head(const PrefixArgs&) const { return word(kSegHead); }
  __device__ __forceinline__ bool next(const PrefixArgs&) {
    const uint32_t n = count % kSegRing;
    lost = !__all_sync(0xffffffffu, bar_wait(sb + U::kSegFull + 8 * n, (count / kSegRing) & 1, sb + U::kFlag));
    if (lost) return false;
    take();
    return b1 > b0;
  }
  __device__ __forceinline__ void take() {
    ++count;
    b0 = word(kSegB0), b1 = word(kSegB1);
  }
  // the warp is done with segment n, or the one at hand
  __device__ __forceinline__ void release(uint32_t n) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(sb + U::kSegEmpty + 8 * (n % kSegRing));
  }
  __device__ __forceinline__ void done() const { release(count - 1); }
};
// The walk's next segment into the ring as number n, or the mark that there is none; whether there is one.
template <int KB, int CG, typename U>
__device__ __forceinline__ bool publish(const PrefixArgs& a, MaskedWalk& w, uint32_t sb, uint32_t n) {
  bool found = false;
  int b0 = 0, b1 = 0, part = -1, chunk = 0, i = 0, h = 0;
  uint32_t rest = 0;  // of the tile's blocks, those of the teams after this one
  MaskedTile t = {};
  while (w.left != 0 && !found) {
    while (w.i >= static_cast<int>(plan_chunk(a)[w.chunk].tiles)) {  // there is work left, so there is a tile
      w.i = 0;
      if (++w.chunk == a.plan_chunks) w.chunk = 0, ++w.h;
    }
    chunk = w.chunk, i = w.i, h = w.h;
    t = plan_tiles(a, chunk)[i];
    const uint32_t cost = plan_tiles(a, chunk)[i + 1].first - t.first, extra = a.tile_cost, took = min(w.left, cost - w.skip);
    const uint32_t from = max(w.skip, extra) - extra, to = max(w.skip + took, extra) - extra;
    w.left -= took;
    w.skip = 0;
    ++w.i;
    found = to > from;
    b0 = t.lo / KB + static_cast<int>(from), b1 = t.lo / KB + static_cast<int>(to);
    part = to - from == cost - extra ? -1 : static_cast<int>(2 * w.team + (from > 0 ? 0 : 1));
    rest = cost - extra - to;
  }
  if (!found) b0 = b1 = 0, t.nrows = 0, t.row0 = 0;
  if (n >= kSegRing && !__all_sync(0xffffffffu, bar_wait(sb + U::kSegEmpty + 8 * (n % kSegRing), (n / kSegRing - 1) & 1, sb + U::kFlag)))
    return false;
  if ((threadIdx.x & 31) == 0) {
    const uint32_t at = sb + U::kSeg + 4 * kSegWords * (n % kSegRing);
    sts128(at, make_uint4(b0, b1, t.row0, t.nrows));
    sts128(at + 16, make_uint4(h, part, t.all_lo, t.all_hi));
    sts128(at + 32, make_uint4(chunk, i, 0, 0));
    bar_arrive(sb + U::kSegFull + 8 * (n % kSegRing));
    // begun and not finished, the team's last segment: one SM notes it for the join
    if (found && part == static_cast<int>(2 * w.team + 1) && blockIdx.x % CG == 0)
      *reinterpret_cast<int4*>(plan_join(a, w.team)) = make_int4(t.row0, t.nrows, h, static_cast<int>(1 + w.teams_of(rest)));
  }
  __syncwarp();
  // its queries into L2, a segment ahead of their loads
  const int G = a.num_q_heads / a.num_kv_heads;
  for (int k = threadIdx.x & 31; k < t.nrows; k += 32)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(a.q + (t.row0 + static_cast<int64_t>(k)) * a.q_stride +
                                                                   static_cast<int64_t>(h) * G * a.head_dim),
                 "r"(static_cast<uint32_t>(2 * G * a.head_dim))
                 : "memory");
  return found;
}
// Missing keys are flagged where a row of the tile sees them.
static __device__ __noinline__ void flag_if_seen(const int32_t* start, const int32_t* end, const int32_t* pos, int window, int max_end, int rows, int p,
                                          uint32_t* status) {
  for (int k = 0; k < rows; ++k) {
    const int e = __ldg(end + k), b = start != nullptr ? __ldg(start + k) : 0, at = pos != nullptr ? __ldg(pos + k) : e - 1;
    if (e > max_end || b < 0 || at < 0 || at > kMaxRowPos) continue;  // an invalid row, which sees nothing
    if (p < e && p >= (window > 0 ? max(b, at - window + 1) : b)) {
      atomicOr(status, QKV_DEV_BAD_INDEX);
      return;
    }
  }
}

// MASK: qkv_masked_attn, with the work list of masked_tiles.cuh. What differs: the tile's keys lie in its sequence's row
// of the block table, a block that not all of a warp's rows see whole is masked row by row, scores may be capped and get the
// distance bias, and a tile that one team has whole is written out here. A value of V that is not finite in a
// block that some row of the tile does not see whole is left out of the product (0 times it would not be 0) and added at
// the end for the rows that see it. A segment's
// blocks are taken from the last to the first: a row's nearest keys, whose bias is smallest, then set its reference at once.
// MODE: kPrefix, kMasked, or kAdjusted, which is masked with capped scores or a bias (their code takes registers that the
// others' softmax would spill).
constexpr int kPrefix = 0, kMasked = 1, kAdjusted = 2;
template <int FMT, int HD, int NT, int CG, int MODE>
__global__ void __launch_bounds__(Umma<FMT, HD, NT, CG, MODE != kPrefix>::kThreads, 1) prefix_umma_kernel(const PrefixArgs a) {
  constexpr bool MASK = MODE != kPrefix;
  using F = Fmt<FMT>;
  using U = Umma<FMT, HD, NT, CG, MASK>;
  constexpr int NS = U::kSlots, KB = U::KB;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CG == 2 ? blockIdx.x & 1 : 0;  // this SM in the team
  const uint32_t sb = (smem_u32(smem) + 1023u) & ~1023u, smem0 = smem_u32(smem), flag = sb + U::kFlag;  // swizzled rows: 1 KB aligned
  const int H = a.num_kv_heads, G = a.num_q_heads / H;
  const uint32_t pairs = static_cast<uint32_t>(a.rows) * G;
  let_next_start();

  if (warp == U::kMmaWarp) {
    team_tmem_alloc<CG>(sb + U::kTmemSlot);
    if (lane == 0) {
      for (int s = 0; s < NS; ++s) {
        bar_init(sb + U::kFull + 8 * s, kProdWarps * CG);
        bar_init(sb + U::kEmpty + 8 * s, 1);
      }
      for (int b = 0; b < 2; ++b) {
        bar_init(sb + U::kSFull + 8 * b, 1);
        bar_init(sb + U::kPFull + 8 * b, U::kSoftWarps * CG);
        bar_init(sb + U::kPvDone + 8 * b, 1);
      }
      for (int s = 0; s < kScRing; ++s) {
        bar_init(sb + U::kScFull + 8 * s, 1);
        bar_init(sb + U::kScEmpty + 8 * s, U::kSoftWarps);
      }
      for (int s = 0; s < kRecRing; ++s) {
        bar_init(sb + U::kRecFull + 8 * s, 1);
        bar_init(sb + U::kRecEmpty + 8 * s, 2 * kProdWarps + 1);  // a K and a V group, and scales
      }
      bar_init(sb + U::kQFull, U::kSoftWarps * CG);
      for (int s = 0; MASK && s < kSegRing; ++s) {
        bar_init(sb + U::kSegFull + 8 * s, 1);
        // the softmax, two groups of producers, the scales and, in the team's first SM, the MMAs
        bar_init(sb + U::kSegEmpty + 8 * s, U::kSoftWarps + 2 * kProdWarps + 1 + (rank == 0 ? 1 : 0));
      }
      bar_init(sb + U::kDrain, 1);
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
      sts32(flag, 0u);
      if (MASK) sts32(sb + U::kOdd, 0u);
    }
    __syncwarp();
  }
  tmem_fence_before_sync();
  __syncthreads();
  team_sync<CG>();
  tmem_fence_after_sync();
  const uint32_t tb = lds32(sb + U::kTmemSlot);
  if (MASK) await_previous();  // the work list
  Segments<MASK, U, CG> seg;
  seg.begin(a, sb);
  Records<MASK> rc;
  if (!MASK) rc.init(a, 0);

  if (warp < U::kSoftWarps) {
    // ================================================================ softmax: kParts threads per pair
    const int wg = warp >> 2, q4 = warp & 3, r = tid & 127;  // part of the columns, quarter of the lanes, lane
    const uint32_t tl = tb + (static_cast<uint32_t>(32 * q4) << 16);  // this warp's lanes
    const float sign = a.softmax_scale < 0.f ? -1.f : 1.f;
    constexpr int HB = KB / kParts;  // this thread's columns of a block
    // this thread's part of the dims, and the place of this warp's rows of it in a query tile
    constexpr int kVec = HD / kParts / 8;
    const int d0 = wg * (HD / kParts), c0 = (d0 >> 3) & 7;
    const uint32_t own_part = sb + U::kQ + (d0 >> 6) * (kTileM * 128) + 32 * q4 * 128;
    uint32_t jb = 0, meet = 0;  // blocks so far; exchanges so far of the row's threads
    bool ok = true;
    // Whether any thread of the kParts warps that share rows says so. They meet at a hardware barrier, which has
    // no time limit: so none of them ever leaves alone. One whose own wait ran out (!ok) goes on without its work
    // to the next vote or exchange, where all of them learn it and leave together.
    auto vote = [&](bool x) -> bool {
      uint32_t any;
      asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                   : "=r"(any)
                   : "r"(static_cast<uint32_t>(x)), "r"(1 + q4), "n"(32 * kParts)
                   : "memory");
      return any != 0u;
    };
    // the threads of each of the warp's rows leave a value, and take all of them in the same order
    auto exchange = [&](float mine, float (&all)[kParts]) -> bool {
      const uint32_t at = sb + U::kRow + 4 * ((meet & 1) * kParts * kTileM + r);
      sts32(at + 4 * wg * kTileM, __float_as_uint(mine));
      ok = !vote(!ok);
#pragma unroll
      for (int i = 0; i < kParts; ++i) all[i] = __uint_as_float(lds32(at + 4 * i * kTileM));
      ++meet;
      return ok;
    };
    // P V of sub-iteration n (block, tile)
    auto await_pv = [&](uint32_t n) -> bool {
      const bool done = __all_sync(0xffffffffu, bar_wait(sb + U::kPvDone + 8 * (n & 1), (n >> 1) & 1, flag));
      tmem_fence_after_sync();
      return done;
    };
    static_assert(!MASK || NT == 1, "masked segments have one tile");
    const uint32_t mask_flat = rank * kTileM + r;  // MASK: the thread's pair in the tile
    int h = 0, row0 = 0;                           // MASK: the segment's KV head and first row
    uint32_t flat0 = mask_flat, flats = pairs;     // the thread's pair in tile 0, and how many there are (MASK: of the tile's rows)
    uint4 asked[MASK ? kVec : 1];                  // MASK: query rows, as loaded
    RowRange range = {kPadRow, 0, 0, 0, 0};        // MASK: the pair's
    float slope = 0.f;
    // kVec lanes fetch the part of a row's dims that a thread has together, 32 / kVec rows at a time
    auto load_query = [&](uint32_t flat, uint4* v) {
      const bool in = flat < flats;
      const uint32_t row = in ? flat / G : 0;
      const uint16_t* src = a.q + (row0 + static_cast<int64_t>(row)) * a.q_stride + static_cast<int64_t>(in ? h * G + (flat - row * G) : 0) * HD + d0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int rr = 32 / kVec * i + lane / kVec;
        const uint64_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), rr);
        const bool there = __shfl_sync(0xffffffffu, in, rr);
        if (MASK) v[i] = load_if(reinterpret_cast<const uint4*>(at) + lane % kVec, there);
        else v[i] = there ? __ldg(reinterpret_cast<const uint4*>(at) + lane % kVec) : make_uint4(0, 0, 0, 0);
      }
    };
    bool begun = false;
    [[maybe_unused]] float next_fac = 0.f;  // MASK: the next segment's factor, and whether the warp has pairs of it
    [[maybe_unused]] bool next_in = false;
    // MASK: what a segment needs from global memory
    auto fetch = [&]() {
      if constexpr (MASK) {
        h = seg.word(kSegHead), row0 = seg.word(kSegRow0), flats = static_cast<uint32_t>(seg.word(kSegRows) * G);
        load_query(mask_flat, asked);
        range = RowRange{kPadRow, 0, 0, 0, 0}, slope = 0.f;
        if (mask_flat < flats) {
          const uint32_t row = mask_flat / G;
          if (MODE == kAdjusted && a.slopes != nullptr) slope = __ldg(a.slopes + h * G + (mask_flat - row * G));
          range = row_range(a, row0 + static_cast<int64_t>(row), false);
          if (range.lo >= range.hi) slope = 0.f;  // no bias that rises from block to block, and the reference with it
        }
      }
    };
    // state of the tile at hand; with two tiles the other one's waits in the second element
    float M[2], R[2], l[2], fac[NT];
    int E[2];
    bool warp_in[NT];
    auto other_tile = [&]() {
      if constexpr (NT == 2) {
        swap_places(M[0], M[1]), swap_places(R[0], R[1]), swap_places(l[0], l[1]), swap_places(E[0], E[1]);
        swap_places(fac[0], fac[NT - 1]), swap_places(warp_in[0], warp_in[NT - 1]);
      }
    };
    // A value as if it were new, so that what a tile's ends compute from it does not stay in registers through the block
    // loop: 2048 rows x 16 heads of 256 behind 30000 e4m3 keys 697 -> 676 us.
    auto here = [](uint32_t x) -> uint32_t {
      asm volatile("" : "+r"(x));
      return x;
    };
    // the pairs' query rows into tile t (bytes pools: fp16, pre-scaled by a power of two), a part of the dims by each of a
    // row's threads; and the factor from products to log2 units
    auto put_queries = [&](int t, uint32_t flat, float& factor) -> bool {
      const uint32_t part = here(own_part) + t * U::kQTile, lane = here(threadIdx.x & 31);
      uint4 v[kVec];
      if (!MASK) load_query(flat, v);
#pragma unroll
      for (int i = 0; MASK && i < kVec; ++i) v[i] = asked[MASK ? i : 0];
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int rr = 32 / kVec * i + lane / kVec;
        if (!F::kBytes && sign < 0.f) v[i].x ^= 0x80008000u, v[i].y ^= 0x80008000u, v[i].z ^= 0x80008000u, v[i].w ^= 0x80008000u;
        sts128(part + rr * 128 + (((c0 + lane % kVec) ^ (rr & 7)) << 4), v[i]);
      }
      float fc = fabsf(a.softmax_scale) * (MODE == kAdjusted && a.softcap > 0.f ? 1.f / a.softcap : kLog2e);
      if (F::kBytes) {
        __syncwarp();
        uint32_t mb = 0;  // largest magnitude, as bits of the 16-bit type (magnitudes order like their bits)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          v[i] = lds128(part + lane * 128 + (((c0 + i) ^ (lane & 7)) << 4));
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) mb = max(mb, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
        }
        float all[kParts];
        if (!exchange(__uint_as_float(mb), all)) return false;
#pragma unroll
        for (int i = 0; i < kParts; ++i) mb = max(mb, __float_as_uint(all[i]));
        const float m = a.q_f16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(mb))) : __uint_as_float(mb << 16);
        int e = m > 0.f ? 14 - (static_cast<int>(__float_as_uint(m) >> 23) - 127) : 0;
        e = max(-112, min(126, e));
        const float up = sign * pow2f(e);
        fc *= pow2f(-e);
        if (FMT == QKV_E4M3) fc *= a.k_scale_layer;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          float x[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = a.q_f16 ? __half22float2(*reinterpret_cast<const __half2*>(&w[k])) : make_float2(bf16lo(w[k]), bf16hi(w[k]));
            x[2 * k] = f.x * up;
            x[2 * k + 1] = f.y * up;
          }
          // int8: dims (0, 2), (1, 3) of each four, the order in which the producers store K
          v[i] = F::kInt8 ? make_uint4(pack_half2(x[0], x[2]), pack_half2(x[1], x[3]), pack_half2(x[4], x[6]), pack_half2(x[5], x[7]))
                          : make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
          sts128(part + lane * 128 + (((c0 + i) ^ (lane & 7)) << 4), v[i]);
        }
      }
      factor = fmaxf(fc, 1e-37f);  // a scale of 0: a missing key's -inf stays -inf
      return true;
    };
    auto queries_there = [&]() {
      proxy_fence();
      __syncwarp();
      if (lane == 0) lead_arrive<CG>(sb + U::kQFull);
    };
    // MASK: a chunk of 16 B of a row in the warp's place for output (eight rows' same chunk, and eight chunks in a row, are in
    // different banks), and what the warp stored there to its rows' `to` (-1: nowhere)
    constexpr int kOutChunks = U::kOutRow / 16, kOutTurn = 8 / kOutChunks;
    auto out_chunk = [&](int row, int c) -> uint32_t {
      return here(sb) + U::kOut + (32 * warp + row) * U::kOutRow + ((c ^ ((row / kOutTurn) & (kOutChunks - 1))) << 4);
    };
    auto write_rows = [&](int to, auto write) {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kOutChunks; ++k) {
        const int rr = 32 / kOutChunks * k + lane / kOutChunks;
        const int rr_to = __shfl_sync(0xffffffffu, to, rr);
        const uint4 x = lds128(out_chunk(rr, lane % kOutChunks));
        if (rr_to >= 0) write(rr_to, lane % kOutChunks, x);
      }
      __syncwarp();
    };
    // ---- the segment's partial results, or (MASK) the output of a tile that is the team's own
    auto finish = [&](int out_h, int out_row0, uint32_t out_flats, int out_part, const Odd& odd) {
#pragma unroll 1
      for (int t = 0; t < NT; ++t, other_tile()) {
        ok = ok && await_pv((jb - 1) * NT + t);
        if (!warp_in[0]) continue;
        float all[kParts];
        if (!exchange(l[0], all)) break;
        const uint32_t flat = flat0 + t * CG * kTileM;
        const bool in = flat < out_flats;
        const uint32_t row = in ? flat / G : 0;
        float sum = (all[0] + all[1]) + (all[2] + all[3]);
        if (MASK) {  // blocks that all rows with keys see whole are not masked for those without
          const uint2 lim = lds64(here(sb) + U::kTab + 16 * (here(threadIdx.x) & 127));
          if (lim.x >= lim.y) sum = 0.f;
        }
        const bool any = sum != 0.f;  // NaN too
        float inv = any ? 1.f / sum : 0.f;
        int64_t part_at = 0;
        int at = static_cast<int>(row * a.num_q_heads + out_h * G + (flat - row * G));
        if constexpr (!MASK) {
          part_at = static_cast<int64_t>(seg.part) * a.rows * a.num_q_heads;
        } else {
          if (!F::kInt8) add_odd<FMT, HD, KB>(a, odd, out_h, tl + U::kO + d0, d0, in);
          if (out_part < 0) {
            at += out_row0 * a.num_q_heads;
            if (in && wg == 0 && a.lse != nullptr) {
              float far = 0.f;
              if (MODE == kAdjusted && a.slopes != nullptr && any) {
                const RowRange x = row_range(a, out_row0 + static_cast<int64_t>(row), false);
                if (x.pos != x.near) far = -__ldg(a.slopes + out_h * G + (flat - row * G)) * fabsf(static_cast<float>(x.pos - x.near));
              }
              a.lse[at] = any ? (R[0] + log2f(sum)) * kLn2 + far : -INFINITY;
            }
            // 32 rows x 16 or 32 dims at a time, rounded, through the warp's own place: two or four lanes write 32 or 64 B of
            // a row. A thread that writes its own row touches a line of its own with each store: 3300 cycles a tile, not 1000.
            inv = any ? inv * a.merge_scale : 0.f;
            const int to = in ? at : -1;
#pragma unroll 1
            for (int c = 0; c < HD / kParts; c += 8 * kOutChunks) {
#pragma unroll 1
              for (int half = 0; half < kOutChunks / 2; ++half) {
                float o[16];
                tmem_load(tl + U::kO + d0 + c + 16 * half, o);
                tmem_loaded(o);
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  // int8: the producers store dims 0, 2, 1, 3 of each four
                  float z[4] = {o[4 * k], F::kInt8 ? o[4 * k + 2] : o[4 * k + 1], F::kInt8 ? o[4 * k + 1] : o[4 * k + 2], o[4 * k + 3]};
#pragma unroll
                  for (int n = 0; n < 4; ++n) z[n] = any ? z[n] * inv : 0.f;
                  w[2 * k] = round2(a.q_f16, z[0], z[1]), w[2 * k + 1] = round2(a.q_f16, z[2], z[3]);
                }
                sts128(out_chunk(lane, 2 * half), make_uint4(w[0], w[1], w[2], w[3]));
                sts128(out_chunk(lane, 2 * half + 1), make_uint4(w[4], w[5], w[6], w[7]));
              }
              write_rows(to, [&](int row_to, int ch, const uint4& x) {
                *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(row_to) * HD + d0 + c + 8 * ch) = x;
              });
            }
            continue;
          }
          part_at = static_cast<int64_t>(out_part) * (NT * CG * kTileM);
          at = static_cast<int>(flat);
        }
        if (in && wg == 0) a.lse_part[part_at + at] = any ? (R[0] + log2f(sum)) * kLn2 : -INFINITY;
        // 32 rows x 16 dims at a time through the warp's place in the query tile, which the segment no longer
        // needs (MASK: the warp's own place): four lanes write 64 B of a row
        const int to = in && any ? at : -1;
        const uint32_t part = own_part + t * U::kQTile;
#pragma unroll 1
        for (int c = 0; c < HD / kParts; c += 16) {
          float o[16];
          tmem_load(tl + U::kO + t * HD + d0 + c, o);
          tmem_loaded(o);
          auto four = [&](int k) {
            // int8: the producers store dims 0, 2, 1, 3 of each four
            const float x1 = F::kInt8 ? o[4 * k + 2] : o[4 * k + 1], x2 = F::kInt8 ? o[4 * k + 1] : o[4 * k + 2];
            return make_uint4(__float_as_uint(o[4 * k] * inv), __float_as_uint(x1 * inv), __float_as_uint(x2 * inv),
                              __float_as_uint(o[4 * k + 3] * inv));
          };
          if constexpr (MASK) {
#pragma unroll
            for (int k0 = 0; k0 < 4; k0 += kOutChunks) {
#pragma unroll
              for (int k = 0; k < kOutChunks; ++k) sts128(out_chunk(lane, k), four(k0 + k));
              write_rows(to, [&](int row_to, int ch, const uint4& x) {
                *reinterpret_cast<uint4*>(a.o_part + (part_at + row_to) * HD + d0 + c + 4 * (k0 + ch)) = x;
              });
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) sts128(part + lane * 128 + (((c0 + k) ^ (lane & 7)) << 4), four(k));
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rr = 8 * k + (lane >> 3) + (lane & 4);
              const int rr_to = __shfl_sync(0xffffffffu, to, rr);
              const uint4 x = lds128(part + rr * 128 + (((c0 + (lane & 3)) ^ (rr & 7)) << 4));
              if (rr_to >= 0) *reinterpret_cast<uint4*>(a.o_part + (part_at + rr_to) * HD + d0 + c + 4 * (lane & 3)) = x;
            }
            __syncwarp();
          }
        }
      }
      tmem_fence_before_sync();  // ordered before the next segment's first arrival
    };
    while (true) {
      if constexpr (MASK) {
        // the segment at hand, whose words stay until it is released
        int out_h = 0, out_row0 = 0, out_part = 0;
        uint32_t out_flats = 0;
        const uint32_t used = seg.count - 1;
        if (begun) {
          out_h = seg.word(kSegHead), out_row0 = seg.word(kSegRow0), out_part = seg.word(kSegPart);
          out_flats = static_cast<uint32_t>(seg.word(kSegRows) * G);
        }
        Odd odd = {};
        if (!F::kInt8 && begun)
          odd = Odd{plan_tiles(a, seg.word(kSegChunk)) + seg.word(kSegTile), seg.b0, seg.b1, sb + U::kOdd, sb + U::kTab + 16 * r};
        const bool more = ok && seg.next(a);
        if (seg.lost) ok = false;
        if (vote(!ok)) break;  // from here on the row's threads do the same
        // the next segment's queries first, so that its first products run under the output of the one before: prompts of
        // documents of about 700 bf16 rows 243 -> 231 us
        if (more) {
          fetch();
          next_in = __any_sync(0xffffffffu, mask_flat < flats);
          if (!put_queries(0, mask_flat, next_fac)) break;
          queries_there();
        }
        if (begun) {
          finish(out_h, out_row0, out_flats, out_part, odd);
          if (vote(!ok)) break;
          seg.release(used);
        }
        if (!more) break;
        begun = true;
        // ---- the pairs' masks: of each row once (by the first part's threads), and what all of a warp's rows see that see
        // anything
        if (wg == 0) sts128(sb + U::kTab + 16 * r, make_uint4(range.lo, range.hi, range.near, __float_as_uint(-slope * kLog2e)));
        const int lo = __reduce_max_sync(0xffffffffu, mask_flat < flats ? range.lo : 0);
        const int hi = __reduce_min_sync(0xffffffffu, range.lo < range.hi ? range.hi : INT_MAX);
        if (lane == 0) sts32(sb + U::kAll + 8 * warp, lo), sts32(sb + U::kAll + 8 * warp + 4, hi);
        __syncwarp();
        if (vote(!ok)) break;  // the table is read from here on
      } else {
        if (!seg.next(a)) break;
        h = seg.head(a);
        flat0 = (static_cast<uint32_t>(seg.tile - h * a.umma_ptiles) * NT * CG + rank) * kTileM + r;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) M[i] = -INFINITY, R[i] = 0.f, l[i] = 0.f, E[i] = F::kInt8 ? -90 : 0;
#pragma unroll
      for (int i = 0; i < NT; ++i) fac[i] = 0.f, warp_in[i] = false;
      if constexpr (!MASK) {
#pragma unroll 1
        for (int t = 0; t < NT; ++t, other_tile()) {
          const uint32_t flat = flat0 + t * CG * kTileM;
          warp_in[0] = __any_sync(0xffffffffu, flat < flats);
          if (!put_queries(t, flat, fac[0])) break;
        }
        if (!ok) break;
        queries_there();
      } else {
        fac[0] = next_fac, warp_in[0] = next_in;
      }

      int from = MASK ? (seg.b1 - 1) * KB : 0;  // MASK: the block's first position
      const uint32_t end = (jb + (seg.b1 - seg.b0)) * NT;
#pragma unroll 1
      for (uint32_t n = jb * NT; n != end; ++n) {
        const int t = NT == 2 ? n & 1 : 0;
        const uint32_t blk = n / NT, b = n & 1;
        const uint32_t sc = sb + U::kSc + (blk & (kScRing - 1)) * U::kScStage;
        if (t == 0) ok = ok && bar_wait(sb + U::kScFull + 8 * (blk & (kScRing - 1)), (blk / kScRing) & 1, flag);
        ok = ok && bar_wait(sb + U::kSFull + 8 * b, (n >> 1) & 1, flag);
        ok = __all_sync(0xffffffffu, ok);
        tmem_fence_after_sync();
        if (warp_in[0]) {  // the same in the kParts warps
          const uint4 mw = lds128(sc + U::kScMask);
          bool whole = (mw.x & mw.y & mw.z & mw.w) == 0xffffffffu;
          uint32_t seen = ~0u;  // MASK: the thread's columns that its row sees
          bool ranged = false;  // MASK: some row of the warp does not see all of the block's positions
          const int base = from + wg * HB;  // MASK: position of the thread's first column
          if (MASK) {
            const uint2 all = lds64(sb + U::kAll + 8 * (t * U::kSoftWarps + warp));
            ranged = from < static_cast<int>(all.x) || from + KB > static_cast<int>(all.y);
            whole = whole && !ranged;
            if (!whole) {
              const uint2 range = lds64(sb + U::kTab + 16 * (t * kTileM + r));
              const int lo = min(max(static_cast<int>(range.x) - base, 0), HB), hi = min(max(static_cast<int>(range.y) - base, 0), HB);
              seen = static_cast<uint32_t>((1ull << hi) - 1) & ~static_cast<uint32_t>((1ull << lo) - 1);
              seen &= lds32(sc + U::kScMask + 4 * ((wg * HB) >> 5)) >> ((wg * HB) & 31);
            }
          }
          const float4* ksp = reinterpret_cast<const float4*>(smem + (sc - smem0)) + wg * (HB / 4);
          const float4* vsp = ksp + U::kScVs / 16;
          const uint32_t ts = tl + U::kS + KB * b + wg * HB;  // this thread's columns of S, and its half of P over them
          // ---- the columns' logits (before fac) and their largest
          float x[HB];
          tmem_load(ts, x);
          tmem_loaded(x);
          if (F::kInt8) {
            // the compiler may ask for the scales early where it has registers for them: 2048 rows x 16 heads of 256 behind
            // 30000 keys 964 us, 1015 with every load at its place; capped, 4096 causal rows, 237 and 235
            if (MODE == kAdjusted) scale_by(x, sc + 4 * wg * HB);
            else scale_by(x, ksp);
          }
          float fc = fac[0];
          if (MODE == kAdjusted) {
            adjust_scores<HB>(x, fc, a.softcap, a.slopes != nullptr, sb + U::kTab + 16 * (t * kTileM + r) + 8, base);
            fc = 1.f;  // x holds the scores, in log2 units
          }
          if (__builtin_expect(!whole, 0)) mask_by(x, MASK ? seen : lds32(sc + U::kScMask + 4 * ((wg * HB) >> 5)) >> ((wg * HB) & 31));
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, all[kParts];
#pragma unroll
          for (int k = 0; k < HB; k += 2) m4[(k >> 1) & 3] = max3(m4[(k >> 1) & 3], x[k], x[k + 1]);
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          float tm = mx == -INFINITY ? mx : mx * fc;
          int En = E[0];
          if (F::kInt8) {
            uint32_t vmax = lds32(sc + U::kScVmax);
            // Of the keys that the row sees: the others' scales may be anything. (Missing keys count as 0 anyway, so that the
            // warps meet here by their rows' ranges alone, on which they agree even when a wait ran out.)
            if (MASK && ranged) {
              vmax = 0;
#pragma unroll
              for (int k = 0; k < HB; ++k)
                if ((seen >> k) & 1) vmax = max(vmax, lds32(sc + U::kScVs + 4 * (wg * HB + k)) & 0x7fffffffu);
              if (!exchange(__uint_as_float(vmax), all)) break;
#pragma unroll
              for (int k = 0; k < kParts; ++k) vmax = max(vmax, __float_as_uint(all[k]));
            }
            const int e = min(98, static_cast<int>(vmax >> 23) - 126);  // largest V scale < 2^e
            if (e > En) En = e + U::kHeadroom;
          }
          // most blocks need no more than the answer that no thread's columns pass the reference by too much
          const bool raise = vote(!ok || tm > M[0] + U::kRaise || En != E[0]);
          float f = 1.f;
          if (raise) {
            // ---- raise the reference: the sums and O so far go down by f
            if (!exchange(tm, all)) break;
            tm = fmaxf(fmaxf(all[0], all[1]), fmaxf(all[2], all[3]));
            const bool up_m = tm > M[0] + U::kRaise;  // the same for the row's threads
            const float Mn = up_m ? tm : M[0];
            const float Rn = Mn == -INFINITY ? 0.f : Mn + static_cast<float>(En) - U::kShift;
            if (F::kInt8) {
              // the reference may rise by more than fp32's exponents go down, by E alone: the sum carries E from
              // -90 to 99 and stays in range, so it is scaled in two steps (O then held V scales 2^-126 of the
              // new one's, and is lost)
              const float half = M[0] != -INFINITY ? fast_exp2(0.5f * (R[0] - Rn)) : 1.f;
              l[0] = l[0] * half * half;
              f = half * half;
            } else {
              if (M[0] != -INFINITY) f = fast_exp2(R[0] - Rn);
              l[0] *= f;
            }
            M[0] = Mn, R[0] = Rn, E[0] = En;
          }
          // ---- p = 2^(y - R), its sum, and (times the V scale) the operand
          const uint64_t fac2 = f2pack(fc, fc), ref2 = f2pack(-R[0], -R[0]);
          uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < HB; k += 2) {
            float y0, y1;
            f2unpack(f2fma(f2pack(x[k], x[k + 1]), fac2, ref2), y0, y1);
            x[k] = fast_exp2(y0);
            x[k + 1] = fast_exp2(y1);
            sum[(k >> 1) & 3] = f2add(sum[(k >> 1) & 3], f2pack(x[k], x[k + 1]));
          }
          if (F::kInt8) {
            if (MODE == kAdjusted) scale_by(x, sc + U::kScVs + 4 * wg * HB);
            else scale_by(x, vsp);  // a missing key's scale is 0
            if (MASK && !whole) {
#pragma unroll
              for (int k = 0; k < HB; ++k)
                if (!((seen >> k) & 1)) x[k] = 0.f;
            }
          }
          // Rounded once, to the 16 bits of the MMA's operands: a bf16 pool's V needs bf16 (its values pass fp16's range, and both
          // operands have one type), the others' is fp16. A weight in two such parts would take twice the P V. The sum
          // above is of the unrounded weights, whose errors are independent from key to key. Against 64 bits (root mean
          // square, relative): documents over a bf16 pool 0.0021, where rounding the output alone gives 0.0016; e4m3 with fp16
          // outputs 0.00025, 0.00021; int8 with bf16 outputs 0.0017 both.
          uint32_t p[HB / 2];
#pragma unroll
          for (int k = 0; k < HB; k += 2) p[k / 2] = F::kBf16 ? pack_bf162(x[k], x[k + 1]) : pack_half2(x[k], x[k + 1]);
          tmem_store(ts, p);
          float s0, s1;
          f2unpack(f2add(f2add(sum[0], sum[1]), f2add(sum[2], sum[3])), s0, s1);
          l[0] += s0 + s1;
          // MASK: f is 1 in a segment's first block
          if (MASK ? __any_sync(0xffffffffu, raise && f != 1.f) : raise && n >= (jb + 1) * NT) {
            // O of the blocks before, once their P V is done (with two tiles S was issued after it); last, when the
            // columns' registers are free for a part of the dims at once
            if (NT == 1) ok = await_pv(n - 1);
            const uint64_t f2 = f2pack(f, f);
            const uint32_t to = tl + U::kO + t * HD + wg * (HD / kParts);
#pragma unroll 1
            for (int c = 0; c < HD / kParts; c += 32) {
              float o[32];
              tmem_ld32(to + c, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 32; k += 2) f2scale(o + k, f2);
              tmem_st32(to + c, o);
            }
          }
          tmem_wait_st();
        }
        tmem_fence_before_sync();
        __syncwarp();
        if (ok && lane == 0) {
          lead_arrive<CG>(sb + U::kPFull + 8 * b);
          if (t == NT - 1) bar_arrive(sb + U::kScEmpty + 8 * (blk & (kScRing - 1)));
        }
        other_tile();
        if (MASK && t == NT - 1) from -= KB;
      }
      jb = end / NT;
      if constexpr (!MASK) {
        finish(h, 0, flats, 0, Odd{});
        if (vote(!ok)) break;
      }
    }
  } else if (warp < U::kRecWarp) {
    // ================================================================ producers
    using KOp = Operand<FMT, HD, U::kKRows, HD>;
    using VOp = Operand<FMT, HD, KB, U::kVDims>;
    const int pg = (warp - U::kSoftWarps) >> 2, pw = warp & 3;  // group, warp of the group
    const int voff = rank * VOp::kBytes;  // this SM's dims
    const uint32_t krow = 4 * (rank * U::kKRows + KOp::kWarpRows * pw), vrow = 4 * VOp::kWarpRows * pw;  // of a ring entry
    Rows kr, vr;
    if (F::kBytes) {
      kr = rows_of<KOp>(a.k_cache, pw, lane, rank * U::kKRows);
      vr = rows_of<VOp>(a.v_cache + voff, pw, lane, 0);
    }
    uint32_t base = 0, jb = 0;            // slots and blocks of earlier segments
    bool ok = true;
    auto await = [&](uint32_t s) -> bool {
      if (s < NS) return true;
      return __all_sync(0xffffffffu, bar_wait(sb + U::kEmpty + 8 * (s % NS), (s / NS - 1) & 1, flag));
    };
    auto hand_over = [&](uint32_t s) {
      proxy_fence();
      __syncwarp();
      if (lane == 0) lead_arrive<CG>(sb + U::kFull + 8 * (s % NS));
    };
    while (ok && seg.next(a)) {
      const int B = seg.b1 - seg.b0;
      int all_lo = 0, all_hi = 0;
      if constexpr (MASK) all_lo = seg.word(kSegAllLo), all_hi = seg.word(kSegAllHi);
      // MASK: whether some row of the tile does not see slot e's block whole; values that are not finite are left out then
      auto in_part = [&](int e, auto is_v, auto block_of) -> bool {
        if constexpr (MASK) {
          if (F::kInt8 || !is_v(e)) return false;
          const int p = (seg.b1 - 1 - block_of(e)) * KB;
          return p < all_lo || p + KB > all_hi;
        }
        return false;
      };
      // what the segment's slot e holds
      auto is_v = [&](int e) -> bool { return e == 2 * B - 1 || (e > 0 && !(e & 1)); };
      auto block_of = [&](int e) -> int { return is_v(e) ? (e == 2 * B - 1 ? B - 1 : e / 2 - 1) : (e + 1) / 2; };
      // the records of slot e's block, awaited; each group takes a block's once for K and once for V
      uint32_t rec = 0;
      auto await_records = [&](int e) -> bool {
        const uint32_t n = jb + block_of(e);
        rec = sb + U::kRec + (n % kRecRing) * 4 * KB;
        return __all_sync(0xffffffffu, bar_wait(sb + U::kRecFull + 8 * (n % kRecRing), (n / kRecRing) & 1, flag));
      };
      auto free_records = [&](int e) {
        __syncwarp();
        if (lane == 0) bar_arrive(sb + U::kRecEmpty + 8 * ((jb + block_of(e)) % kRecRing));
      };
      if (F::kBytes) {
        static_assert(KOp::kInstr == VOp::kInstr, "one code for both");
        constexpr int N = KOp::kInstr;
        uint4 raw[N];
        auto load = [&](int e) -> bool {
          if (e >= 2 * B) return true;
          if (!await_records(e)) return false;
          load_rows<FMT, HD, N>(raw, is_v(e) ? vr : kr, rec);
          free_records(e);
          return true;
        };
        ok = load(pg);
#pragma unroll 1
        for (int e = pg; ok && e < 2 * B; e += 2) {
          const uint32_t n = base + e;
          if (!(ok = await(n))) break;
          if (MASK && FMT == QKV_E4M3 && in_part(e, is_v, block_of)) {
            uint32_t odd = 0;
#pragma unroll
            for (int u = 0; u < N; ++u) odd |= drop_odd_e4m3(raw[u]);
            if (odd) note_odd<CG>(sb + U::kOdd, seg.b1 - 1 - block_of(e));
          }
          convert_rows<FMT, N>(sb + U::kRing + (n % NS) * U::kSlotBytes, is_v(e) ? vr : kr, raw);
          hand_over(n);
          ok = load(e + 2);
        }
      } else {
        // A slot is handed over when its copies have arrived; with a ring of five or more after those of the group's next
        // one have been asked for -- unless that one's place is still taken: what frees it may be waiting for this slot.
        // bf16, us, at once | one ahead: 2048 rows behind 30000 keys, 32 heads of 128 (eight slots) 1224 | 1097, 16 heads
        // of 256 (four slots) 743 | 807; 64 x 4 rows x 64 heads of 128 behind 8000 (five slots) 437 | 403. The shared prefix
        // (eight slots): 16 rows x 64 heads of 128 behind 32768 keys 42.1 | 40.0, 32 rows behind 16384 37.0 | 38.6, 256 rows x 32
        // heads behind 32768 137.5 | 138.1.
        constexpr bool kOneAhead = NS >= 5;
        int last = -1;  // the slot whose copies are on their way
        auto arrived = [&](int e) {
          const uint32_t n = base + e;
          if (MASK && in_part(e, is_v, block_of) && VOp::template drop_odd<F::kBf16>(sb + U::kRing + (n % NS) * U::kSlotBytes, pw, lane))
            note_odd<CG>(sb + U::kOdd, seg.b1 - 1 - block_of(e));
          hand_over(n);
        };
        for (int e = pg; ok && e < 2 * B; e += 2) {
          const uint32_t n = base + e, slot = sb + U::kRing + (n % NS) * U::kSlotBytes;
          const bool ahead = kOneAhead && (n < NS || __all_sync(0xffffffffu, bar_test(sb + U::kEmpty + 8 * (n % NS), (n / NS - 1) & 1)));
          if (last >= 0 && !ahead) {
            cp_async_wait<0>();
            arrived(last);
            last = -1;
          }
          if (!(ok = await_records(e)) || !(ok = await(n))) break;
          if (is_v(e)) VOp::copy(slot, a.v_cache, pw, lane, rec + vrow, voff);
          else KOp::copy(slot, a.k_cache, pw, lane, rec + krow, 0);
          free_records(e);
          cp_async_commit();
          if (last >= 0) {
            cp_async_wait<1>();
            arrived(last);
          }
          last = e;
        }
        cp_async_wait<0>();
        if (ok && last >= 0) arrived(last);
      }
      base += 2 * B;
      jb += B;
      seg.done();
    }
  } else if (warp == U::kRecWarp) {
    // ================================================================ records
    if (MASK) rc.init(a, 0);
    uint32_t jb = 0;
    bool ok = true;
    [[maybe_unused]] MaskedWalk walk;
    if constexpr (MASK) {
      walk.begin(a, blockIdx.x / CG);
      if (lane == 0 && rank == 0) *reinterpret_cast<int4*>(plan_join(a, walk.team)) = make_int4(0, 0, 0, 0);
    }
    auto next_segment = [&]() -> bool {
      if constexpr (MASK) {
        if (!publish<KB, CG, U>(a, walk, sb, seg.count)) return false;
        seg.take();
        return true;
      } else {
        return seg.next(a);
      }
    };
    while (ok && next_segment()) {
      rc.h = seg.head(a);
      if constexpr (MASK) rc.of_tile(a, plan_tiles(a, seg.word(kSegChunk))[seg.word(kSegTile)]);
      int blk[KB / 32];
#pragma unroll
      for (int i = 0; i < KB / 32; ++i) blk[i] = rc.lookup((MASK ? seg.b1 - 1 : seg.b0) * KB + 32 * i + lane);
      for (int j = seg.b0; j < seg.b1; ++j, ++jb) {
        const uint32_t n = jb % kRecRing;
        int rec[KB / 32];
#pragma unroll
        for (int i = 0; i < KB / 32; ++i) {
          const int p = (MASK ? seg.b1 - 1 - (j - seg.b0) : j) * KB + 32 * i + lane;
          rec[i] = rc.record(p, blk[i]);
          if constexpr (MASK) {
            if (rec[i] < 0 && rc.in(p) && a.dev_status != nullptr) {
              const int row = seg.word(kSegRow0);
              flag_if_seen(a.row_start != nullptr ? a.row_start + row : nullptr, a.row_len + row, a.row_pos != nullptr ? a.row_pos + row : nullptr,
                           a.window, a.max_row_len, seg.word(kSegRows), p, a.dev_status);
            }
          } else {
            if (rec[i] < 0 && p < a.prefix_len && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_INDEX);
          }
          blk[i] = j + 1 < seg.b1 ? rc.lookup(MASK ? p - KB : p + KB) : -1;  // the next block's, a block ahead of its use
        }
        if (jb >= kRecRing) {
          ok = __all_sync(0xffffffffu, bar_wait(sb + U::kRecEmpty + 8 * n, (jb / kRecRing - 1) & 1, flag));
          if (!ok) break;
        }
#pragma unroll
        for (int i = 0; i < KB / 32; ++i) sts32(sb + U::kRec + n * 4 * KB + 4 * (32 * i + lane), static_cast<uint32_t>(rec[i]));
        __syncwarp();
        if (lane == 0 && jb != a.umma_drop) bar_arrive(sb + U::kRecFull + 8 * n);
      }
    }
  } else if (warp == U::kScWarp) {
    // ================================================================ scales and masks
    uint32_t jb = 0;
    bool ok = true;
    while (ok && seg.next(a)) {
      for (int j = seg.b0; j < seg.b1; ++j, ++jb) {
        const uint32_t n = jb & (kScRing - 1), sc = sb + U::kSc + n * U::kScStage, rn = jb % kRecRing;
        float ks[KB / 32], vs[KB / 32];
        uint32_t mask[4] = {~0u, ~0u, ~0u, ~0u}, vmax = 0;  // words past the block count as whole
        ok = __all_sync(0xffffffffu, bar_wait(sb + U::kRecFull + 8 * rn, (jb / kRecRing) & 1, flag));
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < KB / 32; ++i) {
          const int rec = static_cast<int>(lds32(sb + U::kRec + rn * 4 * KB + 4 * (32 * i + lane)));
          mask[i] = __ballot_sync(0xffffffffu, rec >= 0);
          ks[i] = vs[i] = 0.f;
          if (F::kInt8 && rec >= 0) {
            if (F::kInline) {
              const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(rec)) * (HD + 4) + HD;
              ks[i] = __ldg(reinterpret_cast<const float*>(a.k_cache + off));
              vs[i] = __ldg(reinterpret_cast<const float*>(a.v_cache + off));
            } else {
              ks[i] = __ldg(a.k_scale_tok + rec);
              vs[i] = __ldg(a.v_scale_tok + rec);
            }
          }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(sb + U::kRecEmpty + 8 * rn);
        if (jb >= kScRing) {
          ok = __all_sync(0xffffffffu, bar_wait(sb + U::kScEmpty + 8 * n, (jb / kScRing - 1) & 1, flag));
          if (!ok) break;
        }
        if (F::kInt8) {
#pragma unroll
          for (int i = 0; i < KB / 32; ++i) {
            sts32(sc + 4 * (32 * i + lane), __float_as_uint(ks[i]));
            sts32(sc + U::kScVs + 4 * (32 * i + lane), __float_as_uint(vs[i]));
            vmax = max(vmax, __float_as_uint(vs[i]) & 0x7fffffffu);  // magnitudes: bits order like values
          }
          vmax = __reduce_max_sync(0xffffffffu, vmax);
        }
        if (lane == 0) {
          sts128(sc + U::kScMask, make_uint4(mask[0], mask[1], mask[2], mask[3]));
          sts32(sc + U::kScVmax, vmax);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(sb + U::kScFull + 8 * n);
      }
      seg.done();
    }
  } else if (rank == 0) {
    // ================================================================ MMA issuer
    uint32_t base = 0, jb = 0, segs = 0;
    bool ok = true;
    const uint32_t lead = elect_one();
    const uint32_t tu = __shfl_sync(0xffffffffu, tb, 0);  // warp-uniform
    // This warp's path from a barrier to the next MMA is part of every block: what is probably there already (a slot's
    // values) is awaited first, ahead of what the tensor cores and the softmax have just been asked for. All lanes agree on
    // every wait: with each lane's own answer the descriptors leave the uniform registers (256 rows x 16 heads behind 65536
    // int8 keys 235 -> 250 us).
    auto wait = [&](uint32_t bar, uint32_t ph) -> bool { return __all_sync(0xffffffffu, bar_wait(bar, ph, flag)); };
    auto await_full = [&](uint32_t s) -> bool { return wait(sb + U::kFull + 8 * (s % NS), (s / NS) & 1); };
    // S of sub-iteration n (of tile t) into its buffer, from the K slot s (awaited by the first tile, freed by the
    // last). The buffer holds P of sub-iteration n - 2. MMAs are only sure to run in the order of their issue where
    // they have the same shape and accumulator, which S and O are not, so that P V has to be over first.
    auto qk = [&](int t, uint32_t n, uint32_t s) {
      const uint32_t b = n & 1;
      if (t == 0 && !(ok = await_full(s))) return;
      if (n >= 2 && !(ok = wait(sb + U::kPvDone + 8 * b, ((n >> 1) - 1) & 1))) return;
      tmem_fence_after_sync();
      const uint32_t d = tu + U::kS + KB * b;
      const uint64_t qd = sw128_desc(sb + U::kQ + t * U::kQTile, 16, 1024);
      const uint64_t kd = sw128_desc(sb + U::kRing + (s % NS) * U::kSlotBytes, 16, 1024);
#pragma unroll
      for (int ks = 0; ks < HD / 16; ++ks)  // 64 dims are one column of 128 B rows
        mma_ss<CG>(d, qd + (ks >> 2) * ((kTileM * 128) >> 4) + 2 * (ks & 3), kd + (ks >> 2) * ((U::kKRows * 128) >> 4) + 2 * (ks & 3),
                   U::kIdS, ks > 0 ? 1u : 0u, lead);
      if (lead) {
        if (t == NT - 1) commit_to<CG>(sb + U::kEmpty + 8 * (s % NS));
        commit_to<CG>(sb + U::kSFull + 8 * b);
      }
      __syncwarp();
    };
    // O of tile t += P (in buffer b) times the V slot s
    auto pv = [&](int t, uint32_t b, uint32_t ph, uint32_t s, bool first) {
      if (t == 0 && !(ok = await_full(s))) return;
      if (!(ok = wait(sb + U::kPFull + 8 * b, ph))) return;
      tmem_fence_after_sync();
      constexpr int kPer = KB / kParts / 16;  // 16 keys a step
      const uint32_t d = tu + U::kO + t * HD, p = tu + U::kS + KB * b;
      const uint64_t vd = sw128_desc(sb + U::kRing + (s % NS) * U::kSlotBytes, KB * 128, 1024);
#pragma unroll
      for (int ks = 0; ks < KB / 16; ++ks)  // each part of the keys' P lies over its S
        mma_ts<CG>(d, p + (ks / kPer) * (KB / kParts) + 8 * (ks % kPer), vd + 128 * ks, U::kIdO, !first || ks > 0 ? 1u : 0u, lead);
      if (lead) {
        if (t == NT - 1) commit_to<CG>(sb + U::kEmpty + 8 * (s % NS));
        commit_to<CG>(sb + U::kPvDone + 8 * b);
      }
      __syncwarp();
    };
    while (ok && seg.next(a)) {
      const int B = seg.b1 - seg.b0;
      ok = wait(sb + U::kQFull, segs & 1);
      ++segs;
      // two tiles: P V of block j of a tile, then its S of block j + 1; one tile: S of block j + 1, then P V of j
#pragma unroll 1
      for (int j = -1; ok && j < B; ++j) {
        const uint32_t n = jb + j;
        if constexpr (NT == 1) {
          if (j + 1 < B) qk(0, n + 1, base + k_slot(j + 1));
          if (ok && j >= 0) pv(0, n & 1, (n >> 1) & 1, base + v_slot(j, B), j == 0);
        } else {
#pragma unroll 1
          for (int t = 0; ok && t < NT; ++t) {
            if (j >= 0) pv(t, (n * NT + t) & 1, ((n * NT + t) >> 1) & 1, base + v_slot(j, B), j == 0);
            if (ok && j + 1 < B) qk(t, (n + 1) * NT + t, base + k_slot(j + 1));
          }
        }
      }
      jb += B;
      base += 2 * B;
      seg.done();
    }
    if (lead) commit_to<CG>(sb + U::kDrain);
    __syncwarp();
  }
  __syncwarp();
  tmem_fence_before_sync();
  __syncthreads();
  // Nothing may still write tensor memory, read a slot or arrive on a barrier when the team leaves. (After the others are
  // done: the second SM's MMA warp has nothing to do until here, and a call may be longer than a wait's limit.)
  if (warp == U::kMmaWarp && lane == 0) bar_wait(sb + U::kDrain, 0, flag, false);
  __syncwarp();
  team_sync<CG>();
  tmem_fence_after_sync();
  if (warp == U::kMmaWarp) team_tmem_dealloc<CG>(tb);
  if (tid == 0 && lds32(flag) != 0u && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_TIMEOUT);
}

template <int FMT, int HD, int NT, int CG, int MODE>
cudaError_t launch_umma(const PrefixArgs& a, cudaStream_t stream) {
  using U = Umma<FMT, HD, NT, CG, MODE != kPrefix>;
  auto kern = prefix_umma_kernel<FMT, HD, NT, CG, MODE>;
  static std::atomic<bool> done[64] = {};
  cudaError_t e = allow_smem(kern, U::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.umma_teams * CG));
  cfg.blockDim = dim3(U::kThreads);
  cfg.dynamicSmemBytes = U::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  cfg.attrs = at;
  cfg.numAttrs = 0;
  if (CG > 1) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
  }
  if (MODE != kPrefix) {  // starts while the work list is made
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int FMT, int MODE = kPrefix>
cudaError_t launch_umma(PrefixArgs a, cudaStream_t stream) {
  // Test of the lost-wait path: QKV_TEST_PREFIX_DROP_HANDOFF=<block> makes the records' warp leave out the hand-off of
  // that block in each CTA (read at each launch; unset in any other use).
  if (const char* t = std::getenv("QKV_TEST_PREFIX_DROP_HANDOFF")) {
    char* end = nullptr;
    const long n = std::strtol(t, &end, 10);
    if (end != t && n >= 0 && n < (1 << 30)) a.umma_drop = static_cast<uint32_t>(n);
  }
  if (a.head_dim == 256) return a.umma_cg == 2 ? launch_umma<FMT, 256, 1, 2, MODE>(a, stream) : launch_umma<FMT, 256, 1, 1, MODE>(a, stream);
  // masked: one tile of 256 pairs, not two: half of the work at a tile's ends, and no second tile's state
  if (a.umma_cg == 2) return launch_umma<FMT, 128, MODE == kPrefix ? 2 : 1, 2, MODE>(a, stream);
  return launch_umma<FMT, 128, 1, 1, MODE>(a, stream);
}

template <int FMT>
cudaError_t launch_masked_umma(const PrefixArgs& a, cudaStream_t stream) {
  return a.softcap > 0.f || a.slopes != nullptr ? launch_umma<FMT, kAdjusted>(a, stream) : launch_umma<FMT, kMasked>(a, stream);
}

}  // namespace prefix
}  // namespace qkv
