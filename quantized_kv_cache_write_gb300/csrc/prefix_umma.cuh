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
// producers, one for the records, one for the scales, one MMA issuer (of the team's first SM). Slots
// (rows of 128 B, 128 B swizzle) pass from the producers to the MMA warp in the order
// K_0 K_1 V_0 K_2 V_1 ..., one group every second one; K is K-major, V MN-major, and both are stored alike, one
// 128 B row per key and 64 dims.
//   records: block list -> record numbers of a block's keys, into a ring, eight blocks ahead.
//   producers: 16 B loads into registers, converted to fp16 (codes are exact) and stored to the slot once it is
//     free; then the registers take the group's next slot. 16-bit pools are copied straight into the slot
//     (cp.async).
//   scales: K and V scales, the mask of the block's keys and the largest V scale into a small ring.
//   MMA: one thread. P is the A operand in tensor memory, in the columns of the S it was made from.
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

#include "prefix_attn.cuh"

namespace qkv {
namespace prefix {

constexpr int kTileM = 128;  // pairs of a tile on one SM
constexpr int kProdWarps = 4;  // of a group; two groups
constexpr int kParts = 4;      // threads of a pair: each takes a part of a block's columns
constexpr uint64_t kWaitNs = 2000000000;  // after which a wait is declared lost
constexpr int kScRing = 4, kRecRing = 8;
// keys of a block: 128; 64 where one SM holds 256-wide heads alone
constexpr int umma_block_keys(int head_dim, int cg) { return head_dim == 256 && cg == 1 ? 64 : 128; }

template <int FMT, int HD, int NT, int CG>
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
  static constexpr uint32_t kBar = kRow + 2 * kParts * 4 * kTileM;
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
__device__ __forceinline__ void mask_by(float (&v)[N], uint32_t mask) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (!((mask >> k) & 1)) v[k] = -INFINITY;
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
struct Records {
  const int32_t* blocks;
  int64_t num_slots;
  int bsz, shift, len, H, h;
  bool pow2;
  __device__ __forceinline__ int block_of(int p) const { return pow2 ? p >> shift : p / bsz; }
  // block id of position p, -1 past the prefix
  __device__ __forceinline__ int lookup(int p) const { return p < len ? __ldg(blocks + block_of(p)) : -1; }
  // record of position p in block blk, -1: none
  __device__ __forceinline__ int record(int p, int blk) const {
    const int64_t slot = static_cast<int64_t>(blk) * bsz + (p - block_of(p) * bsz);
    return (p < len && blk >= 0 && slot < num_slots) ? static_cast<int>(slot) * H + h : -1;
  }
};

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

template <int FMT, int HD, int NT, int CG>
__global__ void __launch_bounds__(Umma<FMT, HD, NT, CG>::kThreads, 1) prefix_umma_kernel(const PrefixArgs a) {
  using F = Fmt<FMT>;
  using U = Umma<FMT, HD, NT, CG>;
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
      bar_init(sb + U::kDrain, 1);
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
      sts32(flag, 0u);
    }
    __syncwarp();
  }
  tmem_fence_before_sync();
  __syncthreads();
  team_sync<CG>();
  tmem_fence_after_sync();
  const uint32_t tb = lds32(sb + U::kTmemSlot);
  Segment seg = first_segment<CG>(a);
  Records rc;
  rc.blocks = a.prefix_blocks, rc.num_slots = a.num_slots, rc.bsz = a.block_size, rc.len = a.prefix_len, rc.H = H;
  rc.pow2 = (rc.bsz & (rc.bsz - 1)) == 0, rc.shift = __ffs(rc.bsz) - 1;

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
    while (seg.next(a)) {
      const int h = seg.tile / a.umma_ptiles;
      const uint32_t flat0 = (static_cast<uint32_t>(seg.tile - h * a.umma_ptiles) * NT * CG + rank) * kTileM + r;
      // state of the tile at hand; with two tiles the other one's waits in the second element
      float M[2] = {-INFINITY, -INFINITY}, R[2] = {0.f, 0.f}, l[2] = {0.f, 0.f}, fac[NT] = {};
      int E[2] = {F::kInt8 ? -90 : 0, F::kInt8 ? -90 : 0};
      bool warp_in[NT] = {};
      auto other_tile = [&]() {
        if (NT == 2) {
          float x;
          x = M[0], M[0] = M[1], M[1] = x;
          x = R[0], R[0] = R[1], R[1] = x;
          x = l[0], l[0] = l[1], l[1] = x;
          x = fac[0], fac[0] = fac[NT - 1], fac[NT - 1] = x;
          const int e = E[0];
          E[0] = E[1], E[1] = e;
          const bool w = warp_in[0];
          warp_in[0] = warp_in[NT - 1], warp_in[NT - 1] = w;
        }
      };
      // ---- the pairs' query rows into the tiles (bytes pools: fp16, pre-scaled by a power of two), a part of the
      // dims by each of a row's threads; kVec lanes fetch a row's part together, 32 / kVec rows at a time
#pragma unroll 1
      for (int t = 0; t < NT; ++t, other_tile()) {
        const uint32_t flat = flat0 + t * CG * kTileM;
        const bool in = flat < pairs;
        const uint32_t row = in ? flat / G : 0;
        warp_in[0] = __any_sync(0xffffffffu, in);
        const uint16_t* src = a.q + row * a.q_stride + static_cast<int64_t>(in ? h * G + (flat - row * G) : 0) * HD + d0;
        const uint32_t part = own_part + t * U::kQTile;
        uint4 v[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int rr = 32 / kVec * i + lane / kVec;
          const uint64_t from = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), rr);
          const bool there = __shfl_sync(0xffffffffu, in, rr);
          v[i] = there ? __ldg(reinterpret_cast<const uint4*>(from) + lane % kVec) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int rr = 32 / kVec * i + lane / kVec;
          if (!F::kBytes && sign < 0.f) v[i].x ^= 0x80008000u, v[i].y ^= 0x80008000u, v[i].z ^= 0x80008000u, v[i].w ^= 0x80008000u;
          sts128(part + rr * 128 + (((c0 + lane % kVec) ^ (rr & 7)) << 4), v[i]);
        }
        float fc = fabsf(a.softmax_scale) * kLog2e;
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
          if (!exchange(__uint_as_float(mb), all)) break;
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
        fac[0] = fmaxf(fc, 1e-37f);  // a scale of 0: a missing key's -inf stays -inf
      }
      if (!ok) break;
      proxy_fence();
      __syncwarp();
      if (lane == 0) lead_arrive<CG>(sb + U::kQFull);

      const int subs = (seg.b1 - seg.b0) * NT;
#pragma unroll 1
      for (int i = 0; i < subs; ++i) {
        const int t = NT == 2 ? i & 1 : 0;
        const uint32_t blk = jb + i / NT, n = jb * NT + i, b = n & 1;
        const uint32_t sc = sb + U::kSc + (blk & (kScRing - 1)) * U::kScStage;
        if (t == 0) ok = ok && bar_wait(sb + U::kScFull + 8 * (blk & (kScRing - 1)), (blk / kScRing) & 1, flag);
        ok = ok && bar_wait(sb + U::kSFull + 8 * b, (n >> 1) & 1, flag);
        ok = __all_sync(0xffffffffu, ok);
        tmem_fence_after_sync();
        if (warp_in[0]) {  // the same in the kParts warps
          const uint4 mw = lds128(sc + U::kScMask);
          const bool whole = (mw.x & mw.y & mw.z & mw.w) == 0xffffffffu;
          const float4* ksp = reinterpret_cast<const float4*>(smem + (sc - smem0)) + wg * (HB / 4);
          const float4* vsp = ksp + U::kScVs / 16;
          const uint32_t ts = tl + U::kS + KB * b + wg * HB;  // this thread's columns of S, and its half of P over them
          // ---- the columns' logits (before fac) and their largest
          float x[HB];
          tmem_load(ts, x);
          tmem_loaded(x);
          if (F::kInt8) scale_by(x, ksp);
          if (__builtin_expect(!whole, 0)) mask_by(x, lds32(sc + U::kScMask + 4 * ((wg * HB) >> 5)) >> ((wg * HB) & 31));
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, all[kParts];
#pragma unroll
          for (int k = 0; k < HB; k += 2) m4[(k >> 1) & 3] = max3(m4[(k >> 1) & 3], x[k], x[k + 1]);
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          float tm = mx == -INFINITY ? mx : mx * fac[0];
          int En = E[0];
          if (F::kInt8) {
            const int e = min(98, static_cast<int>(lds32(sc + U::kScVmax) >> 23) - 126);  // largest V scale < 2^e
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
          const uint64_t fac2 = f2pack(fac[0], fac[0]), ref2 = f2pack(-R[0], -R[0]);
          uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < HB; k += 2) {
            float y0, y1;
            f2unpack(f2fma(f2pack(x[k], x[k + 1]), fac2, ref2), y0, y1);
            x[k] = fast_exp2(y0);
            x[k + 1] = fast_exp2(y1);
            sum[(k >> 1) & 3] = f2add(sum[(k >> 1) & 3], f2pack(x[k], x[k + 1]));
          }
          if (F::kInt8) scale_by(x, vsp);  // a masked key's scale is 0
          uint32_t p[HB / 2];
#pragma unroll
          for (int k = 0; k < HB; k += 2) p[k / 2] = F::kBf16 ? pack_bf162(x[k], x[k + 1]) : pack_half2(x[k], x[k + 1]);
          tmem_store(ts, p);
          float s0, s1;
          f2unpack(f2add(f2add(sum[0], sum[1]), f2add(sum[2], sum[3])), s0, s1);
          l[0] += s0 + s1;
          if (raise && i >= NT) {
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
      }
      jb += seg.b1 - seg.b0;
      // ---- the segment's partial results
#pragma unroll 1
      for (int t = 0; t < NT; ++t, other_tile()) {
        ok = ok && await_pv((jb - 1) * NT + t);
        if (!warp_in[0]) continue;
        float all[kParts];
        if (!exchange(l[0], all)) break;
        const uint32_t flat = flat0 + t * CG * kTileM;
        const bool in = flat < pairs;
        const uint32_t row = in ? flat / G : 0;
        const float sum = (all[0] + all[1]) + (all[2] + all[3]);
        const bool any = sum != 0.f;  // NaN too
        const float inv = any ? 1.f / sum : 0.f;
        const int64_t part_at = static_cast<int64_t>(seg.part) * a.rows * a.num_q_heads;
        const int at = static_cast<int>(row * a.num_q_heads + h * G + (flat - row * G));
        if (in && wg == 0) a.lse_part[part_at + at] = any ? (R[0] + log2f(sum)) * kLn2 : -INFINITY;
        // 32 rows x 16 dims at a time through the warp's place in the query tile, which the segment no longer
        // needs: four lanes write 64 B of a row
        const int to = in && any ? at : -1;
        const uint32_t part = own_part + t * U::kQTile;
#pragma unroll 1
        for (int c = 0; c < HD / kParts; c += 16) {
          float o[16];
          tmem_load(tl + U::kO + t * HD + d0 + c, o);
          tmem_loaded(o);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // int8: the producers store dims 0, 2, 1, 3 of each four
            const float x1 = F::kInt8 ? o[4 * k + 2] : o[4 * k + 1], x2 = F::kInt8 ? o[4 * k + 1] : o[4 * k + 2];
            sts128(part + lane * 128 + (((c0 + k) ^ (lane & 7)) << 4),
                   make_uint4(__float_as_uint(o[4 * k] * inv), __float_as_uint(x1 * inv), __float_as_uint(x2 * inv),
                              __float_as_uint(o[4 * k + 3] * inv)));
          }
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
      tmem_fence_before_sync();  // ordered before the next segment's first arrival
      if (vote(!ok)) break;
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
          convert_rows<FMT, N>(sb + U::kRing + (n % NS) * U::kSlotBytes, is_v(e) ? vr : kr, raw);
          hand_over(n);
          ok = load(e + 2);
        }
      } else {
        for (int e = pg; ok && e < 2 * B; e += 2) {
          const uint32_t n = base + e, slot = sb + U::kRing + (n % NS) * U::kSlotBytes;
          if (!(ok = await_records(e)) || !(ok = await(n))) break;
          if (is_v(e)) VOp::copy(slot, a.v_cache, pw, lane, rec + vrow, voff);
          else KOp::copy(slot, a.k_cache, pw, lane, rec + krow, 0);
          free_records(e);
          cp_async_commit();
          cp_async_wait<0>();
          hand_over(n);
        }
      }
      base += 2 * B;
      jb += B;
    }
  } else if (warp == U::kRecWarp) {
    // ================================================================ records
    uint32_t jb = 0;
    bool ok = true;
    while (ok && seg.next(a)) {
      rc.h = seg.tile / a.umma_ptiles;
      int blk[KB / 32];
#pragma unroll
      for (int i = 0; i < KB / 32; ++i) blk[i] = rc.lookup(seg.b0 * KB + 32 * i + lane);
      for (int j = seg.b0; j < seg.b1; ++j, ++jb) {
        const uint32_t n = jb % kRecRing;
        int rec[KB / 32];
#pragma unroll
        for (int i = 0; i < KB / 32; ++i) {
          const int p = j * KB + 32 * i + lane;
          rec[i] = rc.record(p, blk[i]);
          if (rec[i] < 0 && p < a.prefix_len && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_INDEX);
          blk[i] = j + 1 < seg.b1 ? rc.lookup(p + KB) : -1;  // the next block's, a block ahead of its use
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
    }
  } else if (rank == 0) {
    // ================================================================ MMA issuer
    uint32_t base = 0, jb = 0, segs = 0;
    bool ok = true;
    const uint32_t lead = elect_one();
    const uint32_t tu = __shfl_sync(0xffffffffu, tb, 0);  // warp-uniform
    auto wait = [&](uint32_t bar, uint32_t ph) -> bool { return __all_sync(0xffffffffu, bar_wait(bar, ph, flag)); };
    auto await_full = [&](uint32_t s) -> bool { return wait(sb + U::kFull + 8 * (s % NS), (s / NS) & 1); };
    // S of sub-iteration n (of tile t) into its buffer, from the K slot s (awaited by the first tile, freed by the
    // last). The buffer holds P of sub-iteration n - 2. MMAs are only sure to run in the order of their issue where
    // they have the same shape and accumulator, which S and O are not, so that P V has to be over first.
    auto qk = [&](int t, uint32_t n, uint32_t s) {
      const uint32_t b = n & 1;
      if (n >= 2 && !(ok = wait(sb + U::kPvDone + 8 * b, ((n >> 1) - 1) & 1))) return;
      if (t == 0 && !(ok = await_full(s))) return;
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
      if (!(ok = wait(sb + U::kPFull + 8 * b, ph))) return;
      if (t == 0 && !(ok = await_full(s))) return;
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
#pragma unroll 1
        for (int i = 0; ok && i < 2; ++i) {
          const int t = NT == 2 ? i : 0;
          if (j >= 0 && (NT == 2 || i == 1))
            pv(t, (n * NT + t) & 1, ((n * NT + t) >> 1) & 1, base + v_slot(j, B), j == 0);
          if (ok && j + 1 < B && (NT == 2 || i == 0)) qk(t, (n + 1) * NT + t, base + k_slot(j + 1));
        }
      }
      jb += B;
      base += 2 * B;
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

template <int FMT, int HD, int NT, int CG>
cudaError_t launch_umma(const PrefixArgs& a, cudaStream_t stream) {
  using U = Umma<FMT, HD, NT, CG>;
  auto kern = prefix_umma_kernel<FMT, HD, NT, CG>;
  static std::atomic<bool> done[64] = {};
  cudaError_t e = allow_smem(kern, U::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.umma_teams * CG));
  cfg.blockDim = dim3(U::kThreads);
  cfg.dynamicSmemBytes = U::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CG;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CG > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int FMT>
cudaError_t launch_umma(PrefixArgs a, cudaStream_t stream) {
  // Test of the lost-wait path: QKV_TEST_PREFIX_DROP_HANDOFF=<block> makes the records' warp leave out the hand-off of
  // that block in each CTA (read at each launch; unset in any other use).
  if (const char* t = std::getenv("QKV_TEST_PREFIX_DROP_HANDOFF")) {
    char* end = nullptr;
    const long n = std::strtol(t, &end, 10);
    if (end != t && n >= 0 && n < (1 << 30)) a.umma_drop = static_cast<uint32_t>(n);
  }
  if (a.head_dim == 256) return a.umma_cg == 2 ? launch_umma<FMT, 256, 1, 2>(a, stream) : launch_umma<FMT, 256, 1, 1>(a, stream);
  if (a.umma_cg == 2) return launch_umma<FMT, 128, 2, 2>(a, stream);
  return launch_umma<FMT, 128, 1, 1>(a, stream);
}

}  // namespace prefix
}  // namespace qkv
