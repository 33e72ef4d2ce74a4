// Dense decode attention over a paged pool for a batch whose sequences share a prefix: the part of
// the work that runs on mma.sync tiles of 16 or 8 (row, query head) pairs.
//
// For row r, query head h and the keys j the row sees (positions 0 .. row_len - 1 of its sequence;
// those below prefix_len through the shared block list, the others through its own table row):
//   y_j = log2(e) scale q . K_j,  o = sum_j 2^(y_j - M) V_j / sum_j 2^(y_j - M),  lse = ln 2 (M + log2 sum)
// in one pass over the keys with a running reference M and sum per pair; M is raised (and the
// accumulators rescaled) only when a logit exceeds it by 2^8, so p <= 2^8.
//
// A CTA of four warps takes one tile of pairs, one KV head and one range of keys, either of the shared
// prefix (pairs taken across rows, row-major, so every key that is read serves 16 pairs of whatever
// rows) or of the keys behind it (pairs of consecutive rows of one sequence); one launch holds both kinds.
// Each warp streams its own key tiles through a cp.async ring; warps meet once, at the end, to join
// their sums. Tiles start at positions that are multiples of their size, so where blocks are such
// multiples too a tile is one run of slots and costs one table lookup. Quantised pools are multiplied
// in fp16: codes are exact fp16 values, the query is pre-scaled by a power of two into fp16 (its largest
// value between 2^14 and 2^15, so that bf16 values lose bits from 2^-31 of it on and fp16 values from 2^-28; both
// vanish below 2^-39), the K scale multiplies the logit, the V scale p. p (times the V
// scale and a power of two) is rounded to the 16-bit operand type once: relative 2^-11 (fp16) or
// 2^-8 (bf16) at most, independent from key to key. The sum is that of the unrounded p, so a single heavy key's
// rounding stays in the output: at most as much again as the output's own rounding. Measured against 64 bits
// (relative, root mean square; a plain fp32 form in brackets): bf16 pool 0.0022 (0.0017), fp16 outputs behind 65536
// int8 keys 0.00029 (0.00021), the other cases as the plain form.
//
// Measured: 64 rows x 64 heads of 128 over 0 to 8192 e4m3 keys of their own, no prefix (539 MB), 101 us in this
// kernel (5.3 TB/s); 128 rows x 32 heads over 16 to 2048 bf16 keys (270 MB) 58 us (4.7 TB/s). Between its start and
// its join a CTA streams at more than its share of the memory rate; the block list, table and query that it waits for
// before the first key, and the join, are 40 to 60 % of a short range's time and are hidden by the SM's other one
// to three CTAs only in part.
#pragma once

#include <atomic>

#include "qkv_internal.cuh"

namespace qkv {
namespace prefix {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTau = 8.0f;    // lazy-rescale threshold (log2 units)
constexpr float kPShift = 7.f;  // fp16 operand: p 2^7 stays below 2^15, and small p out of the subnormals
constexpr int kEuHeadroom = 2;  // int8: the V-scale bound 2^eu sits up to 2^2 above the largest scale seen

template <int FMT>
struct Fmt {
  static constexpr bool kInt8 = FMT == QKV_INT8_SIDE || FMT == QKV_INT8_INLINE;
  static constexpr bool kInline = FMT == QKV_INT8_INLINE;
  static constexpr bool kBytes = kInt8 || FMT == QKV_E4M3;  // one byte per value
  static constexpr bool kBf16 = FMT == QKV_BF16;            // multiplied as bf16; every other pool as fp16
};

// NP: (row, query head) pairs of a CTA. 16: they are the M of the MMAs, keys (dims) the N; 8: keys (dims) are the M,
// pairs the N.
template <int FMT, int HD, int NP>
struct Geom {
  using F = Fmt<FMT>;
  static constexpr int kRow = F::kBytes ? HD : 2 * HD;              // bytes of a record's values
  static constexpr int kGlobalRow = F::kInline ? HD + 4 : kRow;     // bytes between records
  // Keys of a warp tile (32 where rows are short: the softmax step's fixed cost is shared), ring stages and CTAs
  // per SM. A warp starts the copy of a tile when it is done with the one before: kStages - 1 tiles are in flight while
  // it waits, kStages - 2 while it computes, and the SM's other warps cover that (8 to 16 of them; up to 128 KB in
  // flight). Started before the tile at hand is computed instead, us after that | before: heads of 128, 8 pairs, e4m3
  // 106 | 105, inline int8 127 | 129, bf16 59.6 | 58.4, 16 pairs, int8 66 | 62.5; heads of 256, 8 pairs, e4m3 83 | 78,
  // bf16 78 | 81, 16 pairs, int8 61.5 | 63; drafts 42.6 | 44: no gain on the whole. Tiles of 8 pairs with rows of
  // 128 B, us with 16 keys in three stages on four CTAs | 32 keys in two on three, the next tile ahead in L2: e4m3, 64
  // rows x 64 heads of 0 to 8192 keys 114 | 105, 4 rows of 1000 9.0 | 8.3, 256 rows of 50 to 300 35 | 37; inline int8,
  // 64 rows of 0 to 4096 131 | 125; int8 with side scales 79 | 86 (the cause is not known), so that one keeps the former.
  static constexpr bool kShort = kRow == 128 && (NP == 16 || FMT != QKV_INT8_SIDE);
  static constexpr int kKeys = kShort ? 32 : 16;
  static constexpr int kStages = kShort || (kRow == 256 && NP == 8) ? 2 : 3;
  static constexpr int kMinBlocks = kShort ? 3 : kRow == 128 ? 4 : kRow == 256 ? (NP == 16 ? 2 : 3) : 1;
  // The next tile fetched into L2 ahead of its copy, where the ring holds two tiles of 8 KB and the tile has 8
  // pairs: 128 rows x 32 heads over 16 to 2048 own keys, heads of 128 in bf16 64 -> 60 us, of 256 in e4m3 90 ->
  // 83, in inline int8 118 -> 104; with the other rings it costs (e4m3, 16 keys in three stages: 110 -> 114 us).
  static constexpr bool kAhead = NP == 8 && kStages == 2;
  static constexpr int kScales = 2 * kKeys * kRow;
  static constexpr int kMask = kScales + (F::kInt8 ? 2 * kKeys * 4 : 0);
  static constexpr int kStage = kMask + 16;  // K, V, scales, key mask
  static constexpr int kQPad = F::kBytes ? 16 : 64;  // two rows of a quarter-warp fall on disjoint banks
  static constexpr int kQRow = 2 * HD + kQPad;
  static constexpr int kORow = HD + 4;  // floats per pair of the final join
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kJoin = kWarps * NP * kORow * 4;
  static constexpr int kArea = kRing > kJoin ? kRing : kJoin;
  static constexpr int kSmem = kArea + NP * kQRow;
};

// Row (of 16) feeding column n of N-tile nt (of 2) of q.K^T, so that the p a lane holds are those of the
// keys its transposed V fragments hold (bytes: keys 4c .. 4c + 3 in one register).
template <int FMT>
__device__ __forceinline__ int key_of(int nt, int n) {
  if (Fmt<FMT>::kInt8) return 2 * n + nt;
  if (Fmt<FMT>::kBytes) return 4 * (n >> 1) + (n & 1) + 2 * nt;
  return 8 * nt + n;
}
// 16 B chunk ch of tile row r sits at chunk ch ^ swz(r): the eight rows of a transposed load and
// the two rows a quarter-warp reads together fall on distinct banks.
template <int FMT>
__device__ __forceinline__ int swz(int r) {
  return Fmt<FMT>::kInt8 ? (((r >> 1) & 1) << 2) | (r & 1) | (((r >> 2) & 1) << 1) : ((r & 1) << 2) | ((r >> 1) & 3);
}

// Keys of its own that a row sees; kEmptyRow: it sees nothing; kPadRow: no row at all.
constexpr int kEmptyRow = -1, kPadRow = -2;
__device__ __forceinline__ int row_state(const PrefixArgs& a, int seq, int len, bool flags) {
  if (seq == -1) return kPadRow;
  if (seq < 0 || seq >= a.num_seqs || len < 0 || len > a.max_row_len || (len > 0 && len < a.prefix_len)) {
    if (flags && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_INDEX);
    return kEmptyRow;
  }
  return len == 0 ? kEmptyRow : len - a.prefix_len;
}
__device__ __forceinline__ int row_state(const PrefixArgs& a, int64_t r, bool flags) {
  return row_state(a, __ldg(a.row_seq + r), __ldg(a.row_len + r), flags);
}
// A kernel that a later one of the call need not wait for, and the wait itself (programmatic launches).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]

// out (16-bit) of one value pair
__device__ __forceinline__ uint32_t round2(bool f16, float x, float y) { return f16 ? pack_half2(x, y) : pack_bf162(x, y); }

// The 8 x 8 matrix of 16-bit values that the warp holds (row lane / 4, columns 2 (lane % 4) and the next),
// transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16) mma_bf16(d, a, b0, b1);
  else mma_f16(d, a, b0, b1);
}

template <int FMT, int HD, int NP>
__global__ void __launch_bounds__(kThreads, Geom<FMT, HD, NP>::kMinBlocks) prefix_mma_kernel(const PrefixArgs a) {
  using F = Fmt<FMT>;
  using GM = Geom<FMT, HD, NP>;
  constexpr bool kWide = NP == 16;     // pairs are the MMAs' M
  constexpr int KL = kWide ? 2 : 1;    // keys of eight whose logits a lane holds, for each of its two pairs
  constexpr int RB = GM::kRow, ST = GM::kStages, CH = RB / 16, TK = GM::kKeys, NH = TK / 16;
  constexpr uint32_t kAll = TK == 32 ? 0xffffffffu : 0xffffu;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sFac[NP], sM[kWarps][NP], sL[kWarps][NP];
  __shared__ float sW[kWarps][NP], sInv[NP], sUp[NP];
  __shared__ int64_t sAt[NP];
  __shared__ int sEu[kWarps][NP];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, hn = lane >> 2;
  const int H = a.num_kv_heads, G = a.num_q_heads / H;
  let_next_start();
  const bool own_part = blockIdx.x >= a.prefix_items;
  uint32_t item = own_part ? blockIdx.x - static_cast<uint32_t>(a.prefix_items) : blockIdx.x;
  const uint32_t parts = own_part ? a.own_parts : a.prefix_parts;
  const int part = static_cast<int>(item % parts);
  item /= parts;
  const int h = static_cast<int>(item % static_cast<uint32_t>(H));
  const uint32_t tile = item / static_cast<uint32_t>(H);

  // ---------------- the tile's pairs: lane i < NP holds pair i (row, head of the group, keys of its own)
  int my_row = -1, my_g = 0, my_own = kPadRow;
  uint32_t r0 = 0;  // own part: its first row
  int nrows = 0;    //           its rows, all of one sequence
  int seq = 0;
  if (own_part) {
    const int T = G >= NP ? 1 : NP / G, chunks = (G + NP - 1) / NP;
    r0 = tile / static_cast<uint32_t>(chunks);
    const int ch = static_cast<int>(tile % static_cast<uint32_t>(chunks));
    // lane t holds row r0 + t, lane 31 the row before
    const int64_t rr = static_cast<int64_t>(r0) + (lane == 31 ? -1 : lane);
    const bool there = rr >= 0 && rr < a.rows && (lane == 31 || lane < T);
    const int rs = there ? __ldg(a.row_seq + rr) : 0, rl = there ? __ldg(a.row_len + rr) : 0;
    seq = __shfl_sync(0xffffffffu, rs, 0);
    const uint32_t same = __ballot_sync(0xffffffffu, there && rs == seq);
    // rows [r0, r0 + n) up to the next multiple of T, while the sequence stays the same; a row that
    // continues such a run is in its first row's tile
    const int into = static_cast<int>(r0 % static_cast<uint32_t>(T));
    if (into != 0 && (same >> 31)) return;
    nrows = min(__ffs(~same) - 1, T - into);
    const int state = row_state(a, rs, rl, false);
    const int t = G >= NP ? 0 : lane / G;
    my_g = G >= NP ? ch * NP + lane : lane - t * G;
    const int st = __shfl_sync(0xffffffffu, state, t & 31);
    if (lane < NP && t < nrows && my_g < G) my_row = static_cast<int>(r0) + t, my_own = st;
  } else {
    const uint32_t flat = tile * NP + lane, row = flat / static_cast<uint32_t>(G);  // below 2^31 + 32
    my_g = static_cast<int>(flat - row * G);
    if (lane < NP && row < a.rows) my_row = static_cast<int>(row), my_own = 0;
  }

  // ---------------- its keys: positions [k0, k1) in tiles from a0 (a multiple of TK) on
  int k0, k1, own_min = INT_MAX;  // own_min: the shortest row's end
  if (own_part) {
    const int n = max(0, __reduce_max_sync(0xffffffffu, my_own));
    own_min = a.prefix_len + __reduce_min_sync(0xffffffffu, my_row >= 0 ? max(my_own, 0) : INT_MAX - a.prefix_len);
    // ranges end at multiples of a CTA's step
    const int first = a.prefix_len & ~(TK - 1), len = a.prefix_len + n - first, np = static_cast<int>(parts);
    const int per = ((len + np - 1) / np + TK * kWarps - 1) / (TK * kWarps) * (TK * kWarps);
    const int64_t lo = first + static_cast<int64_t>(part) * per;
    k0 = static_cast<int>(max(static_cast<int64_t>(a.prefix_len), min(lo, static_cast<int64_t>(a.prefix_len) + n)));
    k1 = static_cast<int>(min(lo + per, static_cast<int64_t>(a.prefix_len) + n));
    if (n == 0) k1 = k0;
  } else {
    k0 = static_cast<int>(min(static_cast<int64_t>(a.prefix_len), static_cast<int64_t>(part) * a.prefix_chunk));
    k1 = static_cast<int>(min(static_cast<int64_t>(a.prefix_len), static_cast<int64_t>(k0) + a.prefix_chunk));
  }
  const int a0 = k0 & ~(TK - 1);
  const int ntiles = k1 > k0 ? (k1 - a0 + TK - 1) / TK : 0;
  const int my = ntiles > warp ? (ntiles - warp + kWarps - 1) / kWarps : 0;

  // ---------------- block lookups and copies
  const int32_t* table = a.prefix_blocks;
  if (own_part) table = a.block_table + static_cast<int64_t>(seq >= 0 && seq < a.num_seqs ? seq : 0) * a.max_blocks;
  const int bsz = a.block_size;
  const bool pow2 = (bsz & (bsz - 1)) == 0, runs = bsz % TK == 0;  // runs: a tile never leaves its block
  const int shift = __ffs(bsz) - 1;
  auto block_of = [&](int pos) -> int { return pow2 ? pos >> shift : pos / bsz; };
  auto tile_pos = [&](int i) -> int { return a0 + (warp + kWarps * i) * TK; };
  // block id of key `lane` of this warp's tile i (loaded a tile ahead of its use)
  auto load_blk = [&](int i) -> int {
    const int pos = tile_pos(i) + lane;
    return (i < my && lane < TK && pos >= k0 && pos < k1) ? __ldg(table + block_of(pos)) : -1;
  };
  uint8_t* ring = smem + warp * ST * GM::kStage;
  const int key_sub = lane >> 3, chunk_sub = lane & 7;
  const int64_t rec_bytes = static_cast<int64_t>(H) * GM::kGlobalRow;  // bytes between slots
  auto issue = [&](int i, int blk) {
    if (i < my) {
      uint8_t* st = ring + (i % ST) * GM::kStage;
      const uint32_t sk = smem_u32(st), sv = sk + TK * RB;
      const int p0 = tile_pos(i);
      // all keys wanted and one run of slots: no lookups per key
      const int blk0 = __shfl_sync(0xffffffffu, blk, 0);
      const int64_t slot0 = static_cast<int64_t>(blk0) * bsz + (p0 - block_of(p0) * bsz);
      const bool run = runs && p0 >= k0 && p0 + TK <= k1 && blk0 >= 0 && slot0 + TK <= a.num_slots;
      int rec_l = -1;  // record of key `lane`, -1: none
      uint32_t mask = kAll;
      if (!run) {
        const int pos = p0 + lane;
        if (lane < TK && pos >= k0 && pos < k1) {
          const int64_t slot = static_cast<int64_t>(blk) * bsz + (pos - block_of(pos) * bsz);
          if (blk < 0 || slot >= a.num_slots) {
            if (a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_INDEX);
          } else {
            rec_l = static_cast<int>(slot) * H + h;  // the host keeps num_slots * H below 2^31
          }
        }
        mask = __ballot_sync(0xffffffffu, rec_l >= 0);
      } else {
        rec_l = (static_cast<int>(slot0) + lane) * H + h;  // lanes past the tile: not used
      }
      if (lane == 0) sts32(sk + GM::kMask, mask);
      if (!F::kInline) {
        // four keys per instruction, one 128 B line of each; a masked key zero-fills its rows
        const int64_t run_off = run ? (static_cast<int64_t>(slot0 + key_sub) * H + h) * RB + 16 * chunk_sub : 0;
#pragma unroll
        for (int t = 0; t < TK / 4; ++t) {
          const int kr = key_sub + 4 * t;
          int nb = 16;
          int64_t off = run_off + 4 * t * rec_bytes;
          if (!run) {
            const int rec = __shfl_sync(0xffffffffu, rec_l, kr);
            nb = rec >= 0 ? 16 : 0;
            off = static_cast<int64_t>(max(rec, 0)) * RB + 16 * chunk_sub;
          }
#pragma unroll
          for (int u = 0; u < CH / 8; ++u) {
            const uint32_t d = kr * RB + (((chunk_sub + 8 * u) ^ swz<FMT>(kr & 15)) << 4);
            cp_async16(sk + d, a.k_cache + off + 128 * u, nb);
            cp_async16(sv + d, a.v_cache + off + 128 * u, nb);
          }
        }
        if (F::kInt8 && lane < TK) {
          cp_async4(sk + GM::kScales + 4 * lane, a.k_scale_tok + max(rec_l, 0), rec_l >= 0 ? 4 : 0);
          cp_async4(sk + GM::kScales + 4 * (TK + lane), a.v_scale_tok + max(rec_l, 0), rec_l >= 0 ? 4 : 0);
        }
      } else {
        // inline records sit on 4 B boundaries: 4 B copies, one key per instruction
#pragma unroll 4
        for (int kr = 0; kr < TK; ++kr) {
          const int rec = __shfl_sync(0xffffffffu, rec_l, kr);
          const int nb = rec >= 0 ? 4 : 0;
          const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(max(rec, 0))) * GM::kGlobalRow;
#pragma unroll
          for (int u = 0; u < HD / 128; ++u) {
            const int w = lane + 32 * u;
            const uint32_t d = kr * RB + (((w >> 2) ^ swz<FMT>(kr & 15)) << 4) + 4 * (w & 3);
            cp_async4(sk + d, a.k_cache + off + 4 * w, nb);
            cp_async4(sv + d, a.v_cache + off + 4 * w, nb);
          }
        }
        if (lane < TK) {
          const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(max(rec_l, 0))) * GM::kGlobalRow + HD;
          cp_async4(sk + GM::kScales + 4 * lane, a.k_cache + off, rec_l >= 0 ? 4 : 0);
          cp_async4(sk + GM::kScales + 4 * (TK + lane), a.v_cache + off, rec_l >= 0 ? 4 : 0);
        }
      }
    }
    cp_async_commit();
  };

  // The tile after the one whose copy has just been started into L2, while that one is copied and computed.
  auto prefetch = [&](int i, int blk) {
    if (!GM::kAhead || i >= my) return;
    const int key = lane & (TK - 1), pos = tile_pos(i) + key;
    const int b = __shfl_sync(0xffffffffu, blk, key);
    const int64_t slot = static_cast<int64_t>(b) * bsz + (pos - block_of(pos) * bsz);
    if (b < 0 || slot >= a.num_slots) return;
    const int64_t off = (slot * H + h) * GM::kGlobalRow;
#pragma unroll
    for (int u = 0; u < RB / 128; ++u) {
      if (TK == 32 || lane < TK) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(a.k_cache + off + 128 * u));
      if (TK == 32 || lane >= TK) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(a.v_cache + off + 128 * u));
    }
  };

  int blk = load_blk(0), next0 = load_blk(1);  // before the query's loads: the copies wait for them

  // ---------------- query rows into registers, each warp a quarter of the pairs
  constexpr int kPer = HD / 32, kQPairs = NP / kWarps;  // dims per lane, pairs per warp
  uint32_t qw[kQPairs][kPer / 2];
#pragma unroll
  for (int i = 0; i < kQPairs; ++i) {
    const int row = __shfl_sync(0xffffffffu, my_row, warp * kQPairs + i), g = __shfl_sync(0xffffffffu, my_g, warp * kQPairs + i);
    const uint16_t* src = a.q + static_cast<int64_t>(max(row, 0)) * a.q_stride + static_cast<int64_t>(row >= 0 ? h * G + g : 0) * HD;
    if (kPer == 8) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + lane);
      qw[i][0] = v.x, qw[i][1] = v.y, qw[i][kPer / 2 - 2] = v.z, qw[i][kPer / 2 - 1] = v.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + lane);
      qw[i][0] = v.x, qw[i][1] = v.y;
    }
  }

#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) {
    const int next = i == 0 ? next0 : load_blk(i + 1);
    issue(i, blk);
    blk = next;
  }
  prefetch(ST - 1, blk);

  // ---------------- the query into shared memory; bytes pools: fp16, in the fragments' dim order
  uint8_t* sQ = smem + GM::kArea;
#pragma unroll
  for (int i = 0; i < kQPairs; ++i) {
    const int pair = warp * kQPairs + i;
    const bool in = __shfl_sync(0xffffffffu, my_row, pair) >= 0;
    uint32_t w[kPer / 2];
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) w[k] = in ? qw[i][k] : 0u;
    uint8_t* row = sQ + pair * GM::kQRow;
    float fac = fabsf(a.softmax_scale) * kLog2e;
    const float sign = a.softmax_scale < 0.f ? -1.f : 1.f;  // into the query: the logit factor stays >= 0
    if (F::kBytes) {
      float x[kPer], m = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const uint32_t b = w[k / 2];
        if (a.q_f16) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&b));
          x[k] = (k & 1) ? f.y : f.x;
        } else {
          x[k] = (k & 1) ? bf16hi(b) : bf16lo(b);
        }
        m = fmaxf(m, fabsf(x[k]));
      }
      m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // magnitudes: bits order like values
      // largest magnitude into [2^14, 2^15): e = 14 - floor(log2 m), kept where 2^e and 2^-e are normal
      int e = m > 0.f ? 14 - (static_cast<int>(__float_as_uint(m) >> 23) - 127) : 0;
      e = max(-112, min(126, e));
      const float up = sign * pow2f(e);
#pragma unroll
      for (int k = 0; k < kPer; k += 4) {
        // int8: dims (0, 2), (1, 3) of each four, the pairs of the code splice
        const float y0 = x[k] * up, y1 = x[k + 1] * up, y2 = x[k + 2] * up, y3 = x[k + 3] * up;
        const uint2 v = F::kInt8 ? make_uint2(pack_half2(y0, y2), pack_half2(y1, y3))
                                 : make_uint2(pack_half2(y0, y1), pack_half2(y2, y3));
        *reinterpret_cast<uint2*>(row + (lane * kPer + k) * 2) = v;
      }
      fac *= pow2f(-e);
      if (FMT == QKV_E4M3) fac *= a.k_scale_layer;
    } else {
      const uint32_t flip = sign < 0.f ? 0x80008000u : 0u;
#pragma unroll
      for (int k = 0; k < kPer; k += 4)
        *reinterpret_cast<uint2*>(row + (lane * kPer + k) * 2) = make_uint2(w[k / 2] ^ flip, w[k / 2 + 1] ^ flip);
    }
    if (lane == 0) sFac[pair] = fac;
  }
  __syncthreads();

  // kWide: pairs hn, hn + 8 (rows) by dims 8t + 2c, 2c + 1 (columns) of tile t; else dims 16t + hn, hn + 8 by
  // pairs 2c, 2c + 1
  constexpr int kOTiles = kWide ? HD / 8 : HD / 16;
  float o[kOTiles][4];
#pragma unroll
  for (int t = 0; t < kOTiles; ++t)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[t][k] = 0.f;
  float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int eu[2] = {-120, -120};  // int8: a pair's accumulators hold values times 2^-eu
  const int pr[2] = {kWide ? hn : 2 * c, kWide ? hn + 8 : 2 * c + 1};  // the lane's two pairs
  const float fac[2] = {sFac[pr[0]], sFac[pr[1]]};
  // first position past each of the lane's two rows
  int end[2], row_of[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int ow = __shfl_sync(0xffffffffu, my_own, pr[p]);
    end[p] = own_part ? a.prefix_len + max(ow, 0) : INT_MAX;
    row_of[p] = __shfl_sync(0xffffffffu, my_row, pr[p]);
  }
  const uint32_t qa = smem_u32(sQ) + hn * GM::kQRow, qb = qa + (kWide ? 8 * GM::kQRow : 0);
  // 128-wide heads: the query's fragments stay in registers
  constexpr bool kQReg = HD == 128;
  uint4 qf[kQReg ? HD / 32 : 1][KL];
  if (kQReg) {
#pragma unroll
    for (int j = 0; j < HD / 32; ++j) {
      const uint32_t qo = F::kBytes ? 128 * (j >> 1) + 32 * c + 16 * (j & 1) : 64 * j + 16 * c;
      qf[j % (kQReg ? HD / 32 : 1)][0] = lds128(qa + qo);
      if (kWide) qf[j % (kQReg ? HD / 32 : 1)][KL - 1] = lds128(qb + qo);
    }
  }

#pragma unroll 1
  for (int i = 0; i < my; ++i) {
    const int next = load_blk(i + ST);
    cp_async_wait<ST - 2>();
    __syncwarp();
    const uint32_t sk = smem_u32(ring + (i % ST) * GM::kStage), sv = sk + TK * RB;
    const uint32_t mask = lds32(sk + GM::kMask);
    const int base = tile_pos(i);
    // every key wanted by every row: no masks
    const bool whole = mask == kAll && base + TK <= own_min;

    // ---- logits of 2 NH groups of eight keys. kWide: N-tiles, s[n][2p + k]: pair p, key 2c + k of the group;
    // else halves of M-tiles, s[n / 2][2 (n % 2) + p]: key hn of the group, pair p
    float s[KL * NH][4];
#pragma unroll
    for (int n = 0; n < KL * NH; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[n][k] = 0.f;
    auto S = [&](int n, int p, int k) -> float& { return kWide ? s[n % (KL * NH)][2 * p + k] : s[(n >> 1) % (KL * NH)][2 * (n & 1) + p]; };
    auto key_at = [&](int n, int k) -> int { return 16 * (n >> 1) + key_of<FMT>(n & 1, kWide ? 2 * c + k : hn); };
    uint4 kb[2 * NH];  // bytes pools: 16 dims per lane, for two j
#pragma unroll
    for (int j = 0; j < HD / 32; ++j) {  // two k-steps of 16 dims
      uint4 x, y;
      if (kQReg) {
        x = qf[j % (kQReg ? HD / 32 : 1)][0], y = qf[j % (kQReg ? HD / 32 : 1)][KL - 1];
      } else {
        const uint32_t qo = F::kBytes ? 128 * (j >> 1) + 32 * c + 16 * (j & 1) : 64 * j + 16 * c;
        x = lds128(qa + qo), y = kWide ? lds128(qb + qo) : x;
      }
      uint32_t kf[2 * NH][4];  // a key's dims of the two k-steps
#pragma unroll
      for (int n = 0; n < 2 * NH; ++n) {
        const int kr = key_of<FMT>(n & 1, hn);
        const uint32_t krow = sk + (kr + 16 * (n >> 1)) * RB;
        if (F::kBytes) {
          if ((j & 1) == 0) kb[n] = lds128(krow + (((4 * (j >> 1) + c) ^ swz<FMT>(kr)) << 4));
          const uint2 kw = (j & 1) ? make_uint2(kb[n].z, kb[n].w) : make_uint2(kb[n].x, kb[n].y);  // four dims per k-step
          kf[n][0] = F::kInt8 ? i8pair_to_f16x2(kw.x) : e4m3pair_to_f16x2(kw.x);
          kf[n][1] = F::kInt8 ? i8pair_to_f16x2(kw.x >> 8) : e4m3pair_to_f16x2(kw.x >> 16);
          kf[n][2] = F::kInt8 ? i8pair_to_f16x2(kw.y) : e4m3pair_to_f16x2(kw.y);
          kf[n][3] = F::kInt8 ? i8pair_to_f16x2(kw.y >> 8) : e4m3pair_to_f16x2(kw.y >> 16);
        } else {
          const uint4 kw = lds128(krow + (((4 * j + c) ^ swz<FMT>(kr)) << 4));
          kf[n][0] = kw.x, kf[n][1] = kw.y, kf[n][2] = kw.z, kf[n][3] = kw.w;
        }
        if (kWide) {
          const uint32_t a0f[4] = {x.x, y.x, x.y, y.y}, a1f[4] = {x.z, y.z, x.w, y.w};
          mma16<F::kBf16>(s[n % (KL * NH)], a0f, kf[n][0], kf[n][1]);
          mma16<F::kBf16>(s[n % (KL * NH)], a1f, kf[n][2], kf[n][3]);
        } else if (n & 1) {
          const uint32_t a0f[4] = {kf[n - 1][0], kf[n][0], kf[n - 1][1], kf[n][1]};
          const uint32_t a1f[4] = {kf[n - 1][2], kf[n][2], kf[n - 1][3], kf[n][3]};
          mma16<F::kBf16>(s[(n >> 1) % (KL * NH)], a0f, x.x, x.y);
          mma16<F::kBf16>(s[(n >> 1) % (KL * NH)], a1f, x.z, x.w);
        }
      }
    }

    // ---- softmax step
    float vs[2 * NH][KL];  // int8: V scales of the lane's keys
    float vmax[2] = {0.f, 0.f};  // the largest that a pair sees: what lies behind its row's end is not its own
#pragma unroll
    for (int g = 0; g < NH; ++g) {
      float ks[2][KL];
      if (F::kInt8) {  // the lane's keys of 16: 4c .. 4c + 3 (kWide), 2 hn and the next
        const uint32_t at = sk + GM::kScales + 4 * (16 * g + 2 * KL * (kWide ? c : hn));
        uint32_t kw[4], vw[4];
        if (kWide) {
          const uint4 k4 = lds128(at), v4 = lds128(at + 4 * TK);
          kw[0] = k4.x, kw[1] = k4.y, kw[2] = k4.z, kw[3] = k4.w;
          vw[0] = v4.x, vw[1] = v4.y, vw[2] = v4.z, vw[3] = v4.w;
        } else {
          kw[0] = lds32(at), kw[1] = lds32(at + 4);
          vw[0] = lds32(at + 4 * TK), vw[1] = lds32(at + 4 * TK + 4);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < KL; ++k) {  // key 2 (2c + k) + n, or 2 hn + n
            ks[n][k] = __uint_as_float(kw[2 * k + n]);
            vs[2 * g + n][k] = __uint_as_float(vw[2 * k + n]);
            vmax[0] = fmaxf(vmax[0], fabsf(vs[2 * g + n][k]));
          }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int k = 0; k < KL; ++k)
#pragma unroll
          for (int p = 0; p < 2; ++p) S(2 * g + n, p, k) *= F::kInt8 ? ks[n][k] * fac[p] : fac[p];
    }
    vmax[1] = vmax[0];
    if (!whole) {
      vmax[0] = vmax[1] = 0.f;
#pragma unroll
      for (int n = 0; n < 2 * NH; ++n)
#pragma unroll
        for (int k = 0; k < KL; ++k) {
          const int key = key_at(n, k);
          const bool valid = (mask >> key) & 1;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            if (!valid || base + key >= end[p]) S(n, p, k) = -INFINITY;
            else if (F::kInt8) vmax[p] = fmaxf(vmax[p], fabsf(vs[n][k]));
          }
        }
    }
    float tm[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      tm[p] = -INFINITY;
#pragma unroll
      for (int n = 0; n < 2 * NH; ++n)
#pragma unroll
        for (int k = 0; k < KL; ++k) tm[p] = fmaxf(tm[p], S(n, p, k));
    }
    // over the lanes that hold the pairs' other keys: four (c) or eight (hn)
#pragma unroll
    for (int off = kWide ? 1 : 4; off <= (kWide ? 2 : 16); off <<= 1) {
      tm[0] = fmaxf(tm[0], __shfl_xor_sync(0xffffffffu, tm[0], off));
      tm[1] = fmaxf(tm[1], __shfl_xor_sync(0xffffffffu, tm[1], off));
      if (F::kInt8) {
        vmax[0] = fmaxf(vmax[0], __shfl_xor_sync(0xffffffffu, vmax[0], off));
        vmax[1] = whole ? vmax[0] : fmaxf(vmax[1], __shfl_xor_sync(0xffffffffu, vmax[1], off));
      }
    }
    int eu_new[2] = {eu[0], eu[1]};
    if (F::kInt8) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int e = min(120, static_cast<int>(__float_as_uint(vmax[p]) >> 23) - 126);  // vmax < 2^e
        if (e > eu[p]) eu_new[p] = min(120, e + kEuHeadroom);
      }
    }
    // a first finite logit has no reference to be compared with: M = -inf lies below any
    const bool raise0 = tm[0] > M[0] + kTau, raise1 = tm[1] > M[1] + kTau;
    if (__any_sync(0xffffffffu, raise0 || raise1 || eu_new[0] != eu[0] || eu_new[1] != eu[1])) {
      float f[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const bool up = p ? raise1 : raise0;
        const float m = up ? tm[p] : M[p];
        const float al = (up && M[p] != -INFINITY) ? fast_exp2(M[p] - m) : 1.f;
        M[p] = m;
        l[p] *= al;
        f[p] = F::kInt8 ? al * pow2f(max(eu[p] - eu_new[p], -126)) : al;
        eu[p] = eu_new[p];
      }
#pragma unroll
      for (int t = 0; t < kOTiles; ++t) {
        o[t][0] *= f[0];
        o[t][1] *= f[kWide ? 0 : 1];
        o[t][2] *= f[kWide ? 1 : 0];
        o[t][3] *= f[1];
      }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float ref = M[p] == -INFINITY ? 0.f : M[p] - (F::kBf16 ? 0.f : kPShift);
      const float vdown = F::kInt8 ? pow2f(-eu[p]) : 1.f;
#pragma unroll
      for (int n = 0; n < 2 * NH; ++n)
#pragma unroll
        for (int k = 0; k < KL; ++k) {
          const float y = S(n, p, k);
          float e = fast_exp2(y - ref);
          l[p] += e;
          if (F::kInt8) {
            e *= vs[n][k] * vdown;
            if (!whole && y == -INFINITY) e = 0.f;  // a masked key's scale may be anything (0 x inf): its p stays 0
          }
          S(n, p, k) = e;
        }
    }
    // kWide: the A operand, pairs by keys; else the B operand, keys by pairs (a lane's pairs were the columns)
    uint32_t pa[NH][2 * KL];
#pragma unroll
    for (int n = 0; n < 2 * NH; ++n)
#pragma unroll
      for (int p = 0; p < KL; ++p) {
        const float e0 = S(n, p, 0), e1 = kWide ? S(n, p, KL - 1) : S(n, 1, 0);
        const uint32_t w = F::kBf16 ? pack_bf162(e0, e1) : pack_half2(e0, e1);
        pa[n >> 1][KL * (n & 1) + p] = kWide ? w : transpose8x8(w);
      }

    // ---- p V
    // b0, b1 of the four N-tiles of eight dims from 32 q on, 16 keys from 16 g on
    auto v_frags = [&](int g, int q, uint32_t (&v)[8]) {
      const uint32_t sg = sv + 16 * g * RB;
      if (F::kBytes) {
        // matrices of 16 keys x 16 dims: chunk 2q for lanes 0-15's addresses, 2q + 1 for the others
        uint32_t m[4];
        const int r = lane & 15;
        ldmatrix_x2_trans_b8(sg + r * RB + (((2 * q + (lane >> 4)) ^ swz<FMT>(r)) << 4), m[0], m[1], m[2], m[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (F::kInt8) {
            v[2 * k] = i8pair_to_f16x2(m[k]);
            v[2 * k + 1] = i8pair_to_f16x2(m[k] >> 8);
          } else {
            v[2 * k] = e4m3pair_to_f16x2(m[k]);
            v[2 * k + 1] = e4m3pair_to_f16x2(m[k] >> 16);
          }
        }
      } else {
        // four 8 x 8 matrices: keys 0-7 and 8-15 of chunks ch and ch + 1
        const int r = (lane & 7) + (lane & 8), chs = lane >> 4;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int ch = 4 * q + 2 * k + chs;
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                       : "=r"(v[4 * k]), "=r"(v[4 * k + 1]), "=r"(v[4 * k + 2]), "=r"(v[4 * k + 3])
                       : "r"(sg + r * RB + ((ch ^ swz<FMT>(r)) << 4)));
        }
      }
    };
    // tile k of the four of 8 dims (kWide) or the two of 16 that v holds
    auto pv = [&](float (&d)[4], const uint32_t (&pw)[2 * KL], const uint32_t (&v)[8], int k) {
      if constexpr (kWide) {
        mma16<F::kBf16>(d, pw, v[2 * k], v[2 * k + 1]);
      } else {
        const uint32_t av[4] = {v[4 * k], v[4 * k + 2], v[4 * k + 1], v[4 * k + 3]};
        mma16<F::kBf16>(d, av, pw[0], pw[1]);
      }
    };
    // Rows of different lengths in one tile: a key that one row sees and another does not may hold
    // anything there (0 x NaN), so such a tile goes row by row, each with its own keys only, and only
    // that row's sums are taken.
    if (!F::kInt8 && own_part && nrows > 1 && base + TK > own_min) {
#pragma unroll 1
      for (int t = 0; t < nrows; ++t) {
        const int row = static_cast<int>(r0) + t;
        const int n_end = a.prefix_len + max(0, __shfl_sync(0xffffffffu, my_own, t * G));
#pragma unroll 1
        for (int g = 0; g < NH; ++g) {
          uint32_t keep[2], pg[2 * KL];  // halves of b0 / b1 (the lane's keys) that the row sees
#pragma unroll
          for (int k = 0; k < 2; ++k)
            keep[k] = (base + 16 * g + key_of<FMT>(k, 2 * c) < n_end ? 0x0000ffffu : 0u) |
                      (base + 16 * g + key_of<FMT>(k, 2 * c + 1) < n_end ? 0xffff0000u : 0u);
#pragma unroll
          for (int k = 0; k < 2 * KL; ++k) pg[k] = g == 0 ? pa[0][k] : pa[NH - 1][k];
#pragma unroll
          for (int q = 0; q < HD / 32; ++q) {
            uint32_t v[8];
            v_frags(g, q, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] &= keep[k & 1];
#pragma unroll
            for (int k = 0; k < 2 * KL; ++k) {
              float x[4] = {0.f, 0.f, 0.f, 0.f};
              pv(x, pg, v, k);
              float* acc = o[2 * KL * q + k];
              if (row_of[0] == row) acc[0] += x[0], acc[kWide ? 1 : 2] += x[kWide ? 1 : 2];
              if (row_of[1] == row) acc[kWide ? 2 : 1] += x[kWide ? 2 : 1], acc[3] += x[3];
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int g = 0; g < NH; ++g)
#pragma unroll
        for (int q = 0; q < HD / 32; ++q) {
          uint32_t v[8];
          v_frags(g, q, v);
#pragma unroll
          for (int k = 0; k < 2 * KL; ++k) pv(o[2 * KL * q + k], pa[g], v, k);
        }
    }
    __syncwarp();
    issue(i + ST - 1, blk);
    prefetch(i + ST, next);
    blk = next;
  }

  // ---------------- join the four warps
  cp_async_wait<0>();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int off = kWide ? 1 : 4; off <= (kWide ? 2 : 16); off <<= 1) l[p] += __shfl_xor_sync(0xffffffffu, l[p], off);
    if ((kWide ? c : hn) == 0) {
      sM[warp][pr[p]] = M[p];
      sL[warp][pr[p]] = l[p];
      if (F::kInt8) sEu[warp][pr[p]] = eu[p];
    }
  }
  __syncthreads();  // every ring is drained
  float* sO = reinterpret_cast<float*>(smem);
  if (my > 0) {
#pragma unroll
    for (int t = 0; t < kOTiles; ++t)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float* row = sO + (warp * NP + pr[p]) * GM::kORow;
        if (kWide) *reinterpret_cast<float2*>(row + 8 * t + 2 * c) = make_float2(o[t][2 * p], o[t][2 * p + 1]);
        else row[16 * t + hn] = o[t][p], row[16 * t + 8 + hn] = o[t][2 + p];
      }
  }
  __syncthreads();
  const bool direct = a.o_part == nullptr;  // the only part: its result is the row's
  // one thread per pair: the warps' weights, log-sum-exp and where the result goes
  if (tid < NP) {
    const int head = h * G + my_g;
    int64_t at = -1;
    if (my_row >= 0) {
      const int state = direct ? row_state(a, static_cast<int64_t>(my_row), head == 0) : 0;
      const int64_t pair = static_cast<int64_t>(my_row) * a.num_q_heads + head;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sM[w][lane]);
      const float ref = m == -INFINITY ? 0.f : m;
      // int8: the warps' outputs are joined as values times 2^-top, and get 2^top last, after the division: sums of
      // keys with V scales up to 2^98 would not fit otherwise
      int top = -126;
      if (F::kInt8) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = max(top, sEu[w][lane]);
      }
      sUp[lane] = F::kInt8 ? pow2f(top) : 1.f;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float al = fast_exp2(sM[w][lane] - ref);  // 2^-inf = 0 for a warp without keys
        sum += al * sL[w][lane];
        // no keys, no values: -1. A warp with keys counts though its weight is 0: its values may be NaN
        const bool none = sM[w][lane] == -INFINITY && sL[w][lane] == 0.f;
        sW[w][lane] = none ? -1.f : F::kInt8 ? al * pow2f(max(sEu[w][lane] - top, -126)) : al;
      }
      const bool any = state != kEmptyRow && (m != -INFINITY || sum != sum);
      sInv[lane] = any ? (direct && FMT == QKV_E4M3 ? a.v_scale_layer : 1.f) / sum : 0.f;
      if (state != kPadRow) {
        const int64_t part_at = static_cast<int64_t>(own_part ? a.prefix_parts + part : part) * a.rows * a.num_q_heads + pair;
        const float v = any ? (m - (F::kBf16 ? 0.f : kPShift) + log2f(sum)) * kLn2 : -INFINITY;
        if (!direct) a.lse_part[part_at] = v;
        else if (a.lse != nullptr) a.lse[pair] = v;
        if (direct) at = pair;
        else if (any) at = part_at;  // a part without keys leaves no values
        if (!any) {
#pragma unroll
          for (int w = 0; w < kWarps; ++w) sW[w][lane] = -1.f;
        }
      }
    }
    sAt[lane] = at;
  }
  __syncthreads();
#pragma unroll
  for (int i0 = 0; i0 < NP; i0 += kWarps) {
    const int i = i0 + warp;
    const int64_t at = sAt[i];
    const float inv = sInv[i], up = sUp[i];
#pragma unroll
    for (int d = 4 * lane; d < HD; d += 128) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = sW[w][i];
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (f >= 0.f && at >= 0) x = *reinterpret_cast<const float4*>(sO + (w * NP + i) * GM::kORow + d);  // else none there
        acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
      }
      acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
      if (F::kInt8) acc.x *= up, acc.y *= up, acc.z *= up, acc.w *= up;
      if (at >= 0 && direct)
        *reinterpret_cast<uint2*>(a.out + at * HD + d) = make_uint2(round2(a.q_f16, acc.x, acc.y), round2(a.q_f16, acc.z, acc.w));
      else if (at >= 0)
        *reinterpret_cast<float4*>(a.o_part + at * HD + d) = acc;
    }
  }
  // the prefix's launch is over before this one is, so what waits for this one need not wait for both
  if (blockIdx.x == 0 && tid == 0) await_previous();
}

// A launch that may start while the call's previous kernel still runs (`overlaps`).
template <typename K>
cudaError_t launch_after(K kern, unsigned grid, unsigned block, int smem, bool overlaps, cudaStream_t stream,
                         const PrefixArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = overlaps ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// Opt a kernel into its dynamic shared memory, once per device (`done`: the kernel's own flags). Host threads may
// race here on a device's first call: both set the same attribute, and the flags are atomic.
template <typename K>
cudaError_t allow_smem(K kern, int smem, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

template <int FMT, int HD, int NP>
cudaError_t launch_mma(const PrefixArgs& a, bool overlaps, cudaStream_t stream) {
  static std::atomic<bool> done[64] = {};
  constexpr int smem = Geom<FMT, HD, NP>::kSmem;
  auto kern = prefix_mma_kernel<FMT, HD, NP>;
  cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  return launch_after(kern, static_cast<unsigned>(a.prefix_items + a.own_items), kThreads, smem, overlaps, stream, a);
}

template <int FMT>
cudaError_t launch_mma(const PrefixArgs& a, bool overlaps, cudaStream_t stream) {
  if (a.head_dim == 256)
    return a.mma_pairs == 8 ? launch_mma<FMT, 256, 8>(a, overlaps, stream) : launch_mma<FMT, 256, 16>(a, overlaps, stream);
  return a.mma_pairs == 8 ? launch_mma<FMT, 128, 8>(a, overlaps, stream) : launch_mma<FMT, 128, 16>(a, overlaps, stream);
}

}  // namespace prefix
}  // namespace qkv
