// Dense decode attention over a paged pool for a batch whose sequences share a prefix: the part of
// the work that runs on mma.sync tiles of 16 (row, query head) pairs.
//
// For row r, query head h and the keys j the row sees (positions 0 .. row_len - 1 of its sequence;
// those below prefix_len through the shared block list, the others through its own table row):
//   y_j = log2(e) scale q . K_j,  o = sum_j 2^(y_j - M) V_j / sum_j 2^(y_j - M),  lse = ln 2 (M + log2 sum)
// in one pass over the keys with a running reference M and sum per pair; M is raised (and the
// accumulators rescaled) only when a logit exceeds it by 2^8, so p <= 2^8.
//
// A CTA of four warps takes one tile of pairs, one KV head and one range of keys. OWN = false: the
// shared prefix, pairs taken across rows (row-major), so every key that is read serves 16 pairs of
// whatever rows. OWN = true: the keys behind the prefix, pairs of consecutive rows of one sequence.
// Each warp streams its own 16-key tiles through a cp.async ring; warps meet once, at the end, to
// join their sums. Quantised pools are multiplied in fp16: codes are exact fp16 values, the query is
// pre-scaled by a power of two into fp16 (exact except for values 2^-39 below the row's largest), the K
// scale multiplies the logit, the V scale p. p (times the V scale and a power of two) is rounded to
// the 16-bit operand type once: relative 2^-12 (fp16) or 2^-9 (bf16), independent from key to key,
// so an output has about the rounding error of its own 16-bit type or less.
// One CTA tile is bound by memory: a tile of 16 keys costs about 500 warp instructions against
// 8 KB of int8 records.
#pragma once

#include "qkv_internal.cuh"

namespace qkv {
namespace prefix {

constexpr int kKeys = 16;   // keys of a warp tile
constexpr int kPairs = 16;  // (row, query head) pairs of a CTA: the M of the MMAs
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

template <int FMT, int HD>
struct Geom {
  using F = Fmt<FMT>;
  static constexpr int kRow = F::kBytes ? HD : 2 * HD;              // bytes of a record's values
  static constexpr int kGlobalRow = F::kInline ? HD + 4 : kRow;     // bytes between records
  // ring stages: two CTAs per SM (one for 512 B rows), 24 to 48 KB of copies in flight per CTA
  static constexpr int kStages = kRow == 128 ? 4 : 3;
  static constexpr int kMinBlocks = kRow == 512 ? 1 : 2;
  static constexpr int kStage = 2 * kKeys * kRow + (F::kInt8 ? 2 * kKeys * 4 : 0) + 16;  // K, V, scales, key mask
  static constexpr int kScales = 2 * kKeys * kRow;
  static constexpr int kMask = kStage - 16;
  static constexpr int kQPad = F::kBytes ? 16 : 64;  // two rows of a quarter-warp fall on disjoint banks
  static constexpr int kQRow = 2 * HD + kQPad;
  static constexpr int kORow = HD + 4;  // floats per pair of the final join
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kJoin = kWarps * kPairs * kORow * 4;
  static constexpr int kArea = kRing > kJoin ? kRing : kJoin;
  static constexpr int kSmem = kArea + kPairs * kQRow;
};

// Tile row feeding column n of N-tile nt of q.K^T, so that the p a lane holds are those of the
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

// Keys of its own that row r sees; kEmptyRow: it sees nothing; kPadRow: no row at all.
constexpr int kEmptyRow = -1, kPadRow = -2;
__device__ __forceinline__ int row_state(const PrefixArgs& a, int64_t r, bool flags) {
  const int seq = __ldg(a.row_seq + r), len = __ldg(a.row_len + r);
  if (seq == -1) return kPadRow;
  if (seq < 0 || seq >= a.num_seqs || len < 0 || len > a.max_row_len || (len > 0 && len < a.prefix_len)) {
    if (flags && a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_INDEX);
    return kEmptyRow;
  }
  return len == 0 ? kEmptyRow : len - a.prefix_len;
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]

// out (16-bit) of one value pair
__device__ __forceinline__ uint32_t round2(bool f16, float x, float y) { return f16 ? pack_half2(x, y) : pack_bf162(x, y); }

template <int FMT, int HD, bool OWN>
__global__ void __launch_bounds__(kThreads, Geom<FMT, HD>::kMinBlocks) prefix_mma_kernel(const PrefixArgs a) {
  using F = Fmt<FMT>;
  using GM = Geom<FMT, HD>;
  constexpr int RB = GM::kRow, ST = GM::kStages, CH = RB / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int sRow[kPairs], sHead[kPairs], sOwn[kPairs];
  __shared__ float sFac[kPairs], sM[kWarps][kPairs], sL[kWarps][kPairs];
  __shared__ int sEu[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, hn = lane >> 2;
  const int H = a.num_kv_heads, G = a.num_q_heads / H;
  const int parts = OWN ? a.own_parts : a.prefix_parts;
  uint32_t item = blockIdx.x;
  const int part = static_cast<int>(item % static_cast<uint32_t>(parts));
  item /= static_cast<uint32_t>(parts);
  const int h = static_cast<int>(item % static_cast<uint32_t>(H));
  const uint32_t tile = item / static_cast<uint32_t>(H);

  // ---------------- the tile's pairs
  int64_t r0 = 0;   // OWN: its first row
  int nrows = 0;    // OWN: its rows, all of one sequence
  if (OWN) {
    const int T = G >= kPairs ? 1 : kPairs / G, chunks = (G + kPairs - 1) / kPairs;
    r0 = tile / static_cast<uint32_t>(chunks);
    const int ch = static_cast<int>(tile % static_cast<uint32_t>(chunks));
    const int seq = __ldg(a.row_seq + r0);
    // rows [r0, r0 + n) up to the next multiple of T, while the sequence stays the same; a row that
    // continues such a run is in its first row's tile
    if (r0 % T != 0 && __ldg(a.row_seq + r0 - 1) == seq) return;
    nrows = 1;
    while ((r0 + nrows) % T != 0 && r0 + nrows < a.rows && __ldg(a.row_seq + r0 + nrows) == seq) ++nrows;
    if (tid < kPairs) {
      const int t = G >= kPairs ? 0 : tid / G, g = G >= kPairs ? ch * kPairs + tid : tid % G;
      const bool in = t < nrows && g < G;
      sRow[tid] = in ? static_cast<int>(r0 + t) : -1;
      sHead[tid] = h * G + g;
      sOwn[tid] = in ? row_state(a, r0 + t, false) : kPadRow;
    }
  } else if (tid < kPairs) {
    const int64_t flat = static_cast<int64_t>(tile) * kPairs + tid;
    const int64_t row = flat / G;
    const bool in = row < a.rows;
    sRow[tid] = in ? static_cast<int>(row) : -1;
    sHead[tid] = h * G + static_cast<int>(flat - row * G);
    sOwn[tid] = 0;
  }
  __syncthreads();

  // ---------------- its keys [k0, k1), counted from the prefix's or the own part's first
  int k0, k1, own_min = 0;
  if (OWN) {
    int n = 0;
    own_min = INT_MAX;
    for (int i = 0; i < kPairs; ++i) {
      if (sRow[i] < 0) continue;
      n = max(n, sOwn[i]);
      own_min = min(own_min, max(sOwn[i], 0));
    }
    const int per = ((n + parts - 1) / parts + kKeys * kWarps - 1) / (kKeys * kWarps) * (kKeys * kWarps);
    k0 = static_cast<int>(min(static_cast<int64_t>(n), static_cast<int64_t>(part) * per));
    k1 = static_cast<int>(min(static_cast<int64_t>(n), static_cast<int64_t>(k0) + per));
  } else {
    k0 = static_cast<int>(min(static_cast<int64_t>(a.prefix_len), static_cast<int64_t>(part) * a.prefix_chunk));
    k1 = static_cast<int>(min(static_cast<int64_t>(a.prefix_len), static_cast<int64_t>(k0) + a.prefix_chunk));
  }
  const int ntiles = (k1 - k0 + kKeys - 1) / kKeys;
  const int my = ntiles > warp ? (ntiles - warp + kWarps - 1) / kWarps : 0;

  // ---------------- block lookups and copies
  const int32_t* table = a.prefix_blocks;
  const int pos0 = OWN ? a.prefix_len : 0;  // position of key 0
  if (OWN) {
    const int seq = __ldg(a.row_seq + r0);
    table = a.block_table + static_cast<int64_t>(seq >= 0 && seq < a.num_seqs ? seq : 0) * a.max_blocks;
  }
  const int bsz = a.block_size;
  const bool pow2 = (bsz & (bsz - 1)) == 0;
  const int shift = __ffs(bsz) - 1;
  auto block_of = [&](int pos) -> int { return pow2 ? pos >> shift : pos / bsz; };
  // block id of key `lane` of this warp's tile i (loaded a tile ahead of its use)
  auto load_blk = [&](int i) -> int {
    const int key = k0 + (warp + kWarps * i) * kKeys + lane;
    return (i < my && lane < kKeys && key < k1) ? __ldg(table + block_of(pos0 + key)) : -1;
  };
  uint8_t* ring = smem + warp * ST * GM::kStage;
  const int key_sub = lane >> 3, chunk_sub = lane & 7;
  auto issue = [&](int i, int blk) {
    if (i < my) {
      uint8_t* st = ring + (i % ST) * GM::kStage;
      const uint32_t sk = smem_u32(st), sv = sk + kKeys * RB;
      const int key = k0 + (warp + kWarps * i) * kKeys + lane;
      int rec_l = -1;  // record of key `lane`, -1: none
      if (lane < kKeys && key < k1) {
        const int pos = pos0 + key;
        const int64_t slot = static_cast<int64_t>(blk) * bsz + (pos - block_of(pos) * bsz);
        if (blk < 0 || slot >= a.num_slots) {
          if (a.dev_status != nullptr) atomicOr(a.dev_status, QKV_DEV_BAD_INDEX);
        } else {
          rec_l = static_cast<int>(slot) * H + h;  // the host keeps num_slots * H below 2^31
        }
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, rec_l >= 0);
      if (lane == 0) sts32(sk + GM::kMask, mask);
      if (!F::kInline) {
        // four keys per instruction, one 128 B line of each; a masked key zero-fills its rows
#pragma unroll
        for (int t = 0; t < kKeys / 4; ++t) {
          const int kr = key_sub + 4 * t;
          const int rec = __shfl_sync(0xffffffffu, rec_l, kr);
          const int nb = rec >= 0 ? 16 : 0;
          const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(max(rec, 0))) * RB;
#pragma unroll
          for (int u = 0; u < CH / 8; ++u) {
            const int ch = chunk_sub + 8 * u;
            const uint32_t d = kr * RB + ((ch ^ swz<FMT>(kr)) << 4);
            cp_async16(sk + d, a.k_cache + off + 16 * ch, nb);
            cp_async16(sv + d, a.v_cache + off + 16 * ch, nb);
          }
        }
        if (F::kInt8 && lane < kKeys) {
          cp_async4(sk + GM::kScales + 4 * lane, a.k_scale_tok + max(rec_l, 0), rec_l >= 0 ? 4 : 0);
          cp_async4(sk + GM::kScales + 4 * (kKeys + lane), a.v_scale_tok + max(rec_l, 0), rec_l >= 0 ? 4 : 0);
        }
      } else {
        // inline records sit on 4 B boundaries: 4 B copies, one key per instruction
#pragma unroll 4
        for (int kr = 0; kr < kKeys; ++kr) {
          const int rec = __shfl_sync(0xffffffffu, rec_l, kr);
          const int nb = rec >= 0 ? 4 : 0;
          const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(max(rec, 0))) * GM::kGlobalRow;
#pragma unroll
          for (int u = 0; u < HD / 128; ++u) {
            const int w = lane + 32 * u;
            const uint32_t d = kr * RB + (((w >> 2) ^ swz<FMT>(kr)) << 4) + 4 * (w & 3);
            cp_async4(sk + d, a.k_cache + off + 4 * w, nb);
            cp_async4(sv + d, a.v_cache + off + 4 * w, nb);
          }
        }
        if (lane < kKeys) {
          const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(max(rec_l, 0))) * GM::kGlobalRow + HD;
          cp_async4(sk + GM::kScales + 4 * lane, a.k_cache + off, rec_l >= 0 ? 4 : 0);
          cp_async4(sk + GM::kScales + 4 * (kKeys + lane), a.v_cache + off, rec_l >= 0 ? 4 : 0);
        }
      }
    }
    cp_async_commit();
  };

  int blk = load_blk(0);
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) {
    const int next = load_blk(i + 1);
    issue(i, blk);
    blk = next;
  }

  // ---------------- stage the query: each warp four pairs; bytes pools in the fragments' dim order
  uint8_t* sQ = smem + GM::kArea;
  for (int i = warp * (kPairs / kWarps); i < (warp + 1) * (kPairs / kWarps); ++i) {
    const bool in = sRow[i] >= 0;
    const uint16_t* src = a.q + (in ? static_cast<int64_t>(sRow[i]) * a.q_stride : 0) + static_cast<int64_t>(in ? sHead[i] : 0) * HD;
    constexpr int kPer = HD / 32;  // dims per lane: 4 or 8
    uint32_t w[kPer / 2];
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) w[k] = 0u;
    if (in) {
      if (kPer == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + lane);
        w[0] = v.x, w[1] = v.y, w[kPer / 2 - 2] = v.z, w[kPer / 2 - 1] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + lane);
        w[0] = v.x, w[1] = v.y;
      }
    }
    uint8_t* row = sQ + i * GM::kQRow;
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
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
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
    if (lane == 0) sFac[i] = fac;
  }
  __syncthreads();

  float o[HD / 8][4];
#pragma unroll
  for (int t = 0; t < HD / 8; ++t)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[t][k] = 0.f;
  float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int eu = -120;  // int8: the accumulators hold values times 2^-eu
  const float fac[2] = {sFac[hn], sFac[hn + 8]};
  const int own[2] = {sOwn[hn], sOwn[hn + 8]};
  const int row_of[2] = {sRow[hn], sRow[hn + 8]};
  const uint32_t qa = smem_u32(sQ) + hn * GM::kQRow, qb = qa + 8 * GM::kQRow;
  int kr[2];  // tile rows of this lane's K fragments
  kr[0] = key_of<FMT>(0, hn);
  kr[1] = key_of<FMT>(1, hn);

#pragma unroll 1
  for (int i = 0; i < my; ++i) {
    const int next = load_blk(i + ST);
    cp_async_wait<ST - 2>();
    __syncwarp();
    const uint32_t sk = smem_u32(ring + (i % ST) * GM::kStage), sv = sk + kKeys * RB;
    const uint32_t mask = lds32(sk + GM::kMask);

    // ---- logits: two N-tiles of eight keys, two chains each
    float s[2][2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[n][0][k] = s[n][1][k] = 0.f;
    if (F::kBytes) {
#pragma unroll
      for (int jb = 0; jb < HD / 64; ++jb) {
        uint4 kw[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) kw[n] = lds128(sk + kr[n] * RB + (((4 * jb + c) ^ swz<FMT>(kr[n])) << 4));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t qo = 128 * jb + 32 * c + 16 * half;
          const uint4 x = lds128(qa + qo), y = lds128(qb + qo);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t af[4] = {w ? x.z : x.x, w ? y.z : y.x, w ? x.w : x.y, w ? y.w : y.y};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint32_t kk = half ? (w ? kw[n].w : kw[n].z) : (w ? kw[n].y : kw[n].x);
              uint32_t b0, b1;
              if (F::kInt8) {
                b0 = i8pair_to_f16x2(kk);
                b1 = i8pair_to_f16x2(kk >> 8);
              } else {
                b0 = e4m3pair_to_f16x2(kk);
                b1 = e4m3pair_to_f16x2(kk >> 16);
              }
              mma_f16(s[n][w], af, b0, b1);
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int jb = 0; jb < HD / 32; ++jb) {
        uint4 kw[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) kw[n] = lds128(sk + kr[n] * RB + (((4 * jb + c) ^ swz<FMT>(kr[n])) << 4));
        const uint4 x = lds128(qa + 64 * jb + 16 * c), y = lds128(qb + 64 * jb + 16 * c);
        const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (F::kBf16) {
            mma_bf16(s[n][0], a0, kw[n].x, kw[n].y);
            mma_bf16(s[n][1], a1, kw[n].z, kw[n].w);
          } else {
            mma_f16(s[n][0], a0, kw[n].x, kw[n].y);
            mma_f16(s[n][1], a1, kw[n].z, kw[n].w);
          }
        }
      }
    }

    // ---- softmax step. Lane's columns: keys key_of(n, 2c + {0, 1}); rows hn, hn + 8
    const int base = k0 + (warp + kWarps * i) * kKeys;
    float y[2][2][2];  // [pair][n][column]
    float vs[2][2];    // int8: V scales of the lane's keys, times 2^-eu below
    float vmax = 0.f;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int key = key_of<FMT>(n, 2 * c + k);
        const bool valid = (mask >> key) & 1;
        float ks = 1.f;
        if (F::kInt8) {
          ks = __uint_as_float(lds32(sk + GM::kScales + 4 * key));
          vs[n][k] = __uint_as_float(lds32(sk + GM::kScales + 4 * (kKeys + key)));
          vmax = fmaxf(vmax, fabsf(vs[n][k]));
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float z = (s[n][0][2 * p + k] + s[n][1][2 * p + k]) * ks * fac[p];
          y[p][n][k] = (valid && (!OWN || base + key < own[p])) ? z : -INFINITY;
        }
      }
    }
    float tm[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      tm[p] = fmaxf(fmaxf(y[p][0][0], y[p][0][1]), fmaxf(y[p][1][0], y[p][1][1]));
      tm[p] = fmaxf(tm[p], __shfl_xor_sync(0xffffffffu, tm[p], 1));
      tm[p] = fmaxf(tm[p], __shfl_xor_sync(0xffffffffu, tm[p], 2));
    }
    int eu_new = eu;
    if (F::kInt8) {
      vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 1));
      vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2));
      const int e = min(120, static_cast<int>(__float_as_uint(vmax) >> 23) - 126);  // vmax < 2^e
      if (e > eu) eu_new = min(120, e + kEuHeadroom);
    }
    // a first finite logit has no reference to be compared with: M = -inf lies below any
    const bool raise0 = tm[0] > M[0] + kTau, raise1 = tm[1] > M[1] + kTau;
    if (__any_sync(0xffffffffu, raise0 || raise1 || eu_new != eu)) {
      float f[2];
      const float down = F::kInt8 ? pow2f(max(eu - eu_new, -126)) : 1.f;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const bool up = p ? raise1 : raise0;
        const float m = up ? tm[p] : M[p];
        const float al = (up && M[p] != -INFINITY) ? fast_exp2(M[p] - m) : 1.f;
        M[p] = m;
        l[p] *= al;
        f[p] = al * down;
      }
#pragma unroll
      for (int t = 0; t < HD / 8; ++t) {
        o[t][0] *= f[0];
        o[t][1] *= f[0];
        o[t][2] *= f[1];
        o[t][3] *= f[1];
      }
      eu = eu_new;
    }
    const float vdown = F::kInt8 ? pow2f(-eu) : 1.f;
    uint32_t pa[4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float ref = M[p] == -INFINITY ? 0.f : M[p] - (F::kBf16 ? 0.f : kPShift);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float e0 = fast_exp2(y[p][n][0] - ref), e1 = fast_exp2(y[p][n][1] - ref);
        l[p] += e0 + e1;
        if (F::kInt8) {
          // a masked key's scale may be anything (0 x inf): its p stays 0
          e0 = y[p][n][0] == -INFINITY ? 0.f : e0 * (vs[n][0] * vdown);
          e1 = y[p][n][1] == -INFINITY ? 0.f : e1 * (vs[n][1] * vdown);
        }
        pa[2 * n + p] = F::kBf16 ? pack_bf162(e0, e1) : pack_half2(e0, e1);
      }
    }

    // ---- p V. Rows of different lengths in one tile: a key that one row sees and another does not
    // may hold anything there (0 x NaN), so such a tile goes row by row, each with its own keys only, and
    // only that row's sums are taken.
    const bool ragged = OWN && !F::kInt8 && nrows > 1 && base + kKeys > own_min;
    const int passes = ragged ? nrows : 1;
#pragma unroll 1
    for (int t = 0; t < passes; ++t) {
      uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // halves of b0 / b1 (the lane's keys) that the row sees
      if (ragged) {
        const int n = sOwn[t * G];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          keep[k] = (base + key_of<FMT>(k, 2 * c) < n ? 0x0000ffffu : 0u) | (base + key_of<FMT>(k, 2 * c + 1) < n ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int q = 0; q < HD / 32; ++q) {
        uint32_t v[8];  // b0, b1 of four N-tiles of eight dims
        if (F::kBytes) {
          // matrices of 16 keys x 16 dims: chunk 2q for lanes 0-15's addresses, 2q + 1 for the others
          uint32_t m[4];
          const int r = lane & 15;
          ldmatrix_x2_trans_b8(sv + r * RB + (((2 * q + (lane >> 4)) ^ swz<FMT>(r)) << 4), m[0], m[1], m[2], m[3]);
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
            const uint32_t addr = sv + r * RB + ((ch ^ swz<FMT>(r)) << 4);
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                         : "=r"(v[4 * k]), "=r"(v[4 * k + 1]), "=r"(v[4 * k + 2]), "=r"(v[4 * k + 3])
                         : "r"(addr));
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float* acc = o[4 * q + k];
          if (!ragged) {
            if (F::kBf16)
              mma_bf16(acc, pa, v[2 * k], v[2 * k + 1]);
            else
              mma_f16(acc, pa, v[2 * k], v[2 * k + 1]);
          } else {
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (F::kBf16)
              mma_bf16(x, pa, v[2 * k] & keep[0], v[2 * k + 1] & keep[1]);
            else
              mma_f16(x, pa, v[2 * k] & keep[0], v[2 * k + 1] & keep[1]);
            const int row = static_cast<int>(r0) + t;
            if (row_of[0] == row) acc[0] += x[0], acc[1] += x[1];
            if (row_of[1] == row) acc[2] += x[2], acc[3] += x[3];
          }
        }
      }
    }
    __syncwarp();
    issue(i + ST - 1, blk);
    blk = next;
  }

  // ---------------- join the four warps
  cp_async_wait<0>();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    l[p] += __shfl_xor_sync(0xffffffffu, l[p], 1);
    l[p] += __shfl_xor_sync(0xffffffffu, l[p], 2);
    if (c == 0) {
      sM[warp][hn + 8 * p] = M[p];
      sL[warp][hn + 8 * p] = l[p];
    }
  }
  if (lane == 0) sEu[warp] = eu;
  __syncthreads();  // every ring is drained
  float* sO = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int t = 0; t < HD / 8; ++t)
#pragma unroll
    for (int p = 0; p < 2; ++p)
      *reinterpret_cast<float2*>(sO + (warp * kPairs + hn + 8 * p) * GM::kORow + 8 * t + 2 * c) =
          make_float2(o[t][2 * p], o[t][2 * p + 1]);
  __syncthreads();
  const bool direct = a.o_part == nullptr;  // the only part: its result is the row's
  for (int i = warp; i < kPairs; i += kWarps) {
    const int row = sRow[i];
    if (row < 0) continue;
    bool empty = false;
    if (direct) {
      const int state = row_state(a, row, lane == 0 && sHead[i] == 0);
      if (state == kPadRow) continue;
      empty = state == kEmptyRow;
    }
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sM[w][i]);
    const float ref = m == -INFINITY ? 0.f : m;
    float f[kWarps], sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float al = fast_exp2(sM[w][i] - ref);  // 2^-inf = 0 for a warp without keys
      sum += al * sL[w][i];
      f[w] = F::kInt8 ? al * pow2f(sEu[w]) : al;
    }
    const bool any = !empty && (m != -INFINITY || sum != sum);
    const float inv = any ? (direct && FMT == QKV_E4M3 ? a.v_scale_layer : 1.f) / sum : 0.f;
    const int64_t at = static_cast<int64_t>(row) * a.num_q_heads + sHead[i];
    const int64_t part_at = (static_cast<int64_t>(OWN ? a.prefix_parts + part : part) * a.rows) * a.num_q_heads + at;
    if (lane == 0) {
      const float v = any ? (m - (F::kBf16 ? 0.f : kPShift) + log2f(sum)) * kLn2 : -INFINITY;
      if (!direct) a.lse_part[part_at] = v;
      else if (a.lse != nullptr) a.lse[at] = v;
    }
    if (!any && !direct) continue;
#pragma unroll
    for (int d = 4 * lane; d < HD; d += 128) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(sO + (w * kPairs + i) * GM::kORow + d);
        if (f[w] != 0.f) {
          acc.x += f[w] * x.x, acc.y += f[w] * x.y, acc.z += f[w] * x.z, acc.w += f[w] * x.w;
        }
      }
      acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
      if (direct) {
        *reinterpret_cast<uint2*>(a.out + at * HD + d) = make_uint2(round2(a.q_f16, acc.x, acc.y), round2(a.q_f16, acc.z, acc.w));
      } else {
        *reinterpret_cast<float4*>(a.o_part + part_at * HD + d) = acc;
      }
    }
  }
}

template <int FMT, int HD, bool OWN>
cudaError_t launch_mma(const PrefixArgs& a, cudaStream_t stream) {
  constexpr int smem = Geom<FMT, HD>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(prefix_mma_kernel<FMT, HD, OWN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prefix_mma_kernel<FMT, HD, OWN><<<static_cast<unsigned>(OWN ? a.own_items : a.prefix_items), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_mma(const PrefixArgs& a, bool own, cudaStream_t stream) {
  if (a.head_dim == 256) return own ? launch_mma<FMT, 256, true>(a, stream) : launch_mma<FMT, 256, false>(a, stream);
  return own ? launch_mma<FMT, 128, true>(a, stream) : launch_mma<FMT, 128, false>(a, stream);
}

}  // namespace prefix
}  // namespace qkv
