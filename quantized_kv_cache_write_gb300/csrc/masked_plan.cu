// The work list of qkv_masked_attn's tcgen05 tiles, and the join of the tiles that teams share (masked_tiles.cuh).
#include "prefix_umma.cuh"

namespace qkv {
namespace prefix {
namespace {

constexpr int kPlanWarps = kPlanThreads / 32;

// Inclusive sum over the block's threads; `total` is the last one's.
__device__ __forceinline__ uint32_t scan(uint32_t x, uint32_t* sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t s = sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) x += sums[warp - 1];
  total = sums[kPlanWarps - 1];
  __syncthreads();
  return x;
}

// A chunk of rows per block, a thread per row.
__global__ void __launch_bounds__(kPlanThreads) masked_plan_kernel(const PrefixArgs a) {
  __shared__ int sSeq[kPlanThreads], sLo[kPlanThreads], sHi[kPlanThreads];
  __shared__ int tLo[kPlanThreads], tHi[kPlanThreads], tAllLo[kPlanThreads], tAllHi[kPlanThreads], tRow[kPlanThreads], tRows[kPlanThreads];
  __shared__ uint32_t sums[kPlanWarps];
  let_next_start();
  const int tid = threadIdx.x, T = a.tile_rows, KB = a.block_keys, step = static_cast<int>(plan_chunk_rows(T));
  MaskedChunk* chunk = static_cast<MaskedChunk*>(a.plan) + blockIdx.x;
  MaskedTile* tiles = const_cast<MaskedTile*>(plan_tiles(a, static_cast<int>(blockIdx.x)));
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * step, row = r0 + tid;
  const bool there = tid < step && row < a.rows;
  RowRange x = {kPadRow, 0, 0, 0, 0};
  int seq = -1;
  if (there) x = row_range(a, row, true), seq = __ldg(a.row_seq + row);
  const bool live = x.state != kPadRow, sees = x.lo < x.hi;
  sSeq[tid] = live ? seq : -1, sLo[tid] = x.lo, sHi[tid] = x.hi;
  tLo[tid] = INT_MAX, tHi[tid] = 0, tAllLo[tid] = 0, tAllHi[tid] = INT_MAX, tRows[tid] = 0;
  __syncthreads();
  // A run: rows of one sequence one after the other whose ranges meet. Its tiles count from its first row: 8 x 5 rows
  // whose tiles have up to 16 are 8 tiles, and ten if they were cut at every 16th row (8 x 5 rows x 16 heads of 256 behind
  // 60000 bf16 keys: 164 us, 124 so).
  bool begins = live;
  if (live && tid > 0) {
    const int lo = sLo[tid - 1], hi = sHi[tid - 1];
    const bool apart = sees && lo < hi && max(lo, x.lo) > min(hi, x.hi);
    begins = sSeq[tid - 1] != seq || apart;  // a padding row before: another sequence (-1)
  }
  const uint32_t begin_bits = __ballot_sync(0xffffffffu, begins), upto = begin_bits & (0xffffffffu >> (31 - (tid & 31)));
  if ((tid & 31) == 0) sums[tid >> 5] = begin_bits != 0 ? (tid | 31) - __clz(begin_bits) : 0;
  __syncthreads();
  int run = static_cast<int>(__reduce_max_sync(0xffffffffu, (tid & 31) < (tid >> 5) ? sums[tid & 31] : 0));
  if (upto != 0) run = (tid | 31) - __clz(upto);
  const bool first = live && (tid - run) % T == 0;
  __syncthreads();
  uint32_t n;
  const uint32_t i = scan(first ? 1 : 0, sums, n) - 1;  // the row's tile of these
  // a tile's rows of the warp to the first of them, and from there into the tile
  const int tile = live ? static_cast<int>(i) : -1, lane = tid & 31;
  int rows = 1, lo = sees ? x.lo : INT_MAX, hi = x.hi, all_lo = x.lo, all_hi = sees ? x.hi : INT_MAX;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o_tile = __shfl_down_sync(0xffffffffu, tile, off), o_rows = __shfl_down_sync(0xffffffffu, rows, off);
    const int o_lo = __shfl_down_sync(0xffffffffu, lo, off), o_hi = __shfl_down_sync(0xffffffffu, hi, off);
    const int o_all_lo = __shfl_down_sync(0xffffffffu, all_lo, off), o_all_hi = __shfl_down_sync(0xffffffffu, all_hi, off);
    if (lane + off < 32 && o_tile == tile) {
      rows += o_rows, lo = min(lo, o_lo), hi = max(hi, o_hi), all_lo = max(all_lo, o_all_lo), all_hi = min(all_hi, o_all_hi);
    }
  }
  const int before = __shfl_up_sync(0xffffffffu, tile, 1);
  if (live && first) tRow[i] = static_cast<int>(row);
  if (live && (lane == 0 || before != tile)) {
    atomicAdd(tRows + i, rows);
    atomicMin(tLo + i, lo), atomicMax(tHi + i, hi);
    atomicMax(tAllLo + i, all_lo), atomicMin(tAllHi + i, all_hi);
  }
  __syncthreads();
  MaskedTile t = {};
  uint32_t cost = 0, sum;
  if (tid < n) {
    t.row0 = tRow[tid], t.nrows = tRows[tid], t.seq = sSeq[t.row0 - r0];
    if (tHi[tid] > 0) t.lo = tLo[tid], t.hi = tHi[tid], t.all_lo = tAllLo[tid], t.all_hi = tAllHi[tid];
    // rows that see nothing have a block without keys
    cost = a.tile_cost + max(1, (t.hi + KB - 1) / KB - t.lo / KB);
  }
  t.first = scan(cost, sums, sum) - cost;  // the host keeps a chunk's work below 2^32
  if (tid < n) tiles[tid] = t;
  if (tid == 0) {
    tiles[n].first = sum;
    chunk->work = sum, chunk->tiles = n;
  }
}

// Four values of a part, or zeros; issued here, however late they are used.
__device__ __forceinline__ float4 load_part(const float4* p, uint32_t there) {
  float4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
      " @p ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=&f"(v.x), "=&f"(v.y), "=&f"(v.z), "=&f"(v.w)
      : "l"(p), "r"(there)
      : "memory");
  return v;
}

// A tile that teams share: its (row, head) pairs, one warp each, from the parts that the teams left.
constexpr int kJoinWarps = 8;
template <int HD>
__global__ void __launch_bounds__(32 * kJoinWarps) masked_join_kernel(const PrefixArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  await_previous();
  const uint32_t team = blockIdx.x;
  const int4 t = __ldcg(reinterpret_cast<const int4*>(plan_join(a, team)));
  const int row0 = t.x, nrows = t.y, h = t.z;
  const uint32_t parts = static_cast<uint32_t>(t.w);
  const int G = a.num_q_heads / a.num_kv_heads;
  const int flat = static_cast<int>(blockIdx.y) * kJoinWarps + warp;
  if (parts == 0 || flat >= nrows * G) return;
  const int64_t row = row0 + flat / G, at = row * a.num_q_heads + h * G + flat % G;
  // part i: place 1 of the team that begins, place 0 of those after it
  auto place = [&](uint32_t i) -> int64_t { return static_cast<int64_t>(i == 0 ? 2 * team + 1 : 2 * (team + i)) * a.umma_pairs + flat; };
  float m = -INFINITY;
  bool nan = false;
  for (uint32_t i = lane; i < parts; i += 32) {
    const float v = __ldcg(a.lse_part + place(i));
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
  // a part without keys wrote no values; one with keys counts, its values may be NaN. Eight parts' values are in flight at
  // once
  constexpr uint32_t kAtOnce = 8;
  for (uint32_t i0 = 0; any && i0 < parts; i0 += 32) {
    const float l = i0 + lane < parts ? __ldcg(a.lse_part + place(i0 + lane)) : -INFINITY;
    const uint32_t some = __ballot_sync(0xffffffffu, l != -INFINITY);
    const float w = l != -INFINITY ? expf(l - ref) : 0.f;
    sum += w;
    for (uint32_t i = 0; i < min(parts - i0, 32u); i += kAtOnce) {
      float4 x[kAtOnce][kVec];
#pragma unroll
      for (uint32_t k = 0; k < kAtOnce; ++k) {
        const float4* src = reinterpret_cast<const float4*>(a.o_part + place(i0 + i + k) * HD);
#pragma unroll
        for (int v = 0; v < kVec; ++v) x[k][v] = load_part(src + lane + 32 * v, (some >> (i + k)) & 1);
      }
#pragma unroll
      for (uint32_t k = 0; k < kAtOnce; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, i + k);
#pragma unroll
        for (int v = 0; v < kVec; ++v) acc[v].x += wk * x[k][v].x, acc[v].y += wk * x[k][v].y, acc[v].z += wk * x[k][v].z, acc[v].w += wk * x[k][v].w;
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const float f = any ? a.merge_scale / sum : 0.f;
#pragma unroll
  for (int v = 0; v < kVec; ++v)
    *reinterpret_cast<uint2*>(a.out + at * HD + 4 * (lane + 32 * v)) =
        make_uint2(round2(a.q_f16, acc[v].x * f, acc[v].y * f), round2(a.q_f16, acc[v].z * f, acc[v].w * f));
  if (lane == 0 && a.lse != nullptr) {
    const RowRange x = row_range(a, row, false);
    float far = 0.f;
    if (a.slopes != nullptr && x.pos != x.near) far = -__ldg(a.slopes + h * G + flat % G) * fabsf(static_cast<float>(x.pos - x.near));
    a.lse[at] = any ? ref + logf(sum) + far : -INFINITY;
  }
}

template <int HD>
cudaError_t launch_join(const PrefixArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.umma_teams, (a.umma_pairs + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, masked_join_kernel<HD>, a);
}

}  // namespace
}  // namespace prefix

size_t masked_plan_tiles_at(int64_t rows, int tile_rows, uint32_t teams) {
  return (static_cast<size_t>(prefix::plan_chunks(rows, tile_rows)) * sizeof(prefix::MaskedChunk) + teams * sizeof(prefix::MaskedJoin) + 31) / 32 * 32;
}
size_t masked_plan_bytes(int64_t rows, int tile_rows, uint32_t teams) {
  return masked_plan_tiles_at(rows, tile_rows, teams) +
         static_cast<size_t>(prefix::plan_chunks(rows, tile_rows)) * (prefix::kPlanThreads + 1) * sizeof(prefix::MaskedTile);
}
int masked_plan_chunks(int64_t rows, int tile_rows) { return static_cast<int>(prefix::plan_chunks(rows, tile_rows)); }
cudaError_t launch_masked_plan(const PrefixArgs& a, cudaStream_t stream) {
  prefix::masked_plan_kernel<<<static_cast<unsigned>(a.plan_chunks), prefix::kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_masked_join(const PrefixArgs& a, cudaStream_t stream) {
  return a.head_dim == 256 ? prefix::launch_join<256>(a, stream) : prefix::launch_join<128>(a, stream);
}

}  // namespace qkv
