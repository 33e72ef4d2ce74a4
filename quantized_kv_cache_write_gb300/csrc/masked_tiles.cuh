// The work list of qkv_masked_attn's tcgen05 tiles. A tile is up to tile_rows consecutive rows of one sequence (cut every
// tile_rows rows from where the sequence changes or a row's range lies apart from that of the row before) and the key blocks
// that any of them sees. A KV head's work is its tiles' costs: a tile's blocks, and tile_cost more for what it costs besides them (its
// queries, its first and last products, its output). The kernel that makes the list runs first, a block for each chunk of
// rows; the teams of the tile kernel then each take an equal contiguous share of all heads' work, so that causal, ragged and
// windowed rows balance without the host knowing them. A tile that one team has whole is written out by it; of one that
// teams share each leaves a partial result, which a last kernel joins. A team has at most two of those: the end of
// a tile that a team before began (place 0), and the beginning of one that it does not finish (place 1).
// Measured, 8192 causal rows x 16 heads of 256, bf16: shares of equal blocks left the team with the shortest tiles at work
// for 834 us, the others for 415.
#pragma once

#include "prefix_attn.cuh"

namespace qkv {
namespace prefix {

constexpr int kPlanThreads = 1024;  // rows of a chunk, at most: a multiple of tile_rows

struct MaskedTile {
  uint32_t first;      // its work within its chunk
  int row0, nrows;     // its rows
  int seq;
  int lo, hi;          // positions that any of its rows sees (none: both 0)
  int all_lo, all_hi;  // positions that every row sees that sees anything
};
// The list: every chunk's work and number of tiles; then the chunks' tiles, kPlanThreads + 1 places each, a last entry's
// `first` being the chunk's work.
struct MaskedChunk {
  uint32_t work, tiles;
};
// What the tile kernel leaves for the join, one for each team: the tile that it begins and does not finish, and the teams that
// have a part of it (0: there is none).
struct MaskedJoin {
  int row0, nrows, h;
  uint32_t parts;
};
__host__ __device__ inline int64_t plan_chunk_rows(int tile_rows) { return kPlanThreads / tile_rows * tile_rows; }
__host__ __device__ inline int64_t plan_chunks(int64_t rows, int tile_rows) {
  return (rows + plan_chunk_rows(tile_rows) - 1) / plan_chunk_rows(tile_rows);
}
__device__ __forceinline__ const MaskedChunk* plan_chunk(const PrefixArgs& a) { return static_cast<const MaskedChunk*>(a.plan); }
__device__ __forceinline__ const MaskedTile* plan_tiles(const PrefixArgs& a, int chunk) {
  return reinterpret_cast<const MaskedTile*>(static_cast<const uint8_t*>(a.plan) + a.plan_tiles_at) + static_cast<int64_t>(chunk) * (kPlanThreads + 1);
}
// The joins lie before the tiles.
__device__ __forceinline__ MaskedJoin* plan_join(const PrefixArgs& a, uint32_t team) {
  return reinterpret_cast<MaskedJoin*>(static_cast<uint8_t*>(a.plan) + a.plan_tiles_at) - a.umma_teams + team;
}

// The teams' shares: each of the first `extra` has one unit of work more.
struct Shares {
  uint64_t share, extra;
  __device__ __forceinline__ Shares(uint64_t total, uint32_t teams) : share(total / teams), extra(total % teams) {}
  __device__ __forceinline__ uint64_t first(uint64_t team) const { return team * share + min(team, extra); }
  __device__ __forceinline__ uint64_t of(uint64_t team) const { return share + (team < extra ? 1 : 0); }
};

// A KV head's work; the warp's lanes together.
__device__ __forceinline__ uint64_t plan_work(const PrefixArgs& a) {
  uint64_t sum = 0;
  for (int c = threadIdx.x & 31; c < a.plan_chunks; c += 32) sum += plan_chunk(a)[c].work;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return sum;
}
// The tile that holds unit `rem` of a KV head's work (0 <= rem < plan_work), and its place in it; the warp's lanes together.
struct PlanPlace {
  int chunk, tile;
  uint32_t into;  // units of the tile before
};
__device__ __forceinline__ PlanPlace plan_find(const PrefixArgs& a, uint64_t rem) {
  PlanPlace p = {0, 0, 0};
  uint64_t before = 0;  // units of the chunks before
  const int lane = threadIdx.x & 31;
  uint64_t base = 0;
  for (int c0 = 0; c0 < a.plan_chunks; c0 += 32) {
    const uint64_t own = c0 + lane < a.plan_chunks ? plan_chunk(a)[c0 + lane].work : 0;
    uint64_t sum = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += x;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + sum > rem);
    if (past != 0) {
      const int at = __ffs(past) - 1;
      p.chunk = c0 + at;
      before = base + __shfl_sync(0xffffffffu, sum - own, at);
      break;
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  const MaskedTile* tiles = plan_tiles(a, p.chunk);
  const uint32_t in = static_cast<uint32_t>(rem - before);
  const int n = static_cast<int>(plan_chunk(a)[p.chunk].tiles);
  // the last tile that starts there or before, in two steps of 32 (a chunk has at most 1024): ten dependent loads by halves
  int lo = 0;
  for (int step = 32; step > 0; step /= 32) {
    const int at = lo + lane * step;
    lo += step * (31 - __clz(__ballot_sync(0xffffffffu, at < n && tiles[min(at, n - 1)].first <= in)));
  }
  p.tile = lo;
  p.into = in - tiles[lo].first;
  return p;
}

// A team's walk through its share, a segment at a time: its part of the blocks of one tile of one KV head. One warp of each
// SM walks and publishes the segments to the other roles (SegWord); a walk in every role costs each of them a thousand
// cycles of loads per segment, and the instruction cache a copy.
struct MaskedWalk {
  uint32_t left;    // work still to do
  uint32_t share, extra;  // the teams' shares
  uint32_t skip;    // work of the next tile that a team before has
  int chunk, i, h;  // the next tile and its KV head
  uint32_t team;
  __device__ __forceinline__ void begin(const PrefixArgs& a, uint32_t of_team) {
    team = of_team;
    const uint64_t work = plan_work(a);
    const Shares s(work * a.num_kv_heads, a.umma_teams);
    left = static_cast<uint32_t>(s.of(team));  // the host keeps a share below 2^32
    share = static_cast<uint32_t>(s.share), extra = static_cast<uint32_t>(s.extra);
    skip = 0, chunk = 0, i = 0, h = 0;
    if (left == 0) return;
    const uint64_t u = s.first(team);
    h = static_cast<int>(u / work);
    const PlanPlace p = plan_find(a, u - h * work);
    chunk = p.chunk, i = p.tile, skip = p.into;
  }
  // how many of the teams after this one `rest` units of work go to
  __device__ __forceinline__ uint32_t teams_of(uint32_t rest) const {
    const uint32_t more = max(extra, team + 1) - (team + 1);  // of them have a unit more
    const uint64_t theirs = static_cast<uint64_t>(more) * (share + 1);
    return rest <= theirs ? (rest + share) / (share + 1) : more + (rest - static_cast<uint32_t>(theirs) + share - 1) / share;
  }
};
// A published segment, in shared memory: its first block and the last one's next (equal: there is none; blocks are numbered
// from position 0), the tile's rows, its KV head, its place among the partial results (-1: the tile is whole), what all
// of its rows see, and where the tile's entry is.
enum SegWord { kSegB0, kSegB1, kSegRow0, kSegRows, kSegHead, kSegPart, kSegAllLo, kSegAllHi, kSegChunk, kSegTile, kSegWords = 12 };
constexpr int kSegRing = 4;  // the softmax holds a segment while it asks for the next one

}  // namespace prefix
}  // namespace qkv
