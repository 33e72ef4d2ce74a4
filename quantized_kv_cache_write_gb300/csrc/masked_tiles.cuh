// The work list of qkv_masked_attn's tcgen05 tiles. A tile is up to tile_rows consecutive rows of one sequence (cut at
// multiples of tile_rows, where the sequence changes, and between rows whose ranges lie apart) and the key blocks that any of
// them sees; a KV head's tiles by their blocks are its units. The kernel that makes the list runs first, on one SM; the
// teams of the tile kernel then each take an equal contiguous share of all heads' units, so that causal, ragged and
// windowed rows balance without the host knowing them. A tile that one team has whole is written out by it; of one that
// teams share each leaves a partial result, which a last kernel joins. A team has at most two of those: the end of
// a tile that the team before began (place 0), and the beginning of one that it does not finish (place 1).
#pragma once

#include "prefix_attn.cuh"

namespace qkv {
namespace prefix {

struct MaskedTile {
  uint64_t first;    // its first unit within a KV head
  int row0, nrows;   // its rows
  int seq;
  int lo, hi;        // positions that any of its rows sees (none: both 0)
  int all_lo, all_hi;  // positions that every row sees that sees anything
  int pad;
};
struct MaskedHead {
  uint64_t units;  // of a KV head
  uint32_t tiles;
  uint32_t pad;
};
// The list: the head, then the tiles and a last entry whose `first` is the number of units.
__device__ __forceinline__ const MaskedHead* plan_head(const PrefixArgs& a) { return static_cast<const MaskedHead*>(a.plan); }
__device__ __forceinline__ const MaskedTile* plan_tiles(const PrefixArgs& a) {
  return reinterpret_cast<const MaskedTile*>(plan_head(a) + 1);
}

// The teams' shares: each of the first `extra` has one unit more.
struct Shares {
  uint64_t share, extra;
  __device__ __forceinline__ Shares(uint64_t total, uint32_t teams) : share(total / teams), extra(total % teams) {}
  __device__ __forceinline__ uint64_t first(uint64_t team) const { return team * share + min(team, extra); }
  __device__ __forceinline__ uint64_t of(uint64_t team) const { return share + (team < extra ? 1 : 0); }
};

// A team's next segment: the part of its units that lies in one tile of one KV head. Blocks are numbered from position 0.
template <int KB>
struct MaskedSegment {
  uint32_t left;  // units still to do
  uint32_t skip;  // the first tile's units that the team before has
  int i, h;       // tile and KV head to come
  uint32_t tiles;
  MaskedTile t;
  int b0, b1, part;
  __device__ __forceinline__ void begin(const PrefixArgs& a, uint32_t team) {
    const MaskedHead head = *plan_head(a);
    tiles = head.tiles;
    const Shares s(head.units * a.num_kv_heads, a.umma_teams);
    left = static_cast<uint32_t>(s.of(team));  // the host keeps a share below 2^32
    skip = 0, i = 0, h = 0;
    if (left == 0) return;
    const uint64_t u = s.first(team);
    h = static_cast<int>(u / head.units);
    const uint64_t rem = u - h * head.units;
    int lo = 0, hi = static_cast<int>(tiles);  // the last tile that starts at rem or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (plan_tiles(a)[mid].first <= rem) lo = mid;
      else hi = mid;
    }
    i = lo;
    skip = static_cast<uint32_t>(rem - plan_tiles(a)[i].first);
  }
  __device__ __forceinline__ bool next(const PrefixArgs& a, uint32_t team) {
    if (left == 0) return false;
    t = plan_tiles(a)[i];
    const uint32_t nb = static_cast<uint32_t>(plan_tiles(a)[i + 1].first - t.first);
    const uint32_t n = min(left, nb - skip);
    b0 = t.lo / KB + static_cast<int>(skip);
    b1 = b0 + static_cast<int>(n);
    part = n == nb ? -1 : static_cast<int>(2 * team + (skip > 0 ? 0 : 1));
    left -= n;
    skip = 0;
    h_now = h;
    if (++i == static_cast<int>(tiles)) i = 0, ++h;
    return true;
  }
  int h_now;  // the segment's KV head
};

}  // namespace prefix
}  // namespace qkv
