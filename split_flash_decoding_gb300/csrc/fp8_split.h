// fp8_split.h -- arithmetic of the 8-bit decode's balanced split (fp8_items.cuh has
// the whole of it): plain integers, the same on the device and on the host.
#pragma once

#ifdef __CUDACC__
#define ATTN_SPLIT_FN __host__ __device__ __forceinline__
#else
#define ATTN_SPLIT_FN inline
#endif

namespace attn {

// In eighths of a tile of up to four columns: the cost of a tile of 16 columns, and
// of opening a unit.
constexpr int kFp8MostTileCost = 11;
constexpr int kFp8UnitCost = 32;

// Cost of a tile whose queries (rows x heads) fill this many columns.
ATTN_SPLIT_FN int fp8_cost_of_columns(int columns) {
    const int chunks = (columns + 3) / 4;
    return 7 + (chunks < 1 ? 1 : chunks > 4 ? 4 : chunks);
}

// Groups that take part, of the grid's: at most one per tile, and no more than leave
// each at least the cost of the dearest tile.  W: the cost of all units, T: their
// tiles.  A group takes the tiles that start in its range, and ranges are W / C long
// (rounded down or up), so each one that lies between a unit's first and last tile
// then has a tile of that unit: the merge reads the slots of all of them.  (With one
// cost for all tiles the second bound is never the smaller, as W / cost >= T.)
ATTN_SPLIT_FN int fp8_split_groups(int groups, int T, int W, int dearest) {
    const int wide = W / dearest;
    const int C = groups < T ? groups : T;
    return C < wide ? C : wide < 1 ? 1 : wide;
}

// First position of group c: c W / C, in 32 bits (c <= C, and C C fits).
ATTN_SPLIT_FN int first_position(int c, int W, int C) {
    const int q = W / C;
    return c * q + c * (W - q * C) / C;
}

// Group that a position belongs to.
ATTN_SPLIT_FN int group_of_position(int y, int W, int C) {
    return static_cast<int>((static_cast<long long>(y + 1) * C - 1) / W);
}

}  // namespace attn
