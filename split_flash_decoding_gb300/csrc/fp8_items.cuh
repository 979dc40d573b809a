// fp8_items.cuh -- the work list of decode attention over an 8-bit cache: a
// balanced split whose CTAs walk the KV heads of a sequence side by side.
//
// The grid is cut into groups of H CTAs (H the largest power of two up to 8
// that divides the KV heads).  CTA x is member x % H of group x / H, and the
// members of a group take the same tiles of H consecutive KV heads: a token's
// codes of one head are only 128 bytes, and neighbouring heads' codes are
// neighbours in memory, so whole DRAM bursts and pages are read at about the
// same time.  (Heads dealt to CTAs one after the other, as the bf16 kernel does
// with its 256-byte rows, read 64 sequences of Llama-3-8B shapes at 114.9 us.)
//
// A unit is (sequence b, group of H heads).  The 128-key tiles of all units,
// concatenated, are dealt out in contiguous ranges of equal cost, in eighths of a
// tile's: a tile costs 8 + (chunks of four columns that the sequence's rows fill
// - 1), as the softmax of more columns takes longer (1 to 4 rows of 4 heads:
// 1.58, 1.77, 1.89 and 2.11 us a tile), and every unit is preceded by kFp8UnitCost
// (opening it: its queries, the pipeline refill, the epilogue).  Group c of C
// takes the tiles that start in [c W / C, (c + 1) W / C), W the cost of all; C is
// such that every group inside a unit gets one of its tiles (fp8_split_groups).
#pragma once

#include "cache_ops.h"
#include "ptx.cuh"

namespace attn {

struct Fp8Range {
    int x0, x1;            // this group's tiles of the concatenation
    int u0, u1;            // its first and last unit
    int groups;            // C: groups that take part
    int cost;              // W
    __device__ __forceinline__ int count() const { return x1 > x0 ? u1 - u0 + 1 : 0; }
};

struct Fp8Item {
    int b, kvh, L, start, end, ntiles;
    int unit, unit_tiles;
    int slot;              // partial slot
    bool first, direct;    // holds the unit's first tile; holds all of it
};

__device__ __forceinline__ int fp8_tiles(uint32_t len, uint32_t cap) {
    return max(static_cast<int>((min(len, cap) + kGqaTcTileKeys - 1) / kGqaTcTileKeys), 1);
}

// By the number of head groups, which usually is 1 (an integer division is some
// forty instructions, on the way to a CTA's first load).
__device__ __forceinline__ int by_groups(int x, int hg) { return hg == 1 ? x : x / hg; }

// Cost of a tile of sequence b.
__device__ __forceinline__ int fp8_tile_cost(const Fp8DecodeParams &p, int b) {
    if (!p.q_row_offsets) return fp8_cost_of_columns(p.group);
    const int rows = static_cast<int>(p.q_row_offsets[b + 1] - p.q_row_offsets[b]);
    return fp8_cost_of_columns(rows * p.group);
}

// cum[b].x: tiles of the concatenation before sequence b (head groups included),
// cum[b].y: their cost, b up to the batch; and this group's range.  Three warps, all
// lanes: warp 0 finds where the range begins, warp 1 where it ends, warp 2 writes
// cum.  (The host bounds the tiles of a call so that costs fit an int.)
__device__ __forceinline__ void fp8_build_items(const Fp8DecodeParams &p, int2 *cum, int warp,
                                                int lane, Fp8Range *out) {
    const int hg = p.head_groups;
    const uint32_t cap = uint32_t(p.max_kv_len);
    const int per_lane = (p.batch + 31) / 32;
    const int b0 = min(lane * per_lane, p.batch), b1 = min(b0 + per_lane, p.batch);
    int local = 0, cost = 0, dearest = 1;      // (a lane without sequences: 1)
    for (int b = b0; b < b1; ++b) {
        const uint32_t len = p.kv_len[b];
        if (len > cap && blockIdx.x == 0 && warp == 0) atomicOr(p.err, kErrBadLength);
        const int n = fp8_tiles(len, cap), tile = fp8_tile_cost(p, b);
        local += n * hg;
        cost += hg * (n * tile + kFp8UnitCost);
        dearest = max(dearest, tile);
    }
    int incl = local, cost_incl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        const int w = __shfl_up_sync(0xffffffffu, cost_incl, o);
        if (lane >= o) {
            incl += v;
            cost_incl += w;
        }
    }
    if (warp == 2) {
        int2 run = make_int2(incl - local, cost_incl - cost);
        for (int b = b0; b < b1; ++b) {
            cum[b] = run;
            const int n = fp8_tiles(p.kv_len[b], cap);
            run.x += n * hg;
            run.y += hg * (n * fp8_tile_cost(p, b) + kFp8UnitCost);
        }
        if (lane == 31) cum[p.batch] = make_int2(incl, cost_incl);
        return;
    }

    const int T = __shfl_sync(0xffffffffu, incl, 31);
    const int W = __shfl_sync(0xffffffffu, cost_incl, 31);
    const int C = fp8_split_groups(static_cast<int>(gridDim.x) >> p.head_shift, T, W,
                                   __reduce_max_sync(0xffffffffu, dearest));
    const int c = static_cast<int>(blockIdx.x) >> p.head_shift;
    const int w_lo = cost_incl - cost, w_hi = cost_incl;
    // First tile that starts at or after position y, and its unit; first: it
    // opens that unit.
    const auto locate = [&](int y, int &unit, bool &first) -> int {
        const bool mine = w_lo <= y && y < w_hi;
        const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        int x = 0, u = 0, f = 0;
        if (lane == src) {
            int xs = incl - local, ws = w_lo;   // the chunk's first tile / position
            for (int b = b0; b < b1; ++b) {
                const int n = fp8_tiles(p.kv_len[b], cap);
                const int tile = fp8_tile_cost(p, b);
                const int unit_span = n * tile + kFp8UnitCost;
                const int span = hg * unit_span;
                if (y < ws + span) {
                    const int h = hg == 1 ? 0 : (y - ws) / unit_span;
                    const int o = (y - ws) - h * unit_span - kFp8UnitCost;
                    const int i = o <= 0 ? 0 : (o + tile - 1) / tile;
                    x = xs + h * n + i;
                    u = b * hg + h + (i == n);   // past the unit's last tile: the next opens
                    f = i == 0 || i == n;
                    break;
                }
                xs += hg * n;
                ws += span;
            }
        }
        unit = __shfl_sync(0xffffffffu, u, src);
        first = __shfl_sync(0xffffffffu, f, src) != 0;
        return __shfl_sync(0xffffffffu, x, src);
    };
    int u = 0, x = 0;
    bool opens;
    if (warp == 0) {
        if (c < C) x = locate(first_position(c, W, C), u, opens);
        if (lane == 0) {
            out->x0 = x;
            out->u0 = u;
            out->groups = C;
            out->cost = W;
        }
    } else {
        if (c + 1 < C) {
            x = locate(first_position(c + 1, W, C), u, opens);
            u -= opens;    // tile x - 1 lies in the unit before when x opens one
        } else if (c + 1 == C) {
            x = T;
            u = p.batch * hg - 1;
        }
        if (lane == 0) {
            out->x1 = x;
            out->u1 = u;
        }
    }
}

// The piece of unit u0 + j inside the range.
__device__ __forceinline__ Fp8Item fp8_item(const Fp8DecodeParams &p, const int2 *cum,
                                            const Fp8Range &r, int j) {
    const int hg = p.head_groups;
    Fp8Item it;
    it.unit = r.u0 + j;
    it.b = by_groups(it.unit, hg);
    const int h = it.unit - it.b * hg;
    const int member = static_cast<int>(blockIdx.x) & ((1 << p.head_shift) - 1);
    it.kvh = (h << p.head_shift) + member;
    it.unit_tiles = by_groups(cum[it.b + 1].x - cum[it.b].x, hg);
    const int x = cum[it.b].x + h * it.unit_tiles;
    const int tb = max(r.x0 - x, 0), te = min(r.x1 - x, it.unit_tiles);
    it.L = static_cast<int>(min(p.kv_len[it.b], uint32_t(p.max_kv_len)));
    it.start = tb * kGqaTcTileKeys;
    it.end = min(te * kGqaTcTileKeys, it.L);
    it.ntiles = it.start < it.end ? (it.end - it.start + kGqaTcTileKeys - 1) / kGqaTcTileKeys : 0;
    it.first = tb == 0;
    it.direct = tb == 0 && te == it.unit_tiles;
    // the pieces of one (sequence, head) are consecutive: (groups + units) slots a member
    const int per_member = (static_cast<int>(gridDim.x) >> p.head_shift) + p.batch * hg;
    it.slot = member * per_member + (static_cast<int>(blockIdx.x) >> p.head_shift) + it.unit;
    return it;
}

// Pieces of the unit whose first tile this group holds: position y is group
// ((y + 1) C - 1) / W's, and the unit's last piece is the group's that its last
// tile starts in.
__device__ __forceinline__ int fp8_pieces(const Fp8DecodeParams &p, const int2 *cum,
                                          const Fp8Range &r, const Fp8Item &it) {
    const int h = it.unit - it.b * p.head_groups;
    const int tile = fp8_tile_cost(p, it.b);
    const int last =
        cum[it.b].y + (h + 1) * (it.unit_tiles * tile + kFp8UnitCost) - tile;
    const int c_last = group_of_position(last, r.cost, r.groups);
    return c_last - (static_cast<int>(blockIdx.x) >> p.head_shift) + 1;
}

}  // namespace attn
