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
// concatenated, are dealt out in contiguous ranges of equal cost: every unit is
// preceded by kUnitCost virtual tiles in a weighted concatenation (the
// fixed cost of opening it: its queries, the pipeline refill, the epilogue), and
// group c of C takes weighted positions [c W / C, (c + 1) W / C).  A unit of n
// tiles from tile x on sits at [x + kUnitCost u, x + kUnitCost (u + 1) + n); a
// position in its virtual block maps to its first tile.
#pragma once

#include "cache_ops.h"
#include "ptx.cuh"

namespace attn {

constexpr int kUnitCost = 4;

struct Fp8Range {
    int x0, x1;            // this group's tiles of the concatenation
    int u0, count;         // its first unit, and how many it meets
    int groups;            // C, after leaving out groups without tiles
    long long wtiles;      // W
};

struct Fp8Item {
    int b, kvh, L, start, end, ntiles;
    int unit, unit_x, unit_tiles;
    int slot;              // partial slot
    bool first, direct;    // holds the unit's first tile; holds all of it
};

__device__ __forceinline__ int fp8_tiles(uint32_t len, uint32_t cap) {
    return max(static_cast<int>((min(len, cap) + kGqaTcTileKeys - 1) / kGqaTcTileKeys), 1);
}

// cum[0..batch]: tiles of the concatenation before sequence b (head groups
// included); and this group's range.  One warp, all lanes.
__device__ __forceinline__ void fp8_build_items(const Fp8DecodeParams &p, int *cum, int lane,
                                                Fp8Range *out) {
    const int hg = p.head_groups;
    const uint32_t cap = uint32_t(p.max_kv_len);
    const int per_lane = (p.batch + 31) / 32;
    const int b0 = min(lane * per_lane, p.batch), b1 = min(b0 + per_lane, p.batch);
    int local = 0;
    for (int b = b0; b < b1; ++b) {
        const uint32_t len = p.kv_len[b];
        if (len > cap && blockIdx.x == 0) atomicOr(p.err, kErrBadLength);
        local += fp8_tiles(len, cap) * hg;
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    int run = incl - local;
    for (int b = b0; b < b1; ++b) {
        cum[b] = run;
        run += fp8_tiles(p.kv_len[b], cap) * hg;
    }
    if (lane == 31) cum[p.batch] = incl;

    const long long per_seq = static_cast<long long>(kUnitCost) * hg;
    const int T = __shfl_sync(0xffffffffu, incl, 31);
    const long long W = T + per_seq * p.batch;
    const int C = min(static_cast<int>(gridDim.x) >> p.head_shift, T);
    const int c = static_cast<int>(blockIdx.x) >> p.head_shift;
    const long long w_lo = (incl - local) + per_seq * b0, w_hi = incl + per_seq * b1;
    // Tile of weighted position y, its unit, and whether it is the unit's first.
    const auto locate = [&](long long y, int &unit, bool &at_first) -> int {
        const bool mine = w_lo <= y && y < w_hi;
        const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        int x = 0, u = 0, f = 0;
        if (lane == src) {
            int xs = incl - local;
            long long ws = w_lo;   // the chunk's first tile / position
            for (int b = b0; b < b1; ++b) {
                const int n = fp8_tiles(p.kv_len[b], cap);
                const long long span = static_cast<long long>(hg) * (n + kUnitCost);
                if (y < ws + span) {
                    const int off = static_cast<int>(y - ws);
                    const int h = off / (n + kUnitCost);
                    const int o = off - h * (n + kUnitCost) - kUnitCost;
                    x = xs + h * n + min(max(o, 0), n);
                    u = b * hg + h;
                    f = o <= 0;
                    break;
                }
                xs += hg * n;
                ws += span;
            }
        }
        unit = __shfl_sync(0xffffffffu, u, src);
        at_first = __shfl_sync(0xffffffffu, f, src) != 0;
        return __shfl_sync(0xffffffffu, x, src);
    };
    Fp8Range r;
    r.x0 = r.x1 = r.u0 = r.count = 0;
    r.groups = C;
    r.wtiles = W;
    if (c < C) {
        int u0, u1, u_last;
        bool f0, f1;
        r.x0 = locate(c * W / C, u0, f0);
        if (c + 1 == C) {
            r.x1 = T;
            u_last = p.batch * hg - 1;
        } else {
            r.x1 = locate((c + 1) * W / C, u1, f1);
            u_last = f1 ? u1 - 1 : u1;   // x1 - 1 lies in the unit before when x1 opens one
        }
        r.u0 = u0;
        r.count = r.x1 > r.x0 ? u_last - u0 + 1 : 0;
    }
    if (lane == 0) *out = r;
}

// The piece of unit u0 + j inside the range.
__device__ __forceinline__ Fp8Item fp8_item(const Fp8DecodeParams &p, const int *cum,
                                            const Fp8Range &r, int j) {
    const int hg = p.head_groups;
    Fp8Item it;
    it.unit = r.u0 + j;
    it.b = it.unit / hg;
    const int h = it.unit - it.b * hg;
    const int member = static_cast<int>(blockIdx.x) & ((1 << p.head_shift) - 1);
    it.kvh = (h << p.head_shift) + member;
    it.unit_tiles = (cum[it.b + 1] - cum[it.b]) / hg;
    it.unit_x = cum[it.b] + h * it.unit_tiles;
    const int tb = max(r.x0 - it.unit_x, 0), te = min(r.x1 - it.unit_x, it.unit_tiles);
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

// Pieces of the unit whose first piece is this one: groups c hold weighted
// position y if c = ((y + 1) C - 1) / W.
__device__ __forceinline__ int fp8_pieces(const Fp8DecodeParams &p, const Fp8Range &r,
                                          const Fp8Item &it) {
    const long long last = it.unit_x + it.unit_tiles - 1 +
                           static_cast<long long>(kUnitCost) * (it.unit + 1);
    const int c_last = static_cast<int>(((last + 1) * r.groups - 1) / r.wtiles);
    return c_last - (static_cast<int>(blockIdx.x) >> p.head_shift) + 1;
}

}  // namespace attn
