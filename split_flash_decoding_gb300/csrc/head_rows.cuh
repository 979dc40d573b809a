// head_rows.cuh -- the norm and rotation of one head vector, and where a row of
// a call falls in the cache.
#pragma once

#include "cache_ops.h"
#include "ptx.cuh"

namespace attn {

// cos and sin of pair i's angle at a position, times mscale.  The phase is a
// 64-bit fraction of a turn, so the product wraps exactly; its top 32 bits as
// a signed fraction lie in [-1/2, 1/2) turns, and their rounding to fp32 moves
// the angle by at most 2^-25 pi.
__device__ __forceinline__ void rope_cos_sin(const RopeParams &r, int i, int pos, float &c,
                                             float &s) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * r.turns[i];
    const float half_turns =
        static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
    sincospif(half_turns, &s, &c);
    c *= r.mscale;
    s *= r.mscale;
}

// Sequence of row r (one row per sequence without offsets); -1: none.
__device__ __forceinline__ int sequence_of_row(const RowsParams &p, int r) {
    if (!p.q_row_offsets) return r;
    if (r >= static_cast<int>(p.q_row_offsets[p.batch])) return -1;
    int lo = 0, hi = p.batch;   // off[lo] <= r < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int>(p.q_row_offsets[mid]) <= r) lo = mid; else hi = mid;
    }
    return lo;
}

// Page of token t of sequence b; -1 (and error bit 1) if it is not in the pool.
__device__ __forceinline__ int page_of(const RowsParams &p, int b, int t) {
    if (!p.page_table) return b;
    const int e = p.page_table[static_cast<size_t>(b) * p.max_pages + t / p.page_size];
    if (e < 0 || e >= p.num_pages) {
        atomicOr(p.err, kErrBadPage);
        return -1;
    }
    return e;
}

}  // namespace attn
