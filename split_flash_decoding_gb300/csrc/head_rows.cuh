// head_rows.cuh -- the norm and rotation of one head vector, and where a row of
// a call falls in the cache.
#pragma once

#include "cache_ops.h"
#include "ptx.cuh"

namespace attn {

// cos and sin of pair i's angle at a position, times mscale.  The phase is a
// 64-bit fraction of a turn, so the product wraps exactly.  Its two top bits
// (rounded) are the quadrant; what is left, within an eighth of a turn, becomes
// an fp32 angle and the rest of it, and the Taylor series end where the next term
// is below 2^-28.  Within 1.3 steps of the exact cos and sin: a plain fp32 angle
// would miss by up to 2^-25 pi, which moves roundings to 8 bits.
__device__ __forceinline__ void rope_cos_sin(const RopeParams &rope, int i, int pos, float &c,
                                             float &s) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * rope.turns[i];
    const uint32_t top = static_cast<uint32_t>(phase >> 32);
    const uint32_t quadrant = (top + 0x20000000u) >> 30;
    const int left = static_cast<int>(top - (quadrant << 30));        // 2^-32 turns
    const float below = static_cast<float>(static_cast<uint32_t>(phase)) * 2.3283064e-10f;   // 2^-32
    // radians of 2^-32 turns, as a float and its rest
    constexpr double kUnitExact = 6.283185307179586 / 4294967296.0;
    constexpr float kUnit = static_cast<float>(kUnitExact);
    constexpr float kUnitRest = static_cast<float>(kUnitExact - static_cast<double>(kUnit));
    const float hi = static_cast<float>(left);
    const float lo = static_cast<float>(left - static_cast<int>(hi)) + below;
    const float r = hi * kUnit;
    const float rest = fmaf(hi, kUnit, -r) + fmaf(hi, kUnitRest, lo * kUnit);
    const float r2 = r * r;
    const float ps = fmaf(r2, fmaf(r2, fmaf(r2, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f),
                          -1.f / 6.f);
    const float pc = fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, -1.f / 3628800.f, 1.f / 40320.f),
                                            -1.f / 720.f), 1.f / 24.f), -0.5f);
    const float sr = fmaf(r * r2, ps, rest) + r;
    const float cr = fmaf(r2, pc, -rest * r) + 1.f;
    const bool swap = quadrant & 1;
    const float x = swap ? sr : cr, y = swap ? cr : sr;
    c = ((quadrant + 1) & 2 ? -x : x) * rope.mscale;
    s = (quadrant & 2 ? -y : y) * rope.mscale;
}

// Where a row falls: its sequence and token, and the sequence's first row and row
// count.  b < 0: the row belongs to no sequence.
struct RowPlace {
    int b, row0, n;
    uint32_t L;
    long long t;
};

// Place of row r, found by the whole warp: the offsets are searched 32 at a time.
__device__ __forceinline__ RowPlace place_of_row(const RowsParams &p, int r, int lane) {
    RowPlace at;
    at.b = r;
    at.row0 = r;
    at.n = 1;
    at.L = 0;
    at.t = 0;
    if (p.q_row_offsets) {
        int lo = 0, len = p.batch + 1;   // off[lo] <= r, the answer in [lo, lo + len)
        while (len > 1) {
            const int step = (len + 31) / 32;
            const int i = lane * step;
            const bool below =
                i < len && static_cast<int>(p.q_row_offsets[lo + i]) <= r;
            const int count = __popc(__ballot_sync(0xffffffffu, below));
            if (count == 0) {            // r < off[0]
                at.b = -1;
                return at;
            }
            lo += (count - 1) * step;
            len = min(step, len - (count - 1) * step);
        }
        at.b = lo < p.batch ? lo : -1;
        if (at.b < 0) return at;
        at.row0 = static_cast<int>(p.q_row_offsets[lo]);
        at.n = static_cast<int>(p.q_row_offsets[lo + 1]) - at.row0;
    }
    at.L = p.kv_len[at.b];
    at.t = static_cast<long long>(at.L) - at.n + (r - at.row0);
    return at;
}

// Page of token t of sequence b; -1 (and error bit 1) if it is not in the pool.
// (Pages of a table are a power of two long.)
__device__ __forceinline__ int page_of(const RowsParams &p, int b, int t) {
    if (!p.page_table) return b;
    const int e = p.page_table[static_cast<size_t>(b) * p.max_pages + (t >> (31 - __clz(p.page_size)))];
    if (e < 0 || e >= p.num_pages) {
        atomicOr(p.err, kErrBadPage);
        return -1;
    }
    return e;
}

// Head h of row r, normed and (rotate) rotated, into y (shared memory); one warp.
// kStepwise: each operation rounded by itself, as in the 4-bit tiles (see there): a head's codes
// then do not depend on which of the two kernels took it.
template <bool kStepwise = false>
__device__ __forceinline__ void load_head(const RowsParams &p, const HeadRows &x, int r, int h,
                                          int pos, bool rotate, float *y, int lane) {
    const uint16_t *src = x.in + r * x.in_row + h * x.in_head;
    float sq = 0.f;
    for (int c = lane; c < x.dim; c += 32) {
        const float v = bf16_lo(src[c]);
        y[c] = v;
        if (c < x.norm_dim) sq += v * v;
    }
    __syncwarp();
    if (x.norm_dim > 0) {
        const float inv = rsqrtf(warp_sum(sq) / static_cast<float>(x.norm_dim) + x.eps);
        for (int c = lane; c < x.norm_dim; c += 32) {
            const float g = x.norm ? bf16_lo(x.norm[c]) : 1.f;
            y[c] = kStepwise ? __fmul_rn(__fmul_rn(y[c], inv), g) : y[c] * (inv * g);
        }
        __syncwarp();
    }
    if (rotate) {
        const int half = p.rope.rot_dim / 2;
        for (int i = lane; i < half; i += 32) {
            const int a = x.rot_start + (p.rope.interleaved ? 2 * i : i);
            const int b = a + (p.rope.interleaved ? 1 : half);
            float c, s;
            rope_cos_sin(p.rope, i, pos, c, s);
            const float ya = y[a], yb = y[b];
            if (kStepwise) {
                y[a] = __fsub_rn(__fmul_rn(ya, c), __fmul_rn(yb, s));
                y[b] = __fadd_rn(__fmul_rn(yb, c), __fmul_rn(ya, s));
            } else {
                y[a] = fmaf(ya, c, -yb * s);
                y[b] = fmaf(yb, c, ya * s);
            }
        }
        __syncwarp();
    }
}

}  // namespace attn
