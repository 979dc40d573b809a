// head_tiles.cuh -- norm and rotation of query and key heads over tiles of rows,
// with the three ways the results go: rows of memory, slots of a bf16 cache, slots
// of a cache held in 8 bits.
//
// Bound by memory for prompts (each channel read and written once) and by latency
// for a few rows.  A CTA takes a tile of rows and some of their heads.  Its threads
// first look the rows' places up and compute the cos and sin of every (row, pair)
// once, into shared memory; then they walk the heads, whose rotation costs no more
// than reading that table.
//
// An item is one head of one row, on L lanes.  A lane holds two 16-byte vectors of
// it, chosen so that a pair of channels is always in one lane: in the half layout
// a vector of the rotated channels' lower half and the one rot_dim / 2 above it,
// otherwise vector i and the one half the head above it, so that lanes side by
// side read and write whole lines.  A CTA has 256 / L items in work at once: the
// tile's rows (padded to a power of two), then the next heads', so that a tile of
// one row has many heads in work.  A thread keeps its place in the list of heads
// (pointers, channels, weights) and adds to it; a first form, which found all that
// for every item, spent 437 instructions on 512 channels and took 142 us for 24768
// rows of 48 heads (now 98.5: 609 MB at 6.2 TB/s).  8191 rows of 40 heads with norms:
// 32.6 us (5.1 TB/s; a little over two waves of CTAs); 64 rows of 48 heads 3.3 us, one
// row 2.7.
//
// The 8-bit cache needs the largest value of a block of tokens before the first
// code: a tile then is the new tokens of one sequence inside an aligned group of
// 128 tokens (whole blocks of up to 128), the transformed values stay in registers
// while the rows' maxima are joined over the block, and what the block holds from
// before is rounded to a scale that grew.  64 single rows of 48 heads 4.4 us.  Runs
// of more than 32 tokens have a kernel of their own (append_fp8_runs.cu).
#pragma once

#include <cuda_fp8.h>
#include <float.h>

#include "head_rows.cuh"

namespace attn {
namespace tiles {

constexpr int kGroupTokens = 128;     // 8-bit cache: aligned tokens of a tile
constexpr int kMinExp = -60, kMaxExp = 120;

// The launch's cut of the work.
struct Cut {
    int tile_rows;                    // rows of a tile (8-bit cache: up to kGroupTokens)
    int chunks;                       // CTAs of a tile
    int chunk_heads;                  // heads of a CTA
    int heads;                        // q, k and v heads together
    int any_norm;
};

constexpr int kThreads = 256;
constexpr int kAhead = 3;             // heads whose vectors are on their way

// Items of L lanes at once: also the most rows of a tile.
template <int L>
constexpr int kItemsOf = kThreads / L;

// Where a row of the tile goes.
struct Place {
    long long k_at, v_at;             // element offsets into the caches
    int pos, token, page, slot;
    int stored;                       // -1: the row belongs to no sequence; 0: not stored; 1
};

// The m-th vector (8 channels) of a head, the rotated ones first: R of them from
// vector `start` on.
__device__ __forceinline__ int ordered(int m, int R, int start) {
    return m < R ? start + m : m - R < start ? m - R : m;
}

// The vectors of lane i in that order (-1: none), `vecs` in all, R of them rotated.
__device__ __forceinline__ void pair_of(bool inter, int vecs, int R, int i, int &a, int &b) {
    if (!inter && i < R / 2) {
        a = i;
        b = i + R / 2;
        return;
    }
    const int base = inter ? 0 : R;
    const int j = inter ? i : i - R / 2;
    const int H = (vecs - base + 1) / 2;
    a = j < H ? base + j : -1;
    b = j < H && base + j + H < vecs ? base + j + H : -1;
}

__device__ __forceinline__ void copy_16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}

__device__ __forceinline__ void unpack8(const uint4 &w, float2 (&x)[4]) {
    x[0] = bf16x2_to_float2(w.x);
    x[1] = bf16x2_to_float2(w.y);
    x[2] = bf16x2_to_float2(w.z);
    x[3] = bf16x2_to_float2(w.w);
}

__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
    return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                      pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
}

__device__ __forceinline__ void add_squares(const float2 (&y)[4], float2 &sum) {
#pragma unroll
    for (int c = 0; c < 4; ++c) sum = __ffma2_rn(y[c], y[c], sum);
}

// y *= f * weights (1 without weights)
__device__ __forceinline__ void scale8(float2 (&y)[4], const uint4 &w, float f) {
    float2 g[4];
    unpack8(w, g);
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = __fmul2_rn(y[c], __fmul2_rn(g[c], make_float2(f, f)));
}

// Exponent of the scale of a block whose largest finite value is amax: the least e
// with amax <= 448 * 2^e (448 = 0.875 * 2^9), clamped.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int e = static_cast<int>(bits >> 23) - 127;            // (0 and subnormal: clamped)
    return min(max(e - ((bits & 0x7fffffu) > 0x600000u ? 7 : 8), kMinExp), kMaxExp);
}

__device__ __forceinline__ float pow2i(int e) {   // -126 <= e <= 127
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Largest finite |value| (infinities and NaN do not count).
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= FLT_MAX ? a : 0.f;
}

// Four finite (or NaN) values times f as e4m3 codes.
__device__ __forceinline__ uint32_t encode4_finite(const float2 &a, const float2 &b, float f) {
    const float2 x = __fmul2_rn(a, make_float2(f, f)), y = __fmul2_rn(b, make_float2(f, f));
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// The same of any values; there is no infinity: it becomes NaN.
__device__ __forceinline__ uint32_t encode4(const float2 &a, const float2 &b, float f) {
    float2 x = __fmul2_rn(a, make_float2(f, f)), y = __fmul2_rn(b, make_float2(f, f));
    const float nan = __uint_as_float(0x7fffffffu);
    if (!(fabsf(x.x) <= FLT_MAX)) x.x = nan;
    if (!(fabsf(x.y) <= FLT_MAX)) x.y = nan;
    if (!(fabsf(y.x) <= FLT_MAX)) y.x = nan;
    if (!(fabsf(y.y) <= FLT_MAX)) y.y = nan;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ float2 decode2(uint32_t c) {
    return __half22float2(__half2(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xffffu), __NV_E4M3)));
}

// A lane's 16 channels as codes.
__device__ __forceinline__ void store_codes(uint8_t *a, uint8_t *b, const float2 (&ya)[4],
                                            const float2 (&yb)[4], float f, bool infinite) {
    uint2 wa, wb;
    if (infinite) {
        wa = make_uint2(encode4(ya[0], ya[1], f), encode4(ya[2], ya[3], f));
        wb = make_uint2(encode4(yb[0], yb[1], f), encode4(yb[2], yb[3], f));
    } else {
        wa = make_uint2(encode4_finite(ya[0], ya[1], f), encode4_finite(ya[2], ya[3], f));
        wb = make_uint2(encode4_finite(yb[0], yb[1], f), encode4_finite(yb[2], yb[3], f));
    }
    *reinterpret_cast<uint2 *>(a) = wa;
    *reinterpret_cast<uint2 *>(b) = wb;
}

// Four held codes at a scale that grew: ratio is the old one over the new.
__device__ __forceinline__ uint32_t recode4(uint32_t c, float ratio) {
    return encode4(decode2(c), decode2(c >> 16), ratio);
}

// Largest |value| of a lane's channels; NaN does not count.
__device__ __forceinline__ float largest(const float2 (&ya)[4], const float2 (&yb)[4]) {
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        top = fmax3(top, fabsf(ya[k].x), fabsf(ya[k].y));
        top = fmax3(top, fabsf(yb[k].x), fabsf(yb[k].y));
    }
    return top;
}

// The same where there is an infinity: it does not count either.
__device__ __forceinline__ float largest_finite(const float2 (&ya)[4], const float2 (&yb)[4]) {
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        top = fmaxf(fmaxf(fmaxf(finite_abs(ya[k].x), finite_abs(ya[k].y)), top),
                    fmaxf(finite_abs(yb[k].x), finite_abs(yb[k].y)));
    return top;
}

// Turn entry k of a lane's two vectors (turn_b: the second is rotated as well; in
// the half layout always).
template <bool kInter>
__device__ __forceinline__ void rotate_pairs(float2 &ya, float2 &yb, const float4 &v, bool turn_b) {
    const float2 y = ya, z = yb;
    if (kInter) {
        ya = make_float2(fmaf(y.x, v.x, -y.y * v.y), fmaf(y.y, v.x, y.x * v.y));
        if (turn_b) yb = make_float2(fmaf(z.x, v.z, -z.y * v.w), fmaf(z.y, v.z, z.x * v.w));
    } else {
        const float2 c = make_float2(v.x, v.z), n = make_float2(v.y, v.w);
        ya = __ffma2_rn(y, c, __fmul2_rn(z, make_float2(-n.x, -n.y)));
        yb = __ffma2_rn(z, c, __fmul2_rn(y, n));
    }
}

// Entry k of lane i's angles {cos, sin, cos, sin}: half layout those of channels 2k
// and 2k + 1 of its vectors, interleaved those of pair k of each vector.
template <bool kInter>
__device__ __forceinline__ float4 angle_entry(const RopeParams &rope, int vecs, int k, int i,
                                              int pos) {
    const int R = rope.rot_dim / 8;
    int a, b;
    pair_of(kInter, vecs, R, i, a, b);
    const int j0 = kInter ? 4 * a + k : 8 * i + 2 * k;
    const int j1 = kInter ? 4 * b + k : j0 + 1;
    float4 v = make_float4(1.f, 0.f, 1.f, 0.f);
    if (a >= 0 && a < R) rope_cos_sin(rope, j0, pos, v.x, v.y);
    if (b >= 0 && b < R) rope_cos_sin(rope, j1, pos, v.z, v.w);
    return v;
}

// Sequence of row r; -1: none.  (One thread a row; a warp's rows read the same lines.)
__device__ __forceinline__ int sequence_of(const RowsParams &p, int r) {
    if (!p.q_row_offsets) return r;
    if (r < static_cast<int>(p.q_row_offsets[0]) ||
        r >= static_cast<int>(p.q_row_offsets[p.batch]))
        return -1;
    int lo = 0, hi = p.batch;   // off[lo] <= r < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int>(p.q_row_offsets[mid]) <= r) lo = mid; else hi = mid;
    }
    return lo;
}

// Tile `tile` of the 8-bit cache: the new tokens of one sequence in one aligned
// group of kGroupTokens (tokens below 0 included: their queries are written);
// false: there is no such tile.  With single rows tile = row.  One warp, all lanes.
struct Tokens {
    int b, row, count;
    long long first, begin;   // the tile's first token; the sequence's first new token
};

__device__ __forceinline__ bool tile_tokens(const RowsParams &p, int tile, int lane, Tokens &out) {
    static_assert(kGroupTokens == 128, "token >> 7 is its group");
    int row0 = 0, n = 0, found = -1, index = 0;
    long long begin = 0;
    const auto look = [&](int b, bool report) {
        row0 = p.q_row_offsets ? static_cast<int>(p.q_row_offsets[b]) : b;
        n = p.q_row_offsets ? static_cast<int>(p.q_row_offsets[b + 1]) - row0 : 1;
        const uint32_t len = p.kv_len[b];
        begin = static_cast<long long>(len) - n;
        if (report && n > 0 && len != 0 &&
            (begin < 0 || len > static_cast<uint32_t>(p.max_kv_len)))
            atomicOr(p.err, kErrBadLength);
        n = min(n, p.num_rows - row0);
    };
    if (!p.q_row_offsets) {
        found = tile;
    } else {
        // 32 sequences at a time: a scan of their tile counts.  (The first CTA looks
        // at all of them, to report their lengths.)
        int before = 0;
        for (int b0 = 0; b0 < p.batch && (found < 0 || blockIdx.x == 0); b0 += 32) {
            int count = 0;
            if (b0 + lane < p.batch) {
                look(b0 + lane, blockIdx.x == 0);
                if (n > 0) count = static_cast<int>(((begin + n - 1) >> 7) - (begin >> 7)) + 1;
            }
            int incl = count;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const int start = before + incl - count;
            const unsigned who =
                __ballot_sync(0xffffffffu, found < 0 && tile >= start && tile < start + count);
            if (who) {
                const int src = __ffs(who) - 1;
                found = b0 + src;
                index = tile - __shfl_sync(0xffffffffu, start, src);
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (found < 0) return false;
    }
    look(found, !p.q_row_offsets && lane == 0);
    if (n <= 0) return false;
    const long long group = (begin >> 7) + index;
    out.b = found;
    out.begin = begin;
    out.first = max(begin, group * kGroupTokens);
    out.count = static_cast<int>(min(begin + n, (group + 1) * kGroupTokens) - out.first);
    out.row = row0 + static_cast<int>(out.first - begin);
    return true;
}

// At least as many tiles as a call has: a sequence of n rows meets at most
// (n - 1) / kGroupTokens + 2 groups.
inline long long fp8_tile_count(const RowsParams &p) {
    const long long bound = p.num_rows / kGroupTokens + 2LL * p.batch;
    return p.q_row_offsets && bound < p.num_rows ? bound : p.num_rows;
}

// The kind of head h of the list (q, then k, then v), its number among them and
// the end of its kind (within h1).
struct KindOf {
    int kind, head, end;
};

__device__ __forceinline__ KindOf kind_of(const RowsParams &p, int h, int h1) {
    const int k0 = p.q.heads, v0 = p.q.heads + p.k.heads;
    KindOf x;
    x.kind = h < k0 ? 0 : h < v0 ? 1 : 2;
    x.head = h - (x.kind == 0 ? 0 : x.kind == 1 ? k0 : v0);
    x.end = min(h1, x.kind == 0 ? k0 : x.kind == 1 ? v0 : h1);
    return x;
}

__device__ __forceinline__ const HeadRows &rows_of_kind(const RowsParams &p, int kind) {
    return kind == 0 ? p.q : kind == 1 ? p.k : p.v;
}

// First channels of lane i's two vectors; -1: none.
template <bool kInter>
__device__ __forceinline__ void channels_of(const RowsParams &p, const HeadRows &x, int kind, int i,
                                            int &ca, int &cb) {
    const int turning = kind < 2 ? p.rope.rot_dim / 8 : 0, start = x.rot_start / 8;
    int a, b;
    pair_of(kInter, x.dim / 8, turning, i, a, b);
    ca = a >= 0 ? 8 * ordered(a, turning, start) : -1;
    cb = b >= 0 ? 8 * ordered(b, turning, start) : -1;
}

// Where a thread's next vectors come from.
struct Source {
    const uint16_t *src;              // the head vector
    long long step;                   // to the thread's next head
    int h, h_end, ca, cb;

    template <bool kInter>
    __device__ __forceinline__ void open(const RowsParams &p, int row, int i0, int h1,
                                         int step_heads) {
        ca = cb = -1;
        h_end = 0x7fffffff;
        src = nullptr;
        step = 0;
        if (h >= h1) return;
        const KindOf k = kind_of(p, h, h1);
        const HeadRows &x = rows_of_kind(p, k.kind);
        channels_of<kInter>(p, x, k.kind, i0, ca, cb);
        h_end = k.end;
        src = x.in + row * x.in_row + k.head * x.in_head;
        step = step_heads * x.in_head;
    }

    // Sends for the vectors (if any) and moves on.
    template <bool kInter>
    __device__ __forceinline__ void fetch(const RowsParams &p, int row, int i0, int h1,
                                          int step_heads, uint4 *to) {
        if (ca >= 0) copy_16(to, src + ca);
        if (cb >= 0) copy_16(to + kThreads, src + cb);
        asm volatile("cp.async.commit_group;" ::: "memory");
        h += step_heads;
        src += step;
        if (h >= h_end) open<kInter>(p, row, i0, h1, step_heads);
    }
};

// A thread's item: where it is in the list of heads.
struct Item {
    enum { kNormA = 1, kNormB = 2, kTurnA = 4, kTurnB = 8 };
    uint16_t *dst;                    // rows: its output; a cache: the head's offset
    long long dst_step;               // to the thread's next head
    uint4 ga, gb;                     // the norm's weights of its channels
    float mean, eps;
    int row, h, h_end, kind, head;
    int ca, cb;                       // its two first channels; -1: none
    int flags;
    bool to_cache;

    template <bool kInter>
    __device__ __forceinline__ void open(const RowsParams &p, int r0, int i0, int h1,
                                         int step_heads) {
        ca = cb = -1;
        flags = 0;
        kind = 0;
        head = 0;
        h_end = 0x7fffffff;
        dst = nullptr;
        dst_step = 0;
        mean = eps = 0.f;
        to_cache = false;
        ga = gb = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);   // 1
        if (h >= h1) return;
        const KindOf k = kind_of(p, h, h1);
        const HeadRows &x = rows_of_kind(p, k.kind);
        kind = k.kind;
        head = k.head;
        h_end = k.end;
        channels_of<kInter>(p, x, kind, i0, ca, cb);
        to_cache = x.out == nullptr;
        if (to_cache) {
            const CacheOut &c = kind == 1 ? p.kc : p.vc;
            dst = reinterpret_cast<uint16_t *>(c.base) + head * c.head_stride;
            dst_step = step_heads * c.head_stride;
        } else {
            dst = x.out + (r0 + row) * x.out_row + head * x.out_head;
            dst_step = step_heads * x.out_head;
        }
        mean = x.mean;
        eps = x.eps;
        if (ca >= 0 && ca < x.norm_dim) {
            flags |= kNormA;
            if (x.norm) ga = *reinterpret_cast<const uint4 *>(x.norm + ca);
        }
        if (cb >= 0 && cb < x.norm_dim) {
            flags |= kNormB;
            if (x.norm) gb = *reinterpret_cast<const uint4 *>(x.norm + cb);
        }
        const int turn0 = x.rot_start, turn1 = kind < 2 ? turn0 + p.rope.rot_dim : turn0;
        if (ca >= turn0 && ca < turn1) flags |= kTurnA;
        if (cb >= turn0 && cb < turn1) flags |= kTurnB;
    }

    // step_heads heads on
    template <bool kInter>
    __device__ __forceinline__ void advance(const RowsParams &p, int r0, int i0, int h1,
                                            int step_heads) {
        h += step_heads;
        head += step_heads;
        dst += dst_step;
        if (h >= h_end) open<kInter>(p, r0, i0, h1, step_heads);
    }
};

// kMany: a CTA has more heads than it works on at once (never with kFp8).
template <int L, bool kInter, bool kFp8, bool kMany>
__global__ void __launch_bounds__(kThreads, kFp8 ? 2 : kMany ? 3 : 4)
head_tiles_kernel(const __grid_constant__ RowsParams p, const __grid_constant__ Cut cut) {
    constexpr int kItems = kItemsOf<L>;
    extern __shared__ __align__(16) float4 angles[];             // [rows][4][lanes]
    __shared__ Place places[kItems];
    __shared__ float row_max[kFp8 ? kItems : 1];                 // then 1 / scale
    __shared__ Tokens s_tile;
    __shared__ int s_any;
    const int tid = threadIdx.x, lane = tid & 31;
    if (!kFp8) pdl_launch_dependents();        // (the keys and values of an 8-bit append)
    const int tile = static_cast<int>(blockIdx.x) / cut.chunks;
    const int chunk = static_cast<int>(blockIdx.x) - tile * cut.chunks;
    const int h0 = chunk * cut.chunk_heads, h1 = min(h0 + cut.chunk_heads, cut.heads);

    // ---- rows of the tile and their places -------------------------------------
    int r0, n;
    if (kFp8) {
        for (int i = tid; i < kItems; i += kThreads) row_max[i] = 0.f;
        if (tid < 32) {
            Tokens t;
            const bool any = tile_tokens(p, tile, lane, t);
            if (lane == 0) {
                s_any = any;
                s_tile = t;
            }
        }
        __syncthreads();
        if (!s_any) return;
        r0 = s_tile.row;
        n = min(s_tile.count, cut.tile_rows);
        if (n < s_tile.count && tid == 0) atomicOr(p.err, kErrBadLength);   // above max_q_len
    } else {
        r0 = tile * cut.tile_rows;
        n = min(cut.tile_rows, p.num_rows - r0);
    }

    // ---- items: the first heads' loads go out before anything else ----------------
    int shift = 0;                                               // rows padded to 2^shift
    while ((1 << shift) < n) ++shift;
    const int step_heads = kItems >> shift;                      // heads in work at once
    const int i0 = tid & (L - 1);
    const int item0 = tid / L;
    const int half = p.rope.rot_dim / 2;
    Item it;
    it.row = item0 & ((1 << shift) - 1);
    it.h = it.row < n ? h0 + (item0 >> shift) : h1;
    it.row = min(it.row, n - 1);
    Source from;
    from.h = it.h;
    from.open<kInter>(p, r0 + it.row, i0, h1, step_heads);
    // kMany: the vectors go through shared memory, each thread's own, three heads ahead;
    // as many bytes as that have to be on their way for the memory's rate (in
    // registers and none ahead, 24768 rows of 48 heads took 131.7 us, two ahead 108.2;
    // 2, 3, 4 ahead, 8191 rows of 40 heads: 33.4, 32.5, 34.4).
    uint4 *ring = reinterpret_cast<uint4 *>(angles) + (half > 0 ? cut.tile_rows * 4 * L : 0) + tid;
    uint4 ra = make_uint4(0u, 0u, 0u, 0u), rb = ra;
    if (kMany) {
#pragma unroll
        for (int s = 0; s < kAhead; ++s)
            from.fetch<kInter>(p, r0 + it.row, i0, h1, step_heads, ring + 2 * s * kThreads);
    } else {
        if (from.ca >= 0) ra = *reinterpret_cast<const uint4 *>(from.src + from.ca);
        if (from.cb >= 0) rb = *reinterpret_cast<const uint4 *>(from.src + from.cb);
    }
    it.open<kInter>(p, r0, i0, h1, step_heads);
    int slot = 0;                                                // of this head's vectors

    // ---- places ----------------------------------------------------------------------
    for (int i = tid; i < n; i += kThreads) {
        Place at;
        at.pos = 0;
        at.stored = 0;
        at.k_at = at.v_at = 0;
        at.token = at.page = at.slot = 0;
        if (p.kv_len) {
            const int b = kFp8 ? s_tile.b : sequence_of(p, r0 + i);
            if (b < 0) {
                at.stored = -1;
            } else {
                long long t;
                if (kFp8) {
                    t = s_tile.first + i;
                } else {
                    const int row0 =
                        p.q_row_offsets ? static_cast<int>(p.q_row_offsets[b]) : b;
                    const int rows =
                        p.q_row_offsets ? static_cast<int>(p.q_row_offsets[b + 1]) - row0 : 1;
                    const uint32_t len = p.kv_len[b];
                    t = static_cast<long long>(len) - rows + (r0 + i - row0);
                    if ((t < 0 || t >= p.max_kv_len) && len != 0) atomicOr(p.err, kErrBadLength);
                }
                at.pos = static_cast<int>(max(t, 0LL));
                if (t >= 0 && t < p.max_kv_len && p.k.heads > 0) {
                    const int page = page_of(p, b, at.pos);
                    const int slot = p.page_table ? at.pos & (p.page_size - 1) : at.pos;
                    at.stored = page >= 0;
                    at.token = at.pos;
                    at.page = page;
                    at.slot = slot;
                    at.k_at = page * p.kc.page_stride + slot * p.kc.token_stride;
                    at.v_at = page * p.vc.page_stride + slot * p.vc.token_stride;
                }
            }
        }
        if (p.positions) at.pos = p.positions[r0 + i];
        places[i] = at;
    }
    __syncthreads();

    // ---- angles: one entry (two pairs) a thread ---------------------------------
    const int q_vecs = p.q.heads > 0 ? p.q.dim / 8 : p.k.dim / 8;
    if (half > 0 && h0 < p.q.heads + p.k.heads) {
        for (int e = tid; e < n * 4 * L; e += kThreads) {
            const int row = e / (4 * L);
            angles[e] = angle_entry<kInter>(p.rope, q_vecs, e / L & 3, e & (L - 1), places[row].pos);
        }
    }
    __syncthreads();

#pragma unroll 1
    for (int hs = h0; hs < h1; hs += step_heads) {
        if (kMany) {
            const int last = slot == 0 ? kAhead : slot - 1;      // used up one head ago
            from.fetch<kInter>(p, r0 + it.row, i0, h1, step_heads, ring + 2 * last * kThreads);
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
            ra = rb = make_uint4(0u, 0u, 0u, 0u);
            if (it.ca >= 0) ra = ring[2 * slot * kThreads];
            if (it.cb >= 0) rb = ring[(2 * slot + 1) * kThreads];
            slot = slot == kAhead ? 0 : slot + 1;
        }
        float2 ya[4], yb[4];
        unpack8(ra, ya);
        unpack8(rb, yb);
        const Place &at = places[it.row];
        if (cut.any_norm) {
            float2 sq = make_float2(0.f, 0.f);                   // (no vector: zeros)
            if (it.flags & Item::kNormA) add_squares(ya, sq);
            if (it.flags & Item::kNormB) add_squares(yb, sq);
            float sum = sq.x + sq.y;
#pragma unroll
            for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = rsqrtf(fmaf(sum, it.mean, it.eps));
            if (it.flags & Item::kNormA) scale8(ya, it.ga, inv);
            if (it.flags & Item::kNormB) scale8(yb, it.gb, inv);
        }
        if (it.flags & Item::kTurnA) {
            const float4 *t = angles + it.row * 4 * L + i0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                rotate_pairs<kInter>(ya[k], yb[k], t[k * L], it.flags & Item::kTurnB);
        }
        if (!kFp8 || it.kind == 0) {
            uint16_t *dst = it.dst;
            bool store = at.stored >= 0;
            if (!kFp8 && it.to_cache) {
                dst += it.kind == 1 ? at.k_at : at.v_at;
                store = at.stored > 0;
            }
            // (what is neither normed nor rotated goes as it is, NaN payloads too)
            const bool plain = !(it.flags & (Item::kNormA | Item::kNormB | Item::kTurnA));
            if (store && it.ca >= 0)
                *reinterpret_cast<uint4 *>(dst + it.ca) = plain ? ra : pack8(ya);
            if (store && it.cb >= 0)
                *reinterpret_cast<uint4 *>(dst + it.cb) = plain ? rb : pack8(yb);
        }
        if (!kFp8) {
            if (!kMany) return;
            it.advance<kInter>(p, r0, i0, h1, step_heads);
            continue;
        }
        if (hs + step_heads <= p.q.heads) return;                // queries only: uniform

        // ---- 8-bit cache: scales of the blocks -----------------------------------------
        const int B = p.block_tokens, base = static_cast<int>(s_tile.first);   // row 0's token
        // earlier tokens of the first row's block, uniform over the CTA
        const int held = s_tile.first == s_tile.begin && base >= 0 && places[0].stored > 0
                             ? base & (B - 1) : 0;
        float ratio = 1.f;                                       // of a held block's row 0
        // (NaN never counts; infinities do not either, but cost a second look)
        float top = largest(ya, yb);
        const bool infinite = top > FLT_MAX;
        if (infinite) top = largest_finite(ya, yb);
#pragma unroll
        for (int o = 1; o < L; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (i0 == 0) row_max[item0] = top;                       // (no item: 0)
        __syncthreads();
        // The thread of a block's first stored row in the tile takes the maximum over
        // the block's rows, writes the scale and leaves 1 / scale in their places.
        const int row = tid & ((1 << shift) - 1), h = hs + (tid >> shift);
        if (tid < kItems && row < n && h < h1 && h >= p.q.heads && places[row].stored > 0) {
            const int t = places[row].token;
            const int block0 = t & ~(B - 1);
            const int first = max(block0 - base, max(-base, 0));
            const int last = min(block0 + B, min(base + n, p.max_kv_len)) - base;
            if (row == first) {
                float most = 0.f;
                for (int i = first; i < last; ++i) most = fmaxf(most, row_max[(tid - row) + i]);
                const bool is_k = h < p.q.heads + p.k.heads;
                const int head = h - p.q.heads - (is_k ? 0 : p.k.heads);
                const CacheOut &c = is_k ? p.kc : p.vc;
                float *where = c.scale + places[row].page * c.scale_page +
                               (places[row].slot >> p.block_shift) * c.scale_block +
                               head * c.scale_head;
                float scale = pow2i(scale_exponent(most));
                if (row == 0 && held > 0) {
                    const float old = *where;
                    if (scale > old) ratio = old / scale; else scale = old;
                }
                *where = scale;
                const float inv = __frcp_rn(scale);
                for (int i = first; i < last; ++i) row_max[(tid - row) + i] = inv;
            }
        }
        // What the first block held, where its scale grew: eight tokens a warp at a
        // time, all their loads before the first store.
        if (held > 0) {
            __shared__ float s_ratio[kItems];
            const int heads_now = min(step_heads, h1 - hs);
            if (tid < kItems && (tid & ((1 << shift) - 1)) == 0) s_ratio[tid >> shift] = ratio;
            const int batches = __syncthreads_or(ratio != 1.f) ? (held + 7) / 8 : 0;
            for (int w = tid >> 5; w < heads_now * batches; w += kThreads / 32) {
                const int hh = w / batches, g = hs + hh;
                if (g < p.q.heads || s_ratio[hh] == 1.f) continue;
                const bool is_k = g < p.q.heads + p.k.heads;
                const int head = g - p.q.heads - (is_k ? 0 : p.k.heads);
                const CacheOut &c = is_k ? p.kc : p.vc;
                // the held tokens are the slots just before the tile's first row's
                const int i1 = 8 * (w - hh * batches) + 1;
                uint32_t *to = reinterpret_cast<uint32_t *>(
                                   c.base + (is_k ? places[0].k_at : places[0].v_at) +
                                   head * c.head_stride - i1 * c.token_stride) + lane;
                const long long step = c.token_stride / 4;
                uint32_t old[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i1 + i <= held) old[i] = *(to - i * step);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i1 + i <= held) *(to - i * step) = recode4(old[i], s_ratio[hh]);
            }
        } else {
            __syncthreads();                                     // 1 / scale is in place
        }
        // ---- codes ---------------------------------------------------------------------
        if (it.ca >= 0 && it.kind != 0 && at.stored > 0) {
            const CacheOut &c = it.kind == 1 ? p.kc : p.vc;
            const float f = row_max[item0];
            uint8_t *dst = c.base + (it.kind == 1 ? at.k_at : at.v_at) + it.head * c.head_stride;
            store_codes(dst + it.ca, dst + it.cb, ya, yb, f, infinite);
        }
        return;
    }
}

template <int L, bool kFp8, bool kMany>
cudaError_t launch(const RowsParams &p, const Cut &cut, long long tiles, cudaStream_t stream) {
    const long long blocks = tiles * cut.chunks;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const size_t smem =                                              // up to 48 KB
        (p.rope.rot_dim > 0 ? size_t(cut.tile_rows) * 4 * L * sizeof(float4) : 0) +
        (kMany ? size_t(kAhead + 1) * 2 * kThreads * sizeof(uint4) : 0);
    auto kern = p.rope.interleaved ? head_tiles_kernel<L, true, kFp8, kMany>
                                   : head_tiles_kernel<L, false, kFp8, kMany>;
    if (smem > 40 * 1024) {                                          // (48 KB with the static part)
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    kern<<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(p, cut);
    return cudaGetLastError();
}

}  // namespace tiles
}  // namespace attn
