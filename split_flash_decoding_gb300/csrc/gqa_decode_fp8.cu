// gqa_decode_fp8.cu -- split-K decode attention over a cache held in 8 bits
// (e4m3 codes, an fp32 scale per block of tokens and KV head), head_dim 128.
//
//   s_j = scale q . (ks_j K8_j),  p_j = e^(s_j - m)
//   out = sum_j p_j (vs_j V8_j) / (sum_j p_j + e^(sink - m))
//
// The work list is the balanced split of fp8_items.cuh (the 128-key tiles of
// the sequences dealt out in ranges of equal cost, KV heads side by side), with
// two CTAs per SM.  Both contractions of a tile run on the codes as they are,
// as tcgen05 kind::f8f6f4 MMAs with the keys / the channels on the 128 rows of
// M and the folded query rows and heads on N:
//
//   S^T [128 keys x N] = K8 [128 keys x 128 ch] . Q^T       (K-major A, B)
//   O^T [128 ch x N]  += V8^T [128 ch x 128 keys] . P^T     (MN-major A)
//
// Both operands of such an MMA are 8 bits wide, so the side that is not in the
// cache is a sum of e4m3 terms, each in a column of its own: N is padded to 16
// anyway, and the time of an MMA this narrow is that of reading A.
//   q = 2^-a (q0 + q1 / 16): a puts the row's largest channel in [128, 256);
//     8 significant bits are two terms of 4, so bf16 channels down to 2^-13 of
//     the largest are exact and smaller ones miss at most 2^-21 of it.
//   weights = w0 + 2^-5 w1 + 2^-10 w2 + 2^-25 w3, each term what those before leave,
//     rounded to nearest.  e4m3 numbers end at 2^-9, so what terms hold of a small weight
//     is bounded below: an error of at most 2^-13 of the weight, or 2^-29 of the piece's
//     reference where that is more (a weight of 2^-20 of it keeps 9 bits, as in bf16),
//     though never more than a sixteenth of a weight of 2^-35 and more; what is below
//     2^-40 is lost.  The last term starts that low because the first three already hold
//     the larger weights; it saturates there.  (Three terms 2^-4 apart dropped all below
//     2^-21: a key that takes nearly all the weight and has no V, 15 nats above 131072
//     others, left 0 of them.)
// A thread owns one key of the tile (its TMEM lane), so the scales cost it two
// multiplications: ks_j goes into the score, and V's scale into the weight.
// With vs_j = r_j 2^(e_j) (e_j its exponent, clamped to [-64, 64]), the running
// reference m is that of s_j + e_j, so the largest weight sits at the top of
// the e4m3 range whatever the scales are; the row sum takes the weights
// without 2^(e_j).  m, the sum and O keep one reference, which is what the
// split-K reduce merges.  The reference is lazy: it follows a tile's maximum
// only when that exceeds it by more than 2^kLazy.
//
// Warp roles: softmax and epilogue (four warps, or two groups of four for more
// than 4 columns), K producer and V producer (TMA), MMA issue, and one warp that
// turns q into its terms and fetches the scales of each tile's keys (cp.async).
//
// What bounds it.  Up to 4 columns the stream of codes: 64 sequences of 32 + 8
// heads and 512 to 8192 keys (580 MB) take 98 us, 5.9 TB/s with everything,
// about 7 while the stream runs.  The rest is 5 us until the first scores
// (range, page table, first tile), the ends of the CTAs and the reduce.  With 16
// columns the softmax of a tile takes longer than its bytes (1 to 4 draft
// rows of 4 heads: 89 us for 318 MB; 83 with three terms of the weights).  What runs
// once an item (opening it, the first tile's maxima, the epilogue) runs from a cold
// instruction cache, at 100 cycles and more per eight instructions: hence the rolled
// loops and the care for code length there.  (Heads taken one after the other 114.9 us, P through a swizzled
// K-major layout 201 instead of 158 us for the draft rows, one group of warps for
// 16 columns 147 instead of 103, 3 V stages the same.)
#include <cuda_fp8.h>

#include "cache_ops.h"
#include "fp8_items.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace attn {
namespace {

constexpr int kD = 128;
constexpr int kBK = kGqaTcTileKeys;          // 128 keys per tile
constexpr int kStages = 3;                   // K tiles in flight
constexpr int kVStages = 2;                  // V tiles in flight (three measured the same)
constexpr int kTileBytes = kBK * kD;         // 16 KB
constexpr int kScStages = 6;                 // tiles of scales in flight
constexpr int kQBufs = 2;
constexpr int kCtasPerSm = 2;
// A lower kLazy leaves more of the e4m3 range below the reference, a higher one moves it
// less often (kLazy 1, 2, 3, 4: 64 single rows 100 us each, 1 to 4 draft rows of 4 heads 107,
// 98, 93, 92).
constexpr float kLazy = 3.f;                 // base 2
constexpr float kWeightTop = 16.f;           // weights reach 2^kLazy * 2 * kWeightTop = 256
// Each term's unit over the next one's (see above).
__host__ __device__ constexpr float term_ratio(int u) { return u < 2 ? 32.f : 32768.f; }
constexpr int kBarBytes = 304;
constexpr int kMinVExp = -64, kMaxVExp = 64;

// Columns (query rows x heads) come in chunks of four: a chunk's S columns (and Q
// rows) are [2 terms][4], its O columns (and P columns) [4 terms][4].  More than one
// chunk takes two groups of four softmax warps; group g has the chunks g, g + 2.  Chunks
// past an item's columns are skipped.
template <int NC>
struct Cfg {
    static constexpr int kChunks = NC / 4;
    static constexpr int kGroups = NC > 4 ? 2 : 1;
    static constexpr int NCH = kChunks / kGroups;                    // chunks per group
    static constexpr int NS = kChunks < 2 ? 16 : 8 * kChunks;        // N of the score MMA
    static constexpr int NP = 16 * kChunks;                          // N of the output MMA
    static constexpr int kTmemO = 2 * NS;                            // after two score buffers
    static constexpr int kTmemCols = 2 * NS + NP <= 64 ? 64 : 128;
    static constexpr int kWarpK = 4 * kGroups, kWarpV = kWarpK + 1, kWarpMma = kWarpK + 2,
                         kWarpAux = kWarpK + 3;
    static constexpr int kThreads = 32 * (4 * kGroups + 4);
    // shared memory
    static constexpr int kring = 0;
    static constexpr int vring = kring + kStages * kTileBytes;
    static constexpr int q = vring + kVStages * kTileBytes;          // [kQBufs][NS rows][128 B]
    static constexpr int p = q + kQBufs * NS * 128;                  // [chunks][128 keys][16 B]
    static constexpr int sc = p + NP * 128;                          // [kScStages][128] {ks, vs}
    static constexpr int red = sc + kScStages * kBK * 8;             // float [4][16] tile max
    static constexpr int lred = red + 4 * 16 * 4;                    // float [2][5][16] row sums, references
    static constexpr int qf = lred + 2 * 5 * 16 * 4;                 // float [kQBufs][16] 2^-a
    static constexpr int bars = qf + 2 * 16 * 4;
    static constexpr int tmem_slot = bars + kBarBytes;
    static constexpr int range = tmem_slot + 16;
    static constexpr int items = range + 32;
};

enum Bar {
    kKFull = 0, kKEmpty = 3, kVFull = 6, kVEmpty = 9,   // [kStages] each
    kScFull = 12, kScEmpty = 12 + kScStages,         // [kScStages] each
    kQFull = 12 + 2 * kScStages, kQEmpty = kQFull + 2,   // [2] each
    kSFull = kQEmpty + 2, kSFree = kSFull + 2,          // [2] each
    kPFull = kSFree + 2, kODone = kPFull + 1,
    kNumBars = kODone + 1
};
static_assert(kStages == 3 && kNumBars * 8 <= kBarBytes, "barrier layout");
static_assert(sizeof(Fp8Range) <= 32, "range slot");

template <int NC>
size_t smem_bytes(int batch) {
    return size_t(Cfg<NC>::items) + sizeof(int2) * size_t(batch + 1);
}

// Instruction descriptor of kind::f8f6f4 with e4m3 A and B, fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) |
           (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Shared-memory matrix descriptor without a swizzle; lbo/sbo in bytes.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= uint64_t((saddr & 0x3FFFFu) >> 4);
    d |= uint64_t((lbo >> 4) & 0x3FFFu) << 16;
    d |= uint64_t((sbo >> 4) & 0x3FFFu) << 32;
    d |= uint64_t(1) << 46;
    return d;
}

// N (a multiple of 8) consecutive TMEM columns of the thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i + 8 <= N; i += 8) {
        float a[8];
        tc::tmem_ld_n<8>(taddr + i, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i + j] = a[j];
    }
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i + 8 <= N; i += 8) {
        float a[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = v[i + j];
        tc::tmem_st_n<8>(taddr + i, a);
    }
}

// The four terms of two O columns side by side, four columns apart.
__device__ __forceinline__ void tmem_ld_terms(uint32_t taddr, float (&o)[4][2]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%8];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x2.b32 {%2, %3}, [%9];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x2.b32 {%4, %5}, [%10];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x2.b32 {%6, %7}, [%11];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&f"(o[0][0]), "=&f"(o[0][1]), "=&f"(o[1][0]), "=&f"(o[1][1]), "=&f"(o[2][0]),
          "=&f"(o[2][1]), "=&f"(o[3][0]), "=&f"(o[3][1])
        : "r"(taddr), "r"(taddr + 4), "r"(taddr + 8), "r"(taddr + 12)
        : "memory");
}

// Eight columns at each of the thread's chunks, one wait for all.
__device__ __forceinline__ void tmem_ld_scores(uint32_t t0, uint32_t, float (&v)[1][8]) {
    tc::tmem_ld_n<8>(t0, v[0]);
}
__device__ __forceinline__ void tmem_ld_scores(uint32_t t0, uint32_t t1, float (&v)[2][8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&f"(v[0][0]), "=&f"(v[0][1]), "=&f"(v[0][2]), "=&f"(v[0][3]), "=&f"(v[0][4]),
          "=&f"(v[0][5]), "=&f"(v[0][6]), "=&f"(v[0][7]), "=&f"(v[1][0]), "=&f"(v[1][1]),
          "=&f"(v[1][2]), "=&f"(v[1][3]), "=&f"(v[1][4]), "=&f"(v[1][5]), "=&f"(v[1][6]),
          "=&f"(v[1][7])
        : "r"(t0), "r"(t1)
        : "memory");
}

// Maximum over the 32 lanes of the warp (NaN ignored; every lane gets it).
__device__ __forceinline__ float warp_max_redux(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Named barrier over a subset of warps that returns the OR of their predicates.
__device__ __forceinline__ bool named_or(int id, int threads, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(pred ? 1u : 0u)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float pow2i(int e) {   // -126 <= e <= 127
    return __uint_as_float(uint32_t(e + 127) << 23);
}

// Two values to e4m3 (a in the low byte).
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// What two codes leave of (a, b): exact, in a mixed-precision FMA, no unpacking.
__device__ __forceinline__ void take_rest(uint32_t c, float &a, float &b) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
    const unsigned short minus1 = 0xbc00;   // f16
    asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(a) : "h"(h.x), "h"(minus1));
    asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(b) : "h"(h.y), "h"(minus1));
}

// Byte of element (row r, byte c) of an operand of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t operand_offset(int r, int c) {
    return uint32_t(r * 128 + (((c >> 4) ^ (r & 7)) << 4) + (c & 15));
}

// First query row and row count of sequence b.
__device__ __forceinline__ void seq_rows(const Fp8DecodeParams &p, int b, int &row0, int &nrows) {
    if (p.q_row_offsets) {
        row0 = int(p.q_row_offsets[b]);
        nrows = int(p.q_row_offsets[b + 1]) - row0;
    } else {
        row0 = b;
        nrows = 1;
    }
}

// Page and first slot of the item's 32 row boxes from box 32 * chunk on, one
// per lane; page -1: past the end or outside the pool.
__device__ __forceinline__ void lookup_boxes(const Fp8DecodeParams &p, const Fp8Item &it, int chunk,
                                             int lane, bool report, int &page, int &slot) {
    const int tk = it.start + ((chunk << 5) + lane) * p.box_rows;
    page = -1;
    slot = 0;
    if (tk >= it.L) return;
    if (!p.page_table) {
        page = it.b;
        slot = tk;
        return;
    }
    const int pidx = tk >> (31 - __clz(p.page_size));   // (pages of a table: powers of two)
    const int e = pidx < p.max_pages ? p.page_table[size_t(it.b) * p.max_pages + pidx] : -1;
    if (e < 0 || e >= p.num_pages) {
        if (report) atomicOr(p.err, kErrBadPage);
        return;
    }
    page = e;
    slot = tk & (p.page_size - 1);
}

// K or V producer: walks this CTA's items and tiles and lets lane 0 issue the
// boxes of each tile into the ring.
template <bool kIsK, int NC>
__device__ __forceinline__ void produce(const Fp8DecodeParams &p, const int2 *cum, const Fp8Range &w,
                                        uint8_t *smem, uint64_t *bar, int lane) {
    const CUtensorMap *map = kIsK ? &p.k_map : &p.v_map;
    uint64_t *full = bar + (kIsK ? kKFull : kVFull);
    uint64_t *empty = bar + (kIsK ? kKEmpty : kVEmpty);
    uint8_t *ring = smem + (kIsK ? Cfg<NC>::kring : Cfg<NC>::vring);
    constexpr int kN = kIsK ? kStages : kVStages;
    const int box_rows = p.box_rows;        // 128, 64, 32, 16 or 8
    const int box_shift = 31 - __clz(box_rows);
    const int nb = kBK >> box_shift;        // row boxes per tile
    const uint32_t box_bytes = uint32_t(box_rows) * 128u;
    int g = 0;
    bool aborted = false;
    for (int j = 0, items = w.count(); j < items && !aborted; ++j) {
        const Fp8Item it = fp8_item(p, cum, w, j);
        if (it.ntiles == 0) continue;
        int cached = -1, my_page = -1, my_slot = 0;
        for (int t = 0; t < it.ntiles && !aborted; ++t) {
            const int gg = g + t;
            const int s = gg % kN;
            const int key0 = it.start + t * kBK;
            const int live = min(nb, (it.L - key0 + box_rows - 1) >> box_shift);
            if (lane == 0) {
                if (gg >= kN && !mbar_wait(&empty[s], ((gg / kN) - 1) & 1, p.err))
                    aborted = true;
                else
                    mbar_arrive_expect_tx(&full[s], uint32_t(live) * box_bytes);
            }
            aborted = __shfl_sync(0xffffffffu, aborted, 0);
            if (aborted) break;
            uint8_t *dst = ring + s * kTileBytes;
            for (int r = 0; r < live; ++r) {
                const int gb = t * nb + r;                           // box index in the item
                if ((gb >> 5) != cached) {                           // warp-uniform refill
                    cached = gb >> 5;
                    lookup_boxes(p, it, cached, lane, kIsK, my_page, my_slot);
                }
                const int page = __shfl_sync(0xffffffffu, my_page, gb & 31);
                const int slot = __shfl_sync(0xffffffffu, my_slot, gb & 31);
                if (lane == 0) {
                    if (page < 0)
                        mbar_complete_tx(&full[s], box_bytes);       // skipped bad page
                    else
                        tma_load_4d(dst + r * box_bytes, map, &full[s], 0, slot, it.kvh, page);
                }
            }
        }
        g += it.ntiles;
    }
    // Every copy this warp issued must land before the CTA may leave.
    if (lane == 0)
        for (int i = max(0, g - kN); i < g; ++i)
            mbar_wait(&full[i % kN], (i / kN) & 1, p.err);
}

__device__ __forceinline__ void cp_async_4(void *dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}
// Arrive (without raising the pending count) when this thread's copies so far are done.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// Auxiliary warp: the terms of each item's queries and the scales of each
// tile's keys.
template <int NC>
__device__ __forceinline__ void feed(const Fp8DecodeParams &p, const int2 *cum, const Fp8Range &w,
                                     uint8_t *smem, uint64_t *bar, int lane) {
    using C = Cfg<NC>;
    const int G = p.group;
    const int g_inv = (1 << 16) / G + 1;            // (c * g_inv) >> 16 = c / G for c < 16
    const int box_shift = 31 - __clz(p.box_rows);   // a power of two
    const int nb_shift = 7 - box_shift;             // boxes per tile
    int g = 0, itq = 0;
    bool ok = true;
    for (int j = 0, items = w.count(); ok && j < items; ++j) {
        const Fp8Item it = fp8_item(p, cum, w, j);
        if (it.ntiles == 0) continue;
        const int qb = itq % kQBufs;
        if (itq >= kQBufs)
            ok = mbar_wait(&bar[kQEmpty + qb], ((itq / kQBufs) - 1) & 1, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        int row0, nrows;
        seq_rows(p, it.b, row0, nrows);
        uint8_t *qs = smem + C::q + qb * C::NS * 128;
        float *qf = reinterpret_cast<float *>(smem + C::qf) + qb * 16;
        const int want = min(nrows, p.num_q_rows - row0) * G, cols = min(want, NC);
        if (want > NC && lane == 0) atomicOr(p.err, kErrBadLength);   // above max_q_len
        // Four columns at a time, 16 channels a lane.  The bf16 rows are first copied
        // to where their own terms go; both loops are rolled, as they run from a
        // cold instruction cache (8 columns unrolled: 13000 cycles for 16 columns).
        const int cq = lane >> 3, li = lane & 7;
#pragma unroll 1
        for (int c = cq; c < cols; c += 4) {
            const int i = (c * g_inv) >> 16, h = c - i * G;
            const uint16_t *src =
                p.q + (size_t(row0 + i) * p.num_q_heads + it.kvh * G + h) * kD + 16 * li;
            uint8_t *dst = qs + (2 * (c - cq) + cq + (li & 4)) * 128 + (li & 3) * 32;
            cp_async_16(dst, src);
            cp_async_16(dst + 16, src + 8);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 4) {
            const int c = c0 + cq, r = 2 * c0 + cq;              // rows r and r + 4: its terms
            const uint4 *raw =
                reinterpret_cast<const uint4 *>(qs + (r + (li & 4)) * 128 + (li & 3) * 32);
            const uint4 u = raw[0], v = raw[1];
            float2 x[8] = {bf16x2_to_float2(u.x), bf16x2_to_float2(u.y), bf16x2_to_float2(u.z),
                           bf16x2_to_float2(u.w), bf16x2_to_float2(v.x), bf16x2_to_float2(v.y),
                           bf16x2_to_float2(v.z), bf16x2_to_float2(v.w)};
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmax3(top, fabsf(x[k].x), fabsf(x[k].y));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // 2^a * top in [128, 256) (a clamped where the factor would leave fp32)
            const int e = int(__float_as_uint(top) >> 23) - 127;
            const int a = min(max(7 - e, -120), 120);
            const float f = pow2i(a);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[k] = __fmul2_rn(x[k], make_float2(f, f));
                // an infinite channel has no e4m3 code: it becomes NaN
                if (!(fabsf(x[k].x) < INFINITY)) x[k].x = __uint_as_float(0x7fffffffu);
                if (!(fabsf(x[k].y) < INFINITY)) x[k].y = __uint_as_float(0x7fffffffu);
                const uint32_t h = to_e4m3x2(x[k].x, x[k].y);
                take_rest(h, x[k].x, x[k].y);
                x[k] = __fmul2_rn(x[k], make_float2(16.f, 16.f));
                const uint32_t l = to_e4m3x2(x[k].x, x[k].y);
                hi[k >> 1] = k & 1 ? hi[k >> 1] | (h << 16) : h;
                lo[k >> 1] = k & 1 ? lo[k >> 1] | (l << 16) : l;
            }
            __syncwarp();                                        // the four rows are read
            if (c < cols) {
                *reinterpret_cast<uint4 *>(qs + operand_offset(r, 16 * li)) =
                    make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(qs + operand_offset(r + 4, 16 * li)) =
                    make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if (li == 0) qf[c] = pow2i(-a);
            }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kQFull + qb]);

        // One box per lane and refill, as in the producers; the 32 keys of a step
        // lie in one box or in whole boxes, within one refill.
        const float *ksp = p.k_scale + it.kvh * p.ks_head;
        const float *vsp = p.v_scale + it.kvh * p.vs_head;
        int cached = -1, my_page = -1, my_slot = 0;
        for (int t = 0; t < it.ntiles; ++t) {
            const int gg = g + t;
            const int s = gg % kScStages;
            const int left = it.L - (it.start + t * kBK);            // keys of the tile on
            if (gg >= kScStages)
                ok = mbar_wait(&bar[kScEmpty + s], ((gg / kScStages) - 1) & 1, p.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            float2 *dst = reinterpret_cast<float2 *>(smem + C::sc) + s * kBK + lane;
#pragma unroll
            for (int u = 0; u < kBK / 32; ++u) {
                const int k = 32 * u + lane;                         // key of the tile
                const int box = (t << nb_shift) + (k >> box_shift);
                if ((box >> 5) != cached) {                          // uniform: see above
                    cached = box >> 5;
                    lookup_boxes(p, it, cached, lane, false, my_page, my_slot);
                }
                const int page = __shfl_sync(0xffffffffu, my_page, box);
                const int slot = __shfl_sync(0xffffffffu, my_slot, box) + (k & (p.box_rows - 1));
                if (page >= 0 && slot < p.page_size && k < left) {
                    const long long blk = slot >> p.block_shift;
                    cp_async_4(&dst[32 * u].x, ksp + page * p.ks_page + blk * p.ks_block);
                    cp_async_4(&dst[32 * u].y, vsp + page * p.vs_page + blk * p.vs_block);
                }
            }
            cp_async_arrive(&bar[kScFull + s]);
        }
        g += it.ntiles;
        ++itq;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int NC>
__global__ void __launch_bounds__(Cfg<NC>::kThreads, kCtasPerSm)
gqa_decode_fp8_kernel(const __grid_constant__ Fp8DecodeParams p) {
    using C = Cfg<NC>;
    constexpr int NCH = C::NCH;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::tmem_slot);
    Fp8Range *range = reinterpret_cast<Fp8Range *>(smem + C::range);
    int2 *cum = reinterpret_cast<int2 *>(smem + C::items);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = p.group;

    if (warp < 3) fp8_build_items(p, cum, warp, lane, range);
    if (lane == 0 && (warp == C::kWarpK || warp == C::kWarpV))
        prefetch_tensormap(warp == C::kWarpK ? &p.k_map : &p.v_map);
    if (threadIdx.x == 96) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t n = 1;
            if (i == kSFree || i == kSFree + 1 || i == kPFull) n = 4 * C::kGroups;
            if (i >= kScEmpty && i < kScEmpty + kScStages) n = 4 * C::kGroups;
            if (i == kQEmpty || i == kQEmpty + 1) n = 4 * C::kGroups + 1;
            if (i >= kScFull && i < kScFull + kScStages) n = 32;
            mbar_init(&bar[i], n);
        }
        fence_mbar_init();
    }
    if (warp == C::kWarpMma) {
        tc::tmem_alloc(tmem_slot, C::kTmemCols);
        tc::tmem_relinquish();
    }
    // Rows of Q and P past the columns in use stay zero.
    if (warp >= 3)
        for (int i = threadIdx.x - 96; i < (kQBufs * C::NS + C::NP) * 8; i += C::kThreads - 96)
            reinterpret_cast<uint4 *>(smem + C::q)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const Fp8Range walk = *range;
    const int items = walk.count();

    if (warp == C::kWarpK) {
        produce<true, NC>(p, cum, walk, smem, bar, lane);
    } else if (warp == C::kWarpV) {
        produce<false, NC>(p, cum, walk, smem, bar, lane);
    } else if (warp == C::kWarpAux) {
        feed<NC>(p, cum, walk, smem, bar, lane);
    } else if (warp == C::kWarpMma) {
        // ---------------------------------------------------------- MMA issue
        if (lane == 0) {
            constexpr uint32_t idesc_s = idesc_e4m3(128, C::NS, 0, 0);
            constexpr uint32_t idesc_o = idesc_e4m3(128, C::NP, 1, 1);
            const uint32_t k_base = smem_addr(smem + C::kring);
            const uint32_t v_base = smem_addr(smem + C::vring);
            const uint32_t q_base = smem_addr(smem + C::q);
            // MN-major without a swizzle: 16 bytes per key, 8-key groups 128 bytes
            // apart, 16-column blocks kBK * 16
            const uint64_t pd = smem_desc_plain(smem_addr(smem + C::p), 128, kBK * 16);
            int g = 0, itq = 0;
            bool ok = true;
            for (int j = 0; ok && j < items; ++j) {
                const Fp8Item it = fp8_item(p, cum, walk, j);
                if (it.ntiles == 0) continue;
                const int qb = itq % kQBufs;
                ok = mbar_wait(&bar[kQFull + qb], (itq / kQBufs) & 1, p.err);
                for (int t = 0; ok && t <= it.ntiles; ++t) {
                    if (t < it.ntiles) {
                        const int gg = g + t;
                        const int ks = gg % kStages;
                        const int sb = gg & 1;
                        ok = mbar_wait(&bar[kKFull + ks], (gg / kStages) & 1, p.err);
                        if (ok && gg >= 2)
                            ok = mbar_wait(&bar[kSFree + sb], ((gg >> 1) - 1) & 1, p.err);
                        if (!ok) break;
                        tc::fence_after_sync();
                        const uint64_t kd =
                            tc::smem_desc_sw128(k_base + ks * kTileBytes, 16, 1024);
                        const uint64_t qd =
                            tc::smem_desc_sw128(q_base + qb * C::NS * 128, 16, 1024);
#pragma unroll
                        for (int kk = 0; kk < kD / 32; ++kk)   // 32 channels = 32 bytes a step
                            mma_e4m3(tmem + sb * C::NS, kd + uint64_t(kk * 2), qd + uint64_t(kk * 2),
                                     idesc_s, kk > 0);
                        tc::mma_commit(&bar[kSFull + sb]);
                        tc::mma_commit(&bar[kKEmpty + ks]);
                        if (t == it.ntiles - 1) tc::mma_commit(&bar[kQEmpty + qb]);
                    }
                    if (t >= 1) {
                        const int gp = g + t - 1;
                        const int vs = gp % kVStages;
                        ok = mbar_wait(&bar[kPFull], gp & 1, p.err);
                        if (ok) ok = mbar_wait(&bar[kVFull + vs], (gp / kVStages) & 1, p.err);
                        if (!ok) break;
                        tc::fence_after_sync();
                        // V^T as the MN-major A operand: 128 channels are one 128-byte
                        // atom, 8-key groups 1 KB apart, 32 keys a step.
                        const uint64_t vd =
                            tc::smem_desc_sw128(v_base + vs * kTileBytes, kTileBytes, 1024);
#pragma unroll
                        for (int kk = 0; kk < kBK / 32; ++kk)
                            mma_e4m3(tmem + C::kTmemO, vd + uint64_t((kk * 32 * 128) >> 4),
                                     pd + uint64_t((kk * 32 * 16) >> 4), idesc_o,
                                     t > 1 || kk > 0);
                        tc::mma_commit(&bar[kODone]);
                        tc::mma_commit(&bar[kVEmpty + vs]);
                    }
                }
                g += it.ntiles;
                ++itq;
            }
        }
    } else {
        // ---------------------------------------------------- softmax + epilogue
        const int kw = warp & 3;                     // key warp: TMEM lanes 32 kw ..
        const int grp = warp >> 2;                   // column group
        const int k = kw * 32 + lane;                // key of the tile == TMEM lane
        const uint32_t lane_base = uint32_t(kw * 32) << 16;
        float *red = reinterpret_cast<float *>(smem + C::red);
        float *lred = reinterpret_cast<float *>(smem + C::lred);
        const int g_inv = (1 << 16) / G + 1;         // (cg * g_inv) >> 16 = cg / G for cg < 16
        int g = 0, iter = 0, itq = 0;
        int ss = 0, sph = 0;                         // stage and phase of the scale ring
        bool ok = true;
        for (int j = 0; j < items; ++j, ++iter) {
            const Fp8Item it = fp8_item(p, cum, walk, j);
            int row0, nrows;
            seq_rows(p, it.b, row0, nrows);
            nrows = min(nrows, p.num_q_rows - row0);
            // Column cg = (row cg / G, head cg % G); chunk h of this group holds the
            // columns col(h) .. col(h) + 3.  Columns past the item's rows hold an
            // earlier item's scores and are never written out.
            const auto col = [&](int h) { return 4 * (h * C::kGroups + grp); };
            const int cols = nrows * G;
            // Pairs of columns go through the packed fp32 instructions.  m is 0 until
            // the first tile sets it: a column that sees no key there sees none at
            // all in this item, as the mask only hides a sequence's last keys.
            float2 f[NCH][2], m[NCH][2], l[NCH][2];
#pragma unroll
            for (int h = 0; h < NCH; ++h)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    m[h][c] = l[h][c] = f[h][c] = make_float2(0.f, 0.f);
            if (it.ntiles > 0) {
                const int qb = itq % kQBufs;
                ok = ok && mbar_wait(&bar[kQFull + qb], (itq / kQBufs) & 1, p.err);
                const float *qf = reinterpret_cast<const float *>(smem + C::qf) + qb * 16;
#pragma unroll
                for (int h = 0; h < NCH; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        f[h][c] = make_float2(qf[col(h) + 2 * c] * p.qk_scale_log2,
                                              qf[col(h) + 2 * c + 1] * p.qk_scale_log2);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kQEmpty + qb]);
                ++itq;
            }
            // First key that some row may not see: row i sees keys j < full + i (all
            // L without the causal mask).
            const bool masked_rows = p.causal && nrows > 1;
            const int full = masked_rows ? it.L - nrows + 1 : it.L;
            const auto sees = [&](int cg, int key) {
                return key < it.L && (!masked_rows || key < full + ((cg * g_inv) >> 16));
            };
            // Every warp runs every named barrier of every tile, even after a
            // wait gave up (ok == false), so no warp can strand the others.
            for (int t = 0; t < it.ntiles; ++t) {
                const int gg = g + t;
                const int sb = gg & 1;
                const int t0 = it.start + t * kBK;
                const bool tail = t0 + kBK > full;               // uniform over the CTA
                // ---- scales and scores of this key -------------------------------
                // both polls in flight together
                const bool sc_in = mbar_try_wait(&bar[kScFull + ss], sph);
                const bool s_in = mbar_try_wait(&bar[kSFull + sb], (gg >> 1) & 1);
                if (!sc_in) ok = ok && mbar_wait(&bar[kScFull + ss], sph, p.err);
                float2 sc = reinterpret_cast<const float2 *>(smem + C::sc)[ss * kBK + k];
                if (!s_in) ok = ok && mbar_wait(&bar[kSFull + sb], (gg >> 1) & 1, p.err);
                tc::fence_after_sync();
                float2 s[NCH][2];                                // score, then score - m
                float raw[NCH][8];
                const uint32_t s_at = tmem + lane_base + sb * C::NS;
                tmem_ld_scores(s_at + 2 * col(0), s_at + 2 * col(NCH - 1), raw);
#pragma unroll
                for (int h = 0; h < NCH; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        s[h][c] = __ffma2_rn(make_float2(raw[h][4 + 2 * c], raw[h][5 + 2 * c]),
                                             make_float2(0.0625f, 0.0625f),
                                             make_float2(raw[h][2 * c], raw[h][2 * c + 1]));
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar[kSFree + sb]);
                    mbar_arrive(&bar[kScEmpty + ss]);
                }
                if (++ss == kScStages) { ss = 0; sph ^= 1; }
                if (tail && t0 + k >= it.L) sc = make_float2(0.f, 0.f);
                const int ve_raw = int((__float_as_uint(sc.y) >> 23) & 0xffu) - 127;
                const int ve = min(max(ve_raw, kMinVExp), kMaxVExp);
                const float vexp = static_cast<float>(ve);
                const float v_inv = pow2i(-ve);
                // (a scale past the range would saturate: NaN instead)
                const float v_mul = ve_raw > kMaxVExp ? __uint_as_float(0x7fffffffu)
                                                      : sc.y * v_inv * kWeightTop;
                float top = -INFINITY;
#pragma unroll
                for (int h = 0; h < NCH; ++h) {
                    if (col(h) >= cols) continue;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        s[h][c] = __ffma2_rn(__fmul2_rn(s[h][c], make_float2(sc.x, sc.x)), f[h][c],
                                             make_float2(vexp, vexp));
                        if (tail) {
                            if (!sees(col(h) + 2 * c, t0 + k)) s[h][c].x = -INFINITY;
                            if (!sees(col(h) + 2 * c + 1, t0 + k)) s[h][c].y = -INFINITY;
                        }
                        s[h][c] = __fadd2_rn(s[h][c], make_float2(-m[h][c].x, -m[h][c].y));
                        top = fmax3(top, s[h][c].x, s[h][c].y);
                    }
                }
                // ---- does any column's reference have to move? --------------------
                // One barrier with an OR answers for the group; the columns' maxima
                // are only taken where it says yes (the first tile and a few more).
                const bool moved = t == 0 || named_or(1 + grp, 128, top > kLazy);
                float2 alpha[NCH][2];
                if (moved) {
#pragma unroll
                    for (int h = 0; h < NCH; ++h) {
                        if (col(h) >= cols) continue;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float w0 = warp_max_redux(s[h][c].x);
                            const float w1 = warp_max_redux(s[h][c].y);
                            if (lane == 0)
                                *reinterpret_cast<float2 *>(red + kw * 16 + col(h) + 2 * c) =
                                    make_float2(w0, w1);
                        }
                    }
                    named_sync(1 + grp, 128);
                    const float lazy = t == 0 ? -INFINITY : kLazy;
                    const auto raise = [&](int cg, float &sx, float &mx, float &lx, float &ax) {
                        const float up = fmaxf(fmaxf(red[cg], red[16 + cg]),
                                               fmaxf(red[32 + cg], red[48 + cg]));
                        const bool move = up > lazy;
                        ax = move && t > 0 ? fast_exp2(-up) : 1.f;
                        if (move) {
                            mx += up;
                            sx -= up;
                            lx *= ax;
                        }
                    };
#pragma unroll
                    for (int h = 0; h < NCH; ++h) {
                        if (col(h) >= cols) continue;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            raise(col(h) + 2 * c, s[h][c].x, m[h][c].x, l[h][c].x, alpha[h][c].x);
                            raise(col(h) + 2 * c + 1, s[h][c].y, m[h][c].y, l[h][c].y,
                                  alpha[h][c].y);
                        }
                    }
                }
                uint32_t code[NCH][4];   // four columns of a term to a word
#pragma unroll
                for (int h = 0; h < NCH; ++h) {
                    if (col(h) >= cols) continue;
                    float2 w[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float2 e = make_float2(fast_exp2(s[h][c].x), fast_exp2(s[h][c].y));
                        l[h][c] = __ffma2_rn(e, make_float2(v_inv, v_inv), l[h][c]);
                        w[c] = __fmul2_rn(e, make_float2(v_mul, v_mul));
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t lo = to_e4m3x2(w[0].x, w[0].y);
                        const uint32_t hi = to_e4m3x2(w[1].x, w[1].y);
                        code[h][u] = lo | (hi << 16);
                        if (u < 3) {
                            take_rest(lo, w[0].x, w[0].y);
                            take_rest(hi, w[1].x, w[1].y);
                            const float2 ratio = make_float2(term_ratio(u), term_ratio(u));
                            w[0] = __fmul2_rn(w[0], ratio);
                            w[1] = __fmul2_rn(w[1], ratio);
                        }
                    }
                }
                if (t >= 1) {
                    // O^T(t-1) is complete: P^T may be overwritten and O^T
                    // rescaled (thread = channel lane).
                    ok = ok && mbar_wait(&bar[kODone], (gg - 1) & 1, p.err);
                    tc::fence_after_sync();
                    if (moved) {   // identical in every thread of the group
#pragma unroll
                        for (int h = 0; h < NCH; ++h) {
                            if (col(h) >= cols) continue;
                            float o[16];
                            const uint32_t oc = tmem + lane_base + C::kTmemO + 4 * col(h);
                            tmem_ld_cols<16>(oc, o);
#pragma unroll
                            for (int c = 0; c < 16; c += 2) {
                                o[c] *= alpha[h][(c >> 1) & 1].x;
                                o[c + 1] *= alpha[h][(c >> 1) & 1].y;
                            }
                            tmem_st_cols<16>(oc, o);
                        }
                        tc::tmem_wait_st();
                    }
                }
                // ---- V rows that some or all rows must not see --------------------
                if (tail) {
                    const int vs = gg % kVStages;
                    ok = ok && mbar_wait(&bar[kVFull + vs], (gg / kVStages) & 1, p.err);
                    uint4 *row = reinterpret_cast<uint4 *>(smem + C::vring + vs * kTileBytes) + k * 8;
                    bool clear = t0 + k >= it.L;     // past the end: may hold anything
                    if (t0 + k >= full && t0 + k < it.L) {
                        // A later token of the call: a NaN in its V, or a scale that counts
                        // as NaN, must not reach the rows before it through 0 * NaN.  Its V
                        // becomes 0, and its weight NaN for the rows that see it and 0 for
                        // the others.
                        bool nan = v_mul != v_mul;
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const uint4 x = row[u];
                            const uint32_t word[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                nan |= __vcmpeq4(word[v] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u;
                        }
                        if (nan) {
                            clear = true;
#pragma unroll
                            for (int h = 0; h < NCH; ++h)
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    if (col(h) >= cols) continue;
                                    const bool seen = sees(col(h) + c, t0 + k);
#pragma unroll
                                    for (int u = 0; u < 4; ++u)
                                        code[h][u] &= ~(0xffu << (8 * c));
                                    code[h][0] |= (seen ? 0x7fu : 0u) << (8 * c);
                                }
                        }
                    }
                    named_sync(3, 128 * C::kGroups);
                    if (clear && grp == 0) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) row[u] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
#pragma unroll
                for (int h = 0; h < NCH; ++h)
                    if (col(h) < cols)
                        *reinterpret_cast<uint4 *>(smem + C::p + 4 * col(h) * kBK + 16 * k) =
                            make_uint4(code[h][0], code[h][1], code[h][2], code[h][3]);
                tc::fence_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kPFull]);
            }

            // ---- item epilogue ----------------------------------------------------
            // Rolled over pairs of columns and short on purpose: it runs once an item,
            // from a cold instruction cache (all 8 columns of a warp unrolled: 10000
            // cycles; a pair at a time: 3000 to 5000).  The row sums and references go
            // through shared memory while the last P.V is still in flight.
            float *lb = lred + (iter & 1) * 80;   // [4 key warps][16 columns], then m[16]
            // (halving butterfly: the warp's sum of column n ends up in the lanes whose
            // upper bits are n)
            float part[4 * NCH];
#pragma unroll
            for (int n = 0; n < 4 * NCH; ++n)
                part[n] = n & 1 ? l[n >> 2][(n >> 1) & 1].y : l[n >> 2][(n >> 1) & 1].x;
            int at = 0, o = 16;
#pragma unroll
            for (int n = 2 * NCH; n > 0; n >>= 1, o >>= 1) {
                const bool upper = lane & o;
                at += upper ? n : 0;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float keep = upper ? part[n + i] : part[i];
                    const float give = upper ? part[i] : part[n + i];
                    part[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
            for (; o > 0; o >>= 1) part[0] += __shfl_xor_sync(0xffffffffu, part[0], o);
            if ((lane & (32 / (4 * NCH) - 1)) == 0) lb[kw * 16 + col(at >> 2) + (at & 3)] = part[0];
            if (kw == 0 && lane == 0) {
#pragma unroll
                for (int h = 0; h < NCH; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<float2 *>(lb + 64 + col(h) + 2 * c) = m[h][c];
            }
            named_sync(1 + grp, 128);
            if (it.ntiles > 0)
                ok = ok && mbar_wait(&bar[kODone], (g + it.ntiles - 1) & 1, p.err);
            tc::fence_after_sync();
            const bool has_o = ok && it.ntiles > 0;
            const int ch = k;   // output channel of this thread
            const size_t head0 = size_t(row0) * p.num_q_heads + it.kvh * G;
            const size_t slot0 = size_t(it.slot) * kGqaSlotCols;
#pragma unroll 1
            for (int x = 0; x < 4 * NCH; x += 2) {
                const int c0 = col(x >> 2) + (x & 3);
                if (c0 >= cols) break;
                float term[4][2];
                tmem_ld_terms(tmem + lane_base + C::kTmemO + 4 * (c0 & ~3) + (c0 & 3), term);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int cg = c0 + u, i = (cg * g_inv) >> 16;
                    if (i >= nrows) continue;
                    float acc = term[3][u];
#pragma unroll
                    for (int v = 2; v >= 0; --v) acc = fmaf(acc, 1.f / term_ratio(v), term[v][u]);
                    acc = has_o ? acc * (1.f / kWeightTop) : 0.f;
                    const float lsum = (lb[cg] + lb[16 + cg]) + (lb[32 + cg] + lb[48 + cg]);
                    // no visible key: no sum, no reference
                    const float mx = lsum == 0.f ? -INFINITY : lb[64 + cg];
                    if (it.direct) {
                        const float t2 = p.sink ? p.sink[it.kvh * G + cg - i * G] * kLog2e : -INFINITY;
                        const float Mf = fmaxf(mx, t2);
                        float so = 1.f, Z = lsum;
                        if (Mf != -INFINITY) {
                            so = fast_exp2(mx - Mf);    // 0 when mx = -inf
                            Z = lsum * so + fast_exp2(t2 - Mf);
                        }
                        const float v = Z == 0.f ? 0.f : __fdividef(acc * so, Z);
                        const size_t row = head0 + i * p.num_q_heads + cg - i * G;
                        p.out[row * kD + ch] = static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xffffu);
                        if (ch == 0 && p.lse)
                            p.lse[row] = Z == 0.f ? -INFINITY : (Mf + fast_log2(Z)) * kLn2;
                    } else {
                        const size_t base = slot0 + cg;
                        p.ws_o[base * kD + ch] = acc;
                        if (ch == 0) {
                            p.ws_m[base] = mx * kLn2;
                            p.ws_l[base] = lsum;
                        }
                    }
                }
            }
            tc::fence_before_sync();
            // The CTA holding the unit's first tile publishes where its pieces are.
            if (it.first && threadIdx.x == 0 && p.unit_slots)
                p.unit_slots[it.b * (p.num_q_heads / G) + it.kvh] =
                    make_int2(it.slot, fp8_pieces(p, cum, walk, it));
            g += it.ntiles;
        }
        pdl_launch_dependents();
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == C::kWarpMma) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int NC>
cudaError_t launch_nc(const Fp8DecodeParams &p, int ctas, cudaStream_t stream) {
    const size_t smem = smem_bytes<NC>(p.batch);
    auto kern = gqa_decode_fp8_kernel<NC>;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    kern<<<dim3(static_cast<unsigned>(ctas)), Cfg<NC>::kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

int fp8_decode_ctas(int num_sms) { return kCtasPerSm * num_sms; }

cudaError_t launch_gqa_decode_fp8(const Fp8DecodeParams &p, int ctas, cudaStream_t stream) {
    const int cols = p.max_q_len * p.group;
    if (cols < 1 || cols > 16) return cudaErrorInvalidValue;
    if (cols <= 4) return launch_nc<4>(p, ctas, stream);
    if (cols <= 8) return launch_nc<8>(p, ctas, stream);
    return launch_nc<16>(p, ctas, stream);
}

}  // namespace attn
