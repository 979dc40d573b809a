// gqa_decode_codes.cuh -- split-K decode attention over a cache held in codes, head_dim 128:
// 8 bits (e4m3, an fp32 scale per block of tokens and KV head) or 4 (e2m1; keys with a power of
// two for every 32 channels, values with an fp32 scale a token).
//
//   s_j = scale q . (ks_j K_j),  p_j = e^(s_j - m)
//   out = sum_j p_j (vs_j V_j) / (sum_j p_j + e^(sink - m))
//
// First for 8 bits; what 4 bits change follows.
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
// 4 bits.  A copy unpacks 16 codes into the first 8 of 16 bytes, as the MMAs (e2m1 times e4m3
// or e5m2) want them, so a tile is as large in shared memory and half as large in memory: its
// softmax, not its stream, is what has to be quick.
//   A key's scale differs between its four groups of channels, so each group's product goes to
//     columns of its own and the thread that owns the key adds the four up.  With 16 columns
//     the two terms of q are two MMAs into the same columns (q1 in e5m2, which holds q1 / 16).
//   weights = w0 + 2^-4 (w1 + w2) + 2^-10 w3 in e5m2 (3 bits; the upper byte of an f16 number is
//     one): w0 and w3 rounded, w1 and w2 what is left cut off.  Half a step of w0 is at most
//     2^-3 of it, a cut leaves three bits less, half a step of w3 is three bits and one down: at
//     most 2^-13 of a weight, 2^-15 more where what w0 leaves becomes an f16 number, so 2^-12;
//     or 2^-34 of the reference's where that is more (what is below 2^-38 of it is lost).  w3
//     cannot start lower: 64 times what is left of the largest weight is 2^15.  (Four cuts of
//     an f16 number, all in one unit, erred by 2^-11, or 2^-27 and always toward 0, for the same
//     time but with draft rows, 71.3 and 72.1 us.  Four e4m3 terms are those of 8 bits; they
//     were not timed since the MMA warp walks as one.)
//   Up to 4 columns two groups of softmax warps take the tiles in turns, each with its own
//     weights, reference and output, joined at an item's end: what one waits for (scores, the
//     barrier, the last P.V) the other uses.  A warp for each contraction's MMAs (one for both
//     held the scores of the next tile back: 72.5 and 62.0 us), and one producer for both.
//
// What bounds it, 8 bits.  Up to 4 columns the stream of codes: 64 sequences of 32 + 8
// heads and 512 to 8192 keys (580 MB) take 98 us, 5.9 TB/s with everything,
// about 7 while the stream runs.  The rest is 5 us until the first scores
// (range, page table, first tile), the ends of the CTAs and the reduce.  With 16
// columns the softmax of a tile takes longer than its bytes (1 to 4 draft
// rows of 4 heads: 82 us for 318 MB).  What runs
// once an item (opening it, the first tile's maxima, the epilogue) runs from a cold
// instruction cache, at 100 cycles and more per eight instructions: hence the rolled
// loops and the care for code length there.  (Heads taken one after the other 114.9 us, P
// through a swizzled K-major layout 201 instead of 158 us for the draft rows, one group of
// warps for 16 columns 147 instead of 103, 3 V stages the same.)
// 4 bits: the same 64 sequences (309 MB) take 57.2 us, 5.4 TB/s; 131072 keys of one sequence
// (143 MB) 33.0 us, of which 5.5 are the reduce and about 6 the start; 1 to 4 draft rows 72 us,
// the softmax's issue slots (half of all, the rest lost to waits between its steps and to
// instructions that are not yet there).
#pragma once

#include <cuda_fp8.h>

#include "cache_ops.h"
#include "fp8_items.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace attn {
namespace codes {

constexpr int kD = 128;
constexpr int kBK = kGqaTcTileKeys;          // 128 keys per tile
constexpr int kStages = 3;                   // K tiles in flight
// V tiles in flight (kVs): as many as leave two CTAs room (8 bits: three measured the same).
// 4 bits, 4 columns: three, and two where the table of that many sequences takes the third's
// room (512 sequences of 512 to 1024 keys: 135 us, 168 with three and one CTA an SM; 1024 of 64
// keys 97 and 183; 120 and 87 since).
__host__ __device__ constexpr int v_stages(bool fp4, int nc) { return fp4 && nc == 4 ? 3 : 2; }
constexpr size_t kCtaSmem = 113 * 1024;      // a CTA of two on an SM
constexpr int kTileBytes = kBK * kD;         // 16 KB (4 bits: 16 codes in the first 8 of 16 bytes)
constexpr int kKGroups = 4;                  // 4 bits: scales of a key, 32 channels each
constexpr int kScStages = 4;                 // tiles of scales in flight
constexpr int kQBufs = 2;
constexpr int kCtasPerSm = 2;
// A lower kLazy leaves more of the e4m3 range below the reference, a higher one moves it
// less often (kLazy 1, 2, 3, 4: 64 single rows 100 us each, 1 to 4 draft rows of 4 heads 107,
// 98, 93, 92).
constexpr float kLazy = 3.f;                 // base 2
// Weights reach 2^kLazy * 2 * this: 256 of e4m3's 448, 2^15 of e5m2's 57344.
__host__ __device__ constexpr float weight_top(bool fp4) { return fp4 ? 2048.f : 16.f; }
// Each term's unit over the next one's (see above).
__host__ __device__ constexpr float term_ratio(bool fp4, int u) {
    return fp4 ? (u == 0 ? 16.f : u == 1 ? 1.f : 64.f) : u < 2 ? 32.f : 32768.f;
}
constexpr int kBarBytes = 304;
constexpr int kMinVExp = -64, kMaxVExp = 64;

// Columns (query rows x heads) come in chunks of four: a chunk's S columns (and Q
// rows) are [2 terms][4], its O columns (and P columns) [4 terms][4].  More than one
// chunk takes two groups of four softmax warps; group g has the chunks g, g + 2.  Chunks
// past an item's columns are skipped.
template <int NC, bool kFp4, int kVs>
struct Cfg {
    static constexpr int kChunks = NC / 4;
    // kTurns: the two groups of softmax warps take the tiles in turns, each with weights,
    // references and an output of its own, which an item's end joins.
    static constexpr bool kTurns = kFp4 && NC == 4;
    static constexpr int kGroups = NC > 4 || kTurns ? 2 : 1;
    static constexpr int kColGroups = kTurns ? 1 : kGroups;          // that share a tile's columns
    static constexpr int kBufs = kTurns ? 2 : 1;                     // of P and O
    static constexpr int NCH = kChunks / kColGroups;                 // chunks per group
    // 4 bits: queries' two terms in columns of their own (as in 8 bits), or added up.
    static constexpr bool kTermCols = !kFp4 || NC <= 8;
    // N of a score MMA, and the columns of a score buffer: 4 bits, a block of NS columns
    // for each group of channels
    static constexpr int NS = !kTermCols || kChunks < 2 ? 16 : 8 * kChunks;
    static constexpr int kSCols = kFp4 ? kKGroups * NS : NS;
    static constexpr int NP = 16 * kChunks;                          // N of the output MMA
    static constexpr int kTmemO = 2 * kSCols;                        // after two score buffers
    static constexpr int kTmemUsed = kTmemO + kBufs * NP;
    static constexpr int kTmemCols = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : 256;
    static constexpr int kQBytes = (kTermCols ? 1 : 2) * NS * 128;   // added up: a tile a term
    // Rows of Q: the first of column c's, and from there to its second term's.
    static constexpr int kTermRows = kTermCols ? 4 : NS;
    static __host__ __device__ constexpr int term0(int c) { return kTermCols ? 2 * c - (c & 3) : c; }
    static constexpr int kWarpK = 4 * kGroups, kWarpV = kWarpK + 1, kWarpMma = kWarpK + 2,
                         kWarpAux = kWarpK + 3;
    static constexpr bool kTwoMmaWarps = kFp4;   // kWarpV's is the outputs' (kWarpK loads both)
    static constexpr int kThreads = 32 * (4 * kGroups + 4);
    // shared memory
    static constexpr int kring = 0;
    static constexpr int vring = kring + kStages * kTileBytes;
    static constexpr int q = vring + kVs * kTileBytes;          // [kQBufs][terms, rows][128 B]
    static constexpr int p = q + kQBufs * kQBytes;                   // [chunks][128 keys][16 B]
    static constexpr int sc = p + kBufs * NP * 128;                  // [kScStages]: 128 {ks, vs}; 4 bits: ks, vs
    static constexpr int red = sc + kScStages * kBK * 8;             // float [4][16] tile max
    // (turns: of each group; the maxima have room for one row of 4 columns a group)
    // float [2][kBufs][5][16]: row sums, references
    static constexpr int lred = red + 4 * 16 * 4;
    static constexpr int qf = lred + 2 * kBufs * 5 * 16 * 4;         // float [kQBufs][16] 2^-a
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
    kPFull = kSFree + 2, kODone = kPFull + 2,           // [2] each: of a buffer of P and O
    kNumBars = kODone + 2
};
static_assert((kScStages & (kScStages - 1)) == 0, "stages of scales are found with shifts");
static_assert(kStages == 3 && kNumBars * 8 <= kBarBytes, "barrier layout");
static_assert(sizeof(Fp8Range) <= 32, "range slot");

template <int NC, bool kFp4, int kVs>
size_t smem_bytes(int batch) {
    return size_t(Cfg<NC, kFp4, kVs>::items) + sizeof(int2) * size_t(batch + 1);
}

// Element types of kind::f8f6f4.
constexpr uint32_t kE4m3 = 0, kE5m2 = 1, kE2m1 = 5;

// Instruction descriptor of kind::f8f6f4, fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f8f6f4(uint32_t a, uint32_t b, int M, int N, int a_mn,
                                                    int b_mn) {
    return (1u << 4) | (a << 7) | (b << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
           (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void mma_f8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// One lane of the warp (all lanes take part).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(one));
    return one != 0;
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

// Eight columns of each of the four groups' blocks, one wait for all.
__device__ __forceinline__ void tmem_ld_group_terms(uint32_t t, float (&v)[kKGroups][8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%33];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%34];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%24, %25, %26, %27, %28, %29, %30, %31}, [%35];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&f"(v[0][0]), "=&f"(v[0][1]), "=&f"(v[0][2]), "=&f"(v[0][3]),
          "=&f"(v[0][4]), "=&f"(v[0][5]), "=&f"(v[0][6]), "=&f"(v[0][7]),
          "=&f"(v[1][0]), "=&f"(v[1][1]), "=&f"(v[1][2]), "=&f"(v[1][3]),
          "=&f"(v[1][4]), "=&f"(v[1][5]), "=&f"(v[1][6]), "=&f"(v[1][7]),
          "=&f"(v[2][0]), "=&f"(v[2][1]), "=&f"(v[2][2]), "=&f"(v[2][3]),
          "=&f"(v[2][4]), "=&f"(v[2][5]), "=&f"(v[2][6]), "=&f"(v[2][7]),
          "=&f"(v[3][0]), "=&f"(v[3][1]), "=&f"(v[3][2]), "=&f"(v[3][3]),
          "=&f"(v[3][4]), "=&f"(v[3][5]), "=&f"(v[3][6]), "=&f"(v[3][7])
        : "r"(t), "r"(t + 16), "r"(t + 32), "r"(t + 48)
        : "memory");
}
// Four columns of each of the four groups' blocks, of two chunks, one wait for all.
__device__ __forceinline__ void tmem_ld_groups(uint32_t t0, uint32_t t1,
                                               float (&v)[2][kKGroups][4]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%4, %5, %6, %7}, [%33];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%8, %9, %10, %11}, [%34];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%12, %13, %14, %15}, [%35];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%16, %17, %18, %19}, [%36];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%20, %21, %22, %23}, [%37];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%24, %25, %26, %27}, [%38];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%28, %29, %30, %31}, [%39];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&f"(v[0][0][0]), "=&f"(v[0][0][1]), "=&f"(v[0][0][2]), "=&f"(v[0][0][3]),
          "=&f"(v[0][1][0]), "=&f"(v[0][1][1]), "=&f"(v[0][1][2]), "=&f"(v[0][1][3]),
          "=&f"(v[0][2][0]), "=&f"(v[0][2][1]), "=&f"(v[0][2][2]), "=&f"(v[0][2][3]),
          "=&f"(v[0][3][0]), "=&f"(v[0][3][1]), "=&f"(v[0][3][2]), "=&f"(v[0][3][3]),
          "=&f"(v[1][0][0]), "=&f"(v[1][0][1]), "=&f"(v[1][0][2]), "=&f"(v[1][0][3]),
          "=&f"(v[1][1][0]), "=&f"(v[1][1][1]), "=&f"(v[1][1][2]), "=&f"(v[1][1][3]),
          "=&f"(v[1][2][0]), "=&f"(v[1][2][1]), "=&f"(v[1][2][2]), "=&f"(v[1][2][3]),
          "=&f"(v[1][3][0]), "=&f"(v[1][3][1]), "=&f"(v[1][3][2]), "=&f"(v[1][3][3])
        : "r"(t0), "r"(t0 + 16), "r"(t0 + 32), "r"(t0 + 48), "r"(t1), "r"(t1 + 16), "r"(t1 + 32),
          "r"(t1 + 48)
        : "memory");
}

// Whether the phase with the given parity is complete, now.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
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

// r minus sixteen times the f16 numbers of c.
__device__ __forceinline__ void take_sixteenfold(uint32_t c, float2 &r) {
    const unsigned short minus16 = 0xcc00;   // f16
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "fma.rn.f32.f16 %0, l, %3, %0;\n\tfma.rn.f32.f16 %1, h, %3, %1;\n\t}"
        : "+f"(r.x), "+f"(r.y)
        : "r"(c), "h"(minus16));
}

// The same in e5m2.
__device__ __forceinline__ uint32_t to_e5m2x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
}

// Four weights as four e5m2 terms each, a term of all four to a word.  The first is the
// nearest; sixteen times what it leaves (exact in fp32, of either sign) becomes an f16 number.
// The upper byte of such a number is an e5m2 number: that is the next term, cut off, and so
// once more; 64 times the rest is rounded again.  (Every product is by a power of two.)
__device__ __forceinline__ void e5m2_terms(const float2 &a, const float2 &b, uint32_t (&code)[4]) {
    code[0] = to_e5m2x2(a.x, a.y) | (to_e5m2x2(b.x, b.y) << 16);
    const float2 unit = make_float2(term_ratio(true, 0), term_ratio(true, 0));
    float2 ra = __fmul2_rn(a, unit), rb = __fmul2_rn(b, unit);
    take_sixteenfold(__byte_perm(code[0], 0, 0x1404), ra);
    take_sixteenfold(__byte_perm(code[0], 0, 0x3424), rb);
    uint32_t x, y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(ra.y), "f"(ra.x));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(rb.y), "f"(rb.x));
#pragma unroll
    for (int u = 1; u < 3; ++u) {
        code[u] = __byte_perm(x, y, 0x7531);
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(x & 0xff00ff00u));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(y) : "r"(y & 0xff00ff00u));
    }
    const uint32_t last = 0x54005400u;                           // term_ratio(true, 2), twice
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(last));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(y) : "r"(last));
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(lo) : "r"(x));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(hi) : "r"(y));
    code[3] = uint32_t(lo) | (uint32_t(hi) << 16);
}

// The scales that the four e8m0 bytes of w stand for (255: NaN), by way of bf16.
__device__ __forceinline__ void e8m0x4(uint32_t w, float (&f)[kKGroups]) {
    uint32_t a, b;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\tcvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
    f[0] = __uint_as_float(a << 16);
    f[1] = __uint_as_float(a & 0xffff0000u);
    f[2] = __uint_as_float(b << 16);
    f[3] = __uint_as_float(b & 0xffff0000u);
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

// The CTA holding the unit's first tile publishes where its pieces are.  (4 bits: from the
// producer warp, as the softmax warps' time between items counts: draft rows 73.7 us and 71.4.)
__device__ __forceinline__ void publish(const Fp8DecodeParams &p, const int2 *cum,
                                        const Fp8Range &w, const Fp8Item &it) {
    if (it.first && p.unit_slots)
        p.unit_slots[it.b * (p.num_q_heads / p.group) + it.kvh] =
            make_int2(it.slot, it.direct ? 1 : fp8_pieces(p, cum, w, it));
}

// K or V producer: walks this CTA's items and tiles and lets lane 0 issue the
// boxes of each tile into the ring.
template <bool kIsK, int NC, int kVs>
__device__ __forceinline__ void produce(const Fp8DecodeParams &p, const int2 *cum, const Fp8Range &w,
                                        uint8_t *smem, uint64_t *bar, int lane) {
    const CUtensorMap *map = kIsK ? &p.k_map : &p.v_map;
    uint64_t *full = bar + (kIsK ? kKFull : kVFull);
    uint64_t *empty = bar + (kIsK ? kKEmpty : kVEmpty);
    uint8_t *ring = smem + (kIsK ? Cfg<NC, false, kVs>::kring : Cfg<NC, false, kVs>::vring);
    constexpr int kN = kIsK ? kStages : kVs;
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

// Where one operand's producer is in the walk of a CTA's tiles.
struct Walk {
    Fp8Item it;
    int j, t, g;                   // item, tile of it, tile of the walk
    int cached, page, slot;        // 32 boxes' places, one per lane
    bool more;
};

// Producer of the 4-bit kernel: the boxes of both operands, a box a lane.  Keys and values go
// at their own pace: a value stage is free a softmax later than its tile's key stage, and keys
// that waited for it came too late (64 sequences 62.0 us in step and 60.2 so, 131072 keys 35.9
// and 33.5; keys sent a tile ahead of the values, each wait blocking, 1.5 more than so).
template <int NC, int kVs>
__device__ __forceinline__ void produce_both(const Fp8DecodeParams &p, const int2 *cum,
                                             const Fp8Range &w, uint8_t *smem, uint64_t *bar,
                                             int lane) {
    using C = Cfg<NC, true, kVs>;
    const int box_rows = p.box_rows;        // 128, 64, 32, 16 or 8
    const int box_shift = 31 - __clz(box_rows);
    const int nb = kBK >> box_shift;        // row boxes per tile
    const uint32_t box_bytes = uint32_t(box_rows) * 64u;        // in memory: what a copy counts
    const int items = w.count();
    Walk k, v;
    const auto open = [&](Walk &x) {        // the next item with tiles
        x.more = false;
        x.t = 0;
        x.cached = -1;
        while (!x.more && ++x.j < items) {
            x.it = fp8_item(p, cum, w, x.j);
            x.more = x.it.ntiles > 0;
            if (&x == &k && lane == 0 && !x.more) publish(p, cum, w, x.it);   // (else: step)
        }
    };
    // Sends for the walk's tile, if its stage is free; n stages.
    const auto step = [&](Walk &x, bool is_k, uint64_t *full, uint64_t *empty, int n,
                          const CUtensorMap *map, uint8_t *ring) -> bool {
        if (!x.more) return false;
        const int s = x.g % n;
        if (x.g >= n) {
            const bool is_free = mbar_test(&empty[s], ((x.g / n) - 1) & 1);
            if (!__shfl_sync(0xffffffffu, is_free, 0)) return false;
        }
        const int key0 = x.it.start + x.t * kBK;
        const int live = min(nb, (x.it.L - key0 + box_rows - 1) >> box_shift);
        const int box0 = x.t * nb;                               // box index in the item
        if ((box0 >> 5) != x.cached) {
            x.cached = box0 >> 5;
            lookup_boxes(p, x.it, x.cached, lane, is_k, x.page, x.slot);
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[s], uint32_t(live) * box_bytes);
        __syncwarp();
        const int r = lane - (box0 & 31);
        if (r >= 0 && r < live) {
            if (x.page < 0)
                mbar_complete_tx(&full[s], box_bytes);           // skipped bad page
            else
                tma_load_4d(ring + s * kTileBytes + r * box_rows * 128, map, &full[s], 0, x.slot,
                            x.it.kvh, x.page);
        }
        __syncwarp();
        if (is_k && x.t == 0 && lane == 0) publish(p, cum, w, x.it);
        ++x.g;
        if (++x.t == x.it.ntiles) open(x);
        return true;
    };
    k.j = v.j = -1;
    k.g = v.g = 0;
    open(k);
    open(v);
    unsigned long long since = 0;           // of the last step that found neither stage free
    while (k.more || v.more) {
        const bool a =
            step(k, true, bar + kKFull, bar + kKEmpty, kStages, &p.k_map, smem + C::kring);
        const bool b = step(v, false, bar + kVFull, bar + kVEmpty, kVs, &p.v_map, smem + C::vring);
        if (a || b) {
            since = 0;
            continue;
        }
        const unsigned long long now = __shfl_sync(0xffffffffu, global_ns(), 0);
        if (since == 0) since = now;
        if (now - since > kWaitLimitNs) {
            if (lane == 0) atomicOr(p.err, kErrWaitTimeout);
            break;
        }
    }
    // (after a wait that gave up: the merge reads what every unit publishes)
    if (lane == 0) {
        if (k.more && k.t == 0) publish(p, cum, w, k.it);
        for (int j = k.j + 1; j < items; ++j) publish(p, cum, w, fp8_item(p, cum, w, j));
    }
    // Every copy this warp issued must land before the CTA may leave.
    if (lane == 0) {
        for (int i = max(0, k.g - kStages); i < k.g; ++i)
            mbar_wait(&bar[kKFull + i % kStages], (i / kStages) & 1, p.err);
        for (int i = max(0, v.g - kVs); i < v.g; ++i)
            mbar_wait(&bar[kVFull + i % kVs], (i / kVs) & 1, p.err);
    }
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
template <int NC, bool kFp4, int kVs>
__device__ __forceinline__ void feed(const Fp8DecodeParams &p, const int2 *cum, const Fp8Range &w,
                                     uint8_t *smem, uint64_t *bar, int lane) {
    using C = Cfg<NC, kFp4, kVs>;
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
        uint8_t *qs = smem + C::q + qb * C::kQBytes;
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
            uint8_t *dst = qs + (C::term0(c) + (li & 4) / 4 * C::kTermRows) * 128 + (li & 3) * 32;
            cp_async_16(dst, src);
            cp_async_16(dst + 16, src + 8);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 4) {
            const int c = c0 + cq, r = C::term0(c);              // rows r and r + kTermRows: its terms
            const uint4 *raw = reinterpret_cast<const uint4 *>(
                qs + (r + (li & 4) / 4 * C::kTermRows) * 128 + (li & 3) * 32);
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
                if (C::kTermCols) x[k] = __fmul2_rn(x[k], make_float2(16.f, 16.f));
                const uint32_t l = C::kTermCols ? to_e4m3x2(x[k].x, x[k].y)
                                                : to_e5m2x2(x[k].x, x[k].y);
                hi[k >> 1] = k & 1 ? hi[k >> 1] | (h << 16) : h;
                lo[k >> 1] = k & 1 ? lo[k >> 1] | (l << 16) : l;
            }
            __syncwarp();                                        // the four rows are read
            if (c < cols) {
                *reinterpret_cast<uint4 *>(qs + operand_offset(r, 16 * li)) =
                    make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(qs + operand_offset(r + C::kTermRows, 16 * li)) =
                    make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if (li == 0) qf[c] = pow2i(-a);
            }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kQFull + qb]);

        // One box per lane and refill, as in the producers; the 32 keys of a step
        // lie in one box or in whole boxes, within one refill.  (4 bits: a tile takes half as
        // long, so the words of four keys side by side go in one copy, and those of a page of
        // 128 and more from one address: a warp has an instruction in ten cycles here, and a
        // copy a key took 1100 to 1600 of a tile's 1900 to 4400.  64 sequences 58.9 us and
        // 57.2 so; draft rows, heads of a token side by side, 78.1 and 73.8.)
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
            if constexpr (kFp4) {                                // keys' words, then values'
                float *dst = reinterpret_cast<float *>(smem + C::sc) + s * 2 * kBK;
                // A tile's boxes lie within one refill, four keys side by side in one box.
                const int box0 = t << nb_shift;
                if ((box0 >> 5) != cached) {
                    cached = box0 >> 5;
                    lookup_boxes(p, it, cached, lane, false, my_page, my_slot);
                }
                if (p.scale_runs) {
                    const int k = 4 * lane, box = box0 + (k >> box_shift);
                    const int page = __shfl_sync(0xffffffffu, my_page, box);
                    const int slot =
                        __shfl_sync(0xffffffffu, my_slot, box) + (k & (p.box_rows - 1));
                    const float *ks = ksp + page * p.ks_page + slot;
                    const float *vs = vsp + page * p.vs_page + slot;
                    if (page >= 0 && k < left && slot + 4 <= p.page_size) {
                        cp_async_16(dst + k, ks);
                        cp_async_16(dst + kBK + k, vs);
                    } else if (page >= 0) {                      // (a cache's end)
                        for (int i = 0; i < 4 && k + i < left && slot + i < p.page_size; ++i) {
                            cp_async_4(dst + k + i, ks + i);
                            cp_async_4(dst + kBK + k + i, vs + i);
                        }
                    }
                } else if (box_shift == 7) {
                    const int page = __shfl_sync(0xffffffffu, my_page, box0);
                    const int slot = __shfl_sync(0xffffffffu, my_slot, box0) + lane;
                    const int live = page < 0 ? 0 : min(left, p.page_size - (slot - lane));
                    const float *ks = ksp + page * p.ks_page + slot * p.ks_block;
                    const float *vs = vsp + page * p.vs_page + slot * p.vs_block;
#pragma unroll
                    for (int u = 0; u < kBK / 32; ++u)
                        if (lane + 32 * u < live) {
                            cp_async_4(dst + lane + 32 * u, ks + 32 * u * p.ks_block);
                            cp_async_4(dst + kBK + lane + 32 * u, vs + 32 * u * p.vs_block);
                        }
                } else {
#pragma unroll
                    for (int u = 0; u < kBK / 32; ++u) {
                        const int k = 32 * u + lane, box = box0 + (k >> box_shift);
                        const int page = __shfl_sync(0xffffffffu, my_page, box);
                        const int slot =
                            __shfl_sync(0xffffffffu, my_slot, box) + (k & (p.box_rows - 1));
                        if (page >= 0 && k < left) {
                            cp_async_4(dst + k, ksp + page * p.ks_page + slot * p.ks_block);
                            cp_async_4(dst + kBK + k, vsp + page * p.vs_page + slot * p.vs_block);
                        }
                    }
                }
                cp_async_arrive(&bar[kScFull + s]);
                continue;
            }
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

template <int NC, bool kFp4, int kVs>
__global__ void __launch_bounds__(Cfg<NC, kFp4, kVs>::kThreads, kCtasPerSm)
gqa_decode_codes_kernel(const __grid_constant__ Fp8DecodeParams p) {
    using C = Cfg<NC, kFp4, kVs>;
    constexpr int NCH = C::NCH;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::tmem_slot);
    Fp8Range *range = reinterpret_cast<Fp8Range *>(smem + C::range);
    int2 *cum = reinterpret_cast<int2 *>(smem + C::items);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (uniform)
    const int lane = threadIdx.x & 31;
    const int G = p.group;

    if (warp < 3) fp8_build_items(p, cum, warp, lane, range);
    if (lane == 0 && (warp == C::kWarpK || warp == C::kWarpV))
        prefetch_tensormap(warp == C::kWarpK ? &p.k_map : &p.v_map);
    if (threadIdx.x == 96) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t n = 1;
            if (i == kSFree || i == kSFree + 1 || i == kPFull || i == kPFull + 1)
                n = 4 * C::kColGroups;
            if (i >= kScEmpty && i < kScEmpty + kScStages) n = 4 * C::kColGroups;
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
        for (int i = threadIdx.x - 96; i < (kQBufs * C::kQBytes + C::kBufs * C::NP * 128) / 16;
             i += C::kThreads - 96)
            reinterpret_cast<uint4 *>(smem + C::q)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const Fp8Range walk = *range;
    const int items = walk.count();

    if (warp == C::kWarpK) {
        if constexpr (kFp4) {
            produce_both<NC, kVs>(p, cum, walk, smem, bar, lane);
        } else {
            produce<true, NC, kVs>(p, cum, walk, smem, bar, lane);
        }
    } else if (!C::kTwoMmaWarps && warp == C::kWarpV) {
        produce<false, NC, kVs>(p, cum, walk, smem, bar, lane);
    } else if (warp == C::kWarpAux) {
        feed<NC, kFp4, kVs>(p, cum, walk, smem, bar, lane);
    } else if (warp == C::kWarpMma || (C::kTwoMmaWarps && warp == C::kWarpV)) {
        // ---------------------------------------------------------- MMA issue
        // A warp for both contractions, or (4 bits, whose tiles come twice as fast) one for
        // each.  The whole warp walks, with numbers that are the same in all lanes, and one
        // lane issues: what the tensor core is given then is in uniform registers (one lane
        // that walks by itself took 130 cycles an MMA to move it there).
        const bool scores = !C::kTwoMmaWarps || warp == C::kWarpMma;
        const bool outputs = !C::kTwoMmaWarps || warp == C::kWarpV;
        constexpr uint32_t held = kFp4 ? kE2m1 : kE4m3;
        constexpr uint32_t idesc_s = idesc_f8f6f4(held, kE4m3, 128, C::NS, 0, 0);
        constexpr uint32_t idesc_s1 = idesc_f8f6f4(held, kE5m2, 128, C::NS, 0, 0);
        constexpr uint32_t idesc_o = idesc_f8f6f4(held, kFp4 ? kE5m2 : kE4m3, 128, C::NP, 1, 1);
        const uint32_t k_base = smem_addr(smem + C::kring);
        const uint32_t v_base = smem_addr(smem + C::vring);
        const uint32_t q_base = smem_addr(smem + C::q);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        // MN-major without a swizzle: 16 bytes per key, 8-key groups 128 bytes
        // apart, 16-column blocks kBK * 16
        const uint64_t pd = smem_desc_plain(smem_addr(smem + C::p), 128, kBK * 16);
        const int count = __shfl_sync(0xffffffffu, items, 0);
        const auto arrived = [&](int b, int phase) {
            return __all_sync(0xffffffffu, mbar_wait(&bar[b], phase, p.err)) != 0;
        };
        int g = 0, itq = 0;
        bool ok = true;
        // S of tile gg of the walk, whose item's queries are in buffer qb; last: of the item
        const auto issue_scores = [&](int gg, int qb, bool last) {
            const int ks = gg % kStages;
            const int sb = gg & 1;
            ok = arrived(kKFull + ks, (gg / kStages) & 1);
            if (ok && gg >= 2) ok = arrived(kSFree + sb, ((gg >> 1) - 1) & 1);
            if (!ok) return;
            tc::fence_after_sync();
            const uint64_t kd = tc::smem_desc_sw128(k_base + ks * kTileBytes, 16, 1024);
            const uint64_t qd = tc::smem_desc_sw128(q_base + qb * C::kQBytes, 16, 1024);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kD / 32; ++kk) {           // 32 channels = 32 bytes a step
                    const uint64_t ka = kd + uint64_t(kk * 2), qa = qd + uint64_t(kk * 2);
                    if constexpr (kFp4) {                        // a group's block
                        const uint32_t to = tm + sb * C::kSCols + kk * C::NS;
                        mma_f8f6f4(to, ka, qa, idesc_s, false);
                        if (!C::kTermCols)
                            mma_f8f6f4(to, ka, qa + uint64_t((C::NS * 128) >> 4), idesc_s1, true);
                    } else {
                        mma_f8f6f4(tm + sb * C::kSCols, ka, qa, idesc_s, kk > 0);
                    }
                }
                tc::mma_commit(&bar[kSFull + sb]);
                tc::mma_commit(&bar[kKEmpty + ks]);
                if (last) tc::mma_commit(&bar[kQEmpty + qb]);
            }
            __syncwarp();
        };
        // O += V P of tile gp, the t-th of its item
        const auto issue_outputs = [&](int gp, int t) {
            const int vs = gp % kVs;
            const int ob = C::kTurns ? gp & 1 : 0;               // buffer of P and O
            const int turn = C::kTurns ? gp >> 1 : gp;
            ok = arrived(kPFull + ob, turn & 1);
            if (ok) ok = arrived(kVFull + vs, (gp / kVs) & 1);
            if (!ok) return;
            tc::fence_after_sync();
            // V^T as the MN-major A operand: 128 channels are one 128-byte
            // atom, 8-key groups 1 KB apart, 32 keys a step.
            const uint64_t vd = tc::smem_desc_sw128(v_base + vs * kTileBytes, kTileBytes, 1024);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kBK / 32; ++kk)
                    mma_f8f6f4(tm + C::kTmemO + ob * C::NP, vd + uint64_t((kk * 32 * 128) >> 4),
                               pd + uint64_t((ob * C::NP * 128 + kk * 32 * 16) >> 4), idesc_o,
                               t >= C::kBufs || kk > 0);
                tc::mma_commit(&bar[kODone + ob]);
                tc::mma_commit(&bar[kVEmpty + vs]);
            }
            __syncwarp();
        };
        for (int j = 0; ok && j < count; ++j) {
            const int ntiles = __shfl_sync(0xffffffffu, fp8_item(p, cum, walk, j).ntiles, 0);
            if (ntiles == 0) continue;
            const int qb = itq % kQBufs;
            if (scores) ok = arrived(kQFull + qb, (itq / kQBufs) & 1);
            if (C::kTwoMmaWarps) {
                for (int t = 0; ok && t < ntiles; ++t) {
                    if (scores) issue_scores(g + t, qb, t == ntiles - 1);
                    else issue_outputs(g + t, t);
                }
            } else {
                for (int t = 0; ok && t <= ntiles; ++t) {
                    if (t < ntiles) issue_scores(g + t, qb, t == ntiles - 1);
                    if (ok && t >= 1) issue_outputs(g + t - 1, t - 1);
                }
            }
            g += ntiles;
            ++itq;
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
        const int buf = C::kTurns ? grp : 0;         // of P and O
        bool ok = true;
        for (int j = 0; j < items; ++j, ++iter) {
            const Fp8Item it = fp8_item(p, cum, walk, j);
            int row0, nrows;
            seq_rows(p, it.b, row0, nrows);
            nrows = min(nrows, p.num_q_rows - row0);
            // Column cg = (row cg / G, head cg % G); chunk h of this group holds the
            // columns col(h) .. col(h) + 3.  Columns past the item's rows hold an
            // earlier item's scores and are never written out.
            const auto col = [&](int h) { return 4 * (h * C::kColGroups + (C::kTurns ? 0 : grp)); };
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
            const int t_first = C::kTurns ? (grp ^ g) & 1 : 0;
            for (int t = t_first; t < it.ntiles; t += C::kBufs) {
                const int gg = g + t;
                const int sb = gg & 1;
                const bool first = t == t_first;
                const int ss = gg % kScStages, sph = gg / kScStages & 1;   // of the scale ring
                const int turn = C::kTurns ? gg >> 1 : gg;                 // of the buffer
                const int t0 = it.start + t * kBK;
                const bool tail = t0 + kBK > full;               // uniform over the CTA
                // ---- scales and scores of this key -------------------------------
                // both polls in flight together
                const bool sc_in = mbar_try_wait(&bar[kScFull + ss], sph);
                const bool s_in = mbar_try_wait(&bar[kSFull + sb], (gg >> 1) & 1);
                if (!sc_in) ok = ok && mbar_wait(&bar[kScFull + ss], sph, p.err);
                float2 sc;
                if constexpr (kFp4) {
                    const float *at = reinterpret_cast<const float *>(smem + C::sc) + ss * 2 * kBK;
                    sc = make_float2(at[k], at[kBK + k]);
                } else {
                    sc = reinterpret_cast<const float2 *>(smem + C::sc)[ss * kBK + k];
                }
                if (!s_in) ok = ok && mbar_wait(&bar[kSFull + sb], (gg >> 1) & 1, p.err);
                tc::fence_after_sync();
                float2 s[NCH][2];                                // score, then score - m
                const uint32_t s_at = tmem + lane_base + sb * C::kSCols;
                // (4 bits: the key's scales, a group of channels each)
                float by_group[kKGroups];
                if constexpr (kFp4) e8m0x4(__float_as_uint(sc.x), by_group);
                if constexpr (kFp4 && C::kTermCols) {
                    float raw[kKGroups][8];
                    tmem_ld_group_terms(s_at + 2 * col(0), raw);
                    float2 lo[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) s[0][c] = lo[c] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int kk = 0; kk < kKGroups; ++kk) {
                        const float f4 = by_group[kk];
                        const float2 f2 = make_float2(f4, f4);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            s[0][c] = __ffma2_rn(make_float2(raw[kk][2 * c], raw[kk][2 * c + 1]), f2,
                                                 s[0][c]);
                            lo[c] = __ffma2_rn(make_float2(raw[kk][4 + 2 * c], raw[kk][5 + 2 * c]),
                                               f2, lo[c]);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        s[0][c] = __ffma2_rn(lo[c], make_float2(0.0625f, 0.0625f), s[0][c]);
                } else if constexpr (kFp4) {
                    float raw[NCH][kKGroups][4];
                    tmem_ld_groups(s_at + col(0), s_at + col(NCH - 1), raw);
#pragma unroll
                    for (int h = 0; h < NCH; ++h)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            s[h][c] = make_float2(0.f, 0.f);
#pragma unroll
                            for (int kk = 0; kk < kKGroups; ++kk) {
                                const float f4 = by_group[kk];
                                s[h][c] = __ffma2_rn(
                                    make_float2(raw[h][kk][2 * c], raw[h][kk][2 * c + 1]),
                                    make_float2(f4, f4), s[h][c]);
                            }
                        }
                } else {
                    float raw[NCH][8];
                    tmem_ld_scores(s_at + 2 * col(0), s_at + 2 * col(NCH - 1), raw);
#pragma unroll
                    for (int h = 0; h < NCH; ++h)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            s[h][c] = __ffma2_rn(make_float2(raw[h][4 + 2 * c], raw[h][5 + 2 * c]),
                                                 make_float2(0.0625f, 0.0625f),
                                                 make_float2(raw[h][2 * c], raw[h][2 * c + 1]));
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar[kSFree + sb]);
                    mbar_arrive(&bar[kScEmpty + ss]);
                }
                if (tail && t0 + k >= it.L) sc = make_float2(0.f, 0.f);
                const int ve_raw = int((__float_as_uint(sc.y) >> 23) & 0xffu) - 127;
                const int ve = min(max(ve_raw, kMinVExp), kMaxVExp);
                const float vexp = static_cast<float>(ve);
                const float v_inv = pow2i(-ve);
                // (a scale past the range would saturate: NaN instead)
                const float v_mul = ve_raw > kMaxVExp ? __uint_as_float(0x7fffffffu)
                                                      : sc.y * v_inv * weight_top(kFp4);
                float top = -INFINITY;
#pragma unroll
                for (int h = 0; h < NCH; ++h) {
                    if (col(h) >= cols) continue;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (!kFp4) s[h][c] = __fmul2_rn(s[h][c], make_float2(sc.x, sc.x));
                        s[h][c] = __ffma2_rn(s[h][c], f[h][c], make_float2(vexp, vexp));
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
                const bool moved = first || named_or(1 + grp, 128, top > kLazy);
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
                                *reinterpret_cast<float2 *>(red + kw * 16 + 4 * buf + col(h) + 2 * c) =
                                    make_float2(w0, w1);
                        }
                    }
                    named_sync(1 + grp, 128);
                    const float lazy = first ? -INFINITY : kLazy;
                    const auto raise = [&](int cg, float &sx, float &mx, float &lx, float &ax) {
                        const float *r = red + 4 * buf + cg;
                        const float up = fmaxf(fmaxf(r[0], r[16]), fmaxf(r[32], r[48]));
                        const bool move = up > lazy;
                        ax = move && !first ? fast_exp2(-up) : 1.f;
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
                    if constexpr (kFp4) {
                        e5m2_terms(w[0], w[1], code[h]);
                    } else {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint32_t lo = to_e4m3x2(w[0].x, w[0].y);
                            const uint32_t hi = to_e4m3x2(w[1].x, w[1].y);
                            code[h][u] = lo | (hi << 16);
                            if (u < 3) {
                                take_rest(lo, w[0].x, w[0].y);
                                take_rest(hi, w[1].x, w[1].y);
                                const float2 ratio = make_float2(term_ratio(kFp4, u), term_ratio(kFp4, u));
                                w[0] = __fmul2_rn(w[0], ratio);
                                w[1] = __fmul2_rn(w[1], ratio);
                            }
                        }
                    }
                }
                if (!first) {
                    // The last P.V of this buffer is complete: P^T may be overwritten and
                    // O^T rescaled (thread = channel lane).
                    ok = ok && mbar_wait(&bar[kODone + buf], (turn - 1) & 1, p.err);
                    tc::fence_after_sync();
                    if (moved) {   // identical in every thread of the group
#pragma unroll
                        for (int h = 0; h < NCH; ++h) {
                            if (col(h) >= cols) continue;
                            float o[16];
                            const uint32_t oc =
                                tmem + lane_base + C::kTmemO + buf * C::NP + 4 * col(h);
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
                if constexpr (kFp4) {
                    // No code is NaN, so a weight of 0 hides whatever a row holds; but a scale
                    // that counts as NaN must not reach the rows before its token.
                    if (tail && v_mul != v_mul) {
#pragma unroll
                        for (int h = 0; h < NCH; ++h)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (col(h) < cols && !sees(col(h) + c, t0 + k)) {
#pragma unroll
                                    for (int u = 0; u < 4; ++u) code[h][u] &= ~(0xffu << (8 * c));
                                }
                    }
                } else if (tail) {
                    const int vs = gg % kVs;
                    ok = ok && mbar_wait(&bar[kVFull + vs], (gg / kVs) & 1, p.err);
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
                        *reinterpret_cast<uint4 *>(smem + C::p + buf * C::NP * 128 +
                                                   4 * col(h) * kBK + 16 * k) =
                            make_uint4(code[h][0], code[h][1], code[h][2], code[h][3]);
                tc::fence_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kPFull + buf]);
            }

            // ---- item epilogue ----------------------------------------------------
            // Rolled over pairs of columns and short on purpose: it runs once an item,
            // from a cold instruction cache (all 8 columns of a warp unrolled: 10000
            // cycles; a pair at a time: 3000 to 5000).  The row sums and references go
            // through shared memory while the last P.V is still in flight.
            // [4 key warps][16 columns], then m[16]; turns: each group's
            const float *both = lred + (iter & 1) * 80 * C::kBufs;
            float *lb = lred + ((iter & 1) * C::kBufs + buf) * 80;
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
            if (C::kTurns) named_sync(3, 256); else named_sync(1 + grp, 128);
            // the last P.V of each buffer that had a tile of the item
            const int tiles_of[2] = {
                C::kTurns ? (it.ntiles + 1 - (g & 1)) >> 1 : it.ntiles, (it.ntiles + (g & 1)) >> 1};
#pragma unroll
            for (int q = 0; q < C::kBufs; ++q) {
                const int last = C::kTurns ? ((g + it.ntiles - 1 - q) >> 1) : g + it.ntiles - 1;
                if (tiles_of[q] > 0) ok = ok && mbar_wait(&bar[kODone + q], last & 1, p.err);
            }
            tc::fence_after_sync();
            const int ch = k;   // output channel of this thread
            const size_t head0 = size_t(row0) * p.num_q_heads + it.kvh * G;
            const size_t slot0 = size_t(it.slot) * kGqaSlotCols;
            // (turns: a group has two of the columns)
#pragma unroll 1
            for (int x = C::kTurns ? 2 * grp : 0; x < (C::kTurns ? 2 * grp + 2 : 4 * NCH); x += 2) {
                const int c0 = col(x >> 2) + (x & 3);
                if (c0 >= cols) break;
                float o[C::kBufs][2];
#pragma unroll
                for (int q = 0; q < C::kBufs; ++q) {
                    float term[4][2];
                    tmem_ld_terms(
                        tmem + lane_base + C::kTmemO + q * C::NP + 4 * (c0 & ~3) + (c0 & 3), term);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float acc = term[3][u];
#pragma unroll
                        for (int v = 2; v >= 0; --v)
                            acc = fmaf(acc, 1.f / term_ratio(kFp4, v), term[v][u]);
                        o[q][u] = ok && tiles_of[q] > 0 ? acc * (1.f / weight_top(kFp4)) : 0.f;
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int cg = c0 + u, i = (cg * g_inv) >> 16;
                    if (i >= nrows) continue;
                    float acc = o[0][u];
                    float lsum = (both[cg] + both[16 + cg]) + (both[32 + cg] + both[48 + cg]);
                    // no visible key: no sum, no reference
                    float mx = lsum == 0.f ? -INFINITY : both[64 + cg];
                    if constexpr (C::kTurns) {
                        const float *b2 = both + 80;
                        const float l2 = (b2[cg] + b2[16 + cg]) + (b2[32 + cg] + b2[48 + cg]);
                        const float m2 = l2 == 0.f ? -INFINITY : b2[64 + cg];
                        const float top = fmaxf(mx, m2);
                        const float a1 = l2 == 0.f ? 0.f : fast_exp2(m2 - top);
                        const float a0 = lsum == 0.f ? 0.f : fast_exp2(mx - top);
                        acc = fmaf(acc, a0, o[1][u] * a1);
                        lsum = fmaf(lsum, a0, l2 * a1);
                        mx = top;
                    }
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
            if (C::kTurns) named_sync(3, 256);   // both groups have read both outputs
            if (!kFp4 && threadIdx.x == 0) publish(p, cum, walk, it);   // (4 bits: its producer)
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

template <int NC, bool kFp4, int kVs>
cudaError_t launch_nc(const Fp8DecodeParams &p, int ctas, cudaStream_t stream) {
    const size_t smem = smem_bytes<NC, kFp4, kVs>(p.batch);
    auto kern = gqa_decode_codes_kernel<NC, kFp4, kVs>;
    const cudaError_t e = allow_smem(kern, smem_bytes<NC, kFp4, kVs>(kGqaMaxBatch));
    if (e != cudaSuccess) return e;
    kern<<<dim3(static_cast<unsigned>(ctas)), Cfg<NC, kFp4, kVs>::kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <bool kFp4>
cudaError_t launch(const Fp8DecodeParams &p, int ctas, cudaStream_t stream) {
    const int cols = p.max_q_len * p.group;
    if (cols < 1 || cols > 16) return cudaErrorInvalidValue;
    if (cols <= 4) {
        constexpr int kVs = v_stages(kFp4, 4);
        if (kVs > 2 && smem_bytes<4, kFp4, kVs>(p.batch) > kCtaSmem)
            return launch_nc<4, kFp4, 2>(p, ctas, stream);
        return launch_nc<4, kFp4, kVs>(p, ctas, stream);
    }
    if (cols <= 8) return launch_nc<8, kFp4, 2>(p, ctas, stream);
    return launch_nc<16, kFp4, 2>(p, ctas, stream);
}

}  // namespace codes
}  // namespace attn
