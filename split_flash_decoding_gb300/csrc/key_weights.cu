// key_weights.cu -- the attention weight that every key of a bf16 cache gathers
// from a call's query rows (attn_key_weights):
//
//   w_t <- [t < L - n] decay w_t + sum_(rows that see t, heads of the group) e^(scale q.k_t - lse)
//
// The rows' log-sum-exps are known (the attention call before returned them), so a
// weight is final as soon as its score is: nothing runs along the keys, no key needs
// another, and a sum over the rows of one key is all there is.  Scores are tcgen05
// MMAs with the keys on the 128 rows of M and (query row, head) columns on N,
//
//   S^T [128 keys x N] = K [128 x d] . Q^T [d x N],
//
// so a thread that reads one TMEM lane sums one key's weights over the columns in
// registers: no shuffles, no atomics, one store a key.
//
// An item is KT tiles of 128 keys of one (sequence, KV head); its steps are the
// column tiles of the rows that see one of its keys.
//   Few columns (decode, draft rows): KT = 1, steps of 16 columns.  Bound by the stream of
//   keys up to 32 columns.  Two CTAs per SM walk the units of all sequences, a unit being a
//   tile of up to four KV heads, an item each: a thread then has its key's weights of four
//   heads, neighbours in memory, and reads and writes them at once (a head at a time, four
//   bytes of every 32 were 15 of 125 us).  64 sequences of 512 to 8192 keys 95 to 98 us, 6.2 TB/s.
//   More (prompts): KT = 2, steps of 256 columns (MMAs of 128 columns wait for shared
//   memory: 128 bytes a cycle for A and B).  Both key tiles stay in shared memory while
//   column tiles pass; the score tiles of the two alternate in the two halves of tensor
//   memory, one being filled while the other is read.  A CTA takes one item; those that the
//   most rows see come first.  4 prompts of 2070 to 4062 rows, 32 + 8 heads: 149 us, 1.1 PFLOP/s
//   (101 us with the epilogue left out; 197 with column tiles of 128 and eight epilogue warps,
//   174 with sixteen).  The exponential unit gives 32 a cycle and SM, as long as the MMAs take;
//   a part of them as polynomials on the FMA units lost, as the instructions are as scarce.
//
// Warp roles: epilogue (four warps, or sixteen in four parts of the columns), K producer
// and Q producer (TMA), MMA issue, and one warp that fetches the rows' lse.
#include "evict_ops.h"
#include "launch.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace attn {
namespace {

constexpr int kKeys = 128;                   // keys of a tile: the rows of M

template <int D, bool kMany>
struct Cfg {
    static constexpr int KT = kMany ? 2 : 1;                 // key tiles of an item
    static constexpr int NQ = kMany ? kManyColumns : kFewColumns;
    static constexpr int kKStages = kMany ? 1 : 3;           // items in flight
    static constexpr int kQStages = 2;
    static constexpr int kLseStages = 4;
    static constexpr int kHeads = kMany ? 1 : 4;             // KV heads of a unit, at most
    static constexpr int kParts = kMany ? 4 : 1;             // of a tile's columns, four warps each
    static constexpr int kCols = NQ / kParts;
    static constexpr int kEpiWarps = 4 * kParts;
    static constexpr int kWarpK = kEpiWarps, kWarpQ = kWarpK + 1, kWarpMma = kWarpK + 2,
                         kWarpAux = kWarpK + 3;
    static constexpr int kThreads = 32 * (kEpiWarps + 4);
    static constexpr int kTileBytes = kKeys * D * 2;
    static constexpr int kQBytes = NQ * D * 2;
    static constexpr int kTmemCols = 2 * NQ;                 // two score tiles: 32 or 512
    // shared memory
    static constexpr int k = 0;
    static constexpr int q = k + kKStages * KT * kTileBytes;
    static constexpr int lse = q + kQStages * kQBytes;
    static constexpr int part = lse + kLseStages * NQ * 4;   // many: the parts' sums
    static constexpr int bars = part + (kMany ? kParts * KT * kKeys * 4 : 0);
    static constexpr int tmem_slot = bars + 256;
    static constexpr int items = tmem_slot + 16;
    // barriers
    static constexpr int bKFull = 0, bKEmpty = bKFull + kKStages, bQFull = bKEmpty + kKStages,
                         bQEmpty = bQFull + kQStages, bLFull = bQEmpty + kQStages,
                         bLEmpty = bLFull + kLseStages, bSFull = bLEmpty + kLseStages,
                         bSFree = bSFull + 2, kNumBars = bSFree + 2;
    static_assert(kNumBars * 8 <= 256, "barrier space");
};

struct Unit {
    int b, kvh, heads;              // KV heads [kvh, kvh + heads), an item each
    int L, n, row0, rows;           // n: the sequence's rows; rows: those the call has
    int key0;                       // first key
    int step0, steps;               // column tiles [step0, step0 + steps)
};

// Key tiles of a sequence: KT * 128 keys each.
template <int KT>
__device__ __forceinline__ int tiles_of(const WeightsParams &p, int b) {
    const uint32_t L = min(p.kv_len[b], uint32_t(p.max_kv_len));
    return static_cast<int>((L + KT * kKeys - 1) / (KT * kKeys));
}

template <bool kMany>
__device__ __forceinline__ void open_unit(const WeightsParams &p, int b, int kvh, int tile, Unit &it) {
    constexpr int KT = kMany ? 2 : 1;
    it.b = b;
    it.kvh = kvh;
    it.heads = kMany ? 1 : min(Cfg<64, kMany>::kHeads, p.hkv - kvh);
    it.L = static_cast<int>(min(p.kv_len[b], uint32_t(p.max_kv_len)));
    it.row0 = b;
    it.n = 1;
    if (p.q_row_offsets) {
        it.row0 = static_cast<int>(p.q_row_offsets[b]);
        it.n = max(static_cast<int>(p.q_row_offsets[b + 1]) - it.row0, 0);
    }
    it.rows = max(min(it.n, p.num_q_rows - it.row0), 0);
    it.key0 = tile * (KT * kKeys);
    const int first = p.causal ? max(it.key0 - (it.L - it.n), 0) : 0;   // first row that sees a key
    it.step0 = first / p.tile_rows;
    it.steps = max((it.rows + p.tile_rows - 1) / p.tile_rows - it.step0, 0);
}

// The columns of step t that see key tile kt of an item: [lo, hi), and from which on a key
// of it is seen.
struct Columns {
    int lo, hi, first, group;
    bool causal;
    __device__ __forceinline__ bool any() const { return lo < hi; }
    __device__ __forceinline__ int seen_by(int k) const {
        return causal ? max(first + k, 0) * group : 0;
    }
};
__device__ __forceinline__ Columns columns_of(const WeightsParams &p, const Unit &it, int kt, int t) {
    Columns c;
    const int i0 = (it.step0 + t) * p.tile_rows;         // first row of the step
    c.group = p.group;
    c.causal = p.causal;
    c.first = it.key0 + kt * kKeys - (it.L - it.n) - i0; // row of the step that is key 0 itself
    c.lo = c.seen_by(0);
    c.hi = min(p.tile_rows, it.rows - i0) * p.group;
    return c;
}

// Unit j of the call's list; false: there is none of that number (a later one may be).
//   few:  (sequence, tile, four KV heads), the last fastest; cum: tiles before each sequence
//   many: (tile from the sequence's end, falling; sequence, KV head): where the rows are
//         the last tokens, that many of them see the tile, so the dearest come first
template <bool kMany>
__device__ __forceinline__ bool find_unit(const WeightsParams &p, const int *cum, int j, Unit &it) {
    if (kMany) {
        const int units = p.batch * p.hkv, last = (p.max_kv_len - 1) / (2 * kKeys);
        const int e = last - j / units, u = j % units;
        const int b = u / p.hkv, tiles = tiles_of<2>(p, b);
        if (e >= tiles) return false;
        open_unit<kMany>(p, b, u - b * p.hkv, tiles - 1 - e, it);
        return true;
    }
    const int x = j / p.head_groups;
    int lo = 0, hi = p.batch;       // cum[lo] <= x < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= x) lo = mid; else hi = mid;
    }
    open_unit<kMany>(p, lo, (j - x * p.head_groups) * Cfg<64, kMany>::kHeads, x - cum[lo], it);
    return true;
}

// Page of token t of sequence b (-1: outside the pool) and its slot.  report: the threads that
// own the keys, as they walk the units without rows too (the key producer skips those).
__device__ __forceinline__ int page_at(const WeightsParams &p, int b, int t, bool report, int &slot) {
    if (!p.page_table) {
        slot = t;
        return b;
    }
    const int shift = 31 - __clz(p.page_size);   // (pages of a table: powers of two)
    const int pidx = t >> shift;
    slot = t & (p.page_size - 1);
    const int e = pidx < p.max_pages ? p.page_table[size_t(b) * p.max_pages + pidx] : -1;
    if (e < 0 || e >= p.num_pages) {
        if (report) atomicOr(p.err, kErrBadPage);
        return -1;
    }
    return e;
}

// One lane of the warp (all lanes take part).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void cp_async_4(void *dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}
// Arrive (without raising the pending count) when this thread's copies so far are done.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// N scores of the thread's key: adds their weights to sum.  kPart: only columns [lo, hi)
// count.
//   kFast: e^(scale s - lse) = 2^(a s - b), a = scale log2 e and b = lse log2 e (in `lse`)
//     rounded: the exponent errs by up to 2^-24 (|a s| + |b|) more than below, and a pair of
//     columns takes five instructions instead of six.  (For many columns: 149.7 us, 152.3 with
//     the form below, whose weights were no nearer to 64 bits, 1.2e-7 off and 1.1e-7 so: a
//     score of that size errs as much in its own sum, and so does a sum of thousands of terms.)
//   else: scale s - lse first, then the product with log2 e, which errs by a part of that
//     small number only.
template <int N, bool kPart, bool kFast>
__device__ __forceinline__ void add_weights(const float (&v)[N], const float *lse, float scale,
                                            int lo, int hi, float2 (&sum)[2]) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(lse + c);
        // (precise: lse - score, and a negative factor: packed numbers have no minus sign)
        const float2 f = kFast ? make_float2(scale, scale) : make_float2(-scale, -scale);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float2 x = __ffma2_rn(make_float2(v[c + 2 * u], v[c + 2 * u + 1]), f,
                                  u ? make_float2(l.z, l.w) : make_float2(l.x, l.y));
            if (!kFast) x = __fmul2_rn(x, make_float2(-kLog2e, -kLog2e));
            float2 w = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            if (kPart) {
                const int at = c + 2 * u;
                if (at < lo || at >= hi) w.x = 0.f;
                if (at + 1 < lo || at + 1 >= hi) w.y = 0.f;
            }
            sum[u] = __fadd2_rn(sum[u], w);
        }
    }
}

template <int D, bool kMany>
__global__ void __launch_bounds__(Cfg<D, kMany>::kThreads, kMany ? 1 : 2)
key_weights_kernel(const __grid_constant__ WeightsParams p) {
    using C = Cfg<D, kMany>;
    constexpr int KT = C::KT, NQ = C::NQ;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::bars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::tmem_slot);
    int *cum = reinterpret_cast<int *>(smem + C::items);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int stride = static_cast<int>(gridDim.x);

    if (blockIdx.x == 0 && warp == 0)
        for (int b = lane; b < p.batch; b += 32)
            if (p.kv_len[b] > uint32_t(p.max_kv_len)) atomicOr(p.err, kErrBadLength);
    int total;
    if (kMany) {
        // (one item a CTA: most of those past a sequence's end leave here)
        total = ((p.max_kv_len - 1) / (KT * kKeys) + 1) * p.batch * p.hkv;
        if (stride >= total) {
            Unit it;
            if (!find_unit<kMany>(p, cum, blockIdx.x, it)) return;
        }
    } else if (warp == 0) {
        int before = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            const int n = b0 + lane < p.batch ? tiles_of<KT>(p, b0 + lane) : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (b0 + lane < p.batch) cum[b0 + lane] = before + incl - n;
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) cum[p.batch] = before;
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < C::kNumBars; ++i) {
            uint32_t n = 1;
            if (i >= C::bLFull && i < C::bLFull + C::kLseStages) n = 32;
            if (i >= C::bLEmpty && i < C::bLEmpty + C::kLseStages) n = C::kEpiWarps;
            if (i >= C::bSFree) n = C::kEpiWarps;
            mbar_init(&bar[i], n);
        }
        fence_mbar_init();
    }
    if (warp == C::kWarpMma) {
        tc::tmem_alloc(tmem_slot, C::kTmemCols);
        tc::tmem_relinquish();
    }
    if (lane == 0 && (warp == C::kWarpK || warp == C::kWarpQ))
        prefetch_tensormap(warp == C::kWarpK ? &p.k_map : &p.q_map);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    if (!kMany) total = cum[p.batch] * p.head_groups;

    Unit it;
    if (warp == C::kWarpK) {
        // ------------------------------------------------------------ K producer
        const int box_rows = p.box_rows, box_shift = 31 - __clz(box_rows);
        const int nb = (KT * kKeys) >> box_shift;                // boxes of an item
        const uint32_t box_bytes = uint32_t(box_rows) * D * 2;
        int g = 0;
        bool ok = true;
        for (int j = blockIdx.x; ok && j < total; j += stride) {
            if (!find_unit<kMany>(p, cum, j, it) || it.steps == 0) continue;
            const int live = min(nb, (it.L - it.key0 + box_rows - 1) >> box_shift);
            int page = -1, slot = 0;                             // of the lane's box
            if (lane < live) page = page_at(p, it.b, it.key0 + (lane << box_shift), false, slot);
            const int row = lane << box_shift;                   // in the item
            uint8_t *dst = smem + C::k + (row / kKeys) * C::kTileBytes + (row % kKeys) * 128;
            for (int h = 0; ok && h < it.heads; ++h) {
                const int s = g % C::kKStages;
                if (lane == 0) {
                    if (g >= C::kKStages)
                        ok = mbar_wait(&bar[C::bKEmpty + s], ((g / C::kKStages) - 1) & 1, p.err);
                    if (ok) mbar_arrive_expect_tx(&bar[C::bKFull + s], uint32_t(live) * box_bytes);
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                ++g;
                if (lane < live) {
                    if (page < 0) {
                        mbar_complete_tx(&bar[C::bKFull + s], box_bytes);   // skipped bad page
                    } else {
#pragma unroll
                        for (int cb = 0; cb < D / 64; ++cb)
                            tma_load_4d(dst + s * (KT * C::kTileBytes) + cb * (kKeys * 128), &p.k_map,
                                        &bar[C::bKFull + s], cb * 64, slot, it.kvh + h, page);
                    }
                }
                __syncwarp();
            }
        }
        // every copy this warp issued must land before the CTA may leave
        if (lane == 0)
            for (int i = max(0, g - C::kKStages); i < g; ++i)
                mbar_wait(&bar[C::bKFull + i % C::kKStages], (i / C::kKStages) & 1, p.err);
    } else if (warp == C::kWarpQ) {
        // ------------------------------------------------------------ Q producer
        const uint32_t bytes = uint32_t(p.tile_rows * p.group) * D * 2;
        int g = 0;
        bool ok = true;
        if (lane == 0) {
            for (int j = blockIdx.x; ok && j < total; j += stride) {
                if (!find_unit<kMany>(p, cum, j, it)) continue;
                for (int x = 0; ok && x < it.steps * it.heads; ++x) {
                    const int h = kMany ? 0 : x / it.steps, t = x - h * it.steps;
                    const int s = g % C::kQStages;
                    if (g >= C::kQStages)
                        ok = mbar_wait(&bar[C::bQEmpty + s], ((g / C::kQStages) - 1) & 1, p.err);
                    if (!ok) break;
                    ++g;
                    mbar_arrive_expect_tx(&bar[C::bQFull + s], bytes);
#pragma unroll
                    for (int cb = 0; cb < D / 64; ++cb)
                        tma_load_4d(smem + C::q + s * C::kQBytes + cb * (NQ * 128), &p.q_map,
                                    &bar[C::bQFull + s], cb * 64, 0, it.kvh + h,
                                    it.row0 + (it.step0 + t) * p.tile_rows);
                }
            }
            for (int i = max(0, g - C::kQStages); i < g; ++i)
                mbar_wait(&bar[C::bQFull + i % C::kQStages], (i / C::kQStages) & 1, p.err);
        }
    } else if (warp == C::kWarpMma) {
        // ------------------------------------------------------------ MMA issue
        // (The whole warp walks, with numbers that are the same in all lanes, and one lane
        // issues: what the tensor core is given then is in uniform registers.)
        constexpr uint32_t idesc = tc::idesc_bf16_f32(128, NQ, 0, 0);
        const uint32_t k_base = smem_addr(smem + C::k), q_base = smem_addr(smem + C::q);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const auto arrived = [&](int b, int phase) {
            return __all_sync(0xffffffffu, mbar_wait(&bar[b], phase, p.err)) != 0;
        };
        int g = 0, gk = 0;
        bool ok = true;
        for (int j = blockIdx.x; ok && j < total; j += stride) {
            if (!find_unit<kMany>(p, cum, j, it)) continue;
            const int steps = __shfl_sync(0xffffffffu, it.steps, 0);
            const int heads = __shfl_sync(0xffffffffu, it.heads, 0);
            if (steps == 0) continue;
            for (int h = 0; ok && h < heads; ++h, ++gk) {
                const int ks = gk % C::kKStages;
                ok = arrived(C::bKFull + ks, (gk / C::kKStages) & 1);
                for (int t = 0; ok && t < steps; ++t, ++g) {
                    const int qs = g % C::kQStages;
                    ok = arrived(C::bQFull + qs, (g / C::kQStages) & 1);
                    const uint64_t qd = tc::smem_desc_sw128(q_base + qs * C::kQBytes, 16, 1024);
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        const int x = g * KT + kt, sb = x & 1;   // score tile and its buffer
                        if (ok && x >= 2) ok = arrived(C::bSFree + sb, ((x >> 1) - 1) & 1);
                        if (!ok) break;
                        tc::fence_after_sync();
                        const uint64_t kd = tc::smem_desc_sw128(
                            k_base + (ks * KT + kt) * C::kTileBytes, 16, 1024);
                        const bool any =
                            __all_sync(0xffffffffu, columns_of(p, it, kt, t).any()) != 0;
                        if (elect_one()) {
                            if (any) {
#pragma unroll
                                for (int kk = 0; kk < D / 16; ++kk) {
                                    const uint32_t in = (kk & 3) * 32;   // in the 64 channels' rows
                                    tc::mma_bf16(
                                        tm + sb * NQ,
                                        kd + uint64_t(((kk >> 2) * (kKeys * 128) + in) >> 4),
                                        qd + uint64_t(((kk >> 2) * (NQ * 128) + in) >> 4), idesc,
                                        kk > 0);
                                }
                            }
                            tc::mma_commit(&bar[C::bSFull + sb]);
                            if (kt == KT - 1) tc::mma_commit(&bar[C::bQEmpty + qs]);
                            if (kt == KT - 1 && t == steps - 1) tc::mma_commit(&bar[C::bKEmpty + ks]);
                        }
                        __syncwarp();
                    }
                }
            }
        }
    } else if (warp == C::kWarpAux) {
        // ------------------------------------------------------------ lse and earlier weights
        constexpr int kPer = (NQ + 31) / 32;
        int row_in[kPer], head_in[kPer];         // of this lane's columns
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int c = lane + 32 * u;
            row_in[u] = c < p.tile_rows * p.group ? c / p.group : 0x3fffffff;
            head_in[u] = c % p.group;
        }
        int g = 0;
        bool ok = true;
        for (int j = blockIdx.x; ok && j < total; j += stride) {
            if (!find_unit<kMany>(p, cum, j, it)) continue;
            // Many columns: -lse log2 e, a step's numbers loaded before the last one's are
            // stored; few: the numbers as they are.
            const auto row_of = [&](int t, int u) { return (it.step0 + t) * p.tile_rows + row_in[u]; };
            const auto lse_of = [&](int t, int u) {
                return p.lse + size_t(it.row0 + row_of(t, u)) * p.num_q_heads + it.kvh * p.group +
                       head_in[u];
            };
            float next[kPer];
            const auto load = [&](int t) {
#pragma unroll
                for (int u = 0; u < kPer; ++u)
                    next[u] = t < it.steps && row_of(t, u) < it.rows ? *lse_of(t, u) : 0.f;
            };
            if (kMany) load(0);
            for (int x = 0; x < it.steps * it.heads; ++x) {
                const int h = kMany ? 0 : x / it.steps, t = x - h * it.steps;
                const int s = g % C::kLseStages;
                float *to = reinterpret_cast<float *>(smem + C::lse) + s * NQ + lane;
                float now[kPer];
                if (kMany) {
#pragma unroll
                    for (int u = 0; u < kPer; ++u) now[u] = next[u] * -kLog2e;
                    load(t + 1);
                }
                if (g >= C::kLseStages)
                    ok = mbar_wait(&bar[C::bLEmpty + s], ((g / C::kLseStages) - 1) & 1, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++g;
                if (kMany) {
#pragma unroll
                    for (int u = 0; u < kPer; ++u) to[32 * u] = now[u];
                    mbar_arrive(&bar[C::bLFull + s]);
                } else {
#pragma unroll
                    for (int u = 0; u < kPer; ++u)
                        if (row_of(t, u) < it.rows)
                            cp_async_4(to + 32 * u, lse_of(t, u) + h * p.group);
                    cp_async_arrive(&bar[C::bLFull + s]);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ------------------------------------------------------------ epilogue
        const int part = warp >> 2;                              // of the columns
        const int k = (warp & 3) * 32 + lane;                    // key of a tile == TMEM lane
        const uint32_t s_base = tmem + (uint32_t((warp & 3) * 32) << 16);
        const float scale2 = p.scale * kLog2e;
        int g = 0;
        bool ok = true;
        // Every warp runs every item's named barriers, even after a wait gave up (ok ==
        // false), so no warp can strand the others.
        for (int j = blockIdx.x; j < total && (ok || C::kParts > 1); j += stride) {
            if (!find_unit<kMany>(p, cum, j, it)) continue;
            // The key that this thread stores, and its earlier weights on their way (many: the
            // threads of part i have key tile i).
            const int tile = part < KT ? part : 0, key = it.key0 + tile * kKeys + k;
            float *where = nullptr;
            float old[C::kHeads], w[C::kHeads];
#pragma unroll
            for (int h = 0; h < C::kHeads; ++h) old[h] = w[h] = 0.f;
            if (part < KT && key < it.L) {
                int slot;
                const int page = page_at(p, it.b, key, true, slot);
                if (page >= 0)
                    where = p.w.base + page * p.w.page + slot * p.w.token + it.kvh * p.w.head;
            }
            const bool together = C::kHeads == 4 && it.heads == 4 && p.w.head == 1 &&
                                  (reinterpret_cast<uintptr_t>(where) & 15) == 0;
            if (where && key < it.L - it.n && p.decay != 0.f) {
                if (together) {
                    const float4 v = *reinterpret_cast<const float4 *>(where);
                    old[0] = v.x;
                    if (C::kHeads == 4) { old[1] = v.y; old[2] = v.z; old[3] = v.w; }
                } else {
#pragma unroll
                    for (int h = 0; h < C::kHeads; ++h)
                        if (h < it.heads) old[h] = where[h * p.w.head];
                }
            }
#pragma unroll
            for (int h = 0; h < C::kHeads; ++h) {
                if (h >= it.heads) break;
                float2 sum[KT][2];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) sum[kt][0] = sum[kt][1] = make_float2(0.f, 0.f);
                for (int t = 0; ok && t < it.steps; ++t, ++g) {
                    const int ls = g % C::kLseStages;
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&bar[C::bLFull + ls], (g / C::kLseStages) & 1, p.err));
                    const float *lse = reinterpret_cast<const float *>(smem + C::lse) + ls * NQ;
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        const int x = g * KT + kt, sb = x & 1;
                        if (ok)
                            ok = __all_sync(0xffffffffu,
                                            mbar_wait(&bar[C::bSFull + sb], (x >> 1) & 1, p.err));
                        if (!ok) break;
                        tc::fence_after_sync();
                        const Columns cols = columns_of(p, it, kt, t);
                        const int lo = cols.seen_by(k), c1 = min((part + 1) * C::kCols, cols.hi);
                        const uint32_t s_at = s_base + sb * NQ;
                        if constexpr (kMany) {
                            // The warp's 32 keys see none of a chunk of 32 columns, all of it, or some.
                            const int none = cols.seen_by(k & ~31), all = cols.seen_by(k | 31);
#pragma unroll 1
                            for (int c = max(part * C::kCols, none & ~31); c < c1; c += 32) {
                                float v[32];
                                tc::tmem_ld32(s_at + c, v);
                                if (c >= all && c + 32 <= c1)
                                    add_weights<32, false, true>(v, lse + c, scale2, 0, 32, sum[kt]);
                                else
                                    add_weights<32, true, true>(v, lse + c, scale2, lo - c, c1 - c,
                                                                sum[kt]);
                            }
                        } else {
#pragma unroll 1
                            for (int c = 0; c < c1; c += 8) {
                                float v[8];
                                tc::tmem_ld_n<8>(s_at + c, v);
                                add_weights<8, true, false>(v, lse + c, p.scale, lo - c, c1 - c, sum[kt]);
                            }
                        }
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar[C::bSFree + sb]);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[C::bLEmpty + ls]);
                }
                w[h] = (sum[0][0].x + sum[0][0].y) + (sum[0][1].x + sum[0][1].y);
                if constexpr (C::kParts > 1) {       // the parts' sums of a key
                    float *parts = reinterpret_cast<float *>(smem + C::part);
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
                        parts[(part * KT + kt) * kKeys + k] =
                            (sum[kt][0].x + sum[kt][0].y) + (sum[kt][1].x + sum[kt][1].y);
                    named_sync(1, 32 * C::kEpiWarps);
                    w[h] = 0.f;
#pragma unroll
                    for (int i = 0; i < C::kParts; ++i) w[h] += parts[(i * KT + tile) * kKeys + k];
                    named_sync(1, 32 * C::kEpiWarps);
                }
            }
            if (!ok || !where) continue;
            if (key < it.L - it.n) {
#pragma unroll
                for (int h = 0; h < C::kHeads; ++h) w[h] = fmaf(old[h], p.decay, w[h]);
            }
            if (together) {
                *reinterpret_cast<float4 *>(where) =
                    make_float4(w[0], w[C::kHeads > 1 ? 1 : 0], w[C::kHeads > 2 ? 2 : 0],
                                w[C::kHeads > 3 ? 3 : 0]);
            } else {
#pragma unroll
                for (int h = 0; h < C::kHeads; ++h)
                    if (h < it.heads) where[h * p.w.head] = w[h];
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == C::kWarpMma) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int D, bool kMany>
cudaError_t launch(const WeightsParams &p, int sms, cudaStream_t stream) {
    using C = Cfg<D, kMany>;
    const auto bytes = [](int batch) {
        return size_t(C::items) + (kMany ? 0 : sizeof(int) * size_t(batch + 1));
    };
    const size_t smem = bytes(p.batch);
    auto kern = key_weights_kernel<D, kMany>;
    const cudaError_t e = allow_smem(kern, bytes(kGqaMaxBatch));
    if (e != cudaSuccess) return e;
    const long long units = (static_cast<long long>(p.max_kv_len - 1) / (C::KT * kKeys) + 1) *
                            p.batch * (kMany ? p.hkv : p.head_groups);
    long long ctas = kMany ? 64LL * sms : 2LL * sms;
    if (ctas > units) ctas = units;
    kern<<<static_cast<unsigned>(ctas), C::kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights(const WeightsParams &p, int head_dim, bool few, int sms,
                               cudaStream_t stream) {
    if (head_dim == 64)
        return few ? launch<64, false>(p, sms, stream) : launch<64, true>(p, sms, stream);
    return few ? launch<128, false>(p, sms, stream) : launch<128, true>(p, sms, stream);
}

}  // namespace attn
