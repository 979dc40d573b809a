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
//   Few columns (rows x group <= 16, decode): KT = 1, one step of 16 columns.  Bound by
//   the stream of keys; two CTAs per SM walk the items of all sequences, KV heads
//   side by side.
//   More (prompts): KT = 2, steps of 128 columns.  Both key tiles stay in shared memory
//   while column tiles pass, each read once for 256 keys.  Bound by the exponentials and
//   the MMAs.  A CTA takes one item; those that the most rows see come first.
//
// Warp roles: four epilogue warps per key tile, K producer and Q producer (TMA), MMA
// issue, and one warp that fetches what the epilogue needs from memory (the rows' lse,
// the keys' earlier weights and where the new ones go).
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
    static constexpr int kKStages = kMany ? 2 : 3;           // items in flight
    static constexpr int kQStages = 2;
    static constexpr int kLseStages = 4;
    static constexpr int kOldStages = 2;                     // items of earlier weights
    static constexpr int kEpiWarps = 4 * KT;
    static constexpr int kWarpK = kEpiWarps, kWarpQ = kWarpK + 1, kWarpMma = kWarpK + 2,
                         kWarpAux = kWarpK + 3;
    static constexpr int kThreads = 32 * (kEpiWarps + 4);
    static constexpr int kTileBytes = kKeys * D * 2;
    static constexpr int kQBytes = NQ * D * 2;
    static constexpr int kTmemCols = 2 * KT * NQ;            // 32 or 512
    // shared memory
    static constexpr int k = 0;
    static constexpr int q = k + kKStages * KT * kTileBytes;
    static constexpr int lse = q + kQStages * kQBytes;
    static constexpr int old = lse + kLseStages * NQ * 4;
    static constexpr int at = old + kOldStages * KT * kKeys * 4;
    static constexpr int bars = at + kOldStages * KT * kKeys * 8;
    static constexpr int tmem_slot = bars + 256;
    static constexpr int items = tmem_slot + 16;
    // barriers
    static constexpr int bKFull = 0, bKEmpty = bKFull + kKStages, bQFull = bKEmpty + kKStages,
                         bQEmpty = bQFull + kQStages, bLFull = bQEmpty + kQStages,
                         bLEmpty = bLFull + kLseStages, bOFull = bLEmpty + kLseStages,
                         bOEmpty = bOFull + kOldStages, bSFull = bOEmpty + kOldStages,   // [2][KT]
                         bSFree = bSFull + 2 * KT, kNumBars = bSFree + 2 * KT;
    static_assert(kNumBars * 8 <= 256, "barrier space");
};

struct Item {
    int b, kvh, L, n, row0, rows;   // n: the sequence's rows; rows: those the call has
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
__device__ __forceinline__ void open_item(const WeightsParams &p, int b, int kvh, int tile, Item &it) {
    constexpr int KT = kMany ? 2 : 1;
    it.b = b;
    it.kvh = kvh;
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

// Item j of the call's list; false: there is none of that number (a later one may be).
//   few:  (sequence, tile, KV head), the last fastest; cum: tiles before each sequence
//   many: (tile from the sequence's end, falling; sequence, KV head): where the rows are
//         the last tokens, that many of them see the tile, so the dearest come first
template <bool kMany>
__device__ __forceinline__ bool find_item(const WeightsParams &p, const int *cum, int j, Item &it) {
    if (kMany) {
        const int units = p.batch * p.hkv, last = (p.max_kv_len - 1) / (2 * kKeys);
        const int e = last - j / units, u = j % units;
        const int b = u / p.hkv, tiles = tiles_of<2>(p, b);
        if (e >= tiles) return false;
        open_item<kMany>(p, b, u - b * p.hkv, tiles - 1 - e, it);
        return true;
    }
    const int x = j / p.hkv;
    int lo = 0, hi = p.batch;       // cum[lo] <= x < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= x) lo = mid; else hi = mid;
    }
    open_item<kMany>(p, lo, j - x * p.hkv, x - cum[lo], it);
    return true;
}

// Page of token t of sequence b (-1: outside the pool) and its slot.
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

__device__ __forceinline__ void cp_async_4(void *dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}
// Arrive (without raising the pending count) when this thread's copies so far are done.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// N scores of the thread's key, columns c0 on: adds their weights to sum.  kPart:
// only columns [lo, hi) count.
template <int N, bool kPart>
__device__ __forceinline__ void add_weights(const float (&v)[N], const float *lse, float scale,
                                            int c0, int lo, int hi, float2 (&sum)[2]) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(lse + c0 + c);
        const float2 f = make_float2(scale, scale), g = make_float2(kLog2e, kLog2e);
        // (score - lse first: the product with log2 e then errs by a part of that small number)
        const float2 x =
            __fmul2_rn(__ffma2_rn(make_float2(v[c], v[c + 1]), f, make_float2(-l.x, -l.y)), g);
        const float2 y =
            __fmul2_rn(__ffma2_rn(make_float2(v[c + 2], v[c + 3]), f, make_float2(-l.z, -l.w)), g);
        float w[4] = {fast_exp2(x.x), fast_exp2(x.y), fast_exp2(y.x), fast_exp2(y.y)};
        if (kPart) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + c + i < lo || c0 + c + i >= hi) w[i] = 0.f;
        }
        sum[0] = __fadd2_rn(sum[0], make_float2(w[0], w[1]));
        sum[1] = __fadd2_rn(sum[1], make_float2(w[2], w[3]));
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stride = static_cast<int>(gridDim.x);

    if (blockIdx.x == 0 && warp == 0)
        for (int b = lane; b < p.batch; b += 32)
            if (p.kv_len[b] > uint32_t(p.max_kv_len)) atomicOr(p.err, kErrBadLength);
    int total;
    if (kMany) {
        // (one item a CTA: most of those past a sequence's end leave here)
        total = ((p.max_kv_len - 1) / (KT * kKeys) + 1) * p.batch * p.hkv;
        if (stride >= total) {
            Item it;
            if (!find_item<kMany>(p, cum, blockIdx.x, it)) return;
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
            if (i >= C::bOFull && i < C::bOFull + C::kOldStages) n = 64;
            if (i >= C::bOEmpty && i < C::bOEmpty + C::kOldStages) n = C::kEpiWarps;
            if (i >= C::bSFree) n = 4;
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
    if (!kMany) total = cum[p.batch] * p.hkv;

    Item it;
    if (warp == C::kWarpK) {
        // ------------------------------------------------------------ K producer
        const int box_rows = p.box_rows, box_shift = 31 - __clz(box_rows);
        const int nb = (KT * kKeys) >> box_shift;                // boxes of an item
        const uint32_t box_bytes = uint32_t(box_rows) * D * 2;
        int g = 0;
        bool ok = true;
        for (int j = blockIdx.x; ok && j < total; j += stride) {
            if (!find_item<kMany>(p, cum, j, it) || it.steps == 0) continue;
            const int s = g % C::kKStages;
            const int live = min(nb, (it.L - it.key0 + box_rows - 1) >> box_shift);
            if (lane == 0) {
                if (g >= C::kKStages)
                    ok = mbar_wait(&bar[C::bKEmpty + s], ((g / C::kKStages) - 1) & 1, p.err);
                if (ok) mbar_arrive_expect_tx(&bar[C::bKFull + s], uint32_t(live) * box_bytes);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            ++g;
            uint8_t *dst = smem + C::k + s * (KT * C::kTileBytes);
            for (int r = lane; r < live; r += 32) {              // a box a lane
                int slot;
                const int page = page_at(p, it.b, it.key0 + (r << box_shift), true, slot);
                const int row = r << box_shift;                  // in the item
                uint8_t *to = dst + (row / kKeys) * C::kTileBytes + (row % kKeys) * 128;
                if (page < 0) {
                    mbar_complete_tx(&bar[C::bKFull + s], box_bytes);   // skipped bad page
                } else {
#pragma unroll
                    for (int cb = 0; cb < D / 64; ++cb)
                        tma_load_4d(to + cb * (kKeys * 128), &p.k_map, &bar[C::bKFull + s], cb * 64,
                                    slot, it.kvh, page);
                }
            }
            __syncwarp();
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
                if (!find_item<kMany>(p, cum, j, it)) continue;
                for (int t = 0; ok && t < it.steps; ++t) {
                    const int s = g % C::kQStages;
                    if (g >= C::kQStages)
                        ok = mbar_wait(&bar[C::bQEmpty + s], ((g / C::kQStages) - 1) & 1, p.err);
                    if (!ok) break;
                    ++g;
                    mbar_arrive_expect_tx(&bar[C::bQFull + s], bytes);
#pragma unroll
                    for (int cb = 0; cb < D / 64; ++cb)
                        tma_load_4d(smem + C::q + s * C::kQBytes + cb * (NQ * 128), &p.q_map,
                                    &bar[C::bQFull + s], cb * 64, 0, it.kvh,
                                    it.row0 + (it.step0 + t) * p.tile_rows);
                }
            }
            for (int i = max(0, g - C::kQStages); i < g; ++i)
                mbar_wait(&bar[C::bQFull + i % C::kQStages], (i / C::kQStages) & 1, p.err);
        }
    } else if (warp == C::kWarpMma) {
        // ------------------------------------------------------------ MMA issue
        if (lane == 0) {
            constexpr uint32_t idesc = tc::idesc_bf16_f32(128, NQ, 0, 0);
            const uint32_t k_base = smem_addr(smem + C::k), q_base = smem_addr(smem + C::q);
            int g = 0, gk = 0;
            bool ok = true;
            for (int j = blockIdx.x; ok && j < total; j += stride) {
                if (!find_item<kMany>(p, cum, j, it) || it.steps == 0) continue;
                const int ks = gk % C::kKStages;
                ok = mbar_wait(&bar[C::bKFull + ks], (gk / C::kKStages) & 1, p.err);
                for (int t = 0; ok && t < it.steps; ++t, ++g) {
                    const int qs = g % C::kQStages, sb = g & 1;
                    ok = mbar_wait(&bar[C::bQFull + qs], (g / C::kQStages) & 1, p.err);
                    const uint64_t qd = tc::smem_desc_sw128(q_base + qs * C::kQBytes, 16, 1024);
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        if (ok && g >= 2)
                            ok = mbar_wait(&bar[C::bSFree + sb * KT + kt], ((g >> 1) - 1) & 1, p.err);
                        if (!ok) break;
                        tc::fence_after_sync();
                        const uint64_t kd = tc::smem_desc_sw128(
                            k_base + (ks * KT + kt) * C::kTileBytes, 16, 1024);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t in = (kk & 3) * 32;   // within the 64 channels' rows
                            tc::mma_bf16(tmem + (sb * KT + kt) * NQ,
                                         kd + uint64_t(((kk >> 2) * (kKeys * 128) + in) >> 4),
                                         qd + uint64_t(((kk >> 2) * (NQ * 128) + in) >> 4), idesc,
                                         kk > 0);
                        }
                        tc::mma_commit(&bar[C::bSFull + sb * KT + kt]);
                    }
                    if (ok) tc::mma_commit(&bar[C::bQEmpty + qs]);
                }
                if (ok) tc::mma_commit(&bar[C::bKEmpty + ks]);
                ++gk;
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
        int g = 0, gi = 0;
        bool ok = true;
        for (int j = blockIdx.x; ok && j < total; j += stride) {
            if (!find_item<kMany>(p, cum, j, it)) continue;
            const int os = gi % C::kOldStages;
            if (gi >= C::kOldStages)
                ok = mbar_wait(&bar[C::bOEmpty + os], ((gi / C::kOldStages) - 1) & 1, p.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++gi;
            float *old = reinterpret_cast<float *>(smem + C::old) + os * (KT * kKeys);
            long long *at = reinterpret_cast<long long *>(smem + C::at) + os * (KT * kKeys);
#pragma unroll
            for (int u = 0; u < KT * kKeys / 32; ++u) {
                const int k = lane + 32 * u, t = it.key0 + k;
                long long where = -1;
                if (t < it.L) {
                    int slot;
                    const int page = page_at(p, it.b, t, false, slot);
                    if (page >= 0)
                        where = page * p.w.page + slot * p.w.token + it.kvh * p.w.head;
                }
                at[k] = where;
                if (where >= 0 && t < it.L - it.n)
                    cp_async_4(old + k, p.w.base + where);
                else
                    old[k] = 0.f;
            }
            cp_async_arrive(&bar[C::bOFull + os]);
            mbar_arrive(&bar[C::bOFull + os]);
            for (int t = 0; t < it.steps; ++t) {
                const int s = g % C::kLseStages;
                if (g >= C::kLseStages)
                    ok = mbar_wait(&bar[C::bLEmpty + s], ((g / C::kLseStages) - 1) & 1, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++g;
                const int i0 = (it.step0 + t) * p.tile_rows;
                float *to = reinterpret_cast<float *>(smem + C::lse) + s * NQ + lane;
#pragma unroll
                for (int u = 0; u < kPer; ++u)
                    if (i0 + row_in[u] < it.rows)
                        cp_async_4(to + 32 * u, p.lse + size_t(it.row0 + i0 + row_in[u]) * p.num_q_heads +
                                                    it.kvh * p.group + head_in[u]);
                cp_async_arrive(&bar[C::bLFull + s]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ------------------------------------------------------------ epilogue
        const int kt = warp >> 2;                                // key tile of the item
        const int k = (warp & 3) * 32 + lane;                    // key == TMEM lane
        const uint32_t s_base = tmem + (uint32_t((warp & 3) * 32) << 16) + kt * NQ;
        int g = 0, gi = 0;
        bool ok = true;
        for (int j = blockIdx.x; ok && j < total; j += stride) {
            if (!find_item<kMany>(p, cum, j, it)) continue;
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const int tile0 = it.key0 + kt * kKeys;
            for (int t = 0; ok && t < it.steps; ++t, ++g) {
                const int sb = g & 1, ls = g % C::kLseStages;
                const int i0 = (it.step0 + t) * p.tile_rows;     // first row of the columns
                const int hi = min(p.tile_rows, it.rows - i0) * p.group;
                // columns from which on this thread's key is seen
                const int lo = p.causal ? max(tile0 + k - (it.L - it.n) - i0, 0) * p.group : 0;
                const bool part = hi < NQ || (p.causal && tile0 + kKeys - 1 > it.L - it.n + i0);
                ok = mbar_wait(&bar[C::bLFull + ls], (g / C::kLseStages) & 1, p.err);
                if (ok) ok = mbar_wait(&bar[C::bSFull + sb * KT + kt], (g >> 1) & 1, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::fence_after_sync();
                const float *lse = reinterpret_cast<const float *>(smem + C::lse) + ls * NQ;
                const uint32_t s_at = s_base + sb * (KT * NQ);
                if constexpr (kMany) {
#pragma unroll 1
                    for (int c0 = 0; c0 < NQ && c0 < hi; c0 += 32) {
                        float v[32];
                        tc::tmem_ld32(s_at + c0, v);
                        if (part)
                            add_weights<32, true>(v, lse, p.scale, c0, lo, hi, sum);
                        else
                            add_weights<32, false>(v, lse, p.scale, c0, lo, hi, sum);
                    }
                } else {
#pragma unroll 1
                    for (int c0 = 0; c0 < NQ && c0 < hi; c0 += 8) {
                        float v[8];
                        tc::tmem_ld_n<8>(s_at + c0, v);
                        add_weights<8, true>(v, lse, p.scale, c0, lo, hi, sum);
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar[C::bSFree + sb * KT + kt]);
                    mbar_arrive(&bar[C::bLEmpty + ls]);
                }
            }
            if (!ok) break;
            const int os = gi % C::kOldStages;
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&bar[C::bOFull + os], (gi / C::kOldStages) & 1, p.err));
            if (!ok) break;
            ++gi;
            const float old =
                reinterpret_cast<const float *>(smem + C::old)[(os * KT + kt) * kKeys + k];
            const long long where =
                reinterpret_cast<const long long *>(smem + C::at)[(os * KT + kt) * kKeys + k];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[C::bOEmpty + os]);
            const float w = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            if (where >= 0)
                p.w.base[where] = tile0 + k < it.L - it.n ? fmaf(old, p.decay, w) : w;
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
    const size_t smem = size_t(C::items) + (kMany ? 0 : sizeof(int) * size_t(p.batch + 1));
    auto kern = key_weights_kernel<D, kMany>;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const long long items = (static_cast<long long>(p.max_kv_len - 1) / (C::KT * kKeys) + 1) *
                            p.batch * p.hkv;
    long long ctas = kMany ? 64LL * sms : 2LL * sms;
    if (ctas > items) ctas = items;
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
