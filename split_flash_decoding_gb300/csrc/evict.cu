// evict.cu -- keeps the keys of a cache that gathered the most attention weight and
// moves them together (attn_evict_kv).
//
// Of a sequence's L tokens n = min(L, keep) stay, for every KV head its own: the last
// r = min(recent, n), the first f = min(first, n - r), and of those in between the n - r - f
// of the largest weight (equal weights: the lowest token).  They go, in their order, to
// slots 0 to n - 1 of other pages.
//
// Two kernels.  The first finds, for a (sequence, KV head), the smallest weight that
// stays, by the digits of the weights' bit patterns (11, 11 and 10 bits: counts in shared
// memory, then the digit in which the wanted rank falls), and writes the list of kept
// tokens.  A unit's tokens are split over a cluster of up to 8 CTAs, which join their counts
// through distributed shared memory, so the weights are read once from memory and stay
// on chip.  Nothing depends on the order of atomics: they count.
// The second copies the rows the list names, 16 bytes a thread.
// Bound by the rows' bytes (read and written once) for prompts, by the chain of the
// digits for short calls.  8 KV heads of 128 channels: 16 prompts of 1024 to 8192 tokens to a
// quarter 39.9 us, 10.6 of them the choice; 131072 tokens to an eighth 46.3 us, 21.6 of them the
// choice (4 bytes of every 32-byte sector where a token's heads lie side by side) and the rows at
// 5.4 TB/s; 2 sequences of up to 300 tokens 6.0 us.  (Counts of the first digit in 4 or 8 copies
// by lane the same, clusters of 16 slower.  Keys in shared memory, counts joined by every CTA of a
// cluster and a row's place found anew for each vector, all three together: 75.0 instead of 46.9.)
#include <cooperative_groups.h>

#include "evict_ops.h"
#include "launch.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace attn {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMostPer = 16;                 // weights of a thread kept in registers
constexpr int kHeldKeys = 32768;             // of a CTA, past that, kept in shared memory (128 KB)

// A weight as a number whose order is that of weights: -0 counts as 0, NaN as -inf.
// (kStays is above all of them, 0 below.)
constexpr uint32_t kStays = 0xffffffffu;
__device__ __forceinline__ uint32_t sort_key(float w) {
    if (!(w == w)) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Page of token t of sequence b in a table (-1: outside the pool) and its slot.
__device__ __forceinline__ int page_in(const int32_t *table, int max_pages, int num_pages,
                                       int page_size, int b, int t, unsigned *err, int &slot) {
    if (!table) {
        slot = t;
        return b;
    }
    const int pidx = t >> (31 - __clz(page_size));   // (pages of a table: powers of two)
    slot = t & (page_size - 1);
    const int e = pidx < max_pages ? table[size_t(b) * max_pages + pidx] : -1;
    if (e < 0 || e >= num_pages) {
        atomicOr(err, kErrBadPage);
        return -1;
    }
    return e;
}

// Lengths of sequence b: L tokens, n kept, the last r and the first f of them always.
struct Lengths {
    int L, n, r, f;
};
__device__ __forceinline__ Lengths lengths_of(const EvictParams &p, int b) {
    Lengths x;
    x.L = static_cast<int>(min(p.kv_len[b], uint32_t(p.max_kv_len)));
    x.n = min(x.L, min(max(p.keep[b], 0), p.max_keep));
    x.r = min(p.recent, x.n);
    x.f = min(p.first, x.n - x.r);
    return x;
}

constexpr int kPasses = 3;                   // digits of 11, 11 and 10 bits

struct Shared {
    int hist[kPasses][kBins];        // this CTA's counts
    int warp_sum[kWarps];
    int warp_more[kWarps], warp_equal[kWarps];
    int counts[2];                   // this CTA's kept for sure, and equal to the threshold
    int merged[kPasses][kBins];      // first CTA of a cluster: the counts of all
    int digit, rest, all;            // of a pass: the digit, the keys wanted of it, all of its keys
};

// Sum over the warps before this one, of a value for each warp (in shared memory), by
// every warp for itself; total: of all.
__device__ __forceinline__ int before_warp(const int *sums, int warp, int lane, int &total) {
    static_assert(kWarps == 32, "a lane a warp");
    const int mine = sums[lane];
    total = __reduce_add_sync(0xffffffffu, mine);
    return __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0);
}

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// kPer: tokens of a thread, whose keys stay in registers; 0: any number, their keys in
// shared memory or, past held_keys, read again for every digit.
template <int kRanks, int kPer>
__global__ void __launch_bounds__(kThreads, 1)
evict_select_kernel(const __grid_constant__ EvictParams p, int held_keys) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    uint32_t *keys = reinterpret_cast<uint32_t *>(raw + sizeof(Shared));
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = kRanks > 1 ? static_cast<int>(cluster.block_rank()) : 0;
    const int unit = static_cast<int>(blockIdx.x) / kRanks;
    const int b = unit / p.hkv, kvh = unit - b * p.hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();

    const Lengths x = lengths_of(p, b);
    if (kvh == 0 && rank == 0 && tid == 0) {
        if (p.kv_len[b] > uint32_t(p.max_kv_len) || p.keep[b] > p.max_keep)
            atomicOr(p.err, kErrBadLength);
        if (p.kept_len) p.kept_len[b] = uint32_t(x.n);
    }
    // Tokens [t0, t1) are this CTA's; a warp has a run of them, of whole 32s.
    const int slice = ((x.L + kRanks - 1) / kRanks + kThreads - 1) / kThreads * kThreads;
    const int t0 = min(rank * slice, x.L), t1 = min(t0 + slice, x.L);
    const int run = slice / kWarps;
    const int w0 = min(t0 + warp * run, t1), w1 = min(w0 + run, t1);
    const int c0 = x.f, c1 = x.L - x.r;      // the tokens that are chosen among
    const int wanted = x.n - x.r - x.f;      // of them
    const bool choose = wanted > 0 && wanted < c1 - c0;
    const bool held = slice <= held_keys;

    const float *weights = p.w.base + kvh * p.w.head;
    const auto where = [&](int t) -> const float * {
        int slot;
        const int page = page_in(p.page_table, p.max_pages, p.num_pages, p.page_size, b, t, p.err,
                                 slot);
        return page < 0 ? nullptr : weights + page * p.w.page + slot * p.w.token;
    };
    // The key of token t of this CTA: kStays for those that stay whatever their weight.
    const auto read_key = [&](int t) -> uint32_t {
        if (t < c0 || t >= c1) return kStays;
        if (!choose) return 0u;
        const float *at = where(t);
        return at ? sort_key(*at) : 0u;
    };
    uint32_t mine[kPer > 0 ? kPer : 1] = {};
    // f(t, index) for this thread's tokens and, all lanes of a warp at once, what is past them
    const auto each = [&](auto f) {
        if constexpr (kPer > 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (32 * i < run) f(w0 + lane + 32 * i, i);      // (uniform)
            }
        } else {
            for (int t = w0 + lane; t - lane < w1; t += 32) f(t, 0);
        }
    };
    const auto key_of = [&](int t, int i) -> uint32_t {
        if (kPer > 0) return mine[i];
        return t >= w1 ? 0u : held ? keys[t - t0] : read_key(t);
    };

    if constexpr (kPer > 0) {
        // eight tokens' page numbers first, then their weights: two waits for eight
        constexpr int kBatch = kPer < 8 ? kPer : 8;
#pragma unroll
        for (int i0 = 0; i0 < kPer; i0 += kBatch) {
            const float *at[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u, t = w0 + lane + 32 * i;
                const bool stays = t < c0 || t >= c1;
                mine[i] = stays ? kStays : 0u;
                at[u] = choose && !stays && 32 * i < run && t < w1 ? where(t) : nullptr;
            }
            float w[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) w[u] = at[u] ? *at[u] : 0.f;
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (at[u]) mine[i0 + u] = sort_key(w[u]);
        }
    } else if (held) {
        for (int t = w0 + lane; t < w1; t += 32) keys[t - t0] = read_key(t);
    }

    // the smallest weight that stays, its known digits
    uint32_t least = 0, mask = choose ? 0u : ~0u;
    int rest = wanted;                       // how many of those equal to it, as far as known
    if (choose) {
        for (int i = tid; i < kPasses * kBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
        if (kRanks > 1) {
            for (int i = tid; i < kPasses * kBins; i += kThreads) (&sh.merged[0][0])[i] = 0;
            cluster.sync();                  // (before other CTAs add to them)
        }
        __syncthreads();
#pragma unroll 1
        for (int pass = 0; pass < kPasses; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t bits = pass == 2 ? 1023u : 2047u;
            int *hist = sh.hist[pass];
            each([&](int t, int i) {
                const uint32_t key = key_of(t, i);
                if ((key & mask) == least && key != kStays && t < w1)
                    atomicAdd(&hist[(key >> shift) & bits], 1);
            });
            __syncthreads();
            if (kRanks > 1) {                // to the first CTA of the cluster, which does the rest
                int *to = cluster.map_shared_rank(sh.merged[pass], 0);
                for (int i = tid; i < kBins; i += kThreads) {
                    const int c = hist[i];
                    if (c) atomicAdd(to + i, c);
                }
                cluster.sync();
                hist = sh.merged[pass];
            }
            // The digit with fewer than `rest` keys above it, and at least that many from it
            // on; thread t has the bins 2 t and 2 t + 1 from above.
            static_assert(kBins == 2 * kThreads, "two bins a thread");
            if (rank == 0) {
                const int top = kBins - 1 - 2 * tid;
                const int n0 = hist[top], n1 = hist[top - 1], local = n0 + n1;
                const int incl = warp_inclusive(local, lane);
                if (lane == 31) sh.warp_sum[warp] = incl;
                __syncthreads();
                int total;
                const int above = before_warp(sh.warp_sum, warp, lane, total) + incl - local;
                if (above < rest && above + local >= rest) {
                    const bool first = above + n0 >= rest;
                    for (int r = 0; r < kRanks; ++r) {
                        Shared *to = kRanks > 1 ? cluster.map_shared_rank(&sh, r) : &sh;
                        to->digit = first ? top : top - 1;
                        to->rest = rest - above - (first ? 0 : n0);
                        to->all = first ? n0 : n1;
                    }
                }
            }
            if (kRanks > 1) cluster.sync(); else __syncthreads();
            least |= uint32_t(sh.digit) << shift;
            mask |= bits << shift;
            rest = sh.rest;
            if (rest == sh.all) break;       // all keys of these digits stay: no need of the others
            // (the next pass writes these behind its first barriers)
        }
    }

    // ---- what stays, per warp and CTA -------------------------------------------------
    // more: above the least key that stays; equal: that key, of which the first `rest` stay
    int more = 0, equal = 0;
    each([&](int t, int i) {
        const uint32_t key = key_of(t, i) & mask;
        if (t < w1) {
            more += key > least;
            equal += key == least;
        }
    });
    more = __reduce_add_sync(0xffffffffu, more);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        sh.warp_more[warp] = more;
        sh.warp_equal[warp] = equal;
    }
    __syncthreads();
    int all_more, all_equal;
    int base = before_warp(sh.warp_more, warp, lane, all_more);
    int equals = before_warp(sh.warp_equal, warp, lane, all_equal);   // before this warp
    if constexpr (kRanks > 1) {
        if (tid == 0) {
            sh.counts[0] = all_more;
            sh.counts[1] = all_equal;
        }
        cluster.sync();
        const int *c = cluster.map_shared_rank(sh.counts, lane < rank ? lane : rank);
        const int m = c[0], e = c[1];
        base += __reduce_add_sync(0xffffffffu, lane < rank ? m : 0);
        equals += __reduce_add_sync(0xffffffffu, lane < rank ? e : 0);
    }
    base += min(equals, rest);
    int32_t *out = p.indices + (size_t(b) * p.hkv + kvh) * p.max_keep;
    const uint32_t below = (1u << lane) - 1u;
    each([&](int t, int i) {
        const uint32_t key = key_of(t, i) & mask;
        bool stays = key > least && t < w1;
        const uint32_t eq = __ballot_sync(0xffffffffu, key == least && t < w1);
        if (eq) {                                  // (uniform)
            stays = stays || ((eq >> lane & 1u) && equals + __popc(eq & below) < rest);
            equals += __popc(eq);
        }
        const uint32_t in = __ballot_sync(0xffffffffu, stays);
        const int j = base + __popc(in & below);
        if (stays && j < x.n) out[j] = t;          // (j < n unless weights change meanwhile)
        base += __popc(in);
    });
    if (kRanks > 1) cluster.sync();          // (the others have read this CTA's counts)
}

// ---- the rows -----------------------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kMoveEntries = 256;            // (slot, head) pairs of a CTA, at most
constexpr int kMoveAhead = 4;                // rows of a warp's lanes on their way

// Where an entry's rows are and go, in bytes from the caches' bases; k_from < 0: nowhere.
struct Entry {
    long long k_from, v_from, k_to, v_to;
};

__device__ __forceinline__ uint4 load_once(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Copies the entries' rows of one cache, 2^lanes_shift lanes a row.
template <bool kIsK>
__device__ __forceinline__ void move_rows(const MovedRows &m, const Entry *entries, int count,
                                          int lanes_shift) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_warp = 32 >> lanes_shift, step = kMoveWarps * per_warp;
    const int e_of = warp * per_warp + (lane >> lanes_shift), c_of = lane & ((1 << lanes_shift) - 1);
    for (int e0 = e_of; e0 < count; e0 += step * kMoveAhead) {
        long long from[kMoveAhead], to[kMoveAhead];
#pragma unroll
        for (int u = 0; u < kMoveAhead; ++u) {
            const int e = e0 + u * step;
            const Entry *at = entries + (e < count ? e : e0);
            from[u] = e < count && at->k_from >= 0 ? (kIsK ? at->k_from : at->v_from) : -1;
            to[u] = kIsK ? at->k_to : at->v_to;
        }
        for (int c = c_of; c < m.vecs; c += 32) {
            uint4 v[kMoveAhead];
#pragma unroll
            for (int u = 0; u < kMoveAhead; ++u)
                if (from[u] >= 0) v[u] = load_once(m.from + from[u] + 16 * c);
#pragma unroll
            for (int u = 0; u < kMoveAhead; ++u)
                if (from[u] >= 0) *reinterpret_cast<uint4 *>(m.to + to[u] + 16 * c) = v[u];
        }
    }
}

__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const __grid_constant__ EvictParams p, int slots_of_cta, int k_shift, int v_shift) {
    __shared__ Entry entries[kMoveEntries];
    const int b = blockIdx.y, j0 = static_cast<int>(blockIdx.x) * slots_of_cta;
    const int tid = threadIdx.x;
    const Lengths x = lengths_of(p, b);
    const int slots = min(slots_of_cta, x.n - j0);
    if (slots <= 0) {
        // (where no sequence keeps a token, this grid still ends after the one before it)
        if (blockIdx.x == 0 && b == 0) pdl_wait_primary();
        return;
    }
    const int count = slots * p.hkv;
    // an entry a thread, a token's heads side by side
    const int s = tid / p.hkv, h = tid - s * p.hkv;
    int page_to = -1, slot_to = 0;
    if (tid < count)
        page_to = page_in(p.to_table, p.to_max_pages, p.to_num_pages, p.to_page_size, b, j0 + s, p.err,
                          slot_to);
    pdl_wait_primary();
    if (tid < count) {
        const int t = p.indices[(size_t(b) * p.hkv + h) * p.max_keep + j0 + s];
        int slot = 0, page = -1;
        if (t >= 0 && t < x.L)
            // (reported here too: of tokens that stay in any case the choice has read no weight)
            page = page_in(p.page_table, p.max_pages, p.num_pages, p.page_size, b, t, p.err, slot);
        Entry at;
        at.k_from = page * p.k.from_page + slot * p.k.from_token + h * p.k.from_head;
        at.v_from = page * p.v.from_page + slot * p.v.from_token + h * p.v.from_head;
        at.k_to = page_to * p.k.to_page + slot_to * p.k.to_token + h * p.k.to_head;
        at.v_to = page_to * p.v.to_page + slot_to * p.v.to_token + h * p.v.to_head;
        const bool moves = page >= 0 && page_to >= 0;
        if (!moves) at.k_from = -1;
        entries[tid] = at;
        if (moves && p.w_to.base)
            p.w_to.base[page_to * p.w_to.page + slot_to * p.w_to.token + h * p.w_to.head] =
                p.w.base[page * p.w.page + slot * p.w.token + h * p.w.head];
    }
    __syncthreads();
    move_rows<true>(p.k, entries, count, k_shift);
    if (p.v.vecs > 0) move_rows<false>(p.v, entries, count, v_shift);
}

// Lanes of a row of `vecs` vectors, as a power of two.
int lanes_of(int vecs) {
    int shift = 0;
    while (shift < 5 && (1 << shift) < vecs) ++shift;
    return shift;
}

template <int kRanks, int kPer>
cudaError_t launch_select(const EvictParams &p, int slice, cudaStream_t stream) {
    const int held = kPer > 0 ? 0 : slice < kHeldKeys ? slice : kHeldKeys;
    auto kern = evict_select_kernel<kRanks, kPer>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch * p.hkv * kRanks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared) + sizeof(uint32_t) * size_t(held);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kRanks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        allow_smem(kern, sizeof(Shared) + (kPer > 0 ? 0 : sizeof(uint32_t) * size_t(kHeldKeys)));
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, kern, p, held);
}

template <int kRanks>
cudaError_t launch_ranks(const EvictParams &p, cudaStream_t stream) {
    const int slice = ((p.max_kv_len + kRanks - 1) / kRanks + kThreads - 1) / kThreads * kThreads;
    if constexpr (kRanks == 1) {
        if (slice <= kThreads) return launch_select<kRanks, 1>(p, slice, stream);
    }
    if (slice <= 4 * kThreads) return launch_select<kRanks, 4>(p, slice, stream);
    if (slice <= 8 * kThreads) return launch_select<kRanks, 8>(p, slice, stream);
    // (fewer CTAs than a cluster's most never have longer slices)
    if constexpr (kRanks == kMaxCluster) {
        if (slice > kMostPer * kThreads) return launch_select<kRanks, 0>(p, slice, stream);
    }
    return launch_select<kRanks, kMostPer>(p, slice, stream);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t stream) {
    // CTAs of a unit (one an SM, of 1024 threads): as many as fill the GPU once, and more
    // where a thread would have more weights than its registers hold.
    const long long units = static_cast<long long>(p.batch) * p.hkv;
    int ranks = 1;
    while (ranks < kMaxCluster && p.max_kv_len > 2 * kThreads * ranks &&
           (units * ranks * 2 <= sms || p.max_kv_len > kMostPer * kThreads * ranks))
        ranks *= 2;
    cudaError_t e = ranks == 1   ? launch_ranks<1>(p, stream)
                    : ranks == 2 ? launch_ranks<2>(p, stream)
                    : ranks == 4 ? launch_ranks<4>(p, stream)
                                 : launch_ranks<8>(p, stream);
    if (e != cudaSuccess || p.max_keep == 0) return e;

    int slots = kMoveEntries / p.hkv;
    if (slots > 32) slots = 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.max_keep + slots - 1) / slots),
                       static_cast<unsigned>(p.batch));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p, slots, lanes_of(p.k.vecs),
                              lanes_of(p.v.vecs));
}

}  // namespace attn
