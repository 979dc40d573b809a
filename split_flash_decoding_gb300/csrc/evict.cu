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
// digits for short calls.
#include <cooperative_groups.h>

#include "evict_ops.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace attn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kHeldKeys = 32768;             // weights of a CTA kept in shared memory (128 KB)

// A weight as a number whose order is that of weights: -0 counts as 0, NaN as -inf.
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
        if (err) atomicOr(err, kErrBadPage);
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

struct Shared {
    int hist[kBins];
    int merged[kBins];               // counts of all CTAs of the cluster
    int warp_sum[kWarps];
    int warp_more[kWarps], warp_equal[kWarps];
    int counts[2];                   // this CTA's kept for sure, and equal to the threshold
    int digit, rest;                 // of the last pass: the digit, and what is wanted inside it
};

__global__ void __launch_bounds__(kThreads)
evict_select_kernel(const __grid_constant__ EvictParams p, int held_keys) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    uint32_t *keys = reinterpret_cast<uint32_t *>(raw + sizeof(Shared));
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int unit = static_cast<int>(blockIdx.x) / ranks;
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
    const int slice = ((x.L + ranks - 1) / ranks + kThreads - 1) / kThreads * kThreads;
    const int t0 = min(rank * slice, x.L), t1 = min(t0 + slice, x.L);
    const int run = slice / kWarps;
    const int w0 = min(t0 + warp * run, t1), w1 = min(w0 + run, t1);
    const int c0 = x.f, c1 = x.L - x.r;      // the tokens that are chosen among
    const int wanted = x.n - x.r - x.f;      // of them
    const bool choose = wanted > 0 && wanted < c1 - c0;
    const bool held = slice <= held_keys;

    const auto read_key = [&](int t) -> uint32_t {
        int slot;
        const int page = page_in(p.page_table, p.max_pages, p.num_pages, p.page_size, b, t, p.err,
                                 slot);
        return page < 0 ? 0u : sort_key(p.w.base[page * p.w.page + slot * p.w.token +
                                                 kvh * p.w.head]);
    };
    const auto key_of = [&](int t) -> uint32_t { return held ? keys[t - t0] : read_key(t); };

    uint32_t least = 0;                      // the smallest weight that stays
    int take = 0;                            // how many of those equal to it
    if (choose) {
        if (held)
            for (int t = t0 + tid; t < t1; t += kThreads) keys[t - t0] = read_key(t);
        int rest = wanted;
        uint32_t mask = 0;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t bits = pass == 2 ? 1023u : 2047u;
            for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
            __syncthreads();
            for (int t = max(t0, c0) + tid; t < min(t1, c1); t += kThreads) {
                const uint32_t key = key_of(t);
                if ((key & mask) == least) atomicAdd(&sh.hist[(key >> shift) & bits], 1);
            }
            cluster.sync();
            for (int i = tid; i < kBins; i += kThreads) {
                int sum = 0;
                for (int r = 0; r < ranks; ++r) sum += *cluster.map_shared_rank(&sh.hist[i], r);
                sh.merged[i] = sum;
            }
            __syncthreads();
            // the digit d with fewer than `rest` keys above it, and at least that many from it on
            int mine[kBins / kThreads], local = 0;
#pragma unroll
            for (int i = 0; i < kBins / kThreads; ++i) {
                mine[i] = sh.merged[kBins - 1 - (tid * (kBins / kThreads) + i)];
                local += mine[i];
            }
            int incl = local;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) sh.warp_sum[warp] = incl;
            __syncthreads();
            int above = incl - local;
            for (int i = 0; i < warp; ++i) above += sh.warp_sum[i];
            if (above < rest && above + local >= rest) {
#pragma unroll
                for (int i = 0; i < kBins / kThreads; ++i) {
                    if (above < rest && above + mine[i] >= rest) {
                        sh.digit = kBins - 1 - (tid * (kBins / kThreads) + i);
                        sh.rest = rest - above;
                    }
                    above += mine[i];
                }
            }
            cluster.sync();                  // (also: the others have read this CTA's counts)
            least |= uint32_t(sh.digit) << shift;
            mask |= bits << shift;
            rest = sh.rest;
            __syncthreads();
        }
        take = rest;
    }

    // ---- what stays, per warp and CTA -------------------------------------------------
    // 0: goes; 1: stays; 2: stays if it is among the first `take` of its weight
    const auto kind_of = [&](int t) -> int {
        if (t < c0 || t >= c1) return 1;
        if (!choose) return wanted > 0;
        const uint32_t key = key_of(t);
        return key > least ? 1 : key == least ? 2 : 0;
    };
    int more = 0, equal = 0;
    for (int t = w0 + lane; t < w1; t += 32) {
        const int kind = kind_of(t);
        more += kind == 1;
        equal += kind == 2;
    }
    more = __reduce_add_sync(0xffffffffu, more);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        sh.warp_more[warp] = more;
        sh.warp_equal[warp] = equal;
    }
    __syncthreads();
    if (tid == 0) {
        int m = 0, e = 0;
        for (int i = 0; i < kWarps; ++i) {
            m += sh.warp_more[i];
            e += sh.warp_equal[i];
        }
        sh.counts[0] = m;
        sh.counts[1] = e;
    }
    cluster.sync();
    int base = 0, equals = 0;                // before this warp
    for (int r = 0; r < rank; ++r) {
        const int *c = cluster.map_shared_rank(sh.counts, r);
        base += c[0];
        equals += c[1];
    }
    for (int i = 0; i < warp; ++i) {
        base += sh.warp_more[i];
        equals += sh.warp_equal[i];
    }
    base += min(equals, take);
    int32_t *out = p.indices + (size_t(b) * p.hkv + kvh) * p.max_keep;
    for (int t = w0; t < w1; t += 32) {
        const int kind = t + lane < w1 ? kind_of(t + lane) : 0;
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t eq = __ballot_sync(0xffffffffu, kind == 2);
        const bool stays = kind == 1 || (kind == 2 && equals + __popc(eq & below) < take);
        const uint32_t in = __ballot_sync(0xffffffffu, stays);
        const int j = base + __popc(in & below);
        if (stays && j < x.n) out[j] = t + lane;   // (j < n unless weights change meanwhile)
        base += __popc(in);
        equals += __popc(eq);
    }
    cluster.sync();                          // (the others have read this CTA's counts)
}

// ---- the rows -----------------------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kMoveSlots = 16;               // kept tokens of a CTA
constexpr int kMoveAhead = 4;                // vectors of a thread on their way

__device__ __forceinline__ uint4 load_once(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ __align__(16) int2 from[];         // {page, slot} [kMoveSlots][hkv]
    __shared__ int2 to[kMoveSlots];
    const int b = blockIdx.y, j0 = static_cast<int>(blockIdx.x) * kMoveSlots;
    const int tid = threadIdx.x;
    const Lengths x = lengths_of(p, b);
    const int slots = min(kMoveSlots, x.n - j0);
    if (slots <= 0) return;
    if (tid < slots) {
        int slot;
        const int page = page_in(p.to_table, p.to_max_pages, p.to_num_pages, p.to_page_size, b,
                                 j0 + tid, p.err, slot);
        to[tid] = make_int2(page, slot);
    }
    pdl_wait_primary();
    for (int i = tid; i < slots * p.hkv; i += kMoveThreads) {
        const int h = i / slots, s = i - h * slots;
        const int t = p.indices[(size_t(b) * p.hkv + h) * p.max_keep + j0 + s];
        int slot = 0, page = -1;
        if (t >= 0 && t < x.L)
            page = page_in(p.page_table, p.max_pages, p.num_pages, p.page_size, b, t, nullptr, slot);
        from[s * p.hkv + h] = make_int2(page, slot);
    }
    __syncthreads();
    if (p.w_to.base)
        for (int i = tid; i < slots * p.hkv; i += kMoveThreads) {
            const int s = i / p.hkv, h = i - s * p.hkv;
            const int2 f = from[i], d = to[s];
            if (f.x >= 0 && d.x >= 0)
                p.w_to.base[d.x * p.w_to.page + d.y * p.w_to.token + h * p.w_to.head] =
                    p.w.base[f.x * p.w.page + f.y * p.w.token + h * p.w.head];
        }
    // vectors of a token: its heads' K, then its heads' V
    const int kv = p.k.vecs + p.v.vecs, per_slot = p.hkv * kv, all = slots * per_slot;
    for (int i0 = tid; i0 < all; i0 += kMoveThreads * kMoveAhead) {
        uint4 v[kMoveAhead];
        uint8_t *dst[kMoveAhead];
#pragma unroll
        for (int u = 0; u < kMoveAhead; ++u) {
            const int i = i0 + u * kMoveThreads;
            dst[u] = nullptr;
            if (i >= all) continue;
            const int s = i / per_slot;
            int c = i - s * per_slot;
            const bool is_k = c < p.hkv * p.k.vecs;
            const MovedRows &m = is_k ? p.k : p.v;
            if (!is_k) c -= p.hkv * p.k.vecs;
            const int h = c / m.vecs;
            c -= h * m.vecs;
            const int2 f = from[s * p.hkv + h], d = to[s];
            if (f.x < 0 || d.x < 0) continue;
            v[u] = load_once(m.from + f.x * m.from_page + f.y * m.from_token + h * m.from_head +
                             16 * c);
            dst[u] = m.to + d.x * m.to_page + d.y * m.to_token + h * m.to_head + 16 * c;
        }
#pragma unroll
        for (int u = 0; u < kMoveAhead; ++u)
            if (dst[u]) *reinterpret_cast<uint4 *>(dst[u]) = v[u];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t stream) {
    // CTAs of a unit: until the GPU is full, or the weights of one no longer fit it.
    const long long units = static_cast<long long>(p.batch) * p.hkv;
    int ranks = 1;
    while (ranks < kMaxCluster && p.max_kv_len > 2048 * ranks &&
           (units * ranks < sms || p.max_kv_len > kHeldKeys * ranks))
        ranks *= 2;
    const int slice = ((p.max_kv_len + ranks - 1) / ranks + kThreads - 1) / kThreads * kThreads;
    const int held = slice < kHeldKeys ? slice : kHeldKeys;
    const size_t smem = sizeof(Shared) + sizeof(uint32_t) * size_t(held);
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, held);
    if (e != cudaSuccess || p.max_keep == 0) return e;

    const size_t move_smem = sizeof(int2) * size_t(kMoveSlots) * size_t(p.hkv);
    cfg.gridDim = dim3(static_cast<unsigned>((p.max_keep + kMoveSlots - 1) / kMoveSlots),
                       static_cast<unsigned>(p.batch));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = move_smem;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

}  // namespace attn
