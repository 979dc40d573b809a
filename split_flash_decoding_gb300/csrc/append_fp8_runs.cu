// append_fp8_runs.cu -- keys and values of long runs of new tokens (prompts) into
// a cache held in 8 bits (attn_append_kv_fp8).
//
// A CTA takes the new tokens of one sequence inside an aligned group of 128 tokens
// (whole blocks of up to 128) and some heads, keys' first.  Thread (item, lane)
// of 32 x 8 stands for the group's tokens 4 item .. 4 item + 3 and two 16-byte
// vectors of their heads, the ones that tiles::pair_of gives (a rotation's pairs
// are in one thread); values use the same two.  A warp then holds 16 tokens in
// order, a block's largest value is a few shuffles away, and only blocks of 32 and
// more tokens need shared memory and a barrier a head.  What a block holds from
// before belongs to the same threads as its new tokens, so each rounds its own to
// a scale that grew.
//
// The work on one head is a chain (load, sum of squares, maximum, codes), so the
// next head's vectors are fetched into shared memory meanwhile, each thread's own
// (in registers, they would spill).  cos and sin of the tokens' positions are
// shared by the CTA's heads.
#include "head_tiles.cuh"

namespace attn {

using namespace tiles;

namespace {

constexpr int kT = 256, kL = 8, kS = 4;        // threads, lanes of a head, tokens of a thread
constexpr int kMaxChunk = 32;                  // heads of a CTA

struct SlotPlace {
    long long k_at, v_at, ks_at, vs_at;        // offsets into the caches and their scales
    int pos, stored;
};

// Shared memory: angles [128][4][8] {c, s, c, s} when there is a rotation, then
// the vectors in flight [kS][2][kT].
size_t run_smem(const RowsParams &p) {
    return (p.rope.rot_dim > 0 ? size_t(kGroupTokens) * 4 * kL * sizeof(float4) : 0) +
           size_t(kT) * 2 * kS * sizeof(uint4);
}

__device__ __forceinline__ void copy_16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
                 : "memory");
}

template <bool kInter>
__global__ void __launch_bounds__(kT, 2)
append_fp8_runs_kernel(const __grid_constant__ RowsParams p, int chunks, int chunk_heads) {
    extern __shared__ __align__(16) float4 angles[];
    __shared__ SlotPlace places[kGroupTokens];
    __shared__ float s_old[kMaxChunk];         // scales of the block that holds earlier tokens
    __shared__ float s_part[2][kT / 32];       // maxima of 16 tokens
    __shared__ Tokens s_tile;
    __shared__ int s_any;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tile = static_cast<int>(blockIdx.x) / chunks;
    const int h0 = (static_cast<int>(blockIdx.x) - tile * chunks) * chunk_heads;
    const int h1 = min(h0 + chunk_heads, p.k.heads + p.v.heads);

    if (warp == 0) {
        Tokens t;
        const bool any = tile_tokens(p, tile, lane, t);
        if (lane == 0) {
            s_any = any;
            s_tile = t;
        }
    }
    __syncthreads();
    if (!s_any || s_tile.first < 0) return;    // (a group of tokens below 0 is stored nowhere)
    const int first = static_cast<int>(s_tile.first), count = s_tile.count, r0 = s_tile.row;
    const int group0 = first & ~(kGroupTokens - 1);
    const int B = p.block_tokens;

    // ---- this thread's tokens and channels; the first head's loads -------------------
    const int item = tid / kL, i0 = tid & (kL - 1);
    const int R = p.rope.rot_dim / 8, half = p.rope.rot_dim / 2;
    const int start = p.k.rot_start / 8;
    int va, vb;
    pair_of(kInter, 16, R, i0, va, vb);        // of 16 vectors no lane goes without
    const bool turn_a = va < R, turn_b = vb < R;
    const int ca = 8 * ordered(va, R, start), cb = 8 * ordered(vb, R, start);
    const bool norm_a = ca < p.k.norm_dim, norm_b = cb < p.k.norm_dim;
    uint4 ga = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), gb = ga;   // 1
    if (p.k.norm && norm_a) ga = *reinterpret_cast<const uint4 *>(p.k.norm + ca);
    if (p.k.norm && norm_b) gb = *reinterpret_cast<const uint4 *>(p.k.norm + cb);
    uint4 *ahead = reinterpret_cast<uint4 *>(angles + (half > 0 ? kGroupTokens * 4 * kL : 0)) + tid;
    const int row0 = 4 * item - (first - group0);                // row of its first token
    const auto fetch = [&](int h) {
        const bool is_k = h < p.k.heads;
        const long long step = is_k ? p.k.in_row : p.v.in_row;
        const uint16_t *src = (is_k ? p.k.in + h * p.k.in_head
                                    : p.v.in + (h - p.k.heads) * p.v.in_head) + (r0 + row0) * step;
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            if (row0 + s < 0 || row0 + s >= count) continue;
            copy_16(ahead + 2 * s * kT, src + s * step + ca);
            copy_16(ahead + (2 * s + 1) * kT, src + s * step + cb);
        }
    };
#pragma unroll
    for (int s = 0; s < kS; ++s)
        if (row0 + s < 0 || row0 + s >= count)                   // never fetched
            ahead[2 * s * kT] = ahead[(2 * s + 1) * kT] = make_uint4(0u, 0u, 0u, 0u);
    fetch(h0);

    // ---- places ----------------------------------------------------------------------
    for (int i = tid; i < kGroupTokens; i += kT) {
        SlotPlace at;
        at.k_at = at.v_at = at.ks_at = at.vs_at = 0;
        at.stored = 0;
        const int t = group0 + i, row = t - first;
        at.pos = t;
        // (tokens that the first block holds from before have a place too)
        if (t >= (first & ~(B - 1)) && row < count && t < p.max_kv_len) {
            const int page = page_of(p, s_tile.b, t);
            const int slot = p.page_table ? t & (p.page_size - 1) : t;
            if (page >= 0) {
                at.stored = 1;
                at.k_at = page * p.kc.page_stride + slot * p.kc.token_stride;
                at.v_at = page * p.vc.page_stride + slot * p.vc.token_stride;
                at.ks_at = page * p.kc.scale_page + (slot >> p.block_shift) * p.kc.scale_block;
                at.vs_at = page * p.vc.scale_page + (slot >> p.block_shift) * p.vc.scale_block;
            }
        }
        if (p.positions && row >= 0 && row < count) at.pos = p.positions[r0 + row];
        places[i] = at;
    }
    __syncthreads();

    // ---- the first block's old scales; angles, one entry (two pairs) a thread -------
    const int first_slot = first - group0;
    // (B is at most 128, and a first block without a place has no held tokens)
    const int held = s_tile.first == s_tile.begin && places[first_slot].stored ? first & (B - 1) : 0;
    if (held > 0 && tid < h1 - h0) {
        const int h = h0 + tid;
        const SlotPlace &at = places[first_slot];
        s_old[tid] = h < p.k.heads ? p.kc.scale[at.ks_at + h * p.kc.scale_head]
                                   : p.vc.scale[at.vs_at + (h - p.k.heads) * p.vc.scale_head];
    }
    if (half > 0 && h0 < p.k.heads) {
        for (int e = tid; e < kGroupTokens * 4 * kL; e += kT) {
            const int slot = e / (4 * kL), k = e / kL & 3, i = e & (kL - 1);
            if (slot < first_slot || slot >= first_slot + count) continue;
            int a, b;
            pair_of(kInter, 16, R, i, a, b);
            const int j0 = kInter ? 4 * a + k : 8 * i + 2 * k;
            const int j1 = kInter ? 4 * b + k : j0 + 1;
            float4 v = make_float4(1.f, 0.f, 1.f, 0.f);
            if (a < R) rope_cos_sin(p.rope, j0, places[slot].pos, v.x, v.y);
            if (b < R) rope_cos_sin(p.rope, j1, places[slot].pos, v.z, v.w);
            angles[e] = v;
        }
    }
    __syncthreads();

#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
        const bool is_k = h < p.k.heads;
        float2 ya[kS][4], yb[kS][4];
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            unpack8(ahead[2 * s * kT], ya[s]);
            unpack8(ahead[(2 * s + 1) * kT], yb[s]);
        }
        if (is_k && p.k.norm_dim > 0) {
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                float2 sq = make_float2(0.f, 0.f);
                if (norm_a) add_squares(ya[s], sq);
                if (norm_b) add_squares(yb[s], sq);
                float sum = sq.x + sq.y;
#pragma unroll
                for (int o = 1; o < kL; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float inv = rsqrtf(fmaf(sum, p.k.mean, p.k.eps));
                if (norm_a) scale8(ya[s], ga, inv);
                if (norm_b) scale8(yb[s], gb, inv);
            }
        }
        if (is_k && turn_a) {
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                const float4 *t = angles + (4 * item + s) * 4 * kL + i0;
#pragma unroll
                for (int k = 0; k < 4; ++k) rotate_pairs<kInter>(ya[s][k], yb[s][k], t[k * kL], turn_b);
            }
        }

        // ---- largest value of each token's block --------------------------------------
        float top[kS];
        unsigned infinite = 0;                                   // tokens with an infinity
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            top[s] = largest(ya[s], yb[s]);
            if (top[s] > FLT_MAX) {
                infinite |= 1u << s;
                top[s] = largest_finite(ya[s], yb[s]);
            }
            if (row0 + s < 0 || row0 + s >= count || !places[4 * item + s].stored) top[s] = 0.f;
        }
        if (B >= 4) {
            float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
#pragma unroll
            for (int o = 1; o < kL; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (B >= 8) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            if (B >= 16) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            if (B >= 32) {
                float *part = s_part[(h - h0) & 1];              // (two heads: one barrier each)
                if (lane == 0) part[warp] = m;
                __syncthreads();
                const int w0 = warp & ~(B / 16 - 1);
                for (int w = 0; w < B / 16; ++w) m = fmaxf(m, part[w0 + w]);
            }
#pragma unroll
            for (int s = 0; s < kS; ++s) top[s] = m;
        } else {
#pragma unroll
            for (int s = 0; s < kS; ++s)
#pragma unroll
                for (int o = 1; o < kL; o <<= 1)
                    top[s] = fmaxf(top[s], __shfl_xor_sync(0xffffffffu, top[s], o));
            if (B == 2) {
                top[0] = top[1] = fmaxf(top[0], top[1]);
                top[2] = top[3] = fmaxf(top[2], top[3]);
            }
        }
        // This head's vectors have all been used: the next one's may take their place.
        if (h + 1 < h1) fetch(h + 1);

        // ---- scales and codes ------------------------------------------------------------
        const CacheOut &c = is_k ? p.kc : p.vc;
        const int head = is_k ? h : h - p.k.heads;
        float scale = 0.f, f = 0.f, ratio = 1.f;
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const int slot = 4 * item + s, row = row0 + s;
            if (s == 0 || B < 4) {                               // (four tokens share blocks of 4)
                scale = pow2i(scale_exponent(top[s]));
                ratio = 1.f;
                if (held > 0 && (slot ^ first_slot) < B) {       // the block of the first token
                    const float old = s_old[h - h0];
                    if (scale > old) ratio = old / scale; else scale = old;
                }
                f = __frcp_rn(scale);
            }
            const SlotPlace &at = places[slot];
            if (!at.stored) continue;
            uint8_t *dst = c.base + (is_k ? at.k_at : at.v_at) + head * c.head_stride;
            if (row < 0) {                                       // held from before
                if (ratio != 1.f) {
                    uint2 *wa = reinterpret_cast<uint2 *>(dst + ca);
                    uint2 *wb = reinterpret_cast<uint2 *>(dst + cb);
                    const uint2 oa = *wa, ob = *wb;
                    *wa = make_uint2(recode4(oa.x, ratio), recode4(oa.y, ratio));
                    *wb = make_uint2(recode4(ob.x, ratio), recode4(ob.y, ratio));
                }
                continue;
            }
            if (i0 == 0 && ((slot & (B - 1)) == 0 || row == 0))
                c.scale[(is_k ? at.ks_at : at.vs_at) + head * c.scale_head] = scale;
            store_codes(dst + ca, dst + cb, ya[s], yb[s], f, infinite >> s & 1);
        }
    }
}

}  // namespace

cudaError_t launch_fp8_runs(const RowsParams &p, cudaStream_t stream) {
    // A tile's angles cost about as much as two heads; as many heads to a CTA as
    // leave the waves full.
    constexpr int kWave = 2 * 152;
    const int heads = p.k.heads + p.v.heads;
    const long long likely = p.num_rows / kGroupTokens + p.batch;
    int best = 1;
    long long least = 0;
    for (int chunk = 1; chunk <= heads && chunk <= kMaxChunk; ++chunk) {
        const long long ctas = likely * ((heads + chunk - 1) / chunk);
        const long long cost = (ctas + kWave - 1) / kWave * (chunk + 2);
        if (chunk == 1 || cost < least) {
            least = cost;
            best = chunk;
        }
    }
    const int chunks = (heads + best - 1) / best;
    const long long blocks = fp8_tile_count(p) * chunks;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto kern = p.rope.interleaved ? append_fp8_runs_kernel<true> : append_fp8_runs_kernel<false>;
    const size_t smem = run_smem(p);
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(blocks), kT, smem, stream>>>(p, chunks, best);
    return cudaGetLastError();
}

}  // namespace attn
