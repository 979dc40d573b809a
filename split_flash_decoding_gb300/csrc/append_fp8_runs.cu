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
// shared by the CTA's heads.  Bound by that chain, with the two CTAs an SM that the
// registers allow: 24768 rows of 8 + 8 heads (152 MB) take 49 us where their bytes
// take 22; the tile kernel of the short runs with four items a thread took 77.
#include "head_tiles.cuh"

namespace attn {

using namespace tiles;

namespace {

constexpr int kT = 256, kL = 8, kS = 4;        // threads, lanes of a head, tokens of a thread
constexpr int kMaxChunk = 32;                  // heads of a CTA

// Heads of a CTA and CTAs of a tile, keys and values apart; CTAs of all keys.
struct RunCut {
    int k_chunk, v_chunk, k_chunks, v_chunks, k_ctas;
};

// Shared memory: angles [128][4][8] when there is a rotation, then the vectors in
// flight [kS][2][kT].
size_t run_smem(const RowsParams &p) {
    return (p.rope.rot_dim > 0 ? size_t(kGroupTokens) * 4 * kL * sizeof(float4) : 0) +
           size_t(kT) * 2 * kS * sizeof(uint4);
}

template <bool kInter>
__global__ void __launch_bounds__(kT, 2)
append_fp8_runs_kernel(const __grid_constant__ RowsParams p, const __grid_constant__ RunCut cut) {
    extern __shared__ __align__(16) float4 angles[];
    __shared__ float s_old[kMaxChunk];         // scales of the block that holds earlier tokens
    __shared__ float s_part[2][kT / 32];       // maxima of 16 tokens
    __shared__ Tokens s_tile;
    __shared__ int s_any;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // keys' CTAs first: they take longer
    const int x = static_cast<int>(blockIdx.x) - cut.k_ctas;
    const bool is_k = x < 0;
    const int chunks = is_k ? cut.k_chunks : cut.v_chunks;
    const int y = is_k ? static_cast<int>(blockIdx.x) : x;
    const int tile = y / chunks, chunk = is_k ? cut.k_chunk : cut.v_chunk;
    const int h0 = (y - tile * chunks) * chunk, h1 = min(h0 + chunk, p.k.heads);

    if (warp == 0) {
        Tokens t;
        const bool any = tile_tokens(p, tile, lane, t);
        if (lane == 0) {
            s_any = any;
            s_tile = t;
        }
    }
    __syncthreads();
    // A group of tokens below 0 or past the bound is stored nowhere.  (A length of up to
    // 2^32 - 1 may come; below the bound, tokens fit an int.)
    if (!s_any || s_tile.first < 0 || s_tile.first >= p.max_kv_len) {
        pdl_wait_primary();
        return;
    }
    const int first = static_cast<int>(s_tile.first), count = s_tile.count, r0 = s_tile.row;
    const int group0 = first & ~(kGroupTokens - 1), first_slot = first - group0;
    const int B = p.block_tokens;

    // ---- this thread's tokens and channels; the first head's loads -------------------
    const HeadRows &in = is_k ? p.k : p.v;
    const CacheOut &c = is_k ? p.kc : p.vc;
    const int item = tid / kL, i0 = tid & (kL - 1);
    const int R = p.rope.rot_dim / 8, half = is_k ? p.rope.rot_dim / 2 : 0;
    const int start = p.k.rot_start / 8;
    int va, vb;
    pair_of(kInter, 16, R, i0, va, vb);        // of 16 vectors no lane goes without
    const bool turn_a = half > 0 && va < R, turn_b = half > 0 && vb < R;
    const int ca = 8 * ordered(va, R, start), cb = 8 * ordered(vb, R, start);
    const bool norm_a = ca < in.norm_dim, norm_b = cb < in.norm_dim;
    uint4 ga = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), gb = ga;   // 1
    if (in.norm && norm_a) ga = *reinterpret_cast<const uint4 *>(in.norm + ca);
    if (in.norm && norm_b) gb = *reinterpret_cast<const uint4 *>(in.norm + cb);
    // Its four tokens lie in one page, side by side (pages have at least 8 slots); so
    // do the tokens that the first block holds from before.
    const int t0 = group0 + 4 * item, row0 = t0 - first;
    int page = -1, slot0 = t0;
    if (t0 + 3 >= (first & ~(B - 1)) && row0 < count && t0 < p.max_kv_len) {
        page = page_of(p, s_tile.b, t0);
        if (p.page_table) slot0 = t0 & (p.page_size - 1);
    }
    unsigned stored = 0;                       // new tokens, a bit each
#pragma unroll
    for (int s = 0; s < kS; ++s)
        if (page >= 0 && row0 + s >= 0 && row0 + s < count && t0 + s < p.max_kv_len)
            stored |= 1u << s;
    uint4 *ahead = reinterpret_cast<uint4 *>(angles + (half > 0 ? kGroupTokens * 4 * kL : 0)) + tid;
    const uint16_t *src = in.in + (r0 + row0) * in.in_row + h0 * in.in_head;
    const auto fetch = [&]() {
#pragma unroll
        for (int s = 0; s < kS; ++s)
            if (stored >> s & 1) {
                copy_16(ahead + 2 * s * kT, src + s * in.in_row + ca);
                copy_16(ahead + (2 * s + 1) * kT, src + s * in.in_row + cb);
            }
    };
#pragma unroll
    for (int s = 0; s < kS; ++s)
        if (!(stored >> s & 1))                // never fetched: 0, which no maximum sees
            ahead[2 * s * kT] = ahead[(2 * s + 1) * kT] = make_uint4(0u, 0u, 0u, 0u);
    fetch();

    // ---- the first block's old scales; angles, one entry a thread ---------------------
    int held = s_tile.first == s_tile.begin ? first & (B - 1) : 0;
    if (held > 0) {
        const int at = first < p.max_kv_len ? page_of(p, s_tile.b, first) : -1;
        if (at < 0) held = 0;                  // the first token is not stored
        const int slot = p.page_table ? first & (p.page_size - 1) : first;
        if (held > 0 && tid < h1 - h0)
            s_old[tid] = c.scale[at * c.scale_page + (slot >> p.block_shift) * c.scale_block +
                                 (h0 + tid) * c.scale_head];
    }
    if (half > 0)
        for (int e = tid; e < kGroupTokens * 4 * kL; e += kT) {
            const int row = e / (4 * kL) - first_slot;
            if (row < 0 || row >= count) continue;
            angles[e] = angle_entry<kInter>(p.rope, 16, e / kL & 3, e & (kL - 1),
                                            p.positions ? p.positions[r0 + row] : first + row);
        }
    __syncthreads();

#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
        float2 ya[kS][4], yb[kS][4];
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            unpack8(ahead[2 * s * kT], ya[s]);
            unpack8(ahead[(2 * s + 1) * kT], yb[s]);
        }
        if (in.norm_dim > 0) {
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                float2 sq = make_float2(0.f, 0.f);
                if (norm_a) add_squares(ya[s], sq);
                if (norm_b) add_squares(yb[s], sq);
                float sum = sq.x + sq.y;
#pragma unroll
                for (int o = 1; o < kL; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float inv = rsqrtf(fmaf(sum, in.mean, in.eps));
                if (norm_a) scale8(ya[s], ga, inv);
                if (norm_b) scale8(yb[s], gb, inv);
            }
        }
        if (turn_a) {
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
        src += in.in_head;
        if (h + 1 < h1) fetch();

        // ---- scales and codes ------------------------------------------------------------
        if (page < 0) continue;
        uint8_t *dst = c.base + page * c.page_stride + slot0 * c.token_stride + h * c.head_stride;
        float *scales = c.scale + page * c.scale_page + h * c.scale_head;
        float scale = 0.f, f = 0.f, ratio = 1.f;
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const int slot = 4 * item + s;
            if (s == 0 || B < 4) {                               // (four tokens share blocks of 4)
                scale = pow2i(scale_exponent(top[s]));
                ratio = 1.f;
                if (held > 0 && (slot ^ first_slot) < B) {       // the block of the first token
                    const float old = s_old[h - h0];
                    if (scale > old) ratio = old / scale; else scale = old;
                }
                f = __frcp_rn(scale);
            }
            uint8_t *at = dst + s * c.token_stride;
            if (stored >> s & 1) {
                if (i0 == 0 && ((slot & (B - 1)) == 0 || slot == first_slot))
                    scales[((slot0 + s) >> p.block_shift) * c.scale_block] = scale;
                store_codes(at + ca, at + cb, ya[s], yb[s], f, infinite >> s & 1);
            } else if (ratio != 1.f && slot < first_slot) {      // held from before
                uint2 *wa = reinterpret_cast<uint2 *>(at + ca);
                uint2 *wb = reinterpret_cast<uint2 *>(at + cb);
                const uint2 oa = *wa, ob = *wb;
                *wa = make_uint2(recode4(oa.x, ratio), recode4(oa.y, ratio));
                *wb = make_uint2(recode4(ob.x, ratio), recode4(ob.y, ratio));
            }
        }
    }
    pdl_wait_primary();
}

}  // namespace

cudaError_t launch_fp8_runs(const RowsParams &p, bool behind_queries, cudaStream_t stream) {
    // In units of a values' head: a keys' head costs about two, the angles of a tile
    // six, opening a tile one.  The cut with the least estimate is taken: the work of
    // a resident CTA, and half of a CTA of the last ones.  (24768 rows of 8 + 8 heads,
    // 8 keys' and 4 values' heads a CTA: 47.7 us; 8 and 2 47.8, 4 and 4 51.0, 4 and 8
    // 57.7.)
    constexpr int kWave = 2 * 152;
    const long long likely = p.num_rows / kGroupTokens + p.batch;
    const int heads = p.k.heads;
    const int angles = p.rope.rot_dim > 0 ? 6 : 0;
    RunCut cut;
    cut.k_chunk = cut.v_chunk = 1;
    long long least = 0;
    for (int ck = 1; ck <= heads && ck <= kMaxChunk; ++ck)
        for (int cv = 1; cv <= heads && cv <= kMaxChunk; ++cv) {
            const int nk = (heads + ck - 1) / ck, nv = (heads + cv - 1) / cv;
            const long long work = likely * (nk * (1 + angles) + nv + 3 * heads) / kWave;
            const long long most = max(1 + angles + 2 * ck, 1 + cv);
            const long long cost = 2 * max(work, most) + 1 + cv;
            if ((ck == 1 && cv == 1) || cost < least) {
                least = cost;
                cut.k_chunk = ck;
                cut.v_chunk = cv;
            }
        }
    cut.k_chunks = (heads + cut.k_chunk - 1) / cut.k_chunk;
    cut.v_chunks = (heads + cut.v_chunk - 1) / cut.v_chunk;
    const long long tiles = fp8_tile_count(p), blocks = tiles * (cut.k_chunks + cut.v_chunks);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cut.k_ctas = static_cast<int>(tiles * cut.k_chunks);
    auto kern = p.rope.interleaved ? append_fp8_runs_kernel<true> : append_fp8_runs_kernel<false>;
    const size_t smem = run_smem(p);
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // Behind the queries' launch, which it does not depend on: CTAs start as that
    // one's last ones leave, and wait for its end before they leave themselves.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind_queries ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p, cut);
}

}  // namespace attn
