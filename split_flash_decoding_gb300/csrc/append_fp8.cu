// append_fp8.cu -- keys and values of new tokens into a cache held in 8 bits,
// shapes that the tile kernel does not take: blocks of more than 128 tokens and
// rotations whose pairs do not fall on whole 16-byte vectors.
//
// One CTA per (row, KV head, K or V); the CTA of a block's first new row does
// the block: the new tokens' largest value gives the scale, codes already held
// are rounded to a scale that grew, and the new tokens are encoded.
#include <cuda_fp8.h>
#include <float.h>

#include "head_tiles.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kD = 128;
__device__ __forceinline__ uint8_t encode(float x) {
    if (!(fabsf(x) <= FLT_MAX)) x = __uint_as_float(0x7fffffffu);   // no infinity: NaN
    return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3));
}

__device__ __forceinline__ float decode(uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(__half(h));
}

__global__ void __launch_bounds__(kThreads)
append_fp8_kernel(const __grid_constant__ RowsParams p) {
    __shared__ float buf[kWarps][kD];
    __shared__ float top[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.x, h = blockIdx.y;
    const bool is_k = blockIdx.z == 0;
    const HeadRows &x = is_k ? p.k : p.v;
    const CacheOut &cache = is_k ? p.kc : p.vc;

    const RowPlace at = place_of_row(p, r, lane);
    const int b = at.b;
    if (b < 0) return;
    const uint32_t L = at.L;
    const long long t0 = static_cast<long long>(L) - at.n;   // token of the first row
    const long long tl = at.t;
    if (tl < 0 || tl >= p.max_kv_len) {
        if (L != 0 && threadIdx.x == 0) atomicOr(p.err, kErrBadLength);
        return;
    }
    const int t = static_cast<int>(tl);
    const int first = static_cast<int>(max(t0, 0LL));
    const int B = p.block_tokens;
    if (t != first && t % B) return;                      // not its block's first new row
    const int page = page_of(p, b, t);
    if (page < 0) return;
    const int slot = t % p.page_size;
    const int held = t == first ? t % B : 0;              // earlier tokens of the block
    const int count = static_cast<int>(
        min(min(static_cast<long long>(B - t % B), static_cast<long long>(L) - t),
            min(static_cast<long long>(p.max_kv_len) - t,
                static_cast<long long>(p.num_rows) - r)));
    uint8_t *dst = cache.base + page * cache.page_stride + h * cache.head_stride;
    float *scale = cache.scale + page * cache.scale_page + (slot / B) * cache.scale_block +
                   h * cache.scale_head;
    const bool rotate = is_k && p.rope.rot_dim > 0;
    float *y = buf[warp];

    float amax = 0.f;
    for (int i = warp; i < count; i += kWarps) {
        load_head(p, x, r + i, h, p.positions ? p.positions[r + i] : t + i, rotate, y, lane);
        for (int c = lane; c < kD; c += 32) {
            const float a = fabsf(y[c]);
            if (a <= FLT_MAX) amax = fmaxf(amax, a);
        }
        __syncwarp();
    }
    amax = warp_max(amax);
    if (lane == 0) top[warp] = amax;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, top[w]);
    float s = tiles::pow2i(tiles::scale_exponent(amax));
    if (held) {
        const float old = *scale;
        if (s > old) {
            const float ratio = old / s;
            for (int i = warp; i < held; i += kWarps) {
                uint8_t *row = dst + (slot - held + i) * cache.token_stride;
                for (int c = lane; c < kD; c += 32) row[c] = encode(decode(row[c]) * ratio);
            }
        } else {
            s = old;
        }
    }
    __syncthreads();   // every thread has read the old scale
    if (threadIdx.x == 0) *scale = s;
    const float inv = 1.f / s;
    for (int i = warp; i < count; i += kWarps) {
        load_head(p, x, r + i, h, p.positions ? p.positions[r + i] : t + i, rotate, y, lane);
        uint8_t *row = dst + (slot + i) * cache.token_stride;
        for (int c = lane; c < kD; c += 32) row[c] = encode(y[c] * inv);
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_append_fp8(const RowsParams &p, cudaStream_t stream) {
    const bool small_blocks = p.block_tokens <= tiles::kGroupTokens;
    if (small_blocks && fp8_tiles_take_queries(p)) return launch_fp8_tiles(p, false, stream);
    RowsParams kv = p;
    if (p.q.heads > 0) {
        RowsParams q = p;
        q.k.heads = q.v.heads = 0;
        const cudaError_t e = launch_head_rows(q, stream);
        if (e != cudaSuccess) return e;
        kv.q.heads = 0;
    }
    if (small_blocks && head_tiles_fit(kv)) return launch_fp8_tiles(kv, p.q.heads > 0, stream);
    append_fp8_kernel<<<dim3(p.num_rows, p.k.heads, 2), kThreads, 0, stream>>>(kv);
    return cudaGetLastError();
}

}  // namespace attn
