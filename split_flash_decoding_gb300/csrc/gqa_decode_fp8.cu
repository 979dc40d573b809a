// gqa_decode_fp8.cu -- decode attention over a cache held in 8 bits.
//
// One CTA per (query row, query head): warps take keys in turn with a running
// maximum and sum, joined at the end.
#include <cuda_fp8.h>

#include "cache_ops.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float4 decode4(uint32_t w) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(w & 0xffffu, __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(w >> 16, __NV_E4M3);
    const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
    return make_float4(x.x, x.y, y.x, y.y);
}

__global__ void __launch_bounds__(kWarps * 32)
gqa_decode_fp8_kernel(const __grid_constant__ Fp8DecodeParams p) {
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x, h = blockIdx.y, kvh = h / p.group;
    int b = row, row0 = row, n = 1;
    if (p.q_row_offsets) {
        if (row >= static_cast<int>(p.q_row_offsets[p.batch])) return;
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (static_cast<int>(p.q_row_offsets[mid]) <= row) lo = mid; else hi = mid;
        }
        b = lo;
        row0 = p.q_row_offsets[b];
        n = p.q_row_offsets[b + 1] - row0;
    }
    const uint32_t cap = p.num_partitions;   // max_kv_len
    if (p.kv_len[b] > cap && threadIdx.x == 0) atomicOr(p.err, kErrBadLength);
    const int L = static_cast<int>(min(p.kv_len[b], cap));
    const int lim = p.causal ? min(L, L - n + (row - row0) + 1) : L;
    const uint16_t *q = p.q + (static_cast<size_t>(row) * p.num_q_heads + h) * 128;
    float4 qv;
    qv.x = bf16_lo(q[4 * lane]);
    qv.y = bf16_lo(q[4 * lane + 1]);
    qv.z = bf16_lo(q[4 * lane + 2]);
    qv.w = bf16_lo(q[4 * lane + 3]);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t = warp; t < lim; t += kWarps) {
        int page = b;
        if (p.page_table) {
            page = p.page_table[static_cast<size_t>(b) * p.max_pages + t / p.page_size];
            if (page < 0 || page >= p.num_pages) {
                if (lane == 0) atomicOr(p.err, kErrBadPage);
                continue;
            }
        }
        const int slot = t % p.page_size;
        const long long blk = slot >> p.block_shift;
        const float4 kx = decode4(*reinterpret_cast<const uint32_t *>(
            p.k_base + page * p.k_page + slot * p.k_token + kvh * p.k_head + 4 * lane));
        const float4 vx = decode4(*reinterpret_cast<const uint32_t *>(
            p.v_base + page * p.v_page + slot * p.v_token + kvh * p.v_head + 4 * lane));
        const float ks = p.k_scale[page * p.ks_page + blk * p.ks_block + kvh * p.ks_head];
        const float vs = p.v_scale[page * p.vs_page + blk * p.vs_block + kvh * p.vs_head];
        const float s = warp_sum(qv.x * kx.x + qv.y * kx.y + qv.z * kx.z + qv.w * kx.w) * ks *
                        p.qk_scale_log2;
        const float mn = fmaxf(m, s);
        const float a = mn == -INFINITY ? 1.f : exp2f(m - mn);
        const float w = mn == -INFINITY ? 0.f : exp2f(s - mn);
        m = mn;
        l = l * a + w;
        o.x = o.x * a + w * (vs * vx.x);
        o.y = o.y * a + w * (vs * vx.y);
        o.z = o.z * a + w * (vs * vx.z);
        o.w = o.w * a + w * (vs * vx.w);
    }
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
    *reinterpret_cast<float4 *>(&so[warp][4 * lane]) = o;
    __syncthreads();
    if (threadIdx.x >= 128) return;
    const int ch = threadIdx.x;
    const float t2 = p.sink ? p.sink[h] * kLog2e : -INFINITY;
    float M = t2;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    float Z = 0.f, acc = 0.f;
    if (M != -INFINITY) {
        Z = exp2f(t2 - M);
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(sm[w] - M);
            Z += f * sl[w];
            acc += f * so[w][ch];
        }
    }
    const size_t at = static_cast<size_t>(row) * p.num_q_heads + h;
    p.out[at * 128 + ch] = static_cast<uint16_t>(pack_bf16x2(Z == 0.f ? 0.f : acc / Z, 0.f));
    if (ch == 0 && p.lse) p.lse[at] = Z == 0.f ? -INFINITY : (M + log2f(Z)) * kLn2;
}

}  // namespace

int fp8_decode_ctas(int num_sms) { return num_sms; }

cudaError_t launch_gqa_decode_fp8(const Fp8DecodeParams &p, int, cudaStream_t stream) {
    gqa_decode_fp8_kernel<<<dim3(p.num_q_rows, p.num_q_heads), kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace attn
