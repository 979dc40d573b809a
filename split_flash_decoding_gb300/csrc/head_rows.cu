// head_rows.cu -- norm and rotation of query and key heads, stored to rows
// (attn_qk_norm_rope) or, keys and values, to their slots of a bf16 cache
// (attn_append_kv).
//
// One warp per (row, head): the head vector goes through shared memory in
// fp32, so that any rotation layout finds its pairs.
#include "head_rows.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxDim = 1024;

__global__ void __launch_bounds__(kWarps * 32)
head_rows_kernel(const __grid_constant__ RowsParams p) {
    __shared__ float buf[kWarps][kMaxDim];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = p.q.heads + p.k.heads + p.v.heads;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
    if (item >= static_cast<long long>(p.num_rows) * heads) return;
    const int r = static_cast<int>(item / heads);
    int h = static_cast<int>(item - static_cast<long long>(r) * heads);
    const int kind = h < p.q.heads ? 0 : h < p.q.heads + p.k.heads ? 1 : 2;   // q, k, v
    const HeadRows &x = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    h -= kind == 0 ? 0 : kind == 1 ? p.q.heads : p.q.heads + p.k.heads;

    uint16_t *dst = x.out ? x.out + r * x.out_row + h * x.out_head : nullptr;
    int pos = 0;
    if (p.kv_len) {
        const int b = sequence_of_row(p, r);
        if (b < 0) return;
        const int row0 = p.q_row_offsets ? static_cast<int>(p.q_row_offsets[b]) : r;
        const int n = p.q_row_offsets ? static_cast<int>(p.q_row_offsets[b + 1]) - row0 : 1;
        const uint32_t L = p.kv_len[b];
        const long long t = static_cast<long long>(L) - n + (r - row0);
        pos = static_cast<int>(max(t, 0LL));
        if (kind > 0) {
            if (t < 0 || t >= p.max_kv_len) {
                if (L != 0 && lane == 0) atomicOr(p.err, kErrBadLength);
                return;
            }
            const int page = page_of(p, b, pos);
            if (page < 0) return;
            const CacheOut &c = kind == 1 ? p.kc : p.vc;
            dst = reinterpret_cast<uint16_t *>(c.base) + page * c.page_stride +
                  (pos % p.page_size) * c.token_stride + h * c.head_stride;
        }
    }
    if (p.positions) pos = p.positions[r];

    const uint16_t *src = x.in + r * x.in_row + h * x.in_head;
    float *y = buf[warp];
    float sq = 0.f;
    for (int c = lane; c < x.dim; c += 32) {
        const float v = bf16_lo(src[c]);
        y[c] = v;
        if (c < x.norm_dim) sq += v * v;
    }
    __syncwarp();
    if (x.norm_dim > 0) {
        const float inv = rsqrtf(warp_sum(sq) / static_cast<float>(x.norm_dim) + x.eps);
        for (int c = lane; c < x.norm_dim; c += 32)
            y[c] *= inv * (x.norm ? bf16_lo(x.norm[c]) : 1.f);
        __syncwarp();
    }
    if (kind < 2 && p.rope.rot_dim > 0) {
        const int half = p.rope.rot_dim / 2;
        for (int i = lane; i < half; i += 32) {
            const int a = x.rot_start + (p.rope.interleaved ? 2 * i : i);
            const int b = a + (p.rope.interleaved ? 1 : half);
            float c, s;
            rope_cos_sin(p.rope, i, pos, c, s);
            const float ya = y[a], yb = y[b];
            y[a] = ya * c - yb * s;
            y[b] = yb * c + ya * s;
        }
        __syncwarp();
    }
    for (int c = lane; c < x.dim; c += 32)
        dst[c] = static_cast<uint16_t>(pack_bf16x2(y[c], 0.f) & 0xffffu);
}

}  // namespace

cudaError_t launch_head_rows(const RowsParams &p, cudaStream_t stream) {
    const long long heads = p.q.heads + p.k.heads + p.v.heads;
    const long long blocks = (p.num_rows * heads + kWarps - 1) / kWarps;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    head_rows_kernel<<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace attn
