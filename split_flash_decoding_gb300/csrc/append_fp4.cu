// append_fp4.cu -- keys and values of new tokens into a cache held in 4 bits, queries
// normed and rotated on the way (attn_append_kv_fp4).
//
// Every token's codes depend on that token alone, so this is the bf16 append with
// another end: the tile kernel (head_tiles.cuh) takes the rows, and the lanes of a head
// join their largest values before they store.  Prompts are bound by issue slots (72% in
// use: conversions, scales and rotation of vectors that are there already; 24,768 rows of
// 32 + 8 heads, keys normed, 121 us, 5.2 TB/s), 64 rows by latency (3.8 us).  Rotations
// whose pairs do not fall on whole 16-byte vectors have the kernel here, one warp a row and
// head, with the same roundings.
#include "head_tiles.cuh"

namespace attn {
namespace {

constexpr int kD = 128;
constexpr int kWarps = 4;

// Lane l has channels 4 l to 4 l + 3: eight lanes are a group of 32.
__global__ void __launch_bounds__(kWarps * 32)
append_fp4_kernel(const __grid_constant__ RowsParams p) {
    __shared__ float buf[kWarps][kD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = p.k.heads + p.v.heads;
    const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
    if (item >= static_cast<long long>(p.num_rows) * heads) return;
    const int r = static_cast<int>(item / heads);
    int h = static_cast<int>(item - static_cast<long long>(r) * heads);
    const bool is_k = h < p.k.heads;
    if (!is_k) h -= p.k.heads;
    const HeadRows &x = is_k ? p.k : p.v;
    const CacheOut &c = is_k ? p.kc : p.vc;
    const RowPlace at = place_of_row(p, r, lane);
    if (at.b < 0) return;
    int pos = static_cast<int>(max(at.t, 0LL)), page = -1, slot = 0;
    if (at.t < 0 || at.t >= p.max_kv_len) {
        if (at.L != 0 && lane == 0) atomicOr(p.err, kErrBadLength);
    } else {
        page = page_of(p, at.b, pos);
        slot = p.page_table ? pos & (p.page_size - 1) : pos;
    }
    if (p.positions) pos = p.positions[r];
    float *y = buf[warp];
    load_head<true>(p, x, r, h, pos, is_k && p.rope.rot_dim > 0, y, lane);
    __syncwarp();
    const float4 v = *reinterpret_cast<const float4 *>(y + 4 * lane);
    uint32_t top = max(max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))),
                       max(__float_as_uint(fabsf(v.z)), __float_as_uint(fabsf(v.w))));
    for (int o = 1; o < (is_k ? 8 : 32); o <<= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool whole = top < 0x7f800000u;
    const int e = tiles::fp4_exponent(top);
    const float f = tiles::pow2i(-e);
    const float s = whole ? tiles::pow2i(e) : __uint_as_float(0x7fffffffu);
    const float2 z[4] = {make_float2(v.x * f, v.y * f), make_float2(v.z * f, v.w * f),
                         make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const uint32_t word = whole ? tiles::to_fp4x8(z) : 0u;
    if (page >= 0) {
        *reinterpret_cast<uint16_t *>(c.base + page * c.page_stride + slot * c.token_stride +
                                      h * c.head_stride + 2 * lane) = static_cast<uint16_t>(word);
        float *scale = c.scale + page * c.scale_page + slot * c.scale_block + h * c.scale_head;
        if (!is_k) {
            if (lane == 0) *scale = s;
        } else if ((lane & 7) == 0) {
            reinterpret_cast<uint8_t *>(scale)[lane >> 3] = whole ? uint8_t(e + 127) : 255;
        }
    }
    if (x.out) {
        const uint4 n = tiles::from_fp4x8(word, s);
        *reinterpret_cast<uint2 *>(x.out + r * x.out_row + h * x.out_head + 4 * lane) =
            make_uint2(n.x, n.y);
    }
}

// Whether four lanes side by side hold a whole group of 32 channels (four vectors) of a key in
// their first vectors, and one in their second.
bool lanes_hold_groups(const RowsParams &p) {
    const int turning = p.rope.rot_dim / 8, start = p.k.rot_start / 8;
    for (int i = 0; i < 8; ++i) {
        int a, b, a0, b0;
        tiles::pair_of(p.rope.interleaved != 0, kD / 8, turning, i, a, b);
        tiles::pair_of(p.rope.interleaved != 0, kD / 8, turning, i & ~3, a0, b0);
        if (tiles::ordered(a, turning, start) / 4 != tiles::ordered(a0, turning, start) / 4 ||
            tiles::ordered(b, turning, start) / 4 != tiles::ordered(b0, turning, start) / 4)
            return false;
    }
    return true;
}

}  // namespace

cudaError_t launch_append_fp4(const RowsParams &p, cudaStream_t stream) {
    RowsParams kv = p;
    if (p.q.heads > 0 && (p.q.dim > kD || !head_tiles_fit(p))) {
        RowsParams q = p;
        q.k.heads = q.v.heads = 0;
        const cudaError_t e = launch_head_rows(q, stream);
        if (e != cudaSuccess) return e;
        kv.q.heads = 0;
    }
    if (head_tiles_fit(kv))
        return tiles::launch_lanes<8, tiles::kFp4>(kv, stream, lanes_hold_groups(kv));
    const long long items = static_cast<long long>(p.num_rows) * (p.k.heads + p.v.heads);
    const long long blocks = (items + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    append_fp4_kernel<<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(kv);
    return cudaGetLastError();
}

}  // namespace attn
