// head_rows.cu -- norm and rotation of query and key heads, stored to rows
// (attn_qk_norm_rope) or, keys and values, to their slots of a bf16 cache
// (attn_append_kv).
//
// Heads of up to 256 channels take the tile kernel (head_tiles.cuh).  The kernel
// here is for longer ones (latent rows), and for q and k of unequal dims, which have
// no table of angles in common.
//
// Bound by memory (each channel read and written once) or, for a few rows, by
// latency.  A head vector is split over the lanes of a warp, 8 channels (16
// bytes) a lane and up to four such vectors for dims above 256; smaller dims put
// several heads side by side.  A warp takes one row, or a part of its heads when
// there are few rows, and nothing is shared between warps: it looks its row's
// place up, computes the cos and sin of its lanes' channels once, and then walks
// the heads with the next ones' loads in flight.  Sums of squares and the
// partners of the half layout travel by shuffles.  The loop is rolled: the code
// stays small enough that a call for a few rows does not wait for instructions.
// 47 rows of 128 heads of 576 channels (14 MB) take 6.1 us.
#include "head_rows.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

// One row's heads as a list of steps, a step being what a warp does at a time:
// 32 >> shift heads of q, then of k, then of v.
struct Steps {
    int shift[3];                  // log2 of the lanes of a head
    int first[4];                  // first step of q, k, v; their count
    int per_warp;                  // steps of a warp
    int chunks;                    // warps of a row
};

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x);
    x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z);
    x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}

// Step `step` of a row: its kind (0 q, 1 k, 2 v), and the lane's head and vector.
struct Part {
    int kind, shift, head, vec;
};

__device__ __forceinline__ Part part_of(const Steps &st, int step, int lane) {
    Part x;
    x.kind = step < st.first[1] ? 0 : step < st.first[2] ? 1 : 2;
    x.shift = st.shift[x.kind];
    x.head = ((step - st.first[x.kind]) << (5 - x.shift)) + (lane >> x.shift);
    x.vec = lane & ((1 << x.shift) - 1);
    return x;
}

// V: 16-byte vectors of a lane (2 and more: dims above 256, a head per warp).
template <int V>
__device__ __forceinline__ void load_part(const RowsParams &p, const Steps &st, int step, int r,
                                          int lane, uint4 (&raw)[V]) {
    const Part at = part_of(st, step, lane);
    const HeadRows &x = at.kind == 0 ? p.q : at.kind == 1 ? p.k : p.v;
    const uint16_t *src = x.in + r * x.in_row + at.head * x.in_head + at.vec * 8;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        raw[v] = make_uint4(0u, 0u, 0u, 0u);
        if (at.head < x.heads && (at.vec + 32 * v) * 8 < x.dim)
            raw[v] = *reinterpret_cast<const uint4 *>(src + 256 * v);
    }
}

template <int V>
__global__ void __launch_bounds__(kThreads)
head_rows_kernel(const __grid_constant__ RowsParams p, const __grid_constant__ Steps st) {
    const int lane = threadIdx.x & 31;
    const long long id = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int r = static_cast<int>(id / st.chunks);
    const int s0 = static_cast<int>(id - static_cast<long long>(r) * st.chunks) * st.per_warp;
    const int s1 = min(s0 + st.per_warp, st.first[3]);
    if (r >= p.num_rows || s0 >= s1) return;

    uint4 next[V];
    load_part<V>(p, st, s0, r, lane, next);

    // ---- the row's place ------------------------------------------------------
    int pos = 0, page = -1, slot = 0;              // page -1: not stored
    if (p.kv_len) {
        const RowPlace at = place_of_row(p, r, lane);
        if (at.b < 0) return;
        const bool fits = at.t >= 0 && at.t < p.max_kv_len;
        if (!fits && at.L != 0 && lane == 0) atomicOr(p.err, kErrBadLength);
        pos = static_cast<int>(max(at.t, 0LL));
        if (fits && s1 > st.first[1]) {
            page = page_of(p, at.b, pos);
            slot = p.page_table ? pos & (p.page_size - 1) : pos;
        }
    }
    if (p.positions) pos = p.positions[r];

    // ---- cos and sin of the lane's eight channels -------------------------------
    // y' = C y + S z, z the pair's other channel.  The rotated channels lie in one
    // of the V vectors of each lane; q and k may have them in different places.
    const int half = p.rope.rot_dim / 2;
    float cs[8], sn[8];
    int angles_of = -1;                            // the lane's first rotated channel

#pragma unroll 1
    for (int step = s0; step < s1; ++step) {
        uint4 raw[V];
#pragma unroll
        for (int v = 0; v < V; ++v) raw[v] = next[v];
        if (step + 1 < s1) load_part<V>(p, st, step + 1, r, lane, next);

        const Part at = part_of(st, step, lane);
        const HeadRows &x = at.kind == 0 ? p.q : at.kind == 1 ? p.k : p.v;
        uint16_t *dst;
        if (x.out) {
            dst = x.out + r * x.out_row + at.head * x.out_head;
        } else {
            if (page < 0) continue;
            const CacheOut &c = at.kind == 1 ? p.kc : p.vc;
            dst = reinterpret_cast<uint16_t *>(c.base) + page * c.page_stride +
                  slot * c.token_stride + at.head * c.head_stride;
        }
        const bool rotate = at.kind < 2 && half > 0;
        const int v_rot = V == 1 ? 0 : x.rot_start >> 8;         // the vector that is rotated
        const int rot = (at.vec + 32 * v_rot) * 8 - x.rot_start;
        const bool turns = rotate && rot >= 0 && rot < p.rope.rot_dim;
        if (turns && rot != angles_of) {
            angles_of = rot;
            if (p.rope.interleaved) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    rope_cos_sin(p.rope, rot / 2 + k, pos, cs[2 * k], sn[2 * k + 1]);
                    cs[2 * k + 1] = cs[2 * k];
                    sn[2 * k] = -sn[2 * k + 1];
                }
            } else {
                const bool low = rot < half;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    rope_cos_sin(p.rope, (low ? rot : rot - half) + k, pos, cs[k], sn[k]);
                    if (low) sn[k] = -sn[k];
                }
            }
        }
        float inv = 0.f;
        if (x.norm_dim > 0) {
            float sq = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if ((at.vec + 32 * v) * 8 < x.norm_dim) {
                    float y[8];
                    unpack8(raw[v], y);
#pragma unroll
                    for (int c = 0; c < 8; ++c) sq = fmaf(y[c], y[c], sq);
                }
#pragma unroll 1
            for (int o = 1; o < (1 << at.shift); o <<= 1)
                sq += __shfl_xor_sync(0xffffffffu, sq, o);
            inv = rsqrtf(sq / static_cast<float>(x.norm_dim) + x.eps);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c0 = (at.vec + 32 * v) * 8;                // the lane's first channel
            uint4 w = raw[v];
            const bool normed = c0 < x.norm_dim;
            const bool rotated = rotate && v == v_rot;           // uniform over the warp
            if (normed || rotated) {
                float y[8];
                unpack8(w, y);
                if (normed) {
                    if (x.norm) {
                        float g[8];
                        unpack8(*reinterpret_cast<const uint4 *>(x.norm + c0), g);
#pragma unroll
                        for (int c = 0; c < 8; ++c) y[c] *= inv * g[c];
                    } else {
#pragma unroll
                        for (int c = 0; c < 8; ++c) y[c] *= inv;
                    }
                }
                w.x = pack_bf16x2(y[0], y[1]);
                w.y = pack_bf16x2(y[2], y[3]);
                w.z = pack_bf16x2(y[4], y[5]);
                w.w = pack_bf16x2(y[6], y[7]);
                if (rotated) {
                    __syncwarp();
                    float z[8];
                    if (p.rope.interleaved) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) z[c] = y[c ^ 1];
                    } else {
                        // the partner is half / 8 lanes up or down
                        const int partner =
                            turns ? lane + (rot < half ? half / 8 : -(half / 8)) : lane;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            z[c] = __shfl_sync(0xffffffffu, y[c], partner);
                    }
                    if (turns) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) y[c] = fmaf(y[c], cs[c], z[c] * sn[c]);
                        w.x = pack_bf16x2(y[0], y[1]);
                        w.y = pack_bf16x2(y[2], y[3]);
                        w.z = pack_bf16x2(y[4], y[5]);
                        w.w = pack_bf16x2(y[6], y[7]);
                    }
                }
            }
            if (at.head < x.heads && c0 < x.dim) *reinterpret_cast<uint4 *>(dst + c0) = w;
        }
    }
}

// Any shape: one warp per (row, head), the vector in shared memory.  Rotations
// whose pairs do not fall on whole 16-byte vectors come here.
constexpr int kAnyWarps = 4;
constexpr int kMaxDim = 1024;

__global__ void __launch_bounds__(kAnyWarps * 32)
head_rows_any_kernel(const __grid_constant__ RowsParams p) {
    __shared__ float buf[kAnyWarps][kMaxDim];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = p.q.heads + p.k.heads + p.v.heads;
    const long long item = static_cast<long long>(blockIdx.x) * kAnyWarps + warp;
    if (item >= static_cast<long long>(p.num_rows) * heads) return;
    const int r = static_cast<int>(item / heads);
    int h = static_cast<int>(item - static_cast<long long>(r) * heads);
    const int kind = h < p.q.heads ? 0 : h < p.q.heads + p.k.heads ? 1 : 2;   // q, k, v
    const HeadRows &x = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    h -= kind == 0 ? 0 : kind == 1 ? p.q.heads : p.q.heads + p.k.heads;

    uint16_t *dst = x.out ? x.out + r * x.out_row + h * x.out_head : nullptr;
    int pos = 0;
    if (p.kv_len) {
        const RowPlace at = place_of_row(p, r, lane);
        if (at.b < 0) return;
        pos = static_cast<int>(max(at.t, 0LL));
        if (kind > 0) {
            if (at.t < 0 || at.t >= p.max_kv_len) {
                if (at.L != 0 && lane == 0) atomicOr(p.err, kErrBadLength);
                return;
            }
            const int page = page_of(p, at.b, pos);
            if (page < 0) return;
            const CacheOut &c = kind == 1 ? p.kc : p.vc;
            dst = reinterpret_cast<uint16_t *>(c.base) + page * c.page_stride +
                  (p.page_table ? pos % p.page_size : pos) * c.token_stride + h * c.head_stride;
        }
    }
    if (p.positions) pos = p.positions[r];
    float *y = buf[warp];
    load_head(p, x, r, h, pos, kind < 2 && p.rope.rot_dim > 0, y, lane);
    for (int c = lane; c < x.dim; c += 32)
        dst[c] = static_cast<uint16_t>(pack_bf16x2(y[c], 0.f) & 0xffffu);
}

// Whether a rotation's pairs are whole 16-byte vectors that one shuffle reaches.
bool on_vectors(const RopeParams &rope, const HeadRows &x) {
    if (x.heads == 0 || rope.rot_dim == 0) return true;
    const int first = x.rot_start / 8, last = (x.rot_start + rope.rot_dim - 1) / 8;
    return rope.rot_dim % (rope.interleaved ? 8 : 16) == 0 && first / 32 == last / 32;
}

template <int V>
cudaError_t launch_v(const RowsParams &p, const Steps &st, cudaStream_t stream) {
    const long long blocks =
        (static_cast<long long>(p.num_rows) * st.chunks + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    head_rows_kernel<V><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p, st);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_head_rows(const RowsParams &p, cudaStream_t stream) {
    const long long heads = p.q.heads + p.k.heads + p.v.heads;
    if (p.num_rows == 0 || heads == 0) return cudaSuccess;
    if (head_tiles_fit(p)) return launch_head_tiles(p, stream);
    if (!on_vectors(p.rope, p.q) || !on_vectors(p.rope, p.k)) {
        const long long blocks = (p.num_rows * heads + kAnyWarps - 1) / kAnyWarps;
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        head_rows_any_kernel<<<static_cast<unsigned>(blocks), kAnyWarps * 32, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const HeadRows *seg[3] = {&p.q, &p.k, &p.v};
    Steps st;
    int vectors = 1;
    st.first[3] = 0;
    for (int k = 0; k < 3; ++k) {
        const int vecs = (seg[k]->dim + 7) / 8;
        st.shift[k] = 3;
        while (st.shift[k] < 5 && (1 << st.shift[k]) < vecs) ++st.shift[k];
        if (seg[k]->heads > 0 && (vecs + 31) / 32 > vectors) vectors = (vecs + 31) / 32;
        st.first[k] = st.first[3];
        const int per = 32 >> st.shift[k];
        st.first[3] += (seg[k]->heads + per - 1) / per;
    }
    // A warp a row once the rows fill the GPU's warps; fewer heads a warp below
    // that.  (The angles cost about as much as three steps.)
    constexpr long long kFill = 152 * 32;
    long long chunks = (kFill + p.num_rows - 1) / p.num_rows;
    if (chunks > st.first[3]) chunks = st.first[3];
    st.per_warp = static_cast<int>((st.first[3] + chunks - 1) / chunks);
    st.chunks = (st.first[3] + st.per_warp - 1) / st.per_warp;
    switch (vectors) {
        case 1: return launch_v<1>(p, st, stream);
        case 2: return launch_v<2>(p, st, stream);
        case 3: return launch_v<3>(p, st, stream);
        default: return launch_v<4>(p, st, stream);
    }
}

}  // namespace attn
