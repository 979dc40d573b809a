// head_tiles_fp8.cu -- the tile kernel's keys and values to slots of a cache held
// in 8 bits, queries to rows on the way (attn_append_kv_fp8).
#include "head_tiles.cuh"

namespace attn {

using namespace tiles;

namespace {

template <int S, int T>
cudaError_t launch_steps(const RowsParams &p, int tile_rows, int chunk_heads, cudaStream_t stream) {
    Cut cut;
    cut.heads = p.q.heads + p.k.heads + p.v.heads;
    cut.any_norm = (p.q.heads > 0 && p.q.norm_dim > 0) || p.k.norm_dim > 0;
    cut.tile_rows = tile_rows;
    cut.chunk_heads = chunk_heads;
    cut.chunks = (cut.heads + chunk_heads - 1) / chunk_heads;
    // a sequence of n rows meets at most (n - 1) / kGroupTokens + 2 groups
    long long tiles = p.num_rows;
    if (p.q_row_offsets) {
        const long long bound = p.num_rows / kGroupTokens + 2LL * p.batch;
        if (bound < tiles) tiles = bound;
    }
    return p.rope.interleaved ? launch<8, S, T, true, true>(p, cut, tiles, stream)
                              : launch<8, S, T, false, true>(p, cut, tiles, stream);
}

}  // namespace

cudaError_t launch_fp8_tiles(const RowsParams &p, cudaStream_t stream) {
    const int longest = p.q_row_offsets ? p.max_q_len : 1;
    if (longest <= Shape<8, 1, 256>::kMaxRows) {
        int rows = 1;
        while (rows < longest) rows *= 2;
        const int now = Shape<8, 1, 256>::kItems / rows;              // heads at once
        return launch_steps<1, 256>(p, rows, now, stream);
    }
    // Long runs: the queries go through the row tiles, which are better at them
    // (their heads side by side), in a launch of their own.
    RowsParams kv = p;
    if (p.q.heads > 0) {
        RowsParams q = p;
        q.k.heads = q.v.heads = 0;
        const cudaError_t e = launch_head_tiles(q, stream);
        if (e != cudaSuccess) return e;
        kv.q.heads = 0;
    }
    // A tile's angles cost about as much as two heads; as many heads to a CTA as
    // leave the waves full.
    constexpr int kWave = 2 * 152;
    const int heads = p.k.heads + p.v.heads;
    const long long tiles = p.num_rows / kGroupTokens + p.batch;
    int best = 1;
    long long least = 0;
    for (int chunk = 1; chunk <= heads; ++chunk) {
        const long long ctas = tiles * ((heads + chunk - 1) / chunk);
        const long long cost = (ctas + kWave - 1) / kWave * (chunk + 2);
        if (chunk == 1 || cost < least) {
            least = cost;
            best = chunk;
        }
    }
    return launch_steps<4, 256>(kv, kGroupTokens, best, stream);
}

}  // namespace attn
