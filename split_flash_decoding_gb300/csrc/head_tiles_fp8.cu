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

constexpr int kShortRun = Shape<8, 1, 256>::kMaxRows;

int longest_run(const RowsParams &p) { return p.q_row_offsets ? p.max_q_len : 1; }

}  // namespace

// Queries join the keys' and values' launch when their heads have as many lanes
// and the runs are short; the row tiles are better at long ones (a row's heads
// side by side).
bool fp8_tiles_take_queries(const RowsParams &p) {
    return p.q.dim <= 128 && longest_run(p) <= kShortRun && head_tiles_fit(p);
}

cudaError_t launch_fp8_tiles(const RowsParams &p, cudaStream_t stream) {
    const int longest = longest_run(p);
    if (longest <= kShortRun) {
        int rows = 1;
        while (rows < longest) rows *= 2;
        const int now = Shape<8, 1, 256>::kItems / rows;              // heads at once
        return launch_steps<1, 256>(p, rows, now, stream);
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
    return launch_steps<4, 256>(p, kGroupTokens, best, stream);
}

}  // namespace attn
