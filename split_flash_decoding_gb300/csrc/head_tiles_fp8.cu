// head_tiles_fp8.cu -- the tile kernel's keys and values to slots of a cache held
// in 8 bits, queries to rows on the way (attn_append_kv_fp8): runs of up to 32 new
// tokens.
#include "head_tiles.cuh"

namespace attn {

using namespace tiles;

static int longest_run(const RowsParams &p) { return p.q_row_offsets ? p.max_q_len : 1; }

// Queries join the keys' and values' launch when their heads have as many lanes
// and the runs are short; the row tiles are better at long ones (a row's heads
// side by side).
bool fp8_tiles_take_queries(const RowsParams &p) {
    return p.q.dim <= 128 && longest_run(p) <= kItemsOf<8> && head_tiles_fit(p);
}

cudaError_t launch_fp8_tiles(const RowsParams &p, bool behind_queries, cudaStream_t stream) {
    const int longest = longest_run(p);
    if (longest > kItemsOf<8>) return launch_fp8_runs(p, behind_queries, stream);
    Cut cut;
    cut.heads = p.q.heads + p.k.heads + p.v.heads;
    cut.any_norm = (p.q.heads > 0 && p.q.norm_dim > 0) || p.k.norm_dim > 0;
    cut.tile_rows = 1;
    while (cut.tile_rows < longest) cut.tile_rows *= 2;
    cut.chunk_heads = kItemsOf<8> / cut.tile_rows;               // heads at once
    cut.chunks = (cut.heads + cut.chunk_heads - 1) / cut.chunk_heads;
    return launch<8, true, false>(p, cut, fp8_tile_count(p), stream);
}

}  // namespace attn
