// head_tiles_rows.cu -- the tile kernel's results to rows of memory and to slots
// of a bf16 cache.
#include "head_tiles.cuh"

namespace attn {

using namespace tiles;

// Whether a rotation's pairs of channels fall into the lanes' pairs of vectors.
static bool rotates_on_vectors(const RopeParams &rope, const HeadRows &x) {
    if (x.heads == 0 || rope.rot_dim == 0) return true;
    return rope.rot_dim % (rope.interleaved ? 8 : 16) == 0;
}

bool head_tiles_fit(const RowsParams &p) {
    const HeadRows *seg[3] = {&p.q, &p.k, &p.v};
    for (const HeadRows *x : seg)
        if (x->heads > 0 && x->dim > 256) return false;
    // one table of angles for q and k
    if (p.rope.rot_dim > 0 && p.q.heads > 0 && p.k.heads > 0 && p.q.dim != p.k.dim) return false;
    return rotates_on_vectors(p.rope, p.q) && rotates_on_vectors(p.rope, p.k);
}

namespace {

template <int L, int S>
cudaError_t launch_shape(const RowsParams &p, int tile_rows, int chunk_heads, cudaStream_t stream) {
    Cut cut;
    cut.heads = p.q.heads + p.k.heads + p.v.heads;
    cut.any_norm = (p.q.heads > 0 && p.q.norm_dim > 0) || (p.k.heads > 0 && p.k.norm_dim > 0);
    cut.tile_rows = tile_rows;
    cut.chunk_heads = chunk_heads;
    cut.chunks = (cut.heads + chunk_heads - 1) / chunk_heads;
    const long long tiles = (static_cast<long long>(p.num_rows) + tile_rows - 1) / tile_rows;
    return p.rope.interleaved ? launch<L, S, true, false>(p, cut, tiles, stream)
                              : launch<L, S, false, false>(p, cut, tiles, stream);
}

template <int L>
cudaError_t launch_lanes(const RowsParams &p, cudaStream_t stream) {
    const int heads = p.q.heads + p.k.heads + p.v.heads;
    constexpr int kWave = 2 * 152;                 // CTAs of a wave
    const long long items = static_cast<long long>(p.num_rows) * heads;
    if (items < static_cast<long long>(kWave) * (kThreads / L) * 4) {
        // few rows: small tiles, so that the angles take no time, one step a CTA
        int rows = 8;
        while (rows > 1 && rows / 2 >= p.num_rows) rows /= 2;
        return launch_shape<L, 1>(p, rows, Shape<L, 1>::kItems / rows, stream);
    }
    // Many: the angles of a tile serve up to 16 heads a CTA, fewer where the tiles
    // would not fill the GPU.
    constexpr int rows = Shape<L, 4>::kMaxRows;
    const long long tiles = (p.num_rows + rows - 1) / rows;
    long long chunk = heads * tiles / kWave;
    if (chunk > 16) chunk = 16;
    if (chunk < 1) chunk = 1;
    return launch_shape<L, 4>(p, rows, static_cast<int>(chunk), stream);
}

}  // namespace

cudaError_t launch_head_tiles(const RowsParams &p, cudaStream_t stream) {
    int dim = 0;
    const HeadRows *seg[3] = {&p.q, &p.k, &p.v};
    for (const HeadRows *x : seg)
        if (x->heads > 0 && x->dim > dim) dim = x->dim;
    if (dim <= 64) return launch_lanes<4>(p, stream);
    if (dim <= 128) return launch_lanes<8>(p, stream);
    return launch_lanes<16>(p, stream);
}

}  // namespace attn
