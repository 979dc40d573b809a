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

template <int L>
cudaError_t launch_lanes(const RowsParams &p, cudaStream_t stream) {
    // Tiles of 8 rows: a step then reads 256 / L / 8 heads side by side of every row
    // (1 KB at 128 channels), and the angles of a tile are two a thread.  A CTA
    // takes all heads of its rows once the tiles fill the GPU, fewer below.
    // us for 24768 rows of 48 heads / 8191 of 40 with norm: 4 rows 136 / 40, 8 rows
    // 132 / 38, 16 rows 135 / 53, 32 rows and 16 heads 135 / 39.
    constexpr int kWave = 4 * 152;                 // resident CTAs
    Cut cut;
    cut.heads = p.q.heads + p.k.heads + p.v.heads;
    cut.any_norm = (p.q.heads > 0 && p.q.norm_dim > 0) || (p.k.heads > 0 && p.k.norm_dim > 0);
    cut.tile_rows = 8;
    while (cut.tile_rows > 1 && cut.tile_rows / 2 >= p.num_rows) cut.tile_rows /= 2;
    const long long tiles = (static_cast<long long>(p.num_rows) + cut.tile_rows - 1) / cut.tile_rows;
    const int step = kItemsOf<L> / cut.tile_rows;        // heads at once
    const int steps = (cut.heads + step - 1) / step;
    long long per_cta = steps * tiles / kWave;
    if (per_cta < 1) per_cta = 1;
    if (per_cta > steps) per_cta = steps;
    cut.chunk_heads = static_cast<int>(per_cta) * step;
    cut.chunks = (cut.heads + cut.chunk_heads - 1) / cut.chunk_heads;
    return per_cta > 1 ? launch<L, false, true>(p, cut, tiles, stream)
                       : launch<L, false, false>(p, cut, tiles, stream);
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
