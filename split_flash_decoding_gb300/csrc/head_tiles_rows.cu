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
    // (1 KB at 128 channels), and the angles of a tile are two a thread.  16 rows where
    // each row's place has to be found and there are enough of them: a CTA's start is
    // longer then.  A CTA takes all heads of its rows once the tiles fill the GPU,
    // fewer below.  us with 4, 8, 16 rows:
    //   norms, 40 heads: 1000 rows 8.6, 8.2, 8.9; 8191 37.7, 32.7, 34.9; 16384 69.4, 57.3,
    //   60.2; 32768 132.8, 107.3, 108.0
    //   to a cache, 48 heads: 3096 rows (8, 16) 20.6, 21.8; 6192 34.1, 33.1; 24768 104.8, 98.6
    constexpr int kWave = 3 * 152;                 // resident CTAs
    Cut cut;
    cut.heads = p.q.heads + p.k.heads + p.v.heads;
    cut.any_norm = (p.q.heads > 0 && p.q.norm_dim > 0) || (p.k.heads > 0 && p.k.norm_dim > 0);
    cut.tile_rows = p.kv_len && p.num_rows >= 16 * 2 * 152 ? 16 : 8;
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
