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

cudaError_t launch_head_tiles(const RowsParams &p, cudaStream_t stream) {
    int dim = 0;
    const HeadRows *seg[3] = {&p.q, &p.k, &p.v};
    for (const HeadRows *x : seg)
        if (x->heads > 0 && x->dim > dim) dim = x->dim;
    if (dim <= 64) return launch_lanes<4, kBf16>(p, stream);
    if (dim <= 128) return launch_lanes<8, kBf16>(p, stream);
    return launch_lanes<16, kBf16>(p, stream);
}

}  // namespace attn
