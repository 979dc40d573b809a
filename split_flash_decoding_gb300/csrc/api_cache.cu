// api_cache.cu -- the extern "C" entry points that fill a KV cache and read one
// held in 8 bits: host-side validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn_decode.h"
#include "cache_ops.h"

namespace attn {
namespace {

bool is_pow2(long long x) { return x > 0 && (x & (x - 1)) == 0; }
bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int map_cuda(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

// Head rows of an entry point; to_rows: they go to rows of memory (out), else
// to a cache.
int take_heads(const attn_head_rows_t &h, bool to_rows, const attn_rope_t *rope, int num_rows,
               HeadRows *x) {
    if (h.reserved != 0 || h.num_heads <= 0 || h.dim <= 0 || h.norm_dim < 0 || h.rot_start < 0)
        return ATTN_ERR_INVALID_ARG;
    if (h.dim % 8 || h.dim > 1024 || h.norm_dim % 8 || h.rot_start % 8) return ATTN_ERR_UNSUPPORTED;
    if (h.norm_dim > h.dim) return ATTN_ERR_INVALID_ARG;
    if (rope && (h.rot_start > h.dim || rope->rot_dim > h.dim - h.rot_start))
        return ATTN_ERR_INVALID_ARG;
    if (h.norm_dim > 0 && !(h.norm_eps >= 0.f)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(h.norm_weight, 16)) return ATTN_ERR_INVALID_ARG;
    if (to_rows != (h.out != nullptr) && num_rows > 0) return ATTN_ERR_INVALID_ARG;
    if (num_rows > 0 && !h.in) return ATTN_ERR_INVALID_ARG;
    if (!aligned(h.in, 16) || !aligned(h.out, 16)) return ATTN_ERR_INVALID_ARG;
    if (h.in_row_stride % 8 || h.in_head_stride % 8) return ATTN_ERR_INVALID_ARG;
    if (to_rows && (h.out_row_stride % 8 || h.out_head_stride % 8)) return ATTN_ERR_INVALID_ARG;
    x->in = static_cast<const uint16_t *>(h.in);
    x->out = static_cast<uint16_t *>(h.out);
    x->norm = static_cast<const uint16_t *>(h.norm_weight);
    x->in_row = h.in_row_stride;
    x->in_head = h.in_head_stride;
    x->out_row = h.out_row_stride;
    x->out_head = h.out_head_stride;
    x->eps = h.norm_eps;
    x->mean = h.norm_dim > 0 ? 1.f / static_cast<float>(h.norm_dim) : 0.f;
    x->norm_dim = h.norm_dim;
    x->heads = h.num_heads;
    x->dim = h.dim;
    x->rot_start = h.rot_start;
    return ATTN_OK;
}

int take_rope(const attn_rope_t *rope, RopeParams *r) {
    r->turns = nullptr;
    r->rot_dim = 0;
    r->interleaved = 0;
    r->mscale = 1.f;
    if (!rope) return ATTN_OK;
    if (rope->reserved != 0 || rope->rot_dim < 0 || rope->rot_dim % 2) return ATTN_ERR_INVALID_ARG;
    if (!(rope->mscale == rope->mscale)) return ATTN_ERR_INVALID_ARG;
    if (rope->rot_dim > 0 && (!rope->turns || !aligned(rope->turns, 8))) return ATTN_ERR_INVALID_ARG;
    r->turns = rope->turns;
    r->rot_dim = rope->rot_dim;
    r->interleaved = rope->interleaved ? 1 : 0;
    r->mscale = rope->mscale;
    return ATTN_OK;
}

// A cache operand that rows are stored to; unit: elements per 16 bytes.
int take_cache(const attn_kv_t *kv, int batch, int dim, int num_kv_heads, int max_kv_len, int unit,
               CacheOut *c) {
    if (!kv || !kv->base || kv->reserved != 0) return ATTN_ERR_INVALID_ARG;
    if (!aligned(kv->base, 16)) return ATTN_ERR_INVALID_ARG;
    if (kv->page_size <= 0 || kv->num_pages <= 0) return ATTN_ERR_INVALID_ARG;
    if (kv->token_stride <= 0 || kv->head_stride <= 0 || kv->page_stride <= 0)
        return ATTN_ERR_INVALID_ARG;
    if (kv->token_stride % unit || kv->head_stride % unit || kv->page_stride % unit)
        return ATTN_ERR_INVALID_ARG;
    if (kv->token_stride < dim || (num_kv_heads > 1 && kv->head_stride < dim))
        return ATTN_ERR_INVALID_ARG;
    if (kv->page_table) {
        if (!is_pow2(kv->page_size) || kv->page_size < 8) return ATTN_ERR_UNSUPPORTED;
        if (kv->max_pages <= 0) return ATTN_ERR_INVALID_ARG;
        if ((static_cast<long long>(max_kv_len) + kv->page_size - 1) / kv->page_size > kv->max_pages)
            return ATTN_ERR_INVALID_ARG;
    } else {
        if (kv->page_size < max_kv_len || kv->num_pages < batch) return ATTN_ERR_INVALID_ARG;
    }
    c->base = static_cast<uint8_t *>(const_cast<void *>(kv->base));
    c->page_stride = kv->page_stride;
    c->token_stride = kv->token_stride;
    c->head_stride = kv->head_stride;
    return ATTN_OK;
}

bool same_layout(const attn_kv_t *a, const attn_kv_t *b) {
    return a->page_table == b->page_table && a->page_size == b->page_size &&
           a->max_pages == b->max_pages && a->num_pages == b->num_pages;
}

int check_scale(const attn_kv_scale_t *s, const attn_kv_t *kv) {
    if (!s || !s->base || s->reserved != 0 || !aligned(s->base, 4)) return ATTN_ERR_INVALID_ARG;
    if (s->page_stride <= 0 || s->block_stride <= 0 || s->head_stride <= 0)
        return ATTN_ERR_INVALID_ARG;
    if (!is_pow2(s->block_tokens) || kv->page_size % s->block_tokens) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

void take_scale(const attn_kv_scale_t *s, CacheOut *c) {
    c->scale = s->base;
    c->scale_page = s->page_stride;
    c->scale_block = s->block_stride;
    c->scale_head = s->head_stride;
}

// Shared part of the two appending entry points.
int take_append(const attn_head_rows_t *q, const attn_head_rows_t *k, const attn_head_rows_t *v,
                const attn_rope_t *rope, const int32_t *positions, const attn_kv_t *k_cache,
                const attn_kv_t *v_cache, const uint32_t *kv_len, const uint32_t *q_row_offsets,
                int batch, int num_q_rows, int max_kv_len, int unit, RowsParams *p) {
    std::memset(p, 0, sizeof(*p));
    if (batch < 0 || num_q_rows < 0 || max_kv_len < 0) return ATTN_ERR_INVALID_ARG;
    if (!q_row_offsets && num_q_rows != batch) return ATTN_ERR_INVALID_ARG;
    if (batch == 0 || num_q_rows == 0) return ATTN_OK;   // num_rows stays 0: nothing to do
    if (!k || !kv_len || (v == nullptr) != (v_cache == nullptr)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || !aligned(kv_len, 4) || !aligned(q_row_offsets, 4))
        return ATTN_ERR_INVALID_ARG;
    int st = take_rope(rope, &p->rope);
    if (st) return st;
    if (q && (st = take_heads(*q, true, rope, num_q_rows, &p->q))) return st;
    if ((st = take_heads(*k, false, rope, num_q_rows, &p->k))) return st;
    if ((st = take_cache(k_cache, batch, k->dim, k->num_heads, max_kv_len, unit, &p->kc))) return st;
    if (v) {
        if ((st = take_heads(*v, false, nullptr, num_q_rows, &p->v))) return st;
        if (v->norm_dim != 0 || v->num_heads != k->num_heads) return ATTN_ERR_INVALID_ARG;
        if ((st = take_cache(v_cache, batch, v->dim, v->num_heads, max_kv_len, unit, &p->vc)))
            return st;
        if (!same_layout(k_cache, v_cache)) return ATTN_ERR_UNSUPPORTED;
    }
    p->positions = positions;
    p->num_rows = num_q_rows;
    p->kv_len = kv_len;
    p->q_row_offsets = q_row_offsets;
    p->page_table = k_cache->page_table;
    p->batch = batch;
    p->max_kv_len = max_kv_len;
    p->page_size = k_cache->page_size;
    p->num_pages = k_cache->num_pages;
    p->max_pages = k_cache->max_pages;
    return ATTN_OK;
}

// Partial slots of the balanced split (CTAs + units) of 16 columns x 128
// channels, m and l per column, then the unit table {first slot, pieces}.
size_t fp8_layout(int ctas, long long units, size_t *off_m, size_t *off_l, size_t *off_table) {
    const size_t n = (size_t(ctas) + size_t(units)) * size_t(kGqaSlotCols);
    const size_t o_bytes = align256(n * 128 * sizeof(float));
    const size_t m_bytes = align256(n * sizeof(float));
    if (off_m) *off_m = o_bytes;
    if (off_l) *off_l = o_bytes + m_bytes;
    if (off_table) *off_table = o_bytes + 2 * m_bytes;
    return o_bytes + 2 * m_bytes + align256(size_t(units) * 8);
}

int device_sms(int *sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return ATTN_ERR_CUDA;
    return ATTN_OK;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" int attn_rope_turns(int rot_dim, double theta, int scaling, double factor,
                               double original_len, double low, double high, uint64_t *turns,
                               float *mscale) {
    if (rot_dim <= 0 || rot_dim % 2 || !turns || !(theta > 0.0) || !std::isfinite(theta))
        return ATTN_ERR_INVALID_ARG;
    if (scaling < ATTN_ROPE_PLAIN || scaling > ATTN_ROPE_BANDS) return ATTN_ERR_INVALID_ARG;
    if (scaling != ATTN_ROPE_PLAIN && !(factor > 0.0 && std::isfinite(factor)))
        return ATTN_ERR_INVALID_ARG;
    const bool parts = scaling == ATTN_ROPE_YARN || scaling == ATTN_ROPE_BANDS;
    if (parts && !(original_len > 0.0 && low > 0.0 && high > low && std::isfinite(high) &&
                   std::isfinite(original_len)))
        return ATTN_ERR_INVALID_ARG;
    if (scaling == ATTN_ROPE_YARN && theta == 1.0) return ATTN_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    const int half = rot_dim / 2;
    double base = theta;
    if (scaling == ATTN_ROPE_NTK && rot_dim > 2)
        base = theta * std::pow(factor, rot_dim / (rot_dim - 2.0));
    // YARN: pair indices at which the period fits `high` and `low` times into
    // the original length
    double i_lo = 0.0, i_hi = 0.0;
    if (scaling == ATTN_ROPE_YARN) {
        const auto index = [&](double n) {
            return rot_dim * std::log(original_len / (n * two_pi)) / (2.0 * std::log(theta));
        };
        i_lo = std::fmax(0.0, std::floor(index(high)));
        i_hi = std::fmin(rot_dim - 1.0, std::ceil(index(low)));
        if (i_hi - i_lo < 1e-3) i_hi = i_lo + 1e-3;
    }
    for (int i = 0; i < half; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == ATTN_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == ATTN_ROPE_YARN) {
            const double x = std::fmin(1.0, std::fmax(0.0, (i - i_lo) / (i_hi - i_lo)));
            f = f * (1.0 - x) + f / factor * x;
        } else if (scaling == ATTN_ROPE_BANDS) {
            const double n = original_len * f / two_pi;   // turns in the original length
            const double x = std::fmin(1.0, std::fmax(0.0, (n - low) / (high - low)));
            f = (1.0 - x) * f / factor + x * f;
        }
        if (!std::isfinite(f)) return ATTN_ERR_INVALID_ARG;
        double t = f / two_pi;
        t -= std::floor(t);
        turns[i] = static_cast<uint64_t>(std::ldexp(t, 64));
    }
    if (mscale)
        *mscale = scaling == ATTN_ROPE_YARN && factor > 1.0
                      ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return ATTN_OK;
}

extern "C" int attn_qk_norm_rope(const attn_head_rows_t *q, const attn_head_rows_t *k,
                                 const attn_rope_t *rope, const int32_t *positions, int num_rows,
                                 attn_stream_t stream) {
    if (num_rows < 0 || !q) return ATTN_ERR_INVALID_ARG;
    RowsParams p;
    std::memset(&p, 0, sizeof(p));
    int st = take_rope(rope, &p.rope);
    if (st) return st;
    if ((st = take_heads(*q, true, rope, num_rows, &p.q))) return st;
    if (k && (st = take_heads(*k, true, rope, num_rows, &p.k))) return st;
    if (num_rows == 0) return ATTN_OK;
    if ((p.rope.rot_dim > 0 && !positions) || !aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
    p.positions = positions;
    p.num_rows = num_rows;
    return map_cuda(launch_head_rows(p, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int attn_append_kv(const attn_head_rows_t *q, const attn_head_rows_t *k,
                              const attn_head_rows_t *v, const attn_rope_t *rope,
                              const int32_t *positions, const attn_kv_t *k_cache,
                              const attn_kv_t *v_cache, const uint32_t *kv_len,
                              const uint32_t *q_row_offsets, int batch, int num_q_rows,
                              int max_kv_len, attn_stream_t stream) {
    RowsParams p;
    int st = take_append(q, k, v, rope, positions, k_cache, v_cache, kv_len, q_row_offsets, batch,
                         num_q_rows, max_kv_len, 8, &p);
    if (st || p.num_rows == 0) return st;
    if ((st = device_error_word(&p.err))) return st;
    return map_cuda(launch_head_rows(p, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int attn_append_kv_fp8(const attn_head_rows_t *q, const attn_head_rows_t *k,
                                  const attn_head_rows_t *v, const attn_rope_t *rope,
                                  const int32_t *positions, const attn_kv_t *k_cache,
                                  const attn_kv_t *v_cache, const attn_kv_scale_t *k_scale,
                                  const attn_kv_scale_t *v_scale, const uint32_t *kv_len,
                                  const uint32_t *q_row_offsets, int batch, int num_q_rows,
                                  int max_q_len, int max_kv_len, attn_stream_t stream) {
    RowsParams p;
    int st = take_append(q, k, v, rope, positions, k_cache, v_cache, kv_len, q_row_offsets, batch,
                         num_q_rows, max_kv_len, 16, &p);
    if (st || p.num_rows == 0) return st;
    if (!v || max_q_len < 1 || (!q_row_offsets && max_q_len != 1)) return ATTN_ERR_INVALID_ARG;
    if (k->dim != 128 || v->dim != 128 || max_kv_len > kMaxFp8Tokens) return ATTN_ERR_UNSUPPORTED;
    if ((st = check_scale(k_scale, k_cache)) || (st = check_scale(v_scale, v_cache))) return st;
    if (k_scale->block_tokens != v_scale->block_tokens) return ATTN_ERR_UNSUPPORTED;
    take_scale(k_scale, &p.kc);
    take_scale(v_scale, &p.vc);
    p.block_tokens = k_scale->block_tokens;
    while ((1 << p.block_shift) < p.block_tokens) ++p.block_shift;
    p.max_q_len = max_q_len;
    if ((st = device_error_word(&p.err))) return st;
    return map_cuda(launch_append_fp8(p, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int attn_decode_fp8_workspace(int num_sms, int batch, int num_q_heads, int group,
                                         size_t *workspace_bytes) {
    if (!workspace_bytes || batch < 0 || num_q_heads <= 0 || group <= 0 || num_q_heads % group)
        return ATTN_ERR_INVALID_ARG;
    if (num_sms <= 0) {
        const int st = device_sms(&num_sms);
        if (st) return st;
    }
    *workspace_bytes = fp8_layout(fp8_decode_ctas(num_sms),
                                  static_cast<long long>(batch > 0 ? batch : 1) *
                                      (num_q_heads / group),
                                  nullptr, nullptr, nullptr);
    return ATTN_OK;
}

extern "C" int attn_decode_fp8(const void *q, const attn_kv_t *k, const attn_kv_t *v,
                               const attn_kv_scale_t *k_scale, const attn_kv_scale_t *v_scale,
                               const uint32_t *kv_len, const uint32_t *q_row_offsets, int batch,
                               int num_q_rows, int num_q_heads, int group, int head_dim,
                               int max_q_len, int max_kv_len, float scale, const float *sink,
                               int causal, void *workspace, size_t workspace_bytes, void *out,
                               float *lse, attn_stream_t stream) {
    if (batch < 0 || num_q_rows < 0 || num_q_heads <= 0 || group <= 0 || max_kv_len < 0 ||
        max_q_len < 1)
        return ATTN_ERR_INVALID_ARG;
    if (num_q_heads % group) return ATTN_ERR_INVALID_ARG;
    if (!(scale == scale)) return ATTN_ERR_INVALID_ARG;
    if (!q_row_offsets && (num_q_rows != batch || max_q_len != 1)) return ATTN_ERR_INVALID_ARG;
    if (batch == 0 || num_q_rows == 0) return ATTN_OK;
    if (!q || !kv_len || !out) return ATTN_ERR_INVALID_ARG;
    if (head_dim != 128 || static_cast<long long>(max_q_len) * group > 16 || batch > kGqaMaxBatch)
        return ATTN_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16)) return ATTN_ERR_INVALID_ARG;
    const int hkv = num_q_heads / group;
    int head_shift = 0;
    while (head_shift < 3 && hkv % (2 << head_shift) == 0) ++head_shift;
    // the split counts the costs of its tiles in ints
    const long long most = (max_kv_len / kGqaTcTileKeys + 1) * kFp8MostTileCost + kFp8UnitCost;
    if (max_kv_len > kMaxFp8Tokens || most * batch * (hkv >> head_shift) > 0x7fffffffLL)
        return ATTN_ERR_UNSUPPORTED;
    CacheOut kc, vc;
    int st = take_cache(k, batch, head_dim, hkv, max_kv_len, 16, &kc);
    if (st) return st;
    if ((st = take_cache(v, batch, head_dim, hkv, max_kv_len, 16, &vc))) return st;
    if (!same_layout(k, v)) return ATTN_ERR_UNSUPPORTED;
    if ((st = check_scale(k_scale, k)) || (st = check_scale(v_scale, v))) return st;
    if (k_scale->block_tokens != v_scale->block_tokens) return ATTN_ERR_UNSUPPORTED;
    // Units of one tile are never cut: no partials, nothing to merge.
    const bool cut = max_kv_len > kGqaTcTileKeys;
    int sms = 0;
    if (cut && (!workspace || !aligned(workspace, 256))) return ATTN_ERR_WORKSPACE;
    if ((st = device_sms(&sms))) return st;
    const int ctas = fp8_decode_ctas(sms);
    size_t off_m = 0, off_l = 0, off_table = 0;
    if (cut && workspace_bytes < fp8_layout(ctas, static_cast<long long>(batch) * hkv, &off_m, &off_l,
                                     &off_table))
        return ATTN_ERR_WORKSPACE;

    Fp8DecodeParams p;
    std::memset(&p, 0, sizeof(p));
    if ((st = device_error_word(&p.err))) return st;
    p.q = static_cast<const uint16_t *>(q);
    p.kv_len = kv_len;
    p.q_row_offsets = q_row_offsets;
    p.page_table = k->page_table;
    p.sink = sink;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.batch = batch;
    p.num_q_rows = num_q_rows;
    p.num_q_heads = num_q_heads;
    p.group = group;
    p.max_q_len = max_q_len;
    p.causal = causal ? 1 : 0;
    p.max_pages = k->max_pages;
    p.page_size = k->page_size;
    p.num_pages = k->num_pages;
    p.qk_scale_log2 = scale * 1.4426950408889634f;
    p.max_kv_len = max_kv_len;
    p.head_shift = head_shift;
    p.head_groups = hkv >> p.head_shift;
    if (cut) {
        uint8_t *ws = static_cast<uint8_t *>(workspace);
        p.ws_o = reinterpret_cast<float *>(ws);
        p.ws_m = reinterpret_cast<float *>(ws + off_m);
        p.ws_l = reinterpret_cast<float *>(ws + off_l);
        p.unit_slots = reinterpret_cast<int2 *>(ws + off_table);
    }
    p.box_rows = k->page_table && k->page_size < kGqaTcTileKeys ? k->page_size : kGqaTcTileKeys;
    if ((st = encode_kv_map_8bit(&p.k_map, k->base, k->token_stride, k->head_stride,
                                 k->page_stride, head_dim, k->page_size, hkv, k->num_pages,
                                 p.box_rows)))
        return st;
    if ((st = encode_kv_map_8bit(&p.v_map, v->base, v->token_stride, v->head_stride,
                                 v->page_stride, head_dim, v->page_size, hkv, v->num_pages,
                                 p.box_rows)))
        return st;
    p.k_scale = k_scale->base;
    p.ks_page = k_scale->page_stride;
    p.ks_block = k_scale->block_stride;
    p.ks_head = k_scale->head_stride;
    p.v_scale = v_scale->base;
    p.vs_page = v_scale->page_stride;
    p.vs_block = v_scale->block_stride;
    p.vs_head = v_scale->head_stride;
    p.block_shift = 0;
    while ((1 << p.block_shift) < k_scale->block_tokens) ++p.block_shift;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    st = map_cuda(launch_gqa_decode_fp8(p, ctas, s));
    if (st || !cut) return st;
    ReduceParams r;
    std::memset(&r, 0, sizeof(r));
    r.ws_o = p.ws_o;
    r.ws_m = p.ws_m;
    r.ws_l = p.ws_l;
    r.sink = sink;
    r.out = p.out;
    r.lse = lse;
    r.q_row_offsets = q_row_offsets;
    r.batch = batch;
    r.num_partitions = ctas;   // the most pieces a unit can have
    r.rows = num_q_rows;
    r.num_q_heads = num_q_heads;
    r.dim_v = head_dim;
    r.unit_slots = p.unit_slots;
    r.group = group;
    r.hkv = hkv;
    return map_cuda(launch_splitk_reduce(r, s, /*pdl=*/true));
}
