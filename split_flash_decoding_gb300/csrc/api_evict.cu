// api_evict.cu -- the extern "C" entry points around the weights that a cache's keys
// gather: host-side validation and launches.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "attn_decode.h"
#include "cache_ops.h"
#include "evict_ops.h"

namespace attn {
namespace {

bool is_pow2(long long x) { return x > 0 && (x & (x - 1)) == 0; }
bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int map_cuda(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

// A cache operand of 2-byte elements that holds up to `tokens` of each sequence.
int check_cache(const attn_kv_t *kv, int batch, int dim, int heads, int tokens) {
    if (!kv || !kv->base || kv->reserved != 0 || !aligned(kv->base, 16)) return ATTN_ERR_INVALID_ARG;
    if (kv->page_size <= 0 || kv->num_pages <= 0) return ATTN_ERR_INVALID_ARG;
    if (kv->token_stride < dim || kv->head_stride <= 0 || kv->page_stride <= 0 ||
        (heads > 1 && kv->head_stride < dim))
        return ATTN_ERR_INVALID_ARG;
    if (kv->token_stride % 8 || kv->head_stride % 8 || kv->page_stride % 8)
        return ATTN_ERR_INVALID_ARG;
    if (!kv->page_table)
        return kv->page_size < tokens || kv->num_pages < batch ? ATTN_ERR_INVALID_ARG : ATTN_OK;
    if (!is_pow2(kv->page_size) || kv->page_size < 8) return ATTN_ERR_UNSUPPORTED;
    if (kv->max_pages <= 0 ||
        (static_cast<long long>(tokens) + kv->page_size - 1) / kv->page_size > kv->max_pages)
        return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

int take_floats(const attn_kv_scale_t *w, TokenFloats *x) {
    if (!w || !w->base || w->reserved != 0 || !aligned(w->base, 4) || w->block_tokens != 1)
        return ATTN_ERR_INVALID_ARG;
    if (w->page_stride <= 0 || w->block_stride <= 0 || w->head_stride <= 0)
        return ATTN_ERR_INVALID_ARG;
    *x = {w->base, w->page_stride, w->block_stride, w->head_stride};
    return ATTN_OK;
}

MovedRows moved(const attn_kv_t *from, const attn_kv_t *to, int dim) {
    MovedRows m;
    m.from = static_cast<const uint8_t *>(from->base);
    m.to = static_cast<uint8_t *>(const_cast<void *>(to->base));
    m.from_page = 2 * from->page_stride;
    m.from_token = 2 * from->token_stride;
    m.from_head = 2 * from->head_stride;
    m.to_page = 2 * to->page_stride;
    m.to_token = 2 * to->token_stride;
    m.to_head = 2 * to->head_stride;
    m.vecs = dim / 8;
    return m;
}

bool same_layout(const attn_kv_t *a, const attn_kv_t *b) {
    return a->page_table == b->page_table && a->page_size == b->page_size &&
           a->max_pages == b->max_pages && a->num_pages == b->num_pages;
}

// Whether an output of n bytes shares any with an input of m bytes.
bool overlap(const void *out, long long n, const void *in, long long m) {
    if (!out || !in || n <= 0 || m <= 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(out), b = reinterpret_cast<uintptr_t>(in);
    return a < b + m && b < a + n;
}

// Whether key weights take the kernel of few columns, whose CTAs walk units of four KV heads in
// steps of kFewColumns, or the one of many, of whose CTAs there are `items`, one for 256 keys of a
// head.  The latter takes 5.5 us for a round of them over the GPU whatever the columns, up to 256;
// the former reads keys at the memory's rate up to 32 columns and about 14.5 us for each 16
// more of 64 sequences.  us, few and many, 8 KV heads of 128 channels:
//   columns                                32         64          128         160         192
//   64 sequences, 512 to 8192 keys     95, 330   145, 339    259, 348    315, 351    373, 360
//   131072 keys                        49, 150    72, 153    127, 159    155, 161    182, 167
//   16 sequences, 300 to 700           8.1, 16   10.7, 17    16.5, 18    19.7, 18    22.5, 18
//   4 sequences, 1024 to 4096          7.9, 13   10.8, 14    16.6, 14    19.6, 14    22.6, 15
//   500 keys                          7.4, 6.4  10.2, 6.7   16.1, 6.7   19.1, 6.9   22.1, 7.3
// (2 KV heads, 4 sequences of 1024 to 4096: 5.9, 6.8; 7.3, 6.8; 10.3, 6.9.)
bool few_columns(long long columns, int group, long long items, int sms) {
    return group <= kFewColumns && columns <= (items <= sms ? 32 : items <= 4LL * sms ? 64 : 128);
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

extern "C" int attn_key_weights(const void *q, const attn_kv_t *k, const float *lse,
                                const uint32_t *kv_len, const uint32_t *q_row_offsets, int batch,
                                int num_q_rows, int num_q_heads, int group, int head_dim,
                                int max_q_len, int max_kv_len, float scale, int causal,
                                float decay, const attn_kv_scale_t *weights,
                                attn_stream_t stream) {
    if (batch < 0 || num_q_rows < 0 || num_q_heads <= 0 || group <= 0 || max_kv_len < 0 ||
        max_q_len < 1 || num_q_heads % group)
        return ATTN_ERR_INVALID_ARG;
    if (!(scale == scale) || !(decay == decay)) return ATTN_ERR_INVALID_ARG;
    if (!q_row_offsets && (num_q_rows != batch || max_q_len != 1)) return ATTN_ERR_INVALID_ARG;
    if (batch == 0 || max_kv_len == 0) return ATTN_OK;
    if ((!q || !lse) && num_q_rows > 0) return ATTN_ERR_INVALID_ARG;
    if (!kv_len || !aligned(q, 16) || !aligned(lse, 4) || !aligned(kv_len, 4) ||
        !aligned(q_row_offsets, 4))
        return ATTN_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || group > 128 || batch > kGqaMaxBatch ||
        max_kv_len > kMaxFp8Tokens)
        return ATTN_ERR_UNSUPPORTED;
    const int hkv = num_q_heads / group;
    // items are counted in ints
    if ((max_kv_len / 128 + 1LL) * batch * hkv > 0x3fffffffLL) return ATTN_ERR_UNSUPPORTED;
    WeightsParams p;
    std::memset(&p, 0, sizeof(p));
    int st = check_cache(k, batch, head_dim, hkv, max_kv_len);
    if (st || (st = take_floats(weights, &p.w))) return st;
    int sms = 0;
    if ((st = device_sms(&sms))) return st;
    const bool few = few_columns(static_cast<long long>(max_q_len) * group, group,
                                 (max_kv_len / 256 + 1LL) * batch * hkv, sms);
    p.tile_rows = (few ? kFewColumns : kManyColumns) / group;
    p.box_rows = k->page_table && k->page_size < 128 ? k->page_size : 128;
    // (the error word first: see error_word)
    if ((st = device_error_word(&p.err)) ||
        (st = encode_kv_map_bf16(&p.k_map, k->base, k->token_stride, k->head_stride, k->page_stride,
                                 head_dim, k->page_size, hkv, k->num_pages, p.box_rows)) ||
        // (without rows the map is not used, but has to be one)
        (st = encode_q_map_bf16(&p.q_map, num_q_rows > 0 ? q : k->base, head_dim, group, hkv,
                                num_q_rows > 0 ? num_q_rows : 1, p.tile_rows)))
        return st;
    p.lse = lse;
    p.kv_len = kv_len;
    p.q_row_offsets = q_row_offsets;
    p.page_table = k->page_table;
    p.batch = batch;
    p.num_q_rows = num_q_rows;
    p.num_q_heads = num_q_heads;
    p.group = group;
    p.hkv = hkv;
    p.head_groups = (hkv + 3) / 4;
    p.max_kv_len = max_kv_len;
    p.causal = causal ? 1 : 0;
    p.max_pages = k->max_pages;
    p.page_size = k->page_size;
    p.num_pages = k->num_pages;
    p.scale = scale;
    p.decay = decay;
    return map_cuda(launch_key_weights(p, head_dim, few, sms, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int attn_evict_kv(const attn_kv_t *k, const attn_kv_t *v, const attn_kv_scale_t *weights,
                             const uint32_t *kv_len, const int32_t *keep, int batch,
                             int num_kv_heads, int dim_k, int dim_v, int max_kv_len, int max_keep,
                             int first, int recent, const attn_kv_t *k_out, const attn_kv_t *v_out,
                             const attn_kv_scale_t *weights_out, uint32_t *kept_len,
                             int32_t *indices, attn_stream_t stream) {
    if (batch < 0 || num_kv_heads <= 0 || max_kv_len < 0 || max_keep < 0 || first < 0 || recent < 0)
        return ATTN_ERR_INVALID_ARG;
    if ((v == nullptr) != (v_out == nullptr)) return ATTN_ERR_INVALID_ARG;
    if (batch == 0) return ATTN_OK;
    if (!kv_len || !keep || (!indices && max_keep > 0)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(kv_len, 4) || !aligned(keep, 4) || !aligned(kept_len, 4) || !aligned(indices, 4))
        return ATTN_ERR_INVALID_ARG;
    if (dim_k <= 0 || (v && dim_v <= 0)) return ATTN_ERR_INVALID_ARG;
    if (dim_k % 8 || dim_k > 1024 || (v && (dim_v % 8 || dim_v > 1024)) || num_kv_heads > 256 ||
        batch > kGqaMaxBatch || max_kv_len > kMaxFp8Tokens)
        return ATTN_ERR_UNSUPPORTED;
    EvictParams p;
    std::memset(&p, 0, sizeof(p));
    int st = check_cache(k, batch, dim_k, num_kv_heads, max_kv_len);
    if (st || (st = check_cache(k_out, batch, dim_k, num_kv_heads, max_keep))) return st;
    if (v) {
        if ((st = check_cache(v, batch, dim_v, num_kv_heads, max_kv_len)) ||
            (st = check_cache(v_out, batch, dim_v, num_kv_heads, max_keep)))
            return st;
        if (!same_layout(k, v) || !same_layout(k_out, v_out)) return ATTN_ERR_UNSUPPORTED;
        p.v = moved(v, v_out, dim_v);
    }
    if ((st = take_floats(weights, &p.w))) return st;
    if (weights_out && (st = take_floats(weights_out, &p.w_to))) return st;
    // Both kernels read the lengths, and every CTA for itself: nothing that the call writes may
    // lie in what it reads, lengths brought up to date in place least of all.
    const long long lens = 4LL * batch, list = 4LL * batch * num_kv_heads * max_keep;
    const struct {
        const void *at;
        long long bytes;
    } read[] = {{kv_len, lens},
                {keep, lens},
                {k->page_table, lens * k->max_pages},
                {k_out->page_table, lens * k_out->max_pages}};
    for (const auto &x : read)
        if (overlap(kept_len, lens, x.at, x.bytes) || overlap(indices, list, x.at, x.bytes))
            return ATTN_ERR_INVALID_ARG;
    if (overlap(kept_len, lens, indices, list)) return ATTN_ERR_INVALID_ARG;
    if ((st = device_error_word(&p.err))) return st;
    p.k = moved(k, k_out, dim_k);
    p.kv_len = kv_len;
    p.keep = keep;
    p.page_table = k->page_table;
    p.to_table = k_out->page_table;
    p.kept_len = kept_len;
    p.indices = indices;
    p.batch = batch;
    p.hkv = num_kv_heads;
    p.max_kv_len = max_kv_len;
    p.max_keep = max_keep;
    p.first = first;
    p.recent = recent;
    p.page_size = k->page_size;
    p.num_pages = k->num_pages;
    p.max_pages = k->max_pages;
    p.to_page_size = k_out->page_size;
    p.to_num_pages = k_out->num_pages;
    p.to_max_pages = k_out->max_pages;
    int sms = 0;
    if ((st = device_sms(&sms))) return st;
    return map_cuda(launch_evict(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}
