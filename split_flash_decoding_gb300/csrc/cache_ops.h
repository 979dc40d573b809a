// cache_ops.h -- parameter blocks of the kernels that fill a KV cache and of
// decode attention over a cache held in 8 bits.  Everything here is already
// validated.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8_split.h"
#include "launch.h"

namespace attn {

// The 8-bit cache's kernels round token numbers up in ints.
constexpr int kMaxFp8Tokens = 0x7fffffff - 8192;

// Head vectors of a call's rows (attn_head_rows_t).
struct HeadRows {
    const uint16_t *in;
    uint16_t *out;                // nullptr: the rows go to a cache
    const uint16_t *norm;         // [norm_dim] or nullptr (weights 1)
    long long in_row, in_head, out_row, out_head;
    float eps, mean;              // mean: 1 / norm_dim
    int norm_dim, heads, dim, rot_start;
};

struct RopeParams {
    const uint64_t *turns;        // [rot_dim / 2]
    int rot_dim;                  // 0: no rotation
    int interleaved;
    float mscale;
};

// One cache operand that rows are stored to; strides in elements.
struct CacheOut {
    uint8_t *base;
    long long page_stride, token_stride, head_stride;
    float *scale;                 // 8-bit caches
    long long scale_page, scale_block, scale_head;
};

struct RowsParams {
    HeadRows q, k, v;             // heads 0: absent
    RopeParams rope;
    const int32_t *positions;     // [rows] or nullptr: the row's token
    int num_rows;
    // appending: where row r of sequence b goes (kv_len nullptr: nowhere)
    CacheOut kc, vc;
    const uint32_t *kv_len;
    const uint32_t *q_row_offsets;
    const int32_t *page_table;
    int batch, max_kv_len, page_size, num_pages, max_pages;
    int block_tokens, block_shift;  // 8-bit caches: tokens per scale, a power of two
    int max_q_len;
    unsigned *err;
};

struct Fp8DecodeParams {
    CUtensorMap k_map, v_map;     // 4-D: (channel, slot, kv head, page)
    const uint16_t *q;            // bf16 [rows][Hq][128]
    const uint32_t *kv_len;       // [batch]
    const uint32_t *q_row_offsets;  // [batch + 1], or nullptr: row b is sequence b
    const int32_t *page_table;    // [batch][max_pages] or nullptr
    const float *sink;            // [Hq] or nullptr
    float *ws_o, *ws_m, *ws_l;    // partial slots: [16 columns][128], [16], [16]
    int2 *unit_slots;             // [batch * kv heads] {first slot, pieces} for the reduce
    uint16_t *out;                // bf16 [rows][Hq][128]
    float *lse;                   // [rows][Hq] or nullptr
    unsigned *err;
    int batch, num_q_rows, num_q_heads, group, max_q_len, max_kv_len;
    int causal;
    int max_pages, page_size, num_pages;
    int box_rows;                 // tokens per TMA box (min(128, page size))
    int head_shift;               // log2 of the KV heads that a group of CTAs walks side by side
    int head_groups;              // KV heads >> head_shift
    float qk_scale_log2;          // scale * log2(e)
    const float *k_scale, *v_scale;
    long long ks_page, ks_block, ks_head, vs_page, vs_block, vs_head;
    int block_shift;              // log2(tokens per scale)
};

cudaError_t launch_head_rows(const RowsParams &p, cudaStream_t stream);
cudaError_t launch_append_fp8(const RowsParams &p, cudaStream_t stream);
// The tile kernel takes heads of up to 256 channels whose rotated pairs fall on
// whole 16-byte vectors; false: not these.
bool head_tiles_fit(const RowsParams &p);
cudaError_t launch_head_tiles(const RowsParams &p, cudaStream_t stream);
// The same into a cache held in 8 bits: blocks of up to 128 tokens, and q only
// where fp8_tiles_take_queries.
bool fp8_tiles_take_queries(const RowsParams &p);
cudaError_t launch_fp8_tiles(const RowsParams &p, bool behind_queries, cudaStream_t stream);
// Keys and values alone; behind_queries: the launch before it wrote their queries.
cudaError_t launch_fp8_runs(const RowsParams &p, bool behind_queries, cudaStream_t stream);
// CTAs of the 8-bit decode grid on num_sms SMs.
int fp8_decode_ctas(int num_sms);
cudaError_t launch_gqa_decode_fp8(const Fp8DecodeParams &p, int ctas, cudaStream_t stream);

// Address of the device error word in the current device's context (ATTN_OK
// or ATTN_ERR_CUDA).
int device_error_word(unsigned **out);
// 4-D tensor map (channel, slot in page, KV head, page) over a cache operand
// of 1-byte elements: boxes of 128 channels x box_rows slots, 128-byte swizzle.
int encode_kv_map_8bit(CUtensorMap *map, const void *base, long long token_stride,
                       long long head_stride, long long page_stride, int dim, int page_size,
                       int num_kv_heads, int num_pages, int box_rows);

}  // namespace attn
