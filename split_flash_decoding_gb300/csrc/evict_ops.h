// evict_ops.h -- parameter blocks of the kernels that gather the attention weight
// of a cache's keys and move the heaviest ones together.  Everything here is
// already validated.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

// One fp32 value for each token and KV head of a cache (attn_kv_scale_t with
// block_tokens 1); strides in floats.
struct TokenFloats {
    float *base;
    long long page, token, head;
};

struct WeightsParams {
    CUtensorMap q_map;            // 4-D: (channel, head in group, kv head, row)
    CUtensorMap k_map;            // 4-D: (channel, slot, kv head, page)
    const float *lse;             // [rows][Hq]
    const uint32_t *kv_len;       // [batch]
    const uint32_t *q_row_offsets;  // [batch + 1], or nullptr: row b is sequence b
    const int32_t *page_table;    // [batch][max_pages] or nullptr
    TokenFloats w;
    unsigned *err;
    int batch, num_q_rows, num_q_heads, group, hkv, max_kv_len;
    int causal;
    int max_pages, page_size, num_pages;
    int box_rows;                 // tokens per TMA box (min(128, page size))
    int tile_rows;                // query rows per column tile
    int head_groups;              // KV heads in fours, rounded up
    float scale, decay;
};

// Columns (query rows x heads of a group) of a step's score tile.
constexpr int kFewColumns = 16, kManyColumns = 256;

// head_dim 64 or 128; few: column tiles of kFewColumns, else of kManyColumns.
cudaError_t launch_key_weights(const WeightsParams &p, int head_dim, bool few, int sms,
                               cudaStream_t stream);

// A cache operand's rows: `vecs` 16-byte vectors each; strides in bytes.
struct MovedRows {
    const uint8_t *from;
    uint8_t *to;
    long long from_page, from_token, from_head, to_page, to_token, to_head;
    int vecs;
};

struct EvictParams {
    MovedRows k, v;               // v.vecs 0: absent
    TokenFloats w, w_to;          // w_to.base nullptr: not wanted
    const uint32_t *kv_len;       // [batch]
    const int32_t *keep;          // [batch]
    const int32_t *page_table, *to_table;   // [batch][max_pages] / [to_max_pages], or nullptr
    uint32_t *kept_len;           // [batch] or nullptr
    int32_t *indices;             // [batch][hkv][max_keep]
    unsigned *err;
    int batch, hkv, max_kv_len, max_keep, first, recent;
    int page_size, num_pages, max_pages, to_page_size, to_num_pages, to_max_pages;
};

cudaError_t launch_evict(const EvictParams &p, int sms, cudaStream_t stream);

// 4-D tensor map (channel, slot in page, KV head, page) over a bf16 cache operand:
// boxes of 64 channels x box_rows slots, 128-byte swizzle.
int encode_kv_map_bf16(CUtensorMap *map, const void *base, long long token_stride,
                       long long head_stride, long long page_stride, int dim, int page_size,
                       int num_kv_heads, int num_pages, int box_rows);
// 4-D tensor map (channel, head of a group, KV head, row) over queries [rows][heads][dim]:
// boxes of 64 channels x group heads x box_rows rows, 128-byte swizzle.
int encode_q_map_bf16(CUtensorMap *map, const void *q, int dim, int group, int num_kv_heads,
                      int num_q_rows, int box_rows);

}  // namespace attn
