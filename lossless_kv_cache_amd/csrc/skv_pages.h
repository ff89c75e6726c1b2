// skv_pages.h -- private declarations of the paged-cache kernels.
#pragma once

#include "skv_internal.h"
#include "skv_pages_index.h"

namespace skv {

// Strides in elements of the arrays they describe.
struct PlanLaunch {
    const int32_t* lens;
    const int32_t* fresh;         // new tokens per request
    int32_t* table;
    const int32_t* free_list;     // null: the table is only read
    int32_t* slots;
    int32_t* positions;
    int32_t* starts;
    int32_t* taken;
    uint32_t* status;
    int64_t table_stride;
    uint32_t requests, width, free_pages, page_shift, tokens;
};

struct RowsLaunch {
    void* k_pages;
    void* v_pages;
    void* k;
    void* v;
    const int32_t* slots;
    const float* k_scale;
    const float* v_scale;
    uint32_t* status;
    int64_t page_layer, page_page, page_token, page_head;
    int64_t row_layer, row_token, row_head;
    uint32_t layers, tokens, heads, head_dim, page_shift, n_slots;
    uint32_t rows_dtype, pages_dtype;
    bool to_pages;
};

struct AttentionLaunch {
    const uint16_t* q;
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;        // null: one row per request
    const float* k_scale;
    const float* v_scale;
    uint16_t* out;
    float* lse;
    uint32_t* status;
    int64_t page_stride, token_stride, head_stride;                     // bytes
    int64_t table_stride, q_token, q_head, out_token, out_head;         // elements
    uint32_t requests, tokens, heads, group, width, pages, page_shift, max_new, causal;
    float scale;
    uint32_t slots;               // the workspace's, set by launch_tiles
};

hipError_t launch_plan(const PlanLaunch& a, hipStream_t stream);
hipError_t launch_rows(const RowsLaunch& a, hipStream_t stream);
// Whether every request has at most 32 query rows (the split kernel's batches).
bool attention_few_rows(const AttentionLaunch& a);
uint64_t split_work_bytes(uint32_t head_dim);
uint64_t tiles_work_bytes(const AttentionLaunch& a, uint32_t head_dim);
hipError_t launch_split(const AttentionLaunch& a, uint32_t head_dim, uint32_t dtype, void* work, hipStream_t stream);
hipError_t launch_tiles(const AttentionLaunch& a, uint32_t head_dim, uint32_t dtype, void* work, hipStream_t stream);

}  // namespace skv
