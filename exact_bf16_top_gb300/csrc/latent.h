// Launch parameters of the latent-cache operators and the host-side interface
// between their translation units (plain C++: no device code).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "latent4.h"
#include "latent_bf16.h"

namespace topk::latent {

struct AttendParams {
    const uint16_t *query;
    int64_t query_token_stride, query_head_stride;
    const void *cache;           // BF16 rows, or rows in 4 bits
    int64_t cache_stride;        // in elements; of rows in 4 bits in bytes
    const int32_t *selected;     // may be NULL with k = 0
    int64_t selected_stride;
    const int32_t *valid_len;
    const int32_t *table;
    uint16_t *out;
    float *lse;
    int32_t cache_rows, tokens, heads, latent;
    int32_t k;
    int32_t paged;               // which form the call takes
    int32_t width, table_stride, page_shift, block_rows, rows_per_request;
    float scale;
    void *workspace;
    int32_t tiles, tiles_per_request, min_share, sms, tiled, cluster, tile_cost;   // filled in by launch_attend
};

cudaError_t launch_append(const latent_bf16_append_t &a, int sms, cudaStream_t stream);
cudaError_t launch_attend(AttendParams p, cudaStream_t stream);
// Joins the split tiles' parts that an attention kernel of `grid` CTAs left in the workspace (nr: rows of a tile).
cudaError_t launch_join(const AttendParams &p, unsigned grid, int nr, cudaStream_t stream);
int64_t attend_workspace(AttendParams p);   // bytes this call needs, -1 if the device cannot be asked
int64_t workspace_bytes();   // 0 if the device cannot be asked

// The same for rows in 4 bits.
cudaError_t launch_append4(const latent4_append_t &a, int sms, cudaStream_t stream);
cudaError_t launch_rows4(const uint8_t *cache, int64_t cache_stride, int32_t cache_rows, int32_t latent,
                         const int32_t *rows, int32_t count, uint16_t *out, int64_t out_stride, int sms,
                         cudaStream_t stream);
cudaError_t launch_attend4(AttendParams p, cudaStream_t stream);
int64_t attend4_workspace(AttendParams p);
int64_t workspace4_bytes();

}  // namespace topk::latent
