/*
 * latent_bf16.h - operators over a paged cache of shared latent rows on GB300
 * (sm_103a): what a decode step does before and after the top-k of topk_bf16.h.
 * Same library (libtopk_bf16.so), same conventions: plain C functions, device
 * pointers of the current device, nothing allocated, kept or synchronised, all
 * work enqueued on `stream`, argument errors returned as a status with nothing
 * enqueued, device-side data never validated by trapping, device status word
 * as topk_bf16_device_status. The kernels take part in programmatic dependent
 * launch as the top-k's do: they wait for the preceding grid before they read
 * or write anything of the caller's, and release the next grid early, so a
 * successor launched with programmatic stream serialization must execute
 * griddepcontrol.wait before it touches this call's inputs or outputs.
 *
 * The cache. One BF16 row per token, shared by all heads:
 *     row = [ c (latent values) | r (LATENT_ROPE values, rotated by position) ]
 * c is key and value, r is key only. Rows are addressed by physical row number
 * (page * block_rows + offset), which is what the top-k writes with a block
 * table. latent is 128, 256, 384 or 512.
 *
 * Attention in the absorbed form: query row (t, h) holds latent + LATENT_ROPE
 * values (the key up-projection folded into it by the caller), and
 *     s_j   = scale * <query[t, h], row_j>          over the rows j it may see
 *     p_j   = exp(s_j - lse),   lse = log sum_j exp(s_j)
 *     out   = sum_j p_j c_j                          (latent values)
 * A query row that sees nothing, or whose scores are all -inf, gets out = 0 and
 * lse = -inf. A cache row that query row (t, h) may not see, or whose score is
 * -inf there, is no part of out[t, h] and lse[t, h], whatever it holds and whatever
 * other query rows see of it.
 * If a row that query row (t, h) sees makes its s_j NaN or +inf, out[t, h] is NaN.
 * The sums are held in 32 bits, in units of a weight that may lag the largest by
 * 2^16: latent values past 2^96 may overflow them.
 */
#ifndef LATENT_BF16_H
#define LATENT_BF16_H

#include <stddef.h>
#include <stdint.h>

#include "topk_bf16.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LATENT_ROPE 64        /* rotated values of a cache row */
#define LATENT_MAX 512        /* largest latent */
#define LATENT_MAX_HEADS 256  /* query heads per token */
#define LATENT_MAX_LENGTH (1 << 30)  /* list entries or width of an attention call */

/*
 * Appends tokens to the cache: for token t with row slots[t] in [0, cache_rows)
 *     cache[slots[t]][0 .. latent)    = weight ? norm(latents[t]) : latents[t]
 *     cache[slots[t]][latent .. )     = rotate(key_rope[t], positions[t])
 * and, for every token (whatever its slot) when query_rope is given,
 *     query[t][h][latent .. )         = rotate(query_rope[t][h], positions[t]).
 * norm(x) = x * weight / sqrt(mean(x^2) + eps). rotate turns pair i, i < 32, by
 * the angle whose cosine and sine are cos_sin[p][i] and cos_sin[p][32 + i]:
 * (a, b) -> (a cos - b sin, a sin + b cos); pair i is values (2 i, 2 i + 1) when
 * interleaved, else (i, i + 32). Computed in 32 bits and rounded once.
 *
 * cache          device BF16, row r at cache + r * cache_stride; 16-byte aligned,
 *                cache_stride a multiple of 8, >= latent + LATENT_ROPE.
 * latents        device BF16 [tokens], rows of `latent` values latents_stride apart.
 * key_rope       device BF16 [tokens], rows of 64 values key_stride apart.
 * positions      device int32 [tokens], clamped to [0, max_positions).
 * cos_sin        device float [max_positions, 64], 16-byte aligned.
 * slots          device int32 [tokens]; a token whose slot lies outside
 *                [0, cache_rows) is not written. Distinct otherwise.
 * weight         NULL (no norm) or device BF16 [latent].
 * query_rope     NULL, or device BF16 [tokens, heads, 64] with the strides given.
 * query          device BF16 [tokens, heads, latent + 64] with the strides given;
 *                only its last 64 values are written. NULL with query_rope NULL.
 * All BF16 pointers are 16-byte aligned and all strides multiples of 8 elements.
 * Outputs must not overlap inputs, except that query_rope may be query's own last
 * 64 values (query + latent, with query's strides): they are then rotated in place.
 *
 * Errors: TOPK_ERR_ARG (null pointer, negative count, more than 2^27 tokens, heads
 * outside [1, LATENT_MAX_HEADS] with query_rope, max_positions < 1, query_rope without
 * query), TOPK_ERR_WIDTH (latent, or a stride below its row), TOPK_ERR_ALIGN.
 */
typedef struct {
    uint16_t *cache;
    int64_t cache_stride;
    const uint16_t *latents;
    int64_t latents_stride;
    const uint16_t *key_rope;
    int64_t key_stride;
    const int32_t *positions;
    const float *cos_sin;
    const int32_t *slots;
    const uint16_t *weight;
    const uint16_t *query_rope;
    int64_t query_rope_token_stride, query_rope_head_stride;
    uint16_t *query;
    int64_t query_token_stride, query_head_stride;
    int32_t cache_rows, tokens, latent, heads, max_positions, interleaved;
    float eps;
} latent_bf16_append_t;

topk_status_t latent_bf16_append(const latent_bf16_append_t *args, void *stream);

/*
 * Attention of `tokens` query tokens over cache rows. Fields common to both
 * forms:
 *
 * query          device BF16 [tokens, heads, latent + 64], strides in elements
 *                (multiples of 8), 16-byte aligned, unit inner stride.
 * cache          as above, read only; cache_rows rows.
 * scale          factor of the scores.
 * out            device BF16 [tokens, heads, latent], contiguous, 16-byte
 *                aligned, fully written.
 * lse            NULL, or device float [tokens, heads]: lse as above (natural
 *                logarithm), for joining parts of one softmax.
 * workspace      device scratch, 16-byte aligned, of latent_bf16_attend_workspace()
 *                bytes for this call (0 for many: NULL will do) or of
 *                latent_bf16_workspace_bytes(), which is enough for any; used by
 *                this call alone until it completes.
 *
 * latent_bf16_attend_selected: token t sees the cache rows selected[t *
 * selected_stride + i], i < k, that lie in [0, cache_rows); other entries (the
 * top-k's -1) are empty places, in any order. A row listed twice counts twice. A
 * block-mode selection (TOPK_BLOCK8) names 8-token blocks, not rows: it has to be
 * expanded to its tokens' rows first.
 *
 * latent_bf16_attend_paged: token t belongs to request t / rows_per_request and
 * sees that request's first valid_len[t] tokens (clamped to [0, width]); token
 * i of the request is cache row block_table[request * table_stride +
 * i / page_size] * block_rows + i % page_size. A causal chunk is lengths that
 * grow by one; a padded token has length 0. Pages that lead outside the cache
 * are left out. page_size is a power of two, block_rows >= page_size,
 * table_stride >= ceil(width / page_size).
 *
 * Errors: TOPK_ERR_ARG (null pointer, negative count, heads outside
 * [1, LATENT_MAX_HEADS], k above LATENT_MAX_LENGTH, a bad page size, block_rows, table stride, workspace
 * size or rows_per_request, a scale that is not finite), TOPK_ERR_WIDTH
 * (latent, width, or a stride below its row), TOPK_ERR_ALIGN, TOPK_ERR_CUDA.
 */
typedef struct {
    const uint16_t *query;
    int64_t query_token_stride, query_head_stride;
    const uint16_t *cache;
    int64_t cache_stride;
    const int32_t *selected;      /* selected form */
    int64_t selected_stride;
    const int32_t *valid_len;     /* paged form */
    const int32_t *block_table;
    uint16_t *out;
    float *lse;
    void *workspace;
    int64_t workspace_bytes;
    int32_t cache_rows, tokens, heads, latent;
    int32_t k;                    /* selected form: entries per list */
    int32_t width, table_stride, page_size, block_rows, rows_per_request;  /* paged form */
    float scale;
} latent_bf16_attend_t;

topk_status_t latent_bf16_attend_selected(const latent_bf16_attend_t *args, void *stream);
topk_status_t latent_bf16_attend_paged(const latent_bf16_attend_t *args, void *stream);

/* Bytes of scratch that a call with these arguments needs on the current device
   (paged: which form; `workspace` is not looked at); -1 for arguments that the
   call would refuse, or if the device cannot be asked. */
int64_t latent_bf16_attend_workspace(const latent_bf16_attend_t *args, int32_t paged);

/* Bytes of scratch that are enough for any attention call on the current device;
   0 if the device cannot be asked. */
int64_t latent_bf16_workspace_bytes(void);

#ifdef __cplusplus
}
#endif

#endif /* LATENT_BF16_H */
