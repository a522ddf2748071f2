/*
 * latent4.h - operators over a paged cache of shared latent rows held in 4 bits,
 * on GB300 (sm_103a): latent_bf16.h's with rows of 160 + latent / 2 bytes in place
 * of 2 latent + 128. Same library, same conventions (latent_bf16.h).
 *
 * The cache. One row of bytes per token, shared by all heads:
 *     row = [ codes: latent / 2 | key part: 128 | scales: 32 ]
 * Value i < latent is e2m1(code i) * e4m3(scale[i / 16]); code 2 j is the low half
 * of byte j, code 2 j + 1 the high half. The key part is LATENT_ROPE BF16 values,
 * rotated by position, that are key only (in 4 bits they would turn the angles of
 * far positions into noise). Of the 32 scale bytes latent / 16 are used; the others
 * are neither read nor written. e2m1 holds 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
 * negatives (sign in the highest bit); e4m3 has no infinity, 0x7F is NaN. A value is
 * exact in BF16 and in FP16. latent is 128, 256, 384 or 512 (LATENT4_ROW_BYTES:
 * 224, 288, 352, 416). Rows are addressed by physical row number, as BF16 rows are.
 *
 * Rounding to 4 bits, per 16 values v: s = e4m3(max |v| / 6), at least 2^-9 and at
 * most 448, and code = e2m1(v / s), both to the nearest, ties to the even code, past
 * 6 the largest. With s from 2^-6 on and max |v| up to 2688 values are off by at most
 * s / 4 where |v| <= 2 s, s / 2 where |v| <= 4 s and s above, where the largest is at
 * most 6.375 s. Scales below 2^-6 are 2^-9 apart, so there the largest may be 9 s and off
 * by 3 s; values below s / 4 become zero (below 2^-11 in any case), and values past 2688
 * become 2688. A cache whose values are that small or large is better held times a
 * power of two: as part of `weight`, taken out again of the query's latent part and of
 * the outputs. Sixteen values of which one is NaN or infinite read back as NaN.
 */
#ifndef LATENT4_H
#define LATENT4_H

#include <stddef.h>
#include <stdint.h>

#include "latent_bf16.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LATENT4_ROW_BYTES(latent) (160 + (latent) / 2)

/*
 * Appends tokens to the cache, as latent_bf16_append: for token t with row slots[t]
 * in [0, cache_rows)
 *     codes, scales  of  weight ? norm(latents[t]) : latents[t]
 *     key part       =   rotate(key_rope[t], positions[t])
 * and, for every token when query_rope is given, query[t][h][latent .. ) =
 * rotate(query_rope[t][h], positions[t]). The norm x * weight / sqrt(mean(x^2) + eps)
 * is carried to about 2^-44 (pairs of floats; exactly where it is a number of few
 * digits) and rounded to 4 bits once, so the codes are those of exact arithmetic, for
 * rows of any size down to the least BF16 values, with eps = 0 too (|weight| up to 2^60:
 * past that x * weight may overflow). Sums of squares that overflow 32 bits (2^128) read back as NaN, and so do rows
 * of zeros with eps = 0. eps, at least 0, is a double: as a float it would already move
 * values next to a border.
 *
 * cache          device bytes, row r at cache + r * cache_stride; 32-byte aligned,
 *                cache_stride a multiple of 32, >= LATENT4_ROW_BYTES(latent).
 * Everything else as in latent_bf16_append_t, errors too.
 */
typedef struct {
    uint8_t *cache;
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
    double eps;
} latent4_append_t;

topk_status_t latent4_append(const latent4_append_t *args, void *stream);

/*
 * Reads rows back: out[i] = the latent + LATENT_ROPE values of cache row rows[i],
 * exactly; zeros where rows[i] lies outside [0, cache_rows).
 *
 * cache, cache_stride   as above.
 * rows                  device int32 [count].
 * out                   device BF16 [count], rows out_stride apart: 16-byte aligned,
 *                       out_stride a multiple of 8, >= latent + LATENT_ROPE.
 * Errors: TOPK_ERR_ARG (null pointer, negative count), TOPK_ERR_WIDTH (latent, a
 * stride below its row), TOPK_ERR_ALIGN, TOPK_ERR_CUDA.
 */
topk_status_t latent4_rows(const uint8_t *cache, int64_t cache_stride, int32_t cache_rows, int32_t latent,
                           const int32_t *rows, int32_t count, uint16_t *out, int64_t out_stride, void *stream);

/*
 * Attention over rows in 4 bits: the formulas, fields, empty rows and errors of
 * latent_bf16_attend_t, with the cache as above. Values and weights go to the tensor
 * cores as FP16 (values are exact there), a query row's latent part as FP16 times a
 * power of two of its own, which brings its largest finite value to [2^8, 2^9): query
 * values below 2^-22 of the row's largest are rounded to 2^-33 of it. Products are
 * summed in 32 bits in that unit: key parts past 2^96 may overflow them.
 */
typedef struct {
    const uint16_t *query;
    int64_t query_token_stride, query_head_stride;
    const uint8_t *cache;
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
} latent4_attend_t;

topk_status_t latent4_attend_selected(const latent4_attend_t *args, void *stream);
topk_status_t latent4_attend_paged(const latent4_attend_t *args, void *stream);

/* As latent_bf16_attend_workspace and latent_bf16_workspace_bytes, for these calls. */
int64_t latent4_attend_workspace(const latent4_attend_t *args, int32_t paged);
int64_t latent4_workspace_bytes(void);

#ifdef __cplusplus
}
#endif

#endif /* LATENT4_H */
