/*
 * page_step.h - a batch's page tables, taken one step further on the GPU: what the
 * operators of topk_bf16.h, latent_bf16.h and latent4.h take as block table, slots,
 * positions and valid lengths, made from request lengths without the host. Same
 * library, same conventions (latent_bf16.h).
 *
 * A request holds `lengths` tokens in ceil(length / page_size) pages, whose numbers
 * are the first entries of its row of the block table; pages nobody holds are a
 * stack, free_pages[0 .. free_count). A step, in the order of the requests r:
 *
 * new_tokens[r] >= 0   the request gets that many tokens (clamped to
 *     rows_per_request) after those it has, and the pages that they need beyond its
 *     own, from the top of the stack downwards. A request that the table's width has
 *     no room for is refused. So is one that needs pages when those that it and
 *     all requests before it asked for (refused for lack of pages or not) are more
 *     than the stack holds; requests that need no page are served all the same.
 * new_tokens[r] < 0    the request is finished: its length becomes 0 and its pages
 *     go back on the stack, after what the step takes from it: in the order of the
 *     requests, each one's first page first. The step after this one may take them.
 *
 * Rows are rows_per_request (q) to a request, as block tables are shared by the
 * other operators: token j of request r is row r q + j. For j < granted[r]
 *     positions = length + j,  slots = page * block_rows + position % page_size,
 *     valid_len = position + 1  (a causal chunk),
 * with `page` the table's new entry position / page_size; else (a padded row) 0, -1
 * and 0: such a row is not appended and sees nothing. A slot past 31 bits or of a
 * negative page is -1.
 *
 * Lengths that go down between steps (drafted tokens that were rejected) need `held`:
 * how many pages each request has. A request then has max(held, ceil(length /
 * page_size)) pages: one behind its last token stays its own, is used before any of
 * the stack, and goes back when the request is finished. Without `held` a request has
 * what its length says, and a page that a lowered length no longer reaches would be in
 * nobody's hands.
 */
#ifndef PAGE_STEP_H
#define PAGE_STEP_H

#include <stdint.h>

#include "topk_bf16.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PAGE_STEP_MAX_REQUESTS 32768
#define PAGE_STEP_MAX_WIDTH (1 << 30)   /* pages * page_size */

/*
 * block_table       device int32 [requests, pages], rows table_stride apart: the new
 *                   pages' entries are written, nothing else.
 * lengths           device int32 [requests], clamped to [0, pages * page_size].
 * new_tokens        device int32 [requests].
 * free_pages        device int32 [free_size]: read, and written where pages come back.
 * free_count        device int32 [1], clamped to [0, free_size].
 * next_lengths      device int32 [requests], may be `lengths` itself.
 * next_free_count   device int32 [1], may be `free_count` itself.
 * granted           device int32 [requests]: tokens that a request got (0: refused,
 *                   finished or none asked for).
 * positions, slots, valid_len   device int32 [requests * rows_per_request].
 * held              NULL, or device int32 [requests], clamped to [0, pages]: pages that
 *                   each request has, updated in place (zeros to begin with will do).
 * page_size is a power of two, block_rows >= page_size. No other overlap of what is
 * written with anything else is allowed. Pages that come back past free_size are
 * dropped (they were never taken from this stack).
 *
 * Errors: TOPK_ERR_ARG (null pointer but for held, negative count, more than
 * PAGE_STEP_MAX_REQUESTS, a bad page size, block_rows, table stride or
 * rows_per_request, requests * pages or requests * rows_per_request past 31 bits),
 * TOPK_ERR_WIDTH (pages * page_size past PAGE_STEP_MAX_WIDTH), TOPK_ERR_ALIGN,
 * TOPK_ERR_CUDA.
 */
typedef struct {
    int32_t *block_table;
    int64_t table_stride;
    const int32_t *lengths, *new_tokens;
    int32_t *free_pages;
    const int32_t *free_count;
    int32_t *next_lengths, *next_free_count, *granted, *positions, *slots, *valid_len;
    int32_t requests, pages, free_size, page_size, block_rows, rows_per_request;
    int32_t *held;
} page_step_t;

topk_status_t page_step(const page_step_t *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGE_STEP_H */
