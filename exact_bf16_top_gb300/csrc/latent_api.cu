// Host side of the latent-cache operators: argument checks and the C ABI
// declared in latent_bf16.h and latent4.h.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "latent.h"

namespace topk::latent {

namespace {

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
bool bad_latent(int32_t v) { return v != 128 && v != 256 && v != 384 && v != 512; }

// What either cache's rows have to keep to, in units of its type.
bool narrow(const uint16_t *, int64_t stride, int32_t latent) { return stride < latent + LATENT_ROPE; }
bool narrow(const uint8_t *, int64_t stride, int32_t latent) { return stride < LATENT4_ROW_BYTES(latent); }
bool misaligned(const uint16_t *cache, int64_t stride) { return off16(cache) || (stride & 7); }
bool misaligned(const uint8_t *cache, int64_t stride) {
    return ((reinterpret_cast<uintptr_t>(cache) | static_cast<uintptr_t>(stride)) & 31u) != 0;
}

template <class Append>
topk_status_t check_append(const Append *a) {
    if (!a || a->tokens < 0 || a->tokens > (1 << 27) || a->cache_rows < 0) return TOPK_ERR_ARG;
    if (bad_latent(a->latent)) return TOPK_ERR_WIDTH;
    if (a->tokens == 0) return TOPK_OK;
    if ((!a->cache && a->cache_rows > 0) || !a->latents || !a->key_rope || !a->positions || !a->cos_sin || !a->slots)
        return TOPK_ERR_ARG;
    if (a->max_positions < 1) return TOPK_ERR_ARG;
    const int64_t dim = a->latent + LATENT_ROPE;
    if (narrow(a->cache, a->cache_stride, a->latent) || a->latents_stride < a->latent || a->key_stride < LATENT_ROPE)
        return TOPK_ERR_WIDTH;
    if (misaligned(a->cache, a->cache_stride) || off16(a->latents) || off16(a->key_rope) || off16(a->cos_sin) ||
        off16(a->weight) || off4(a->positions) || off4(a->slots))
        return TOPK_ERR_ALIGN;
    if ((a->latents_stride | a->key_stride) & 7) return TOPK_ERR_ALIGN;
    if (a->query_rope || a->query) {
        if (!a->query || !a->query_rope) return TOPK_ERR_ARG;
        if (a->heads < 1 || a->heads > LATENT_MAX_HEADS) return TOPK_ERR_ARG;
        if (off16(a->query) || off16(a->query_rope)) return TOPK_ERR_ALIGN;
        if ((a->query_token_stride | a->query_head_stride | a->query_rope_token_stride |
             a->query_rope_head_stride) & 7)
            return TOPK_ERR_ALIGN;
        if (a->query_head_stride < 0 || a->query_token_stride < 0 || a->query_rope_head_stride < 0 ||
            a->query_rope_token_stride < 0)
            return TOPK_ERR_WIDTH;
        // Output rows must be apart (input rows may be broadcast: stride 0).
        if ((a->heads > 1 && a->query_head_stride < dim) || (a->tokens > 1 && a->query_token_stride < dim))
            return TOPK_ERR_WIDTH;
    }
    return TOPK_OK;
}

template <class Attend>
topk_status_t check_attend(const Attend *a, bool paged) {
    if (!a || a->tokens < 0 || a->cache_rows < 0) return TOPK_ERR_ARG;
    if (bad_latent(a->latent)) return TOPK_ERR_WIDTH;
    if (a->heads < 1 || a->heads > LATENT_MAX_HEADS || !std::isfinite(a->scale)) return TOPK_ERR_ARG;
    if (static_cast<int64_t>(a->tokens) * a->heads > INT32_MAX) return TOPK_ERR_ARG;
    if (paged) {
        if (a->width < 0 || a->width > LATENT_MAX_LENGTH) return TOPK_ERR_WIDTH;
        if (a->page_size < 1 || (a->page_size & (a->page_size - 1)) || a->block_rows < a->page_size ||
            a->rows_per_request < 1)
            return TOPK_ERR_ARG;
        if (a->table_stride < (static_cast<int64_t>(a->width) + a->page_size - 1) / a->page_size) return TOPK_ERR_ARG;
    } else if (a->k < 0 || a->k > LATENT_MAX_LENGTH) {
        return TOPK_ERR_ARG;
    } else if (a->selected_stride < a->k) {
        return TOPK_ERR_WIDTH;
    }
    if (a->tokens == 0) return TOPK_OK;
    if (!a->query || (!a->cache && a->cache_rows > 0) || !a->out) return TOPK_ERR_ARG;
    if (paged ? (!a->valid_len || !a->block_table) : (!a->selected && a->k > 0)) return TOPK_ERR_ARG;
    if (narrow(a->cache, a->cache_stride, a->latent) || a->query_head_stride < 0 || a->query_token_stride < 0)
        return TOPK_ERR_WIDTH;
    if (off16(a->query) || misaligned(a->cache, a->cache_stride) || off16(a->out) || off16(a->workspace) ||
        off4(a->lse) || off4(a->selected) || off4(a->valid_len) || off4(a->block_table))
        return TOPK_ERR_ALIGN;
    if ((a->query_token_stride | a->query_head_stride) & 7) return TOPK_ERR_ALIGN;
    return TOPK_OK;
}

template <class Attend>
AttendParams params_of(const Attend *a, bool paged) {
    AttendParams p = {};
    p.query = a->query;
    p.query_token_stride = a->query_token_stride;
    p.query_head_stride = a->query_head_stride;
    p.cache = a->cache;
    p.cache_stride = a->cache_stride;
    p.paged = paged ? 1 : 0;
    p.selected = paged ? nullptr : a->selected;
    p.selected_stride = a->selected_stride;
    p.valid_len = a->valid_len;
    p.table = a->block_table;
    p.out = a->out;
    p.lse = a->lse;
    p.cache_rows = a->cache_rows;
    p.tokens = a->tokens;
    p.heads = a->heads;
    p.latent = a->latent;
    p.k = a->k;
    p.width = a->width;
    p.table_stride = a->table_stride;
    if (paged)
        while ((1 << p.page_shift) < a->page_size) ++p.page_shift;
    p.block_rows = a->block_rows;
    p.rows_per_request = paged ? a->rows_per_request : 1;
    p.scale = a->scale;
    p.workspace = a->workspace;
    return p;
}

int64_t workspace_of(const latent_bf16_attend_t *, const AttendParams &p) { return attend_workspace(p); }
int64_t workspace_of(const latent4_attend_t *, const AttendParams &p) { return attend4_workspace(p); }
cudaError_t launch(const latent_bf16_attend_t *, const AttendParams &p, cudaStream_t s) { return launch_attend(p, s); }
cudaError_t launch(const latent4_attend_t *, const AttendParams &p, cudaStream_t s) { return launch_attend4(p, s); }

template <class Attend>
topk_status_t attend(const Attend *a, bool paged, void *stream) {
    const topk_status_t st = check_attend(a, paged);
    if (st != TOPK_OK || a->tokens == 0) return st;
    const AttendParams p = params_of(a, paged);
    const int64_t need = workspace_of(a, p);
    if (need < 0) return TOPK_ERR_CUDA;
    if (need > 0 && (!a->workspace || a->workspace_bytes < need)) return TOPK_ERR_ARG;
    return launch(a, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TOPK_OK : TOPK_ERR_CUDA;
}

template <class Attend>
int64_t workspace(const Attend *a, int32_t paged) {
    if (check_attend(a, paged != 0) != TOPK_OK) return -1;
    return a->tokens == 0 ? 0 : workspace_of(a, params_of(a, paged != 0));
}

bool multiprocessors(int &sms) {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
           cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

topk_status_t status_of(cudaError_t e) { return e == cudaSuccess ? TOPK_OK : TOPK_ERR_CUDA; }

}  // namespace

}  // namespace topk::latent

extern "C" {

using namespace topk::latent;

topk_status_t latent_bf16_append(const latent_bf16_append_t *args, void *stream) {
    const topk_status_t st = check_append(args);
    int sms = 0;
    if (st != TOPK_OK || args->tokens == 0) return st;
    if (!multiprocessors(sms)) return TOPK_ERR_CUDA;
    return status_of(launch_append(*args, sms, static_cast<cudaStream_t>(stream)));
}

topk_status_t latent_bf16_attend_selected(const latent_bf16_attend_t *args, void *stream) {
    return attend(args, false, stream);
}

topk_status_t latent_bf16_attend_paged(const latent_bf16_attend_t *args, void *stream) {
    return attend(args, true, stream);
}

int64_t latent_bf16_attend_workspace(const latent_bf16_attend_t *args, int32_t paged) {
    return workspace(args, paged);
}

int64_t latent_bf16_workspace_bytes(void) { return workspace_bytes(); }

topk_status_t latent4_append(const latent4_append_t *args, void *stream) {
    const topk_status_t st = check_append(args);
    int sms = 0;
    if (st != TOPK_OK || args->tokens == 0) return st;
    if (!multiprocessors(sms)) return TOPK_ERR_CUDA;
    return status_of(launch_append4(*args, sms, static_cast<cudaStream_t>(stream)));
}

topk_status_t latent4_rows(const uint8_t *cache, int64_t cache_stride, int32_t cache_rows, int32_t latent,
                           const int32_t *rows, int32_t count, uint16_t *out, int64_t out_stride, void *stream) {
    if (count < 0 || cache_rows < 0) return TOPK_ERR_ARG;
    if (bad_latent(latent)) return TOPK_ERR_WIDTH;
    if (count == 0) return TOPK_OK;
    if ((!cache && cache_rows > 0) || !rows || !out) return TOPK_ERR_ARG;
    if (narrow(cache, cache_stride, latent) || out_stride < latent + LATENT_ROPE) return TOPK_ERR_WIDTH;
    if (misaligned(cache, cache_stride) || off4(rows) || off16(out) || (out_stride & 7)) return TOPK_ERR_ALIGN;
    int sms = 0;
    if (!multiprocessors(sms)) return TOPK_ERR_CUDA;
    return status_of(launch_rows4(cache, cache_stride, cache_rows, latent, rows, count, out, out_stride, sms,
                                  static_cast<cudaStream_t>(stream)));
}

topk_status_t latent4_attend_selected(const latent4_attend_t *args, void *stream) {
    return attend(args, false, stream);
}

topk_status_t latent4_attend_paged(const latent4_attend_t *args, void *stream) { return attend(args, true, stream); }

int64_t latent4_attend_workspace(const latent4_attend_t *args, int32_t paged) { return workspace(args, paged); }

int64_t latent4_workspace_bytes(void) { return workspace4_bytes(); }

}  // extern "C"
