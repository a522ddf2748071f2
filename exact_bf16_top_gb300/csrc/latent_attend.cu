// Attention over latent cache rows: a plain kernel.

#include <cuda_bf16.h>

#include "common.cuh"
#include "latent.h"

namespace topk::latent {

namespace {

constexpr int NT = 256;
constexpr int HG = 8;          // heads of one CTA
constexpr int KEYS = 32;       // cache rows of one tile
constexpr int PAD = 8;

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// One CTA per (token, eight heads): tiles of 32 cache rows in shared memory, one
// thread per (head, row) score, one warp per head for the running maximum and
// sum, two latent columns per thread for the weighted sum.
__global__ void __launch_bounds__(NT) attend_kernel(const AttendParams p) {
    grid_dependents_release();
    grid_dependency_wait();
    extern __shared__ __align__(16) char smem[];
    const int dim = p.latent + LATENT_ROPE, pitch = dim + PAD;
    uint16_t *keys = reinterpret_cast<uint16_t *>(smem);
    float *q = reinterpret_cast<float *>(keys + KEYS * pitch);
    float *prob = q + HG * dim;
    float *fac = prob + HG * KEYS;
    int32_t *rows = reinterpret_cast<int32_t *>(fac + HG);
    const int groups = (p.heads + HG - 1) / HG;
    const int t = blockIdx.x / groups, h0 = (blockIdx.x % groups) * HG;
    const int tid = threadIdx.x, head = tid >> 5, lane = tid & 31;
    for (int i = tid; i < HG * dim; i += NT) {
        const int h = h0 + i / dim;
        q[i] = h < p.heads ? bf(p.query[t * p.query_token_stride + h * p.query_head_stride + i % dim]) * p.scale : 0.0f;
    }
    const int request = !p.paged ? 0 : t / p.rows_per_request;
    int len = !p.paged ? p.k : p.valid_len[t];
    if (p.paged) len = len < 0 ? 0 : len > p.width ? p.width : len;
    float m = -INFINITY, l = 0.0f;       // of head `head`
    float acc[HG][2] = {};
    for (int base = 0; base < len; base += KEYS) {
        __syncthreads();
        if (tid < KEYS) {
            int64_t r = -1;
            const int i = base + tid;
            if (i < len)
                r = !p.paged ? p.selected[t * p.selected_stride + i]
                               : static_cast<int64_t>(p.table[static_cast<int64_t>(request) * p.table_stride +
                                                              (i >> p.page_shift)]) * p.block_rows +
                                     (i & ((1 << p.page_shift) - 1));
            rows[tid] = r >= 0 && r < p.cache_rows ? static_cast<int32_t>(r) : -1;
        }
        __syncthreads();
        const int vecs = dim / 8;
        for (int i = tid; i < KEYS * vecs; i += NT) {
            const int j = i / vecs, c = i % vecs;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (rows[j] >= 0) v = reinterpret_cast<const uint4 *>(p.cache + rows[j] * p.cache_stride)[c];
            reinterpret_cast<uint4 *>(keys + j * pitch)[c] = v;
        }
        __syncthreads();
        float s = -INFINITY;
        if (rows[lane] >= 0) {
            float a = 0.0f;
            for (int d = 0; d < dim; ++d) a += q[head * dim + d] * bf(keys[lane * pitch + d]);
            s = a;
        }
        float mx = s;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        mx = fmaxf(m, mx);
        const float ref = mx == -INFINITY ? 0.0f : mx;
        const float e = rows[lane] >= 0 ? expf(s - ref) : 0.0f;
        float sum = e;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float f = m == -INFINITY ? 0.0f : expf(m - ref);
        l = l * f + sum;
        m = mx;
        prob[head * KEYS + lane] = e;
        if (lane == 0) fac[head] = f;
        __syncthreads();
        if (2 * tid < p.latent) {
            for (int h = 0; h < HG; ++h) {
                float a0 = acc[h][0] * fac[h], a1 = acc[h][1] * fac[h];
                for (int j = 0; j < KEYS; ++j) {
                    a0 += prob[h * KEYS + j] * bf(keys[j * pitch + 2 * tid]);
                    a1 += prob[h * KEYS + j] * bf(keys[j * pitch + 2 * tid + 1]);
                }
                acc[h][0] = a0;
                acc[h][1] = a1;
            }
        }
    }
    __syncthreads();
    if (lane == 0) {
        fac[head] = l == 0.0f ? 0.0f : 1.0f / l;   // NaN stays NaN
        if (p.lse && h0 + head < p.heads)
            p.lse[static_cast<int64_t>(t) * p.heads + h0 + head] = l == 0.0f ? -INFINITY : m + logf(l);
    }
    __syncthreads();
    if (2 * tid < p.latent)
        for (int h = 0; h < HG && h0 + h < p.heads; ++h)
            reinterpret_cast<__nv_bfloat162 *>(p.out + (static_cast<int64_t>(t) * p.heads + h0 + h) * p.latent)[tid] =
                __floats2bfloat162_rn(acc[h][0] * fac[h], acc[h][1] * fac[h]);
}

}  // namespace

cudaError_t launch_attend(const AttendParams &p, cudaStream_t stream) {
    const int dim = p.latent + LATENT_ROPE;
    const size_t smem = KEYS * (dim + PAD) * 2 + (HG * dim + HG * KEYS + HG) * 4 + KEYS * 4;
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&attend_kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int64_t blocks = static_cast<int64_t>(p.tokens) * ((p.heads + HG - 1) / HG);
    attend_kernel<<<static_cast<unsigned>(blocks), NT, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace topk::latent
