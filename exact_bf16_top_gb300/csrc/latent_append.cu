// Appending tokens to the latent cache: norm, rotation, the write to the
// token's slot, and the rotation of the token's query parts, in one launch.

#include <cuda_bf16.h>

#include "common.cuh"
#include "latent.h"

namespace topk::latent {

namespace {

constexpr int NT = 256;
constexpr int ROPE = LATENT_ROPE;
constexpr int HEADS = 16;                    // query heads of a unit

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two values rounded to BF16 (nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The cosines and sines that turn eight consecutive values of 64, held by each
// of eight lanes (`part` = lane & 7). Interleaved: the pairs lie inside a lane's
// eight values; halves: value i pairs with i + 32, which the lane four parts
// away holds.
struct Turn {
    float c[8], s[8];   // interleaved: four of each
    __device__ __forceinline__ Turn(const float *__restrict__ cs, int part, bool interleaved) {
        const int at = interleaved ? 4 * part : 8 * (part & 3);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (interleaved && i) break;
            *reinterpret_cast<float4 *>(c + 4 * i) = __ldg(reinterpret_cast<const float4 *>(cs + at + 4 * i));
            *reinterpret_cast<float4 *>(s + 4 * i) = __ldg(reinterpret_cast<const float4 *>(cs + 32 + at + 4 * i));
        }
    }
    __device__ __forceinline__ uint4 operator()(uint4 v, int part, bool interleaved) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t r[4];
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = lo_f(w[i]), b = hi_f(w[i]);
                r[i] = pack(a * c[i] - b * s[i], a * s[i] + b * c[i]);
            }
        } else {
            const float sign = part < 4 ? -1.0f : 1.0f;   // (a cos - b sin, b cos + a sin)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w[i], 4);
                r[i] = pack(lo_f(w[i]) * c[2 * i] + sign * lo_f(o) * s[2 * i],
                            hi_f(w[i]) * c[2 * i + 1] + sign * hi_f(o) * s[2 * i + 1]);
            }
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
};

// One warp per unit of work: a token's cache row, or up to 16 of a token's query
// heads (eight lanes a head, four heads a round, all rounds' loads together).
// Each is one dependent round of loads (position, angles) and one of stores, so
// the kernel is bound by DRAM on long chunks (8191 tokens x 16 heads: 10.7 us, 5.1
// TB/s; with four heads a unit 15.2 us) and by the launch and that round on short
// ones (1 token: 1.7 us a launch in a graph, 128 tokens x 128 heads: 2.5 us).
template <int VECS>   // 16-byte vectors of the latent part per lane pair: latent / 256 rounded up
__global__ void __launch_bounds__(NT) append_kernel(const latent_bf16_append_t a, uint32_t units, uint32_t groups) {
    grid_dependents_release();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, part = lane & 7;
    const bool interleaved = a.interleaved != 0;
    const uint32_t step = gridDim.x * (NT / 32);
    for (uint32_t u = blockIdx.x * (NT / 32) + (threadIdx.x >> 5); u < units; u += step) {
        const bool key = u < static_cast<uint32_t>(a.tokens);
        const uint32_t q = u - a.tokens;
        const int32_t t = static_cast<int32_t>(key ? u : q / groups);
        int32_t pos = __ldg(a.positions + t);
        if (!key) {
            const int32_t h0 = static_cast<int32_t>(q - t * groups) * HEADS + (lane >> 3);
            const uint16_t *from = a.query_rope + t * a.query_rope_token_stride;
            uint4 v[HEADS / 4];
#pragma unroll
            for (int i = 0; i < HEADS / 4; ++i)
                v[i] = h0 + 4 * i >= a.heads
                           ? make_uint4(0, 0, 0, 0)
                           // (an ordinary load: it may be where the unit's result goes)
                           : reinterpret_cast<const uint4 *>(from + (h0 + 4 * i) * a.query_rope_head_stride)[part];
            pos = pos < 0 ? 0 : pos >= a.max_positions ? a.max_positions - 1 : pos;
            const Turn turn(a.cos_sin + static_cast<int64_t>(pos) * ROPE, part, interleaved);
            uint16_t *to = a.query + t * a.query_token_stride + a.latent;
#pragma unroll
            for (int i = 0; i < HEADS / 4; ++i) {
                const uint4 r = turn(v[i], part, interleaved);
                if (h0 + 4 * i < a.heads)
                    reinterpret_cast<uint4 *>(to + (h0 + 4 * i) * a.query_head_stride)[part] = r;
            }
            continue;
        }
        pos = pos < 0 ? 0 : pos >= a.max_positions ? a.max_positions - 1 : pos;
        const float *cs = a.cos_sin + static_cast<int64_t>(pos) * ROPE;
        const int32_t slot = a.slots[t];
        if (slot < 0 || slot >= a.cache_rows) continue;
        uint16_t *row = a.cache + static_cast<int64_t>(slot) * a.cache_stride;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.latents + t * a.latents_stride);
        const int vecs = a.latent / 8;
        uint4 x[VECS], w[VECS];
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int j = i * 32 + lane;
            x[i] = j < vecs ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
        }
        // The rotated key: lanes 0 to 7 hold it, the others a copy of it.
        const uint4 k = __ldg(reinterpret_cast<const uint4 *>(a.key_rope + t * a.key_stride) + part);
        if (a.weight) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                const int j = i * 32 + lane;
                w[i] = j < vecs ? __ldg(reinterpret_cast<const uint4 *>(a.weight) + j) : make_uint4(0, 0, 0, 0);
            }
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                const uint32_t b[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += lo_f(b[e]) * lo_f(b[e]) + hi_f(b[e]) * hi_f(b[e]);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            const float inv = 1.0f / sqrtf(sum / static_cast<float>(a.latent) + a.eps);
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                uint32_t *b = &x[i].x;
                const uint32_t *g = &w[i].x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    b[e] = pack(lo_f(b[e]) * inv * lo_f(g[e]), hi_f(b[e]) * inv * hi_f(g[e]));
            }
        }
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int j = i * 32 + lane;
            if (j < vecs) reinterpret_cast<uint4 *>(row)[j] = x[i];
        }
        const uint4 r = Turn(cs, part, interleaved)(k, part, interleaved);
        if (lane < 8) reinterpret_cast<uint4 *>(row + a.latent)[part] = r;
    }
}

}  // namespace

cudaError_t launch_append(const latent_bf16_append_t &a, int sms, cudaStream_t stream) {
    uint32_t groups = a.query_rope ? static_cast<uint32_t>((a.heads + HEADS - 1) / HEADS) : 0u;
    uint32_t units = static_cast<uint32_t>(a.tokens) * (1u + groups);   // (at most 2^27 tokens: checked)
    const int64_t want = (static_cast<int64_t>(units) + NT / 32 - 1) / (NT / 32);
    const int64_t most = static_cast<int64_t>(sms) * (2048 / NT);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most), 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    latent_bf16_append_t arg = a;
    void *args[] = {&arg, &units, &groups};
    const void *fn = a.latent <= 256 ? reinterpret_cast<const void *>(&append_kernel<1>)
                                     : reinterpret_cast<const void *>(&append_kernel<2>);
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace topk::latent
