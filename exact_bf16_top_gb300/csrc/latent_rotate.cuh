// What the operators that append to a latent cache share: packed BF16 values and
// the rotation by position of 64 of them by eight lanes.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "latent.h"

namespace topk::latent {

namespace {

constexpr int ROPE = LATENT_ROPE;
constexpr int APPEND_HEADS = 16;             // query heads of a unit

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

// Up to 16 of a token's query heads, eight lanes a head, four heads a round, all
// rounds' loads together. Args: either append's arguments.
template <class Args>
__device__ __forceinline__ void turn_heads(const Args &a, int32_t t, int32_t first, int32_t pos, int lane) {
    const int part = lane & 7;
    const bool interleaved = a.interleaved != 0;
    const int32_t h0 = first + (lane >> 3);
    const uint16_t *from = a.query_rope + t * a.query_rope_token_stride;
    uint4 v[APPEND_HEADS / 4];
#pragma unroll
    for (int i = 0; i < APPEND_HEADS / 4; ++i)
        v[i] = h0 + 4 * i >= a.heads
                   ? make_uint4(0, 0, 0, 0)
                   // (an ordinary load: it may be where the unit's result goes)
                   : reinterpret_cast<const uint4 *>(from + (h0 + 4 * i) * a.query_rope_head_stride)[part];
    pos = pos < 0 ? 0 : pos >= a.max_positions ? a.max_positions - 1 : pos;
    const Turn turn(a.cos_sin + static_cast<int64_t>(pos) * ROPE, part, interleaved);
    uint16_t *to = a.query + t * a.query_token_stride + a.latent;
#pragma unroll
    for (int i = 0; i < APPEND_HEADS / 4; ++i) {
        const uint4 r = turn(v[i], part, interleaved);
        if (h0 + 4 * i < a.heads) reinterpret_cast<uint4 *>(to + (h0 + 4 * i) * a.query_head_stride)[part] = r;
    }
}

}  // namespace

}  // namespace topk::latent
