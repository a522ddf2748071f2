// Appending tokens to the 4-bit latent cache (norm, rounding to 4 bits, rotation,
// the write to the token's slot, and the rotation of the token's query parts, in one
// launch), and reading rows back as BF16.

#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "latent_rotate.cuh"

namespace topk::latent {

namespace {

constexpr int NT = 256;
constexpr uint32_t FULL = 0xFFFFFFFFu;

// A number as the sum of two floats, the second at most half a unit of the first.
struct Two {
    float hi, lo;
};

// a + b of two such numbers; exact but for the last product of errors (2^-48).
__device__ __forceinline__ Two add(Two a, Two b) {
    const float s = __fadd_rn(a.hi, b.hi), d = __fadd_rn(s, -a.hi);
    const float e = __fadd_rn(__fadd_rn(a.hi, -__fadd_rn(s, -d)), __fadd_rn(b.hi, -d));
    return {s, __fadd_rn(__fadd_rn(a.lo, b.lo), e)};
}

// a / n of such a number and a small whole one, over = 1 / n: to 2^-47, and exactly where
// the quotient is a float.
__device__ __forceinline__ Two share(Two a, float n, float over) {
    const float h = __fmul_rn(a.hi, over);
    return {h, __fmul_rn(__fadd_rn(__fmaf_rn(-h, n, a.hi), a.lo), over)};
}

// sqrt(x), and 1 / sqrt(x) as a float. Two of Newton's steps on the hardware's estimate,
// each from the exact remainder: to 2^-46, and exactly where the root is a float (a row
// whose norm is a number of few digits has values that lie on the borders).
struct Root {
    Two g;
    float over;
};

__device__ __forceinline__ Root root(Two x) {
    const float y = rsqrtf(x.hi), half = 0.5f * y;
    const float h = __fmul_rn(x.hi, y);      // (NaN of an infinite x and of 0)
    const float hi = __fmaf_rn(__fadd_rn(__fmaf_rn(-h, h, x.hi), x.lo), half, h);
    return {{hi, __fmul_rn(__fadd_rn(__fmaf_rn(-hi, hi, x.hi), x.lo), half)}, y};
}

// xw / g, rounded to odd: what is not a float becomes the neighbour whose last bit is 1.
// Rounded further to any format of two bits less it gives what the exact quotient would,
// ties included. The quotient is rounded to nearest first, for which of its neighbours the
// remainder then points to is certain (product with a reciprocal of two parts, which may
// be off by 1.5 units, took the wrong side of a border now and then); -0 stays -0.
__device__ __forceinline__ float over_odd(float xw, const Root &r) {
    const float q = __fmul_rn(xw, r.over);
    const float v = __fmaf_rn(__fmaf_rn(q, r.g.lo, __fmaf_rn(q, r.g.hi, -xw)), -r.over, q);
    const float m = __fmaf_rn(v, r.g.lo, __fmaf_rn(v, r.g.hi, -xw));   // v g - xw
    uint32_t b = __float_as_uint(v);
    if (m != 0.0f && !(b & 1u)) b += (__float_as_uint(m) ^ b) >> 31 ? 1u : FULL;   // (away from m; NaN stays NaN)
    return __uint_as_float(b);
}

// The larger of m and |v|, NaN if one of them is.
__device__ __forceinline__ float largest(float m, float v) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(m), "f"(fabsf(v)));
    return y;
}

// v / s rounded to nearest, by Markstein's correction of a quotient from the rounded
// reciprocal: the remainder is exact, and its share of s is taken off with one rounding
// (of that sign, so that -0 stays -0).
__device__ __forceinline__ float quotient(float v, float s, float over_s) {
    const float q = __fmul_rn(v, over_s);
    return __fmaf_rn(__fmaf_rn(q, s, -v), -over_s, q);
}

// A block's 16 values to its scale's e4m3 byte and 16 codes. Both quotients are rounded
// to nearest, which no float near a border can be moved onto it by: a border is the
// quotient of a float of few bits, its neighbours' quotients are floats of their own.
__device__ __forceinline__ uint32_t to_codes(const float (&v)[16], uint32_t (&code)[2]) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) most = largest(most, v[i]);
    uint32_t s8 = 0x7Fu;                     // NaN: one of the values is not finite
    float s = 1.0f;
    if (most <= FLT_MAX) {
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(__fdiv_rn(most, 6.0f)));
        s8 = max(static_cast<uint32_t>(two) & 0xFFu, 1u);
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(s8)));
        s = __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
    }
    const float over_s = __frcp_rn(s);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = s8 == 0x7Fu ? 0.0f : quotient(v[8 * w + i], s, over_s);
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(code[w])
            : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    }
    return s8;
}

struct Norm {
    float over;                              // 1 / latent
    Two eps;
    Two part;                                // eps = part * 4^power, part in [1, 4)
    int32_t power;
};

// Mean squares plus eps between these are as exact as what follows: no square, remainder
// or product of the norm that counts is below the least float. A row outside them is
// scaled by a power of two first.
constexpr float LEAST_MEAN = 0x1p-60f, MOST_MEAN = 0x1p100f;

// Brings a row's largest value, or the root of eps where that is larger, to [1, 2), exactly
// (a lane's 16 values), and returns what eps is then.
__device__ __forceinline__ Two scale_row(float (&v)[16], const Norm &norm) {
    int32_t field = 127 + norm.power;        // exponent fields
#pragma unroll
    for (int i = 0; i < 16; ++i) field = max(field, static_cast<int32_t>(__float_as_uint(v[i]) >> 23 & 0xFFu));
    field = min(max(__reduce_max_sync(FULL, field), 1), 253);
    const float by = __uint_as_float(static_cast<uint32_t>(254 - field) << 23);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(v[i], by);
    const int32_t up = norm.power + 127 - field;
    const float f = up < -60 ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 + 2 * min(up, 60)) << 23);
    return {__fmul_rn(norm.part.hi, f), __fmul_rn(norm.part.lo, f)};
}

// One warp per unit of work, as in the BF16 form: a token's cache row (a block of 16
// values that share a scale per lane, so that none of the rounding crosses lanes), or
// up to 16 of a token's query heads. The sum of squares and the norm are pairs of
// floats: a value next to a border of 4 bits takes the side that exact arithmetic
// gives it, whatever the order of the sums. Bound by that arithmetic: 8191 tokens of 512
// values 8.9 us with the norm, 4.7 without (15 MB either way); with 16 heads' queries
// (another 34 MB) 13.8 and 10.6. (Products with a reciprocal in two parts took 0.6 us less,
// and the wrong side of some borders; by divisions and with one chain of sums the rows took
// 1.1 more.) One token 2.0 us: the launch and two rounds of loads.
__global__ void __launch_bounds__(NT) append4_kernel(const latent4_append_t a, uint32_t units, uint32_t groups,
                                                     const Norm norm) {
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
            turn_heads(a, t, static_cast<int32_t>(q - t * groups) * APPEND_HEADS, pos, lane);
            continue;
        }
        pos = pos < 0 ? 0 : pos >= a.max_positions ? a.max_positions - 1 : pos;
        const float *cs = a.cos_sin + static_cast<int64_t>(pos) * ROPE;
        const int32_t slot = a.slots[t];
        const bool mine = lane < a.latent / 16;
        uint4 x[2] = {}, w[2] = {};
        if (mine) {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.latents + t * a.latents_stride) + 2 * lane;
            x[0] = __ldg(src);
            x[1] = __ldg(src + 1);
            if (a.weight) {
                w[0] = __ldg(reinterpret_cast<const uint4 *>(a.weight) + 2 * lane);
                w[1] = __ldg(reinterpret_cast<const uint4 *>(a.weight) + 2 * lane + 1);
            }
        }
        const uint4 k = __ldg(reinterpret_cast<const uint4 *>(a.key_rope + t * a.key_stride) + part);
        if (slot < 0 || slot >= a.cache_rows) continue;
        uint8_t *row = a.cache + static_cast<int64_t>(slot) * a.cache_stride;
        const uint32_t *b = &x[0].x, *g = &w[0].x;
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = lo_f(b[i]);
            v[2 * i + 1] = hi_f(b[i]);
        }
        if (a.weight) {
            Two mean, eps = norm.eps;
#pragma unroll 1
            for (bool scaled = false;; scaled = true) {
                Two sums[4];                 // (squares that count are exact; four sums side by side)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const Two square = {__fmul_rn(v[i], v[i]), 0.0f};
                    sums[i % 4] = i < 4 ? square : add(sums[i % 4], square);
                }
                Two sum = add(add(sums[0], sums[1]), add(sums[2], sums[3]));
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    sum = add(sum, {__shfl_xor_sync(FULL, sum.hi, o), __shfl_xor_sync(FULL, sum.lo, o)});
                mean = add(share(sum, static_cast<float>(a.latent), norm.over), eps);
                const bool fine = (mean.hi >= LEAST_MEAN && mean.hi <= MOST_MEAN) || !(sum.hi <= FLT_MAX);
                if (scaled || __all_sync(FULL, fine)) [[likely]] break;   // (a sum that overflows stays so: NaN)
                eps = scale_row(v, norm);
            }
            const Root r = root(mean);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[2 * i] = over_odd(__fmul_rn(v[2 * i], lo_f(g[i])), r);
                v[2 * i + 1] = over_odd(__fmul_rn(v[2 * i + 1], hi_f(g[i])), r);
            }
        }
        uint32_t code[2];
        const uint32_t s8 = to_codes(v, code);
        if (mine) {
            reinterpret_cast<uint2 *>(row)[lane] = make_uint2(code[0], code[1]);
            row[a.latent / 2 + 2 * ROPE + lane] = static_cast<uint8_t>(s8);
        }
        const uint4 turned = Turn(cs, part, interleaved)(k, part, interleaved);
        if (lane < 8) reinterpret_cast<uint4 *>(row + a.latent / 2)[part] = turned;
    }
}

// Eight codes and their scale as eight BF16 values.
__device__ __forceinline__ uint4 from_codes(uint32_t w, __half2 scale) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(__hmul2(*reinterpret_cast<const __half2 *>(&h[i]), scale));
        r[i] = pack(f.x, f.y);               // (at most six significant bits: nothing is rounded)
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// R rows of a warp at a time, all their loads together: 16 values of one scale per lane,
// the key part by eight lanes. Bound by DRAM where rows are many (131071 rows 35.5 us,
// 5.8 TB/s), by the launch and two rounds of loads else (2048 rows 2.4 us).
template <int R>
__global__ void __launch_bounds__(NT) rows4_kernel(const uint8_t *__restrict__ cache, int64_t cache_stride,
                                                   int32_t cache_rows, int32_t latent, const int32_t *__restrict__ rows,
                                                   int32_t count, uint16_t *__restrict__ out, int64_t out_stride) {
    grid_dependents_release();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const bool mine = lane < latent / 16;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (NT / 32) * R;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * (NT / 32) + (threadIdx.x >> 5)) * R; i < count; i += step) {
        int32_t r[R];
        uint2 code[R];
        uint32_t s8[R];
        uint4 key[R];
#pragma unroll
        for (int k = 0; k < R; ++k) r[k] = i + k < count ? __ldg(rows + i + k) : -1;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            code[k] = make_uint2(0, 0);
            s8[k] = 0;
            key[k] = make_uint4(0, 0, 0, 0);
            if (r[k] >= 0 && r[k] < cache_rows) {
                const uint8_t *row = cache + r[k] * cache_stride;
                if (mine) {
                    code[k] = __ldg(reinterpret_cast<const uint2 *>(row) + lane);
                    s8[k] = __ldg(row + latent / 2 + 2 * ROPE + lane);
                }
                if (lane < 8) key[k] = __ldg(reinterpret_cast<const uint4 *>(row + latent / 2) + lane);
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (i + k >= count) break;
            uint32_t s;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s) : "h"(static_cast<uint16_t>(s8[k] | s8[k] << 8)));
            const __half2 scale = *reinterpret_cast<const __half2 *>(&s);
            uint4 *to = reinterpret_cast<uint4 *>(out + (i + k) * out_stride);
            if (mine) {
                to[2 * lane] = from_codes(code[k].x, scale);
                to[2 * lane + 1] = from_codes(code[k].y, scale);
            }
            if (lane < 8) to[latent / 8 + lane] = key[k];
        }
    }
}

cudaLaunchConfig_t config(int64_t units, int sms, cudaStream_t stream, cudaLaunchAttribute *attr) {
    const int64_t want = (units + NT / 32 - 1) / (NT / 32), most = static_cast<int64_t>(sms) * (2048 / NT);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most), 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.stream = stream;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

Two two(double v) {
    const float hi = static_cast<float>(v);
    return {hi, static_cast<float>(v - hi)};
}

}  // namespace

cudaError_t launch_append4(const latent4_append_t &a, int sms, cudaStream_t stream) {
    uint32_t groups = a.query_rope ? static_cast<uint32_t>((a.heads + APPEND_HEADS - 1) / APPEND_HEADS) : 0u;
    uint32_t units = static_cast<uint32_t>(a.tokens) * (1u + groups);   // (at most 2^27 tokens: checked)
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(units, sms, stream, &attr);
    latent4_append_t arg = a;
    int at = 0;
    (void)std::frexp(a.eps, &at);            // eps in [2^(at - 1), 2^at)
    const bool some = a.eps != 0.0 && std::isfinite(a.eps);
    const int32_t power = some ? (at - 1 - ((at - 1) & 1)) / 2 : -1000;
    Norm norm = {1.0f / static_cast<float>(a.latent), two(a.eps),
                 two(some ? std::ldexp(a.eps, -2 * power) : a.eps), power};
    void *args[] = {&arg, &units, &groups, &norm};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(&append4_kernel), args);
}

cudaError_t launch_rows4(const uint8_t *cache, int64_t cache_stride, int32_t cache_rows, int32_t latent,
                         const int32_t *rows, int32_t count, uint16_t *out, int64_t out_stride, int sms,
                         cudaStream_t stream) {
    cudaLaunchAttribute attr;
    // Several rows a warp once there are three times as many as warps that run at once
    // (latent 512, four rows a warp / one: 12000 rows 5.2 / 4.9 us, 20000 7.4 / 7.0, 30000
    // 9.5 / 10.0, 60000 17.5 / 19.3, 131071 38.2 / 42.0, of a cache of 400000).
    constexpr int R = 4;
    const bool many = count > 3 * sms * (2048 / 32);
    const cudaLaunchConfig_t cfg = config(many ? (count + R - 1) / R : count, sms, stream, &attr);
    void *args[] = {&cache, &cache_stride, &cache_rows, &latent, &rows, &count, &out, &out_stride};
    return cudaLaunchKernelExC(&cfg,
                               many ? reinterpret_cast<const void *>(&rows4_kernel<R>)
                                    : reinterpret_cast<const void *>(&rows4_kernel<1>),
                               args);
}

}  // namespace topk::latent
