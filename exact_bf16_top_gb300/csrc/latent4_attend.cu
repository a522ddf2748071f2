// Attention over latent cache rows in 4 bits on the tensor cores: one persistent
// kernel for both forms, dealt and joined as the BF16 rows' (latent_attend.cuh).
//
// A tile is up to 64 (token, head) rows that read the same cache rows; blocks of 128
// cache rows become FP16 on their way, once for both products:
//     scores (128 tokens x rows) = K Q^T,  weights = 2^(scores - reference),
//     sums (values x rows)      += V^T weights,   V the latent part of K.
// A thread makes FP16 of 128 values of a row (the conversion and one product are exact)
// and writes them into tensor memory, where they are the scores' left operand; others
// copy them from there into shared memory, where, read across rows, they are the
// sums'. So shared memory, which bounds the BF16 kernel, gives each block away once
// instead of twice, and the scores run at 128 rows a step, ahead of the sums.
// The key part stays BF16 and only goes to tensor memory. Warps have one job each
// (softmax, copies, conversion, issue of either product) and meet at mbarriers only.
//
// Measured, latent part 512: 32 requests x 16 heads x 16384 rows 61 us (2.6 TB/s; the
// rows in BF16 82 us), 128 tokens x 16 heads x 2048 listed rows 48 us (2.4 TB/s; 55), a
// chunk of 509 tokens x 128 heads on 9000 rows 1.42 ms (0.88 PFLOP/s; 1.20 ms). Neither
// memory nor the tensor cores nor the issue slots are full: a block takes 4000 to 5500
// cycles. With few query rows that is the time until its rows are there (converters wait
// for them 1800 to 2400 cycles a block, the warps that send for them hardly ever for a
// place; the copies' issue alone is a quarter of a block).
// With 64 it is a loop: a block's last pairs find a place only when the sums of the one
// before have read theirs, and its scores, softmax and sums come after. So where query
// rows are many the rows in BF16 are faster; these take 36 % of the memory.

#include <cuda_fp16.h>

#include <type_traits>

#include "latent_attend.cuh"

namespace topk::latent {

namespace {

// Warps, each with one job, in groups of four: softmax, query rows and outputs (one
// group, two of 64 query rows); cache rows from 4 bits to FP16 in tensor memory (two, one
// of 64 query rows); values from there to shared memory; and two warps for copies of
// cache rows as they are, two for the tensor cores (scores, sums). 96 registers each.
// (32 requests x 16 heads x 16384: 61 us; 22 warps, two senders more, have 80 registers,
// and what does not fit lies in a first-level cache of 28 KB: 71. Before the other steps:
// 24 warps with two groups for the values too 73 instead of 71, 16 warps of 128 registers
// with one group a job 72; a chunk of 509 tokens x 128 heads with one softmax group 2.05
// ms instead of 1.78.)
constexpr int NT = 640;
constexpr int KEYS = 128;                    // cache rows of a block
constexpr int CHUNK = KEYS * 128;            // bytes of a block's rows at 64 of their values
constexpr int BLOCKS = 8, TURNS = 16;        // blocks; pairs and units that have barriers of their own: more than are
                                             // under way (who waits for one may find later ones done, or earlier ones
                                             // not, and two phases of one barrier look like none)
constexpr int KEY_SLOTS = 2;                 // blocks' key parts in tensor memory
constexpr uint32_t FULL = 0xFFFFFFFFu;
// Weights are FP16 (at most 65504): the reference is set this far below the maximum and
// moves when a weight passes 2^MOST, so that the largest weight of a row is 2^8 at least
// and what FP16 rounds away below 2^-25 is less than 2^-33 of it (1 at least for scores past
// 2^27 in log2 units, whose next weights are 2^-16 and 2^-32). A move stops the sums
// until they are rescaled, so the two lie far apart (chunk of 509 tokens x 128 heads, 2^11
// and 2^15: 1565 us, 2^11 and 2^15.9: 1479, 2^8 and 2^15.9: 1430, 2^4: 1430).
constexpr float BELOW = 8.0f, MOST = 15.9f;

constexpr int HALF = 64;                     // rows of a block that are sent for together
constexpr int UNIT = HALF * 128;             // bytes of a unit as it comes: 128 bytes of each row of a half
constexpr int SCALES = HALF * 32;            // bytes of a half's scales

// How a tile of NR rows uses the memories: pairs of 64-value chunks in shared memory
// (sums) and tensor memory (scores), blocks of weights and of scores, units on their way.
template <int NR>
struct Shape {
    static constexpr int GROUPS = NR == 64 ? 2 : 1, CONVERT = 3 - GROUPS, SOFT = 128 * GROUPS;
    static constexpr int CONVERT_WARP = SOFT / 32, COPY_WARP = CONVERT_WARP + 4 * CONVERT, SEND_WARP = COPY_WARP + 4,
                         SCORES_WARP = SEND_WARP + 2, SUMS_WARP = SCORES_WARP + 1;
    static_assert(NT == 32 * (SUMS_WARP + 1));
    static constexpr int PAIRS = 3, A_PAIRS = NR == 64 ? 2 : 4;
    static constexpr int WEIGHTS = NR == 64 ? 1 : 2, SCORES = NR == 64 ? 1 : 2;
    static constexpr int UNITS = NR == 64 ? 2 : 3, SCALE_SLOTS = NR == 64 ? 1 : 2;
    static constexpr uint32_t O_COL = 0, S_COL = 4 * NR, A_COL = S_COL + SCORES * NR, K_COL = A_COL + A_PAIRS * 64;
    static constexpr uint32_t RING = UNITS * UNIT + SCALE_SLOTS * SCALES, RAW = KEYS / HALF * RING;
    static constexpr uint32_t RINGS = (2 * PAIRS + WEIGHTS) * CHUNK + RAW;
    static_assert(K_COL + KEY_SLOTS * 32 <= 512);
    // Places, what waits in registers and tensor memory hold a block: its scores never wait for its own sums.
    static_assert(PAIRS + 1 + A_PAIRS > LATENT_MAX / 128);
    // A cluster's parts lie where the rings were, and what weighs them behind.
    static_assert(RINGS >= NR * LATENT_MAX * sizeof(float) + ROWS * MAX_CLUSTER * sizeof(float));
};

struct Ctrl : Schedule<NT> {
    u64 unit_full[2][TURNS], unit_empty[2][3]; // a half's unit is in / read
    u64 scales_full[2][2], scales_empty[2][2]; // a half's scales are in (boxes: with the first values) / read
    u64 a_full[4], a_done[TURNS];              // a pair is in tensor memory / its scores are added and it is copied
    u64 pair_full[4], summed[TURNS];           // a pair is in shared memory / its sums are added
    u64 key_full[KEY_SLOTS], key_done[BLOCKS]; // a block's key part is in tensor memory / its scores are added
    u64 s_full[2], s_empty[2];                 // scores written / read
    u64 row_full[BLOCKS];                      // a block's marks are in
    u64 p_full[BLOCKS], o_done[BLOCKS];        // a block's weights are in / its sums are added
    u64 q_full;                                // a tile's query rows are in
    u64 drain[2];
    uint32_t tmem;
    volatile uint32_t abort;
    alignas(16) float ref[ROWS];               // reference (log2), LOWEST at first; +inf: a row that sees nothing here
    alignas(16) float factor[ROWS];
    alignas(16) float unit[ROWS];              // scores in log2 units: times this
    float l[ROWS];
    int32_t lim[ROWS];                         // tokens a row may see
    float across[4][ROWS];
    uint32_t marks[BLOCKS][KEYS / 32];         // which rows of a block there are
    uint32_t bad[4][KEYS / 32];                // which rows of a pair in tensor memory have a scale of NaN
};

using Cursor = CursorOf<KEYS>;
using RowList = RowListOf<KEYS>;

template <int NR>
__host__ __device__ constexpr uint32_t query_bytes(int latent) {
    return static_cast<uint32_t>((latent / 64 + 1) * NR * 128);
}
template <int NR>
constexpr bool fits() {
    return 1024 + query_bytes<NR>(LATENT_MAX) + Shape<NR>::RINGS + sizeof(Ctrl) <= SMEM;
}
static_assert(fits<16>() && fits<32>() && fits<64>());

// As mbar_wait() and wait() where there is mostly nothing to wait for: few instructions
// and branches that a warp takes as one (the time of a block goes to instructions and
// not to what they do: without the conversions, or the exponentials, or either product,
// it took a few percent less).
__device__ __forceinline__ void await(u64 *bar, uint32_t parity, Ctrl &c) {
    if (!mbar_try_wait(bar, parity & 1u)) [[unlikely]] mbar_wait(bar, parity & 1u, &c.abort);
}

__device__ __forceinline__ void await_warp(u64 *bar, uint32_t parity, Ctrl &c) {
    if (__all_sync(FULL, mbar_try_wait(bar, parity & 1u))) [[likely]] return;
    const uint64_t t0 = global_timer_ns();
    while (!__all_sync(FULL, mbar_try_wait(bar, parity & 1u) || c.abort))
        if (__any_sync(FULL, global_timer_ns() - t0 > WAIT_LIMIT_NS)) {
            c.abort = 1u;
            atomicOr(&g_device_status, ERR_WAIT);
        }
}

// An arrival by a warp's first lane, without a branch.
__device__ __forceinline__ void arrive_one(u64 *bar, int lane) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t@p mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(
            smem_addr(bar)),
        "r"(lane)
        : "memory");
}

__device__ __forceinline__ void store_vec(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void tc_mma_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ void tc_store16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
            r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}

// Barriers of a softmax group.
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }

__device__ __forceinline__ bool group_any(int group, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "r"(1 + group)
        : "memory");
    return r != 0;
}

// A pair of FP16 values, zero where not finite.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
    return w & ((w & 0x7C00u) == 0x7C00u ? 0xFFFF0000u : FULL) & ((w & 0x7C000000u) == 0x7C000000u ? 0xFFFFu : FULL);
}

// Eight codes as FP16, times their scale: exact.
__device__ __forceinline__ void from_codes(uint32_t w, __half2 scale, uint32_t *to) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&h[i]), scale);
        to[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
}

// 16 columns of this warp's 32 lanes, one lane per thread, to be waited for.
__device__ __forceinline__ void tc_issue16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

__device__ __forceinline__ uint4 shared_vec(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// ------------------------------------------------------------------ the warps' parts

// The larger of two pairs of BF16 values, numbers before NaN.
__device__ __forceinline__ uint32_t larger_pair(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

// A softmax group's query rows into shared memory, eight threads a row: the latent part
// as FP16, all of it times the power of two that brings the row's largest finite value
// to [2^8, 2^9). Both are exact for values down to 2^-22 of it. (Through shared memory as
// they are, for what is unrolled here is fetched from memory at the start of every
// launch.)
template <int NR>
__device__ __forceinline__ void load_query(const AttendParams &p, const Tile &tile, Ctrl &c, char *query, int group,
                                           int tid) {
    constexpr int SHARE = NR / Shape<NR>::GROUPS;
    const int piece = tid & 7, pairs = p.latent / 128;
#pragma unroll 1
    for (int r = group * SHARE + (tid >> 3); r < (group + 1) * SHARE; r += 16) {
        const bool on = r < tile.rows;
        const int32_t flat = tile.base + (on ? r : 0), token = flat / p.heads, head = flat - token * p.heads;
        const uint16_t *src = p.query + token * p.query_token_stride + head * p.query_head_stride + piece * 8;
        uint4 v[LATENT_MAX / 64 + 1];
#pragma unroll
        for (int k = 0; k <= LATENT_MAX / 64; ++k)
            v[k] = on && k <= 2 * pairs ? __ldg(reinterpret_cast<const uint4 *>(src + k * 64)) : make_uint4(0, 0, 0, 0);
        uint4 *mine = reinterpret_cast<uint4 *>(query + r * 128 + ((piece ^ (r & 7)) << 4));
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k <= LATENT_MAX / 64; ++k) {
            if (k <= 2 * pairs) mine[k * NR * 8] = v[k];
            top = larger_pair(top, larger_pair(larger_pair(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu),
                                               larger_pair(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu)));
        }
        uint32_t most = max(top & 0xFFFFu, top >> 16);
        if (__any_sync(FULL, most == 0x7F80u)) [[unlikely]] {
            most = 0;                          // an infinity: the largest of the others
#pragma unroll 1
            for (int k = 0; k < (2 * pairs + 1) * 8; ++k) {
                const uint32_t h = reinterpret_cast<const uint16_t *>(mine + (k >> 3) * NR * 8)[k & 7] & 0x7FFFu;
                most = max(most, h >= 0x7F80u ? 0u : h);
            }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) most = max(most, __shfl_xor_sync(FULL, most, o));
        const uint32_t up = min(262u - (most >> 7), 253u);       // exponent field of the factor: 2^(8 - exponent)
        const float by = __uint_as_float(up << 23);
        if (piece == 0) {
            const float u = p.scale * __uint_as_float((254u - up) << 23) * LOG2E;   // (so no scale overflows)
            c.unit[r] = fminf(fmaxf(u, -FLT_MAX), FLT_MAX);
        }
#pragma unroll 1
        for (int k = 0; k <= 2 * pairs; ++k, mine += NR * 8) {
            const uint4 x = *mine;
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = __uint_as_float(w[i] << 16) * by, b = __uint_as_float(w[i] & 0xFFFF0000u) * by;
                const __half2 h = __floats2half2_rn(a, b);
                const __nv_bfloat162 e = __floats2bfloat162_rn(a, b);
                w[i] = *reinterpret_cast<const uint32_t *>(&e);
                if (k < 2 * pairs) w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            *mine = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __syncwarp();
    if ((tid & 31) == 0) arrive(&c.q_full);
}

// Cache rows as they are, into a ring for each half of a block's rows, a warp a half:
// units of 128 bytes of each row, the key part, then 256 values after 256 (behind the
// last of an odd number of pairs lies something else, which nobody reads), swizzled so
// that lanes reading a row each meet no conflict; and a block's scales. Pages of 32 rows
// and more come by TMA, a box a unit (two of pages of 32 rows); listed rows by 16-byte
// copies. (Rows read straight into registers, a row a lane, were held up at 7 KB on
// their way per SM: the first-level cache, small beside this much shared memory, keeps a
// line of 128 bytes for each 32 that come: 32 requests x 16 heads x 16384 took 118 us.
// With units of 32 bytes of each row the sender was what all others waited for: a box or
// a group of copies costs it 200 to 300 cycles.)
template <int NR>
__device__ void send_rows(const AttendParams &p, const CUtensorMap *units_map, const CUtensorMap *scales_map, Ctrl &c,
                          uint32_t raw) {
    using S = Shape<NR>;
    const int lane = threadIdx.x & 31, half = (threadIdx.x >> 5) - S::SEND_WARP;
    const int pairs = p.latent / 128, units = 1 + (pairs + 1) / 2;
    const bool one = elected();
    const uint8_t *cache = static_cast<const uint8_t *>(p.cache);
    const uint32_t ring = raw + half * S::RING, scales = ring + S::UNITS * UNIT;
    Cursor at(c);
    uint32_t i = 0, turn = 0;                  // the block and its first unit
    while (at.next(p, lane)) {
        const RowList list(p, at);
        int32_t now[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) now[h] = list.fetch(p, at.b0 * KEYS + half * HALF + h * 32 + lane);
        for (int32_t b = at.b0; b < at.b1; ++b, ++i, turn += units) {
            const uint32_t s = i % S::SCALE_SLOTS;
            int32_t row[2];
            uint32_t mask[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t j = b * KEYS + half * HALF + h * 32 + lane;
                row[h] = list.row(p, now[h], j);
                now[h] = list.fetch(p, j + KEYS);
                mask[h] = __ballot_sync(FULL, row[h] >= 0);
            }
            auto mark = [&]() {
                c.marks[i % BLOCKS][2 * half] = mask[0];
                c.marks[i % BLOCKS][2 * half + 1] = mask[1];
                arrive(&c.row_full[i % BLOCKS]);
            };
            if (p.tiled) {
                // (rows of which there are none, and rows past the cache, come as zeros)
                const int32_t r0 = __shfl_sync(FULL, row[0], 0), r1 = __shfl_sync(FULL, row[1], 0);
                const int32_t y0 = r0 >= 0 ? r0 : p.cache_rows, y1 = r1 >= 0 ? r1 : p.cache_rows;
                if (one) {
                    mark();
                    for (int u = 0; u < units; ++u) {
                        const uint32_t t = turn + u, slot = t % S::UNITS;
                        const int x = u ? (u - 1) * 128 : p.latent / 2;
                        u64 *full = &c.unit_full[half][t % TURNS];
                        await(&c.unit_empty[half][slot], (t / S::UNITS + 1) & 1u, c);
                        if (u == 1) await(&c.scales_empty[half][s], (i / S::SCALE_SLOTS + 1) & 1u, c);
                        mbar_expect_tx(full, u == 1 ? UNIT + SCALES : UNIT);
                        copy_box(ring + slot * UNIT, units_map, x, y0, full);
                        if (p.tiled == 1) copy_box(ring + slot * UNIT + UNIT / 2, units_map, x, y1, full);
                        if (u == 1) {
                            const uint32_t to = scales + s * SCALES;
                            copy_box(to, scales_map, p.latent / 2 + 128, y0, full);
                            if (p.tiled == 1) copy_box(to + SCALES / 2, scales_map, p.latent / 2 + 128, y1, full);
                        }
                    }
                }
                __syncwarp();
                continue;
            }
            // Eight lanes a row, four rows a copy: where this lane's copies come from.
            const uint64_t all = mask[0] | static_cast<uint64_t>(mask[1]) << 32;
            const long long offset[2] = {row[0] >= 0 ? row[0] * p.cache_stride : 0,
                                         row[1] >= 0 ? row[1] * p.cache_stride : 0};
            const uint8_t *src[HALF / 4];
#pragma unroll
            for (int m = 0; m < HALF / 4; ++m)
                src[m] = cache + __shfl_sync(FULL, offset[m / 8], (4 * m + (lane >> 3)) & 31) + (lane & 7) * 16;
            const uint64_t mine = all >> (lane >> 3);   // bit 4 m: there is something to copy
            for (int u = 0; u < units; ++u) {
                const uint32_t t = turn + u, slot = t % S::UNITS, to = ring + slot * UNIT + (lane >> 3) * 128;
                const int x = u ? (u - 1) * 128 : p.latent / 2;
                await_warp(&c.unit_empty[half][slot], t / S::UNITS + 1, c);
#pragma unroll
                for (int m = 0; m < HALF / 4; ++m)
                    copy16(to + m * 512 + (((lane ^ (4 * m + (lane >> 3))) & 7) << 4), src[m] + x, mine >> 4 * m & 1u);
                copies_arrive(&c.unit_full[half][t % TURNS]);
                if (u == 0) {
                    await_warp(&c.scales_empty[half][s], i / S::SCALE_SLOTS + 1, c);
#pragma unroll
                    for (int m = 0; m < HALF / 16; ++m) {
                        const int r = 16 * m + (lane >> 1);
                        copy16(scales + s * SCALES + r * 32 + (lane & 1) * 16,
                               cache + __shfl_sync(FULL, offset[m / 2], r & 31) + p.latent / 2 + 128 + (lane & 1) * 16,
                               all >> r & 1u);
                    }
                    copies_arrive(&c.scales_full[half][s]);
                    if (lane == 0) mark();
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (p.tiled && c.abort) settle(c.unit_full[half], static_cast<int32_t>(turn) - 1, 1, TURNS);
}

// Units into tensor memory, a row a lane, each warp the rows of its own lanes there, 64
// bytes of each row at a time (with two groups of warps each has the same half of every
// unit). 128 values become FP16, the scores' left operand; the key part goes there as it
// is.
template <int NR>
__device__ void convert_rows(const AttendParams &p, Ctrl &c, uint32_t raw, uint32_t tmem) {
    using S = Shape<NR>;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, half = quarter >> 1;
    const int group = S::CONVERT == 2 ? (threadIdx.x - S::SOFT) >> 7 : 0;
    const int pairs = p.latent / 128, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t ring = raw + half * S::RING, scales = ring + S::UNITS * UNIT + (row % HALF) * 32;
    const uint32_t mine = ring + (row % HALF) * 128, turned = (row & 7) << 4;
    Cursor at(c);
    uint32_t i = 0, turn = 0, slot = 0;        // the block, the unit and its place that come next
    auto next_unit = [&]() {
        await_warp(&c.unit_full[half][turn % TURNS], turn / TURNS, c);
        ++turn;
        return mine + slot * UNIT;
    };
    auto read = [&](uint32_t from, int e, uint32_t (&v)[16]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 x = shared_vec(from + ((e * 64 + q * 16) ^ turned));
            v[4 * q] = x.x;
            v[4 * q + 1] = x.y;
            v[4 * q + 2] = x.z;
            v[4 * q + 3] = x.w;
        }
    };
    auto unit_read = [&]() {
        __syncwarp();
        arrive_one(&c.unit_empty[half][slot], lane);
        if (++slot == S::UNITS) slot = 0;
    };
    while (at.next(p, lane))
        for (const uint32_t end = i + (at.b1 - at.b0); i < end; ++i) {
            const uint32_t s = i % S::SCALE_SLOTS, key = i % KEY_SLOTS;
            {
                const uint32_t from = next_unit();
                uint32_t v[2][16];
#pragma unroll
                for (int e = 0; e < 2; e += S::CONVERT) read(from, group + e, v[e]);
                if (i >= KEY_SLOTS) await_warp(&c.key_done[(i - KEY_SLOTS) % BLOCKS], (i - KEY_SLOTS) / BLOCKS, c);
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 2; e += S::CONVERT)
                    tc_store16(lanes + S::K_COL + key * 32 + (group + e) * 16, v[e]);
                unit_read();
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                arrive_one(&c.key_full[key], lane);
            }
            if (!p.tiled) await_warp(&c.scales_full[half][s], i / S::SCALE_SLOTS, c);
#pragma unroll 1
            for (int first = 0; first < pairs; first += 2) {
                const uint32_t from = next_unit();
#pragma unroll 1
                for (int e = group; e < 2 && first + e < pairs; e += S::CONVERT) {
                    const uint32_t n = i * pairs + first + e, a = n % S::A_PAIRS;
                    uint32_t v[16], s8[2];
                    read(from, e, v);
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                                 : "=r"(s8[0]), "=r"(s8[1])
                                 : "r"(scales + s * SCALES + (first + e) * 8));
                    if (n >= S::A_PAIRS)
                        await_warp(&c.a_done[(n - S::A_PAIRS) % TURNS], (n - S::A_PAIRS) / TURNS, c);
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // 32 values with two scales
                        uint32_t both, w[16];
                        asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
                            : "=r"(both)
                            : "h"(static_cast<uint16_t>(s8[q >> 1] >> (16 * (q & 1)))));
                        const __half2 h = *reinterpret_cast<const __half2 *>(&both);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            from_codes(v[4 * q + k], k < 2 ? __low2half2(h) : __high2half2(h), w + 4 * k);
                        tc_store16(lanes + S::A_COL + a * 64 + q * 16, w);
                    }
                    const uint32_t bad = __ballot_sync(FULL, ((((s8[0] & 0x7F7F7F7Fu) + 0x01010101u) |
                                                               ((s8[1] & 0x7F7F7F7Fu) + 0x01010101u)) & 0x80808080u));
                    if (lane == 0) c.bad[a][quarter] = bad;
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    arrive_one(&c.a_full[a], lane);
                }
                unit_read();
            }
            arrive_one(&c.scales_empty[half][s], lane);
        }
}

// The sums' left operand: pairs out of tensor memory into shared memory, a chunk's rows
// of 128 bytes swizzled as the products read them. What waits for its place waits in
// registers, so that tensor memory is free for the pairs behind it. A scale of NaN makes
// every score of its row NaN, and with it the weights of all that see the row; its
// values become zeros here, so that 0 x NaN does not reach those that may not see it.
template <int NR>
__device__ void copy_values(const AttendParams &p, Ctrl &c, uint32_t pairs_at, uint32_t tmem) {
    using S = Shape<NR>;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int row = quarter * 32 + lane, pairs = p.latent / 128;
    const uint32_t mine = pairs_at + row * 128 + ((row & 7) << 4);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + S::A_COL;
    Cursor at(c);
    uint32_t n = 0, end = 0;
    while (at.next(p, lane))
        for (end += (at.b1 - at.b0) * pairs; n < end; ++n) {
            const uint32_t a = n % S::A_PAIRS, place = n % S::PAIRS;
            const uint32_t to = mine + place * 2 * CHUNK;
            uint32_t w[4][16];
            await_warp(&c.a_full[a], n / S::A_PAIRS, c);
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 4; ++q) tc_issue16(lanes + a * 64 + q * 16, w[q]);
            const bool bad = c.bad[a][quarter] >> lane & 1u;
            tc_wait_ld();
            tc_fence_before();
            __syncwarp();
            arrive_one(&c.a_done[n % TURNS], lane);
            if (n >= S::PAIRS) await_warp(&c.summed[(n - S::PAIRS) % TURNS], (n - S::PAIRS) / TURNS, c);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint32_t *x = w[k / 4] + 4 * (k % 4);
                store_vec((to ^ ((k & 7) << 4)) + (k >> 3) * CHUNK, x[0], x[1], x[2], x[3]);
            }
            if (bad) [[unlikely]] {
#pragma unroll 1
                for (int k = 0; k < 16; ++k) {
                    const uint32_t at16 = (to ^ ((k & 7) << 4)) + (k >> 3) * CHUNK;
                    const uint4 x = shared_vec(at16);
                    store_vec(at16, finite_halves(x.x), finite_halves(x.y), finite_halves(x.z), finite_halves(x.w));
                }
            }
            __syncwarp();
            arrive_one(&c.pair_full[place], lane);
        }
}

// Instruction descriptor as instruction(), FP16 operands.
__host__ __device__ constexpr uint32_t half_instruction(int m, int n, bool along) {
    return instruction(m, n, along) & ~((1u << 7) | (1u << 10));
}

// The products, both with the cache as the left operand and the query rows as columns
// (128 x NR x 16 a step): scores out of tensor memory, sums out of shared memory. Each
// has a warp of its own, of which one lane issues.
template <int NR>
__device__ void multiply_scores(const AttendParams &p, Ctrl &c, uint32_t query, uint32_t tmem) {
    using S = Shape<NR>;
    const int lane = threadIdx.x & 31, pairs = p.latent / 128;
    const bool one = elected();
    constexpr uint32_t LATENT_KIND = half_instruction(KEYS, NR, false), KEY_KIND = instruction(KEYS, NR, false);
    constexpr int QCHUNK = NR * 128;
    Cursor at(c);
    uint32_t i = 0, n = 0, piece = 0;
    const uint64_t q = matrix(query, 16);
    while (at.next(p, lane)) {
        if (one) {
            for (int32_t b = at.b0; b < at.b1; ++b, ++i) {
                const uint32_t s = i % S::SCORES, d = tmem + S::S_COL + s * NR, key = i % KEY_SLOTS;
                await(&c.s_empty[s], (i / S::SCORES + 1) & 1u, c);
                if (b == at.b0) {
                    await(&c.q_full, piece & 1u, c);
                    fence_proxy_async();
                }
                for (int u = 0; u < pairs; ++u, ++n) {
                    await(&c.a_full[n % S::A_PAIRS], (n / S::A_PAIRS) & 1u, c);
                    tc_fence_after();
                    const uint32_t k = tmem + S::A_COL + n % S::A_PAIRS * 64;
                    const uint64_t qu = q + u * (2 * QCHUNK >> 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        tc_mma_a(d, k + e * 8, qu + (e >> 2) * (QCHUNK >> 4) + (e & 3) * 2, LATENT_KIND,
                                 u > 0 || e > 0);
                    tc_commit(&c.a_done[n % TURNS]);
                }
                await(&c.key_full[key], (i / KEY_SLOTS) & 1u, c);
                tc_fence_after();
                const uint64_t qk = q + pairs * (2 * QCHUNK >> 4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    tc_mma_a(d, tmem + S::K_COL + key * 32 + e * 8, qk + e * 2, KEY_KIND, true);
                tc_commit(&c.key_done[i % BLOCKS]);
                tc_commit(&c.s_full[s]);
            }
        }
        __syncwarp();
        ++piece;
    }
    drain(&c.drain[0], one);
}

template <int NR>
__device__ void multiply_sums(const AttendParams &p, Ctrl &c, uint32_t pairs_at, uint32_t weights, uint32_t tmem) {
    using S = Shape<NR>;
    const int lane = threadIdx.x & 31, pairs = p.latent / 128;
    const bool one = elected();
    constexpr uint32_t KIND = half_instruction(128, NR, true);
    Cursor at(c);
    uint32_t i = 0, n = 0;
    while (at.next(p, lane)) {
        if (one) {
            for (int32_t b = at.b0; b < at.b1; ++b, ++i) {
                await(&c.p_full[i % BLOCKS], (i / BLOCKS) & 1u, c);
                const uint64_t w = matrix(weights + i % S::WEIGHTS * CHUNK, 16);
                for (int h = 0; h < pairs; ++h, ++n) {
                    const uint32_t slot = n % S::PAIRS;
                    await(&c.pair_full[slot], (n / S::PAIRS) & 1u, c);
                    fence_proxy_async();           // (weights and values were written by ordinary stores)
                    tc_fence_after();
                    const uint64_t v = matrix(pairs_at + slot * 2 * CHUNK, CHUNK);
#pragma unroll
                    for (int k = 0; k < KEYS / 16; ++k)
                        tc_mma(tmem + S::O_COL + h * NR, v + k * 128, w + k * 128, KIND, b > at.b0 || k > 0);
                    tc_commit(&c.summed[n % TURNS]);
                }
                tc_commit(&c.o_done[i % BLOCKS]);
            }
        }
        __syncwarp();
    }
    drain(&c.drain[1], one);
}

// Scores to weights, the running reference and sums, and the outputs. Each group of
// four warps has its share of the query rows and goes its own way. Thread t of a
// group's warp w holds tokens 32 w + t / 4 + 8 h, h < 4, of a block, against the rows
// 8 j + 2 (t % 4) and the next of its share: their references and sums stay in its
// registers. Whether a score outgrows its reference is voted on before the exponentials:
// the scores' place is free from then on.
template <int NR>
__device__ void soften(const AttendParams &p, Ctrl &c, char *query, char *pairs_at, uint32_t weights_at,
                       uint32_t tmem) {
    using S = Shape<NR>;
    constexpr int SHARE = NR / S::GROUPS, N = SHARE / 4;   // query rows of a group, of a thread
    const int tid = threadIdx.x & 127, group = threadIdx.x >> 7, lane = tid & 31, w = tid >> 5, quad = lane & 3;
    const int r0 = group * SHARE, mine_row = r0 + tid;     // the group's first row; a row of a thread < SHARE
    const int t0 = w * 32 + lane / 4, pairs = p.latent / 128;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
    Part *parts = reinterpret_cast<Part *>(p.workspace);
    Joint *joints = reinterpret_cast<Joint *>(parts + 2 * p.sms);
    const bool by_tile = p.tiles <= static_cast<int32_t>(gridDim.x);
    auto row_of = [&](int n) { return r0 + 8 * (n >> 1) + 2 * quad + (n & 1); };   // of the thread's n-th
    // Where the thread's weights go: of its first token, its first rows (the others' a constant away).
    weights_at += t0 * 128 + quad * 4 + (((group * (SHARE / 8)) ^ (t0 & 7)) << 4);
    bool split_here = false;
    Cursor at(c);
    uint32_t i = 0;
    long long done = c.begin;
    bool more = at.next(p, lane);
    if (more) load_query<NR>(p, at.tile, c, query, group, tid);
    while (more) {
        const int32_t start = at.b0 * KEYS;
        // A row that sees nothing of this piece has an infinite reference: whatever its
        // scores, its weights never move it, and its results are written as empty.
        if (tid < SHARE) {
            int32_t lim = 0;
            if (mine_row < at.tile.rows) lim = p.paged ? token_len(p, (at.tile.base + mine_row) / p.heads) : INT32_MAX;
            c.lim[mine_row] = lim;
            c.ref[mine_row] = lim > start ? LOWEST : INFINITY;
        }
        group_sync(group);
        int32_t low = INT32_MAX;
        for (int r = lane; r < SHARE; r += 32) {
            const int32_t lim = c.lim[r0 + r];
            low = min(low, lim > start ? lim : INT32_MAX);
        }
        low = __reduce_min_sync(FULL, low);
        float l[N], ref[N], unit[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            l[n] = 0.0f;
            ref[n] = c.ref[row_of(n)];
            unit[n] = c.unit[row_of(n)];
        }
        for (int32_t b = at.b0; b < at.b1; ++b, ++i) {
            const uint32_t s = i % S::SCORES;
            const int32_t token = b * KEYS + t0;
            await_warp(&c.row_full[i % BLOCKS], i / BLOCKS, c);
            const uint32_t marks = c.marks[i % BLOCKS][w] >> (lane / 4);   // bit 8 h: token h is there
            const bool whole = __all_sync(FULL, (marks & 0x01010101u) == 0x01010101u) && (b + 1) * KEYS <= low;
            const uint32_t scores = lanes + S::S_COL + s * NR + r0;
            const uint32_t weights = weights_at + i % S::WEIGHTS * CHUNK;
            float x[2][2 * N];                 // x[g][4 j + 2 h + e]: token 2 g + h, the thread's row 2 j + e
            // Scores in log2 units less `less` (none, or the references); where masked, -inf.
            auto take = [&](auto less) {
                uint32_t u[2][2 * N];
                tc_issue_groups<SHARE / 8>(scores, u[0]);
                tc_issue_groups<SHARE / 8>(scores + (16u << 16), u[1]);
                tc_wait_ld();
                tc_fence_before();
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int k = 0; k < 2 * N; ++k) {
                        const int n = 2 * (k >> 2) + (k & 1);
                        const float v = __uint_as_float(u[g][k]);
                        x[g][k] = decltype(less)::value ? fmaf(v, unit[n], -ref[n]) : v * unit[n];
                    }
                if (whole) return;
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int k = 0; k < 2 * N; ++k) {
                        const int n = 2 * (k >> 2) + (k & 1), h = 2 * g + ((k >> 1) & 1);
                        if (!((marks >> 8 * h & 1u) && token + 8 * h < c.lim[row_of(n)])) x[g][k] = -INFINITY;
                    }
            };
            await(&c.s_full[s], (i / S::SCORES) & 1u, c);
            __syncwarp();
            tc_fence_after();
            bool moved = true;
            if (b > at.b0) {
                take(std::true_type{});
                float top = x[0][0];
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int k = 0; k < 2 * N; ++k) top = fmaxf(top, x[g][k]);
                moved = group_any(group, top > MOST);
            }
            if (moved) {
                // New references where the rows' largest scores of this block are 2^MOST above
                // the old ones (or the first the row sees).
                take(std::false_type{});
                float top[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int k = 4 * (n >> 1) + (n & 1);
                    top[n] = fmaxf(fmaxf(x[0][k], x[0][k + 2]), fmaxf(x[1][k], x[1][k + 2]));
                }
                across_lanes<N>(top, [](float a, float d) { return fmaxf(a, d); });
                const int mine = across_index<N>();
#pragma unroll
                for (int j = 0; j < (N + 7) / 8; ++j) c.across[w][row_of(mine + j)] = top[j];
                group_sync(group);
                if (tid < SHARE) {
                    const float t = fmaxf(fmaxf(c.across[0][mine_row], c.across[1][mine_row]),
                                          fmaxf(c.across[2][mine_row], c.across[3][mine_row]));
                    const float old = c.ref[mine_row];
                    // (Differences, as the exponents are: sums of large scores round. From 2^27 on t - BELOW
                    // may lie 16 below t, where the weight would be infinite: then t itself is taken.)
                    const bool move = t - old > MOST;  // (of LOWEST: t > old)
                    const float below = t - BELOW, to = t - below > MOST ? t : below;
                    c.factor[mine_row] = move ? exp2_fast(old - to) : 1.0f;
                    if (move) c.ref[mine_row] = to;
                }
                group_sync(group);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    ref[n] = c.ref[row_of(n)];
                    l[n] *= c.factor[row_of(n)];
                }
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int k = 0; k < 2 * N; ++k) x[g][k] -= ref[2 * (k >> 2) + (k & 1)];
                if (b > at.b0) {
                    await_warp(&c.o_done[(i - 1) % BLOCKS], (i - 1) / BLOCKS, c);
                    tc_fence_after();
#pragma unroll 1
                    for (int h = 0; h < pairs; ++h)
#pragma unroll 1
                        for (int v = r0; v < r0 + SHARE; v += 16) {
                            float o[16], f[16];
                            shared16(&c.factor[v], f);
                            tc_load16(lanes + S::O_COL + h * NR + v, o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] *= f[k];
                            latent::tc_store16(lanes + S::O_COL + h * NR + v, o);
                        }
                    tc_wait_st();
                    tc_fence_before();
                }
            }
            __syncwarp();
            arrive_one(&c.s_empty[s], lane);
            if (i >= S::WEIGHTS) {             // (the weights' place is free)
                const uint32_t last = i - S::WEIGHTS;
                await_warp(&c.o_done[last % BLOCKS], last / BLOCKS, c);
            }
            // Weights, rounded once to FP16 for the tensor cores; their sums are of the unrounded
            // ones, in 32 bits.
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float a = exp2_fast(x[g][4 * j + 2 * h]), d = exp2_fast(x[g][4 * j + 2 * h + 1]);
                        const __half2 v = __floats2half2_rn(a, d);
                        l[2 * j] += a;
                        l[2 * j + 1] += d;
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"((weights ^ (j << 4)) + (2 * g + h) * 1024),
                                     "r"(*reinterpret_cast<const uint32_t *>(&v))
                                     : "memory");
                    }
            }
            tc_fence_before();
            __syncwarp();
            arrive_one(&c.p_full[i % BLOCKS], lane);
        }
        // The piece is done: the next one's query rows (the last scores are read), then this
        // one's rows, or its part of them.
        Cursor then = at;
        const bool again = then.next(p, lane);
        across_lanes<N>(l, [](float a, float d) { return a + d; });
        const int mine = across_index<N>();
#pragma unroll
        for (int j = 0; j < (N + 7) / 8; ++j) c.across[w][row_of(mine + j)] = l[j];
        group_sync(group);
        if (again) load_query<NR>(p, then.tile, c, query, group, tid);
        if (tid < SHARE) {
            const bool sees = c.lim[mine_row] > start;
            const float sum = c.across[0][mine_row] + c.across[1][mine_row] + c.across[2][mine_row] +
                              c.across[3][mine_row];
            c.l[mine_row] = sees ? sum : 0.0f;
            c.factor[mine_row] = sees && sum != 0.0f ? 1.0f / sum : 0.0f;   // (0: an empty row, whatever its sums)
            if (!sees) c.ref[mine_row] = -INFINITY;
        }
        group_sync(group);
        await_warp(&c.o_done[(i - 1) % BLOCKS], (i - 1) / BLOCKS, c);
        tc_fence_after();
        const bool direct = at.b0 == 0 && at.b1 == at.blocks;
        if (direct) {
            if (p.lse && tid < SHARE && mine_row < at.tile.rows)
                p.lse[at.tile.base + mine_row] = finished_lse(c.ref[mine_row], c.l[mine_row]);
            // A lane has one value of 16 rows; two lanes trade theirs for pairs of one row each.
            const bool odd = (lane & 1) != 0, all = at.tile.rows == NR;
            uint16_t *out = p.out + (static_cast<int64_t>(at.tile.base) + (lane & 1)) * p.latent + w * 32 + (lane & ~1);
#pragma unroll 1
            for (int h = 0; h < pairs; ++h)
#pragma unroll 1
                for (int v = r0; v < r0 + SHARE; v += 16) {
                    float o[16], f[16];
                    shared16(&c.factor[v], f);
                    tc_load16(lanes + S::O_COL + h * NR + v, o);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const float x = f[k] == 0.0f ? 0.0f : o[k] * f[k];
                        const float y = f[k + 1] == 0.0f ? 0.0f : o[k + 1] * f[k + 1];
                        const float other = __shfl_xor_sync(FULL, odd ? x : y, 1);
                        const __nv_bfloat162 two = __floats2bfloat162_rn(odd ? other : x, odd ? y : other);
                        if (all || v + k + (lane & 1) < at.tile.rows)
                            *reinterpret_cast<__nv_bfloat162 *>(
                                out + static_cast<uint32_t>((v + k) * p.latent + h * 128)) = two;
                    }
                }
        } else {
            // In a cluster the rings are used up: this CTA's part stays there for the others to join.
            Part &part = parts[2 * blockIdx.x + (at.b0 == 0 ? 1 : 0)];
            float *sums = p.cluster ? reinterpret_cast<float *>(pairs_at) : part.sum;
            if (!p.cluster && tid < SHARE) {
                part.m[mine_row] = c.ref[mine_row];
                part.l[mine_row] = c.l[mine_row];
            }
#pragma unroll 1
            for (int h = 0; h < pairs; ++h)
#pragma unroll 1
                for (int v = r0; v < r0 + SHARE; v += 16) {
                    float o[16], f[16];
                    shared16(&c.factor[v], f);
                    tc_load16(lanes + S::O_COL + h * NR + v, o);
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        sums[(v + k) * p.latent + h * 128 + w * 32 + lane] = f[k] == 0.0f ? 0.0f : o[k];
                }
        }
        if (!p.cluster && at.b0 == 0 && threadIdx.x == 0 && (by_tile || !direct)) {
            Joint j;
            j.tile = at.next_tile - 1;
            j.cta = static_cast<int32_t>(blockIdx.x);
            j.parts = direct ? 1 : static_cast<int32_t>((done - at.u0 + at.units - 1) / c.share) - j.cta + 1;
            j.unused = 0;
            joints[by_tile ? j.tile : j.cta] = j;
        }
        split_here |= at.b0 == 0 && !direct;
        done += at.u1 - at.u0;
        tc_fence_before();
        group_sync(group);
        at = then;
        more = again;
    }
    if (!p.cluster && !by_tile && !split_here && threadIdx.x == 0) joints[blockIdx.x] = Joint{0, 0, 0, 0};
}

template <int NR>
__global__ void __launch_bounds__(NT, 1) attend4_kernel(const __grid_constant__ AttendParams p,
                                                        const __grid_constant__ CUtensorMap units_map,
                                                        const __grid_constant__ CUtensorMap scales_map) {
    using S = Shape<NR>;
    extern __shared__ char raw[];
    char *query = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    char *pairs = query + query_bytes<NR>(p.latent), *weights = pairs + S::PAIRS * 2 * CHUNK;
    Ctrl &c = *reinterpret_cast<Ctrl *>(pairs + S::RINGS);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::PAIRS; ++s) mbar_init(&c.pair_full[s], 4);
        for (int s = 0; s < S::A_PAIRS; ++s) mbar_init(&c.a_full[s], 4);
        for (int s = 0; s < TURNS; ++s) {
            mbar_init(&c.a_done[s], 5);
            mbar_init(&c.summed[s], 1);
        }
        for (int h = 0; h < 2; ++h) {
            for (int s = 0; s < TURNS; ++s) mbar_init(&c.unit_full[h][s], p.tiled ? 1 : 32);
            for (int s = 0; s < S::UNITS; ++s) mbar_init(&c.unit_empty[h][s], 2 * S::CONVERT);
            for (int s = 0; s < S::SCALE_SLOTS; ++s) {
                mbar_init(&c.scales_full[h][s], 32);
                mbar_init(&c.scales_empty[h][s], 2 * S::CONVERT);
            }
        }
        for (int s = 0; s < KEY_SLOTS; ++s) mbar_init(&c.key_full[s], 4 * S::CONVERT);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&c.s_full[s], 1);
            mbar_init(&c.s_empty[s], S::SOFT / 32);
            mbar_init(&c.drain[s], 1);
        }
        for (int s = 0; s < BLOCKS; ++s) {
            mbar_init(&c.key_done[s], 1);
            mbar_init(&c.row_full[s], 2);
            mbar_init(&c.p_full[s], S::SOFT / 32);
            mbar_init(&c.o_done[s], 1);
        }
        mbar_init(&c.q_full, S::SOFT / 32);
        c.abort = 0;
        fence_mbar_init();
    }
    if (warp == S::SUMS_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&c.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    grid_dependents_release();
    grid_dependency_wait();
    make_schedule<KEYS, NT>(p, c);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    const uint32_t ring = smem_addr(weights + S::WEIGHTS * CHUNK);
    if (warp < S::SOFT / 32) soften<NR>(p, c, query, pairs, smem_addr(weights), tmem);
    else if (warp < S::COPY_WARP) convert_rows<NR>(p, c, ring, tmem);
    else if (warp < S::SEND_WARP) copy_values<NR>(p, c, smem_addr(pairs), tmem);
    else if (warp < S::SCORES_WARP) send_rows<NR>(p, &units_map, &scales_map, c, ring);
    else if (warp < S::SUMS_WARP) multiply_scores<NR>(p, c, smem_addr(query), tmem);
    else multiply_sums<NR>(p, c, smem_addr(pairs), smem_addr(weights), tmem);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == S::SUMS_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    if (p.cluster > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (c.ranks > 1)
            join_cluster<NT>(p, c, pairs,
                             reinterpret_cast<float(*)[MAX_CLUSTER]>(pairs + NR * LATENT_MAX * sizeof(float)));
        __syncwarp();
        cluster_arrive();                      // no CTA leaves while others read its part
        cluster_wait();
    }
}

// ------------------------------------------------------------------ host side

// Blocks are twice the BF16 form's. Of eight settings at 200 sizes (1 to 150 tokens of 16
// to 128 heads, 256 to 32768 rows) this takes the better side of each: shares against
// the cluster, 1 token of 16 rows x 4 blocks 13.4 / 11.5 us (4 CTAs), x 16 14.1 / 13.5
// (16); 8 tokens x 4 16.0 / 11.9; 1 of 64 rows x 16 17.6 / 21.8 (8), x 32 18.4 / 21.2;
// pages of 64 rows x 32 21.2 / 28.6.
constexpr Costs COSTS = {1, 3, 2, 2, 1};

Device g_device[64];

template <int NR>
const void *attend_fn() {
    return reinterpret_cast<const void *>(&attend4_kernel<NR>);
}

cudaError_t device(Device *&out) {
    return device(g_device, {attend_fn<16>(), attend_fn<32>(), attend_fn<64>()}, NT, out);
}

}  // namespace

int64_t workspace4_bytes() {
    Device *d = nullptr;
    if (device(d) != cudaSuccess) return 0;
    return static_cast<int64_t>(d->sms) * static_cast<int64_t>(2 * sizeof(Part) + sizeof(Joint));
}

cudaError_t status_attend4(uint32_t *v, bool clear) { return unit_status(v, clear); }

int64_t attend4_workspace(AttendParams p) {
    Device *d = nullptr;
    if (device(d) != cudaSuccess) return -1;
    if (p.rows_per_request > p.tokens) p.rows_per_request = p.tokens;
    return deal<KEYS>(p, *d, COSTS).cluster ? 0 : workspace4_bytes();
}

cudaError_t launch_attend4(AttendParams p, cudaStream_t stream) {
    Device *d = nullptr;
    cudaError_t e = device(d);
    if (e != cudaSuccess) return e;
    if (p.rows_per_request > p.tokens) p.rows_per_request = p.tokens;   // (one request)
    const Deal plan = deal<KEYS>(p, *d, COSTS);
    p.tiles_per_request = plan.tiles_per_request;
    p.tiles = static_cast<int32_t>(plan.tiles);
    p.cluster = plan.cluster;
    p.tile_cost = plan.tiles > d->sms ? COSTS.tile : 0;
    p.min_share = COSTS.min_share;
    p.sms = d->sms;

    // Pages of 32 rows (1) or 64 and more (2): as many rows of a half follow each other in the cache.
    CUtensorMap units_map = {}, scales_map = {};
    const int run = p.page_shift >= 6 ? 64 : 32;
    p.tiled = p.paged && p.page_shift >= 5 && p.cache_rows >= run ? run / 32 : 0;
    for (CUtensorMap *map : {&units_map, &scales_map}) {
        if (!p.tiled) break;
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(LATENT4_ROW_BYTES(p.latent)),
                                    static_cast<cuuint64_t>(p.cache_rows)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.cache_stride)};
        const cuuint32_t box[2] = {map == &units_map ? 128u : 32u, static_cast<cuuint32_t>(run)}, steps[2] = {1, 1};
        if (d->encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p.cache), dims, strides, box, steps,
                      CU_TENSOR_MAP_INTERLEAVE_NONE,
                      map == &units_map ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }

    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.grid, 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    void *args[] = {&p, &units_map, &scales_map};
    e = cudaLaunchKernelExC(&cfg, plan.nr == 16 ? attend_fn<16>() : plan.nr == 32 ? attend_fn<32>() : attend_fn<64>(),
                            args);
    if (e != cudaSuccess || p.cluster || plan.blocks <= 1) return e;   // tiles of one block are never split
    return launch_join(p, plan.grid, plan.nr, stream);
}

}  // namespace topk::latent
