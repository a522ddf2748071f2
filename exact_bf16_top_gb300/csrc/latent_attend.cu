// Attention over latent cache rows on the tensor cores: one persistent kernel
// for both forms, and the kernel that joins the parts of split tiles.
//
// A tile is up to 64 (token, head) rows that read the same cache rows; blocks of
// 64 cache rows pass through shared memory once for scores and sums:
//     scores (64 tokens x rows) = K Q^T,  weights = 2^(scores - reference),
//     sums (values x rows) += V^T weights,   V the latent part of K.
// Both products have the cache as the left operand: the sums of 512 values x 64
// rows are 256 columns of tensor memory (as rows x values they would fill all of
// it), and 16 rows cost little more than their share. Warps have one job each
// (softmax, copies, issue of either product) and meet at mbarriers only.
//
// What bounds it. Few heads: DRAM (32 requests x 16 heads x up to 16384 tokens: 83
// us, 5.3 TB/s). 64 rows a tile: shared memory. A block's operands leave it 36 x 4
// KB (scores) and 16 x 6 KB (sums) at 128 bytes a cycle and its rows come in once:
// about 2500 cycles a block, what a chunk of 509 tokens x 128 heads over 9000 takes
// (1.20 ms, 1.0 PFLOP/s; tensor pipes 66 % active). More rows a tile would halve
// that but neither their queries (74 KB for 64) nor their sums have room. Listed
// rows (no TMA boxes) add the copies' latency: 3200 cycles a block at two blocks in
// flight, tile ends included (512 tokens x 128 heads x 2048: 359 us).

#include <type_traits>

#include "latent_attend.cuh"

namespace topk::latent {

namespace {

constexpr int SOFT = 256;                    // warps 0 to 7: softmax and outputs, in two groups
constexpr int LOAD = 128;                    // warps 8 to 11: query rows, the latent part of cache rows
constexpr int ROPE_LOAD = 32;                // warp 12: the rotary part
constexpr int NT = SOFT + LOAD + ROPE_LOAD + 64;   // warps 13 and 14: the tensor cores (scores, sums)
constexpr int KEYS = 64;                     // cache rows of a block
constexpr int CHUNK = KEYS * 128;            // bytes of a block's rows at 64 of their values
constexpr int MAX_SLOTS = 12;                // most slots of either ring
constexpr int BLOCKS = 16;                   // blocks that have row numbers and barriers of their own: more
                                             // than the rings hold
constexpr uint32_t O_COL = 0, S_COL = 256;   // tensor memory columns: sums (4 x NR), scores (2 x NR)
constexpr float LAZY = 16.0f;                // the reference may lag the maximum by this much (log2)

struct Ctrl : Schedule<NT> {
    u64 pair_full[MAX_SLOTS], rope_full[MAX_SLOTS];     // a slot's rows are in
    u64 pair_empty[MAX_SLOTS], rope_empty[MAX_SLOTS];   // a slot is used up
    u64 s_full[2], s_empty[2];                 // scores written / read
    u64 p_full[BLOCKS], o_done[BLOCKS];        // a block's weights are in / its sums are added (one each: who waits
                                               // for one block may find later ones done, and two phases of one
                                               // barrier look like none)
    u64 q_first, q_full, q_empty;              // the first query tile, a later one is in / it is used up
    u64 drain[2];
    uint32_t tmem;
    volatile uint32_t abort;
    alignas(16) float ref[ROWS];               // reference maximum (log2), LOWEST at first; +inf: a row that sees
                                               // nothing here
    alignas(16) float factor[ROWS];
    float l[ROWS];
    int32_t lim[ROWS];                         // tokens a row may see
    float across[4][ROWS];
    int32_t rows[BLOCKS][KEYS];                // cache row numbers of a block, -1: none
};

using Cursor = CursorOf<KEYS>;
using RowList = RowListOf<KEYS>;

// Shared memory: the query tile (chunks of 64 values, NR rows of 128 bytes
// each), a ring of pairs of latent chunks, a ring of rotary chunks (where a
// block's weights go once its scores are out), the control block.
struct Plan {
    int pairs, pair_slots, rope_slots;         // pairs per block; slots: two blocks' at least
    uint32_t query_bytes;
};

template <int NR>
__host__ __device__ constexpr Plan make_plan(int latent) {
    Plan r = {};
    r.pairs = latent / 128;
    r.query_bytes = static_cast<uint32_t>((2 * r.pairs + 1) * NR * 128);
    const int units = static_cast<int>((SMEM - 1024 - sizeof(Ctrl) - r.query_bytes) / CHUNK);
    r.rope_slots = units / (2 * r.pairs + 1);
    r.pair_slots = (units - r.rope_slots) / 2;
    if (r.pair_slots > MAX_SLOTS) r.pair_slots = MAX_SLOTS;
    r.rope_slots = units - 2 * r.pair_slots;
    if (r.rope_slots > MAX_SLOTS) r.rope_slots = MAX_SLOTS;
    return r;
}
static_assert(make_plan<ROWS>(LATENT_MAX).pair_slots >= 2 * LATENT_MAX / 128 &&
              make_plan<ROWS>(LATENT_MAX).rope_slots >= 2);

// Whether either of two BF16 values is NaN or infinite.
__device__ __forceinline__ bool not_finite(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(SOFT) : "memory"); }

__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "n"(SOFT)
        : "memory");
    return r != 0;
}

// ------------------------------------------------------------------ the warps' parts

// A tile's query rows into shared memory, swizzled as the products read them, a
// row's eighth of every chunk per thread. Rows past the tile's are zeros: nothing
// is written for them, but an infinity that lay there would have every block's
// tokens looked over.
template <int NR, int THREADS>
__device__ __forceinline__ void load_query(const AttendParams &p, const Tile &tile, uint32_t query, int chunks,
                                           int tid) {
    const int piece = tid & 7;
    for (int r = tid >> 3; r < NR; r += THREADS / 8) {
        const bool on = r < tile.rows;
        const int32_t flat = tile.base + (on ? r : 0), token = flat / p.heads, head = flat - token * p.heads;
        const uint16_t *src = p.query + token * p.query_token_stride + head * p.query_head_stride + piece * 8;
        const uint32_t dst = query + r * 128 + ((piece ^ (r & 7)) << 4);
        for (int k = 0; k < chunks; ++k) copy16(dst + k * NR * 128, src + k * 64, on);
    }
}

// Query and cache rows into shared memory. Each warp has one pair of every
// block (and with few pairs only some of its rows), so that it waits for one
// slot a block and the pairs of a block are copied side by side as their slots
// come free. Places that hold no cache row are filled with zeros. Pages that hold
// whole blocks come by TMA, 64 rows of 64 values a copy; their rows past the
// context's end then hold whatever the page does, and are masked. A tile's query is
// copied when its first block is on its way (the first tile's by the softmax
// warps, which have nothing else to do yet).
// Measured: listed rows gathered four at a time by TMA came at 12 bytes a
// nanosecond per SM, against up to 100 from L2 by four warps' 16-byte copies;
// boxes in place of those copies took a chunk of 509 tokens x 128 heads over 9000
// from 1647 to 1364 us. Eight copying warps, or prefetching rows into L2 ahead of
// the copies, changed nothing.
template <int NR>
__device__ void load_pairs(const AttendParams &p, const CUtensorMap *map, Ctrl &c, const Plan &plan, uint32_t query,
                           uint32_t pairs) {
    constexpr int SHARE = KEYS / (LOAD / 32);  // rows of a warp
    const int lane = threadIdx.x & 31, warp = (threadIdx.x - SOFT) >> 5;
    const int64_t pitch = p.cache_stride * 2;
    const int half = lane >> 4, piece = lane & 15;
    const char *cache = static_cast<const char *>(p.cache) + piece * 16;
    const int r0 = warp * SHARE + half;        // by copies this lane has rows r0, r0 + 2, .. of every pair
    const uint32_t dst = pairs + (piece >> 3) * CHUNK + r0 * 128;
    const int mine = p.tiled ? 0 : warp * SHARE + (lane & (SHARE - 1));
    Cursor at(c);
    uint32_t ps = 0, pu = 0, piece_no = 0;     // the block's first slot and its use
    while (at.next(p, lane)) {
        const RowList list(p, at);
        int32_t now = list.fetch(p, at.b0 * KEYS + mine);
        for (int32_t b = at.b0; b < at.b1; ++b) {
            const int32_t then = list.fetch(p, (b + 1) * KEYS + mine);
            if (piece_no && b == at.b0 + 1) {
                wait(&c.q_empty, piece_no + 1, c);
                load_query<NR, LOAD>(p, at.tile, query, 2 * plan.pairs + 1, threadIdx.x - SOFT);
                copies_arrive(&c.q_full);
            }
            const int32_t here = list.row(p, now, b * KEYS + mine);
            const char *src[SHARE / 2];
            bool on[SHARE / 2];
#pragma unroll
            for (int k = 0; k < SHARE / 2; ++k) {
                const int32_t v = __shfl_sync(0xFFFFFFFFu, here, 2 * k + half);
                on[k] = v >= 0;
                src[k] = cache + (on[k] ? v * pitch : 0);
            }
            for (int u = p.tiled ? warp : 0; u < plan.pairs; u += p.tiled ? LOAD / 32 : 1) {
                uint32_t slot = ps + u, used = pu;
                if (slot >= static_cast<uint32_t>(plan.pair_slots)) {
                    slot -= plan.pair_slots;
                    ++used;
                }
                wait(&c.pair_empty[slot], used + 1, c);
                if (p.tiled) {
                    if (lane == 0) {
                        mbar_expect_tx(&c.pair_full[slot], 2 * CHUNK);
                        for (int k = 0; k < 2; ++k)
                            copy_box(pairs + (2 * slot + k) * CHUNK, map, (2 * u + k) * 64,
                                     here < 0 ? p.cache_rows : here, &c.pair_full[slot]);
                    }
                    __syncwarp();
                } else {
#pragma unroll
                    for (int k = 0; k < SHARE / 2; ++k)
                        copy16(dst + slot * 2 * CHUNK + k * 256 + (((piece ^ (r0 + 2 * k)) & 7) << 4), src[k] + u * 256,
                               on[k]);
                    copies_arrive(&c.pair_full[slot]);
                }
            }
            ps += plan.pairs;
            if (ps >= static_cast<uint32_t>(plan.pair_slots)) {
                ps -= plan.pair_slots;
                ++pu;
            }
            now = then;
        }
        if (piece_no && at.b1 == at.b0 + 1) {
            wait(&c.q_empty, piece_no + 1, c);
            load_query<NR, LOAD>(p, at.tile, query, 2 * plan.pairs + 1, threadIdx.x - SOFT);
            copies_arrive(&c.q_full);
        }
        ++piece_no;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (p.tiled && warp < plan.pairs && c.abort)
        settle(c.pair_full, static_cast<int32_t>(pu * plan.pair_slots + ps) - plan.pairs + warp, plan.pairs,
               plan.pair_slots);
}

__device__ void load_ropes(const AttendParams &p, const CUtensorMap *map, Ctrl &c, const Plan &plan, uint32_t ropes) {
    const int lane = threadIdx.x & 31, quarter = lane >> 3, piece = lane & 7;
    const int64_t pitch = p.cache_stride * 2;
    const char *cache = static_cast<const char *>(p.cache) + plan.pairs * 256 + piece * 16;
    Cursor at(c);
    uint32_t i = 0, rs = 0, ru = 0;
    while (at.next(p, lane)) {
        const RowList list(p, at);
        int32_t now[2], then[2], here[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) now[h] = list.fetch(p, at.b0 * KEYS + 32 * h + lane);
        for (int32_t b = at.b0; b < at.b1; ++b, ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                then[h] = list.fetch(p, (b + 1) * KEYS + 32 * h + lane);
                here[h] = list.row(p, now[h], b * KEYS + 32 * h + lane);
                c.rows[i % BLOCKS][32 * h + lane] = here[h];
            }
            wait(&c.rope_empty[rs], ru + 1, c);
            if (p.tiled) {
                if (lane == 0) {
                    mbar_expect_tx(&c.rope_full[rs], CHUNK);
                    copy_box(ropes + rs * CHUNK, map, plan.pairs * 128, here[0] < 0 ? p.cache_rows : here[0],
                             &c.rope_full[rs]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < KEYS / 4; ++k) {
                    const int r = 4 * k + quarter;
                    const int32_t v = __shfl_sync(0xFFFFFFFFu, here[k / 8], r & 31);
                    copy16(ropes + rs * CHUNK + r * 128 + ((piece ^ (r & 7)) << 4), cache + (v >= 0 ? v * pitch : 0),
                           v >= 0);
                }
                copies_arrive(&c.rope_full[rs]);
            }
            __syncwarp();
            if (lane == 0) arrive(&c.rope_full[rs]);   // (makes the row numbers visible)
            if (++rs == static_cast<uint32_t>(plan.rope_slots)) {
                rs = 0;
                ++ru;
            }
            now[0] = then[0];
            now[1] = then[1];
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (p.tiled && c.abort)
        settle(c.rope_full, static_cast<int32_t>(ru * plan.rope_slots + rs) - 1, 1, plan.rope_slots);
}

// The products, both with the cache as the left operand and the query rows as
// columns, so that few query rows cost little:
//   scores[token][row] = sum over chunks of K chunk x Q chunk       (64 x NR x 16 a step)
//   sums[value][row]  += V pair (values x tokens) x weights         (128 x NR x 16 a step)
// A step takes the longer of its arithmetic and its operands' way out of shared
// memory at 128 bytes a cycle (measured: 23 and 39 cycles at NR = 16, 32 and 48
// at NR = 64). Each product has a warp of its own, of which one lane issues: the
// tensor cores take the steps in the order in which operands arrive, and one
// product's waiting does not hold up the other.
template <int NR>
__device__ void multiply_scores(const AttendParams &p, Ctrl &c, const Plan &plan, uint32_t query, uint32_t pairs,
                                uint32_t ropes, uint32_t tmem) {
    const int lane = threadIdx.x & 31;
    const bool one = elected();
    constexpr uint32_t KIND = instruction(KEYS, NR, false);
    constexpr int QCHUNK = NR * 128;
    Cursor at(c);
    uint32_t i = 0, piece = 0, ps = 0, pu = 0, rs = 0, ru = 0;
    const uint64_t q = matrix(query, 16);
    while (at.next(p, lane)) {
        if (one) {
            for (int32_t b = at.b0; b < at.b1; ++b, ++i) {
                const uint32_t d = tmem + S_COL + (i & 1) * NR;
                mbar_wait(&c.s_empty[i & 1], ((i >> 1) + 1) & 1u, &c.abort);
                if (b == at.b0) mbar_wait(piece ? &c.q_full : &c.q_first, piece ? (piece - 1) & 1u : 0u, &c.abort);
                for (int u = 0; u < plan.pairs; ++u) {
                    mbar_wait(&c.pair_full[ps], pu & 1u, &c.abort);
                    fence_proxy_async();      // (the rows were written by ordinary copies)
                    tc_fence_after();
                    const uint64_t k = matrix(pairs + ps * 2 * CHUNK, 16), qu = q + u * (2 * QCHUNK >> 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        tc_mma(d, k + (e >> 2) * (CHUNK >> 4) + (e & 3) * 2,
                               qu + (e >> 2) * (QCHUNK >> 4) + (e & 3) * 2, KIND, u > 0 || e > 0);
                    if (++ps == static_cast<uint32_t>(plan.pair_slots)) {
                        ps = 0;
                        ++pu;
                    }
                }
                mbar_wait(&c.rope_full[rs], ru & 1u, &c.abort);
                fence_proxy_async();
                tc_fence_after();
                const uint64_t k = matrix(ropes + rs * CHUNK, 16), qu = q + plan.pairs * (2 * QCHUNK >> 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) tc_mma(d, k + e * 2, qu + e * 2, KIND, true);
                tc_commit(&c.s_full[i & 1]);
                if (++rs == static_cast<uint32_t>(plan.rope_slots)) {
                    rs = 0;
                    ++ru;
                }
            }
            tc_commit(&c.q_empty);
        }
        __syncwarp();
        ++piece;
    }
    drain(&c.drain[0], one);
}

template <int NR>
__device__ void multiply_sums(const AttendParams &p, Ctrl &c, const Plan &plan, uint32_t pairs, uint32_t ropes,
                              uint32_t tmem) {
    const int lane = threadIdx.x & 31;
    const bool one = elected();
    constexpr uint32_t KIND = instruction(128, NR, true);
    Cursor at(c);
    uint32_t i = 0, ps = 0, rs = 0;
    while (at.next(p, lane)) {
        if (one) {
            for (int32_t b = at.b0; b < at.b1; ++b, ++i) {
                mbar_wait(&c.p_full[i % BLOCKS], (i / BLOCKS) & 1u, &c.abort);
                fence_proxy_async();
                tc_fence_after();
                const uint64_t w = matrix(ropes + rs * CHUNK, 16);
                for (int h = 0; h < plan.pairs; ++h) {
                    const uint64_t v = matrix(pairs + ps * 2 * CHUNK, CHUNK);
#pragma unroll
                    for (int k = 0; k < KEYS / 16; ++k)
                        tc_mma(tmem + O_COL + h * NR, v + k * 128, w + k * 128, KIND, b > at.b0 || k > 0);
                    tc_commit(&c.pair_empty[ps]);
                    if (++ps == static_cast<uint32_t>(plan.pair_slots)) ps = 0;
                }
                tc_commit(&c.rope_empty[rs]);
                tc_commit(&c.o_done[i % BLOCKS]);
                if (++rs == static_cast<uint32_t>(plan.rope_slots)) rs = 0;
            }
        }
        __syncwarp();
    }
    drain(&c.drain[1], one);
}

// Scores to weights, the running reference and sums, and the outputs. Each group
// of four warps has half of the query rows. Thread t of a group's warp w holds
// tokens 16 w + t / 4 and 8 further of a block, against the rows 8 j + 2 (t % 4)
// and the next of its half: their references and sums stay in its registers.
// The weights' reference is the maximum of the row's first block; weights may grow
// to 2^16 before it moves (FP32 sums and BF16 weights lose nothing by that), which
// is seen from the packed weights and rarely happens. Bound by latency, not by the
// exponentials (16 a thread and block at 64 rows).
template <int NR>
__device__ void soften(const AttendParams &p, Ctrl &c, const Plan &plan, uint32_t query, char *pairs, char *ropes,
                       uint32_t tmem) {
    constexpr int N = NR / 8;                  // query rows of a thread
    const int tid = threadIdx.x, lane = tid & 31, w = (tid >> 5) & 3, group = tid >> 7, quad = lane & 3;
    const int t0 = w * 16 + lane / 4;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
    const float scale = p.scale * LOG2E;
    Part *parts = reinterpret_cast<Part *>(p.workspace);
    Joint *joints = reinterpret_cast<Joint *>(parts + 2 * p.sms);
    const bool by_tile = p.tiles <= static_cast<int32_t>(gridDim.x);
    auto row_of = [&](int n) { return group * (NR / 2) + 8 * (n >> 1) + 2 * quad + (n & 1); };   // of the thread's n-th
    bool split_here = false;
    Cursor at(c);
    uint32_t i = 0, ps = 0, rs = 0, ru = 0;
    long long done = c.begin;
    while (at.next(p, lane)) {
        const int32_t start = at.b0 * KEYS;
        if (i == 0) {
            load_query<NR, SOFT>(p, at.tile, query, 2 * plan.pairs + 1, tid);
            copies_arrive(&c.q_first);
        }
        // A row that sees nothing of this piece has an infinite reference: whatever its
        // scores, its weights never move it, and its results are written as empty.
        if (tid < ROWS) {
            int32_t lim = 0;
            if (tid < at.tile.rows) lim = p.paged ? token_len(p, (at.tile.base + tid) / p.heads) : INT32_MAX;
            c.lim[tid] = lim;
            c.ref[tid] = lim > start ? LOWEST : INFINITY;
        }
        soft_sync();
        int32_t low = INT32_MAX;
#pragma unroll
        for (int r = 0; r < ROWS; r += 32) {
            const int32_t lim = c.lim[r + lane];
            low = min(low, lim > start ? lim : INT32_MAX);
        }
        low = __reduce_min_sync(0xFFFFFFFFu, low);
        float l[N], ref[N];
        int32_t lim[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            lim[n] = c.lim[row_of(n)];
            l[n] = 0.0f;
            ref[n] = c.ref[row_of(n)];
        }
        for (int32_t b = at.b0; b < at.b1; ++b, ++i) {
            wait(&c.rope_full[rs], ru, c);             // (makes the row numbers visible)
            const int32_t token = b * KEYS + t0;
            const bool there[2] = {c.rows[i % BLOCKS][t0] >= 0, c.rows[i % BLOCKS][t0 + 8] >= 0};
            const bool whole = __all_sync(0xFFFFFFFFu, there[0] && there[1]) && (b + 1) * KEYS <= low;
            const uint32_t scores = lanes + S_COL + (i & 1) * NR + group * (NR / 2);
            char *weights = ropes + rs * CHUNK + t0 * 128 + quad * 4;
            float x[2 * N];                    // x[4 j + 2 h + e]: token h, the thread's row 2 j + e
            float most = 0.0f;                 // the block's largest score (by size): infinity and NaN are rare
            // Scores in log2 units; where masked, -inf.
            auto take = [&]() {
                tc_load_groups<NR / 16>(scores, x);
                tc_fence_before();
#pragma unroll
                for (int e = 0; e < 2 * N; e += 2) most = largest(most, x[e], x[e + 1]);
#pragma unroll
                for (int e = 0; e < 2 * N; ++e) x[e] *= scale;
                if (!whole) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            float &v = x[4 * (n >> 1) + 2 * h + (n & 1)];
                            v = there[h] && token + 8 * h < lim[n] ? v : -INFINITY;
                        }
                }
            };
            // Weights from scores (or from the unscaled scores of a whole block), rounded once
            // to BF16 for the tensor cores; true if one outgrew the reference.
            auto weigh = [&](auto unscaled) -> bool {
                __nv_bfloat162 top = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < N / 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float &a = x[4 * j + 2 * h], &d = x[4 * j + 2 * h + 1];
                        if constexpr (decltype(unscaled)::value) {
                            most = largest(most, a, d);
                            a = exp2_fast(fmaf(a, scale, -ref[2 * j]));
                            d = exp2_fast(fmaf(d, scale, -ref[2 * j + 1]));
                        } else {
                            a = exp2_fast(a - ref[2 * j]);
                            d = exp2_fast(d - ref[2 * j + 1]);
                        }
                        const __nv_bfloat162 v = __floats2bfloat162_rn(a, d);
                        top = __hmax2(top, v);
                        const int at_row = (group * (N / 2) + j) ^ (t0 & 7);
                        *reinterpret_cast<__nv_bfloat162 *>(weights + h * 1024 + (at_row << 4)) = v;
                    }
                return fmaxf(__low2float(top), __high2float(top)) > 65536.0f;   // 2^LAZY
            };
            mbar_wait(&c.s_full[i & 1], (i >> 1) & 1u, &c.abort);
            __syncwarp();
            tc_fence_after();
            bool moved = true;
            if (b == at.b0) {
                take();
            } else if (whole) {
                tc_load_groups<NR / 16>(scores, x);
                tc_fence_before();
                moved = soft_any(weigh(std::true_type{}));
            } else {
                take();
                moved = soft_any(weigh(std::false_type{}));
            }
            if (moved) {
                // New references: the rows' largest scores of this block where they are 2^16
                // above the old ones (or the first the row sees).
                if (b > at.b0) take();
                float top[N];
#pragma unroll
                for (int n = 0; n < N; ++n) top[n] = fmaxf(x[4 * (n >> 1) + (n & 1)], x[4 * (n >> 1) + 2 + (n & 1)]);
                across_lanes<N>(top, [](float a, float d) { return fmaxf(a, d); });
                const int mine = across_index<N>();
#pragma unroll
                for (int j = 0; j < (N + 7) / 8; ++j) c.across[w][row_of(mine + j)] = top[j];
                soft_sync();
                if (tid < NR) {
                    const float t = fmaxf(fmaxf(c.across[0][tid], c.across[1][tid]),
                                          fmaxf(c.across[2][tid], c.across[3][tid]));
                    const float old = c.ref[tid];
                    const bool move = t > old + LAZY;  // (of LOWEST: t > old)
                    c.factor[tid] = move ? exp2_fast(old - t) : 1.0f;
                    if (move) c.ref[tid] = t;
                }
                soft_sync();
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    ref[n] = c.ref[row_of(n)];
                    l[n] *= c.factor[row_of(n)];
                }
                weigh(std::false_type{});
                if (b > at.b0) {
                    wait(&c.o_done[(i - 1) % BLOCKS], (i - 1) / BLOCKS, c);
                    tc_fence_after();
                    for (int h = 0; h < plan.pairs; ++h)
#pragma unroll
                        for (int v = 0; v < NR; v += 16) {
                            if (((h * (NR / 16) + v / 16) & 1) != group) continue;
                            float o[16], f[16];
                            shared16(&c.factor[v], f);
                            tc_load16(lanes + O_COL + h * NR + v, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f[e];
                            tc_store16(lanes + O_COL + h * NR + v, o);
                        }
                    tc_wait_st();
                    tc_fence_before();
                }
            }
            // What is not finite among a token's values must not reach a row that gives the token
            // no weight through 0 x inf: neither one that may not see it nor one whose score of it
            // is -inf. Such a row's score of it is not finite, which marks the token, and what is
            // not finite among its values is zeroed (a row that does weigh it has a score of NaN or
            // +inf, so NaN weights; a query's own NaN marks tokens too, whose values then are fine).
            // Scores are read again for it, here and in small code: marks made in take(), which is
            // inlined three times, cost 10 % of 512 x 128 heads x 2048 (412 us against 375).
            if (__any_sync(0xFFFFFFFFu, !(most < INFINITY))) {
                bool odd[2] = {false, false};
#pragma unroll 1
                for (int j = 0; j < N / 2; ++j) {
                    float v[4];
                    tc_load_groups<1>(scores + 8 * j, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int h = e >> 1, r = row_of(2 * j + (e & 1));
                        const bool seen = there[h] && token + 8 * h < c.lim[r];
                        odd[h] |= r < at.tile.rows && (seen ? v[e] * scale == -INFINITY : !(fabsf(v[e]) < INFINITY));
                    }
                }
                tc_fence_before();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    odd[h] |= __shfl_xor_sync(0xFFFFFFFFu, odd[h], 1);
                    odd[h] |= __shfl_xor_sync(0xFFFFFFFFu, odd[h], 2);
                    if (!odd[h]) continue;
                    uint32_t slot = ps;
#pragma unroll 1
                    for (int u = 0; u < plan.pairs; ++u) {
                        for (int k = quad; k < 16; k += 4) {
                            uint4 *at16 = reinterpret_cast<uint4 *>(pairs + slot * 2 * CHUNK + (k >> 3) * CHUNK +
                                                                    (t0 + 8 * h) * 128 + (k & 7) * 16);
                            const uint4 v = *at16;
                            if (not_finite(v.x) || not_finite(v.y) || not_finite(v.z) || not_finite(v.w))
                                *at16 = make_uint4(0, 0, 0, 0);
                        }
                        if (++slot == static_cast<uint32_t>(plan.pair_slots)) slot = 0;
                    }
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                arrive(&c.s_empty[i & 1]);
                arrive(&c.p_full[i % BLOCKS]);
            }
            // The sums are of the unrounded weights, in 32 bits.
#pragma unroll
            for (int n = 0; n < N; ++n) l[n] += x[4 * (n >> 1) + (n & 1)] + x[4 * (n >> 1) + 2 + (n & 1)];
            ps += plan.pairs;
            if (ps >= static_cast<uint32_t>(plan.pair_slots)) ps -= plan.pair_slots;
            if (++rs == static_cast<uint32_t>(plan.rope_slots)) {
                rs = 0;
                ++ru;
            }
        }
        // The piece is done: write its rows, or its part of them.
        across_lanes<N>(l, [](float a, float d) { return a + d; });
        const int mine = across_index<N>();
#pragma unroll
        for (int j = 0; j < (N + 7) / 8; ++j) c.across[w][row_of(mine + j)] = l[j];
        soft_sync();
        if (tid < NR) {
            const bool sees = c.lim[tid] > start;
            const float sum = c.across[0][tid] + c.across[1][tid] + c.across[2][tid] + c.across[3][tid];
            c.l[tid] = sees ? sum : 0.0f;
            c.factor[tid] = sees && sum != 0.0f ? 1.0f / sum : 0.0f;   // (0: an empty row, whatever its sums)
            if (!sees) c.ref[tid] = -INFINITY;
        }
        soft_sync();
        wait(&c.o_done[(i - 1) % BLOCKS], (i - 1) / BLOCKS, c);
        tc_fence_after();
        const bool direct = at.b0 == 0 && at.b1 == at.blocks;
        if (direct) {
            if (p.lse && tid < at.tile.rows) p.lse[at.tile.base + tid] = finished_lse(c.ref[tid], c.l[tid]);
            // A lane has one value of 16 rows; two lanes trade theirs for pairs of one row
            // each. (Tiles of all rows store without a test a row: 1144 tokens x 128 heads x
            // 175 rows 193 us with it, 160 without; 512 x 128 x 2048 398 and 357.)
            const bool odd = (lane & 1) != 0;
            uint16_t *out = p.out + (static_cast<int64_t>(at.tile.base) + (lane & 1)) * p.latent + w * 32 + (lane & ~1);
            auto write = [&](auto all) {
                for (int h = 0; h < plan.pairs; ++h)
#pragma unroll
                    for (int v = 0; v < NR; v += 16) {
                        if (((h * (NR / 16) + v / 16) & 1) != group) continue;
                        float o[16], f[16];
                        shared16(&c.factor[v], f);
                        tc_load16(lanes + O_COL + h * NR + v, o);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float x = f[e] == 0.0f ? 0.0f : o[e] * f[e];
                            const float y = f[e + 1] == 0.0f ? 0.0f : o[e + 1] * f[e + 1];
                            const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? x : y, 1);
                            const __nv_bfloat162 two = __floats2bfloat162_rn(odd ? other : x, odd ? y : other);
                            if (decltype(all)::value || v + e + (lane & 1) < at.tile.rows)
                                *reinterpret_cast<__nv_bfloat162 *>(
                                    out + static_cast<uint32_t>((v + e) * p.latent + h * 128)) = two;
                        }
                    }
            };
            if (at.tile.rows == NR)
                write(std::true_type{});
            else
                write(std::false_type{});
        } else if (p.cluster) {
            // The rings are used up: this CTA's part stays there for the cluster to join.
            float *sums = reinterpret_cast<float *>(pairs);
            for (int h = 0; h < plan.pairs; ++h)
#pragma unroll
                for (int v = 0; v < NR; v += 16) {
                    if (((h * (NR / 16) + v / 16) & 1) != group) continue;
                    float o[16], f[16];
                    shared16(&c.factor[v], f);
                    tc_load16(lanes + O_COL + h * NR + v, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        sums[(v + e) * p.latent + h * 128 + w * 32 + lane] = f[e] == 0.0f ? 0.0f : o[e];
                }
        } else {
            Part &part = parts[2 * blockIdx.x + (at.b0 == 0 ? 1 : 0)];
            if (tid < NR) {
                part.m[tid] = c.ref[tid];
                part.l[tid] = c.l[tid];
            }
            for (int h = 0; h < plan.pairs; ++h)
#pragma unroll
                for (int v = 0; v < NR; v += 16) {
                    if (((h * (NR / 16) + v / 16) & 1) != group) continue;
                    float o[16], f[16];
                    shared16(&c.factor[v], f);
                    tc_load16(lanes + O_COL + h * NR + v, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        part.sum[(v + e) * p.latent + h * 128 + w * 32 + lane] = f[e] == 0.0f ? 0.0f : o[e];
                }
        }
        if (!p.cluster && at.b0 == 0 && tid == 0 && (by_tile || !direct)) {
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
        soft_sync();
    }
    if (!p.cluster && !by_tile && !split_here && tid == 0) joints[blockIdx.x] = Joint{0, 0, 0, 0};
}

template <int NR>
__global__ void __launch_bounds__(NT, 1) attend_kernel(const __grid_constant__ AttendParams p,
                                                       const __grid_constant__ CUtensorMap map) {
    extern __shared__ char raw[];
    char *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const Plan plan = make_plan<NR>(p.latent);
    char *pairs = smem + plan.query_bytes, *ropes = pairs + plan.pair_slots * 2 * CHUNK;
    Ctrl &c = *reinterpret_cast<Ctrl *>(ropes + plan.rope_slots * CHUNK);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < MAX_SLOTS; ++s) {
            mbar_init(&c.pair_full[s], p.tiled ? 1 : LOAD);
            mbar_init(&c.rope_full[s], p.tiled ? 2 : ROPE_LOAD + 1);
            mbar_init(&c.pair_empty[s], 1);
            mbar_init(&c.rope_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&c.s_full[s], 1);
            mbar_init(&c.s_empty[s], SOFT / 32);
            mbar_init(&c.drain[s], 1);
        }
        for (int s = 0; s < BLOCKS; ++s) {
            mbar_init(&c.p_full[s], SOFT / 32);
            mbar_init(&c.o_done[s], 1);
        }
        mbar_init(&c.q_first, SOFT);
        mbar_init(&c.q_full, LOAD);
        mbar_init(&c.q_empty, 1);
        c.abort = 0;
        fence_mbar_init();
    }
    if (warp == NT / 32 - 1) {
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
    if (warp < SOFT / 32) soften<NR>(p, c, plan, smem_addr(smem), pairs, ropes, tmem);
    else if (warp < (SOFT + LOAD) / 32) load_pairs<NR>(p, &map, c, plan, smem_addr(smem), smem_addr(pairs));
    else if (warp < (SOFT + LOAD + ROPE_LOAD) / 32) load_ropes(p, &map, c, plan, smem_addr(ropes));
    else if (warp < NT / 32 - 1)
        multiply_scores<NR>(p, c, plan, smem_addr(smem), smem_addr(pairs), smem_addr(ropes), tmem);
    else multiply_sums<NR>(p, c, plan, smem_addr(pairs), smem_addr(ropes), tmem);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == NT / 32 - 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    if (p.cluster > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        static_assert(sizeof(c.rows) >= ROWS * MAX_CLUSTER * sizeof(float));
        if (c.ranks > 1) join_cluster<NT>(p, c, pairs, reinterpret_cast<float(*)[MAX_CLUSTER]>(c.rows));
        __syncwarp();
        cluster_arrive();                      // no CTA leaves while others read its part
        cluster_wait();
    }
}

// Joins a split tile's parts: each part's sum weighs 2^(its maximum - the
// largest). Parts are added in an order of their own: results do not depend on
// which CTA finished first.
__device__ __forceinline__ const Part &part_of(const Part *parts, const Joint &j, int i) {
    return parts[2 * (j.cta + i) + (i == 0 ? 1 : 0)];
}

// Many parts of few tiles: a CTA per row, the parts dealt to groups of threads.
template <int THREADS>
__device__ void join_wide(const AttendParams &p, const Part *parts, const Joint &j, const Tile &t, int row) {
    __shared__ float weight[512], red[THREADS / 32];
    __shared__ __align__(16) float partial[THREADS * 4];
    const int tid = threadIdx.x;
    float mine = -INFINITY;
    for (int i = tid; i < j.parts; i += THREADS) mine = fmaxf(mine, part_of(parts, j, i).m[row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mine = fmaxf(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, o));
    if ((tid & 31) == 0) red[tid >> 5] = mine;
    __syncthreads();
    float top = red[0];
#pragma unroll
    for (int i = 1; i < THREADS / 32; ++i) top = fmaxf(top, red[i]);
    __syncthreads();
    float sum = 0.0f;
    for (int i = tid; i < j.parts; i += THREADS) {
        const float f = part_weight(part_of(parts, j, i).m[row], top);
        weight[i] = f;
        sum += f * part_of(parts, j, i).l[row];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    float l = 0.0f;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) l += red[i];
    const int vecs = p.latent / 4, groups = THREADS / vecs, g = tid / vecs, v = tid - g * vecs;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (g < groups) {
#pragma unroll 8
        for (int i = g; i < j.parts; i += groups)
            add4(acc, weight[i], reinterpret_cast<const float4 *>(part_of(parts, j, i).sum + row * p.latent)[v]);
        reinterpret_cast<float4 *>(partial)[tid] = acc;
    }
    __syncthreads();
    if (g == 0) {
        for (int k = 1; k < groups; ++k) add4(acc, 1.0f, reinterpret_cast<const float4 *>(partial)[k * vecs + v]);
        write4(p, static_cast<int64_t>(t.base) + row, v, acc, l);
        if (v == 0 && p.lse) p.lse[t.base + row] = finished_lse(top, l);
    }
}

// Few parts (32 at most) of many tiles: a warp per row.
__device__ void join_narrow(const AttendParams &p, const Part *parts, const Joint &j, const Tile &t, int row) {
    const int lane = threadIdx.x & 31;
    const bool on = lane < j.parts;
    const float m = on ? part_of(parts, j, lane).m[row] : -INFINITY;
    float l = on ? part_of(parts, j, lane).l[row] : 0.0f, top = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float f = part_weight(m, top);
    l *= f;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int quads = p.latent / 128;
#pragma unroll 2
    for (int i = 0; i < j.parts; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, i);
        const float4 *from = reinterpret_cast<const float4 *>(part_of(parts, j, i).sum + row * p.latent);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < quads) add4(acc[k], w, from[k * 32 + lane]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < quads) write4(p, static_cast<int64_t>(t.base) + row, k * 32 + lane, acc[k], l);
    if (lane == 0 && p.lse) p.lse[t.base + row] = finished_lse(top, l);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) join_kernel(const __grid_constant__ AttendParams p, int wide) {
    grid_dependents_release();
    grid_dependency_wait();
    const Part *parts = reinterpret_cast<const Part *>(p.workspace);
    const Joint j = reinterpret_cast<const Joint *>(parts + 2 * p.sms)[blockIdx.x];
    if (j.parts < 2) return;
    const Tile t = tile_at(p, j.tile);
    if (wide) {
        if (static_cast<int>(blockIdx.y) < t.rows) join_wide<THREADS>(p, parts, j, t, blockIdx.y);
        return;
    }
    const int first = blockIdx.y * (THREADS / 32), row = first + (threadIdx.x >> 5);
    if (j.parts <= 32) {
        if (row < t.rows) join_narrow(p, parts, j, t, row);
        return;
    }
    // (A long tile among short ones may have more parts than a warp has lanes.)
    for (int r = first; r < min(first + THREADS / 32, t.rows); ++r) {
        join_wide<THREADS>(p, parts, j, t, r);
        __syncthreads();
    }
}

}  // namespace

// ------------------------------------------------------------------ host side

namespace {

// Fitted to both sides' times in graphs at 230 sizes of listed rows (1 to 152 tiles of
// 16, 32 and 64 rows, 4 to 64 blocks): the choice is 0.4 % slower than the best on
// average, 11 % at most. Some of both sides, shares against the cluster: 1 tile of 16
// rows x 32 blocks 12.1 / 11.8 us (16 CTAs), x 64 12.8 / 14.3; 64 rows x 8 14.0 / 13.6
// (8), x 16 14.3 / 14.8 (8); 36 tiles of 16 rows x 64 39.5 / 36.1 (4); unsplit, 72 x 16
// 28.8 / 26.8, 96 x 32 52.3 / 48.6, 64 x 32 40.2 / 46.2. A cluster of 16 joins tiles of
// 64 rows slower than one of 8 (1 x 16 blocks: 16.5, 14.8). Called one by one, 1 request
// of 16 heads x 64 blocks of pages takes 22.8 us a call in shares, 16.5 as a cluster; in
// graphs 14.5 and 15.0 (2 requests: 16.0, 14.9). TILE: see the schedule.
constexpr Costs COSTS = {2, 5, 4, 3, 2};

Device g_device[64];

template <int NR>
const void *attend_fn() {
    return reinterpret_cast<const void *>(&attend_kernel<NR>);
}

cudaError_t device(Device *&out) {
    return device(g_device, {attend_fn<16>(), attend_fn<32>(), attend_fn<64>()}, NT, out);
}

}  // namespace

int64_t workspace_bytes() {
    Device *d = nullptr;
    if (device(d) != cudaSuccess) return 0;
    return static_cast<int64_t>(d->sms) * static_cast<int64_t>(2 * sizeof(Part) + sizeof(Joint));
}

cudaError_t status_attend(uint32_t *v, bool clear) { return unit_status(v, clear); }

int64_t attend_workspace(AttendParams p) {
    Device *d = nullptr;
    if (device(d) != cudaSuccess) return -1;
    if (p.rows_per_request > p.tokens) p.rows_per_request = p.tokens;
    return deal<KEYS>(p, *d, COSTS).cluster ? 0 : workspace_bytes();
}

cudaError_t launch_attend(AttendParams p, cudaStream_t stream) {
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
    const unsigned grid = plan.grid;
    const int nr = plan.nr;

    // Pages that hold whole blocks: a block is 64 consecutive rows of the cache.
    CUtensorMap map = {};
    p.tiled = p.paged && (1 << p.page_shift) % KEYS == 0 && p.cache_rows >= KEYS ? 1 : 0;
    if (p.tiled) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.latent + LATENT_ROPE),
                                    static_cast<cuuint64_t>(p.cache_rows)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.cache_stride) * 2};
        const cuuint32_t box[2] = {64, KEYS}, steps[2] = {1, 1};
        if (d->encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p.cache), dims, strides, box,
                      steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
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
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    void *args[] = {&p, &map};
    e = cudaLaunchKernelExC(&cfg, nr == 16 ? attend_fn<16>() : nr == 32 ? attend_fn<32>() : attend_fn<64>(), args);
    if (e != cudaSuccess || p.cluster || plan.blocks <= 1) return e;   // tiles of one block are never split
    return launch_join(p, grid, nr, stream);
}

cudaError_t launch_join(const AttendParams &params, unsigned grid, int nr, cudaStream_t stream) {
    AttendParams p = params;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    // A CTA per row where that is few enough CTAs to run at once (many parts each
    // then; the fewer rows, the more threads on each), else a warp per row.
    // (Measured, two tiles of 76 parts: 9.4 us with 256 threads a row, 5.8 with 1024.)
    const unsigned sms = static_cast<unsigned>(p.sms), rows = static_cast<unsigned>(nr);
    const unsigned tiles = static_cast<unsigned>(p.tiles) < grid ? static_cast<unsigned>(p.tiles) : grid;
    int wide = tiles * rows <= 8 * sms ? 1 : 0;
    const bool big = tiles * rows <= sms;
    cfg.gridDim = dim3(tiles, wide ? rows : rows / 8, 1);
    cfg.blockDim = dim3(big ? 1024 : 256, 1, 1);
    void *join_args[] = {&p, &wide};
    return cudaLaunchKernelExC(&cfg,
                               big ? reinterpret_cast<const void *>(&join_kernel<1024>)
                                   : reinterpret_cast<const void *>(&join_kernel<256>),
                               join_args);
}

}  // namespace topk::latent
