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
// What bounds it. Few heads: DRAM (32 requests x 16 heads x up to 16384 tokens: 85
// us, 5.2 TB/s). 64 rows a tile: shared memory. A block's operands leave it 36 x 4
// KB (scores) and 16 x 6 KB (sums) at 128 bytes a cycle and its rows come in once:
// about 2500 cycles a block, what a chunk of 509 tokens x 128 heads over 9000 takes
// (1.22 ms, 1.0 PFLOP/s; tensor pipes 66 % active). More rows a tile would halve
// that but neither their queries (74 KB for 64) nor their sums have room. Listed
// rows (no TMA boxes) add the copies' latency: 3200 cycles a block at two blocks in
// flight, tile ends included (512 tokens x 128 heads x 2048: 356 us).

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <cfloat>
#include <mutex>
#include <type_traits>
#include <utility>

#include "common.cuh"
#include "latent.h"

namespace topk::latent {

namespace {

constexpr int SOFT = 256;                    // warps 0 to 7: softmax and outputs, in two groups
constexpr int LOAD = 128;                    // warps 8 to 11: query rows, the latent part of cache rows
constexpr int ROPE_LOAD = 32;                // warp 12: the rotary part
constexpr int NT = SOFT + LOAD + ROPE_LOAD + 64;   // warps 13 and 14: the tensor cores (scores, sums)
constexpr int ROWS = 64;                     // query rows of a tile
constexpr int KEYS = 64;                     // cache rows of a block
constexpr int CHUNK = KEYS * 128;            // bytes of a block's rows at 64 of their values
constexpr int MAX_SLOTS = 12;                // most slots of either ring
constexpr int BLOCKS = 16;                   // blocks that have row numbers and barriers of their own: more
                                             // than the rings hold
constexpr int SMEM = 232448;                 // all of a CTA's shared memory
constexpr uint32_t O_COL = 0, S_COL = 256;   // tensor memory columns: sums (4 x NR), scores (2 x NR)
constexpr float LAZY = 16.0f;                // the reference may lag the maximum by this much (log2)
constexpr float LOWEST = -FLT_MAX;           // the reference of a row that has seen no score above -inf: finite, so
                                             // that 2^(-inf - reference) is 0 in every block
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
using u64 = unsigned long long;

struct Ctrl {
    u64 pair_full[MAX_SLOTS], rope_full[MAX_SLOTS];     // a slot's rows are in
    u64 pair_empty[MAX_SLOTS], rope_empty[MAX_SLOTS];   // a slot is used up
    u64 s_full[2], s_empty[2];                 // scores written / read
    u64 p_full[BLOCKS], o_done[BLOCKS];        // a block's weights are in / its sums are added (one each: who waits
                                               // for one block may find later ones done, and two phases of one
                                               // barrier look like none)
    u64 q_first, q_full, q_empty;              // the first query tile, a later one is in / it is used up
    u64 drain[2];
    long long sums[NT / 32];
    int32_t longest[NT / 32];
    int32_t first_tile, first_unit;
    int32_t ranks;                             // CTAs of the cluster that have blocks
    long long begin, share, total;
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

__device__ __forceinline__ void arrive(u64 *bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Bounded wait by a whole warp. Once a wait of the CTA gave up, every later one
// returns at once and all warps go on to the end of the schedule on whatever the
// memories hold, inside the same bounds: they meet at barriers, so none may leave
// early.
__device__ __forceinline__ void wait(u64 *bar, uint32_t parity, Ctrl &c) {
    mbar_wait(bar, parity & 1u, &c.abort);
    __syncwarp();
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane of a converged warp, by elect.sync: the compiler then knows that what
// follows is one thread's and keeps descriptors in uniform registers (with
// `lane == 0` in its place a step takes twice as long to issue).
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void tc_commit(u64 *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

// Waits for all that the warp's elected lane issued: nothing may be running on
// the tensor cores when their memory is freed.
__device__ __forceinline__ void drain(u64 *bar, bool one) {
    if (one) tc_commit(bar);
    __syncwarp();
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, 0) && global_timer_ns() - t0 < WAIT_LIMIT_NS) {
    }
}

// Matrix descriptor of a 128-byte-swizzled operand. `lead`: bytes between
// 64-value groups along the major dimension (only where that dimension is not
// the summed one); groups of 8 rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t matrix(uint32_t addr, uint32_t lead) {
    return (static_cast<uint64_t>(addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: BF16 x BF16 -> FP32, M x N; `along`: both operands are
// stored with the summed dimension across rows (else along them).
__host__ __device__ constexpr uint32_t instruction(int m, int n, bool along) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (along ? 3u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// Eight columns of this warp's first 16 lanes, N groups of them: thread t gets
// of group j the values of lane t / 4 (v[4 j], v[4 j + 1]) and of lane t / 4 + 8
// (v[4 j + 2], v[4 j + 3]) at columns 8 j + 2 (t % 4) and the next.
template <int N>
__device__ __forceinline__ void tc_load_groups(uint32_t addr, float (&v)[4 * N]) {
    uint32_t r[4 * N];
    if constexpr (N == 1)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr));
    else if constexpr (N == 2)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(addr));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(addr));
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 columns of this warp's 32 lanes, one lane per thread.
__device__ __forceinline__ void tc_load16(uint32_t addr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Sixteen of a shared array's floats, 16 bytes a load (as single loads they
// outweighed all else of an output: 5.5 us a tile of 64 x 512 values).
__device__ __forceinline__ void shared16(const float *from, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(from + i);
        v[i] = x.x;
        v[i + 1] = x.y;
        v[i + 2] = x.z;
        v[i + 3] = x.w;
    }
}

__device__ __forceinline__ void tc_store16(uint32_t addr, const float (&v)[16]) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
            r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}

// 16 bytes from global to shared memory, or zeros (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// 64 rows of 64 values from column x and row y, completing on `bar`.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, u64 *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// An arrival on `bar` once this thread's copies so far are done.
__device__ __forceinline__ void copies_arrive(u64 *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest of |a|, |b| and m, NaN if one of them is.
__device__ __forceinline__ float largest(float m, float a, float b) {
    float y;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(m), "f"(a), "f"(b));
    return y;
}

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

// ------------------------------------------------------------------ the schedule

// A tile is up to 64 consecutive (token, head) rows of one request (paged form)
// or token (selected form).
struct Tile {
    int32_t base, rows;          // first flat row (token * heads + head), rows
    int32_t token, last;         // first and last token
    int32_t request;
};

__device__ __forceinline__ Tile tile_at(const AttendParams &p, int32_t t) {
    Tile r;
    r.request = t / p.tiles_per_request;
    const int32_t per = p.rows_per_request;
    const int32_t first = r.request * per;
    const int32_t end = min(p.tokens, first + per) * p.heads;
    r.base = first * p.heads + (t - r.request * p.tiles_per_request) * ROWS;
    r.rows = min(ROWS, end - r.base);
    r.token = r.base / p.heads;
    r.last = (r.base + r.rows - 1) / p.heads;
    return r;
}

__device__ __forceinline__ int32_t token_len(const AttendParams &p, int32_t token) {
    return min(max(p.valid_len[token], 0), p.width);
}

// Cache rows that a tile's longest row may see, and blocks of them (at least
// one: a tile that sees nothing still writes its outputs).
__device__ __forceinline__ int32_t tile_len(const AttendParams &p, const Tile &t) {
    if (!p.paged) return p.k;
    int32_t n = 0;
    for (int32_t i = t.token; i <= t.last; ++i) n = max(n, token_len(p, i));
    return n;
}

// What split tiles cost besides their blocks, in blocks / 48 (SPLIT_UNIT): a part
// and a tile to join. (Fitted with deal()'s costs.)
constexpr int SPLIT_UNIT = 48;
__host__ __device__ __forceinline__ int64_t split_cost(int64_t parts, int64_t tiles) { return parts + 3 * tiles; }

__device__ __forceinline__ int32_t blocks_of(int32_t len) { return max(1, (len + KEYS - 1) / KEYS); }

// As tile_len, by a whole warp; low: the tile's smallest length.
__device__ __forceinline__ int32_t tile_len_warp(const AttendParams &p, const Tile &t, int lane, int32_t &low) {
    low = INT32_MAX;
    if (!p.paged) return p.k;
    int32_t n = 0;
    for (int32_t i = t.token + lane; i <= t.last; i += 32) {
        const int32_t v = token_len(p, i);
        n = max(n, v);
        low = min(low, v);
    }
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    return __reduce_max_sync(0xFFFFFFFFu, n);
}

// All blocks of all tiles in order are cut into equal shares, one per CTA: a
// CTA's share is a run of pieces, each part or all of one tile's blocks. Where a
// CTA has several tiles, a tile counts TILE_COST blocks more than it has: its
// query, first reference and outputs (854 tiles of 1 to 4 blocks: 97 us counted
// as none, 72 as five). Or each CTA has one tile: a cluster's CTAs share one where
// the host chose so, and pages whose tiles are about as many as the CTAs and about
// as long as each other are not split, which only the lengths here can tell.
struct Cursor {
    int32_t next_tile, next_unit;
    long long left;
    Tile tile;
    int32_t b0, b1, blocks, len, low;   // the piece: blocks [b0, b1) of `blocks`
    int32_t u0, u1, units;              // the same with the tile's own cost in front
    __device__ Cursor(const Ctrl &c)
        : next_tile(c.first_tile), next_unit(c.first_unit),
          left(min(c.begin + c.share, c.total) - c.begin) {}
    __device__ bool next(const AttendParams &p, int lane) {
        if (left <= 0) return false;
        tile = tile_at(p, next_tile);
        len = tile_len_warp(p, tile, lane, low);
        blocks = blocks_of(len);
        units = blocks + p.tile_cost;
        u0 = next_unit;
        u1 = static_cast<int32_t>(min(static_cast<long long>(units), u0 + left));
        b0 = max(0, u0 - p.tile_cost);
        b1 = max(0, u1 - p.tile_cost);
        left -= u1 - u0;
        ++next_tile;
        next_unit = 0;
        return b1 > b0;                 // (a share that ends in a tile's cost leaves it to the next CTA)
    }
};

// The CTA's share, by all threads of the CTA.
__device__ __forceinline__ void make_schedule(const AttendParams &p, Ctrl &c) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.cluster) {                           // a tile per cluster, its blocks in equal runs
        if (warp == 0) {
            const int32_t tile = blockIdx.x / p.cluster, rank = blockIdx.x - tile * p.cluster;
            int32_t low;
            const int32_t n = blocks_of(tile_len_warp(p, tile_at(p, tile), lane, low));
            const int32_t per = (n + p.cluster - 1) / p.cluster;
            if (lane == 0) {
                c.first_tile = tile;
                c.first_unit = rank * per;
                c.begin = 0;
                c.share = c.total = max(0, min(per, n - rank * per));
                c.ranks = (n + per - 1) / per;
            }
        }
        __syncthreads();
        return;
    }
    if (!p.paged) {
        if (tid == 0) {
            const long long n = blocks_of(p.k) + p.tile_cost;
            c.total = n * p.tiles;
            c.share = max(static_cast<long long>(p.min_share), (c.total + gridDim.x - 1) / gridDim.x);
            c.begin = min(c.total, c.share * blockIdx.x);
            c.first_tile = static_cast<int32_t>(c.begin / n);
            c.first_unit = static_cast<int32_t>(c.begin % n);
        }
        __syncthreads();
        return;
    }
    const int32_t per = (p.tiles + NT - 1) / NT;
    const int32_t t0 = min(p.tiles, tid * per), t1 = min(p.tiles, t0 + per);
    long long sum = 0;
    int32_t longest = 0;
    for (int32_t t = t0; t < t1; ++t) {
        const int32_t n = blocks_of(tile_len(p, tile_at(p, t)));
        sum += n + p.tile_cost;
        longest = max(longest, n);
    }
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    long long pre = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, pre, o);
        if (lane >= o) pre += v;
    }
    if (lane == 31) {
        c.sums[warp] = pre;
        c.longest[warp] = longest;
    }
    __syncthreads();
    long long before = pre - sum, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const long long v = c.sums[w];
        before += w < warp ? v : 0;
        total += v;
        longest = max(longest, c.longest[w]);
    }
    const long long share = max(static_cast<long long>(p.min_share), (total + gridDim.x - 1) / gridDim.x);
    const long long begin = min(total, share * static_cast<long long>(blockIdx.x));
    const int32_t ctas = static_cast<int32_t>(gridDim.x);
    if (p.tiles <= ctas && longest <= share + split_cost(ctas, p.tiles) / SPLIT_UNIT) {
        if (warp == 0) {                       // every tile to a CTA of its own
            const int32_t tile = blockIdx.x;
            int32_t n = 0, low;
            if (tile < p.tiles) n = blocks_of(tile_len_warp(p, tile_at(p, tile), lane, low));
            if (lane == 0) {
                c.first_tile = tile;
                c.first_unit = 0;
                c.begin = 0;
                c.share = c.total = n;
            }
        }
        __syncthreads();
        return;
    }
    if (tid == 0) {
        c.total = total;
        c.share = share;
        c.begin = begin;
    }
    if (begin >= before && begin < before + sum) {
        long long at = before;
        for (int32_t t = t0; t < t1; ++t) {
            const int32_t n = blocks_of(tile_len(p, tile_at(p, t))) + p.tile_cost;
            if (begin < at + n) {
                c.first_tile = t;
                c.first_unit = static_cast<int32_t>(begin - at);
                break;
            }
            at += n;
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------ the warps' parts

// The row numbers of a tile's blocks. fetch() only loads entry j of the list or
// pages, row() makes the cache row of it (-1 for none) a block later: a warp
// that looked at the value at once would stand still until it came.
struct RowList {
    const int32_t *list;
    int32_t len;
    __device__ RowList(const AttendParams &p, const Cursor &at)
        : list(p.paged ? p.table + static_cast<int64_t>(at.tile.request) * p.table_stride
                       : p.selected + static_cast<int64_t>(at.tile.token) * p.selected_stride),
          len(min(at.len, at.b1 * KEYS)) {}
    __device__ int32_t fetch(const AttendParams &p, int32_t j) const {
        return j < len ? __ldg(list + (p.paged ? j >> p.page_shift : j)) : -1;
    }
    __device__ int32_t row(const AttendParams &p, int32_t fetched, int32_t j) const {
        const int64_t v = p.paged ? static_cast<int64_t>(fetched) * p.block_rows + (j & ((1 << p.page_shift) - 1))
                                  : fetched;
        return j < len && v >= 0 && v < p.cache_rows ? static_cast<int32_t>(v) : -1;
    }
};

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

// After a wait that gave up: no copy may be in flight into shared memory when the
// CTA ends, so wait (with its own limit) for the last ones into each slot. Copy q
// went into slot q % slots for the q / slots-th time, q = last, last - step, ..
__device__ __forceinline__ void settle(u64 *full, int32_t last, int step, int slots) {
    const uint64_t t0 = global_timer_ns();
    for (int32_t q = last; q >= 0 && q > last - slots; q -= step)
        while (!mbar_try_wait(&full[q % slots], static_cast<uint32_t>(q / slots) & 1u) &&
               global_timer_ns() - t0 < WAIT_LIMIT_NS) {
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
    const char *cache = reinterpret_cast<const char *>(p.cache) + piece * 16;
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
    const char *cache = reinterpret_cast<const char *>(p.cache) + plan.pairs * 256 + piece * 16;
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

struct Part {                                  // a piece's unfinished rows in the workspace
    float sum[ROWS * LATENT_MAX];
    float m[ROWS], l[ROWS];
};

struct Joint {                                 // a split tile: where its parts are
    int32_t tile, parts, cta, unused;
};

__device__ __forceinline__ float finished_lse(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2; }
__device__ __forceinline__ float finished(float sum, float l) { return l == 0.0f ? 0.0f : sum / l; }   // NaN stays NaN

// Combines v[0 .. N) over the eight lanes that share lane % 4: afterwards a
// lane's v[j] is the eight lanes' value across_index() + j (N / 8 of them).
template <int N, int O = 16, int SIZE, class Op>
__device__ __forceinline__ void across_lanes(float (&v)[SIZE], Op op) {
    if constexpr (O >= 4) {
        constexpr int H = N / 2;
        if constexpr (H > 0) {
            const bool up = (threadIdx.x & O) != 0;
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const float other = __shfl_xor_sync(0xFFFFFFFFu, up ? v[j] : v[j + H], O);
                v[j] = op(up ? v[j + H] : v[j], other);
            }
            across_lanes<H, O / 2>(v, op);
        } else {
            v[0] = op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], O));
            across_lanes<1, O / 2>(v, op);
        }
    }
}

template <int N>
__device__ __forceinline__ int across_index() {
    int r = 0;
#pragma unroll
    for (int o = 16, n = N / 2; o >= 4 && n; o >>= 1, n /= 2) r += threadIdx.x & o ? n : 0;
    return r;
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

__device__ __forceinline__ float part_weight(float m, float top) { return m == -INFINITY ? 0.0f : exp2_fast(m - top); }

__device__ __forceinline__ void add4(float4 &a, float f, const float4 &x) {
    a.x += f * x.x;
    a.y += f * x.y;
    a.z += f * x.z;
    a.w += f * x.w;
}

__device__ __forceinline__ void write4(const AttendParams &p, int64_t row, int v, const float4 &a, float l) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(finished(a.x, l), finished(a.y, l));
    const __nv_bfloat162 hi = __floats2bfloat162_rn(finished(a.z, l), finished(a.w, l));
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t *>(&lo);
    o.y = *reinterpret_cast<const uint32_t *>(&hi);
    reinterpret_cast<uint2 *>(p.out + row * p.latent)[v] = o;
}

__device__ __forceinline__ float ld_peer_f(const void *p, uint32_t rank) {
    return __uint_as_float(ld_peer(peer_addr(p, rank)));
}

__device__ __forceinline__ float4 ld_peer4(const void *p, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(peer_addr(p, rank))
                 : "memory");
    return v;
}

// Joins a cluster's parts of its tile out of its CTAs' shared memory: each CTA
// takes every cluster-th row, the parts are added in the CTAs' order. First the
// parts' weights, a lane per part, then the sums with all parts' loads in flight.
constexpr int MAX_CLUSTER = 16;

__device__ void join_cluster(const AttendParams &p, Ctrl &c, const char *sums) {
    const Tile t = tile_at(p, c.first_tile);
    const int rank = static_cast<int>(cluster_rank()), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    static_assert(sizeof(c.rows) >= ROWS * MAX_CLUSTER * sizeof(float));
    float(*weight)[MAX_CLUSTER] = reinterpret_cast<float(*)[MAX_CLUSTER]>(c.rows);   // (row numbers: used up)
    for (int row = rank + p.cluster * warp; row < t.rows; row += p.cluster * (NT / 32)) {
        const bool on = lane < c.ranks;
        const float m = on ? ld_peer_f(&c.ref[row], lane) : -INFINITY;
        float l = on ? ld_peer_f(&c.l[row], lane) : 0.0f, top = m;
#pragma unroll
        for (int o = MAX_CLUSTER / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float f = part_weight(m, top);
        l *= f;
#pragma unroll
        for (int o = MAX_CLUSTER / 2; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (lane < MAX_CLUSTER) weight[row][lane] = f;
        if (lane == 0) {
            c.factor[row] = l;
            if (p.lse) p.lse[t.base + row] = finished_lse(top, l);
        }
    }
    __syncthreads();
    const int vecs = p.latent / 4, groups = NT / vecs, g = threadIdx.x / vecs, v = threadIdx.x - g * vecs;
    if (g >= groups) return;
    for (int row = rank + p.cluster * g; row < t.rows; row += p.cluster * groups) {
        float4 x[MAX_CLUSTER], acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < MAX_CLUSTER; ++i)
            if (i < c.ranks) x[i] = ld_peer4(sums + (row * p.latent + v * 4) * 4, i);
#pragma unroll
        for (int i = 0; i < MAX_CLUSTER; ++i)
            if (i < c.ranks) add4(acc, weight[row][i], x[i]);
        write4(p, static_cast<int64_t>(t.base) + row, v, acc, c.factor[row]);
    }
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
    make_schedule(p, c);
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
        if (c.ranks > 1) join_cluster(p, c, pairs);
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

struct Device {
    std::once_flag once;
    cudaError_t err = cudaSuccess;
    int sms = 0;
    int clusters[5] = {};                      // of 1, 2, 4, 8, 16 CTAs that run at once
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
};
Device g_device[64];

template <int NR>
const void *attend_fn() {
    return reinterpret_cast<const void *>(&attend_kernel<NR>);
}

cudaError_t device(Device *&out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    Device &d = g_device[dev];
    std::call_once(d.once, [&]() {
        cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        for (const void *fn : {attend_fn<16>(), attend_fn<32>(), attend_fn<64>()})
            for (const auto &set : {std::pair{cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM},
                                    std::pair{cudaFuncAttributeNonPortableClusterSizeAllowed, 1}})
                if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, set.first, set.second);
        d.clusters[0] = d.sms;
        for (int i = 1; i < 5 && e == cudaSuccess; ++i) {
            cudaLaunchAttribute a = {};
            a.id = cudaLaunchAttributeClusterDimension;
            a.val.clusterDim.x = 1u << i;
            a.val.clusterDim.y = a.val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1u << i, 1, 1);
            cfg.blockDim = dim3(NT, 1, 1);
            cfg.dynamicSmemBytes = SMEM;
            cfg.attrs = &a;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&d.clusters[i], attend_fn<64>(), &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                d.clusters[i] = 0;             // (a size that the device does not take)
            }
        }
        cudaDriverEntryPointQueryResult found;
        void *f = nullptr;
        if (e == cudaSuccess)
            e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        if (e == cudaSuccess && (found != cudaDriverEntryPointSuccess || !f)) e = cudaErrorNotSupported;
        d.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        if (e == cudaSuccess && d.sms > 512) e = cudaErrorNotSupported;   // (join_kernel's weights)
        d.err = e;
    });
    out = &d;
    return d.err;
}

}  // namespace

int64_t workspace_bytes() {
    Device *d = nullptr;
    if (device(d) != cudaSuccess) return 0;
    return static_cast<int64_t>(d->sms) * static_cast<int64_t>(2 * sizeof(Part) + sizeof(Joint));
}

cudaError_t status_attend(uint32_t *v, bool clear) { return unit_status(v, clear); }

namespace {

// How a call's blocks are dealt: the tiles, and either equal shares of all blocks
// for every SM with the split tiles joined by a second kernel, or (cluster > 0)
// one cluster per tile, joined through its shared memory.
struct Deal {
    int64_t tiles, blocks;                     // tiles; blocks of a tile at most
    int32_t tiles_per_request, cluster;
    unsigned grid;
    int nr;
};

constexpr int MIN_SHARE = 2;                   // blocks of a CTA in equal shares
constexpr int TILE_COST = 5;                   // what a tile costs besides its blocks, in blocks
constexpr int CLUSTER_COST = 4;                // what a cluster of several costs a tile, in blocks
constexpr int SHARES_COST = 3;                 // what parts and the second kernel cost at least
constexpr int LENGTHS_COST = 2;                // what the shares of pages cost besides: every CTA adds up all lengths

Deal deal(const AttendParams &p, const Device &d) {
    Deal r = {};
    const int64_t per = static_cast<int64_t>(p.rows_per_request) * p.heads;
    const int64_t full = p.tokens / p.rows_per_request;
    const int64_t rest = p.tokens % p.rows_per_request * static_cast<int64_t>(p.heads);
    r.tiles_per_request = static_cast<int32_t>((per + ROWS - 1) / ROWS);
    r.tiles = full * r.tiles_per_request + (rest + ROWS - 1) / ROWS;
    const int64_t rows = full > 0 ? per : rest;
    r.nr = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    r.blocks = (static_cast<int64_t>(p.paged ? p.width : p.k) + KEYS - 1) / KEYS;
    if (r.blocks < 1) r.blocks = 1;
    // The least of the expected times, in blocks of a CTA / 48: equal shares against every
    // cluster size that runs at once. Costs fitted to both sides' times in graphs at 230 sizes
    // of listed rows (1 to 152 tiles of 16, 32 and 64 rows, 4 to 64 blocks): the choice is 0.4 %
    // slower than the best on average, 11 % at most. Shares count half a block more than
    // that: called one by one they cost the host a second launch and scratch (1 request of 16
    // heads x 64 blocks of pages: 22.8 us a call against 16.5). Some of both sides, shares
    // against the cluster: 1 tile of 16 rows x 32 blocks 12.1 / 11.8 us (16 CTAs), x 64 12.8 /
    // 14.3; 64 rows x 8 14.0 / 13.6 (8), x 16 14.3 / 14.8 (8); 36 tiles of 16 rows x 64 39.5 /
    // 36.1 (4); unsplit, 72 x 16 28.8 / 26.8, 96 x 32 52.3 / 48.6, 64 x 32 40.2 / 46.2. A
    // cluster of 16 joins tiles of 64 rows slower than one of 8 (1 x 16 blocks: 16.5, 14.8).
    // How long requests really are is not known here: of pages, shares may come to as little as
    // MIN_SHARE, and a tile goes to a cluster or to one CTA only where that is as fast even then
    // (16 heads x 64 blocks: 1 request 14.5 us in shares, 15.0 as a cluster; 2: 16.0, 14.9).
    // Beyond, make_schedule looks at the lengths.
    const int64_t parts = (r.tiles * r.blocks + MIN_SHARE - 1) / MIN_SHARE;
    const int64_t even = (r.tiles * r.blocks + d.sms - 1) / d.sms;
    const int64_t share = p.paged || even < MIN_SHARE ? MIN_SHARE : even;
    int64_t least = (share + SHARES_COST + (p.paged ? LENGTHS_COST : 0)) * SPLIT_UNIT + SPLIT_UNIT / 2 +
                    split_cost(parts < d.sms ? parts : d.sms, r.tiles);
    for (int i = r.nr > 32 ? 3 : 4; i >= 0; --i) {
        const int64_t size = 1 << i, run = (r.blocks + size - 1) / size;
        const int64_t cost = (run + (size > 1 ? CLUSTER_COST : 0)) * SPLIT_UNIT;
        if (size > r.blocks || r.tiles > d.clusters[i] || cost > least) continue;
        r.cluster = static_cast<int32_t>(size);
        least = cost;
    }
    const int64_t want = r.cluster ? r.tiles * r.cluster : parts;
    r.grid = static_cast<unsigned>(r.cluster || want < d.sms ? want : d.sms);
    return r;
}

}  // namespace

int64_t attend_workspace(AttendParams p) {
    Device *d = nullptr;
    if (device(d) != cudaSuccess) return -1;
    if (p.rows_per_request > p.tokens) p.rows_per_request = p.tokens;
    return deal(p, *d).cluster ? 0 : workspace_bytes();
}

cudaError_t launch_attend(AttendParams p, cudaStream_t stream) {
    Device *d = nullptr;
    cudaError_t e = device(d);
    if (e != cudaSuccess) return e;
    if (p.rows_per_request > p.tokens) p.rows_per_request = p.tokens;   // (one request)
    const Deal plan = deal(p, *d);
    p.tiles_per_request = plan.tiles_per_request;
    p.tiles = static_cast<int32_t>(plan.tiles);
    p.cluster = plan.cluster;
    p.tile_cost = plan.tiles > d->sms ? TILE_COST : 0;
    p.min_share = MIN_SHARE;
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
        if (d->encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(p.cache), dims, strides, box,
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
    cfg.numAttrs = 1;
    // A CTA per row where that is few enough CTAs to run at once (many parts each
    // then; the fewer rows, the more threads on each), else a warp per row.
    // (Measured, two tiles of 76 parts: 9.4 us with 256 threads a row, 5.8 with 1024.)
    const unsigned sms = static_cast<unsigned>(d->sms), rows = static_cast<unsigned>(nr);
    const unsigned tiles = static_cast<unsigned>(p.tiles) < grid ? static_cast<unsigned>(p.tiles) : grid;
    int wide = tiles * rows <= 8 * sms ? 1 : 0;
    const bool big = tiles * rows <= sms;
    cfg.gridDim = dim3(tiles, wide ? rows : rows / 8, 1);
    cfg.blockDim = dim3(big ? 1024 : 256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    void *join_args[] = {&p, &wide};
    return cudaLaunchKernelExC(&cfg,
                               big ? reinterpret_cast<const void *>(&join_kernel<1024>)
                                   : reinterpret_cast<const void *>(&join_kernel<256>),
                               join_args);
}

}  // namespace topk::latent
