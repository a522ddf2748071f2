// What the attention kernels over latent cache rows share, BF16 or in 4 bits: tensor
// core and copy instructions, the dealing of tiles' blocks to CTAs, and the joining of
// split tiles' parts.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <cfloat>
#include <mutex>
#include <utility>

#include "common.cuh"
#include "latent.h"

namespace topk::latent {

namespace {

constexpr int ROWS = 64;                     // query rows of a tile
constexpr int SMEM = 232448;                 // all of a CTA's shared memory
constexpr float LOWEST = -FLT_MAX;           // the reference of a row that has seen no score above -inf: finite, so
                                             // that 2^(-inf - reference) is 0 in every block
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
using u64 = unsigned long long;

__device__ __forceinline__ void arrive(u64 *bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Bounded wait by a whole warp. Once a wait of the CTA gave up, every later one
// returns at once and all warps go on to the end of the schedule on whatever the
// memories hold, inside the same bounds: they meet at barriers, so none may leave
// early.
template <class Ctrl>
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
// (tc_issue_groups: to be waited for.)
template <int N>
__device__ __forceinline__ void tc_issue_groups(uint32_t addr, uint32_t (&r)[4 * N]) {
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
}

template <int N>
__device__ __forceinline__ void tc_load_groups(uint32_t addr, float (&v)[4 * N]) {
    uint32_t r[4 * N];
    tc_issue_groups<N>(addr, r);
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

// The map's box from column x and row y, completing on `bar`.
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

// ------------------------------------------------------------------ the schedule

// A tile is up to 64 consecutive (token, head) rows of one request (paged form)
// or token (selected form).
struct Tile {
    int32_t base, rows;          // first flat row (token * heads + head), rows
    int32_t token, last;         // first and last token
    int32_t request;
};

// What a CTA (of NT threads at most) knows of its share of the blocks: part of its control block.
template <int NT>
struct Schedule {
    long long sums[NT / 32];
    int32_t longest[NT / 32];
    int32_t first_tile, first_unit;
    int32_t ranks;                             // CTAs of the cluster that have blocks
    long long begin, share, total;
    Tile tile;                                 // the first one
    int32_t len, low;
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

// Cache rows that a tile's longest row may see (blocks of them: at least one, for a
// tile that sees nothing still writes its outputs); low: its shortest row.
__device__ __forceinline__ int32_t tile_len(const AttendParams &p, const Tile &t, int32_t &low) {
    low = INT32_MAX;
    int32_t n = 0;
#pragma unroll 1
    for (int32_t i = t.token; i <= t.last; ++i) {
        const int32_t v = token_len(p, i);
        n = max(n, v);
        low = min(low, v);
    }
    return n;
}

// What split tiles cost besides their blocks, in blocks / 48 (SPLIT_UNIT): a part
// and a tile to join. (Fitted with deal()'s costs.)
constexpr int SPLIT_UNIT = 48;
__host__ __device__ __forceinline__ int64_t split_cost(int64_t parts, int64_t tiles) { return parts + 3 * tiles; }

template <int KEYS>
__device__ __forceinline__ int32_t blocks_of(int32_t len) { return max(1, (len + KEYS - 1) / KEYS); }

// As tile_len, by a whole warp.
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
// CTA has several tiles, a tile counts `tile_cost` blocks more than it has: its
// query, first reference and outputs (854 tiles of 1 to 4 blocks: 97 us counted
// as none, 72 as five). Or each CTA has one tile: a cluster's CTAs share one where
// the host chose so, and pages whose tiles are about as many as the CTAs and about
// as long as each other are not split, which only the lengths here can tell. Whoever
// makes the schedule leaves the first tile in it: a CTA begins with code that nobody
// has fetched yet, of which six roles need not each have a copy.
template <int KEYS>
struct CursorOf {
    int32_t next_tile, next_unit;
    long long left;
    Tile tile;
    int32_t b0, b1, blocks, len, low;   // the piece: blocks [b0, b1) of `blocks`
    int32_t u0, u1, units;              // the same with the tile's own cost in front
    bool first = true;
    template <class Ctrl>
    __device__ CursorOf(const Ctrl &c)
        : next_tile(c.first_tile), next_unit(c.first_unit), left(min(c.begin + c.share, c.total) - c.begin),
          tile(c.tile), len(c.len), low(c.low) {}
    __device__ bool next(const AttendParams &p, int lane) {
        if (left <= 0) return false;
        if (!first) [[unlikely]] {
            tile = tile_at(p, next_tile);
            len = tile_len_warp(p, tile, lane, low);
        }
        first = false;
        blocks = blocks_of<KEYS>(len);
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
template <int KEYS, int NT, int SIZE>
__device__ __forceinline__ void make_schedule(const AttendParams &p, Schedule<SIZE> &c) {
    static_assert(NT <= SIZE);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.cluster) {                           // a tile per cluster, its blocks in equal runs
        if (warp == 0) {
            const int32_t tile = blockIdx.x / p.cluster, rank = blockIdx.x - tile * p.cluster;
            const Tile first = tile_at(p, tile);
            int32_t low;
            const int32_t len = tile_len_warp(p, first, lane, low), n = blocks_of<KEYS>(len);
            const int32_t per = (n + p.cluster - 1) / p.cluster;
            if (lane == 0) {
                c.tile = first;
                c.len = len;
                c.low = low;
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
            const long long n = blocks_of<KEYS>(p.k) + p.tile_cost;
            c.total = n * p.tiles;
            c.share = max(static_cast<long long>(p.min_share), (c.total + gridDim.x - 1) / gridDim.x);
            c.begin = min(c.total, c.share * blockIdx.x);
            c.first_tile = static_cast<int32_t>(c.begin / n);
            c.first_unit = static_cast<int32_t>(c.begin % n);
            c.tile = tile_at(p, c.first_tile);
            c.len = p.k;
            c.low = INT32_MAX;
        }
        __syncthreads();
        return;
    }
    const int32_t per = (p.tiles + NT - 1) / NT;
    const int32_t t0 = min(p.tiles, tid * per), t1 = min(p.tiles, t0 + per);
    Tile tile;
    int32_t len = 0, low = 0;
    long long sum = 0;
    int32_t longest = 0;
#pragma unroll 1
    for (int32_t t = t0; t < t1; ++t) {
        tile = tile_at(p, t);
        len = tile_len(p, tile, low);
        const int32_t n = blocks_of<KEYS>(len);
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
            int32_t n = 0;
            if (blockIdx.x < static_cast<unsigned>(p.tiles)) {
                tile = tile_at(p, blockIdx.x);
                len = tile_len_warp(p, tile, lane, low);
                n = blocks_of<KEYS>(len);
            }
            if (lane == 0) {
                c.tile = tile;
                c.len = len;
                c.low = low;
                c.first_tile = blockIdx.x;
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
#pragma unroll 1
        for (int32_t t = t0; t < t1; ++t) {
            if (per > 1) {                     // (of a single tile they are known)
                tile = tile_at(p, t);
                len = tile_len(p, tile, low);
            }
            const int32_t n = blocks_of<KEYS>(len) + p.tile_cost;
            if (begin < at + n) {
                c.tile = tile;
                c.len = len;
                c.low = low;
                c.first_tile = t;
                c.first_unit = static_cast<int32_t>(begin - at);
                break;
            }
            at += n;
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------ rows, parts, outputs

// The row numbers of a tile's blocks. fetch() only loads entry j of the list or
// pages, row() makes the cache row of it (-1 for none) a block later: a warp
// that looked at the value at once would stand still until it came.
template <int KEYS>
struct RowListOf {
    const int32_t *list;
    int32_t len;
    __device__ RowListOf(const AttendParams &p, const CursorOf<KEYS> &at)
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
// parts' weights (`weight`: ROWS of them, shared memory that is used up), a lane per
// part, then the sums with all parts' loads in flight.
constexpr int MAX_CLUSTER = 16;

template <int NT, class Ctrl>
__device__ void join_cluster(const AttendParams &p, Ctrl &c, const char *sums, float (*weight)[MAX_CLUSTER]) {
    const Tile t = tile_at(p, c.first_tile);
    const int rank = static_cast<int>(cluster_rank()), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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

// Looks at the current device once: `fns`, the kernel's forms by query rows, get their
// attributes.
inline cudaError_t device(Device (&devices)[64], const void *const (&fns)[3], int threads, Device *&out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    Device &d = devices[dev];
    std::call_once(d.once, [&]() {
        cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
        for (const void *fn : fns)
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
            cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
            cfg.dynamicSmemBytes = SMEM;
            cfg.attrs = &a;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&d.clusters[i], fns[2], &cfg) != cudaSuccess) {
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

// How a call's blocks are dealt: the tiles, and either equal shares of all blocks
// for every SM with the split tiles joined by a second kernel, or (cluster > 0)
// one cluster per tile, joined through its shared memory.
struct Deal {
    int64_t tiles, blocks;                     // tiles; blocks of a tile at most
    int32_t tiles_per_request, cluster;
    unsigned grid;
    int nr;
};

// What the dealing goes by, in blocks; fitted to a kernel's times.
struct Costs {
    int min_share;                             // blocks of a CTA in equal shares, at least
    int tile;                                  // what a tile costs besides its blocks
    int cluster;                               // what a cluster of several costs a tile
    int shares;                                // what parts and the second kernel cost at least
    int lengths;                               // what the shares of pages cost besides: every CTA adds up all lengths
};

template <int KEYS>
Deal deal(const AttendParams &p, const Device &d, const Costs &c) {
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
    // cluster size that runs at once. Shares count half a block more than what they cost on the
    // device: called one by one they cost the host a second launch and scratch. How long requests
    // really are is not known here: of pages, shares may come to as little as `min_share`, and a
    // tile goes to a cluster or to one CTA only where that is as fast even then. Beyond,
    // make_schedule looks at the lengths.
    const int64_t parts = (r.tiles * r.blocks + c.min_share - 1) / c.min_share;
    const int64_t even = (r.tiles * r.blocks + d.sms - 1) / d.sms;
    const int64_t share = p.paged || even < c.min_share ? c.min_share : even;
    int64_t least = (share + c.shares + (p.paged ? c.lengths : 0)) * SPLIT_UNIT + SPLIT_UNIT / 2 +
                    split_cost(parts < d.sms ? parts : d.sms, r.tiles);
    for (int i = r.nr > 32 ? 3 : 4; i >= 0; --i) {
        const int64_t size = 1 << i, run = (r.blocks + size - 1) / size;
        const int64_t cost = (run + (size > 1 ? c.cluster : 0)) * SPLIT_UNIT;
        if (size > r.blocks || r.tiles > d.clusters[i] || cost > least) continue;
        r.cluster = static_cast<int32_t>(size);
        least = cost;
    }
    const int64_t want = r.cluster ? r.tiles * r.cluster : parts;
    r.grid = static_cast<unsigned>(r.cluster || want < d.sms ? want : d.sms);
    return r;
}

}  // namespace

}  // namespace topk::latent
