// Attention over latent cache rows on the tensor cores: one persistent kernel
// for both forms, and the kernel that joins the parts of split tiles.

#include <cuda_bf16.h>

#include <mutex>

#include "common.cuh"
#include "latent.h"

namespace topk::latent {

namespace {

constexpr int SOFT = 128;                    // warps 0 to 3: softmax and outputs
constexpr int LOAD = 128;                    // warps 4 to 7: cache rows
constexpr int QLOAD = 64;                    // warps 8 and 9: query rows
constexpr int NT = SOFT + LOAD + QLOAD + 32; // warp 10: the tensor cores
constexpr int NT_JOIN = 256;
constexpr int ROWS = 64;                     // query rows of a tile
constexpr int KEYS = 64;                     // cache rows of a block
constexpr int CHUNK = 64 * 128;              // bytes of 64 rows of 64 values
constexpr int CHUNKS = 27;                   // chunks of shared memory: the query's and the stages'
constexpr int MAX_STAGES = 4;
constexpr uint32_t O_COL = 0, S_COL = 256;   // tensor memory columns: output (4 x NR), scores (2 x 64)
constexpr float LAZY = 8.0f;                 // the reference maximum may lag by this much (log2)
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
using u64 = unsigned long long;

struct Ctrl {
    u64 full[MAX_STAGES], empty[MAX_STAGES];   // a stage's rows are in / its values are used up
    u64 s_full[2], s_empty[2];                 // scores written / read
    u64 p_full, o_done;                        // a block's weights are in / its product is added
    u64 q_full, q_empty;                       // the query tile is in / used up
    u64 drain;
    u64 bad;
    long long sums[NT / 32];
    int32_t first_tile, first_block;
    long long begin, share, total;
    uint32_t tmem;
    volatile uint32_t abort;
    float factor[ROWS], m[ROWS], l[ROWS];
    uint8_t there[MAX_STAGES][KEYS];           // which rows of the stage hold a cache row
};

constexpr int SMEM = CHUNKS * CHUNK + static_cast<int>(sizeof(Ctrl)) + 1024;

__device__ __forceinline__ void arrive(u64 *bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Bounded wait by a whole warp; false, on every lane, once any wait of the CTA
// gave up.
__device__ __forceinline__ bool wait(u64 *bar, uint32_t parity, Ctrl &c) {
    mbar_wait(bar, parity & 1u, &c.abort);
    return __all_sync(0xFFFFFFFFu, c.abort == 0);
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

// Matrix descriptor of a 128-byte-swizzled operand. `lead`: bytes between
// 64-value groups along the major dimension (only where that dimension is not
// the summed one); groups of 8 rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t matrix(uint32_t addr, uint32_t lead) {
    return (static_cast<uint64_t>(addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: BF16 x BF16 -> FP32, M x N; a_major: A is stored with
// its rows' dimension contiguous.
__host__ __device__ constexpr uint32_t instruction(int m, int n, bool a_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_major ? 1u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// 64 columns of 16 lanes: thread t gets of every group of 8 columns j the
// values of row t / 4 (v[4 j], v[4 j + 1]) and row t / 4 + 8 (v[4 j + 2], v[4 j + 3])
// at columns 8 j + 2 (t % 4) and the next.
__device__ __forceinline__ void tc_load_scores(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
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

// An arrival on `bar` once this thread's copies so far are done.
__device__ __forceinline__ void copies_arrive(u64 *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
// CTA's share is a run of pieces, each part or all of one tile's blocks.
struct Cursor {
    int32_t next_tile, next_block;
    long long left;
    Tile tile;
    int32_t b0, b1, blocks, len, low;   // the piece: blocks [b0, b1) of `blocks`
    __device__ Cursor(const Ctrl &c)
        : next_tile(c.first_tile), next_block(c.first_block),
          left(min(c.begin + c.share, c.total) - c.begin) {}
    __device__ bool next(const AttendParams &p, int lane) {
        if (left <= 0) return false;
        tile = tile_at(p, next_tile);
        len = tile_len_warp(p, tile, lane, low);
        blocks = blocks_of(len);
        b0 = next_block;
        b1 = static_cast<int32_t>(min(static_cast<long long>(blocks), b0 + left));
        left -= b1 - b0;
        ++next_tile;
        next_block = 0;
        return true;
    }
};

// The CTA's share, by all threads of the CTA.
__device__ __forceinline__ void make_schedule(const AttendParams &p, Ctrl &c) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!p.paged) {
        if (tid == 0) {
            const long long n = blocks_of(p.k);
            c.total = n * p.tiles;
            c.share = max(static_cast<long long>(p.min_share), (c.total + gridDim.x - 1) / gridDim.x);
            c.begin = min(c.total, c.share * blockIdx.x);
            c.first_tile = static_cast<int32_t>(c.begin / n);
            c.first_block = static_cast<int32_t>(c.begin % n);
        }
        __syncthreads();
        return;
    }
    const int32_t per = (p.tiles + NT - 1) / NT;
    const int32_t t0 = min(p.tiles, tid * per), t1 = min(p.tiles, t0 + per);
    long long sum = 0;
    for (int32_t t = t0; t < t1; ++t) sum += blocks_of(tile_len(p, tile_at(p, t)));
    long long pre = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, pre, o);
        if (lane >= o) pre += v;
    }
    if (lane == 31) c.sums[warp] = pre;
    __syncthreads();
    long long before = pre - sum, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const long long v = c.sums[w];
        before += w < warp ? v : 0;
        total += v;
    }
    const long long share = max(static_cast<long long>(p.min_share), (total + gridDim.x - 1) / gridDim.x);
    const long long begin = min(total, share * static_cast<long long>(blockIdx.x));
    if (tid == 0) {
        c.total = total;
        c.share = share;
        c.begin = begin;
    }
    if (begin >= before && begin < before + sum) {
        long long at = before;
        for (int32_t t = t0; t < t1; ++t) {
            const int32_t n = blocks_of(tile_len(p, tile_at(p, t)));
            if (begin < at + n) {
                c.first_tile = t;
                c.first_block = static_cast<int32_t>(begin - at);
                break;
            }
            at += n;
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------ the warps' parts

// Cache rows into the stages, swizzled as the products read them. Eight threads
// copy a row's 128-byte chunks, 16 rows at a time; places that hold no cache
// row are filled with zeros and marked. (Measured: the same rows gathered four
// at a time by TMA come at 12 bytes a nanosecond per SM, a third of what these
// copies reach.)
__device__ void load_rows(const AttendParams &p, Ctrl &c, uint32_t stages, int chunks, int stage_count) {
    const int tid = threadIdx.x - SOFT, lane = tid & 31, piece = tid & 7, r = tid >> 3;
    const int64_t pitch = p.cache_stride * 2;
    const char *cache = reinterpret_cast<const char *>(p.cache) + piece * 16;
    Cursor at(c);
    uint32_t st = 0, use = 0;
    bool ok = true;
    while (ok && at.next(p, lane)) {
        const int32_t *list = p.paged ? p.table + static_cast<int64_t>(at.tile.request) * p.table_stride
                                      : p.selected + static_cast<int64_t>(at.tile.token) * p.selected_stride;
        auto row = [&](int32_t i) -> int32_t {
            if (i >= at.len) return -1;
            int64_t v;
            if (p.paged)
                v = static_cast<int64_t>(__ldg(list + (i >> p.page_shift))) * p.block_rows +
                    (i & ((1 << p.page_shift) - 1));
            else
                v = __ldg(list + i);
            return v >= 0 && v < p.cache_rows ? static_cast<int32_t>(v) : -1;
        };
        int32_t now[4], then[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) now[i] = row(at.b0 * KEYS + r + 16 * i);
        for (int32_t b = at.b0; b < at.b1; ++b) {
            if (b + 1 < at.b1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) then[i] = row((b + 1) * KEYS + r + 16 * i);
            }
            if (!(ok = wait(&c.empty[st], use + 1, c))) break;
            const uint32_t stage = stages + st * chunks * CHUNK + r * 128 + ((piece ^ (r & 7)) << 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool on = now[i] >= 0;
                const char *src = cache + (on ? now[i] * pitch : 0);
                for (int k = 0; k < chunks; ++k) copy16(stage + i * 16 * 128 + k * CHUNK, src + k * 128, on);
                if (piece == 0) c.there[st][r + 16 * i] = on ? 1 : 0;
                now[i] = then[i];
            }
            copies_arrive(&c.full[st]);
            __syncwarp();
            if (lane == 0) arrive(&c.full[st]);
            if (++st == static_cast<uint32_t>(stage_count)) {
                st = 0;
                ++use;
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// The products: scores of block i, then the weighted sum of block i - 1, so
// that the tensor cores work while the softmax warps turn scores into weights.
template <int NR>
__device__ void multiply(const AttendParams &p, Ctrl &c, uint32_t query, uint32_t stages, int chunks, int stage_count,
                         uint32_t tmem) {
    const int lane = threadIdx.x & 31;
    constexpr uint32_t QK = instruction(ROWS, KEYS, false), PV = instruction(128, NR, true);
    const int halves = (chunks - 1) / 2;      // 128-value blocks of the latent part
    Cursor at(c);
    uint32_t i = 0, st = 0, use = 0, piece = 0;
    uint32_t prev_st = 0;
    bool prev_first = true, ok = true;
    auto sum = [&]() -> bool {                // the weighted sum of block i - 1, in stage prev_st
        if (!wait(&c.p_full, i - 1, c)) return false;
        tc_fence_after();
        if (lane == 0) {
            const uint32_t base = stages + prev_st * chunks * CHUNK;
            const uint64_t b = matrix(base + (chunks - 1) * CHUNK, 16);
            for (int h = 0; h < halves; ++h) {
                const uint64_t a = matrix(base + 2 * h * CHUNK, CHUNK);
#pragma unroll
                for (int k = 0; k < KEYS / 16; ++k)
                    tc_mma(tmem + O_COL + h * NR, a + k * (16 * 128 >> 4), b + k * 2, PV, !prev_first || k > 0);
            }
            tc_commit(&c.empty[prev_st]);
            tc_commit(&c.o_done);
        }
        __syncwarp();
        return true;
    };
    bool pending = false;
    while (ok && at.next(p, lane)) {
        for (int32_t b = at.b0; b < at.b1; ++b) {
            if (b == at.b0) {
                // A new query tile waits for its loads: finish the last tile's sum first.
                if (pending && !(ok = sum())) break;
                pending = false;
                if (!(ok = wait(&c.q_full, piece, c))) break;
            }
            if (!(ok = wait(&c.full[st], use, c))) break;
            fence_proxy_async();              // (the stage was written by ordinary copies)
            if (!(ok = wait(&c.s_empty[i & 1], (i >> 1) + 1, c))) break;
            tc_fence_after();
            if (lane == 0) {
                const uint64_t a = matrix(query, 16), k0 = matrix(stages + st * chunks * CHUNK, 16);
                for (int k = 0; k < chunks; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        tc_mma(tmem + S_COL + (i & 1) * KEYS, a + k * (CHUNK >> 4) + e * 2, k0 + k * (CHUNK >> 4) + e * 2,
                               QK, k > 0 || e > 0);
                tc_commit(&c.s_full[i & 1]);
                if (b + 1 == at.b1) tc_commit(&c.q_empty);
            }
            __syncwarp();
            if (pending && !(ok = sum())) break;
            pending = true;
            prev_st = st;
            prev_first = b == at.b0;
            ++i;
            if (++st == static_cast<uint32_t>(stage_count)) {
                st = 0;
                ++use;
            }
        }
        ++piece;
    }
    if (ok && pending) ok = sum();
    // Nothing may be running on the tensor cores when their memory is freed.
    if (lane == 0) tc_commit(&c.drain);
    __syncwarp();
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(&c.drain, 0) && global_timer_ns() - t0 < WAIT_LIMIT_NS) {
    }
}

// A tile's query rows into shared memory, swizzled as the products read them.
// Rows past the tile's are left as they are: every row is apart in scores,
// weights and sums, and nothing is written for those.
__device__ void load_query(const AttendParams &p, Ctrl &c, char *query, int chunks) {
    const int tid = threadIdx.x - SOFT - LOAD, lane = threadIdx.x & 31;
    Cursor at(c);
    uint32_t piece = 0;
    while (at.next(p, lane)) {
        if (!wait(&c.q_empty, piece + 1, c)) return;
        const int vecs = chunks * 8, n = at.tile.rows * vecs;
        for (int i0 = tid; i0 < n; i0 += QLOAD * 8) {
            uint4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * QLOAD;
                if (i < n) {
                    const int r = i / vecs, k = i - r * vecs;
                    const int32_t flat = at.tile.base + r, token = flat / p.heads, head = flat - token * p.heads;
                    v[e] = __ldg(reinterpret_cast<const uint4 *>(p.query + token * p.query_token_stride +
                                                                 head * p.query_head_stride) + k);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * QLOAD;
                if (i < n) {
                    const int r = i / vecs, k = i - r * vecs;
                    *reinterpret_cast<uint4 *>(query + (k >> 3) * CHUNK + r * 128 + (((k & 7) ^ (r & 7)) << 4)) = v[e];
                }
            }
        }
        fence_proxy_async();
        arrive(&c.q_full);
        ++piece;
    }
}

struct Part {                                  // a piece's unfinished rows in the workspace
    float sum[ROWS * LATENT_MAX];
    float m[ROWS], l[ROWS];
};

struct Joint {                                 // a split tile: where its parts are
    int32_t tile, parts, cta, unused;
};

__device__ __forceinline__ float finished_lse(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2; }
__device__ __forceinline__ float reciprocal(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }   // NaN stays NaN

// Scores to weights, the running maximum and sum, and the outputs. Thread t of
// warp w holds rows 16 w + t / 4 and 8 further, a quarter of each one's columns.
template <int NR>
__device__ void soften(const AttendParams &p, Ctrl &c, char *stages, int chunks, int stage_count, uint32_t tmem) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const bool active = w * 16 < NR;
    const int row0 = w * 16 + lane / 4, quad = lane & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
    const float scale = p.scale * LOG2E;
    Part *parts = reinterpret_cast<Part *>(p.workspace);
    Joint *joints = reinterpret_cast<Joint *>(parts + 2 * p.sms);
    const bool by_tile = p.tiles <= static_cast<int32_t>(gridDim.x);
    bool split_here = false;
    Cursor at(c);
    uint32_t i = 0, st = 0, use = 0;
    long long done = c.begin;
    while (at.next(p, lane)) {
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        int32_t lim[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (row0 + 8 * h < at.tile.rows)
                lim[h] = p.paged ? token_len(p, (at.tile.base + row0 + 8 * h) / p.heads) : INT32_MAX;
        for (int32_t b = at.b0; b < at.b1; ++b) {
            char *stage = stages + st * chunks * CHUNK;
            // (These warps meet at barriers, so none leaves early: after a wait that gave
            // up, all go on without waiting, on whatever the memories hold.)
            mbar_wait(&c.s_full[i & 1], (i >> 1) & 1u, &c.abort);
            mbar_wait(&c.full[st], use & 1u, &c.abort);   // (complete: makes the mask visible)
            __syncwarp();
            const u64 mask = static_cast<u64>(__ballot_sync(0xFFFFFFFFu, c.there[st][lane] != 0)) |
                             static_cast<u64>(__ballot_sync(0xFFFFFFFFu, c.there[st][lane + 32] != 0)) << 32;
            float x[32];
            if (active) {
                tc_fence_after();
                tc_load_scores(lanes + S_COL + (i & 1) * KEYS, x);
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) arrive(&c.s_empty[i & 1]);
            bool grow[2] = {false, false};
            float old[2] = {m[0], m[1]};
            if (active) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] *= scale;
            }
            const bool whole = mask == ~0ull && at.low >= (b + 1) * KEYS && at.tile.rows == NR;
            if (!whole) {
                // Keep an entry if its place holds a cache row that this row may see. A
                // cache row that only some of the tile's rows see must not reach the others
                // through 0 x inf: where a score that is masked here is not finite (every
                // row sees its NaN and infinities in its score), the cache row is zeroed and
                // the weights of the rows that do see it are NaN.
                const u64 mine = mask >> (2 * quad);
                u64 bad = 0;
                uint32_t keep = 0;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const int h = (e >> 1) & 1, col = (e >> 2) * 8 + (e & 1);
                    const bool there = (mine >> col) & 1;
                    const bool seen = there && b * KEYS + col + 2 * quad < lim[h];
                    keep |= seen ? 1u << e : 0u;
                    if (active && there && !seen && lim[h] >= 0 && row0 + 8 * h < at.tile.rows &&
                        !(fabsf(x[e]) < INFINITY))
                        bad |= 1ull << (col + 2 * quad);
                }
                if (p.paged && soft_any(bad != 0)) {
                    if (bad) atomicOr(&c.bad, bad);
                    soft_sync();
                    const u64 all = c.bad;
                    const u64 here = all >> (2 * quad);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if ((here >> ((e >> 2) * 8 + (e & 1))) & 1) x[e] = __uint_as_float(0x7FC00000u);
                    for (int v = tid; v < KEYS * (chunks - 1) * 8; v += SOFT) {
                        const int r = v / ((chunks - 1) * 8), k = v - r * (chunks - 1) * 8;
                        if ((all >> r) & 1)
                            *reinterpret_cast<uint4 *>(stage + (k >> 3) * CHUNK + r * 128 + (k & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    soft_sync();
                    if (tid == 0) c.bad = 0;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (!((keep >> e) & 1)) x[e] = -INFINITY;
            }
            if (active) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (((e >> 1) & 1) == h) mx = fmaxf(mx, x[e]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                    grow[h] = mx > m[h] + LAZY || (m[h] == -INFINITY && mx > m[h]);
                    if (grow[h]) m[h] = mx;
                }
            }
            // The reference maximum only moves when it lags by more than 2^8 (the weights
            // then stay below 2^8 and lose nothing): the sums so far are rescaled then.
            if (b > at.b0 && soft_any(grow[0] || grow[1])) {
                if (active) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float f = !grow[h] ? 1.0f : old[h] == -INFINITY ? 0.0f : exp2_fast(old[h] - m[h]);
                        l[h] *= f;
                        if (quad == 0) c.factor[row0 + 8 * h] = f;
                    }
                }
                soft_sync();
                mbar_wait(&c.o_done, (i - 1) & 1u, &c.abort);
                __syncwarp();
                tc_fence_after();
                for (int v = 0; v < (chunks - 1) / 2 * NR; v += 16) {
                    float o[16];
                    tc_load16(lanes + O_COL + v, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= c.factor[(v + e) % NR];
                    tc_store16(lanes + O_COL + v, o);
                }
                tc_wait_st();
                tc_fence_before();
            }
            if (active) {
                // Weights, rounded once to BF16 for the tensor cores; their sum is of the
                // unrounded ones, in 32 bits, a block's 16 per thread first.
                char *weights = stage + (chunks - 1) * CHUNK;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float ref = m[h] == -INFINITY ? 0.0f : m[h];
                    float s = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float a = exp2_fast(x[4 * j + 2 * h] - ref), d = exp2_fast(x[4 * j + 2 * h + 1] - ref);
                        s += a + d;
                        const __nv_bfloat162 v = __floats2bfloat162_rn(a, d);
                        const int r = row0 + 8 * h;
                        *reinterpret_cast<__nv_bfloat162 *>(weights + r * 128 + ((j ^ (r & 7)) << 4) + quad * 4) = v;
                    }
                    l[h] += s;
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(&c.p_full);
            ++i;
            if (++st == static_cast<uint32_t>(stage_count)) {
                st = 0;
                ++use;
            }
        }
        // The piece is done: write its rows, or its part of them.
        if (active) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
                l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
                if (quad == 0) {
                    c.m[row0 + 8 * h] = m[h];
                    c.l[row0 + 8 * h] = l[h];
                }
            }
        }
        soft_sync();
        // (One phase at a time: block i - 1's scores say that block i - 3's sum is done.)
        if (i > 1) mbar_wait(&c.o_done, i & 1u, &c.abort);
        mbar_wait(&c.o_done, (i - 1) & 1u, &c.abort);
        __syncwarp();
        tc_fence_after();
        const bool direct = at.b0 == 0 && at.b1 == at.blocks;
        if (direct) {
            if (p.lse && tid < at.tile.rows) p.lse[at.tile.base + tid] = finished_lse(c.m[tid], c.l[tid]);
            uint16_t *out = p.out + static_cast<int64_t>(at.tile.base) * p.latent;
            for (int v = 0; v < (chunks - 1) / 2 * NR; v += 16) {
                float o[16];
                tc_load16(lanes + O_COL + v, o);
                const int d = v / NR * 128 + w * 32 + lane;
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    // Even lanes take the pair's values of one row, odd lanes of the next.
                    const int r = v % NR + e;
                    const float a = o[e] * reciprocal(c.l[r]), a1 = o[e + 1] * reciprocal(c.l[r + 1]);
                    const float other = __shfl_xor_sync(0xFFFFFFFFu, lane & 1 ? a : a1, 1);
                    const int mine = r + (lane & 1);
                    const __nv_bfloat162 pair = lane & 1 ? __floats2bfloat162_rn(other, a1)
                                                         : __floats2bfloat162_rn(a, other);
                    if (mine < at.tile.rows)
                        *reinterpret_cast<__nv_bfloat162 *>(out + static_cast<int64_t>(mine) * p.latent + (d & ~1)) =
                            pair;
                }
            }
        } else {
            Part &part = parts[2 * blockIdx.x + (at.b0 == 0 ? 1 : 0)];
            if (tid < NR) {
                part.m[tid] = c.m[tid];
                part.l[tid] = c.l[tid];
            }
            for (int v = 0; v < (chunks - 1) / 2 * NR; v += 16) {
                float o[16];
                tc_load16(lanes + O_COL + v, o);
                const int d = v / NR * 128 + w * 32 + lane;
#pragma unroll
                for (int e = 0; e < 16; ++e) part.sum[(v % NR + e) * p.latent + d] = o[e];
            }
        }
        if (at.b0 == 0 && tid == 0 && (by_tile || !direct)) {
            Joint j;
            j.tile = at.next_tile - 1;
            j.cta = static_cast<int32_t>(blockIdx.x);
            j.parts = static_cast<int32_t>((done + at.blocks - 1) / c.share) - j.cta + 1;
            j.unused = 0;
            joints[by_tile ? j.tile : j.cta] = j;
        }
        split_here |= at.b0 == 0 && !direct;
        done += at.b1 - at.b0;
        tc_fence_before();
        soft_sync();
    }
    if (!by_tile && !split_here && tid == 0) joints[blockIdx.x] = Joint{0, 0, 0, 0};
}

template <int NR>
__global__ void __launch_bounds__(NT, 1) attend_kernel(const __grid_constant__ AttendParams p) {
    extern __shared__ char raw[];
    char *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Ctrl &c = *reinterpret_cast<Ctrl *>(smem + CHUNKS * CHUNK);
    const int warp = threadIdx.x >> 5;
    const int chunks = p.latent / 64 + 1;
    const int stage_count = min(MAX_STAGES, (CHUNKS - chunks) / chunks);
    if (threadIdx.x == 0) {
        for (int s = 0; s < MAX_STAGES; ++s) {
            mbar_init(&c.full[s], LOAD + LOAD / 32);
            mbar_init(&c.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&c.s_full[s], 1);
            mbar_init(&c.s_empty[s], SOFT / 32);
        }
        mbar_init(&c.p_full, SOFT / 32);
        mbar_init(&c.o_done, 1);
        mbar_init(&c.q_full, QLOAD);
        mbar_init(&c.q_empty, 1);
        mbar_init(&c.drain, 1);
        c.bad = 0;
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
    char *stages = smem + chunks * CHUNK;
    if (warp < SOFT / 32) soften<NR>(p, c, stages, chunks, stage_count, tmem);
    else if (warp < (SOFT + LOAD) / 32) load_rows(p, c, smem_addr(stages), chunks, stage_count);
    else if (warp < (SOFT + LOAD + QLOAD) / 32) load_query(p, c, smem, chunks);
    else multiply<NR>(p, c, smem_addr(smem), smem_addr(stages), chunks, stage_count, tmem);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == NT / 32 - 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// Joins a split tile's parts, one CTA per row: each part's sum weighs
// 2^(its maximum - the largest). Parts are added in order: results do not
// depend on which CTA finished first.
__global__ void __launch_bounds__(NT_JOIN) join_kernel(const __grid_constant__ AttendParams p) {
    __shared__ float weight[512], red[NT_JOIN / 32];
    __shared__ __align__(16) float partial[NT_JOIN * 4];
    grid_dependents_release();
    grid_dependency_wait();
    const Part *parts = reinterpret_cast<const Part *>(p.workspace);
    const Joint j = reinterpret_cast<const Joint *>(parts + 2 * p.sms)[blockIdx.x];
    if (j.parts < 2) return;
    const Tile t = tile_at(p, j.tile);
    const int row = blockIdx.y, tid = threadIdx.x;
    if (row >= t.rows) return;
    auto part = [&](int i) -> const Part & { return parts[2 * (j.cta + i) + (i == 0 ? 1 : 0)]; };
    float mine = -INFINITY;
    for (int i = tid; i < j.parts; i += NT_JOIN) mine = fmaxf(mine, part(i).m[row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mine = fmaxf(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, o));
    if ((tid & 31) == 0) red[tid >> 5] = mine;
    __syncthreads();
    float top = red[0];
#pragma unroll
    for (int i = 1; i < NT_JOIN / 32; ++i) top = fmaxf(top, red[i]);
    __syncthreads();
    float sum = 0.0f;
    for (int i = tid; i < j.parts; i += NT_JOIN) {
        const float m = part(i).m[row];
        const float f = m == -INFINITY ? 0.0f : exp2_fast(m - top);
        weight[i] = f;
        sum += f * part(i).l[row];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    float l = 0.0f;
#pragma unroll
    for (int i = 0; i < NT_JOIN / 32; ++i) l += red[i];
    const int vecs = p.latent / 4, groups = NT_JOIN / vecs, g = tid / vecs, v = tid - g * vecs;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (g < groups) {
#pragma unroll 8
        for (int i = g; i < j.parts; i += groups) {
            const float4 x = reinterpret_cast<const float4 *>(part(i).sum + row * p.latent)[v];
            const float f = weight[i];
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
        }
        reinterpret_cast<float4 *>(partial)[tid] = acc;
    }
    __syncthreads();
    if (g == 0) {
        for (int k = 1; k < groups; ++k) {
            const float4 x = reinterpret_cast<const float4 *>(partial)[k * vecs + v];
            acc.x += x.x;
            acc.y += x.y;
            acc.z += x.z;
            acc.w += x.w;
        }
        const float inv = reciprocal(l);
        const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        uint2 o;
        o.x = *reinterpret_cast<const uint32_t *>(&a);
        o.y = *reinterpret_cast<const uint32_t *>(&b);
        reinterpret_cast<uint2 *>(p.out + (static_cast<int64_t>(t.base) + row) * p.latent)[v] = o;
        if (v == 0 && p.lse) p.lse[t.base + row] = finished_lse(top, l);
    }
}

}  // namespace

// ------------------------------------------------------------------ host side

namespace {

struct Device {
    std::once_flag once;
    cudaError_t err = cudaSuccess;
    int sms = 0;
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
            if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
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

cudaError_t launch_attend(AttendParams p, cudaStream_t stream) {
    Device *d = nullptr;
    cudaError_t e = device(d);
    if (e != cudaSuccess) return e;
    const int64_t per = static_cast<int64_t>(p.rows_per_request) * p.heads;
    const int64_t full = p.tokens / p.rows_per_request, rest = p.tokens % p.rows_per_request * static_cast<int64_t>(p.heads);
    p.tiles_per_request = static_cast<int32_t>((per + ROWS - 1) / ROWS);
    p.tiles = static_cast<int32_t>(full * p.tiles_per_request + (rest + ROWS - 1) / ROWS);
    p.min_share = 2;
    p.sms = d->sms;
    const int64_t most_blocks = (static_cast<int64_t>(p.paged ? p.width : p.k) + KEYS - 1) / KEYS;
    const int64_t want = (p.tiles * (most_blocks > 1 ? most_blocks : 1) + p.min_share - 1) / p.min_share;
    const unsigned grid = static_cast<unsigned>(want < d->sms ? want : d->sms);
    const int64_t rows = full > 0 ? per : rest;
    const int nr = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&p};
    e = cudaLaunchKernelExC(&cfg, nr == 16 ? attend_fn<16>() : nr == 32 ? attend_fn<32>() : attend_fn<64>(), args);
    if (e != cudaSuccess || most_blocks <= 1) return e;   // tiles of one block are never split
    cfg.blockDim = dim3(NT_JOIN, 1, 1);
    cfg.gridDim = dim3(static_cast<unsigned>(p.tiles < static_cast<int32_t>(grid) ? p.tiles : grid),
                       static_cast<unsigned>(nr), 1);
    cfg.dynamicSmemBytes = 0;
    void *join_args[] = {&p};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(&join_kernel), join_args);
}

}  // namespace topk::latent
