// pages.cu -- the page pool of a paged KV cache: forking, reserving (with
// copies of shared pages), freeing and compacting, all on the device.
//
// The state is four integer arrays of the caller's (spark_page_pool): the page
// table, the pages and tokens of each row, and how many rows hold each page.
// A page is free when no row holds it, so there is no free list to keep in
// step: a call that takes pages scans the counts, and what it takes depends on
// the state alone, never on timing.
//
//   plan kernels   one CTA each: scans over rows and pages (integers, a few
//                  microseconds), the list of page copies left in the workspace
//   page_copy_kernel  the copies, in every layer, K and V; bound by HBM
#include "common.cuh"
#include "spark_attn.h"

namespace spark {

namespace {

constexpr int kPlanThreads = 1024;
static_assert(kPlanThreads == 32 * 32, "block_scan sums 32 warps with one warp");
constexpr int kRowThreads = 128;
constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 8;                                 // 16-byte words in flight per thread
constexpr int kCopyChunk = kCopyThreads * kCopyVec * 16;    // 32 KB

struct PoolParams {
    uint8_t *k_pages, *v_pages;
    int32_t *table, *held, *len, *refs;
    int32_t n_layers, n_pages, page_size, n_rows, max_pages;
    long long page_bytes;       // of one page of one layer, K or V
    unsigned *status;
    // workspace
    int32_t *n_copies;          // copies listed
    int32_t *n_live;            // pages in use (compact)
    int32_t *copy_src, *copy_dst;   // [n_pages]
    int32_t *map;               // [n_pages]: where a page goes (compact)
    int32_t *row_a, *row_b, *row_c;   // [n_rows]
};

// ---------------------------------------------------------------- block scan

// Exclusive prefix sum of one value per thread over the block, and the total.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *total, T *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();  // the sums of the scan before are read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    T s = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    const T before = warp ? __shfl_sync(0xffffffffu, s, warp - 1) : T(0);
    return before + x - v;
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
    return static_cast<int>((static_cast<long long>(tokens) + page_size - 1) / page_size);
}

// Whether a row's counts fit the table (a pool that was not set up, or written
// over, must not lead outside it).
__device__ __forceinline__ bool row_sane(const PoolParams &P, int held, int len) {
    return held >= 0 && held <= P.max_pages && len >= 0 && pages_of(len, P.page_size) <= held;
}

// ---------------------------------------------------------------- fork

// Decides every pair before any row changes.  row_a[r]: the first pair that
// forks into row r; row_b[r]: its pages (-1: refused); row_c[r]: its tokens.
__device__ __forceinline__ void fork_plan(const PoolParams &P, const int32_t *src,
                                          const int32_t *dst, int n) {
    for (int r = threadIdx.x; r < P.n_rows; r += kPlanThreads) P.row_a[r] = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int d = dst[i];
        if (d >= 0 && d < P.n_rows) atomicMin(&P.row_a[d], i);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int s = src[i], d = dst[i];
        const bool row = d >= 0 && d < P.n_rows;
        const bool first = row && P.row_a[d] == i;
        int pages = -1;
        if (first && s >= 0 && s < P.n_rows && P.held[d] == 0) {
            const int held = P.held[s], len = P.len[s];
            if (row_sane(P, held, len)) {
                pages = pages_of(len, P.page_size);
                P.row_c[d] = len;
            }
        }
        if (pages < 0) atomicOr(P.status, kErrRow);
        if (first) P.row_b[d] = pages;
    }
}

// The table row and the counts of pair i, by the threads t, t + step, ...
__device__ __forceinline__ void fork_apply(const PoolParams &P, const int32_t *src,
                                           const int32_t *dst, int i, int t, int step) {
    const int d = dst[i];
    if (d < 0 || d >= P.n_rows || P.row_a[d] != i) return;
    const int count = P.row_b[d];
    if (count < 0) return;
    const int32_t *from = P.table + static_cast<size_t>(src[i]) * P.max_pages;
    int32_t *to = P.table + static_cast<size_t>(d) * P.max_pages;
    for (int j = t; j < P.max_pages; j += step) {
        int p = -1;
        if (j < count) {
            p = from[j];
            if (p < 0 || p >= P.n_pages)
                atomicOr(P.status, kErrPage);
            else
                atomicAdd(&P.refs[p], 1);
        }
        to[j] = p;
    }
    if (t == 0) {
        P.held[d] = count;
        P.len[d] = P.row_c[d];
    }
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(
    const __grid_constant__ PoolParams P, const int32_t *src, const int32_t *dst, int n) {
    grid_dep_wait();
    grid_dep_launch();
    fork_plan(P, src, dst, n);
}

__global__ void __launch_bounds__(kRowThreads) fork_apply_kernel(
    const __grid_constant__ PoolParams P, const int32_t *src, const int32_t *dst, int n) {
    grid_dep_wait();
    grid_dep_launch();
    fork_apply(P, src, dst, blockIdx.x, threadIdx.x, kRowThreads);
}

// Both in one CTA, a warp per pair, where there are few table entries to write:
// one launch less, against a CTA per pair for many (fork and free, in one CTA
// and in two launches: 16 x 64 entries 9.9 and 11.0 us, 64 x 256 9.9 and 10.7,
// 128 x 256 13.6 and 10.6, 256 x 256 23 and 10.6).
constexpr long long kForkSmall = 16384;

__global__ void __launch_bounds__(kPlanThreads) fork_kernel(const __grid_constant__ PoolParams P,
                                                            const int32_t *src, const int32_t *dst,
                                                            int n) {
    grid_dep_wait();
    grid_dep_launch();
    fork_plan(P, src, dst, n);
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < n; i += kPlanThreads / 32)
        fork_apply(P, src, dst, i, threadIdx.x & 31, 32);
}

// ---------------------------------------------------------------- free

__global__ void __launch_bounds__(kRowThreads) free_kernel(const __grid_constant__ PoolParams P,
                                                           const int32_t *rows,
                                                           const int32_t *keep, int n) {
    grid_dep_wait();
    grid_dep_launch();
    const int i = blockIdx.x;
    const int r = rows[i];
    if (r < 0 || r >= P.n_rows) {
        if (threadIdx.x == 0) atomicOr(P.status, kErrRow);
        return;
    }
    bool first = true;
    for (int j = threadIdx.x; j < i; j += kRowThreads) first = first && rows[j] != r;
    if (!__syncthreads_and(first)) return;
    const int held = P.held[r], len = P.len[r];
    if (!row_sane(P, held, len)) {
        if (threadIdx.x == 0) atomicOr(P.status, kErrRow);
        return;
    }
    int tokens = keep ? keep[i] : 0;
    tokens = tokens < 0 ? 0 : (tokens < len ? tokens : len);
    const int stay = pages_of(tokens, P.page_size);
    int32_t *row = P.table + static_cast<size_t>(r) * P.max_pages;
    for (int j = stay + threadIdx.x; j < held; j += kRowThreads) {
        const int p = row[j];
        if (p < 0 || p >= P.n_pages)
            atomicOr(P.status, kErrPage);
        else
            atomicSub(&P.refs[p], 1);
        row[j] = -1;
    }
    __syncthreads();  // every thread has read held and len
    if (threadIdx.x == 0) {
        P.held[r] = stay;
        P.len[r] = tokens;
    }
}

// ---------------------------------------------------------------- reserve

constexpr int kScanPages = 4 * kPlanThreads;  // pages a scan step looks at, four per thread

// Which of the four pages 4 tid .. 4 tid + 3 behind p0 are free, as bits.
__device__ __forceinline__ unsigned free_bits(const PoolParams &P, int p0) {
    unsigned bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = p0 + 4 * static_cast<int>(threadIdx.x) + i;
        if (p < P.n_pages && P.refs[p] == 0) bits |= 1u << i;
    }
    return bits;
}

// What row r asks for: the page it is about to write into although it holds
// tokens already (-1: none), and the fresh pages behind the ones it holds.
__device__ __forceinline__ void row_wish(const PoolParams &P, const int32_t *add, int r, int &page,
                                         int &fresh) {
    page = -1;
    fresh = 0;
    const int more = add[r], held = P.held[r], len = P.len[r];
    if (more <= 0) return;
    const long long end = static_cast<long long>(len) + more;
    if (!row_sane(P, held, len) || end > static_cast<long long>(P.max_pages) * P.page_size) {
        atomicOr(P.status, kErrRow);
        return;
    }
    if (len % P.page_size) {
        page = P.table[static_cast<size_t>(r) * P.max_pages + len / P.page_size];
        if (page < 0 || page >= P.n_pages) {
            atomicOr(P.status, kErrPage);
            page = -1;
            return;
        }
    }
    const int need = static_cast<int>((end + P.page_size - 1) / P.page_size);
    fresh = need > held ? need - held : 0;
    if (fresh > P.n_pages) fresh = P.n_pages + 1;  // too many, whatever the sum
}

// One CTA, a row per thread at a time.  Rows of the first kPlanThreads keep
// their wishes in registers; the arrays in the workspace serve pools with more
// (a trip through L2 costs half a microsecond, and there are several).
__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(
    const __grid_constant__ PoolParams P, const int32_t *add, int32_t *taken) {
    __shared__ int warp_sums[32];
    __shared__ long long wide_sums[32];
    __shared__ int s_page[kPlanThreads];  // row_wish's pages of this chunk of rows
    __shared__ int s_map[kPlanThreads];   // the first pages taken
    constexpr int kCopyBit = 1 << 30;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    const bool one = P.n_rows <= kPlanThreads;
    const unsigned first_free = free_bits(P, 0);  // (its latency overlaps the rows')
    int my_want = 0, my_at = 0;                   // of the chunk's row
    long long base = 0;
    int copies = 0;
    for (int r0 = 0; r0 < P.n_rows; r0 += kPlanThreads) {
        const int r = r0 + tid;
        int page = -1, fresh = 0, refs = 0;
        if (r < P.n_rows) row_wish(P, add, r, page, fresh);
        if (page >= 0) refs = P.refs[page];
        s_page[tid] = page;
        if (!one && r < P.n_rows) P.row_a[r] = page;
        __syncthreads();
        // a copy for all rows that are about to write into the page but the
        // last holder
        int copy = 0;
        if (refs > 1) {
            int before = 0;
            for (int q = 0; q < r0; ++q) before += P.row_a[q] == page;
            for (int q = 0; q < tid; ++q) before += s_page[q] == page;
            copy = refs - before > 1;
        }
        long long total;
        int ctotal;
        const long long at = base + block_scan<long long>(fresh + copy, &total, wide_sums);
        const int cat = copies + block_scan(copy, &ctotal, warp_sums);
        // past n_pages the call will be refused: nothing of it is used
        my_want = fresh | (copy ? kCopyBit : 0);
        my_at = static_cast<int>(at < P.n_pages ? at : P.n_pages);
        if (copy && cat < P.n_pages) {
            P.copy_src[cat] = page;
            P.copy_dst[cat] = my_at;  // its rank among the free pages, for now
        }
        if (!one && r < P.n_rows) {
            P.row_b[r] = my_want;
            P.row_c[r] = my_at;
        }
        base += total;
        copies += ctotal;
    }
    const int want = static_cast<int>(base <= P.n_pages ? base : P.n_pages + 1);
    // the first `want` free pages
    int32_t *map = want <= kPlanThreads ? s_map : P.map;
    int found = 0;
    for (int p0 = 0; p0 < P.n_pages && found < want; p0 += kScanPages) {
        const unsigned bits = p0 == 0 ? first_free : free_bits(P, p0);
        int total;
        int at = found + block_scan(__popc(bits), &total, warp_sums);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (bits >> i & 1u) {
                if (at < want) map[at] = p0 + 4 * tid + i;
                ++at;
            }
        found += total;
    }
    __syncthreads();
    const bool ok = found >= want;
    if (tid == 0) {
        *P.n_copies = ok ? copies : 0;
        if (taken) *taken = ok ? want : -1;
    }
    if (!ok) return;
    for (int i = tid; i < want; i += kPlanThreads) P.refs[map[i]] = 1;
    for (int i = tid; i < copies; i += kPlanThreads) {
        P.copy_dst[i] = map[P.copy_dst[i]];
        atomicSub(&P.refs[P.copy_src[i]], 1);
    }
    for (int r = tid; r < P.n_rows; r += kPlanThreads) {
        const int w = one ? my_want : P.row_b[r];
        if (!w) continue;
        int at = one ? my_at : P.row_c[r];
        int32_t *row = P.table + static_cast<size_t>(r) * P.max_pages;
        if (w & kCopyBit) row[P.len[r] / P.page_size] = map[at++];
        const int fresh = w & ~kCopyBit, held = P.held[r];
        for (int j = 0; j < fresh; ++j) row[held + j] = map[at + j];
        if (fresh) P.held[r] = held + fresh;
    }
}

// ---------------------------------------------------------------- compact

// With U(p) the pages in use below p, of n_live in all: a free page p < n_live
// is hole number p - U(p), a used page p >= n_live mover number U(p) - U(n_live),
// and there are as many of one as of the other.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(
    const __grid_constant__ PoolParams P, int32_t *live) {
    __shared__ int warp_sums[32];
    __shared__ int s_below;  // U(n_live)
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    auto used_bits = [&](int p0) {
        unsigned bits = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 4 * tid + i;
            if (p < P.n_pages && P.refs[p] > 0) bits |= 1u << i;
        }
        return bits;
    };
    const unsigned first = used_bits(0);
    int n = 0;
    for (int p0 = 0; p0 < P.n_pages; p0 += kScanPages)
        n += __popc(p0 == 0 ? first : used_bits(p0));
    int n_live;
    block_scan(n, &n_live, warp_sums);
    if (tid == 0 && n_live >= P.n_pages) s_below = n_live;
    int before = 0;
    for (int p0 = 0; p0 < P.n_pages; p0 += kScanPages) {
        const unsigned bits = p0 == 0 ? first : used_bits(p0);
        int total;
        int u = before + block_scan(__popc(bits), &total, warp_sums);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 4 * tid + i;
            if (p >= P.n_pages) break;
            const bool used = bits >> i & 1u;
            if (p == n_live) s_below = u;
            if (p < n_live) {
                if (!used) P.copy_dst[p - u] = p;
            } else {
                P.map[p] = used ? u : p;  // U(p) of a mover, for now
            }
            u += used;
        }
        before += total;
    }
    __syncthreads();
    const int below = s_below, movers = n_live - below;
    for (int p = n_live + tid; p < P.n_pages; p += kPlanThreads) {
        const int refs = P.refs[p];
        if (refs <= 0) continue;
        const int i = P.map[p] - below, to = P.copy_dst[i];
        P.copy_src[i] = p;
        P.map[p] = to;
        P.refs[to] = refs;
        P.refs[p] = 0;
    }
    if (tid == 0) {
        *P.n_copies = movers;
        *P.n_live = n_live;
        if (live) *live = n_live;
    }
}

// The tables follow their pages: rows r, r + step, ..., one CTA each.
__device__ __forceinline__ void compact_tables(const PoolParams &P) {
    const int n_live = *P.n_live;
    for (int r = blockIdx.x; r < P.n_rows; r += gridDim.x) {
        const int held = P.held[r];
        if (held < 0 || held > P.max_pages) {
            if (threadIdx.x == 0) atomicOr(P.status, kErrRow);
            continue;
        }
        int32_t *row = P.table + static_cast<size_t>(r) * P.max_pages;
        for (int j = threadIdx.x; j < held; j += blockDim.x) {
            const int p = row[j];
            if (p < 0 || p >= P.n_pages)
                atomicOr(P.status, kErrPage);
            else if (p >= n_live)
                row[j] = P.map[p];
        }
    }
}

// ---------------------------------------------------------------- copies

// The listed page copies in every layer, K and V, in chunks of 32 KB (or the
// page, where it is smaller).  No page is the source of one copy and the
// target of another, so their order does not matter.
template <bool kTables>
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(
    const __grid_constant__ PoolParams P) {
    grid_dep_wait();
    grid_dep_launch();
    if (kTables) compact_tables(P);
    const long long per_page = (P.page_bytes + kCopyChunk - 1) / kCopyChunk;
    const long long total = per_page * 2 * P.n_layers * *P.n_copies;
    for (long long c = blockIdx.x; c < total; c += gridDim.x) {
        const long long at = (c % per_page) * kCopyChunk;
        long long u = c / per_page;
        uint8_t *pool = (u & 1) ? P.v_pages : P.k_pages;
        u >>= 1;
        const int i = static_cast<int>(u / P.n_layers);
        const long long layer = (u % P.n_layers) * P.n_pages;
        const uint8_t *src = pool + (layer + P.copy_src[i]) * P.page_bytes + at;
        uint8_t *dst = pool + (layer + P.copy_dst[i]) * P.page_bytes + at;
        const long long left = P.page_bytes - at;
        uint4 w[kCopyVec];
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j) {
            const int off = (j * kCopyThreads + static_cast<int>(threadIdx.x)) * 16;
            if (off < left) w[j] = __ldcs(reinterpret_cast<const uint4 *>(src + off));
        }
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j) {
            const int off = (j * kCopyThreads + static_cast<int>(threadIdx.x)) * 16;
            if (off < left) *reinterpret_cast<uint4 *>(dst + off) = w[j];
        }
    }
}

// ---------------------------------------------------------------- host side

struct PoolPlan {
    size_t counts, copy_src, copy_dst, map, rows, bytes;
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

PoolPlan plan_pool(const spark_page_pool *pool) {
    PoolPlan pl{};
    const size_t pages = up256(static_cast<size_t>(pool->n_pages) * 4);
    const size_t rows = up256(static_cast<size_t>(pool->n_rows > 0 ? pool->n_rows : 1) * 4);
    pl.counts = kWorkspaceHeader;
    pl.copy_src = pl.counts + 256;
    pl.copy_dst = pl.copy_src + pages;
    pl.map = pl.copy_dst + pages;
    pl.rows = pl.map + pages;
    pl.bytes = pl.rows + 3 * rows;
    return pl;
}

spark_status check_pool_sizes(const spark_page_pool *pool) {
    if (!pool) return SPARK_ERR_NULL;
    if (pool->n_layers < 1 || pool->Hkv < 1 || pool->n_pages < 0 || pool->n_rows < 0 ||
        pool->max_pages < 0)
        return SPARK_ERR_SHAPE;
    const int ps = pool->page_size;
    if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return SPARK_ERR_UNSUPPORTED;
    // tokens of a row stay below 2^30, the pages a row wants below bit 30
    if (pool->n_pages >= (1 << 29) || pool->max_pages >= (1 << 30) / ps)
        return SPARK_ERR_UNSUPPORTED;
    return SPARK_OK;
}

spark_status check_pool(const spark_page_pool *pool, const void *workspace,
                        size_t workspace_bytes) {
    spark_status st = check_pool_sizes(pool);
    if (st != SPARK_OK) return st;
    auto bad = [](const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; };
    if ((pool->n_pages > 0 && (!pool->k_pages || !pool->v_pages || !pool->refs)) ||
        (pool->n_rows > 0 && (!pool->held || !pool->len)) ||
        (pool->n_rows > 0 && pool->max_pages > 0 && !pool->table) || !workspace)
        return SPARK_ERR_NULL;
    if (bad(pool->k_pages, 16) || bad(pool->v_pages, 16) || bad(pool->refs, 4) ||
        bad(pool->held, 4) || bad(pool->len, 4) || bad(pool->table, 4) || bad(workspace, 256))
        return SPARK_ERR_ALIGN;
    if (workspace_bytes < plan_pool(pool).bytes) return SPARK_ERR_WORKSPACE;
    return SPARK_OK;
}

// token_bytes: of a token's key, or value, of one KV head.
PoolParams pool_params(const spark_page_pool *pool, void *workspace,
                       int token_bytes = kHeadDim * 2) {
    const PoolPlan pl = plan_pool(pool);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t rows = up256(static_cast<size_t>(pool->n_rows > 0 ? pool->n_rows : 1) * 4);
    PoolParams P{};
    P.k_pages = static_cast<uint8_t *>(pool->k_pages);
    P.v_pages = static_cast<uint8_t *>(pool->v_pages);
    P.table = pool->table;
    P.held = pool->held;
    P.len = pool->len;
    P.refs = pool->refs;
    P.n_layers = pool->n_layers;
    P.n_pages = pool->n_pages;
    P.page_size = pool->page_size;
    P.n_rows = pool->n_rows;
    P.max_pages = pool->max_pages;
    P.page_bytes = static_cast<long long>(pool->Hkv) * pool->page_size * token_bytes;
    P.status = reinterpret_cast<unsigned *>(ws);
    P.n_copies = reinterpret_cast<int32_t *>(ws + pl.counts);
    P.n_live = P.n_copies + 1;
    P.copy_src = reinterpret_cast<int32_t *>(ws + pl.copy_src);
    P.copy_dst = reinterpret_cast<int32_t *>(ws + pl.copy_dst);
    P.map = reinterpret_cast<int32_t *>(ws + pl.map);
    P.row_a = reinterpret_cast<int32_t *>(ws + pl.rows);
    P.row_b = reinterpret_cast<int32_t *>(ws + pl.rows + rows);
    P.row_c = reinterpret_cast<int32_t *>(ws + pl.rows + 2 * rows);
    return P;
}

spark_status done(cudaError_t e) {
    if (e == cudaSuccess) return SPARK_OK;
    cudaGetLastError();
    return SPARK_ERR_CUDA;
}

// The copies listed, `most` at most; with kTables the rows' tables too.
template <bool kTables>
cudaError_t launch_copies(const PoolParams &P, long long most, int sms, cudaStream_t stream) {
    const long long per_page = (P.page_bytes + kCopyChunk - 1) / kCopyChunk;
    long long work = per_page * 2 * P.n_layers * most;
    if (kTables && work < P.n_rows) work = P.n_rows;
    const long long grid = work < sms * 4ll ? work : sms * 4ll;
    return launch_overlapped(page_copy_kernel<kTables>, dim3(static_cast<unsigned>(grid)),
                             dim3(kCopyThreads), 0, stream, P);
}

}  // namespace

// spark_attn.cu
spark_status device_ready(int *sms);

namespace {

spark_status reserve(const spark_page_pool *pool, const int32_t *add, int32_t *taken,
                     void *workspace, size_t workspace_bytes, void *stream, int token_bytes) {
    spark_status st = check_pool(pool, workspace, workspace_bytes);
    if (st != SPARK_OK) return st;
    if (pool->n_rows > 0 && !add) return SPARK_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(add) % 4 || reinterpret_cast<uintptr_t>(taken) % 4)
        return SPARK_ERR_ALIGN;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    const PoolParams P = pool_params(pool, workspace, token_bytes);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = done(launch_overlapped(reserve_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, P, add,
                                taken));
    const long long most = pool->n_rows < pool->n_pages ? pool->n_rows : pool->n_pages;
    if (st != SPARK_OK || most == 0) return st;
    return done(launch_copies<false>(P, most, sms, s));
}

spark_status compact(const spark_page_pool *pool, int32_t *live, void *workspace,
                     size_t workspace_bytes, void *stream, int token_bytes) {
    spark_status st = check_pool(pool, workspace, workspace_bytes);
    if (st != SPARK_OK) return st;
    if (reinterpret_cast<uintptr_t>(live) % 4) return SPARK_ERR_ALIGN;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    const PoolParams P = pool_params(pool, workspace, token_bytes);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = done(launch_overlapped(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, P, live));
    if (st != SPARK_OK || pool->n_rows == 0 || pool->n_pages == 0) return st;
    return done(launch_copies<true>(P, pool->n_pages / 2 + 1, sms, s));
}

}  // namespace

}  // namespace spark

using namespace spark;

extern "C" {

size_t spark_attn_pages_workspace_size(const spark_page_pool *pool) {
    if (check_pool_sizes(pool) != SPARK_OK) return 0;
    return plan_pool(pool).bytes;
}

spark_status spark_attn_pages_fork(const spark_page_pool *pool, const int32_t *src,
                                   const int32_t *dst, int n, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    spark_status st = check_pool(pool, workspace, workspace_bytes);
    if (st != SPARK_OK) return st;
    if (n < 0) return SPARK_ERR_SHAPE;
    if (n == 0) return SPARK_OK;
    if (!src || !dst) return SPARK_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(src) % 4 || reinterpret_cast<uintptr_t>(dst) % 4)
        return SPARK_ERR_ALIGN;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    const PoolParams P = pool_params(pool, workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (static_cast<long long>(n) * pool->max_pages <= kForkSmall)
        return done(launch_overlapped(fork_kernel, dim3(1), dim3(kPlanThreads), 0, s, P, src, dst,
                                      n));
    st = done(launch_overlapped(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, P, src, dst,
                                n));
    if (st != SPARK_OK) return st;
    return done(launch_overlapped(fork_apply_kernel, dim3(n), dim3(kRowThreads), 0, s, P, src, dst,
                                  n));
}

spark_status spark_attn_pages_reserve(const spark_page_pool *pool, const int32_t *add,
                                      int32_t *taken, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    return reserve(pool, add, taken, workspace, workspace_bytes, stream, kHeadDim * 2);
}

spark_status spark_attn_kv4_pages_reserve(const spark_page_pool *pool, const int32_t *add,
                                          int32_t *taken, void *workspace, size_t workspace_bytes,
                                          void *stream) {
    return reserve(pool, add, taken, workspace, workspace_bytes, stream, kKv4TokenBytes);
}

spark_status spark_attn_pages_free(const spark_page_pool *pool, const int32_t *rows,
                                   const int32_t *keep, int n, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    spark_status st = check_pool(pool, workspace, workspace_bytes);
    if (st != SPARK_OK) return st;
    if (n < 0) return SPARK_ERR_SHAPE;
    if (n == 0) return SPARK_OK;
    if (!rows) return SPARK_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(rows) % 4 || reinterpret_cast<uintptr_t>(keep) % 4)
        return SPARK_ERR_ALIGN;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    return done(launch_overlapped(free_kernel, dim3(n), dim3(kRowThreads), 0,
                                  static_cast<cudaStream_t>(stream), pool_params(pool, workspace),
                                  rows, keep, n));
}

spark_status spark_attn_pages_compact(const spark_page_pool *pool, int32_t *live, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    return compact(pool, live, workspace, workspace_bytes, stream, kHeadDim * 2);
}

spark_status spark_attn_kv4_pages_compact(const spark_page_pool *pool, int32_t *live,
                                          void *workspace, size_t workspace_bytes, void *stream) {
    return compact(pool, live, workspace, workspace_bytes, stream, kKv4TokenBytes);
}

}  // extern "C"
