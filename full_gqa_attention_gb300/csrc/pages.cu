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
__device__ __forceinline__ bool row_sane(const PoolParams &P, int row, int held, int len) {
    return held >= 0 && held <= P.max_pages && len >= 0 && pages_of(len, P.page_size) <= held;
}

// ---------------------------------------------------------------- fork

// Decides every pair before any row changes: row_a[i % ...] cannot hold more
// pairs than rows, since a row is the target of one pair at most; pairs past
// n_rows repeat a target and are refused here.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(
    const __grid_constant__ PoolParams P, const int32_t *src, const int32_t *dst, int n) {
    grid_dep_wait();
    grid_dep_launch();
    // row_a[r]: the pair that forks into row r, or -1; row_b[r]: its pages;
    // row_c[r]: its tokens
    for (int r = threadIdx.x; r < P.n_rows; r += kPlanThreads) P.row_a[r] = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int d = dst[i];
        if (d >= 0 && d < P.n_rows) atomicMin(&P.row_a[d], i);  // the first mention
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        const int s = src[i], d = dst[i];
        bool ok = s >= 0 && s < P.n_rows && d >= 0 && d < P.n_rows;
        if (ok) ok = P.row_a[d] == i;
        if (ok) ok = P.held[d] == 0 && row_sane(P, s, P.held[s], P.len[s]);
        if (!ok) {
            atomicOr(P.status, kErrRow);
            // a pair that comes first but is refused leaves the row alone
            if (d >= 0 && d < P.n_rows && P.row_a[d] == i) P.row_b[d] = -1;
        } else {
            P.row_b[d] = pages_of(P.len[s], P.page_size);
            P.row_c[d] = P.len[s];
        }
    }
}

// One CTA per pair: the table row and the counts.
__global__ void __launch_bounds__(kRowThreads) fork_apply_kernel(
    const __grid_constant__ PoolParams P, const int32_t *src, const int32_t *dst, int n) {
    grid_dep_wait();
    grid_dep_launch();
    const int i = blockIdx.x;
    const int d = dst[i];
    if (d < 0 || d >= P.n_rows || P.row_a[d] != i || P.row_b[d] < 0) return;
    const int count = P.row_b[d];
    const int32_t *from = P.table + static_cast<size_t>(src[i]) * P.max_pages;
    int32_t *to = P.table + static_cast<size_t>(d) * P.max_pages;
    for (int j = threadIdx.x; j < P.max_pages; j += kRowThreads) {
        int p = -1;
        if (j < count) {
            p = from[j];
            if (p < 0 || p >= P.n_pages) {
                atomicOr(P.status, kErrPage);
            } else {
                atomicAdd(&P.refs[p], 1);
            }
        }
        to[j] = p;
    }
    if (threadIdx.x == 0) {
        P.held[d] = count;
        P.len[d] = P.row_c[d];
    }
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
    if (!row_sane(P, r, held, len)) {
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

// One CTA.  row_a[r]: the page row r is about to write into although it holds
// tokens already (-1: none); row_b[r]: pages wanted, the copy in bit 30;
// row_c[r]: exclusive prefix of the wants.
__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(
    const __grid_constant__ PoolParams P, const int32_t *add, int32_t *taken) {
    __shared__ int warp_sums[32];
    __shared__ long long wide_sums[32];
    constexpr int kCopyBit = 1 << 30;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    for (int r = tid; r < P.n_rows; r += kPlanThreads) {
        int page = -1, fresh = 0;
        const int more = add[r];
        if (more > 0) {
            const int held = P.held[r], len = P.len[r];
            const long long end = static_cast<long long>(len) + more;
            if (!row_sane(P, r, held, len) ||
                end > static_cast<long long>(P.max_pages) * P.page_size) {
                atomicOr(P.status, kErrRow);
            } else {
                const int need = static_cast<int>((end + P.page_size - 1) / P.page_size);
                fresh = need > held ? need - held : 0;
                if (fresh > P.n_pages) fresh = P.n_pages + 1;  // too many, whatever the sum
                if (len % P.page_size) {
                    page = P.table[static_cast<size_t>(r) * P.max_pages + len / P.page_size];
                    if (page < 0 || page >= P.n_pages) {
                        atomicOr(P.status, kErrPage);
                        page = -1;
                        fresh = 0;
                    }
                }
            }
        }
        P.row_a[r] = page;
        P.row_b[r] = fresh;
    }
    __syncthreads();
    // copies: all rows that share the page but the last holder
    for (int r = tid; r < P.n_rows; r += kPlanThreads) {
        const int page = P.row_a[r];
        if (page < 0) continue;
        const int refs = P.refs[page];
        if (refs <= 1) continue;
        int before = 0;
        for (int q = 0; q < r; ++q) before += P.row_a[q] == page;
        if (refs - before > 1) P.row_b[r] |= kCopyBit;
    }
    __syncthreads();
    // prefix sum of the wants, and of the copies, over the rows
    long long base = 0;
    int copies = 0;
    for (int r0 = 0; r0 < P.n_rows; r0 += kPlanThreads) {
        const int r = r0 + tid;
        const int w = r < P.n_rows ? P.row_b[r] : 0;
        const int cp = (w & kCopyBit) ? 1 : 0;
        long long total;
        int ctotal;
        const long long at =
            base + block_scan<long long>((w & ~kCopyBit) + cp, &total, wide_sums);
        const int cat = copies + block_scan(cp, &ctotal, warp_sums);
        // past n_pages the call will be refused: nothing of it is used
        if (r < P.n_rows) P.row_c[r] = static_cast<int>(at < P.n_pages ? at : P.n_pages);
        if (cp && cat < P.n_pages) {
            P.copy_src[cat] = P.row_a[r];
            P.copy_dst[cat] = static_cast<int>(at < P.n_pages ? at : P.n_pages);  // a rank, for now
        }
        base += total;
        copies += ctotal;
    }
    const int want = static_cast<int>(base <= P.n_pages ? base : P.n_pages + 1);
    // the first `want` free pages, in map[]
    int found = 0;
    for (int p0 = 0; p0 < P.n_pages && found < want; p0 += kPlanThreads) {
        const int p = p0 + tid;
        const int is_free = p < P.n_pages && P.refs[p] == 0;
        int total;
        const int at = block_scan(is_free, &total, warp_sums);
        if (is_free && found + at < want) P.map[found + at] = p;
        found += total;
    }
    __syncthreads();
    if (found < want) {
        if (tid == 0) {
            *P.n_copies = 0;
            if (taken) *taken = -1;
        }
        return;
    }
    if (tid == 0) {
        *P.n_copies = copies;
        if (taken) *taken = want;
    }
    for (int i = tid; i < want; i += kPlanThreads) P.refs[P.map[i]] = 1;
    for (int i = tid; i < copies; i += kPlanThreads) {
        P.copy_dst[i] = P.map[P.copy_dst[i]];
        atomicSub(&P.refs[P.copy_src[i]], 1);
    }
    for (int r = tid; r < P.n_rows; r += kPlanThreads) {
        const int w = P.row_b[r];
        if (!w) continue;
        int at = P.row_c[r];
        int32_t *row = P.table + static_cast<size_t>(r) * P.max_pages;
        if (w & kCopyBit) row[P.len[r] / P.page_size] = P.map[at++];
        const int fresh = w & ~kCopyBit, held = P.held[r];
        for (int j = 0; j < fresh; ++j) row[held + j] = P.map[at + j];
        P.held[r] = held + fresh;
    }
}

// ---------------------------------------------------------------- compact

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(
    const __grid_constant__ PoolParams P, int32_t *live) {
    __shared__ int warp_sums[32];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    int n = 0;
    for (int p = tid; p < P.n_pages; p += kPlanThreads) n += P.refs[p] > 0;
    int n_live;
    block_scan(n, &n_live, warp_sums);
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < P.n_pages; p0 += kPlanThreads) {
        const int p = p0 + tid;
        const bool used = p < P.n_pages && P.refs[p] > 0;
        const int hole = p < n_live && !used, mover = p >= n_live && used;
        int total;
        int at = block_scan(hole, &total, warp_sums);
        if (hole) P.copy_dst[holes + at] = p;
        holes += total;
        at = block_scan(mover, &total, warp_sums);
        if (mover) P.copy_src[movers + at] = p;
        if (p < P.n_pages) P.map[p] = p;
        movers += total;
    }
    __syncthreads();
    for (int i = tid; i < movers; i += kPlanThreads) {  // as many holes as movers
        const int s = P.copy_src[i], d = P.copy_dst[i];
        P.map[s] = d;
        P.refs[d] = P.refs[s];
        P.refs[s] = 0;
    }
    if (tid == 0) {
        *P.n_copies = movers;
        if (live) *live = n_live;
        P.row_a[0] = n_live;
    }
}

// The tables follow their pages: one CTA per row.
__global__ void __launch_bounds__(kRowThreads) compact_table_kernel(
    const __grid_constant__ PoolParams P) {
    grid_dep_wait();
    grid_dep_launch();
    const int r = blockIdx.x, n_live = P.row_a[0];
    const int held = P.held[r];
    if (held < 0 || held > P.max_pages) {
        if (threadIdx.x == 0) atomicOr(P.status, kErrRow);
        return;
    }
    int32_t *row = P.table + static_cast<size_t>(r) * P.max_pages;
    for (int j = threadIdx.x; j < held; j += kRowThreads) {
        const int p = row[j];
        if (p < 0 || p >= P.n_pages)
            atomicOr(P.status, kErrPage);
        else if (p >= n_live)
            row[j] = P.map[p];
    }
}

// ---------------------------------------------------------------- copies

// The listed page copies in every layer, K and V, in chunks of 32 KB (or the
// page, where it is smaller).  No page is the source of one copy and the
// target of another, so their order does not matter.
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(
    const __grid_constant__ PoolParams P) {
    grid_dep_wait();
    grid_dep_launch();
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

PoolParams pool_params(const spark_page_pool *pool, void *workspace) {
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
    P.page_bytes = static_cast<long long>(pool->Hkv) * pool->page_size * kHeadDim * 2;
    P.status = reinterpret_cast<unsigned *>(ws);
    P.n_copies = reinterpret_cast<int32_t *>(ws + pl.counts);
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

cudaError_t launch_copies(const PoolParams &P, long long most, int sms, cudaStream_t stream) {
    const long long per_page = (P.page_bytes + kCopyChunk - 1) / kCopyChunk;
    long long grid = static_cast<long long>(sms) * 4;
    if (grid > per_page * 2 * P.n_layers * most) grid = per_page * 2 * P.n_layers * most;
    return launch_overlapped(page_copy_kernel, dim3(static_cast<unsigned>(grid)),
                             dim3(kCopyThreads), 0, stream, P);
}

}  // namespace

// spark_attn.cu
spark_status device_ready(int *sms);

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
    st = done(launch_overlapped(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, P, src, dst,
                                n));
    if (st != SPARK_OK) return st;
    return done(launch_overlapped(fork_apply_kernel, dim3(n), dim3(kRowThreads), 0, s, P, src, dst,
                                  n));
}

spark_status spark_attn_pages_reserve(const spark_page_pool *pool, const int32_t *add,
                                      int32_t *taken, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    spark_status st = check_pool(pool, workspace, workspace_bytes);
    if (st != SPARK_OK) return st;
    if (pool->n_rows > 0 && !add) return SPARK_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(add) % 4 || reinterpret_cast<uintptr_t>(taken) % 4)
        return SPARK_ERR_ALIGN;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    const PoolParams P = pool_params(pool, workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = done(launch_overlapped(reserve_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, P, add,
                                taken));
    const long long most = pool->n_rows < pool->n_pages ? pool->n_rows : pool->n_pages;
    if (st != SPARK_OK || most == 0) return st;
    return done(launch_copies(P, most, sms, s));
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
    spark_status st = check_pool(pool, workspace, workspace_bytes);
    if (st != SPARK_OK) return st;
    if (reinterpret_cast<uintptr_t>(live) % 4) return SPARK_ERR_ALIGN;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    const PoolParams P = pool_params(pool, workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = done(launch_overlapped(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, P, live));
    if (st != SPARK_OK || pool->n_rows == 0 || pool->n_pages == 0) return st;
    st = done(launch_overlapped(compact_table_kernel, dim3(pool->n_rows), dim3(kRowThreads), 0, s,
                                P));
    if (st != SPARK_OK) return st;
    return done(launch_copies(P, pool->n_pages / 2 + 1, sms, s));
}

}  // extern "C"
