// paged.cu -- packed prompts and a cache in pages: the host side and the
// kernels that are not attention itself.
#include <cstring>

#include "paged.cuh"
#include "spark_attn.h"

namespace spark {

void fill_rope_table(const spark_layer_desc *d, RopeTable *t);
spark_status device_ready(int *sms);
spark_status check_layer_desc(const spark_layer_desc *d, int H, int Hkv);
bool encode_bf16_map(CUtensorMap *map, const void *base, int rank, const uint64_t *dims,
                     const uint64_t *strides, const uint32_t *box);
cudaError_t launch_prefill_packed(const CUtensorMap &tm_q, const CUtensorMap &tm_kv_k,
                                  const CUtensorMap &tm_kv_v, const CUtensorMap &tm_krot,
                                  const CUtensorMap &tm_out, const PrefillParams &P,
                                  long long items, cudaStream_t stream);
cudaError_t launch_decode_paged(const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                const PagedParams &P, int grid, cudaStream_t stream);

namespace {

constexpr int kPrepThreads = 256;
constexpr int kBins = 1024;           // query tiles are sorted by their key tiles, up to this many

// Exclusive prefix sum of one value per thread over the block, and the total.
__device__ __forceinline__ int prep_scan(int v, int *total) {
    __shared__ int sums[kPrepThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();  // the sums of the scan before are read
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPrepThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    *total = all;
    return before + x - v;
}

// The list of query tiles, made by one CTA: every sequence is cut into tiles
// of tq tokens, and the tiles are put in order of the key tiles they visit,
// most first (a counting sort), so that the long ones do not start last.  Tiles
// that all run at once need no order and get none.  The order inside a bin is
// whatever the atomics give; no result depends on it.
//
// A query tile that would outlast the others is split along its keys into
// parts of L key tiles or fewer.  With no more query tiles than SMs, L is the
// least that still fits them all in one wave; else it is an SM's share of all
// the work and kPartCost besides, what a part costs in key tiles (set-up,
// leaving its state, joining).  So uniform batches are not split, and a short
// chunk on top of a long prefix fills the GPU.
//
// kMinPart, 3 to 12: the same on every split measured (one token on 131,072,
// 512 on 65,536, packed prompts of 2500 and 5000 tokens); it decides from which
// length on a call has places for parts at all.  kPartCost 5 / 8 / 12: 512
// tokens on 65,536 442 us each; packed 2500 tokens (8/2 heads) 44 / 46 / 44,
// 5000 tokens (4/1 heads) 72 / 66 / 70, 45 tokens on 16,384 beside 59 short
// chunks 58 / 63 / 65.
constexpr int kMinPart = 6;
constexpr int kPartCost = 8;
constexpr int kPlanSeqs = 1024;       // sequences whose offsets fit in shared memory
constexpr int kMaxSms = 256;

__device__ __forceinline__ void plan_tiles(const PagedParams &P) {
    __shared__ int bins[kBins];
    __shared__ int s_base[kPlanSeqs + 1];
    __shared__ int s_n[kMaxSms];
    __shared__ int s_limit, s_slots, s_splits, s_max;
    __shared__ unsigned long long s_total;
    const int tid = threadIdx.x, tq = 128 / P.G;
    const long long cap = static_cast<long long>(P.max_pages) << P.page_shift;
    int *tile_base = P.S <= kPlanSeqs ? s_base : P.tile_base;
    for (int i = tid; i < kBins; i += kPrepThreads) bins[i] = 0;
    const unsigned call = *P.call;  // the attention kernel counts it on
    if (tid == 0) {
        P.odd_values[(call + 1) & 1] = 0;
        s_total = 0;
        s_max = s_slots = s_splits = 0;
    }
    int base = 0;
    for (int s0 = 0; s0 < P.S; s0 += kPrepThreads) {
        const int s = s0 + tid;
        int n = 0;
        if (s < P.S) {
            const int a = P.cu[s], b = P.cu[s + 1];
            if (a < 0 || a > b || b > P.N) {
                atomicOr(P.status, kErrSeqlens);
            } else if (b > a) {
                const long long st = P.start ? P.start[s] : 0;
                if (st < 0 || (P.start && st + (b - a) > cap))
                    atomicOr(P.status, kErrPosition);
                else
                    n = (b - a + tq - 1) / tq;
            }
        }
        int total;
        const int at = prep_scan(n, &total);
        if (s < P.S) tile_base[s] = base + at;
        // offsets that overlap can ask for more tiles than the list holds, and
        // many times more than 32 bits do
        base = base + total < P.most ? base + total : P.most;
    }
    const int extra = P.slots > 0 ? P.sms / P.Hkv + 1 : 0;
    const int n_tiles = base < P.most - extra ? base : P.most - extra;
    __syncthreads();
    auto tile = [&](int i) {
        int lo = 0, hi = P.S - 1;  // the last s with tile_base[s] <= i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tile_base[mid] <= i)
                lo = mid;
            else
                hi = mid - 1;
        }
        PackedItem t;
        t.seq = lo;
        t.t0 = (i - tile_base[lo]) * tq;
        t.row0 = P.cu[lo];
        t.len = P.cu[lo + 1] - t.row0;
        t.start = P.start ? P.start[lo] : 0;
        t.call = call;
        t.k0 = 0;
        t.tiles = prefill_key_tiles(P.kind, P.window, t.start + t.t0,
                                    t.start + (t.t0 + tq < t.len ? t.t0 + tq : t.len), 128,
                                    P.start != nullptr).ntiles;
        t.part = t.slot = t.pad = 0;
        t.parts = 1;
        return t;
    };
    PackedItem first = {};  // the thread's first tile: in most calls its only one
    if (tid < n_tiles) first = tile(tid);
    const bool wave = static_cast<long long>(n_tiles) * P.Hkv <= P.sms;
    if (P.slots > 0) {
        unsigned long long sum = 0;
        int most = 0;
        for (int i = tid; i < n_tiles; i += kPrepThreads) {
            const int n = i == tid ? first.tiles : tile(i).tiles;
            sum += n;
            most = n > most ? n : most;
            if (wave) s_n[i] = n;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
            most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
        }
        if ((tid & 31) == 0) {
            atomicAdd(&s_total, sum);
            atomicMax(&s_max, most);
        }
        __syncthreads();
    }
    if (tid < 32) {
        // the longest part
        int limit = 1 << 30;
        if (P.slots > 0 && s_max > kMinPart) {
            limit = s_max;
            if (wave) {
                int lo = kMinPart, hi = s_max;  // hi fits
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    int parts = 0;
                    for (int i = tid; i < n_tiles; i += 32) parts += (s_n[i] + mid - 1) / mid;
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
                        parts += __shfl_xor_sync(0xffffffffu, parts, off);
                    if (parts * P.Hkv <= P.sms)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                if (hi + kPartCost < limit) limit = hi;
            } else {
                const unsigned long long share =
                    (s_total * P.Hkv + P.sms - 1) / P.sms + kPartCost;
                if (share < static_cast<unsigned long long>(limit))
                    limit = static_cast<int>(share);
            }
        }
        if (tid == 0) s_limit = limit;
    }
    __syncthreads();
    const int limit = s_limit;
    // (tiles of a single wave start together: they need no order, one bin does)
    auto bin_of = [&](int n) { return wave ? 0 : kBins - 1 - (n < kBins ? n : kBins - 1); };
    int total = 0;
    if (!wave) {
        for (int i = tid; i < n_tiles; i += kPrepThreads) {
            const int n = i == tid ? first.tiles : tile(i).tiles;
            const int parts = (n + limit - 1) / limit;
            atomicAdd(&bins[bin_of((n + parts - 1) / parts)], parts);
        }
        __syncthreads();
        constexpr int kPer = kBins / kPrepThreads;
        int count[kPer], mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            count[i] = bins[tid * kPer + i];
            mine += count[i];
        }
        int at = prep_scan(mine, &total);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            bins[tid * kPer + i] = at;
            at += count[i];
        }
        __syncthreads();
    }
    for (int i = tid; i < n_tiles; i += kPrepThreads) {
        PackedItem t = i == tid ? first : tile(i);
        const int n = t.tiles, parts = (n + limit - 1) / limit;
        int place = atomicAdd(&bins[bin_of((n + parts - 1) / parts)], parts);
        if (parts > 1) {
            t.parts = parts;
            t.slot = atomicAdd(&s_slots, parts * P.Hkv);
            P.splits[atomicAdd(&s_splits, 1)] = t;
        }
        for (int p = 0; p < parts; ++p) {
            t.part = p;
            t.k0 = static_cast<int>(static_cast<long long>(n) * p / parts);
            t.tiles = static_cast<int>(static_cast<long long>(n) * (p + 1) / parts) - t.k0;
            P.work[place++] = t;
        }
    }
    __syncthreads();
    if (wave) total = bins[0];
    for (int i = total + tid; i < P.most; i += kPrepThreads) {
        PackedItem t = {};
        t.seq = -1;
        t.call = call;
        P.work[i] = t;
    }
    if (tid == 0) *P.n_splits = s_splits;
}

// Where the token of `row` goes in the pages (elements), or -1: padding, or a
// place that does not exist.  One warp; lane 0 reports.
__device__ __forceinline__ long long token_slot(const PagedParams &P, int row, int lane) {
    const long long cap = static_cast<long long>(P.max_pages) << P.page_shift;
    const int seq = find_sequence(P.cu, P.S, row, lane);
    if (seq < 0) return -1;
    const int t0 = P.cu[seq], t1 = P.cu[seq + 1];
    const long long st = P.start[seq];
    if (t0 < 0 || t1 > P.N || st < 0 || st + (t1 - t0) > cap) return -1;  // the plan reports it
    const long long a = st + (row - t0);  // index in the sequence
    const int page = P.table[static_cast<size_t>(seq) * P.max_pages + (a >> P.page_shift)];
    if (page < 0 || page >= P.n_pages) {
        if (lane == 0) atomicOr(P.status, kErrPage);
        return -1;
    }
    return ((static_cast<long long>(page) * P.Hkv << P.page_shift) +
            (a & ((1 << P.page_shift) - 1))) * kHeadDim;
}

constexpr int kPrepRows = kPrepThreads / 32;  // tokens per CTA: a warp finds each one's place
constexpr int kPrepHeads = 4;                 // KV heads whose loads are in flight at once

// What the attention kernel needs of the new keys and values.  Paged: every
// token's rotated key and its value go to its pages.  Packed: the leading
// rot_w dims of every key, rotated, go to the workspace (the others are read
// where they are).  The values are looked over for one that is not finite:
// with none, a boundary tile needs no pass over its V but for slots from before
// the call and behind the sequence's end.  A CTA takes kPrepRows
// tokens; one thread per (token, 4 rotated pairs) or (token, 8 copied key dims
// or value dims), over the KV heads, so that each angle is computed once; the
// rotations come first, so that few warps do both.  The first CTA makes the
// list of query tiles instead.
__global__ void __launch_bounds__(kPrepThreads) paged_prep_kernel(
    const __grid_constant__ PagedParams P) {
    __shared__ long long place[kPrepRows];
    // (the lanes' frequencies differ: from the parameters, constant memory, they
    // would come one lane after another)
    __shared__ __align__(16) float2 freq[kHeadDim / 2];
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x == 0) {
        plan_tiles(P);
        return;
    }
    const bool paged = P.k_pages != nullptr;
    const int r = P.rope.rot_dim, half = r / 2;
    const int n_rot = half / 4, n_kcopy = ((paged ? kHeadDim : P.rot_w) - r) / 8;
    const int n_copy = n_kcopy + kHeadDim / 8;
    const long long first = (blockIdx.x - 1ll) * kPrepRows;
    if (paged) {
        const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const long long at =
            first + w < P.N ? token_slot(P, static_cast<int>(first + w), lane) : -1;
        if (lane == 0) place[w] = at;
    }
    if (threadIdx.x < half) freq[threadIdx.x] = P.rope.u[threadIdx.x];
    __syncthreads();
    const size_t width = static_cast<size_t>(P.H + 2 * P.Hkv) * kHeadDim;
    const size_t head_stride = paged ? static_cast<size_t>(kHeadDim) << P.page_shift
                                     : static_cast<size_t>(P.N) * P.rot_w;
    auto dst_of = [&](int w, int row) {
        return paged ? static_cast<size_t>(place[w]) : static_cast<size_t>(row) * P.rot_w;
    };
    auto there = [&](int w) { return first + w < P.N && (!paged || place[w] >= 0); };
    for (int i = threadIdx.x; i < kPrepRows * n_rot; i += kPrepThreads) {
        const int w = i / n_rot, k0 = i % n_rot * 4;
        if (!there(w)) continue;
        const int row = static_cast<int>(first + w);
        const __nv_bfloat16 *src = P.qkv + row * width + static_cast<size_t>(P.H) * kHeadDim + k0;
        __nv_bfloat16 *dst = (paged ? P.k_pages : P.krot) + dst_of(w, row) + k0;
        const int p = P.pos[row];
        uint2 x[kPrepHeads], y[kPrepHeads];
        auto load = [&](int g0) {
#pragma unroll
            for (int g = 0; g < kPrepHeads; ++g) {
                if (g0 + g >= P.Hkv) break;
                x[g] = *reinterpret_cast<const uint2 *>(src + (g0 + g) * kHeadDim);
                y[g] = *reinterpret_cast<const uint2 *>(src + (g0 + g) * kHeadDim + half);
            }
        };
        load(0);
        float c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) rope_cos_sin_fine(p, freq[k0 + j], c[j], s[j]);
        for (int g0 = 0; g0 < P.Hkv; g0 += kPrepHeads) {
            if (g0) load(g0);
#pragma unroll
            for (int g = 0; g < kPrepHeads; ++g) {
                if (g0 + g >= P.Hkv) break;
                const uint32_t xw[2] = {x[g].x, x[g].y}, yw[2] = {y[g].x, y[g].y};
                uint32_t ya[2], yb[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float y1l, y2l, y1h, y2h;
                    rope_rotate(bf16_lo(xw[j]), bf16_lo(yw[j]), c[2 * j], s[2 * j], y1l, y2l);
                    rope_rotate(bf16_hi(xw[j]), bf16_hi(yw[j]), c[2 * j + 1], s[2 * j + 1], y1h,
                                y2h);
                    ya[j] = pack_bf16x2(y1l, y1h);
                    yb[j] = pack_bf16x2(y2l, y2h);
                }
                __nv_bfloat16 *to = dst + (g0 + g) * head_stride;
                *reinterpret_cast<uint2 *>(to) = make_uint2(ya[0], ya[1]);
                *reinterpret_cast<uint2 *>(to + half) = make_uint2(yb[0], yb[1]);
            }
        }
    }
    uint32_t hit = 0;
    // (from the last thread down: the first ones have rotations behind them)
    for (int i = kPrepThreads - 1 - threadIdx.x; i < kPrepRows * n_copy; i += kPrepThreads) {
        const int w = i / n_copy, it = i % n_copy;
        if (!there(w)) continue;
        const int row = static_cast<int>(first + w);
        const bool key = it < n_kcopy;
        const int d0 = key ? r + it * 8 : (it - n_kcopy) * 8;
        const __nv_bfloat16 *src =
            P.qkv + row * width + static_cast<size_t>(P.H + (key ? 0 : P.Hkv)) * kHeadDim + d0;
        __nv_bfloat16 *dst = (key ? (paged ? P.k_pages : P.krot) : P.v_pages) + d0;
        if (key || paged) dst += dst_of(w, row);
        for (int g0 = 0; g0 < P.Hkv; g0 += kPrepHeads) {
            uint4 v[kPrepHeads];
#pragma unroll
            for (int g = 0; g < kPrepHeads; ++g)
                v[g] = g0 + g < P.Hkv
                           ? *reinterpret_cast<const uint4 *>(src + (g0 + g) * kHeadDim)
                           : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int g = 0; g < kPrepHeads; ++g) {
                if (g0 + g >= P.Hkv) break;
                if (key || paged) *reinterpret_cast<uint4 *>(dst + (g0 + g) * head_stride) = v[g];
                if (!key)  // an exponent of all ones carries into the sign's place
                    hit |= ((v[g].x & 0x7F807F80u) + 0x00800080u) |
                           ((v[g].y & 0x7F807F80u) + 0x00800080u) |
                           ((v[g].z & 0x7F807F80u) + 0x00800080u) |
                           ((v[g].w & 0x7F807F80u) + 0x00800080u);
            }
        }
    }
    if (hit & 0x80008000u) atomicOr(&P.odd_values[*P.call & 1], 1u);
}

// ---------------------------------------------------------------- host side

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// Arguments of the pool as an attention call sees it.
spark_status check_pages(const void *k_pages, const void *v_pages, int n_pages, int page_size,
                         const int32_t *table, int max_pages) {
    if (n_pages < 0 || max_pages < 0) return SPARK_ERR_SHAPE;
    if (page_shift_of(page_size) < 0) return SPARK_ERR_UNSUPPORTED;
    if (max_pages >= (1 << 30) / page_size) return SPARK_ERR_UNSUPPORTED;
    if (n_pages == 0 || max_pages == 0) return SPARK_ERR_CAPACITY;
    if (!k_pages || !v_pages || !table) return SPARK_ERR_NULL;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(table, 4))
        return SPARK_ERR_ALIGN;
    return SPARK_OK;
}

spark_status check_packed(int n_tokens, int S, int H, int Hkv, const spark_layer_desc *desc) {
    const spark_status st = check_layer_desc(desc, H, Hkv);
    if (st != SPARK_OK) return st;
    if (n_tokens < 0 || S < 0) return SPARK_ERR_SHAPE;
    return SPARK_OK;
}

PagedParams make_params(const void *qkv, const float *gate, const int32_t *pos,
                        const spark_layer_desc *desc, int N, int S, int H, int Hkv, void *out,
                        void *workspace) {
    PagedParams P;
    std::memset(&P, 0, sizeof(P));
    P.qkv = static_cast<const __nv_bfloat16 *>(qkv);
    P.gate = gate;
    P.pos = pos;
    P.out = static_cast<__nv_bfloat16 *>(out);
    P.status = static_cast<unsigned *>(workspace);
    P.N = N;
    P.S = S;
    P.H = H;
    P.Hkv = Hkv;
    P.G = H / Hkv;
    P.kind = desc->kind;
    // (indices stay below 2^30: a wider window is no narrower, and sums with it
    // stay in 32 bits)
    constexpr int kMostWindow = 1 << 30;
    P.window = desc->kind != SPARK_LAYER_SLIDING  ? 0
               : desc->window < kMostWindow ? desc->window
                                            : kMostWindow;
    P.gate_mode = desc->gate_mode;
    fill_rope_table(desc, &P.rope);
    return P;
}

void set_pages(PagedParams &P, void *k_pages, void *v_pages, int n_pages, int page_size,
               const int32_t *table, int max_pages) {
    P.k_pages = static_cast<__nv_bfloat16 *>(k_pages);
    P.v_pages = static_cast<__nv_bfloat16 *>(v_pages);
    P.table = table;
    P.n_pages = n_pages;
    P.page_shift = page_shift_of(page_size);
    P.max_pages = max_pages;
}

spark_status done(cudaError_t e) {
    if (e == cudaSuccess) return SPARK_OK;
    cudaGetLastError();
    return SPARK_ERR_CUDA;
}

spark_status launch_prep(const PagedParams &P, cudaStream_t s) {
    const long long blocks = (static_cast<long long>(P.N) + kPrepRows - 1) / kPrepRows + 1;
    return done(launch_overlapped(paged_prep_kernel, dim3(static_cast<unsigned>(blocks)),
                                  dim3(kPrepThreads), 0, s, P));
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace of a packed or paged prefill: the status header, the query tiles,
// and (packed) the rotated leading key dims.
struct PackedPlan {
    long long most;  // items at most: full query tiles, a ragged one per sequence, parts
    int rot_w, slots;
    size_t flags, base, splits, work, krot, ml, o, bytes;
};

// Query tiles are split where keys are many: always possible over pages, and in
// a packed prompt of more than kMinPart key tiles.  At most two parts per SM
// then have a state to leave (plan_tiles: a tile is split into parts of at
// least an SM's share, or all parts fit in one wave).
PackedPlan plan_packed(int N, int S, int H, int Hkv, const spark_layer_desc *desc, bool paged,
                       int sms) {
    PackedPlan pl{};
    const int tq = 128 / (H / Hkv);
    pl.most = static_cast<long long>(N / tq) + (S < N ? S : N);
    pl.rot_w = paged ? 0 : (desc->rot_dim + 63) / 64 * 64;
    const bool long_rows = desc->kind == SPARK_LAYER_FULL || desc->window > 128 * kMinPart;
    if (long_rows && (paged || N > 128 * kMinPart) && sms <= kMaxSms) {
        pl.slots = 2 * sms;
        pl.most += sms / Hkv + 1;
    }
    pl.flags = kWorkspaceHeader;
    pl.base = pl.flags + 256;
    pl.splits = pl.base + up256((static_cast<size_t>(S) + 1) * 4);
    pl.work = pl.splits + up256((pl.slots > 0 ? sms : 0) * sizeof(PackedItem));
    pl.krot = pl.work + up256(static_cast<size_t>(pl.most) * sizeof(PackedItem));
    pl.ml = pl.krot + up256(static_cast<size_t>(N) * Hkv * pl.rot_w * 2);
    pl.o = pl.ml + static_cast<size_t>(pl.slots) * 128 * sizeof(float2);
    pl.bytes = pl.o + static_cast<size_t>(pl.slots) * 128 * kHeadDim * sizeof(float);
    return pl;
}

size_t packed_workspace(int N, int S, int H, int Hkv, const spark_layer_desc *desc, bool paged) {
    int sms;
    device_ready(&sms);
    return plan_packed(N, S, H, Hkv, desc, paged, sms).bytes;
}

// The attention kernel's launch: its parameters and tensor maps.
spark_status launch_packed_attn(const PagedParams &P, const PackedPlan &pl, int sms, cudaStream_t stream) {
    const bool paged = P.k_pages != nullptr;
    const int tq = 128 / P.G;
    PrefillParams A;
    std::memset(&A, 0, sizeof(A));
    A.qkv = P.qkv;
    A.gate = P.gate;
    A.pos = P.pos;
    A.v_cache = P.v_pages;
    A.start = P.start;
    A.status = P.status;
    A.B = 1;
    A.T = P.N;
    A.H = P.H;
    A.Hkv = P.Hkv;
    A.G = P.G;
    A.kind = P.kind;
    A.window = P.window;
    A.gate_mode = P.gate_mode;
    A.rot_w = pl.rot_w;
    A.wave = sms;
    A.pk.work = P.work;
    if (pl.slots > 0) {
        A.pk.part_ml = reinterpret_cast<float2 *>(P.part_ml);
        A.pk.part_o = reinterpret_cast<float4 *>(P.part_o);
        A.pk.splits = P.splits;
        A.pk.n_splits = P.n_splits;
    }
    A.pk.odd_values = P.odd_values;
    A.pk.call = P.call;
    A.pk.table = P.table;
    A.pk.n_pages = P.n_pages;
    A.pk.page_shift = P.page_shift;
    A.pk.max_pages = P.max_pages;
    A.pk.out = P.out;
    A.rope = P.rope;

    const uint64_t heads = static_cast<uint64_t>(P.H + 2 * P.Hkv), N = P.N;
    CUtensorMap tm_q, tm_k, tm_v, tm_krot, tm_out;
    std::memset(&tm_krot, 0, sizeof(tm_krot));
    {
        // qkv as [1][N][heads][256]
        const uint64_t dims[4] = {kHeadDim, heads, N, 1};
        const uint64_t strides[3] = {kHeadDim * 2ull, heads * kHeadDim * 2ull,
                                     N * heads * kHeadDim * 2ull};
        const uint32_t box_q[4] = {64, static_cast<uint32_t>(P.G), static_cast<uint32_t>(tq), 1};
        const uint32_t box_k[4] = {64, 1, 128, 1}, box_v[4] = {64, 1, 64, 1};
        if (!encode_bf16_map(&tm_q, P.qkv, 4, dims, strides, box_q)) return SPARK_ERR_CUDA;
        if (!paged && (!encode_bf16_map(&tm_k, P.qkv, 4, dims, strides, box_k) ||
                       !encode_bf16_map(&tm_v, P.qkv, 4, dims, strides, box_v)))
            return SPARK_ERR_CUDA;
    }
    if (paged) {
        // the pool as groups of 8 slots, [groups][4 chunks of 64 dims][8 slots][64]:
        // a box of a few whole groups, which never leaves its page
        const uint64_t page = 1ull << P.page_shift;
        const uint64_t dims[4] = {64, 8, kHeadDim / 64,
                                  static_cast<uint64_t>(P.n_pages) * P.Hkv * page / 8};
        const uint64_t strides[3] = {kHeadDim * 2ull, 128, 8 * kHeadDim * 2ull};
        const uint32_t box_k[4] = {64, 8, 2, static_cast<uint32_t>(page < 64 ? page : 64) / 8};
        const uint32_t box_v[4] = {64, 8, 4, static_cast<uint32_t>(page < 32 ? page : 32) / 8};
        if (!encode_bf16_map(&tm_k, P.k_pages, 4, dims, strides, box_k) ||
            !encode_bf16_map(&tm_v, P.v_pages, 4, dims, strides, box_v))
            return SPARK_ERR_CUDA;
    } else if (pl.rot_w > 0) {
        const uint64_t dims[3] = {static_cast<uint64_t>(pl.rot_w), N,
                                  static_cast<uint64_t>(P.Hkv)};
        const uint64_t strides[2] = {pl.rot_w * 2ull, N * pl.rot_w * 2ull};
        const uint32_t box[3] = {64, 128, 1};
        if (!encode_bf16_map(&tm_krot, P.krot, 3, dims, strides, box)) return SPARK_ERR_CUDA;
    }
    {
        // out as [1][N][H][256]
        const uint64_t H = P.H;
        const uint64_t dims[4] = {kHeadDim, H, N, 1};
        const uint64_t strides[3] = {kHeadDim * 2ull, H * kHeadDim * 2ull, N * H * kHeadDim * 2ull};
        const uint32_t box[4] = {64, static_cast<uint32_t>(P.G), static_cast<uint32_t>(tq), 1};
        if (!encode_bf16_map(&tm_out, P.out, 4, dims, strides, box)) return SPARK_ERR_CUDA;
    }
    return done(launch_prefill_packed(tm_q, tm_k, tm_v, tm_krot, tm_out, A, pl.most, stream));
}

// Workspace of a paged decode: the header (status word, then a byte per CTA
// that counts the finished parts of a shared pair), two partial states per CTA.
struct DecodePagedPlan {
    int grid;
    size_t ml, o, bytes;
};

DecodePagedPlan plan_decode_paged(int H, int Hkv, int sms) {
    DecodePagedPlan pl{};
    constexpr int most = static_cast<int>(kWorkspaceHeader) - 4;
    pl.grid = sms < most ? sms : most;
    const size_t parts = static_cast<size_t>(pl.grid) * 2 * (H / Hkv);
    pl.ml = kWorkspaceHeader;
    pl.o = pl.ml + up256(parts * 2 * 4);
    pl.bytes = pl.o + up256(parts * kHeadDim * 4);
    return pl;
}

spark_status prefill_paged_impl(const void *qkv, const float *gate, const int32_t *pos,
                                const int32_t *cu, const int32_t *start, void *k_pages,
                                void *v_pages, int n_pages, int page_size, const int32_t *table,
                                int max_pages, const spark_layer_desc *desc, int N, int S, int H,
                                int Hkv, void *out, void *workspace, size_t workspace_bytes,
                                void *stream, bool paged) {
    spark_status st = check_packed(N, S, H, Hkv, desc);
    if (st != SPARK_OK) return st;
    if (N == 0 || S == 0) return SPARK_OK;
    if (!qkv || !gate || !pos || !cu || !out || !workspace || (paged && !start))
        return SPARK_ERR_NULL;
    if (!aligned(qkv, 16) || !aligned(out, 16) || !aligned(gate, 4) || !aligned(pos, 4) ||
        !aligned(cu, 4) || !aligned(start, 4) || !aligned(workspace, 256))
        return SPARK_ERR_ALIGN;
    if (paged) {
        st = check_pages(k_pages, v_pages, n_pages, page_size, table, max_pages);
        if (st != SPARK_OK) return st;
        // a box's coordinate counts groups of 8 slots (8.8 TB of them)
        if ((n_pages + 1ll) * Hkv * (page_size / 8) > 0x7fffffffLL) return SPARK_ERR_UNSUPPORTED;
    }
    int sms;
    st = device_ready(&sms);
    const PackedPlan pl = plan_packed(N, S, H, Hkv, desc, paged, sms);
    if (workspace_bytes < pl.bytes) return SPARK_ERR_WORKSPACE;
    if (pl.most * Hkv > 0x7fffffffLL) return SPARK_ERR_UNSUPPORTED;  // the grid
    if (st != SPARK_OK) return st;
    PagedParams P = make_params(qkv, gate, pos, desc, N, S, H, Hkv, out, workspace);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    P.cu = cu;
    P.krot = reinterpret_cast<__nv_bfloat16 *>(ws + pl.krot);
    P.rot_w = pl.rot_w;
    P.tile_base = reinterpret_cast<int32_t *>(ws + pl.base);
    P.work = reinterpret_cast<PackedItem *>(ws + pl.work);
    P.most = static_cast<int>(pl.most);
    P.sms = sms;
    P.slots = pl.slots;
    P.part_ml = reinterpret_cast<float *>(ws + pl.ml);
    P.part_o = reinterpret_cast<float *>(ws + pl.o);
    P.call = reinterpret_cast<unsigned *>(ws + pl.flags);
    P.odd_values = P.call + 1;
    P.n_splits = reinterpret_cast<int *>(P.call) + 3;
    P.splits = reinterpret_cast<PackedItem *>(ws + pl.splits);
    if (paged) {
        P.start = start;
        set_pages(P, k_pages, v_pages, n_pages, page_size, table, max_pages);
    }
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    st = launch_prep(P, cs);
    if (st != SPARK_OK) return st;
    return launch_packed_attn(P, pl, sms, cs);
}

}  // namespace
}  // namespace spark

using namespace spark;

extern "C" {

size_t spark_attn_prefill_packed_workspace_size(int n_tokens, int S, int H, int Hkv,
                                                const spark_layer_desc *desc) {
    if (check_packed(n_tokens, S, H, Hkv, desc) != SPARK_OK) return 0;
    return packed_workspace(n_tokens, S, H, Hkv, desc, false);
}

spark_status spark_attn_prefill_packed(const void *qkv, const float *gate, const int32_t *pos,
                                       const int32_t *cu_seqlens, const spark_layer_desc *desc,
                                       int n_tokens, int S, int H, int Hkv, void *out,
                                       void *workspace, size_t workspace_bytes, void *stream) {
    return prefill_paged_impl(qkv, gate, pos, cu_seqlens, nullptr, nullptr, nullptr, 0, 0, nullptr,
                              0, desc, n_tokens, S, H, Hkv, out, workspace, workspace_bytes,
                              stream, false);
}

size_t spark_attn_prefill_paged_workspace_size(int n_tokens, int S, int H, int Hkv,
                                               const spark_layer_desc *desc) {
    if (check_packed(n_tokens, S, H, Hkv, desc) != SPARK_OK) return 0;
    return packed_workspace(n_tokens, S, H, Hkv, desc, true);
}

spark_status spark_attn_prefill_paged(const void *qkv, const float *gate, const int32_t *pos,
                                      const int32_t *cu_seqlens, const int32_t *start,
                                      void *k_pages, void *v_pages, int n_pages, int page_size,
                                      const int32_t *page_table, int max_pages,
                                      const spark_layer_desc *desc, int n_tokens, int S, int H,
                                      int Hkv, void *out, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    return prefill_paged_impl(qkv, gate, pos, cu_seqlens, start, k_pages, v_pages, n_pages,
                              page_size, page_table, max_pages, desc, n_tokens, S, H, Hkv, out,
                              workspace, workspace_bytes, stream, true);
}

size_t spark_attn_decode_paged_workspace_size(int B, int H, int Hkv, const spark_layer_desc *desc) {
    if (check_layer_desc(desc, H, Hkv) != SPARK_OK || B < 0) return 0;
    int sms;
    device_ready(&sms);
    return plan_decode_paged(H, Hkv, sms).bytes;
}

spark_status spark_attn_decode_paged(const void *qkv, const float *gate, const int32_t *pos,
                                     void *k_pages, void *v_pages, int n_pages, int page_size,
                                     const int32_t *page_table, int max_pages,
                                     const spark_layer_desc *desc, int B, int H, int Hkv,
                                     void *out, void *workspace, size_t workspace_bytes,
                                     void *stream) {
    spark_status st = check_layer_desc(desc, H, Hkv);
    if (st != SPARK_OK) return st;
    if (B < 0) return SPARK_ERR_SHAPE;
    if (B == 0) return SPARK_OK;
    if (!qkv || !gate || !pos || !out || !workspace) return SPARK_ERR_NULL;
    if (!aligned(qkv, 16) || !aligned(out, 16) || !aligned(gate, 4) || !aligned(pos, 4) ||
        !aligned(workspace, 256))
        return SPARK_ERR_ALIGN;
    st = check_pages(k_pages, v_pages, n_pages, page_size, page_table, max_pages);
    if (st != SPARK_OK) return st;
    int sms;
    const spark_status ready = device_ready(&sms);
    const DecodePagedPlan pl = plan_decode_paged(H, Hkv, sms);
    if (workspace_bytes < pl.bytes) return SPARK_ERR_WORKSPACE;
    if (ready != SPARK_OK) return ready;
    PagedParams P = make_params(qkv, gate, pos, desc, B, B, H, Hkv, out, workspace);
    set_pages(P, k_pages, v_pages, n_pages, page_size, page_table, max_pages);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    P.pos_end = max_pages << P.page_shift;
    if (P.rope.rot_dim > 0 && P.pos_end > kRopePositions) P.pos_end = kRopePositions;
    P.counters = reinterpret_cast<unsigned *>(ws) + 1;
    P.part_ml = reinterpret_cast<float *>(ws + pl.ml);
    P.part_o = reinterpret_cast<float *>(ws + pl.o);
    // the pool as [n_pages][Hkv][page][256]; boxes of a page's share of a tile
    const uint64_t page = static_cast<uint64_t>(page_size);
    const uint64_t dims[4] = {kHeadDim, page, static_cast<uint64_t>(Hkv),
                              static_cast<uint64_t>(n_pages)};
    const uint64_t strides[3] = {kHeadDim * 2ull, page * kHeadDim * 2ull,
                                 Hkv * page * kHeadDim * 2ull};
    const uint32_t box[4] = {64, static_cast<uint32_t>(page < 64 ? page : 64), 1, 1};
    CUtensorMap tm_k, tm_v;
    if (!encode_bf16_map(&tm_k, k_pages, 4, dims, strides, box) ||
        !encode_bf16_map(&tm_v, v_pages, 4, dims, strides, box))
        return SPARK_ERR_CUDA;
    return done(launch_decode_paged(tm_k, tm_v, P, pl.grid, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
