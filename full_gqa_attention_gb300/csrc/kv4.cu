// kv4.cu -- a cache in 4 bits: tokens quantised as they are stored, and read
// back, and the host side of the calls on such a cache (format: kv4.cuh).
//
//   store  reads the K and V columns of the projections (1024 bytes per token
//          and KV head), writes 288.  Its instructions bound it, some 220 a key's
//          row and warp, 80 a value's, and their latency: 16 warps per SM issue 2.3
//          of 4 a cycle, no pipe is busy more than 54 % of the time
//   load   reads 288, writes 1024: HBM bounds it
//
// Both walk the groups of 16 slots that the call touches.  The groups of all
// rows behind one another are a list, which the CTAs share out evenly.  A lane
// has 8 dims of a key's or value's row.
#include <cmath>
#include <cstring>

#include "kv4.cuh"
#include "spark_attn.h"

namespace spark {

void fill_rope_table(const spark_layer_desc *d, RopeTable *t);
spark_status device_ready(int *sms);
spark_status check_layer_desc(const spark_layer_desc *d, int H, int Hkv);
bool aligned(const void *p, size_t a);
int page_shift_of(int page_size);
spark_status check_pages(const void *k_pages, const void *v_pages, int n_pages, int page_size,
                         const int32_t *table, int max_pages);
int decode_kv4_ctas(int sms, int G);
cudaError_t launch_decode_kv4(const Kv4Params &P, int grid, cudaStream_t stream);

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// A CTA's stretch [u, end) of a list of units, row behind row, and the row that
// unit u belongs to (whose first unit is base).
struct Stretch {
    long long u, end, base;
    int r;
};

// units(r, report): units of row r; report: the one place to note a fault of it.
// False where nothing is left for this CTA.  All threads.
template <int kThreads, typename Units>
__device__ __forceinline__ bool stretch_of(int S, Units &&units, Stretch &st) {
    constexpr int kWarps = kThreads / 32;
    __shared__ long long sums[kWarps];
    __shared__ long long s_base;
    __shared__ int s_row;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (S + kThreads - 1) / kThreads;
    const int r0 = tid * per;
    long long mine = 0;
    for (int r = r0; r < r0 + per && r < S; ++r) mine += units(r, blockIdx.x == 0);
    long long before = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before += y;
    }
    if (lane == 31) sums[warp] = before;
    before -= mine;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    const long long share = (total + gridDim.x - 1) / gridDim.x;
    st.u = share * blockIdx.x;
    st.end = st.u + share < total ? st.u + share : total;
    if (st.u >= st.end) return false;
    if (st.u >= before && st.u < before + mine) {
        int r = r0;
        long long base = before;
        for (; r + 1 < S; ++r) {
            const long long n = units(r, false);
            if (st.u < base + n) break;
            base += n;
        }
        s_row = r;
        s_base = base;
    }
    __syncthreads();
    st.r = s_row;
    st.base = s_base;
    return true;
}

// Groups of 16 slots that tokens [a, b) touch.
__device__ __forceinline__ int groups_of(int a, int b) {
    return a < b ? ((b + kKv4Group - 1) >> 4) - (a >> 4) : 0;
}

// ---------------------------------------------------------------- store

// Tokens of sequence r: [a, b) of its slots, its first packed row.
struct StoreRow {
    int a, b, row;
};

__device__ __forceinline__ StoreRow store_row(const Kv4Params &P, int r, bool report) {
    StoreRow s{0, 0, 0};
    const int c0 = P.cu[r], c1 = P.cu[r + 1];
    if (c0 < 0 || c1 < c0 || c1 > P.N) {
        if (report) atomicOr(P.status, kErrSeqlens);
        return s;
    }
    if (c1 == c0) return s;
    const int start = P.begin[r];
    const int slots = P.pg.max_pages << P.pg.page_shift;
    if (start < 0 || start > slots - (c1 - c0)) {
        if (report) atomicOr(P.status, kErrPosition);
        return s;
    }
    return StoreRow{start, start + (c1 - c0), c0};
}

// Four words and one that other threads may be writing.
__device__ __forceinline__ void load_relaxed(const uint32_t *four, const uint32_t *one,
                                             uint32_t (&x)[5]) {
    asm volatile("ld.relaxed.gpu.global.v4.b32 {%0, %1, %2, %3}, [%5];\n\t"
                 "ld.relaxed.gpu.global.b32 %4, [%6];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4])
                 : "l"(four), "l"(one)
                 : "memory");
}

// Cosines and sines of a token, as the lanes read them: pairs 8 l + 2 i and the
// next one are the 16 bytes i of lane l.
__device__ __forceinline__ int angle_at(int k) {
    return (k >> 1 & 3) * 32 + (k >> 3) * 2 + (k & 1);  // in float2
}

// One CTA per SM, of 16 warps: a warp takes one of a unit's 16 tokens' keys, of one
// KV head after another with the same angles, and 4 tokens of one KV head's
// values.  The next unit's projections come by bulk copies meanwhile, and its
// angles are written before a unit's keys are: a warp that is late (some rows take
// more arithmetic) may be behind the others by nearly a unit.
//
// 34,200 tokens of 4 KV heads that rotate all dims: 72 us, 2.5 TB/s (0.37 of a
// copy); reading and the angles alone 34, values alone 44, keys alone 64.  Two
// CTAs of 256 threads that load for themselves took 88; 24 or 32 warps, of which
// some take the values, 101 and 132 (80 and 64 registers: spills); units of 2 KV
// heads 101; two keys' rows at a time the same, with more registers.
constexpr int kStoreThreads = 512;
constexpr int kStoreHeads = 4;                                   // of a unit, at most
constexpr int kStoreRow = kStoreHeads * kHeadDim * 2;            // a token's keys, or values
constexpr int kStoreStage = 2 * kKv4Group * kStoreRow;
constexpr int kAngles = kKv4Group * kMaxRopePairs;               // of 16 tokens
constexpr int kAngleSets = 3;
constexpr int kStoreSmem = 2 * kStoreStage + (kAngleSets + 1) * kAngles * 8;

struct StoreUnit {
    int r, slot0, h0, heads;
    int t_lo, t_hi;            // the call's slots of the group
    int first;                 // packed row of slot 0 of the group
    int id;                    // its page
};

// kAll: all 256 dims turn.
template <bool kAll>
__global__ void __launch_bounds__(kStoreThreads, 1)
    kv4_store_kernel(const __grid_constant__ Kv4Params P) {
    extern __shared__ __align__(128) uint8_t smem[];             // two stages: keys, values
    float2 *angles = reinterpret_cast<float2 *>(smem + 2 * kStoreStage);  // of three units
    float2 *steps = angles + kAngleSets * kAngles;               // of 0 .. 15 positions
    __shared__ uint64_t full[2];     // a stage's rows are there
    __shared__ uint64_t turned;      // a unit's angles are
    __shared__ uint64_t emptied[2];  // all warps have read a stage's rows
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int half = P.rope.rot_dim / 2;
    // This thread's pair, and the first of its tokens.
    const int together = half ? kStoreThreads / half : 1;     // tokens the threads take at once
    const int k = half ? tid % half : 0;
    const int t_mine = half && tid < together * half ? tid / half : kKv4Group;
    float2 freq = make_float2(0.f, 0.f);
    if (half) freq = P.rope.u[k];
    if (tid == 0) {
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        mbar_init(&turned, kStoreThreads / 32);
        mbar_init(&emptied[0], kStoreThreads / 32);
        mbar_init(&emptied[1], kStoreThreads / 32);
        fence_mbar_init();
        abort_flag = 0;
    }
    grid_dep_wait();
    grid_dep_launch();
    const int parts = (P.Hkv + kStoreHeads - 1) / kStoreHeads;
    auto units = [&](int r, bool report) {
        const StoreRow s = store_row(P, r, report);
        return static_cast<long long>(groups_of(s.a, s.b)) * parts;
    };
    Stretch st;
    if (!stretch_of<kStoreThreads>(P.S, units, st)) return;
    // Consecutive positions, as nearly always: a group's turns are its first
    // token's and those of 0 .. 15 positions together, 8 instructions for some 70.
    const bool stepwise = st.end - st.u > 2;
    if (stepwise) {
#pragma unroll 1
        for (int t = t_mine; t < kKv4Group; t += together) {
            float2 c;
            rope_cos_sin_fine(t, freq, c.x, c.y);
            steps[t * kMaxRopePairs + k] = c;
        }
        __syncthreads();
    }
    StoreRow row = store_row(P, st.r, false);
    // Unit u, at or behind the one located last; false where there is none, or the
    // offsets changed under the call.
    auto locate = [&](long long u, StoreUnit &unit) {
        if (u >= st.end) return false;
        for (;;) {
            const long long n = static_cast<long long>(groups_of(row.a, row.b)) * parts;
            if (u < st.base + n) break;
            st.base += n;
            if (++st.r >= P.S) return false;
            row = store_row(P, st.r, false);
        }
        const int at = static_cast<int>(u - st.base);
        unit.r = st.r;
        unit.slot0 = ((row.a >> 4) + at / parts) << 4;
        unit.h0 = at % parts * kStoreHeads;
        unit.heads = P.Hkv - unit.h0 < kStoreHeads ? P.Hkv - unit.h0 : kStoreHeads;
        unit.t_lo = row.a > unit.slot0 ? row.a - unit.slot0 : 0;
        unit.t_hi = row.b - unit.slot0 < kKv4Group ? row.b - unit.slot0 : kKv4Group;
        unit.first = row.row + (unit.slot0 - row.a);
        unit.id = P.pg.table[static_cast<size_t>(st.r) * P.pg.max_pages +
                             (unit.slot0 >> P.pg.page_shift)];
        return true;
    };
    const ptrdiff_t width = static_cast<ptrdiff_t>(P.H + 2 * P.Hkv) * kHeadDim;
    // (one warp: lanes 0 .. 15 the tokens' keys, the others their values)
    auto fetch = [&](const StoreUnit &unit, int s) {
        const int t = lane & 15, value = lane >> 4, bytes = unit.heads * kHeadDim * 2;
        if (lane == 0)
            mbar_arrive_expect_tx(&full[s], 2 * (unit.t_hi - unit.t_lo) * bytes);
        __syncwarp();
        if (t >= unit.t_lo && t < unit.t_hi)
            bulk_load(smem + s * kStoreStage + lane * kStoreRow,
                      P.qkv + (unit.first + t) * width +
                          static_cast<ptrdiff_t>(P.H + value * P.Hkv + unit.h0) * kHeadDim,
                      bytes, &full[s]);
    };
    const int turning = P.rope.rot_dim >> 4;                     // lanes of each half of a turn
    const int lane_pairs = lane < turning ? lane : lane < 2 * turning ? lane - turning : 0;
    // The position of this lane's token of a unit: every warp looks at all of them.
    auto token_of = [&](const StoreUnit &unit) {
        return lane < unit.t_lo ? unit.t_lo : lane < unit.t_hi ? lane : unit.t_hi - 1;
    };
    auto position = [&](const StoreUnit &unit) {
        return half ? P.pos[unit.first + token_of(unit)] : 0;
    };
    // Writes unit n's angles.
    auto turn = [&](const StoreUnit &unit, int n, int my_pos) {
        float2 *turns = angles + n % kAngleSets * kAngles;
        const int t_lo = unit.t_lo, t_hi = unit.t_hi, my_t = token_of(unit);
        const int pos_lo = __shfl_sync(0xffffffffu, my_pos, t_lo);
        if (stepwise && __all_sync(0xffffffffu, my_pos == pos_lo + (my_t - t_lo))) {
            float2 c;
            rope_cos_sin_fine(pos_lo, freq, c.x, c.y);
            for (int t = t_lo + t_mine; t < t_hi; t += together) {
                const float2 d = steps[(t - t_lo) * kMaxRopePairs + k];
                turns[t * kMaxRopePairs + angle_at(k)] =
                    make_float2(fmaf(c.x, d.x, -c.y * d.y), fmaf(c.y, d.x, c.x * d.y));
            }
        } else {
#pragma unroll 1
            for (int t = t_lo + t_mine; t < t_hi; t += together) {
                float2 c;
                rope_cos_sin_fine(P.pos[unit.first + t], freq, c.x, c.y);
                turns[t * kMaxRopePairs + angle_at(k)] = c;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&turned);
    };
    StoreUnit next;
    bool more = locate(st.u, next);
    int next_pos = 0, fetched = 0;
    bool alive = true;  // no wait has run out
    if (more) {
        if (warp == 0) fetch(next, fetched++);
        next_pos = position(next);
        turn(next, 0, next_pos);
    }
    for (int n = 0; more; ++n) {
        const StoreUnit unit = next;
        const int s = n & 1, t_lo = unit.t_lo, t_hi = unit.t_hi, my_pos = next_pos;
        const float2 *turns = angles + n % kAngleSets * kAngles;
        more = locate(st.u + n + 1, next);
        if (more) next_pos = position(next);
        alive = alive && mbar_wait_short(&turned, n & 1, &abort_flag, P.status) &&
                mbar_wait_short(&full[s], n >> 1 & 1, &abort_flag, P.status);
        alive = __all_sync(0xffffffffu, alive);
        // In the middle of a unit: the next one's angles (all warps have said that unit
        // n's are there, so that unit n - 2's, whose place these take, are done with) and
        // its rows, into the stage that unit n - 1's have left.
        auto prepare = [&]() {
            if (!more) return;
            turn(next, n + 1, next_pos);
            if (warp != 0) return;
            if (n > 0)
                alive = alive && mbar_wait_short(&emptied[s ^ 1], (n - 1) >> 1 & 1, &abort_flag,
                                                 P.status);
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) return;
            fetch(next, s ^ 1);
            ++fetched;
        };
        // At its end.  (A warp that says so of unit n + 2 has seen that all began unit
        // n + 1: each phase counts every warp once.)
        auto leave = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&emptied[s]);
        };
        if (!alive || unit.id < 0 || unit.id >= P.pg.n_pages) {
            if (tid == 0 && alive) atomicOr(P.status, kErrPage);
            prepare();
            leave();
            continue;
        }
        const uint8_t *keys = smem + s * kStoreStage, *values = keys + kKv4Group * kStoreRow;
        const size_t head_bytes = static_cast<size_t>(kKv4GroupBytes) << (P.pg.page_shift - 4);
        const size_t group0 = P.pg.group(unit.id, unit.h0, P.Hkv, unit.slot0);
        if (warp < unit.heads * 4) {
            const int h = warp >> 2, quad = warp & 3;
            uint32_t codes[4];
            unsigned scales = 0, keep = 0;  // keep: of the group's slots, as masks
            uint32_t mask = 0;
            uint4 raw[4];
            unsigned byte[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)  // (rows beside the call's hold anything and are masked)
                raw[j] = *reinterpret_cast<const uint4 *>(values + (4 * quad + j) * kStoreRow +
                                                          h * (kHeadDim * 2) + lane * 16);
            kv4_value_rows(raw, codes, byte);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * quad + j;
                scales |= byte[j] << (8 * (2 * (j & 1) + (j >> 1)));
                if (t < t_lo || t >= t_hi) {
                    keep |= 0xffu << (8 * (2 * (j & 1) + (j >> 1)));
                    mask |= (j & 1 ? 0xf0f0u : 0x0f0fu) << (16 * (j >> 1));
                }
            }
            if (mask != 0xffffffffu) {
                // dims 2 i, 2 i + 1 of slots 0 and 1, then of 2 and 3
                uint32_t e[2], o[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t a = codes[2 * q], b = codes[2 * q + 1];
                    e[q] = (a & 0x0f0f0f0fu) | (b & 0x0f0f0f0fu) << 4;
                    o[q] = (a >> 4 & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
                }
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = __byte_perm(e[0], o[0], i | (i + 4) << 4);
                    const uint32_t hi = __byte_perm(e[1], o[1], i | (i + 4) << 4);
                    w[i] = __byte_perm(lo, hi, 0x5410);
                }
                uint8_t *group = P.pg.v + group0 + h * head_bytes;
                uint32_t *dst = reinterpret_cast<uint32_t *>(group + kv4_value_at(lane, quad));
                uint32_t *sdst =
                    reinterpret_cast<uint32_t *>(group + kv4_value_scale_at(lane >> 1, quad));
                if (!mask) {
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                    if (!(lane & 1)) *sdst = scales;
                } else {
                    // Slots beside the call's keep what they hold, and other sequences of the
                    // call may be writing there (a row stored as several chunks): only the bits
                    // of this one's slots, which nobody else changes, are turned over.
                    uint32_t old[5];
                    load_relaxed(dst, sdst, old);
#pragma unroll
                    for (int i = 0; i < 4; ++i) atomicXor(dst + i, (old[i] ^ w[i]) & ~mask);
                    if (!(lane & 1)) atomicXor(sdst, (old[4] ^ scales) & ~keep);
                }
            }
        }
        prepare();
        const int t = warp;
        if (t < t_lo || t >= t_hi) {
            leave();
            continue;
        }
        const int p = __shfl_sync(0xffffffffu, my_pos, t);
        float c[8], sn[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 a =
                *reinterpret_cast<const float4 *>(turns + t * kMaxRopePairs + i * 32 + lane_pairs * 2);
            c[2 * i] = a.x, sn[2 * i] = a.y, c[2 * i + 1] = a.z, sn[2 * i + 1] = a.w;
        }
        if (!kAll && lane >= 2 * turning)
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = 1.f, sn[i] = 0.f;
        const KeyTurn turn_of = kv4_key_turn(P.rope.rot_dim, p, lane);
        const uint8_t *key = keys + t * kStoreRow;
        uint8_t *group = P.pg.k + group0;
#pragma unroll 1
        for (int h = 0; h < unit.heads; ++h, key += kHeadDim * 2, group += head_bytes) {
            float y[8];
            uint32_t codes;
            unsigned byte;
            kv4_rotate(turn_of, key, lane, c, sn, y);
            if (kAll && p != 0)
                kv4_key_row<true>(turn_of, key, lane, y, p, P.turns, codes, byte);
            else
                kv4_key_row<false>(turn_of, key, lane, y, p, P.turns, codes, byte);
            *reinterpret_cast<uint32_t *>(group + kv4_key_at(lane, t)) = codes;
            if (!(lane & 1)) group[kv4_key_scale_at(lane >> 1, t)] = static_cast<uint8_t>(byte);
        }
        leave();
    }
    // copies that were waited for in vain must land before the CTA ends
    if (warp == 0 && *static_cast<volatile int *>(&abort_flag))
        for (int i = fetched > 2 ? fetched - 2 : 0; i < fetched; ++i)
            mbar_wait_plain_short(&full[i & 1], i >> 1 & 1);
}

// ---------------------------------------------------------------- load

struct LoadRow {
    int a, b;
};

__device__ __forceinline__ LoadRow load_row(const Kv4LoadParams &P, int r, bool report) {
    const int a = P.begin[r], b = P.end[r];
    if (a == b) return LoadRow{0, 0};
    const int from = P.pg.max_pages << P.pg.page_shift, to = P.to_max_pages << P.to_page_shift;
    if (a < 0 || b < a || b > from || b > to) {
        if (report) atomicOr(P.status, kErrPosition);
        return LoadRow{0, 0};
    }
    return LoadRow{a, b};
}

// Codes of dims 8 l .. and their scale as 8 bf16 (exact).
__device__ __forceinline__ uint4 kv4_to_bf16(uint32_t codes, unsigned byte) {
    uint32_t h[4], w[4];
    kv4_widen(codes, h);
    const float s = kv4_scale(byte);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        w[i] = pack_bf16x2(f.x * s, f.y * s);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp takes 4 slots of a KV head's keys or values.  53,900 tokens of 4 KV heads:
// 52 us, 5.4 TB/s, of which 4.2 are writes (a fill writes 4.0).  Six or eight CTAs
// per SM instead of four, and shares by KV head, are no faster.
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const __grid_constant__ Kv4LoadParams P) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_wait();
    grid_dep_launch();
    auto units = [&](int r, bool report) {
        const LoadRow s = load_row(P, r, report);
        return static_cast<long long>(groups_of(s.a, s.b));
    };
    Stretch st;
    if (!stretch_of<kThreads>(P.S, units, st)) return;
    LoadRow row = load_row(P, st.r, false);
    for (; st.u < st.end; ++st.u) {
        while (st.u >= st.base + groups_of(row.a, row.b)) {
            st.base += groups_of(row.a, row.b);
            if (++st.r >= P.S) return;  // the ranges changed under the call
            row = load_row(P, st.r, false);
        }
        const int slot0 = ((row.a >> 4) + static_cast<int>(st.u - st.base)) << 4;
        const int t_lo = row.a > slot0 ? row.a - slot0 : 0;
        const int t_hi = row.b - slot0 < kKv4Group ? row.b - slot0 : kKv4Group;
        const int id = P.pg.table[static_cast<size_t>(st.r) * P.pg.max_pages +
                                  (slot0 >> P.pg.page_shift)];
        const int to = P.to_table[static_cast<size_t>(st.r) * P.to_max_pages +
                                  (slot0 >> P.to_page_shift)];
        const bool held = id >= 0 && id < P.pg.n_pages;
        if (!held || to < 0 || to >= P.to_n_pages) {
            if (tid == 0) atomicOr(P.status, kErrPage);
            if (to < 0 || to >= P.to_n_pages) continue;
        }
        for (int task = warp; task < P.Hkv * 8; task += kWarps) {
            const int h = task >> 3, quad = task & 3;
            const bool key = !(task & 4);
            uint32_t codes[4] = {0, 0, 0, 0};
            unsigned bytes = 0;  // of slots 4 quad .., in order
            if (held) {
                const uint8_t *group = (key ? P.pg.k : P.pg.v) + P.pg.group(id, h, P.Hkv, slot0);
                if (key) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = 4 * quad + j;
                        codes[j] = __ldcs(
                            reinterpret_cast<const uint32_t *>(group + kv4_key_at(lane, t)));
                        bytes |= static_cast<unsigned>(
                                     __ldcs(group + kv4_key_scale_at(lane >> 1, t)))
                                 << (8 * j);
                    }
                } else {
                    const uint4 w =
                        __ldcs(reinterpret_cast<const uint4 *>(group + kv4_value_at(lane, quad)));
                    bytes = __byte_perm(__ldcs(reinterpret_cast<const unsigned *>(
                                            group + kv4_value_scale_at(lane >> 1, quad))),
                                        0, 0x3120);
#pragma unroll
                    for (int j = 0; j < 4; ++j) codes[j] = kv4_value_codes(w, j);
                }
            }
            __nv_bfloat16 *dst =
                (key ? P.k_pages : P.v_pages) +
                (((static_cast<size_t>(to) * P.Hkv + h) << P.to_page_shift) +
                 (slot0 & ((1 << P.to_page_shift) - 1))) * kHeadDim + lane * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * quad + j;
                if (t >= t_lo && t < t_hi)
                    *reinterpret_cast<uint4 *>(dst + t * kHeadDim) =
                        kv4_to_bf16(codes[j], bytes >> (8 * j) & 255u);
            }
        }
    }
}

// ---------------------------------------------------------------- host side

spark_status done(cudaError_t e) {
    if (e == cudaSuccess) return SPARK_OK;
    cudaGetLastError();
    return SPARK_ERR_CUDA;
}

// The turns of a layer's pairs, in two floats and in units of 2^-64 turns.  A model has a few
// kinds of layers and 128 powers take longer than a launch: each thread keeps the
// last four kinds' (by base and width, nothing else goes into them).
struct LayerTurns {
    double theta = 0.0;
    int rot_dim = -1;
    RopeTable rope;
    unsigned long long turns[kMaxRopePairs];
};

const LayerTurns &turns_of(const spark_layer_desc *desc) {
    constexpr int kKinds = 4;
    static thread_local LayerTurns kept[kKinds];
    static thread_local int oldest = 0;
    for (const LayerTurns &t : kept)
        if (t.rot_dim == desc->rot_dim && t.theta == desc->rope_theta) return t;
    LayerTurns &t = kept[oldest];
    oldest = (oldest + 1) % kKinds;
    t.theta = desc->rope_theta;
    t.rot_dim = desc->rot_dim;
    fill_rope_table(desc, &t.rope);
    std::memset(t.turns, 0, sizeof(t.turns));
    const double two_pi = 6.283185307179586476925286766559;
    for (int k = 0; k < desc->rot_dim / 2; ++k) {
        double u = std::pow(desc->rope_theta, -2.0 * k / desc->rot_dim) / two_pi;
        if (!(u <= 0.5)) {
            // (a base below 1: whole turns per position leave no trace)
            u = std::isfinite(u) ? u - std::rint(u) : 0.0;
            const float hi = static_cast<float>(u);
            t.rope.u[k] = make_float2(hi, static_cast<float>(u - hi));
        }
        t.turns[k] = static_cast<unsigned long long>(std::ldexp(u - std::floor(u), 64));
    }
    return t;
}

void set_layer(Kv4Params &P, const spark_layer_desc *desc, int H, int Hkv) {
    P.H = H;
    P.Hkv = Hkv;
    P.G = H / Hkv;
    P.kind = desc->kind;
    constexpr int kMostWindow = 1 << 30;  // (positions stay below it)
    P.window = desc->kind != SPARK_LAYER_SLIDING ? 0
               : desc->window < kMostWindow     ? desc->window
                                                : kMostWindow;
    P.gate_mode = desc->gate_mode;
    const LayerTurns &t = turns_of(desc);
    P.rope = t.rope;
    std::memcpy(P.turns, t.turns, sizeof(P.turns));
}

Kv4Pages pages_of(void *k4, void *v4, int n_pages, int page_size, const int32_t *table,
                  int max_pages) {
    Kv4Pages pg;
    pg.k = static_cast<uint8_t *>(k4);
    pg.v = static_cast<uint8_t *>(v4);
    pg.table = table;
    pg.n_pages = n_pages;
    pg.page_shift = page_shift_of(page_size);
    pg.max_pages = max_pages;
    return pg;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace of a decode: the header (status word, counts of states left, which every
// call leaves at 0); two partial states per CTA.
struct DecodeKv4Plan {
    int grid;
    size_t ml, o, bytes;
};

DecodeKv4Plan plan_decode_kv4(int H, int Hkv, int sms) {
    DecodeKv4Plan pl{};
    pl.grid = decode_kv4_ctas(sms, H / Hkv);
    const size_t parts = static_cast<size_t>(pl.grid) * 2 * (H / Hkv);
    pl.ml = kWorkspaceHeader;
    pl.o = pl.ml + up256(parts * 2 * 4);
    pl.bytes = pl.o + up256(parts * kHeadDim * 4);
    return pl;
}

}  // namespace
}  // namespace spark

using namespace spark;

extern "C" {

size_t spark_attn_kv4_store_workspace_size(int n_tokens, int S, int H, int Hkv,
                                           const spark_layer_desc *desc) {
    if (check_layer_desc(desc, H, Hkv) != SPARK_OK || n_tokens < 0 || S < 0) return 0;
    return kWorkspaceHeader;
}

spark_status spark_attn_kv4_store(const void *qkv, const int32_t *pos, const int32_t *cu_seqlens,
                                  const int32_t *start, void *k4_pages, void *v4_pages, int n_pages,
                                  int page_size, const int32_t *page_table, int max_pages,
                                  const spark_layer_desc *desc, int n_tokens, int S, int H,
                                  int Hkv, void *workspace, size_t workspace_bytes, void *stream) {
    spark_status st = check_layer_desc(desc, H, Hkv);
    if (st != SPARK_OK) return st;
    if (n_tokens < 0 || S < 0) return SPARK_ERR_SHAPE;
    if (n_tokens == 0 || S == 0) return SPARK_OK;
    if (!qkv || !pos || !cu_seqlens || !start || !workspace) return SPARK_ERR_NULL;
    if (!aligned(qkv, 16) || !aligned(pos, 4) || !aligned(cu_seqlens, 4) || !aligned(start, 4) ||
        !aligned(workspace, 256))
        return SPARK_ERR_ALIGN;
    st = check_pages(k4_pages, v4_pages, n_pages, page_size, page_table, max_pages);
    if (st != SPARK_OK) return st;
    if (workspace_bytes < kWorkspaceHeader) return SPARK_ERR_WORKSPACE;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    Kv4Params P;
    std::memset(&P, 0, sizeof(P));
    P.qkv = static_cast<const __nv_bfloat16 *>(qkv);
    P.pos = pos;
    P.cu = cu_seqlens;
    P.begin = start;
    P.N = n_tokens;
    P.S = S;
    P.status = static_cast<unsigned *>(workspace);
    set_layer(P, desc, H, Hkv);
    P.pg = pages_of(k4_pages, v4_pages, n_pages, page_size, page_table, max_pages);
    auto kernel = desc->rot_dim == kHeadDim ? kv4_store_kernel<true> : kv4_store_kernel<false>;
    st = done(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStoreSmem));
    if (st != SPARK_OK) return st;
    return done(launch_overlapped(kernel, dim3(sms), dim3(kStoreThreads), kStoreSmem,
                                  static_cast<cudaStream_t>(stream), P));
}

size_t spark_attn_kv4_load_workspace_size(int S, int Hkv) {
    if (S < 0 || Hkv < 1) return 0;
    return kWorkspaceHeader;
}

spark_status spark_attn_kv4_load(const void *k4_pages, const void *v4_pages, int n_pages,
                                 int page_size, const int32_t *page_table, int max_pages,
                                 const int32_t *begin, const int32_t *end, void *k_pages,
                                 void *v_pages, int to_n_pages, int to_page_size,
                                 const int32_t *to_page_table, int to_max_pages, int S, int Hkv,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    if (S < 0 || Hkv < 1) return SPARK_ERR_SHAPE;
    if (S == 0) return SPARK_OK;
    if (!begin || !end || !workspace) return SPARK_ERR_NULL;
    if (!aligned(begin, 4) || !aligned(end, 4) || !aligned(workspace, 256)) return SPARK_ERR_ALIGN;
    spark_status st = check_pages(k4_pages, v4_pages, n_pages, page_size, page_table, max_pages);
    if (st != SPARK_OK) return st;
    st = check_pages(k_pages, v_pages, to_n_pages, to_page_size, to_page_table, to_max_pages);
    if (st != SPARK_OK) return st;
    if (workspace_bytes < kWorkspaceHeader) return SPARK_ERR_WORKSPACE;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    Kv4LoadParams P{};
    P.begin = begin;
    P.end = end;
    P.S = S;
    P.Hkv = Hkv;
    P.status = static_cast<unsigned *>(workspace);
    P.pg = pages_of(const_cast<void *>(k4_pages), const_cast<void *>(v4_pages), n_pages, page_size,
              page_table, max_pages);
    P.k_pages = static_cast<__nv_bfloat16 *>(k_pages);
    P.v_pages = static_cast<__nv_bfloat16 *>(v_pages);
    P.to_table = to_page_table;
    P.to_n_pages = to_n_pages;
    P.to_page_shift = page_shift_of(to_page_size);
    P.to_max_pages = to_max_pages;
    return done(launch_overlapped(kv4_load_kernel, dim3(sms * 4), dim3(kThreads), 0,
                                  static_cast<cudaStream_t>(stream), P));
}

size_t spark_attn_decode_kv4_workspace_size(int B, int H, int Hkv, const spark_layer_desc *desc) {
    if (check_layer_desc(desc, H, Hkv) != SPARK_OK || B < 0) return 0;
    int sms;
    device_ready(&sms);
    return plan_decode_kv4(H, Hkv, sms).bytes;
}

spark_status spark_attn_decode_kv4(const void *qkv, const float *gate, const int32_t *pos,
                                   void *k4_pages, void *v4_pages, int n_pages, int page_size,
                                   const int32_t *page_table, int max_pages,
                                   const spark_layer_desc *desc, int B, int H, int Hkv, void *out,
                                   void *workspace, size_t workspace_bytes, void *stream) {
    spark_status st = check_layer_desc(desc, H, Hkv);
    if (st != SPARK_OK) return st;
    if (B < 0) return SPARK_ERR_SHAPE;
    if (B == 0) return SPARK_OK;
    if (!qkv || !gate || !pos || !out || !workspace) return SPARK_ERR_NULL;
    if (!aligned(qkv, 16) || !aligned(out, 16) || !aligned(gate, 4) || !aligned(pos, 4) ||
        !aligned(workspace, 256))
        return SPARK_ERR_ALIGN;
    st = check_pages(k4_pages, v4_pages, n_pages, page_size, page_table, max_pages);
    if (st != SPARK_OK) return st;
    int sms;
    const spark_status ready = device_ready(&sms);
    const DecodeKv4Plan pl = plan_decode_kv4(H, Hkv, sms);
    if (workspace_bytes < pl.bytes) return SPARK_ERR_WORKSPACE;
    if (ready != SPARK_OK) return ready;
    Kv4Params P;
    std::memset(&P, 0, sizeof(P));
    P.qkv = static_cast<const __nv_bfloat16 *>(qkv);
    P.gate = gate;
    P.pos = pos;
    P.out = static_cast<__nv_bfloat16 *>(out);
    P.N = P.S = B;
    P.status = static_cast<unsigned *>(workspace);
    set_layer(P, desc, H, Hkv);
    P.pg = pages_of(k4_pages, v4_pages, n_pages, page_size, page_table, max_pages);
    P.pos_end = max_pages << P.pg.page_shift;
    if (P.rope.rot_dim > 0 && P.pos_end > kRopePositions) P.pos_end = kRopePositions;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    P.counters = P.status + 1;
    P.part_ml = reinterpret_cast<float *>(ws + pl.ml);
    P.part_o = reinterpret_cast<float *>(ws + pl.o);
    return done(launch_decode_kv4(P, pl.grid, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
