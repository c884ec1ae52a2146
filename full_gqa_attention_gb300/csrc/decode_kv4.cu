// decode_kv4.cu -- one decode step over a cache in 4 bits (format: kv4.cuh).
//
// For every row b and KV head g the G query heads of the group attend to the
// cached slots [lo, pos) of the row's pages, as they are held, and to the new
// token itself, as it is:
//     out = sigma(gate) * sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
// with s_j = q.k_j / 16.  The new token's key and value are quantised into
// slot pos.  The step reads 288 bytes per slot and KV head.
//
// The work is shared out as the bf16 step's is (decode_paged.cu): the tiles of
// 64 slots of all pairs are one list, every CTA takes its stretch of it, and a
// pair that several CTAs share is joined by those that arrive last, in the order
// of the CTAs.  No CTA waits for another.  Three CTAs per SM: one warp each feeds
// a ring of stages by bulk copies, as many bytes of a page as the row sees; four
// warps compute.
//
// Widening 4 bits is what the SM has to do besides: a code pair is one
// conversion to two halves and one product with the scale, exact, in the
// registers in which the matrix instructions take them (the pages hold the
// operands' order).  Keys and values are the instructions' A operand, 16 slots
// or dims.  A warp takes 16 slots' scores, and after a barrier a quarter of the
// dims of all 64 slots' values: sums over all dims in every warp would take 64
// registers a thread instead of 16, and with fewer warps on an SM the latency of
// a tile's chain -- scores, maximum, exponentials, products -- shows (262,139
// tokens of 4 KV heads 75 us instead of 67, with everything else as it then was).
// So there is nothing to join over the warps either.
//
// 262,139 tokens of 4 KV heads take 60 us: 5.0 TB/s, 0.74 of a copy's rate.  A tile
// takes an SM some 900 cycles -- 32 words a warp at 17 for their conversions,
// scales and products, and the chain -- where HBM would need 784; 3 us go to the
// start, 5 to the last tiles, the states and their joins.
//
// B has 8 columns.  Up to 4 heads' queries are a sum of two halves each (22
// bits), in two columns; 8 heads' are one half each (11 bits).  Probabilities are
// one half: their roundings are independent and 16 times smaller than that of the
// output.  They are taken relative to a reference that all warps share, the
// largest score so far or up to 2^4 less, so that most tiles need neither a
// maximum over the warps nor a second barrier; they are times 2^11, so that none
// overflows, all of more than 2^-25 of the largest have 11 bits, and smaller ones
// are off by 2^-36 of it.  Their sums are of the same ones in 32 bits.
#include "decode_walk.cuh"
#include "kv4.cuh"
#include "kv4_counts.cuh"

namespace spark {

namespace {

// What setting a pair up and finishing it costs, in tiles: 2 / 3 / 4 / 5 / 7 take
// 27.2 / 27.8 / 28.0 / 28.2 / 29 us for 48 rows of 1 to 16,384 tokens, 29.8 / 29.6 /
// 30.6 / 29.6 / 32 for 256 windows of 512.
constexpr int kPairCost = 3;
constexpr int kTile = 64;                                 // slots per stage
constexpr int kWarps = 4;                                 // consumers
constexpr int kThreads = (kWarps + 1) * 32;               // + one producer warp
constexpr int kTileBytes = kTile * kKv4TokenBytes;        // K or V
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kQBytes = 8 * kHeadDim * 2;                 // 8 columns
constexpr int kRowBytes = kHeadDim * 2;
// Pairs handed over at a time: with 2 the windows take 31 us, with 4 three CTAs no
// longer fit an SM (42).
constexpr int kPairs = 3;
// Partial states loaded at once (2 or 8: 262,139 tokens 62.3 us instead of 60.6).  In the
// first step kSub are joined (kv4_counts.cuh; 32: 20 rows of 8 query heads a KV head 23.5
// instead of 21.6).
constexpr int kFan = 4;
static_assert(kCountWords <= kWorkspaceHeader / 4 - 1, "the counts fit the header");
constexpr int kProbBytes = 2 * kWarps * 32 * 8;           // two tiles' probabilities
// Scores may pass the reference by this (by nothing: 2 to 5 % slower).
constexpr float kHeadroom = 4.f;
constexpr float kProbShift = 11.f;                        // probabilities are times 2^11
constexpr float kProbScale = 2048.f;
constexpr int kSumRow = kHeadDim;                         // floats

// What goes by the query heads of a KV head.  With up to 4, three CTAs per SM of
// three stages; 8 heads' states and joins take more registers, and two CTAs of
// four stages are faster (20 rows of one KV head 25.9 -> 21.8 us, 500,000 tokens
// 45.3 -> 41.9).  Shared memory: the stages, the new tokens (queries, key, value) of
// kPairs pairs, the queries' halves (after the tiles: 4 heads' sums), two tiles'
// probabilities.
template <bool kTwo>
struct Shape {
    static constexpr int kHeads = kTwo ? 4 : 8;
    static constexpr int kCtasPerSm = kTwo ? 3 : 2;
    static constexpr int kStages = kTwo ? 3 : 4;
    static constexpr int kNewBytes = (kHeads + 2) * kRowBytes;
    static constexpr int kSmemBytes =
        kStages * kStageBytes + kPairs * kNewBytes + kQBytes + kProbBytes;
};

using Row = DecodeRow<kTile, kPairCost>;
using Walk = DecodeWalk<kTile, kPairCost>;

__device__ __forceinline__ Row row_of(const Kv4Params &P, int b) {
    return decode_row<kTile, kPairCost>(P, b);
}

// A pair as the producer hands it over: its tiles [t0, t1) for this CTA (none:
// the end), the CTAs [c0, c1] that share it.  A CTA shares its first and its
// last pair at most, and has two places for a state: `second` is 1 where the
// pair is not the first of c0 (it is the first of every other).
struct Pair {
    int pos, lo, b, g, t0, t1, c0, c1, second;
};

__device__ __forceinline__ void consumer_bar() {
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a),
                              *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Two numbers as halves, and what they leave.
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack_half2_rest(float lo, float hi, uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_half2(lo - f.x, hi - f.y);
}

// Two halves times scale `upper` (0, 1) of two.
__device__ __forceinline__ uint32_t mul_scale(uint32_t a, uint32_t scales, int upper) {
    const __half2 s = *reinterpret_cast<const __half2 *>(&scales);
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a),
                              upper ? __high2half2(s) : __low2half2(s));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Counts one up, back to 0 from `all`, and whether that was it.  What was written
// before is seen by who counts later.
__device__ __forceinline__ bool count_last(unsigned *counters, const StateCount &c, unsigned all) {
    unsigned before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
                 : "=r"(before)
                 : "l"(counters + c.word), "r"(1u << c.shift)
                 : "memory");
    const bool last = (before >> c.shift & ((1u << c.bits) - 1u)) == all - 1;
    if (last) atomicSub(counters + c.word, all << c.shift);
    return last;
}

// The CTAs that share a pair with units [first, first + units).
__device__ __forceinline__ int first_cta(long long first, long long share) {
    return static_cast<int>(quotient(first + kPairCost, share));
}
__device__ __forceinline__ int last_cta_of(long long first, long long units, long long share) {
    return static_cast<int>(quotient(first + units - 1, share));
}

__device__ __forceinline__ float nonfinite_part(float x) { return isfinite(x) ? 0.f : x; }

}  // namespace

// kTwo: queries as sums of two halves (4 heads at most).
template <bool kTwo>
__global__ void __launch_bounds__(kThreads, Shape<kTwo>::kCtasPerSm)
    decode_kv4_kernel(const __grid_constant__ Kv4Params P) {
    constexpr int kStages = Shape<kTwo>::kStages;
    constexpr int kNewBytes = Shape<kTwo>::kNewBytes;
    constexpr int kRows = Shape<kTwo>::kHeads / kWarps;                 // heads of a warp: warp, warp + 4
    extern __shared__ __align__(128) uint8_t stages[];
    uint8_t *new_rows = stages + kStages * kStageBytes;
    uint8_t *qs = new_rows + kPairs * kNewBytes;         // queries' halves, as B takes them
    uint2 *probs = reinterpret_cast<uint2 *>(qs + kQBytes);  // [2][4 groups][32 lanes]
    // the sums of 4 heads [4][kSumRow] in the queries' place
    float *sums = reinterpret_cast<float *>(qs);
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ uint64_t pair_full[kPairs], rows_full[kPairs], new_full[kPairs];
    __shared__ uint64_t pair_empty[kPairs];
    __shared__ Pair pairs[kPairs];
    __shared__ int abort_flag, lost, last_cta;
    // Of a tile, by the last bit of its number: someone gave up waiting; some
    // score passes the reference by too much.
    __shared__ int gave_up[2], passed[2];
    __shared__ float red[kWarps][8];            // the warps' maxima, or sums
    __shared__ int s_row;
    __shared__ long long s_base;
    __shared__ long long warp_sum[kThreads / 32];
    __shared__ float q_unit[8];                 // of the queries' halves, in base-2 score units
    __shared__ float s_new[8], s_gate[8];       // the new token's scores, the gates
    // cos and sin of the pair's position: the consumers', the producer's
    __shared__ float2 cs[kHeadDim / 2], cs_new[kHeadDim / 2];
    // the new token's key and value, quantised
    __shared__ uint32_t new_codes[kPairs][2][32];
    __shared__ uint8_t new_scale[kPairs][2][32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < kStages) {
        mbar_init(&full[tid], 1);
        mbar_init(&empty[tid], kWarps);
        fence_mbar_init();
    } else if (tid >= 32 && tid < 32 + kPairs) {
        mbar_init(&pair_full[tid - 32], 1);
        mbar_init(&rows_full[tid - 32], 1);
        mbar_init(&new_full[tid - 32], 1);
        mbar_init(&pair_empty[tid - 32], kWarps);
        fence_mbar_init();
    } else if (tid == 64) {
        abort_flag = 0;
        gave_up[0] = gave_up[1] = passed[0] = passed[1] = 0;
        lost = 0;
    }
    const int half = P.rope.rot_dim / 2;
    grid_dep_wait();  // positions, tables and pages may come from the kernel before

    // ---------------------------------------------------------- this CTA's stretch
    const int per = (P.N + kThreads - 1) / kThreads;  // rows per thread
    const int b0 = tid * per;
    long long mine = 0;
    for (int b = b0; b < b0 + per && b < P.N; ++b) {
        const int p = P.pos[b];
        if (blockIdx.x == 0 && (p < -1 || p >= P.pos_end))
            atomicOr(P.status, kErrPosition);
        mine += row_of(P, b).units();
    }
    long long before = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before += y;
    }
    if (lane == 31) warp_sum[warp] = before;
    before -= mine;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    total *= P.Hkv;
    const long long share = quotient(total + gridDim.x - 1, gridDim.x);
    Walk wk{};
    wk.u = share * blockIdx.x;
    wk.end = wk.u + share < total ? wk.u + share : total;
    if (wk.u >= wk.end) return;
    if (wk.u >= before * P.Hkv && wk.u < (before + mine) * P.Hkv) {
        int b = b0;
        long long base = before * P.Hkv;
        for (;; ++b) {
            const long long n = P.Hkv * row_of(P, b).units();
            if (wk.u < base + n || b + 1 >= P.N) break;
            base += n;
        }
        s_row = b;
        s_base = base;
    }
    __syncthreads();
    wk.b = s_row;
    wk.base = s_base;
    wk.row = row_of(P, wk.b);

    if (warp == kWarps) {
        // ------------------------------------------------------ producer
        // Lane l copies K (or V: bit 0) of piece l / 2 of a tile; a piece is
        // what lies in one page, of it the groups that the row sees.
        const int page = 1 << P.pg.page_shift;
        const int piece_slots = page < kTile ? page : kTile;
        const int pieces = kTile / piece_slots;
        const int piece = lane >> 1, which = lane & 1;
        const size_t width = static_cast<size_t>(P.H + 2 * P.Hkv) * kHeadDim;
        int it = 0, n_pairs = 0;
        bool ok = true;
        // Hands over a pair (or the end), and fetches its new token.  After an
        // abort too: every shared pair has to be counted, so that the counters
        // are 0 again.
        auto hand_over = [&](bool end) {
            const int s = n_pairs % kPairs;
            if (lane == 0) {
                if (n_pairs >= kPairs)
                    mbar_wait_plain_short(&pair_empty[s], ((n_pairs / kPairs) - 1) & 1);
                Pair &p = pairs[s];
                p.pos = wk.row.pos;
                p.lo = wk.row.lo;
                p.b = wk.b;
                p.g = wk.g;
                p.t0 = wk.t0;
                p.t1 = end ? wk.t0 : wk.t1;
                if (!end) {
                    uint8_t *dst = new_rows + s * kNewBytes;
                    const __nv_bfloat16 *src = P.qkv + wk.b * width;
                    mbar_arrive_expect_tx(&rows_full[s], (P.G + 2) * kRowBytes);
                    bulk_load(dst, src + static_cast<size_t>(wk.g) * P.G * kHeadDim,
                              P.G * kRowBytes, &rows_full[s]);
                    bulk_load(dst + P.G * kRowBytes,
                              src + static_cast<size_t>(P.H + wk.g) * kHeadDim, kRowBytes,
                              &rows_full[s]);
                    bulk_load(dst + (P.G + 1) * kRowBytes,
                              src + static_cast<size_t>(P.H + P.Hkv + wk.g) * kHeadDim, kRowBytes,
                              &rows_full[s]);
                    p.c0 = first_cta(wk.first, share);
                    p.c1 = last_cta_of(wk.first, wk.row.units(), share);
                    p.second = share * p.c0 < wk.first ? 1 : 0;
                }
                mbar_arrive(&pair_full[s]);
            }
            __syncwarp();
            ++n_pairs;
        };
        // Quantises the new token of the pair handed over last, while the copies
        // of its first tiles are on their way.
        auto quantise_new = [&]() {
            const int s = (n_pairs - 1) % kPairs;
#pragma unroll 1
            for (int k = lane; k < half; k += 32)
                rope_cos_sin_fine(wk.row.pos, P.rope.u[k], cs_new[k].x, cs_new[k].y);
            mbar_wait_plain_short(&rows_full[s], ((n_pairs - 1) / kPairs) & 1);
            __syncwarp();
            const uint8_t *src = new_rows + s * kNewBytes + P.G * kRowBytes;
            float y[8];
            unsigned byte[1];
            uint32_t codes[1];
            const KeyTurn turn = kv4_key_turn(P.rope.rot_dim, wk.row.pos, lane);
            kv4_rotate(turn, src, lane, cs_new, y);
            kv4_key_row<false>(turn, src, lane, y, wk.row.pos, P.turns, codes[0], byte[0]);
            new_codes[s][0][lane] = codes[0];
            new_scale[s][0][lane] = static_cast<uint8_t>(byte[0]);
            const uint4 value[1] = {kv4_own(src + kRowBytes, lane)};
            kv4_value_rows(value, codes, byte);
            new_codes[s][1][lane] = codes[0];
            new_scale[s][1][lane] = static_cast<uint8_t>(byte[0]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&new_full[s]);
        };
        while (wk.load(P)) {
            // (consumers that have left take no pair any more)
            if (__shfl_sync(0xffffffffu, *static_cast<volatile int *>(&lost), 0)) break;
            hand_over(false);
            int early = kStages;  // tiles before the new token's turn comes
            const int32_t *row = P.pg.table + static_cast<size_t>(wk.b) * P.pg.max_pages;
            const int slot0 = wk.row.slot0();
            const int lo = wk.row.lo & ~15, hi = (wk.row.pos + 15) & ~15;  // groups seen
            int ids = 0;
            bool gaps = false;  // some page number is not in the pool
            for (int t = wk.t0; ok && t < wk.t1; ++t) {
                if (early-- == 0) quantise_new();
                // page numbers of the next 32 pieces, one per lane; -1: none
                const int in = (t - wk.t0) * pieces & 31;
                if (in == 0) {
                    const int slot = slot0 + t * kTile + lane * piece_slots;
                    ids = -1;
                    gaps = false;
                    if (slot < hi && slot + piece_slots > lo && slot < slot0 + wk.t1 * kTile) {
                        ids = row[slot >> P.pg.page_shift];
                        if (ids < 0 || ids >= P.pg.n_pages) {
                            atomicOr(P.status, kErrPage);
                            ids = -1;
                            gaps = true;
                        }
                    }
                    gaps = __any_sync(0xffffffffu, gaps);
                }
                const int s = it % kStages;
                if (it >= kStages && lane == 0)
                    ok = mbar_wait_short(&empty[s], ((it / kStages) - 1) & 1, &abort_flag, P.status);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const int id = __shfl_sync(0xffffffffu, ids, (in + piece) & 31);
                const int at = slot0 + t * kTile + piece * piece_slots;
                const int a = at > lo ? at : lo;
                const int b = at + piece_slots < hi ? at + piece_slots : hi;
                uint8_t *dst = stages + s * kStageBytes + which * kTileBytes +
                               (a & (kTile - 1)) * kKv4TokenBytes;
                const int bytes = piece < pieces && a < b ? (b - a) * kKv4TokenBytes : 0;
                if (gaps) {
                    // A page that is not in the pool reads as zeros: written once every lane
                    // knows that the stage is free, and all before lane 0 tells that it is full.
                    __syncwarp();
                    if (id < 0)
                        for (int i = 0; i < bytes; i += 16)
                            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();  // copies come here later
                    __syncwarp();
                }
                const unsigned all =
                    __reduce_add_sync(0xffffffffu, id < 0 ? 0u : static_cast<unsigned>(bytes));
                if (lane == 0) mbar_arrive_expect_tx(&full[s], all);
                __syncwarp();
                if (bytes && id >= 0)
                    bulk_load(dst, (which ? P.pg.v : P.pg.k) + P.pg.group(id, wk.g, P.Hkv, a),
                              bytes, &full[s]);
                ++it;
            }
            if (early >= 0) quantise_new();
        }
        hand_over(true);
        __syncthreads();
        // copies still in flight after an abort must land before the CTA ends
        if (lane == 0 && abort_flag)
            for (int i = it > kStages ? it - kStages : 0; i < it; ++i)
                mbar_wait_plain_short(&full[i % kStages], (i / kStages) & 1);
        if (lane == 0 && abort_flag)
            for (int i = n_pairs - 1 > kPairs ? n_pairs - 1 - kPairs : 0; i < n_pairs - 1; ++i)
                mbar_wait_plain_short(&rows_full[i % kPairs], (i / kPairs) & 1);
        // Pairs that the consumers have not come to are counted all the same, so that the
        // counts are 0 again; what is joined of them is invalid, as the status word says.
        if (lane == 0 && lost) {
            Walk rest{};
            rest.u = share * blockIdx.x;
            rest.end = wk.end;
            rest.b = s_row;
            rest.base = s_base;
            rest.row = row_of(P, rest.b);
            for (int n = 1; rest.load(P); ++n) {
                if (n < lost) continue;
                const int c0 = first_cta(rest.first, share);
                const StateGroup g = kv4_group(c0, last_cta_of(rest.first, rest.row.units(), share),
                                               static_cast<int>(blockIdx.x));
                if ((g.from == g.to || count_last(P.counters, kv4_first_count(g.from, g.to),
                                                  g.to - g.from + 1)) &&
                    g.groups > 1)
                    count_last(P.counters, kv4_second_count(c0), g.groups);
            }
        }
        return;
    }

    // ---------------------------------------------------------- consumers
    const int row8 = lane >> 2, c4 = lane & 3;           // row and column pair of fragments
    const int tok = 4 * (row8 >> 1) + (row8 & 1);        // slot of row row8; row8 + 8: + 2
    const int h0 = kTwo ? 2 * (c4 & 1) : 2 * c4;         // the first of its two heads
    // (columns of no head keep what they hold: their sums are nobody's)
    if (tid < 8) q_unit[tid] = 0.f;
    float2 freq = make_float2(0.f, 0.f);
    if (tid < half) freq = P.rope.u[tid];
    int it = 0;
    bool aborted = false;  // the same in every consumer thread
    // Waits for a pair; the barrier behind it tells every warp whether all have it.
    auto await_pair = [&](int n) {
        if (!mbar_wait_plain_short(&pair_full[n % kPairs], (n / kPairs) & 1)) {
            atomicOr(P.status, kErrTimeout);
            abort_flag = 1;
            lost = n + 1;
        }
        consumer_bar();
    };
    await_pair(0);
    for (int n = 0; !lost; ++n) {
        const Pair &pair = pairs[n % kPairs];
        const int pos = pair.pos, lo = pair.lo, t0 = pair.t0, t1 = pair.t1;
        if (t0 >= t1) break;
        // The new token's queries, warp w taking heads w and w + 4, and its score
        // (the turns of q and k cancel).
        const int s_pair = n % kPairs, pair_turn = (n / kPairs) & 1;
        const uint8_t *rows = new_rows + s_pair * kNewBytes;
        float gate[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int hq = warp + i * kWarps;
            if (hq < P.G)
                gate[i] = P.gate[static_cast<size_t>(pair.b) * P.H + pair.g * P.G + hq];
        }
        int id_new = 0;
        if (warp == 0)
            id_new = P.pg.table[static_cast<size_t>(pair.b) * P.pg.max_pages +
                                (pos >> P.pg.page_shift)];
        if (tid < half) rope_cos_sin_fine(pos, freq, cs[tid].x, cs[tid].y);
        if (!mbar_wait_plain_short(&rows_full[s_pair], pair_turn)) {
            atomicOr(P.status, kErrTimeout);
            abort_flag = 1;
            gave_up[0] = 1;
        }
        consumer_bar();
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int hh = warp + i * kWarps;
            if (hh >= P.G) break;
            // in halves, scaled by a power of two so that the largest is 1 to 2
            const uint8_t *row = rows + hh * kRowBytes;
            float y[8], k[8];
            kv4_floats(kv4_own(row, lane), y);
            kv4_floats(kv4_own(rows + P.G * kRowBytes, lane), k);
            float d = 0.f, a = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) d = fmaf(y[j], k[j], d);
            kv4_rotate(kv4_key_turn(P.rope.rot_dim, pos, lane), row, lane, cs, y);
            bool odd = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a = fmaxf(a, fabsf(y[j]));
                odd = odd || !isfinite(y[j]);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                d += __shfl_xor_sync(0xffffffffu, d, off);
            }
            // (a query that is not finite is NaN throughout)
            const float z = __any_sync(0xffffffffu, odd) ? NAN : 0.f;
            const unsigned e = __float_as_uint(a) >> 23;
            const unsigned up = (e < 253u ? 254u - e : 1u) << 23;
            const float f = __uint_as_float(up);
            uint32_t hi[4], rest[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = fmaf(y[2 * j], f, z), v = fmaf(y[2 * j + 1], f, z);
                hi[j] = pack_half2(u, v);
                rest[j] = pack_half2_rest(u, v, hi[j]);
            }
            // in the order in which the lanes take B: dims 8 l .. are step
            // 4 (l / 16) + l % 4 of lane 4 column + l % 16 / 4
            uint8_t *dst = qs + (4 * (lane >> 4) + (lane & 3)) * 512 + (lane >> 2 & 3) * 16;
            *reinterpret_cast<uint4 *>(dst + hh * 64) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (kTwo)
                *reinterpret_cast<uint4 *>(dst + (hh + 4) * 64) =
                    make_uint4(rest[0], rest[1], rest[2], rest[3]);
            if (lane == 0) {
                q_unit[hh] = kScaleLog2 * __uint_as_float((254u << 23) - up);
                s_new[hh] = fmaf(d, kScaleLog2, z);
                s_gate[hh] = gate[i];
            }
        }
        consumer_bar();
        const float unit0 = q_unit[h0], unit1 = q_unit[h0 + 1];
        float o[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        // References and sums of the thread's two heads.  All warps have the same
        // references: a head's largest score so far, or up to kHeadroom less.
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        bool ok = !aborted;
        for (int t = t0; ok && t < t1; ++t, ++it) {
            const int s = it % kStages;
            ok = mbar_wait_short(&full[s], (it / kStages) & 1, &abort_flag, P.status);
            const int first = (lo & ~(kTile - 1)) + t * kTile;
            const uint8_t *kt = stages + s * kStageBytes;
            uint2 *pt = probs + (it & 1) * kWarps * 32;
            // S^T (16 slots x 8 columns) = K (16 x 256) Q^T (256 x 8)
            float x[4];
            {
                const uint8_t *kg = kt + warp * kKv4GroupBytes;
                const uint8_t *ks = kg + kKv4Codes + tok * 16 + c4 * 4;
                const uint32_t sa = *reinterpret_cast<const uint32_t *>(ks);
                const uint32_t sb = *reinterpret_cast<const uint32_t *>(ks + 32);
                // blocks 2 c4 and 8 + 2 c4 (first words), and those behind them
                const uint32_t ua[2] = {(sa & 0x00ff00ffu) << 7, (sa >> 1) & 0x7f807f80u};
                const uint32_t ub[2] = {(sb & 0x00ff00ffu) << 7, (sb >> 1) & 0x7f807f80u};
                float acc[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[0][i] = acc[1][i] = acc[2][i] = acc[3][i] = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *kc = kg + h * 1024 + tok * 64 + c4 * 16;
                    const uint4 ka = *reinterpret_cast<const uint4 *>(kc);
                    const uint4 kb = *reinterpret_cast<const uint4 *>(kc + 128);
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w};
                    const uint32_t wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 qf = *reinterpret_cast<const uint4 *>(
                            qs + (4 * h + i) * 512 + lane * 16);
                        uint32_t a[4], b[4];
                        kv4_widen(wa[i], a);
                        kv4_widen(wb[i], b);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            a[j] = mul_scale(a[j], ua[i >> 1], h);
                            b[j] = mul_scale(b[j], ub[i >> 1], h);
                        }
                        mma_f16_16816(acc[2 * (i & 1)], a[0], b[0], a[1], b[1], qf.x, qf.y);
                        mma_f16_16816(acc[2 * (i & 1) + 1], a[2], b[2], a[3], b[3], qf.z, qf.w);
                    }
                }
                // this thread's slots (rows row8 and row8 + 8) and heads
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = (acc[0][i] + acc[1][i]) + (acc[2][i] + acc[3][i]);
                    if (kTwo) x[i] += __shfl_xor_sync(0xffffffffu, x[i], 2);
                    x[i] *= i & 1 ? unit1 : unit0;
                }
                if (first < lo || first + kTile > pos) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int slot = first + warp * kKv4Group + tok + (i & 2);
                        if (slot < lo || slot >= pos) x[i] = -INFINITY;
                    }
                    // Slots that hold no visible token may hold anything: a scale of
                    // zero makes zeros of their values, too.
                    uint32_t seen = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int slot = first + warp * kKv4Group + 4 * c4 + j;
                        if (slot >= lo && slot < pos)
                            seen |= 0xffu << (8 * (2 * (j & 1) + (j >> 1)));
                    }
                    uint2 *sv = reinterpret_cast<uint2 *>(
                        stages + s * kStageBytes + kTileBytes + warp * kKv4GroupBytes + kKv4Codes +
                        lane * 8);
                    *sv = make_uint2(sv->x & seen, sv->y & seen);
                    fence_proxy_async_smem();  // copies come here later
                }
            }
            // P^T of these slots, in the order in which the lanes take B
            float p[4];
            auto exponentiate = [&]() {
                const float z0 = m0 == -INFINITY ? 0.f : m0 - kProbShift;
                const float z1 = m1 == -INFINITY ? 0.f : m1 - kProbShift;
                p[0] = fast_exp2(x[0] - z0);
                p[1] = fast_exp2(x[1] - z1);
                p[2] = fast_exp2(x[2] - z0);
                p[3] = fast_exp2(x[3] - z1);
                pt[warp * 32 + lane] = make_uint2(movmatrix_trans(pack_half2(p[0], p[1])),
                                                  movmatrix_trans(pack_half2(p[2], p[3])));
            };
            exponentiate();
            if (__any_sync(0xffffffffu, fmaxf(x[0], x[2]) > m0 + kHeadroom ||
                                            fmaxf(x[1], x[3]) > m1 + kHeadroom))
                passed[it & 1] = 1;
            if (!ok) gave_up[it & 1] = 1;
            consumer_bar();
            if (gave_up[it & 1]) break;  // (all of them: the next tile has its own word)
            if (passed[it & 1]) {
                // new references: the largest scores so far
                float n0 = fmaxf(x[0], x[2]), n1 = fmaxf(x[1], x[3]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
                    n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
                }
                if (row8 == 0 && (!kTwo || c4 < 2)) {
                    red[warp][h0] = n0;
                    red[warp][h0 + 1] = n1;
                }
                consumer_bar();
                if (tid == 0) passed[it & 1] = 0;
                n0 = m0;
                n1 = m1;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    n0 = fmaxf(n0, red[w][h0]);
                    n1 = fmaxf(n1, red[w][h0 + 1]);
                }
                const float r0 = n0 == -INFINITY ? 1.f : fast_exp2(m0 - n0);
                const float r1 = n1 == -INFINITY ? 1.f : fast_exp2(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= r0;
                l1 *= r1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i][0] *= r0;
                    o[i][1] *= r1;
                    o[i][2] *= r0;
                    o[i][3] *= r1;
                }
                exponentiate();
                consumer_bar();
            }
            l0 += p[0] + p[2];
            l1 += p[1] + p[3];
            // O^T += V^T P^T, 64 dims of all slots
            const uint8_t *vt = kt + kTileBytes;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint2 pb = pt[u * 32 + lane];
                const uint8_t *vu = vt + u * kKv4GroupBytes;
                const uint4 v = *reinterpret_cast<const uint4 *>(vu + warp * 512 + lane * 16);
                const uint32_t w = *reinterpret_cast<const uint32_t *>(vu + kKv4Codes + lane * 8 +
                                                                       4 * (warp >> 1));
                const uint32_t u0 = (w & 0x00ff00ffu) << 7, u1 = (w >> 1) & 0x7f807f80u;
                const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a[4];
                    kv4_widen(wv[i], a);
                    mma_f16_16816(o[i], mul_half2(a[0], u0), mul_half2(a[1], u0),
                                  mul_half2(a[2], u1), mul_half2(a[3], u1), pb.x, pb.y);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }
        aborted = gave_up[0] || gave_up[1];  // (never reset; all have left the loop by one)
        // Where the new token goes; read now, written when the pair is finished.
        const int t_new = pos & 15;
        uint8_t *k_new = nullptr, *v_new = nullptr;
        unsigned old[4] = {0, 0, 0, 0};
        if (warp == 0 && id_new >= 0 && id_new < P.pg.n_pages) {
            const size_t at = P.pg.group(id_new, pair.g, P.Hkv, pos);
            k_new = P.pg.k + at;
            v_new = P.pg.v + at;
            const uint8_t *src = v_new + kv4_value_at(lane, t_new >> 2) + 2 * (t_new >> 1 & 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) old[j] = *reinterpret_cast<const uint16_t *>(src + 4 * j);
        }

        // ---------------------------------------------- this CTA's state of the heads
        // Warp w has heads w and w + 4, lane l their dims 8 l ..
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, off);
            l1 += __shfl_xor_sync(0xffffffffu, l1, off);
        }
        if (row8 == 0 && (!kTwo || c4 < 2)) {
            red[warp][h0] = l0;
            red[warp][h0 + 1] = l1;
        }
        HeadState st[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i) consumer_bar();  // (the heads before are read)
            // dims 32 row8 + 8 warp .. + 7 of two heads; with two columns a head
            // two threads have the same: half each
            if (kTwo || c4 >> 1 == i) {
                const bool upper = kTwo && (c4 & 2);
                float *dst = sums + (h0 & 3) * kSumRow + 32 * row8 + 8 * warp + (upper ? 4 : 0);
#pragma unroll
                for (int j = 0; j < (kTwo ? 2 : 4); j += 2) {
                    float a[4], b[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        a[k] = upper ? o[kTwo ? 2 : j][k] : o[j][k];
                        b[k] = upper ? o[3][k] : o[j + 1][k];
                    }
                    *reinterpret_cast<float4 *>(dst + 2 * j) = make_float4(a[0], a[2], b[0], b[2]);
                    *reinterpret_cast<float4 *>(dst + kSumRow + 2 * j) =
                        make_float4(a[1], a[3], b[1], b[3]);
                }
            }
            consumer_bar();
            const int hq = warp + i * kWarps;
            HeadState &h = st[i];
            h.m = __shfl_sync(0xffffffffu, hq & 1 ? m1 : m0, hq >> 1);
            h.l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) h.l += red[w][hq];
            h.l *= 1.f / kProbScale;
            const float4 *src = reinterpret_cast<const float4 *>(sums + warp * kSumRow + 8 * lane);
            const float4 a = src[0], b = src[1];
            const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) h.o[j] = v[j] * (1.f / kProbScale);
        }

        // ------------------------------------------------------ finish or hand over
        // A pair of one CTA is finished.  Of others the states are joined by the
        // CTA that leaves its own last; of more than kSub in two steps, kSub of
        // them and then what those leave.  The order is that of the CTAs, so that
        // the result does not depend on which one is last.
        const int c0 = pair.c0, c1 = pair.c1;
        bool finish = c0 == c1;
        if (!finish) {
            const int me = static_cast<int>(blockIdx.x), second = pair.second;
            auto place = [&](int cta) { return 2 * cta + (cta == c0 ? second : 0); };
            // Leaves the state in that CTA's place; whether it was the last of `all`.
            auto leave = [&](int cta, const StateCount &count, int all) {
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int hq = warp + i * kWarps;
                    if (hq >= P.G) break;
                    const size_t at = static_cast<size_t>(place(cta)) * P.G + hq;
                    float4 *dst = reinterpret_cast<float4 *>(P.part_o + at * kHeadDim + lane * 8);
                    dst[0] = make_float4(st[i].o[0], st[i].o[1], st[i].o[2], st[i].o[3]);
                    dst[1] = make_float4(st[i].o[4], st[i].o[5], st[i].o[6], st[i].o[7]);
                    if (lane == 0)
                        reinterpret_cast<float2 *>(P.part_ml)[at] = make_float2(st[i].m, st[i].l);
                }
                consumer_bar();
                // behind the whole CTA's state, before the others' are read
                if (tid == 0) last_cta = count_last(P.counters, count, all);
                consumer_bar();
                return last_cta != 0;
            };
            // The states of CTAs from, from + step, .. up to `to`, 32 at most: a lane
            // has one state's maximum and sum, all lanes its output.
            auto join = [&](int from, int to, int step) {
                const int n = step == 1 ? to - from + 1 : (to - from) / kSub + 1;
                auto at = [&](int k, int i) {  // (a warp without a head reads the first)
                    const int hq = warp + i * kWarps < P.G ? warp + i * kWarps : 0;
                    return place(from + (k < n ? k : n - 1) * step) * P.G + hq;
                };
                float w[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    HeadState &h = st[i];
                    const float2 ml =
                        __ldcg(reinterpret_cast<const float2 *>(P.part_ml) + at(lane, i));
                    const float m = lane < n ? ml.x : -INFINITY;
                    h.m = m;
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
                        h.m = fmaxf(h.m, __shfl_xor_sync(0xffffffffu, h.m, off));
                    // (an empty state's sums are 0, or NaN, whatever their weight)
                    w[i] = lane >= n ? 0.f : m == -INFINITY ? 1.f : fast_exp2(m - h.m);
                    h.l = lane < n ? ml.y * w[i] : 0.f;
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
                        h.l += __shfl_xor_sync(0xffffffffu, h.l, off);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h.o[j] = 0.f;
                }
#pragma unroll 1
                for (int k0 = 0; k0 < n; k0 += kFan) {
                    float4 x[kRows][kFan], y[kRows][kFan];
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
#pragma unroll
                        for (int k = 0; k < kFan; ++k) {
                            const float4 *src = reinterpret_cast<const float4 *>(P.part_o) +
                                                at(k0 + k, i) * (kHeadDim / 4) + lane * 2;
                            x[i][k] = __ldcg(src);
                            y[i][k] = __ldcg(src + 1);
                        }
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
#pragma unroll
                        for (int k = 0; k < kFan; ++k) {
                            const float v[8] = {x[i][k].x, x[i][k].y, x[i][k].z, x[i][k].w,
                                                y[i][k].x, y[i][k].y, y[i][k].z, y[i][k].w};
                            add_scaled(st[i], __shfl_sync(0xffffffffu, w[i], (k0 + k) & 31), v);
                        }
                }
            };
            const StateGroup group = kv4_group(c0, c1, me);
            const int from = group.from, to = group.to, subs = group.groups;
            int a = from, b = to, step = 1;
            const bool single = from == to;  // the state is at hand
            finish = single || leave(me, kv4_first_count(from, to), to - from + 1);
#pragma unroll 1
            while (finish) {
                if (!single || step != 1) join(a, b, step);
                if (subs == 1 || step != 1) break;
                finish = leave(from, kv4_second_count(c0), subs);
                a = c0;
                b = c1;
                step = kSub;
            }
        }
        if (finish) {
            // the new token joins, the gate applies
            float v[8];
            kv4_floats(*reinterpret_cast<const uint4 *>(rows + (P.G + 1) * kRowBytes + lane * 16),
                       v);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int hq = warp + i * kWarps;
                if (hq >= P.G) break;
                HeadState &h = st[i];
                const float x_new = s_new[hq];
                const float top = fmaxf(h.m, x_new);
                const float z = top == -INFINITY ? 0.f : top;
                const float wo = h.m == -INFINITY ? 1.f : fast_exp2(h.m - z);
                const float wn = fast_exp2(x_new - z);
                const float scale = gate_act(s_gate[hq], P.gate_mode) / (h.l * wo + wn);
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] = (h.o[j] * wo + v[j] * wn) * scale;
                    // an infinity is one however small its weight
                    if (!isfinite(v[j])) y[j] = (v[j] + nonfinite_part(h.o[j])) * scale;
                }
                *reinterpret_cast<uint4 *>(
                    P.out + (static_cast<size_t>(pair.b) * P.H + pair.g * P.G + hq) * kHeadDim +
                    lane * 8) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                           pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
            }
            if (warp == 0) {
                // the new token's slot: every read of this pair is done
                if (!k_new) {
                    if (lane == 0) atomicOr(P.status, kErrPage);
                } else if (mbar_wait_plain_short(&new_full[s_pair], pair_turn)) {
                    *reinterpret_cast<uint32_t *>(k_new + kv4_key_at(lane, t_new)) =
                        new_codes[s_pair][0][lane];
                    // the other slot of each byte stays
                    const uint32_t codes = new_codes[s_pair][1][lane];
                    uint8_t *dst = v_new + kv4_value_at(lane, t_new >> 2) + 2 * (t_new >> 1 & 1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const unsigned two = codes >> (8 * j);
                        const unsigned c = (two & 15u) | (two & 0xf0u) << 4;
                        *reinterpret_cast<uint16_t *>(dst + 4 * j) = static_cast<uint16_t>(
                            t_new & 1 ? (old[j] & 0x0f0fu) | c << 4 : (old[j] & 0xf0f0u) | c);
                    }
                    if (!(lane & 1)) {
                        k_new[kv4_key_scale_at(lane >> 1, t_new)] = new_scale[s_pair][0][lane];
                        v_new[kv4_value_scale_at(lane >> 1, t_new >> 2) + 2 * (t_new & 1) +
                              (t_new >> 1 & 1)] = new_scale[s_pair][1][lane];
                    }
                } else {
                    atomicOr(P.status, kErrTimeout);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&pair_empty[s_pair]);
        await_pair(n + 1);  // (q, the new token and the sums are read)
    }
    grid_dep_launch();
    __syncthreads();  // with the producer
}

// ---------------------------------------------------------------- launcher

int decode_kv4_ctas(int sms, int G) {
    const int ctas = sms * (G <= 4 ? Shape<true>::kCtasPerSm : Shape<false>::kCtasPerSm);
    return ctas < kMostCtas ? ctas : kMostCtas;
}

template <bool kTwo>
static cudaError_t launch(const Kv4Params &P, int grid, cudaStream_t stream) {
    constexpr int kSmem = Shape<kTwo>::kSmemBytes;
    const cudaError_t err = cudaFuncSetAttribute(
        decode_kv4_kernel<kTwo>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (err != cudaSuccess) return err;
    return launch_overlapped(decode_kv4_kernel<kTwo>, dim3(grid), dim3(kThreads), kSmem, stream,
                             P);
}

cudaError_t launch_decode_kv4(const Kv4Params &P, int grid, cudaStream_t stream) {
    return P.G <= 4 ? launch<true>(P, grid, stream) : launch<false>(P, grid, stream);
}

}  // namespace spark
