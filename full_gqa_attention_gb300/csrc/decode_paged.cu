// decode_paged.cu -- one decode step over a KV cache in pages.
//
// For every row b and KV head g the G query heads of the group attend to the
// cached slots [lo, pos) of the row's pages (lo: 0, or the window's start) and
// to the new token itself:
//     out = sigma(gate) * sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
// with s_j = q.k_j / 16.  The step reads every cached key and value once
// (2 * 512 bytes per slot and KV head) and computes 8 G FLOP per byte pair, so
// HBM bounds it.
//
// One launch of one CTA per SM.  Every row's slots are cut into tiles of 64,
// and the tiles of all (row, KV head) pairs in a row form one list that the
// CTAs share out evenly, whatever the lengths: each reads the positions,
// finds the total, and takes its stretch.  So the split follows what the
// positions ask for on the device, ragged batches leave no SM idle, and a
// captured call serves other lengths.  A stretch crosses from one pair into
// the next while the loads run on: one warp feeds a ring of three 64 KB stages
// (K and V of a tile) by TMA, page by page, four warps consume them.
//
// A pair that lies in one stretch is finished where it was summed.  Otherwise
// each CTA leaves a partial state (max, sum, unnormalised output) in the
// workspace -- its first and its last pair are the only ones it can share, so
// two places per CTA and one counter (a byte of the workspace header) are
// enough -- and the CTA that arrives last at the pair's counter joins them in
// the order of the CTAs, so the result does not depend on which one that is.
// No CTA waits for another.
#include "paged.cuh"

namespace spark {

namespace {

// A pair's own units (Row::units).  None: the ragged batch of 48 rows takes 129
// us; 2, 3 and 5: 93 us, 64 sliding rows 33 to 34.
constexpr int kPairCost = 3;
constexpr int kTile = 64;                                 // slots per stage
constexpr int kStages = 3;
constexpr int kWarps = 4;                                 // consumers, 16 slots each
constexpr int kThreads = (kWarps + 1) * 32;               // + one producer warp
constexpr int kTileBytes = kTile * kHeadDim * 2;          // 32 KB (K or V)
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kQBytes = 8 * kHeadDim * 2;                 // 8 (padded) query heads
constexpr int kJoin = 6;                                  // partial states joined at once (2, 4,
                                                          // 6, 8: 161, 158, 157, 157 us for
                                                          // 262,139 tokens)
constexpr int kRedHeads = 4;                              // heads reduced over the warps at once
constexpr int kRedBytes = kWarps * kRedHeads * kHeadDim * 4;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kQBytes + 2 * kHeadDim * 2 + kRedBytes +
                           3 * kStages * 8;

__device__ __forceinline__ void consumer_bar() {
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}

// What a row asks for: its position, first visible slot and tiles (0: nothing).
struct Row {
    int pos, lo, tiles;
    __device__ __forceinline__ int slot0() const { return lo & ~(kTile - 1); }
    // Units of one of its pairs in the list: its tiles, and what setting a pair
    // up and finishing it costs besides, in tiles.
    __device__ __forceinline__ long long units() const {
        return tiles ? tiles + kPairCost : 0;
    }
};

__device__ __forceinline__ Row row_of(const PagedParams &P, int b) {
    Row r;
    r.pos = P.pos[b];
    r.lo = 0;
    r.tiles = 0;
    if (r.pos < 0 || r.pos >= P.pos_end) return r;
    if (P.kind == kLayerSliding && r.pos >= P.window) r.lo = r.pos - P.window + 1;
    const int n = (r.pos - r.slot0() + kTile - 1) / kTile;
    r.tiles = n > 0 ? n : 1;  // a row with nothing cached still has its new token
    return r;
}

// A CTA's walk over its stretch of the list: the pair (b, g) and the tiles
// [t0, t1) of it.  A pair's units are kPairCost for itself, then its tiles.
struct Walk {
    long long u, end;   // next unit of the stretch, its end
    long long base;     // first unit of row b
    long long first;    // first unit of the pair
    int b, g, t0, t1;
    Row row;

    // The next pair with tiles in the stretch, from unit u on; false at the
    // end.  b and base are at or before it.
    __device__ __forceinline__ bool load(const PagedParams &P) {
        while (u < end) {
            while (u >= base + P.Hkv * row.units()) {
                if (b + 1 >= P.N) return false;  // the positions changed under the call
                base += P.Hkv * row.units();
                row = row_of(P, ++b);
            }
            const long long n = row.units();
            g = static_cast<int>((u - base) / n);
            first = base + g * n;
            const int from = static_cast<int>(u - first) - kPairCost;
            const int to = static_cast<int>(end - first < n ? end - first : n) - kPairCost;
            u = first + to + kPairCost;
            t0 = from > 0 ? from : 0;
            t1 = to;
            if (t1 > t0) return true;
        }
        return false;
    }
};

// The running state of one query head: this lane's 8 dims.
struct HeadState {
    float m, l, o[8];
};

__device__ __forceinline__ void add_scaled(HeadState &s, float w, const float *o) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s.o[i] += o[i] * w;
}

// Values that are not finite.  A visible infinity is infinite in its dims,
// however small its weight, but not in these products: a weight that 32 bits
// hold as zero, or the two terms of a probability, which can have different
// signs, make NaN of it.  So where a sum is not finite, the values that are not
// are added up without weights and take its place: in each CTA's state
// (sum_nonfinite), where states are joined, and where the new token joins.  A
// NaN score makes the sum of the weights NaN, and with it the row.
__device__ __forceinline__ float nonfinite_part(float x) { return isfinite(x) ? 0.f : x; }

}  // namespace

// The sum of the values of the slots [lo, hi) of a pair that are not finite, over
// this warp's share of them, for a lane's 8 dims (from d0).  Groups of 8 slots
// (which lie in one page) are the warps' in turn: one table entry and 8 rows in
// flight.  Rare, and bounded by the CTA's stretch, so that a call takes about
// twice as long: 108 us for a row of 120,000 tokens with one such value (75
// without, and 61 ms where one warp walked the row), 0.42 ms for 262,139 tokens
// with many (0.19 without).
__device__ __noinline__ void sum_nonfinite(const PagedParams &P, int b, int g, int lo, int hi,
                                           int warp, int d0, float (&s)[8]) {
    const int32_t *row = P.table + static_cast<size_t>(b) * P.max_pages;
    for (int j0 = (lo & ~7) + warp * 8; j0 < hi; j0 += kWarps * 8) {
        const int id = row[j0 >> P.page_shift];
        if (id < 0 || id >= P.n_pages) continue;  // read as zeros
        const __nv_bfloat16 *src =
            P.v_pages + (((static_cast<size_t>(id) * P.Hkv + g) << P.page_shift) +
                         (j0 & ((1 << P.page_shift) - 1))) * kHeadDim + d0;
        uint4 w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            w[r] = j0 + r >= lo && j0 + r < hi
                       ? *reinterpret_cast<const uint4 *>(src + r * kHeadDim)
                       : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const uint32_t u[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[2 * i] += nonfinite_part(bf16_lo(u[i]));
                s[2 * i + 1] += nonfinite_part(bf16_hi(u[i]));
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    decode_paged_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __nv_bfloat16 *qs = reinterpret_cast<__nv_bfloat16 *>(stages + kStages * kStageBytes);
    __nv_bfloat16 *kn = qs + 8 * kHeadDim;  // the new token's key (rotated) and value
    __nv_bfloat16 *vn = kn + kHeadDim;
    float *red_o = reinterpret_cast<float *>(vn + kHeadDim);
    uint64_t *full = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(red_o) + kRedBytes);
    uint64_t *fullv = full + kStages;
    uint64_t *empty = fullv + kStages;
    __shared__ int abort_flag, seg_bad, seg_odd, last_cta;
    __shared__ int s_row;
    __shared__ long long s_base;
    __shared__ long long warp_sum[kThreads / 32];
    __shared__ float red_m[kWarps][8], red_l[kWarps][8];
    __shared__ float2 freq[kHeadDim / 2];  // (read by lane: constant memory is slow at that)

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&fullv[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        fence_mbar_init();
        abort_flag = 0;
        seg_bad = 0;
        seg_odd = 0;
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    const int half = P.rope.rot_dim / 2;
    if (tid < half) freq[tid] = P.rope.u[tid];
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
    const long long share = (total + gridDim.x - 1) / gridDim.x;
    Walk wk;
    wk.u = share * blockIdx.x;
    wk.end = wk.u + share < total ? wk.u + share : total;
    if (wk.u >= wk.end) return;
    if (wk.u >= before * P.Hkv && wk.u < (before + mine) * P.Hkv) {
        int b = b0;
        long long base = before * P.Hkv;
        for (;; ++b) {
            const long long n = P.Hkv * row_of(P, b).units();
            if (wk.u < base + n) break;
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
        // ------------------------------------------------------ TMA producer
        // Lane l copies chunk l % 4 (64 dims) of K (or V: bit 2) of piece l / 8
        // of a tile; a piece is what lies in one page.
        const int page = 1 << P.page_shift;
        const int piece_rows = page < kTile ? page : kTile;
        const int pieces = kTile / piece_rows;
        const int piece = lane >> 3, which = (lane >> 2) & 1, c = lane & 3;
        int it = 0;
        bool ok = true;
        while (ok && wk.load(P)) {
            const int32_t *row = P.table + static_cast<size_t>(wk.b) * P.max_pages;
            const int slot0 = wk.row.slot0();
            int ids = 0;
            for (int t = wk.t0; t < wk.t1; ++t) {
                // page numbers for the next 32 pieces, one per lane
                const int in = (t - wk.t0) * pieces & 31;
                if (in == 0) {
                    const int slot = slot0 + t * kTile + lane * piece_rows;
                    const int index = slot >> P.page_shift;
                    ids = P.n_pages;  // past the pool: the copy reads zeros
                    if (slot < wk.row.pos && (index + 1) << P.page_shift > wk.row.lo &&
                        slot < slot0 + wk.t1 * kTile) {
                        ids = row[index];
                        if (ids < 0 || ids >= P.n_pages) {
                            atomicOr(P.status, kErrPage);
                            ids = P.n_pages;
                        }
                    }
                }
                const int s = it % kStages;
                if (it >= kStages && lane == 0)
                    ok = mbar_wait(&empty[s], ((it / kStages) - 1) & 1, &abort_flag, P.status);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], kTileBytes);
                    mbar_arrive_expect_tx(&fullv[s], kTileBytes);
                }
                const int id = __shfl_sync(0xffffffffu, ids, (in + piece) & 31);
                __syncwarp();
                if (piece < pieces)
                    tma_load_4d(stages + s * kStageBytes + which * kTileBytes +
                                    c * (kTileBytes / 4) + piece * piece_rows * 128,
                                which ? &tm_v : &tm_k, which ? &fullv[s] : &full[s], c * 64,
                                (slot0 + t * kTile) & (page - 1), wk.g, id);
                ++it;
            }
        }
        __syncwarp();
        __syncthreads();
        // copies still in flight after an abort must land before the CTA ends
        if (lane == 0 && abort_flag) {
            for (int i = it > kStages ? it - kStages : 0; i < it; ++i) {
                mbar_wait_plain(&full[i % kStages], (i / kStages) & 1);
                mbar_wait_plain(&fullv[i % kStages], (i / kStages) & 1);
            }
        }
        return;
    }

    // ---------------------------------------------------------- consumers
    const size_t width = static_cast<size_t>(P.H + 2 * P.Hkv) * kHeadDim;
    const int arow = warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;  // K rows (ldmatrix)
    const int vrow = warp * 16 + (lane & 7) + (lane >> 4) * 8;        // V rows (ldmatrix.trans)
    const int h0 = 2 * (lane & 3), h1 = h0 + 1;                       // this thread's two heads
    for (int i = tid; i < 8 * (kHeadDim / 8); i += kWarps * 32)
        if (i >= P.G * (kHeadDim / 8))
            *reinterpret_cast<uint4 *>(qs + i * 8) = make_uint4(0, 0, 0, 0);
    int it = 0;
    bool aborted = false;  // the same in every consumer thread
    // The projections of a pair's new token -- q of the group's heads, the key,
    // the value -- and its gates, loaded a pair ahead: warp w brings rows w,
    // w + 4, ... of them.
    uint4 raw[3];
    float gate[2];
    auto fetch = [&](const Walk &w) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int hh = warp + i * kWarps;
            if (hh >= P.G + 2) break;
            const int head = hh < P.G ? w.g * P.G + hh : P.H + (hh - P.G) * P.Hkv + w.g;
            raw[i] = *reinterpret_cast<const uint4 *>(
                P.qkv + w.b * width + static_cast<size_t>(head) * kHeadDim + lane * 8);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int hq = warp + i * kRedHeads;
            if (hq < P.G) gate[i] = P.gate[static_cast<size_t>(w.b) * P.H + w.g * P.G + hq];
        }
    };
    Walk nx = wk;
    bool more = nx.load(P);
    if (more) fetch(nx);
    while (more) {
        wk = nx;
        const Row row = wk.row;
        // q and the new key, rotated and rounded to bf16, and the new value
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int hh = warp + i * kWarps;
            if (hh >= P.G + 2) break;
            __nv_bfloat16 *dst = hh < P.G ? qs + hh * kHeadDim : hh == P.G ? kn : vn;
            *reinterpret_cast<uint4 *>(dst + lane * 8) = raw[i];
        }
        const float gate_now[2] = {gate[0], gate[1]};
        more = nx.load(P);
        if (more) fetch(nx);
        consumer_bar();
        for (int k = tid; k < half; k += kWarps * 32) {
            float c, s;
            rope_cos_sin_fine(row.pos, freq[k], c, s);
            for (int hh = 0; hh <= P.G; ++hh) {
                __nv_bfloat16 *x = hh < P.G ? qs + hh * kHeadDim : kn;
                float y1, y2;
                rope_rotate(__bfloat162float(x[k]), __bfloat162float(x[k + half]), c, s, y1, y2);
                x[k] = __float2bfloat16_rn(y1);
                x[k + half] = __float2bfloat16_rn(y2);
            }
        }
        consumer_bar();
        // Q^T as the B operand of S^T = K Q^T: one (b0, b1) pair per 16 dims
        uint32_t qf[16][2];
        {
            const uint32_t qbase = smem_u32(qs);
#pragma unroll
            for (int ks = 0; ks < 16; ks += 2) {
                const uint32_t addr = qbase + (lane & 7) * (kHeadDim * 2) +
                                      (ks * 16 + (lane >> 3) * 8) * 2;
                ldmatrix_x4(addr, qf[ks][0], qf[ks][1], qf[ks + 1][0], qf[ks + 1][1]);
            }
        }
        float o[16][4];
#pragma unroll
        for (int db = 0; db < 16; ++db) o[db][0] = o[db][1] = o[db][2] = o[db][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        bool ok = !aborted;
        for (int t = wk.t0; ok && t < wk.t1; ++t, ++it) {
            const int s = it % kStages;
            ok = mbar_wait(&full[s], (it / kStages) & 1, &abort_flag, P.status);
            if (!ok) break;
            const uint32_t kt = smem_u32(stages + s * kStageBytes);
            const uint32_t vt = kt + kTileBytes;
            // S^T (16 slots x 8 heads) = K (16 x 256) Q^T (256 x 8)
            float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 16; ++ks) {
                const int gran = ((ks * 16) & 63) / 8 + (lane >> 4);
                const uint32_t addr = kt + (ks >> 2) * (kTileBytes / 4) + arow * 128 +
                                      ((gran ^ (arow & 7)) << 4);
                uint32_t a0, a1, a2, a3;
                ldmatrix_x4(addr, a0, a1, a2, a3);
                mma_bf16_16816(sc, a0, a1, a2, a3, qf[ks][0], qf[ks][1]);
            }
            // this thread's two slots (rows lane/4 and lane/4 + 8) and two heads
            const int first = row.slot0() + t * kTile + warp * 16;
            const int sa = first + (lane >> 2), sb = sa + 8;
            const bool va = sa >= row.lo && sa < row.pos, vb = sb >= row.lo && sb < row.pos;
            const float x0 = va ? sc[0] * kScaleLog2 : -INFINITY;
            const float x1 = va ? sc[1] * kScaleLog2 : -INFINITY;
            const float x2 = vb ? sc[2] * kScaleLog2 : -INFINITY;
            const float x3 = vb ? sc[3] * kScaleLog2 : -INFINITY;
            float n0 = fmaxf(x0, x2), n1 = fmaxf(x1, x3);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
                n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
            }
            n0 = fmaxf(n0, m0);
            n1 = fmaxf(n1, m1);
            const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
            const float r0 = fast_exp2(m0 - z0), r1 = fast_exp2(m1 - z1);
            const float p0 = fast_exp2(x0 - z0), p1 = fast_exp2(x1 - z1);
            const float p2 = fast_exp2(x2 - z0), p3 = fast_exp2(x3 - z1);
            l0 = l0 * r0 + p0 + p2;
            l1 = l1 * r1 + p1 + p3;
            m0 = n0;
            m1 = n1;
#pragma unroll
            for (int db = 0; db < 16; ++db) {
                o[db][0] *= r0;
                o[db][1] *= r1;
                o[db][2] *= r0;
                o[db][3] *= r1;
            }
            // P^T as the B operand of O^T += V^T P^T, in two bf16 terms: the
            // product's operands have V's type, one term would round the
            // probabilities by 2^-9, and the second costs no time while HBM
            // bounds the step.  The sums l stay in 32 bits.
            const uint32_t ph0 = pack_bf16x2(p0, p1), ph1 = pack_bf16x2(p2, p3);
            const uint32_t pb0 = movmatrix_trans(ph0), pb1 = movmatrix_trans(ph1);
            const uint32_t pl0 =
                movmatrix_trans(pack_bf16x2(p0 - bf16_lo(ph0), p1 - bf16_hi(ph0)));
            const uint32_t pl1 =
                movmatrix_trans(pack_bf16x2(p2 - bf16_lo(ph1), p3 - bf16_hi(ph1)));
            ok = mbar_wait(&fullv[s], (it / kStages) & 1, &abort_flag, P.status);
            if (!ok) break;
            // Slots that hold no visible token may hold anything, and 0 * NaN is
            // NaN: this warp zeroes those of its V rows.
            if (first < row.lo || first + 16 > row.pos) {
                uint8_t *vrows = stages + s * kStageBytes + kTileBytes;
                for (int rr = 0; rr < 16; ++rr) {
                    if (first + rr >= row.lo && first + rr < row.pos) continue;
                    *reinterpret_cast<uint4 *>(vrows + (lane >> 3) * (kTileBytes / 4) +
                                               (warp * 16 + rr) * 128 + (lane & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                // the stage is refilled by TMA later: order these writes first
                fence_proxy_async_smem();
                __syncwarp();
            }
#pragma unroll
            for (int db = 0; db < 16; ++db) {
                const int gran = ((db * 16) & 63) / 8 + ((lane >> 3) & 1);
                const uint32_t addr = vt + (db >> 2) * (kTileBytes / 4) + vrow * 128 +
                                      ((gran ^ (vrow & 7)) << 4);
                uint32_t a0, a1, a2, a3;
                ldmatrix_x4_trans(addr, a0, a1, a2, a3);
                mma_bf16_16816(o[db], a0, a1, a2, a3, pb0, pb1);
                mma_bf16_16816(o[db], a0, a1, a2, a3, pl0, pl1);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }

        // ------------------------------------------------------ join the warps
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, off);
            l1 += __shfl_xor_sync(0xffffffffu, l1, off);
        }
        if (lane < 4) {
            red_m[warp][h0] = m0;
            red_m[warp][h1] = m1;
            red_l[warp][h0] = l0;
            red_l[warp][h1] = l1;
        }
        // (a product with zero is NaN where a sum is not finite)
        float odd0 = 0.f, odd1 = 0.f;
#pragma unroll
        for (int db = 0; db < 16; ++db) {
            odd0 += (o[db][0] + o[db][2]) * 0.f;
            odd1 += (o[db][1] + o[db][3]) * 0.f;
        }
        if ((isnan(odd0) && isfinite(l0)) || (isnan(odd1) && isfinite(l1))) seg_odd = 1;
        if (!ok) seg_bad = 1;
        consumer_bar();
        aborted = seg_bad != 0;  // written before the barrier, never reset
        const bool odd = seg_odd != 0 && !aborted;
        float M0 = red_m[0][h0], M1 = red_m[0][h1];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            M0 = fmaxf(M0, red_m[w][h0]);
            M1 = fmaxf(M1, red_m[w][h1]);
        }
        const float s0 = M0 == -INFINITY ? 0.f : fast_exp2(m0 - M0);
        const float s1 = M1 == -INFINITY ? 0.f : fast_exp2(m1 - M1);
        // head hq of this warp, lane l its dims 8l..8l+7; the sums of the warps
        // go through shared memory kRedHeads heads at a time
        HeadState st[2];
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            if (pass * kRedHeads >= P.G) break;
            if (pass) consumer_bar();  // the heads before are read
            if ((lane & 3) >> 1 == pass) {
#pragma unroll
                for (int db = 0; db < 16; ++db) {
                    float *dst = red_o + (warp * kRedHeads + (h0 & 3)) * kHeadDim + db * 16 +
                                 (lane >> 2);
                    dst[0] = o[db][0] * s0;
                    dst[8] = o[db][2] * s0;
                    dst[kHeadDim] = o[db][1] * s1;
                    dst[kHeadDim + 8] = o[db][3] * s1;
                }
            }
            consumer_bar();
            const int hq = warp + pass * kRedHeads;
            HeadState &h = st[pass];
            h.m = -INFINITY;
            h.l = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) h.o[i] = 0.f;
            if (hq < P.G && !aborted) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) h.m = fmaxf(h.m, red_m[w][hq]);
                if (h.m != -INFINITY)
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        h.l += red_l[w][hq] * fast_exp2(red_m[w][hq] - h.m);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 *src = reinterpret_cast<const float4 *>(
                        red_o + (w * kRedHeads + warp) * kHeadDim + lane * 8);
                    const float4 a = src[0], c = src[1];
                    const float v[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
                    add_scaled(h, 1.f, v);
                }
            }
        }

        if (tid == 0) seg_odd = 0;  // (everyone has read it: a barrier lies between)
        if (odd) {
            // the values of this stretch that are not finite, dims 8l..8l+7 in every warp
            float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            const int at = row.slot0() + wk.t0 * kTile;
            const int end = row.slot0() + wk.t1 * kTile;
            sum_nonfinite(P, wk.b, wk.g, at > row.lo ? at : row.lo, end < row.pos ? end : row.pos,
                          warp, lane * 8, s);
            consumer_bar();  // the heads' sums are read
#pragma unroll
            for (int j = 0; j < 8; ++j) red_o[warp * kHeadDim + lane * 8 + j] = s[j];
            consumer_bar();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s[j] += red_o[w * kHeadDim + lane * 8 + j];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    // (with scores of -inf alone the weights are zero in earnest)
                    if (warp + i * kRedHeads < P.G && st[i].m != -INFINITY &&
                        !isfinite(s[j]) && !isfinite(st[i].o[j]))
                        st[i].o[j] = s[j];
            }
        }

        // ------------------------------------------------------ finish or hand over
        const int c0 = static_cast<int>((wk.first + kPairCost) / share);
        const int c1 = static_cast<int>((wk.first + row.units() - 1) / share);
        bool finish = c0 == c1;
        if (!finish) {
            // this CTA's partial state, then the count
            const int place = share * blockIdx.x < wk.first ? 1 : 0;  // not its first pair
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int hq = warp + i * kRedHeads;
                if (hq >= P.G) break;
                const size_t at = (static_cast<size_t>(blockIdx.x) * 2 + place) * P.G + hq;
                float4 *dst = reinterpret_cast<float4 *>(P.part_o + at * kHeadDim + lane * 8);
                dst[0] = make_float4(st[i].o[0], st[i].o[1], st[i].o[2], st[i].o[3]);
                dst[1] = make_float4(st[i].o[4], st[i].o[5], st[i].o[6], st[i].o[7]);
                if (lane == 0)
                    reinterpret_cast<float2 *>(P.part_ml)[at] = make_float2(st[i].m, st[i].l);
            }
            __threadfence();
            consumer_bar();
            if (tid == 0) {
                // c0 is the first CTA of one shared pair at most, which the
                // counter is named by
                unsigned *word = P.counters + (c0 >> 2);
                const int shift = (c0 & 3) * 8;
                last_cta = (atomicAdd(word, 1u << shift) >> shift & 255u) ==
                           static_cast<unsigned>(c1 - c0);
                // everyone has counted: back to 0 for the next call
                if (last_cta) atomicAnd(word, ~(255u << shift));
            }
            consumer_bar();
            finish = last_cta != 0;
            if (finish) {
                __threadfence();  // the others' states are read after the count
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int hq = warp + i * kRedHeads;
                    if (hq >= P.G) break;
                    HeadState &h = st[i];
                    auto at = [&](int cta) {
                        const int pl = static_cast<long long>(cta) * share < wk.first ? 1 : 0;
                        return (static_cast<size_t>(cta) * 2 + pl) * P.G + hq;
                    };
                    // kJoin states at a time, all their loads in flight
                    h.m = -INFINITY;
                    h.l = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) h.o[j] = 0.f;
                    for (int cta = c0; cta <= c1; cta += kJoin) {
                        float2 ml[kJoin];
                        float4 x[kJoin], y[kJoin];
#pragma unroll
                        for (int k = 0; k < kJoin; ++k) {
                            ml[k] = make_float2(-INFINITY, 0.f);
                            x[k] = y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (cta + k > c1) continue;
                            const size_t a = at(cta + k);
                            ml[k] = __ldcg(reinterpret_cast<const float2 *>(P.part_ml) + a);
                            const float4 *src = reinterpret_cast<const float4 *>(
                                P.part_o + a * kHeadDim + lane * 8);
                            x[k] = __ldcg(src);
                            y[k] = __ldcg(src + 1);
                        }
                        float m = h.m;
#pragma unroll
                        for (int k = 0; k < kJoin; ++k) m = fmaxf(m, ml[k].x);
                        const float z = m == -INFINITY ? 0.f : m;
                        const float wo = fast_exp2(h.m - z);
                        h.m = m;
                        h.l *= wo;
#pragma unroll
                        for (int j = 0; j < 8; ++j) h.o[j] *= wo;
#pragma unroll
                        for (int k = 0; k < kJoin; ++k) {
                            const float w = fast_exp2(ml[k].x - z);
                            const float v[8] = {x[k].x, x[k].y, x[k].z, x[k].w,
                                                y[k].x, y[k].y, y[k].z, y[k].w};
                            h.l += ml[k].y * w;
                            add_scaled(h, w, v);
                        }
                    }
                    float any = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) any += h.o[j] * 0.f;
                    if (isnan(any)) {
                        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        for (int cta = c0; cta <= c1; ++cta) {
                            const float4 *src = reinterpret_cast<const float4 *>(
                                P.part_o + at(cta) * kHeadDim + lane * 8);
                            const float4 a = __ldcg(src), c = __ldcg(src + 1);
                            const float v[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
                            for (int j = 0; j < 8; ++j) s[j] += nonfinite_part(v[j]);
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (!isfinite(s[j])) h.o[j] = s[j];
                    }
                }
            }
        }
        if (finish) {
            // the new token joins, the gate applies
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int hq = warp + i * kRedHeads;
                if (hq >= P.G) break;
                HeadState &h = st[i];
                const int head = wk.g * P.G + hq;
                const uint4 qv = *reinterpret_cast<const uint4 *>(qs + hq * kHeadDim + lane * 8);
                const uint4 kv = *reinterpret_cast<const uint4 *>(kn + lane * 8);
                const uint4 vv = *reinterpret_cast<const uint4 *>(vn + lane * 8);
                const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w}, kw[4] = {kv.x, kv.y, kv.z, kv.w};
                const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
                float dot = 0.f, v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = bf16_lo(vw[j]);
                    v[2 * j + 1] = bf16_hi(vw[j]);
                    dot = fmaf(bf16_lo(qw[j]), bf16_lo(kw[j]), dot);
                    dot = fmaf(bf16_hi(qw[j]), bf16_hi(kw[j]), dot);
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    dot += __shfl_xor_sync(0xffffffffu, dot, off);
                const float x = dot * kScaleLog2;
                const float m = fmaxf(h.m, x);
                const float z = m == -INFINITY ? 0.f : m;
                const float wo = h.m == -INFINITY ? 0.f : fast_exp2(h.m - z), wn = fast_exp2(x - z);
                const float scale = gate_act(gate_now[i], P.gate_mode) / (h.l * wo + wn);
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] = (h.o[j] * wo + v[j] * wn) * scale;
                    const float s = nonfinite_part(h.o[j]) + nonfinite_part(v[j]);
                    if (!isfinite(s)) y[j] = s * scale;
                }
                *reinterpret_cast<uint4 *>(
                    P.out + (static_cast<size_t>(wk.b) * P.H + head) * kHeadDim + lane * 8) =
                    make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                               pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
                if (hq == 0) {
                    // the new token's slot: every read of this pair is done
                    const int id = P.table[static_cast<size_t>(wk.b) * P.max_pages +
                                           (row.pos >> P.page_shift)];
                    if (id < 0 || id >= P.n_pages) {
                        if (lane == 0) atomicOr(P.status, kErrPage);
                    } else {
                        const size_t off =
                            (((static_cast<size_t>(id) * P.Hkv + wk.g) << P.page_shift) +
                             (row.pos & ((1 << P.page_shift) - 1))) * kHeadDim + lane * 8;
                        *reinterpret_cast<uint4 *>(P.k_pages + off) = kv;
                        *reinterpret_cast<uint4 *>(P.v_pages + off) = vv;
                    }
                }
            }
        }
        consumer_bar();  // q, the new token and the sums are read: the next pair may come
    }
    grid_dep_launch();
    __syncthreads();  // with the producer
}

// ---------------------------------------------------------------- launcher

cudaError_t launch_decode_paged(const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                const PagedParams &P, int grid, cudaStream_t stream) {
    cudaError_t err = cudaFuncSetAttribute(
        decode_paged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (err != cudaSuccess) return err;
    return launch_overlapped(decode_paged_kernel, dim3(grid), dim3(kThreads), kSmemBytes, stream,
                             tm_k, tm_v, P);
}

}  // namespace spark
