// prefill.cu -- prefill of the gated GQA attention core on the 5th-generation
// tensor cores (tcgen05, accumulators in TMEM, operands staged by TMA).
//
// Spark-X2.5 architecture (4B / 1.7B): §3 Eq. 1 (softmax(QK^T/16) V times the
// per-head sigmoid gate), §4 layered RoPE, §2 causal / sliding-window masks.
//
// Two kernels on one stream:
//   prefill_rope_k_kernel  writes the leading rot_w = roundup(rot_dim, 64)
//       dims of every key, rotated, to a workspace [B][Hkv][T][rot_w].  The
//       other key dims and all of V are read by TMA straight from qkv.
//   prefill_attn_kernel    one CTA per (query tile, KV head, sequence).  A
//       query tile is 128 rows = (128/G) tokens x the G query heads that share
//       the KV head, so every K/V byte brought on chip serves all G heads.
//       Warp roles:
//         warp 0       TMA producer (Q tile once, then K and V through a ring
//                      of 16 KB slots)
//         warp 1       TMEM owner and QK^T issuer (one thread)
//         warp 2       P*V issuer (one thread)
//         warps 4..11  softmax, two warpgroups: query row i (TMEM lane i) is
//                      shared by thread i of each; warpgroup w owns score
//                      columns [64w, 64w+64) and output dims [128w, 128w+128)
//       TMEM (512 columns): O [128 x 256 fp32] in columns 0..255, two score
//       buffers S0/S1 [128 x 128 fp32] in 256..383 and 384..511.  The
//       probabilities P (bf16 pairs) overwrite columns 0..31 (keys 0..63) and
//       64..95 (keys 64..127) of their score buffer, each warpgroup inside the
//       columns it read, and feed P*V as the TMEM A operand.  QK^T of tile j+1 runs on
//       the tensor cores while the softmax of tile j runs on the CUDA cores.
//       Q is rotated in shared memory by the softmax threads (each its own
//       row) before the first product.  Key tiles wholly outside the causal
//       band / window are never visited; boundary tiles are masked per element.
//       Online softmax in base 2 with a lazy rescale: the reference maximum
//       moves only when a row's maximum grows by more than 2^8.
#include <type_traits>

#include "common.cuh"

namespace spark {

// ---------------------------------------------------------------- K RoPE

constexpr int kRopeThreads = 256;

__global__ void __launch_bounds__(kRopeThreads) prefill_rope_k_kernel(
    const __grid_constant__ PrefillParams P) {
    const int r = P.rope.rot_dim, half = r / 2;
    const int n_rot = half / 8;              // groups of 8 rotated pairs
    const int n_copy = (P.rot_w - r) / 8;    // groups of 8 dims copied unrotated
    const int items = n_rot + n_copy;
    grid_dep_wait();  // qkv and pos may come from the previous kernel
    grid_dep_launch();
    const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const long long row = idx / items;
    const int it = static_cast<int>(idx % items);
    if (row >= static_cast<long long>(P.B) * P.T) return;
    const int b = static_cast<int>(row / P.T), t = static_cast<int>(row % P.T);
    const size_t width = static_cast<size_t>(P.H + 2 * P.Hkv) * kHeadDim;
    const __nv_bfloat16 *src = P.qkv + row * width + static_cast<size_t>(P.H) * kHeadDim;
    __nv_bfloat16 *dst0 = P.krot + (static_cast<size_t>(b) * P.Hkv * P.T + t) * P.rot_w;
    const size_t head_stride = static_cast<size_t>(P.T) * P.rot_w;
    if (it < n_rot) {
        const int k0 = it * 8;
        const int p = P.pos[row];
        float c[8], s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) rope_cos_sin(p, P.rope.u[k0 + i], c[i], s[i]);
        for (int g = 0; g < P.Hkv; ++g) {
            const uint4 a = *reinterpret_cast<const uint4 *>(src + g * kHeadDim + k0);
            const uint4 bb = *reinterpret_cast<const uint4 *>(src + g * kHeadDim + k0 + half);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
            const uint32_t bw[4] = {bb.x, bb.y, bb.z, bb.w};
            uint32_t ya[4], yb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y1l, y2l, y1h, y2h;
                rope_rotate(bf16_lo(aw[i]), bf16_lo(bw[i]), c[2 * i], s[2 * i], y1l, y2l);
                rope_rotate(bf16_hi(aw[i]), bf16_hi(bw[i]), c[2 * i + 1], s[2 * i + 1], y1h, y2h);
                ya[i] = pack_bf16x2(y1l, y1h);
                yb[i] = pack_bf16x2(y2l, y2h);
            }
            __nv_bfloat16 *dst = dst0 + g * head_stride;
            *reinterpret_cast<uint4 *>(dst + k0) = make_uint4(ya[0], ya[1], ya[2], ya[3]);
            *reinterpret_cast<uint4 *>(dst + k0 + half) = make_uint4(yb[0], yb[1], yb[2], yb[3]);
        }
    } else {
        const int d0 = r + (it - n_rot) * 8;
        for (int g = 0; g < P.Hkv; ++g)
            *reinterpret_cast<uint4 *>(dst0 + g * head_stride + d0) =
                *reinterpret_cast<const uint4 *>(src + g * kHeadDim + d0);
    }
}

// ---------------------------------------------------------------- KV cache fill

// Stores every token's rotated K (all 256 dims) and its V in the decode cache,
// the step a model takes while it prefills (past_key_values.update): token t
// goes to slot t of a full layer's cache, or to slot t mod cap of a sliding
// layer's ring, where only the last cap tokens survive.  One thread per
// (token, group of 8 rotated pairs / 8 copied K dims / 8 V dims), looping over
// KV heads so each angle is computed once per (token, pair).
__global__ void __launch_bounds__(kRopeThreads) prefill_store_kv_kernel(
    const __grid_constant__ PrefillParams P) {
    grid_dep_wait();
    grid_dep_launch();
    const int r = P.rope.rot_dim, half = r / 2;
    const int n_rot = half / 8, n_kcopy = (kHeadDim - r) / 8, n_v = kHeadDim / 8;
    const int items = n_rot + n_kcopy + n_v;
    const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const long long row = idx / items;
    const int it = static_cast<int>(idx % items);
    if (row >= static_cast<long long>(P.B) * P.T) return;
    const int b = static_cast<int>(row / P.T), t = static_cast<int>(row % P.T);
    if (P.kind == kLayerSliding && t < P.T - P.cap) return;  // overwritten later in the ring
    const long long a = (P.start ? static_cast<long long>(P.start[b]) : 0) + t;  // absolute index
    if (a < 0 || (P.kind == kLayerFull && a >= P.cap)) {
        if (it == 0 && t == 0) atomicOr(P.status, kErrPosition);
        return;
    }
    const long long slot = (P.kind == kLayerFull) ? a : a % P.cap;
    const size_t width = static_cast<size_t>(P.H + 2 * P.Hkv) * kHeadDim;
    const __nv_bfloat16 *src_k = P.qkv + row * width + static_cast<size_t>(P.H) * kHeadDim;
    const __nv_bfloat16 *src_v = src_k + static_cast<size_t>(P.Hkv) * kHeadDim;
    const size_t head_stride = static_cast<size_t>(P.cap) * kHeadDim;
    const size_t base = (static_cast<size_t>(b) * P.Hkv * P.cap + slot) * kHeadDim;
    if (it < n_rot) {
        const int k0 = it * 8;
        const int p = P.pos[row];
        float c[8], s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) rope_cos_sin(p, P.rope.u[k0 + i], c[i], s[i]);
        for (int g = 0; g < P.Hkv; ++g) {
            const uint4 a = *reinterpret_cast<const uint4 *>(src_k + g * kHeadDim + k0);
            const uint4 bb = *reinterpret_cast<const uint4 *>(src_k + g * kHeadDim + k0 + half);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
            const uint32_t bw[4] = {bb.x, bb.y, bb.z, bb.w};
            uint32_t ya[4], yb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y1l, y2l, y1h, y2h;
                rope_rotate(bf16_lo(aw[i]), bf16_lo(bw[i]), c[2 * i], s[2 * i], y1l, y2l);
                rope_rotate(bf16_hi(aw[i]), bf16_hi(bw[i]), c[2 * i + 1], s[2 * i + 1], y1h, y2h);
                ya[i] = pack_bf16x2(y1l, y1h);
                yb[i] = pack_bf16x2(y2l, y2h);
            }
            __nv_bfloat16 *dst = P.k_cache + base + g * head_stride;
            *reinterpret_cast<uint4 *>(dst + k0) = make_uint4(ya[0], ya[1], ya[2], ya[3]);
            *reinterpret_cast<uint4 *>(dst + k0 + half) = make_uint4(yb[0], yb[1], yb[2], yb[3]);
        }
    } else if (it < n_rot + n_kcopy) {
        const int d0 = r + (it - n_rot) * 8;
        for (int g = 0; g < P.Hkv; ++g)
            *reinterpret_cast<uint4 *>(P.k_cache + base + g * head_stride + d0) =
                *reinterpret_cast<const uint4 *>(src_k + g * kHeadDim + d0);
    } else {
        const int d0 = (it - n_rot - n_kcopy) * 8;
        for (int g = 0; g < P.Hkv; ++g)
            *reinterpret_cast<uint4 *>(P.v_cache + base + g * head_stride + d0) =
                *reinterpret_cast<const uint4 *>(src_v + g * kHeadDim + d0);
    }
}

// Zeroes the cache slots that the last key tile of a chunked prefill may read
// past the chunk end but that no token has written yet (a full layer's future
// slots, or ring slots on the first pass): their probabilities are 0, but a
// never-written slot may hold NaN bit patterns and 0 * NaN is NaN in P*V.
// One block per sequence.
__global__ void __launch_bounds__(kRopeThreads) cache_zero_tail_kernel(
    const __grid_constant__ PrefillParams P) {
    grid_dep_wait();
    grid_dep_launch();
    const int b = blockIdx.x;
    if (P.start[b] < 0) return;  // flagged by the store kernel
    const long long a_end = static_cast<long long>(P.start[b]) + P.T;
    const long long a_stop = (a_end + 127) / 128 * 128;
    const long long last = a_stop < P.cap ? a_stop : P.cap;  // slots a_end..last-1
    const int per_slot = P.Hkv * (kHeadDim / 8);             // 16-byte words per slot and tensor
    for (long long w = threadIdx.x; w < (last - a_end) * per_slot; w += blockDim.x) {
        const long long j = a_end + w / per_slot;
        const int g = static_cast<int>((w % per_slot) / (kHeadDim / 8));
        const int d0 = static_cast<int>(w % (kHeadDim / 8)) * 8;
        const size_t off = ((static_cast<size_t>(b) * P.Hkv + g) * P.cap + j) * kHeadDim + d0;
        *reinterpret_cast<uint4 *>(P.k_cache + off) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(P.v_cache + off) = make_uint4(0, 0, 0, 0);
    }
}

// ---------------------------------------------------------------- attention

constexpr int kBM = 128;                  // query rows per tile
constexpr int kBN = 128;                  // keys per tile
constexpr int kSlotBytes = 16384;         // ring slot: 128 keys x 64 dims (K) or 32 keys x 256 (V);
                                          // from pages 32 keys x 256 (both)
constexpr int kSlots = 8;
constexpr int kGroupBytes = 4096;         // from pages: 8 keys, as 4 chunks of 64 dims
constexpr int kQBytes = 4 * kSlotBytes;   // 128 rows x 256 dims, as 4 chunks of 64 dims
constexpr int kAttnThreads = 384;
constexpr int kPrefetchMaxTiles = 8;      // CTAs this short pull the next wave's Q into L2
constexpr int kSoftmaxWarp0 = 4;
constexpr int kSoftmaxThreads = 256;        // two warpgroups, 64 score columns each
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256;

// barriers
constexpr int kBarQFull = 0;
constexpr int kBarQReady = 1;
constexpr int kBarSlotFull = 2;                 // kSlots of them
constexpr int kBarSlotEmpty = 2 + kSlots;       // kSlots of them
constexpr int kBarSFull = 2 + 2 * kSlots;       // 2
constexpr int kBarPReady = 4 + 2 * kSlots;      // 2
constexpr int kBarODone = 6 + 2 * kSlots;
constexpr int kBarMmaDrain = 7 + 2 * kSlots;
constexpr int kBarOFinal = 8 + 2 * kSlots;      // every P*V done (one phase per CTA)
constexpr int kBarMaxX = 9 + 2 * kSlots;        // 2: half-row maxima exchanged (per tile parity)
constexpr int kNumBars = 11 + 2 * kSlots;

constexpr int kAttnSmemBytes = 1024 + kQBytes + kSlots * kSlotBytes + 256;

constexpr uint32_t kIdescQK = idesc_bf16_f32(kBM, kBN, 0, 0);        // Q, K both K-major
constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, kHeadDim, 0, 1);   // V is N(=dim)-major

// Byte offset of 16-byte granule `gran` (0..31 across the 256 dims) of row
// `row` inside a tile stored as 4 chunks of [rows][64 dims] with the 128-byte
// TMA swizzle (granule index XOR row mod 8 inside each 1024-byte atom).
__device__ __forceinline__ uint32_t sw128_offset(int row, int gran) {
    return static_cast<uint32_t>((gran >> 3) * kSlotBytes + row * 128 +
                                 (((gran & 7) ^ (row & 7)) << 4));
}

// RoPE of one query row held in shared memory (the 128-byte-swizzled Q tile),
// for the pair groups of warpgroup `wg`.  The rotated query is rounded to bf16
// once: it is an operand of K's type.  Its angle may be off by 2e-7 rad
// (rope_turns), which moves a query by a ten-thousandth of that rounding; keys
// that are stored in pages take it finer (rope_cos_sin_fine), so that their
// bits agree with 32-bit products.  The G lanes holding the G heads of
// one token compute 8/G of the 8 angles of a group each and exchange them by
// shuffles, so each angle is computed once per token.
template <int G>
__device__ __forceinline__ void rotate_q_row(uint8_t *qbuf, int row, int lane, int wg, int pos,
                                             const RopeTable &rope) {
    const int half = rope.rot_dim / 2;
    const int base = lane & ~(G - 1), sub = lane & (G - 1);
    for (int k0 = wg * 8; k0 < half; k0 += 16) {
        float cw[8 / G], sw[8 / G];
#pragma unroll
        for (int m = 0; m < 8 / G; ++m) rope_cos_sin(pos, rope.u[k0 + sub + G * m], cw[m], sw[m]);
        float c[8], s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = __shfl_sync(0xffffffffu, cw[i / G], base + (i % G));
            s[i] = __shfl_sync(0xffffffffu, sw[i / G], base + (i % G));
        }
        uint4 *pa = reinterpret_cast<uint4 *>(qbuf + sw128_offset(row, k0 / 8));
        uint4 *pb = reinterpret_cast<uint4 *>(qbuf + sw128_offset(row, (k0 + half) / 8));
        const uint4 a = *pa, bb = *pb;
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
        const uint32_t bw[4] = {bb.x, bb.y, bb.z, bb.w};
        uint32_t ya[4], yb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y1l, y2l, y1h, y2h;
            rope_rotate(bf16_lo(aw[i]), bf16_lo(bw[i]), c[2 * i], s[2 * i], y1l, y2l);
            rope_rotate(bf16_hi(aw[i]), bf16_hi(bw[i]), c[2 * i + 1], s[2 * i + 1], y1h, y2h);
            ya[i] = pack_bf16x2(y1l, y1h);
            yb[i] = pack_bf16x2(y2l, y2h);
        }
        *pa = make_uint4(ya[0], ya[1], ya[2], ya[3]);
        *pb = make_uint4(yb[0], yb[1], yb[2], yb[3]);
    }
}

__device__ __forceinline__ void named_bar(int id, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// Where the keys and values come from: the fused projection (one-shot
// prefill), or the KV cache of a chunked prefill -- a full layer's, one slot
// per token, or a sliding layer's ring.  In a chunked prefill the queries are
// chunk tokens at absolute index start[b] + t, the cache already holds this
// chunk's keys and values, and tm_kv_k / tm_kv_v map the caches.  Each source
// is its own instantiation, so that no kernel carries another's addressing
// (the ring's slot arithmetic would sit in every inlined load of the
// producer).
//
// The packed sources: sequences of different lengths behind one another
// (common.cuh: PackedInfo), their keys and values in the fused projection, or
// in pages that hold the chunk and what came before it.  A key tile of the
// last or first kind of place may then reach into another sequence, into slots
// that no token was written to, or behind the window, and all of a tile's
// queries share one V operand: a value there that is not finite would turn its
// zero probability into NaN.  The softmax warps clear those rows in shared
// memory before they hand the tile's probabilities over (clean_v_rows, boundary
// tiles only; one warp doing it alone took 10 us a tile).
enum KvSource : int {
    kKvFromQkv = 0,
    kKvFromCache = 1,
    kKvFromRing = 2,
    kKvPacked = 3,
    kKvPages = 4
};

// The layer kind is a template argument too, so that a kernel carries no
// arithmetic of the other kind; kKindAny reads it from P.kind instead.  Which
// instantiation serves which layer was chosen by timing: the kind-specialised
// builds are faster for both chunked kinds and the one-shot sliding layer,
// the generic one for the one-shot full layer.
constexpr int kKindAny = -1;

// Whether a packed pair of bf16 holds a value that is not finite; and the pair
// with such values replaced by zero.
__device__ __forceinline__ uint32_t nonfinite_mask(uint32_t w) {
    return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) |
           ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// The rows of a key tile (kBN keys from key0) for the queries a0..a_last:
// [none_lo, none_hi) are seen by some of them, [all_lo, all_hi) by all.
struct TileRows {
    int none_lo, none_hi, all_lo, all_hi;
};

__device__ __forceinline__ TileRows tile_rows(int kind, int window, int key0, int a0, int a_last) {
    auto clamp = [](int x) { return x < 0 ? 0 : (x < kBN ? x : kBN); };
    TileRows t;
    t.none_lo = kind == kLayerSliding ? clamp(a0 - window + 1 - key0) : 0;
    t.all_lo = kind == kLayerSliding ? clamp(a_last - window + 1 - key0) : 0;
    t.all_hi = clamp(a0 + 1 - key0);
    t.none_hi = clamp(a_last + 1 - key0);
    return t;
}

// A softmax warp's share of V of a key tile that needs a mask (in the four
// ring slots from `use` on): the rows that not every query sees.  Those that no
// query sees become zero; in the others, values that are not finite become zero
// (returns true if this lane met one: the epilogue gives it back to the queries
// that see it).  Rows [finite_lo, finite_hi) hold finite values only and are
// left alone (pages).
template <bool kPages>
__device__ __forceinline__ bool clean_v_rows(uint8_t *ring, int use, const TileRows &t,
                                             int finite_lo, int finite_hi, int w, int lane) {
    // Row w + 8 i is at a constant distance from row w (`use` is a multiple of
    // 4, so the slots do not wrap): bit i of a mask stands for it, and the
    // passes unroll to plain stores and loads.
    uint8_t *base = ring + (use % kSlots) * kSlotBytes +
                    (lane >> 3) * (kPages ? 1024 : kSlotBytes / 2) + w * 128 + (lane & 7) * 16;
    auto at = [&](int i) {
        return reinterpret_cast<uint4 *>(
            base + (kPages ? i * kGroupBytes : (i >> 3) * 2 * kSlotBytes + (i & 7) * 1024));
    };
    auto below = [&](int row) -> uint32_t {  // rows w + 8 i < row
        const int n = (row - w + 7) >> 3;
        return (1u << (n < 0 ? 0 : (n < 16 ? n : 16))) - 1u;
    };
    const uint32_t unseen = below(t.none_lo) | ~below(t.none_hi);
    const uint32_t all = below(t.all_hi) & ~below(t.all_lo);
    const uint32_t look = kPages ? ~(below(finite_hi) & ~below(finite_lo)) & 0xFFFFu : 0xFFFFu;
    const uint32_t none = unseen & look;
    const uint32_t part = ~(unseen | all) & look;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (none >> i & 1u) *at(i) = make_uint4(0, 0, 0, 0);
    bool found = false;
#pragma unroll
    for (int i0 = 0; i0 < 16; i0 += 4) {
        if (!(part >> i0 & 15u)) continue;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = part >> (i0 + i) & 1u ? *at(i0 + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // an exponent of all ones carries into the sign's place
            const uint32_t hit = ((v[i].x & 0x7F807F80u) + 0x00800080u) |
                                 ((v[i].y & 0x7F807F80u) + 0x00800080u) |
                                 ((v[i].z & 0x7F807F80u) + 0x00800080u) |
                                 ((v[i].w & 0x7F807F80u) + 0x00800080u);
            if (hit & 0x80008000u) {
                *at(i0 + i) = make_uint4(
                    v[i].x & ~nonfinite_mask(v[i].x), v[i].y & ~nonfinite_mask(v[i].y),
                    v[i].z & ~nonfinite_mask(v[i].z), v[i].w & ~nonfinite_mask(v[i].w));
                found = true;
            }
        }
    }
    return found;
}

// The same for tile j of ntiles, once its V has landed; false after a wait that
// ran out.
template <bool kPages>
__device__ __forceinline__ bool clean_tile(uint8_t *ring, uint64_t *bars,
                                           volatile int *abort_flag, unsigned *status,
                                           int *cleaned_any, int j, int ntiles,
                                           int kind, int window, int key0, int a0, int a_last,
                                           int finite_lo, int finite_end, int w, int lane) {
    // V_j comes after min(ntiles, j + 2) K tiles and j V tiles.  The slots' use
    // before it was K_j (the last tile: S_j says that it landed), K0 (the first)
    // or V_{j-1}, which P*V of tile j-1 says: a parity wait must not begin a
    // phase early.
    const int use = 4 * ((ntiles < j + 2 ? ntiles : j + 2) + j);
    bool ok = true;
    if (j > 0 && j + 1 < ntiles) ok = mbar_wait(&bars[kBarODone], (j - 1) & 1, abort_flag, status);
    for (int vs = 0; ok && vs < 4; ++vs)
        ok = mbar_wait(&bars[kBarSlotFull + (use + vs) % kSlots], ((use + vs) / kSlots) & 1,
                       abort_flag, status);
    if (!ok) return false;
    if (clean_v_rows<kPages>(ring, use, tile_rows(kind, window, key0, a0, a_last),
                             finite_lo - key0, finite_end - key0, w, lane))
        *cleaned_any = 1;
    fence_proxy_async_smem();
    return true;
}

// The same out of line: the softmax loop needs it only on boundary tiles, and
// packed only where a value is not finite.  Inlined, a packed sliding prompt of
// 8192 tokens takes 137.5 us instead of 136, one over pages of 16 158 instead
// of 157.
template <bool kPages>
__device__ __noinline__ bool clean_tile_call(uint8_t *ring, uint64_t *bars,
                                             volatile int *abort_flag, unsigned *status,
                                             int *cleaned_any, int j, int ntiles, int kind,
                                             int window, int key0, int a0, int a_last, int w,
                                             int lane, int finite_lo = 0, int finite_end = 0) {
    return clean_tile<kPages>(ring, bars, abort_flag, status, cleaned_any, j, ntiles, kind, window,
                              key0, a0, a_last, finite_lo, finite_end, w, lane);
}

// The copies of a packed source's key and value tiles into the ring, by one
// thread in the order of the issuers: K0, K1, then V_j and K_{j+2} for every
// tile j.  A V tile is two halves of 64 keys, each in two slots of two 64-dim
// chunks (the other sources: four slots of 32 keys): the copy engine takes
// about as long for a box of 32 rows as for one of 64.
//
// With pages, a K or V tile is in groups of 8 keys, each 4 KB of the pool, and
// a box takes several of them: it brings its keys' 64-dim chunks one behind the
// other, so that the groups stand where the products expect them, at a constant
// distance whatever the page size.  V slots hold 32 keys, K slots 64 keys and
// half of the dims, so that QK^T begins with half a tile.  A box per page and
// chunk instead left pages of 16 and 32 bound by the number of copies (64 and
// 32 a tile; 1783 and 1139 us where pages of 64 take 848, chunks of up to 2048
// tokens on up to 24,576; now 1014, 872 and 865).  K in boxes of all dims made
// pages of 64 11 % slower.
//
// What stands between a slot's release and its refill delays every tile, so
// the page numbers are looked up ahead, by the warp's other lanes, and left in
// shared memory: one thread that looked up pages of 16 by itself took 10 %
// longer.  A second thread for V was 5 % slower: its copies then queue behind
// K tiles that are not urgent.
template <int kSrc>
struct PackedTiles {
    const CUtensorMap &tm_k, &tm_v, &tm_krot;
    const PrefillParams &P;
    uint8_t *ring;
    uint64_t *bars;
    volatile int *abort_flag;
    int kind, ntiles, kv_lo, a0, last;  // last: index of the last query
    int row0, seq, g;
    int *groups;  // pages: where the pieces of the tiles of two batches begin

    // Waits until ring use `sc` may be filled, and arms its barrier.
    __device__ __forceinline__ bool take(int sc, int &slot) const {
        slot = sc % kSlots;
        if (sc >= kSlots && !mbar_wait(&bars[kBarSlotEmpty + slot], ((sc / kSlots) - 1) & 1,
                                       abort_flag, P.status))
            return false;
        mbar_arrive_expect_tx(&bars[kBarSlotFull + slot], kSlotBytes);
        return true;
    }

    // Copies every tile; returns the ring uses that were begun.
    __device__ __forceinline__ int load() const {
        if constexpr (kSrc == kKvPages) {
            switch (P.pk.page_shift) {
                case 4: return load_pages<8>();
                case 5: return load_pages<4>();
                case 6: return load_pages<2>();
                default: return load_pages<1>();
            }
        } else {
            int sc = 0;
            auto k_tile = [&](int j) -> bool {
                const int row = row0 + kv_lo + j * kBN;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    int slot;
                    if (!take(sc, slot)) return false;
                    uint8_t *dst = ring + slot * kSlotBytes;
                    if (c * 64 < P.rot_w)
                        tma_load_3d(dst, &tm_krot, &bars[kBarSlotFull + slot], c * 64, row, g);
                    else
                        tma_load_4d(dst, &tm_k, &bars[kBarSlotFull + slot], c * 64, P.H + g, row,
                                    0);
                    ++sc;
                }
                return true;
            };
            auto v_tile = [&](int j) -> bool {
                const int row = row0 + kv_lo + j * kBN;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    int slot;
                    if (!take(sc, slot)) return false;
                    uint8_t *dst = ring + slot * kSlotBytes;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        tma_load_4d(dst + c * (kSlotBytes / 2), &tm_v, &bars[kBarSlotFull + slot],
                                    ((q & 1) * 2 + c) * 64, P.H + P.Hkv + g, row + (q >> 1) * 64,
                                    0);
                    ++sc;
                }
                return true;
            };
            bool ok = k_tile(0);
            if (ok && ntiles > 1) ok = k_tile(1);
            for (int j = 0; ok && j < ntiles; ++j) {
                ok = v_tile(j);
                if (ok && j + 2 < ntiles) ok = k_tile(j + 2);
            }
            return sc;
        }
    }

    // By the whole warp: lane l looks up piece l of the next kBatch tiles, a
    // batch ahead; lane 0 waits and copies.
    template <int kPieces>
    __device__ __forceinline__ int load_pages() const {
        constexpr int kStep = kBN / kPieces;            // keys per piece
        constexpr int kBatch = 32 / kPieces;            // tiles per lookup
        constexpr int kBoxK = kStep < 64 ? kStep : 64;  // keys per K box
        constexpr int kBoxV = kStep < 32 ? kStep : 32;  // keys per V box
        static_assert(kBatch > 2, "V_j is copied after K_{j+2}'s batch has come");
        const int lane = threadIdx.x & 31;
        const int shift = P.pk.page_shift, pmask = (1 << shift) - 1;
        const int lo = kind == kLayerSliding ? a0 - P.window + 1 : 0;
        const int32_t *pages = P.pk.table + static_cast<size_t>(seq) * P.pk.max_pages;
        // pages that no query sees a key of are not looked up
        auto key_of = [&](int n) { return kv_lo + (n * 32 + lane) * kStep; };
        auto seen = [&](int key) { return key <= last && (key | pmask) >= lo; };
        auto look = [&](int n) {
            const int key = key_of(n);
            return seen(key) ? pages[key >> shift] : -1;
        };
        bool bad = false;
        auto place = [&](int n, int id) {  // the piece's first group of 8 slots
            const int key = key_of(n);
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(P.pk.n_pages)) {
                bad = bad || seen(key);
                id = P.pk.n_pages;  // past the pool: the copy reads zeros
            }
            groups[(n & 1) * 32 + lane] =
                ((id * P.Hkv + g) << (shift - 3)) + ((key & pmask) >> 3);
        };
        int sc = 0;
        auto k_tile = [&](int j) -> bool {
            int at[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) at[i] = groups[(j * kPieces + i) & 63];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                int slot;
                if (!take(sc, slot)) return false;
#pragma unroll
                for (int i = 0; i < 64 / kBoxK; ++i) {
                    const int r = (q & 1) * 64 + i * kBoxK;
                    tma_load_4d(ring + slot * kSlotBytes + i * (kBoxK / 8) * (kGroupBytes / 2),
                                &tm_k, &bars[kBarSlotFull + slot], 0, 0, q & 2,
                                at[r / kStep] + r % kStep / 8);
                }
                ++sc;
            }
            return true;
        };
        auto v_tile = [&](int j) -> bool {
            int at[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) at[i] = groups[(j * kPieces + i) & 63];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                int slot;
                if (!take(sc, slot)) return false;
#pragma unroll
                for (int i = 0; i < 32 / kBoxV; ++i) {
                    const int r = q * 32 + i * kBoxV;
                    tma_load_4d(ring + slot * kSlotBytes + i * (kBoxV / 8) * kGroupBytes, &tm_v,
                                &bars[kBarSlotFull + slot], 0, 0, 0,
                                at[r / kStep] + r % kStep / 8);
                }
                ++sc;
            }
            return true;
        };
        place(0, look(0));
        int next = look(1);
        __syncwarp();
        bool ok = true;
        if (lane == 0) ok = k_tile(0) && (ntiles == 1 || k_tile(1));
        for (int j = 0; j < ntiles; ++j) {
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if ((j + 2) % kBatch == 0) {
                const int n = (j + 2) / kBatch;
                __syncwarp();  // the batch before the last is read
                place(n, next);
                next = look(n + 1);
                __syncwarp();
            }
            if (lane == 0) ok = v_tile(j) && (j + 2 >= ntiles || k_tile(j + 2));
        }
        if (bad) atomicOr(P.status, kErrPage);
        return sc;
    }
};

// Gives values of V that are not finite, which clean_v_rows took out, back to
// a row that sees them: adds them to this thread's 128 dims of the row's
// output (TMEM columns from taddr on).  Warp-collective, and rare.  `lo` and
// `end` bound the keys of this CTA, of which only those hidden from some of the
// tile's queries a0..a_last were touched.
template <typename Src>
__device__ __forceinline__ void give_back(uint32_t taddr, bool valid, int kind, int window, int at,
                                          int a0, int a_last, int lo, int end, Src v_row) {
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        tmem_ld32(taddr + c, o);
        tmem_ld_wait();
        for (int key = lo; valid && key < end; ++key) {
            if (key <= a0 && (kind == kLayerFull || a_last - key < window)) continue;
            if (!key_visible(kind, window, at, key)) continue;
            const __nv_bfloat16 *src = v_row(key);
            if (!src) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 w = *reinterpret_cast<const uint4 *>(src + c + q * 8);
                const uint32_t vw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t m = nonfinite_mask(vw[i]);
                    uint32_t &x = o[q * 8 + 2 * i], &y = o[q * 8 + 2 * i + 1];
                    if (m & 0xFFFFu) x = __float_as_uint(__uint_as_float(x) + bf16_lo(vw[i]));
                    if (m >> 16) y = __float_as_uint(__uint_as_float(y) + bf16_hi(vw[i]));
                }
            }
        }
        __syncwarp();
        tmem_st32(taddr + c, o);
    }
    tmem_st_wait();
}

// The same out of line, for the paged kernels: inlined there a sliding prompt of
// 8192 tokens takes 159 us instead of 154.  The packed ones have it inlined: out
// of line mixed prompts take 215.5 us instead of 210.5, 20,011 tokens 2289
// instead of 2258.
template <typename Src>
__device__ __noinline__ void give_back_call(uint32_t taddr, bool valid, int kind, int window,
                                            int at, int a0, int a_last, int lo, int end,
                                            Src v_row) {
    give_back(taddr, valid, kind, window, at, a0, a_last, lo, end, v_row);
}

// Split query tiles: this thread's 128 dims of a row's unnormalised output
// (TMEM columns from taddr on) to the part's state, rows side by side.
__device__ __forceinline__ void leave_part(float4 *o, uint32_t taddr, bool store, bool ok) {
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        uint32_t v[32];
        tmem_ld32(taddr + c, v);
        tmem_ld_wait();
        if (!store) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            o[(c / 4 + q) * kBM] =
                ok ? make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                 __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// kG: the GQA group size when fixed at compile time (the Spark-X2.5 shapes
// all use 4), 0 to read it from P.G.  Timing chose the fixed size for the
// sliding-kind kernels only; the full-kind ones measured faster without it.
template <int kSrc, int kKind, int kG>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prefill_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_kv_k,
                        const __grid_constant__ CUtensorMap tm_kv_v,
                        const __grid_constant__ CUtensorMap tm_krot,
                        const __grid_constant__ CUtensorMap tm_out,
                        const __grid_constant__ PrefillParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *qbuf = smem;
    uint8_t *ring = smem + kQBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + kSlots * kSlotBytes);
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    __shared__ float red_max[2][2][kBM];   // [tile parity][warpgroup][row]: half-row maxima
    __shared__ float red_l[2][kBM];        // [warpgroup][row]: half-row sums
    constexpr bool kIsPacked = kSrc == kKvPacked || kSrc == kKvPages;
    __shared__ int cleaned_any;            // packed: a value was taken out of a partly hidden row
    // packed: the item, read from here where it is needed (held in registers
    // through the softmax it made the kernel spill)
    __shared__ PackedItem s_item;
    __shared__ int s_groups[kSrc == kKvPages ? 64 : 1];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kind = kKind == kKindAny ? P.kind : kKind;
    const int G = kG > 0 ? kG : P.G, tq = kBM / G;
    const int units = P.Hkv * P.B;
    const int qtile = P.n_qtiles - 1 - static_cast<int>(blockIdx.x) / units;  // longest first
    const int rem = static_cast<int>(blockIdx.x) % units;
    const int g = rem % P.Hkv, b = rem / P.Hkv;
    int t0 = qtile * tq;
    int t_end = (t0 + tq < P.T) ? t0 + tq : P.T;  // exclusive
    int seq_end = P.T;                            // tokens of the sequence
    int row0 = 0;                                 // packed: the sequence's first row
    int seq = 0;
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            uint32_t count = 1;
            if (i == kBarQReady || i == kBarPReady || i == kBarPReady + 1 || i == kBarMaxX ||
                i == kBarMaxX + 1)
                count = kSoftmaxThreads;
            if (i == kBarMmaDrain) count = 2;  // one commit from each MMA issuer
            mbar_init(&bars[i], count);
        }
        fence_mbar_init();
        abort_flag = 0;
        if (kIsPacked) cleaned_any = 0;
    }
    if constexpr (kIsPacked) {
        // The tile comes from the list that the kernel before has been making.
        // The grid allows for a ragged tile in every sequence: a CTA past the
        // list has nothing to do.
        // The tensor maps come from the host and wait for nothing.  (As a lambda:
        // written out, the compiler's order of the packed full kernel is 3 to 4 %
        // slower: mixed prompts 209 -> 215 us, 20,011 tokens 2270 -> 2325 us; the
        // other kernels are within 1 % either way.)
        auto prefetch_maps = [&] {
            if (warp == 0 && lane == 0) {
                tma_prefetch_desc(&tm_q);
                tma_prefetch_desc(&tm_kv_k);
                tma_prefetch_desc(&tm_kv_v);
                if (P.rot_w > 0) tma_prefetch_desc(&tm_krot);
                tma_prefetch_desc(&tm_out);
            }
        };
        prefetch_maps();
        grid_dep_wait();
        const PackedItem item = P.pk.work[static_cast<int>(blockIdx.x) / units];
        if (item.seq < 0) return;
        if (tid == 0) s_item = item;
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, kTmemCols);
        tmem_relinquish();
    }
    if (!kIsPacked && warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_kv_k);
        tma_prefetch_desc(&tm_kv_v);
        if (P.rot_w > 0) tma_prefetch_desc(&tm_krot);
        tma_prefetch_desc(&tm_out);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    // Programmatic dependent launch.  The kernel before this one may still run.
    // When it is one of this call's own (rotated K, or the chunk's cache store),
    // it waited for the call's inputs before letting this kernel start, so only
    // the producer waits, before its first key/value load.  Otherwise every
    // thread waits here, before reading any input.
    if (!kIsPacked && !P.defer_wait) grid_dep_wait();

    // Absolute indices: queries t0..t_end-1 of the chunk sit at start + t.
    int start = 0;
    bool skip = false;
    if constexpr (kIsPacked) {
        seq = s_item.seq;
        t0 = s_item.t0;
        row0 = s_item.row0;
        seq_end = s_item.len;
        start = s_item.start;
        t_end = (t0 + tq < seq_end) ? t0 + tq : seq_end;
    } else if constexpr (kSrc != kKvFromQkv) {
        start = P.start[b];
        skip = start < 0 || (kind == kLayerFull && static_cast<long long>(start) + P.T > P.cap);
        if (skip && tid == 0 && qtile == P.n_qtiles - 1 && g == 0) atomicOr(P.status, kErrPosition);
    }
    const int a0 = start + t0;
    // a ring is read in 128-key tiles aligned to its 128-slot boundaries, so
    // that no tile wraps around the end of the ring
    const KeyTiles kt = prefill_key_tiles(kind, P.window, a0, start + t_end, kBN,
                                          kSrc == kKvFromRing || kSrc == kKvPages);
    const int kv_lo = kt.kv_lo + (kIsPacked ? s_item.k0 * kBN : 0);
    const int ntiles = skip ? 0 : (kIsPacked ? s_item.tiles : kt.ntiles);
    const PackedTiles<kSrc> packed_tiles{tm_kv_k, tm_kv_v, tm_krot, P, ring, bars, &abort_flag,
                                         kind, ntiles, kv_lo, a0, start + t_end - 1, row0, seq, g,
                                         s_groups};

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        int sc = 0;  // ring slots filled so far
        if (lane == 0 && !skip) {
            mbar_arrive_expect_tx(&bars[kBarQFull], kQBytes);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                tma_load_4d(qbuf + c * kSlotBytes, &tm_q, &bars[kBarQFull], c * 64, g * G,
                            row0 + t0, b);
            // the CTA one wave later (likely the next one on this SM) finds its
            // query tile in L2 -- when this CTA is short (a sliding layer's, or
            // the last waves of a causal one); behind a long CTA the tile would
            // be evicted before use and read twice
            const long long nb = static_cast<long long>(blockIdx.x) + P.wave;
            if (P.wave > 0 && nb < gridDim.x && ntiles <= kPrefetchMaxTiles) {
                const int nrem = static_cast<int>(nb % units);
                int nt0;
                if constexpr (kIsPacked) {
                    const PackedItem w = P.pk.work[nb / units];
                    nt0 = w.row0 + w.t0;
                } else {
                    nt0 = (P.n_qtiles - 1 - static_cast<int>(nb / units)) * tq;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tma_prefetch_l2_4d(&tm_q, c * 64, (nrem % P.Hkv) * G, nt0, nrem / P.Hkv);
            }
            if (P.defer_wait) grid_dep_wait();  // rotated K / the cache are ready
            bool ok = true;
            auto next_slot = [&](int &slot) -> bool {
                slot = sc % kSlots;
                if (sc >= kSlots &&
                    !mbar_wait(&bars[kBarSlotEmpty + slot], ((sc / kSlots) - 1) & 1, &abort_flag,
                               P.status))
                    return false;
                mbar_arrive_expect_tx(&bars[kBarSlotFull + slot], kSlotBytes);
                return true;
            };
            auto load_k = [&](int j) -> bool {
                const int key0 = kv_lo + j * kBN;
                for (int c = 0; c < 4; ++c) {
                    int slot;
                    if (!next_slot(slot)) return false;
                    uint8_t *dst = ring + slot * kSlotBytes;
                    if constexpr (kSrc != kKvFromQkv) {
                        const int slot0 =
                            kSrc == kKvFromRing ? key0 % static_cast<int>(P.cap) : key0;
                        tma_load_4d(dst, &tm_kv_k, &bars[kBarSlotFull + slot], c * 64, slot0, g,
                                    b);
                    } else if (c * 64 < P.rot_w) {
                        tma_load_3d(dst, &tm_krot, &bars[kBarSlotFull + slot], c * 64, key0,
                                    b * P.Hkv + g);
                    } else {
                        tma_load_4d(dst, &tm_kv_k, &bars[kBarSlotFull + slot], c * 64, P.H + g,
                                    key0, b);
                    }
                    ++sc;
                }
                return true;
            };
            auto load_v = [&](int j) -> bool {
                const int key0 = kv_lo + j * kBN;
                for (int vs = 0; vs < 4; ++vs) {
                    int slot;
                    if (!next_slot(slot)) return false;
                    uint8_t *dst = ring + slot * kSlotBytes;
                    if constexpr (kSrc != kKvFromQkv) {
                        const int slot0 =
                            kSrc == kKvFromRing ? key0 % static_cast<int>(P.cap) : key0;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            tma_load_4d(dst + c * (kSlotBytes / 4), &tm_kv_v,
                                        &bars[kBarSlotFull + slot], c * 64, slot0 + vs * 32, g, b);
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            tma_load_4d(dst + c * (kSlotBytes / 4), &tm_kv_v,
                                        &bars[kBarSlotFull + slot], c * 64, P.H + P.Hkv + g,
                                        key0 + vs * 32, b);
                    }
                    ++sc;
                }
                return true;
            };
            if constexpr (!kIsPacked) {
                ok = load_k(0);
                if (ok && ntiles > 1) ok = load_k(1);
                for (int j = 0; ok && j < ntiles; ++j) {
                    ok = load_v(j);
                    if (ok && j + 2 < ntiles) ok = load_k(j + 2);
                }
            } else if constexpr (kSrc == kKvPacked) {
                sc = packed_tiles.load();
            }
        }
        __syncwarp();
        if constexpr (kSrc == kKvPages) sc = packed_tiles.load();
        tc_fence_before();
        __syncthreads();
        // after an abort, copies in flight must land before shared memory is released
        if (lane == 0 && abort_flag) {
            mbar_wait_plain(&bars[kBarQFull], 0);
            const int first = sc > kSlots ? sc - kSlots : 0;
            for (int s = first; s < sc; ++s)
                mbar_wait_plain(&bars[kBarSlotFull + (s % kSlots)], (s / kSlots) & 1);
        }
    } else if (warp == 1 || warp == 2) {
        // ------------------------------------------------------ MMA issuers
        // Two threads issue the products: warp 1's lane 0 the QK^T of every
        // key tile, warp 2's lane 0 every P*V, so neither waits for the
        // other's issue.  Both replay the producer's load order (K0, K1, then
        // per tile j: V_j, K_{j+2}) to find the ring slots of their chunks.
        // The barriers carry the dependencies between them: P*V of tile j
        // waits for P_j (softmax), and QK^T of tile j+2, which overwrites the
        // score buffer holding P_j, waits for P*V of tile j to complete.
        const bool qk_role = warp == 1;
        if (lane == 0 && !skip) {
            // Shared-memory descriptors built once: the address field holds
            // (address mod 2^18) / 16 in its low bits, and every operand lies
            // below 2^18, so an operand at byte offset o from a base has the
            // base's descriptor plus o / 16.  This keeps the issue loop short.
            const uint64_t q_desc = smem_desc_sw128(smem_u32(qbuf), 16, 1024);
            constexpr bool kPages = kSrc == kKvPages;  // tiles of 8-key groups
            const uint64_t k_desc =
                smem_desc_sw128(smem_u32(ring), 16, kPages ? kGroupBytes / 2 : 1024);
            const uint64_t v_desc = smem_desc_sw128(smem_u32(ring), kPages ? 1024 : kSlotBytes / 4,
                                                    kPages ? kGroupBytes : 1024);
            const uint64_t vp_desc = smem_desc_sw128(smem_u32(ring), kSlotBytes / 2, 1024);
            // (the full-layer cache instance measured faster building each
            // descriptor in place)
            constexpr bool kDescInPlace = kSrc == kKvFromCache;
            const uint32_t q_addr = smem_u32(qbuf), ring_addr = smem_u32(ring);
            int sc = 0;  // ring slots of the producer's loads before the next one
            bool ok = true;
            auto mma_qk = [&](int j) -> bool {
                const uint32_t d = tmem + kColS + (j & 1) * kBN;
                for (int h = 0; kPages && h < 2; ++h) {  // halves of 128 dims, two slots each
                    const int slot = sc % kSlots;
                    const uint32_t parity = (sc / kSlots) & 1;
                    if (!mbar_wait(&bars[kBarSlotFull + slot], parity, &abort_flag, P.status) ||
                        !mbar_wait(&bars[kBarSlotFull + slot + 1], parity, &abort_flag, P.status))
                        return false;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // 16 dims a step
                        mma_ss(d,
                               q_desc + static_cast<uint32_t>(
                                            ((2 * h + (i >> 2)) * kSlotBytes + (i & 3) * 32) >> 4),
                               k_desc + static_cast<uint32_t>(
                                            (slot * kSlotBytes + (i >> 2) * 1024 + (i & 3) * 32) >>
                                            4),
                               kIdescQK, (h | i) != 0);
                    tc_commit(&bars[kBarSlotEmpty + slot]);
                    tc_commit(&bars[kBarSlotEmpty + slot + 1]);
                    sc += 2;
                }
                for (int c = 0; !kPages && c < 4; ++c) {
                    const int slot = sc % kSlots;
                    if (!mbar_wait(&bars[kBarSlotFull + slot], (sc / kSlots) & 1, &abort_flag,
                                   P.status))
                        return false;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t ad =
                            kDescInPlace
                                ? smem_desc_sw128(q_addr + c * kSlotBytes + kk * 32, 16, 1024)
                                : q_desc + static_cast<uint32_t>((c * kSlotBytes + kk * 32) >> 4);
                        const uint64_t bd =
                            kDescInPlace
                                ? smem_desc_sw128(ring_addr + slot * kSlotBytes + kk * 32, 16, 1024)
                                : k_desc + static_cast<uint32_t>((slot * kSlotBytes + kk * 32) >> 4);
                        mma_ss(d, ad, bd, kIdescQK, (c | kk) != 0);
                    }
                    tc_commit(&bars[kBarSlotEmpty + slot]);
                    ++sc;
                }
                tc_commit(&bars[kBarSFull + (j & 1)]);
                return true;
            };
            auto mma_pv = [&](int j) -> bool {
                const uint32_t pcol = tmem + kColS + (j & 1) * kBN;
                if constexpr (kSrc == kKvPacked) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // halves of 64 keys, two slots each
                        const int slot = sc % kSlots;
                        const uint32_t parity = (sc / kSlots) & 1;
                        if (!mbar_wait(&bars[kBarSlotFull + slot], parity, &abort_flag,
                                       P.status) ||
                            !mbar_wait(&bars[kBarSlotFull + slot + 1], parity, &abort_flag,
                                       P.status))
                            return false;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            // P of keys 0..63 sits in packed columns 0..31, of 64..127 in 64..95
                            mma_ts(tmem + kColO, pcol + h * 64 + kk * 8,
                                   vp_desc + static_cast<uint32_t>((slot * kSlotBytes + kk * 2048) >> 4),
                                   kIdescPV, (j > 0 || h + kk > 0));
                        }
                        tc_commit(&bars[kBarSlotEmpty + slot]);
                        tc_commit(&bars[kBarSlotEmpty + slot + 1]);
                        sc += 2;
                    }
                }
                for (int vs = 0; kSrc != kKvPacked && vs < 4; ++vs) {
                    const int slot = sc % kSlots;
                    if (!mbar_wait(&bars[kBarSlotFull + slot], (sc / kSlots) & 1, &abort_flag,
                                   P.status))
                        return false;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        const int ks = vs * 2 + kk;  // 16-key step within the tile
                        const uint64_t bd =
                            kDescInPlace
                                ? smem_desc_sw128(ring_addr + slot * kSlotBytes + kk * 2048,
                                                  kSlotBytes / 4, 1024)
                                : v_desc + static_cast<uint32_t>(
                                               (slot * kSlotBytes +
                                                kk * (kPages ? 2 * kGroupBytes : 2048)) >> 4);
                        // P of keys 0..63 sits in packed columns 0..31, keys 64..127 in 64..95
                        const uint32_t acol = pcol + (ks < 4 ? ks * 8 : 64 + (ks - 4) * 8);
                        mma_ts(tmem + kColO, acol, bd, kIdescPV, (j > 0 || ks > 0));
                    }
                    tc_commit(&bars[kBarSlotEmpty + slot]);
                    ++sc;
                }
                tc_commit(&bars[kBarODone]);
                return true;
            };
            if (qk_role) {
                ok = mbar_wait(&bars[kBarQReady], 0, &abort_flag, P.status);
                tc_fence_after();
                if (ok) ok = mma_qk(0);
                if (ok && ntiles > 1) ok = mma_qk(1);
                for (int j = 0; ok && j < ntiles; ++j) {
                    sc += 4;  // V_j: the other issuer's
                    if (j + 2 < ntiles) {
                        // QK^T of tile j+2 overwrites the score buffer whose
                        // first half holds P_j: wait until P*V of tile j
                        // (accumulator O) has finished reading it.  P*V of tile
                        // j+1 needs QK^T of tile j+1, issued before this wait,
                        // so the barrier is never two phases ahead of it.
                        ok = mbar_wait(&bars[kBarODone], j & 1, &abort_flag, P.status);
                        if (ok) {
                            tc_fence_after();
                            ok = mma_qk(j + 2);
                        }
                    }
                }
            } else {
                sc = ntiles > 1 ? 8 : 4;  // after K0 and K1
                for (int j = 0; ok && j < ntiles; ++j) {
                    ok = mbar_wait(&bars[kBarPReady + (j & 1)], (j >> 1) & 1, &abort_flag,
                                   P.status);
                    if (!ok) break;
                    tc_fence_after();
                    ok = mma_pv(j);
                    if (j + 2 < ntiles) sc += 4;  // K_{j+2}: the other issuer's
                }
                // The epilogue waits on a barrier of its own: a parity wait on
                // kBarODone could be two phases behind when the last softmax
                // tile finishes before P*V of the tile before it.
                if (ok) tc_commit(&bars[kBarOFinal]);
            }
            // every product either thread issued must finish before TMEM is
            // released (the drain barrier counts one arrival from each)
            tc_commit(&bars[kBarMmaDrain]);
            mbar_wait_plain(&bars[kBarMmaDrain], 0);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (qk_role) tmem_dealloc(tmem, kTmemCols);
    } else if (warp >= kSoftmaxWarp0) {
        // ------------------------------------------------------ softmax
        const int wq = warp & 3;                        // TMEM lane quarter of this warp
        const int wg = (warp - kSoftmaxWarp0) >> 2;     // warpgroup: score-column half
        const int row = wq * 32 + lane;                 // TMEM lane, query row
        const int sth = tid - kSoftmaxWarp0 * 32;       // 0..255 among softmax threads
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const int tok = t0 + row / G;
        const int tok_abs = start + tok;                // absolute index for the mask
        const int head = g * G + row % G;
        const bool valid = kIsPacked ? !skip && tok < seq_end : tok < P.T;
        const size_t trow = kIsPacked ? static_cast<size_t>(valid ? row0 + tok : 0)
                                      : static_cast<size_t>(b) * P.T + (valid ? tok : 0);
        const int p = valid ? P.pos[trow] : 0;
        const float gate_logit = valid ? P.gate[trow * P.H + head] : 0.f;
        bool ok = !skip && mbar_wait(&bars[kBarQFull], 0, &abort_flag, P.status);

        // rotate this row of Q in place (bf16 in, fp32 math, bf16 out); the
        // two warpgroups take alternate groups of 8 pairs, and the G rows of a
        // token (adjacent lanes) share the angles
        if (ok) {
            if constexpr (kG > 0) {
                rotate_q_row<kG>(qbuf, row, lane, wg, p, P.rope);
            } else {
                switch (G) {
                    case 1: rotate_q_row<1>(qbuf, row, lane, wg, p, P.rope); break;
                    case 2: rotate_q_row<2>(qbuf, row, lane, wg, p, P.rope); break;
                    case 4: rotate_q_row<4>(qbuf, row, lane, wg, p, P.rope); break;
                    default: rotate_q_row<8>(qbuf, row, lane, wg, p, P.rope); break;
                }
            }
        }
        fence_proxy_async_smem();
        if (!skip) mbar_arrive(&bars[kBarQReady]);

        // Scores stay in raw units s = q.k; probabilities are
        // exp2(s * kScaleLog2 - m * kScaleLog2) with m the row's reference max.
        // The reference moves only when the row max grows past it by the
        // raw equivalent of 2^8.
        constexpr float kLazyRaw = 8.0f / kScaleLog2;
        const int a_last = start + t_end - 1;
        // The kernel before has looked over the values of the call's tokens.
        // Without a cache there are no others; in pages, these are the indices
        // from `start` to finite_end.
        const bool odd = kIsPacked && P.pk.odd_values[s_item.call & 1] != 0;
        const int finite_end = odd ? -1 : start + seq_end;
        const int col0 = wg * 64;                       // first score column of this thread
        float m_run = -INFINITY, l_part = 0.f;
        for (int j = 0; ok && j < ntiles; ++j) {
            ok = mbar_wait(&bars[kBarSFull + (j & 1)], (j >> 1) & 1, &abort_flag, P.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sbase = lane_base + kColS + (j & 1) * kBN;
            uint32_t sv[64];
            tmem_ld32(sbase + col0, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
            tmem_ld32(sbase + col0 + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
            tmem_ld_wait();
            float x[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = __uint_as_float(sv[c]);
            const int key0 = kv_lo + j * kBN;
            if (tile_needs_mask(kind, P.window, key0, kBN, a0, a_last)) {
#pragma unroll
                for (int c = 0; c < 64; ++c) {
                    const bool vis = key_visible(kind, P.window, tok_abs, key0 + col0 + c);
                    x[c] = vis ? x[c] : -INFINITY;
                }
            }
            // row max of this half (8 independent chains), then of the row
            float m8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m8[i] = x[i];
#pragma unroll
            for (int c = 8; c < 64; ++c) m8[c & 7] = fmaxf(m8[c & 7], x[c]);
            const float mloc = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                     fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
            // exchange with the other half of the row (a bounded wait, so a
            // warp that gave up elsewhere cannot strand the others)
            red_max[j & 1][wg][row] = mloc;
            mbar_arrive(&bars[kBarMaxX + (j & 1)]);
            ok = mbar_wait(&bars[kBarMaxX + (j & 1)], (j >> 1) & 1, &abort_flag, P.status);
            if (!ok) break;
            const float m_new = fmaxf(mloc, red_max[j & 1][wg ^ 1][row]);

            // tcgen05.ld/st are warp-collective: the O rescale runs for the
            // whole warp (alpha is 1 on rows that keep their reference)
            const bool bump = m_new > m_run + kLazyRaw;
            const bool rescale_row = bump && m_run != -INFINITY;
            const float alpha = rescale_row ? fast_exp2((m_run - m_new) * kScaleLog2) : 1.f;
            if (bump) {
                l_part *= alpha;
                m_run = m_new;
            }
            if (j > 0 && __any_sync(0xffffffffu, rescale_row)) {
                ok = mbar_wait(&bars[kBarODone], (j - 1) & 1, &abort_flag, P.status);
                if (!ok) break;
                tc_fence_after();
                for (int c = wg * 128; c < wg * 128 + 128; c += 32) {
                    uint32_t ov[32];
                    tmem_ld32(lane_base + kColO + c, ov);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                    tmem_st32(lane_base + kColO + c, ov);
                }
            }
            const float neg = (m_run == -INFINITY) ? 0.f : -m_run * kScaleLog2;
            // Probabilities are rounded to bf16 for P*V, an operand of V's type: with
            // the output's own rounding the error against 64 bits is 2.1e-3 of the
            // output instead of 1.7e-3.  A second term, as in decode, would double
            // the products that bound this kernel.  Their sum stays in 32 bits.
            uint32_t pk[32];
            float l8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const float p0 = fast_exp2(fmaf(x[2 * c], kScaleLog2, neg));
                const float p1 = fast_exp2(fmaf(x[2 * c + 1], kScaleLog2, neg));
                l8[c & 7] += p0 + p1;
                pk[c] = pack_bf16x2(p0, p1);
            }
            l_part += ((l8[0] + l8[1]) + (l8[2] + l8[3])) + ((l8[4] + l8[5]) + (l8[6] + l8[7]));
            tmem_st32(sbase + wg * 64, pk);
            tmem_st_wait();
            tc_fence_before();
            if constexpr (kIsPacked) {
                // (of a page's older slots only the window's start can be hidden)
                const bool clean =
                    kSrc == kKvPages
                        ? key0 + kBN > finite_end || (kind == kLayerSliding && key0 < start &&
                                                      key0 < a_last - P.window + 1)
                        : odd;
                if (clean && tile_needs_mask(kind, P.window, key0, kBN, a0, a_last)) {
                    if constexpr (kSrc == kKvPages)
                        ok = clean_tile_call<true>(ring, bars, &abort_flag, P.status, &cleaned_any,
                                                   j, ntiles, kind, P.window, key0, a0, a_last,
                                                   warp - kSoftmaxWarp0, lane, start, finite_end);
                    else
                        ok = clean_tile_call<false>(ring, bars, &abort_flag, P.status, &cleaned_any,
                                                    j, ntiles, kind, P.window, key0, a0, a_last,
                                                    warp - kSoftmaxWarp0, lane);
                    if (!ok) break;
                }
            }
            mbar_arrive(&bars[kBarPReady + (j & 1)]);
        }

        if (kIsPacked && blockIdx.x == 0 && sth == 0) *P.pk.call = s_item.call + 1;
        // epilogue: O / l * sigmoid(gate) -> bf16 -> staged in the Q buffer -> TMA store
        if (sth == 0) grid_dep_launch();
        if (ok) ok = mbar_wait(&bars[kBarOFinal], 0, &abort_flag, P.status);
        if (skip) ok = false;
        red_l[wg][row] = l_part;
        named_bar(1, kSoftmaxThreads);
        {
            // every softmax thread runs this block (barrier counts must match);
            // only the store below depends on the abort flag
            tc_fence_after();
            const float l_row = l_part + red_l[wg ^ 1][row];
            bool whole = true;  // the same in every softmax thread
            if constexpr (kIsPacked) {
                if (cleaned_any && ok) {
                    const int end = kv_lo + ntiles * kBN < a_last + 1 ? kv_lo + ntiles * kBN
                                                                      : a_last + 1;
                    auto v_row = [&](int key) -> const __nv_bfloat16 * {
                        if constexpr (kSrc == kKvPages) {
                            const int page = P.pk.table[static_cast<size_t>(seq) * P.pk.max_pages +
                                                        (key >> P.pk.page_shift)];
                            if (page < 0 || page >= P.pk.n_pages) return nullptr;
                            return P.v_cache +
                                   (((static_cast<size_t>(page) * P.Hkv + g) << P.pk.page_shift) +
                                    (key & ((1 << P.pk.page_shift) - 1))) * kHeadDim + wg * 128;
                        } else {
                            return P.qkv + ((static_cast<size_t>(row0) + key) * (P.H + 2 * P.Hkv) +
                                            P.H + P.Hkv + g) * kHeadDim + wg * 128;
                        }
                    };
                    const uint32_t taddr = lane_base + kColO + wg * 128;
                    if constexpr (kSrc == kKvPages)
                        give_back_call(taddr, valid, kind, P.window, tok_abs, a0, a_last, kv_lo,
                                       end, v_row);
                    else
                        give_back(taddr, valid, kind, P.window, tok_abs, a0, a_last, kv_lo, end,
                                  v_row);
                }
                whole = s_item.parts == 1;
                if (!whole) {
                    // one of several parts of the query tile: its state goes to
                    // the workspace, and the kernel behind this one joins them
                    const size_t slot =
                        s_item.slot + static_cast<size_t>(g) * s_item.parts + s_item.part;
                    if (wg == 0)
                        P.pk.part_ml[slot * kBM + row] =
                            ok ? make_float2(m_run, l_row) : make_float2(-INFINITY, 0.f);
                    leave_part(P.pk.part_o + (slot * 64 + wg * 32) * kBM + row,
                               lane_base + kColO + wg * 128, valid, ok);
                }
            }
            const float scale = valid ? gate_act(gate_logit, P.gate_mode) / l_row : 0.f;
            // two 32-column loads in flight per wait (the loads' latency overlaps)
            for (int c = wg * 128; whole && c < wg * 128 + 128; c += 64) {
                uint32_t ov[2][32];
                tmem_ld32(lane_base + kColO + c, ov[0]);
                tmem_ld32(lane_base + kColO + c + 32, ov[1]);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint4 w;
                        w.x = pack_bf16x2(__uint_as_float(ov[h][8 * q + 0]) * scale,
                                          __uint_as_float(ov[h][8 * q + 1]) * scale);
                        w.y = pack_bf16x2(__uint_as_float(ov[h][8 * q + 2]) * scale,
                                          __uint_as_float(ov[h][8 * q + 3]) * scale);
                        w.z = pack_bf16x2(__uint_as_float(ov[h][8 * q + 4]) * scale,
                                          __uint_as_float(ov[h][8 * q + 5]) * scale);
                        w.w = pack_bf16x2(__uint_as_float(ov[h][8 * q + 6]) * scale,
                                          __uint_as_float(ov[h][8 * q + 7]) * scale);
                        *reinterpret_cast<uint4 *>(qbuf + sw128_offset(row, (c + 32 * h) / 8 + q)) = w;
                    }
            }
            fence_proxy_async_smem();
            named_bar(1, kSoftmaxThreads);
            if (kIsPacked && t_end - t0 < tq) {
                // a ragged tile: the rows behind it belong to others
                const int nrows = skip || abort_flag || !whole ? 0 : (t_end - t0) * G;
                for (int i = sth; i < nrows * 32; i += kSoftmaxThreads) {
                    const int r = i >> 5, q = i & 31;
                    *reinterpret_cast<uint4 *>(
                        P.pk.out +
                        ((static_cast<size_t>(row0) + t0 + r / G) * P.H + g * G + r % G) *
                            kHeadDim + q * 8) =
                        *reinterpret_cast<const uint4 *>(qbuf + sw128_offset(r, q));
                }
            } else if (sth == 0 && !abort_flag && !skip && whole) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tma_store_4d(&tm_out, qbuf + c * kSlotBytes, c * 64, g * G, row0 + t0, b);
                tma_store_commit();
                tma_store_wait_read();  // the staging buffer is read; the writes land by grid end
            }
        }
        tc_fence_before();
        __syncthreads();
    } else {
        // warp 3 has no role
        __syncthreads();
    }
}

// ---------------------------------------------------------------- joining

// Joins the states of split query tiles: out = sigma(gate) * sum_p w_p O_p /
// sum_p w_p l_p with w_p = exp2((m_p - max m) / 16 log2 e).  A task is 32 rows
// of one tile and KV head and half the dims; lane = row, so that the states
// are read 512 bytes at a time, and each warp takes 16 dims.  Where no tile was
// split there are no tasks.
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads) join_parts_kernel(
    const __grid_constant__ PrefillParams P) {
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = *P.pk.n_splits, tq = kBM / P.G;
    const int per_tile = P.Hkv * (kBM / 32) * 2;
    for (int task = blockIdx.x; task < n * per_tile; task += gridDim.x) {
        const PackedItem t = P.pk.splits[task / per_tile];
        const int u = task % per_tile;
        const int g = u / (2 * (kBM / 32)), row = (u >> 1) % (kBM / 32) * 32 + lane;
        const int tokens = t.len - t.t0 < tq ? t.len - t.t0 : tq;
        if (row >= tokens * P.G) continue;
        const size_t slot0 = t.slot + static_cast<size_t>(g) * t.parts;
        const float2 *ml = P.pk.part_ml + slot0 * kBM + row;
        float m = -INFINITY, l = 0.f;
        for (int p = 0; p < t.parts; ++p) m = fmaxf(m, ml[p * kBM].x);
        const int dim = (u & 1) * 128 + warp * 16;
        const float4 *o = P.pk.part_o + (slot0 * 64 + dim / 4) * kBM + row;
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 4
        for (int p = 0; p < t.parts; ++p) {
            const float2 x = ml[p * kBM];
            const float w = x.x == -INFINITY ? 0.f : fast_exp2((x.x - m) * kScaleLog2);
            l += x.y * w;
            const float4 *src = o + static_cast<size_t>(p) * (kBM * 64);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 y = src[q * kBM];
                acc[4 * q] += y.x * w;
                acc[4 * q + 1] += y.y * w;
                acc[4 * q + 2] += y.z * w;
                acc[4 * q + 3] += y.w * w;
            }
        }
        const size_t token = static_cast<size_t>(t.row0) + t.t0 + row / P.G;
        const size_t head = token * P.H + g * P.G + row % P.G;
        const float scale = gate_act(P.gate[head], P.gate_mode) / l;
        uint4 *dst = reinterpret_cast<uint4 *>(P.pk.out + head * kHeadDim + dim);
#pragma unroll
        for (int q = 0; q < 2; ++q)
            dst[q] = make_uint4(pack_bf16x2(acc[8 * q] * scale, acc[8 * q + 1] * scale),
                                pack_bf16x2(acc[8 * q + 2] * scale, acc[8 * q + 3] * scale),
                                pack_bf16x2(acc[8 * q + 4] * scale, acc[8 * q + 5] * scale),
                                pack_bf16x2(acc[8 * q + 6] * scale, acc[8 * q + 7] * scale));
    }
}

// ---------------------------------------------------------------- launcher

// The attention kernel for a KV source and layer kind; sliding-kind kernels
// are specialised for a group of 4.
template <int kSrc, int kKind>
auto attn_kernel_for(int G) {
    if constexpr (kKind == kLayerSliding)
        return G == 4 ? prefill_attn_kernel<kSrc, kKind, 4> : prefill_attn_kernel<kSrc, kKind, 0>;
    else
        return prefill_attn_kernel<kSrc, kKind, 0>;
}

cudaError_t launch_prefill(const CUtensorMap &tm_q, const CUtensorMap &tm_kv_k,
                           const CUtensorMap &tm_kv_v, const CUtensorMap &tm_krot,
                           const CUtensorMap &tm_out, const PrefillParams &P_in,
                           cudaStream_t stream) {
    PrefillParams P = P_in;
    // a library kernel runs before the attention kernel on every path but the
    // one-shot prefill without rotated dims
    P.defer_wait = (P.start != nullptr || P.rot_w > 0) ? 1 : 0;
    const int r = P.rope.rot_dim;
    const long long store_items = r / 16 + (kHeadDim - r) / 8 + kHeadDim / 8;
    const long long store_blocks =
        (static_cast<long long>(P.B) * P.T * store_items + kRopeThreads - 1) / kRopeThreads;
    const unsigned grid = static_cast<unsigned>(P.n_qtiles) * P.Hkv * P.B;
    cudaError_t err;
    if (P.start != nullptr) {
        // chunked prefill: store the chunk's keys and values first, clear the
        // never-written slots the last key tile may read, then attend over
        // the cache
        err = launch_overlapped(prefill_store_kv_kernel, dim3(static_cast<unsigned>(store_blocks)),
                                dim3(kRopeThreads), 0, stream, P);
        if (err != cudaSuccess) return err;
        err = launch_overlapped(cache_zero_tail_kernel, dim3(P.B), dim3(kRopeThreads), 0, stream,
                                P);
        if (err != cudaSuccess) return err;
        auto kernel = P.kind == kLayerSliding
                          ? attn_kernel_for<kKvFromRing, kLayerSliding>(P.G)
                          : attn_kernel_for<kKvFromCache, kLayerFull>(P.G);
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   kAttnSmemBytes);
        if (err != cudaSuccess) return err;
        return launch_overlapped(kernel, dim3(grid), dim3(kAttnThreads), kAttnSmemBytes, stream,
                                 tm_q, tm_kv_k, tm_kv_v, tm_krot, tm_out, P);
    }
    if (P.rot_w > 0) {
        const long long items = r / 16 + (P.rot_w - r) / 8;
        const long long threads = static_cast<long long>(P.B) * P.T * items;
        const long long blocks = (threads + kRopeThreads - 1) / kRopeThreads;
        err = launch_overlapped(prefill_rope_k_kernel, dim3(static_cast<unsigned>(blocks)),
                                dim3(kRopeThreads), 0, stream, P);
        if (err != cudaSuccess) return err;
    }
    auto kernel = P.kind == kLayerSliding ? attn_kernel_for<kKvFromQkv, kLayerSliding>(P.G)
                                          : attn_kernel_for<kKvFromQkv, kKindAny>(P.G);
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kAttnSmemBytes);
    if (err != cudaSuccess) return err;
    err = launch_overlapped(kernel, dim3(grid), dim3(kAttnThreads), kAttnSmemBytes, stream, tm_q,
                            tm_kv_k, tm_kv_v, tm_krot, tm_out, P);
    if (err != cudaSuccess || P.k_cache == nullptr) return err;
    // fill the decode cache (it reads only qkv and pos)
    return launch_overlapped(prefill_store_kv_kernel, dim3(static_cast<unsigned>(store_blocks)),
                             dim3(kRopeThreads), 0, stream, P);
}

// The attention kernel of a packed prefill: `items` query tiles (and parts of
// them) at most, per KV head, from the list that the kernel before it made; and
// where tiles may be split, the kernel that joins them.
cudaError_t launch_prefill_packed(const CUtensorMap &tm_q, const CUtensorMap &tm_kv_k,
                                  const CUtensorMap &tm_kv_v, const CUtensorMap &tm_krot,
                                  const CUtensorMap &tm_out, const PrefillParams &P,
                                  long long items, cudaStream_t stream) {
    const bool paged = P.pk.table != nullptr;
    const bool sliding = P.kind == kLayerSliding;
    auto kernel = paged ? (sliding ? attn_kernel_for<kKvPages, kLayerSliding>(P.G)
                                   : attn_kernel_for<kKvPages, kLayerFull>(P.G))
                        : (sliding ? attn_kernel_for<kKvPacked, kLayerSliding>(P.G)
                                   : attn_kernel_for<kKvPacked, kLayerFull>(P.G));
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kAttnSmemBytes);
    if (err != cudaSuccess) return err;
    err = launch_overlapped(kernel, dim3(static_cast<unsigned>(items * P.Hkv)),
                            dim3(kAttnThreads), kAttnSmemBytes, stream, tm_q, tm_kv_k, tm_kv_v,
                            tm_krot, tm_out, P);
    if (err != cudaSuccess || P.pk.part_o == nullptr) return err;
    return launch_overlapped(join_parts_kernel, dim3(static_cast<unsigned>(P.wave)),
                             dim3(kJoinThreads), 0, stream, P);
}

}  // namespace spark
