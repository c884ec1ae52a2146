// decode_walk.cuh -- how a decode step over pages is shared out: the list of all
// (row, KV head) pairs' tiles, a CTA's walk over its stretch of it, and the
// running state of a query head.
#pragma once

#include "paged.cuh"

namespace spark {

// A quotient of numbers >= 0 that nearly always have 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}

// What a row asks for: its position, first visible slot and tiles (0: nothing).
// kTile: slots of a tile.  kPairCost: what setting a pair up and finishing it
// costs besides, in tiles.
template <int kTile, int kPairCost>
struct DecodeRow {
    int pos, lo, tiles;
    __device__ __forceinline__ int slot0() const { return lo & ~(kTile - 1); }
    // Units of one of its pairs in the list.
    __device__ __forceinline__ long long units() const {
        return tiles ? tiles + kPairCost : 0;
    }
};

template <int kTile, int kPairCost, typename Params>
__device__ __forceinline__ DecodeRow<kTile, kPairCost> decode_row(const Params &P, int b) {
    DecodeRow<kTile, kPairCost> r;
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
template <int kTile, int kPairCost>
struct DecodeWalk {
    long long u, end;   // next unit of the stretch, its end
    long long base;     // first unit of row b
    long long first;    // first unit of the pair
    int b, g, t0, t1;
    DecodeRow<kTile, kPairCost> row;

    // The next pair with tiles in the stretch, from unit u on; false at the
    // end.  b and base are at or before it.
    template <typename Params>
    __device__ __forceinline__ bool load(const Params &P) {
        while (u < end) {
            while (u >= base + P.Hkv * row.units()) {
                if (b + 1 >= P.N) return false;  // the positions changed under the call
                base += P.Hkv * row.units();
                row = decode_row<kTile, kPairCost>(P, ++b);
            }
            const long long n = row.units();
            g = static_cast<int>(quotient(u - base, n));
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

}  // namespace spark
