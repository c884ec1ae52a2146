// paged.cuh -- launch parameters and helpers of the packed and paged
// attention calls.
#pragma once

#include "common.cuh"

namespace spark {

struct PagedParams {
    const __nv_bfloat16 *qkv;  // [N, (H+2Hkv)*256]
    const float *gate;         // [N, H]
    const int32_t *pos;        // [N] (decode: [B], -1 idle)
    const int32_t *cu;         // [S + 1] (prompts)
    const int32_t *start;      // [S]: tokens in the pages (paged prompts)
    __nv_bfloat16 *k_pages;    // [n_pages, Hkv, page, 256]; nullptr: no cache
    __nv_bfloat16 *v_pages;
    const int32_t *table;      // [rows, max_pages]
    __nv_bfloat16 *out;        // [N, H*256]
    unsigned *status;
    __nv_bfloat16 *krot;       // [Hkv, N, rot_w]: rotated leading key dims (packed prompts)
    int rot_w;
    int32_t *tile_base;        // [S + 1]: query tiles before each sequence
    PackedItem *work;          // query tiles (common.cuh: PackedItem), and -1 behind them
    int most;                  // places in the list
    int sms, slots;            // CTAs at a time, places for states of split tiles
    PackedItem *splits;        // common.cuh: PackedInfo
    int *n_splits;
    unsigned *odd_values;      // common.cuh: PackedInfo
    unsigned *call;
    float *part_ml;            // decode: [grid, 2, G, 2] running max (base-2 units), sum
    float *part_o;             // decode: [grid, 2, G, 256] unnormalised outputs
                               // (prompts: states of split query tiles, PackedInfo)
    unsigned *counters;        // decode: a byte per CTA, left at 0 by every call
    int N, S, H, Hkv, G;
    int kind, window, gate_mode;
    int n_pages, page_shift, max_pages;
    int pos_end;               // decode: positions end here (the table, the rotation)
    RopeTable rope;
};

// Positions that RoPE takes: fp32 holds them (rope_math.cuh).
constexpr int kRopePositions = 1 << 24;

// rope_cos_sin with the last rounding of the angle given back: the sum f + g of
// the reduced angle's two parts (rope_math.cuh: rope_turns) is off by up to
// 2^-25 turns, 2e-7 rad, which TwoSum recovers exactly and a first-order step
// applies.  For keys that go to pages: the angle error then no longer flips the
// last bit of a stored bf16 more often than 32-bit products do.
__device__ __forceinline__ void rope_cos_sin_fine(int pos, float2 u, float &c, float &s) {
    const float fp = static_cast<float>(pos);
    const float p = __fmul_rn(fp, u.x);
    const float f = __fadd_rn(p, -rintf(p));
    const float g = __fmaf_rn(fp, u.y, __fmaf_rn(fp, u.x, -p));
    const float t = __fadd_rn(f, g);
    const float b = __fadd_rn(t, -f);
    const float err = __fadd_rn(__fadd_rn(f, -__fadd_rn(t, -b)), __fadd_rn(g, -b));
    float c0, s0;
    sincospif(__fmul_rn(2.0f, t), &s0, &c0);
    const float d = err * 6.283185307f;
    c = __fmaf_rn(-d, s0, c0);
    s = __fmaf_rn(d, c0, s0);
}

// The sequence whose tokens [cu[s], cu[s+1]) hold `row`, or -1 (padding, or
// offsets that are no prefix sum), by one warp: 32 probes a step.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int S, int row, int lane) {
    int lo = 0, n = S + 1;  // the last s with cu[s] <= row lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const unsigned hit = __ballot_sync(0xffffffffu, at < n && cu[lo + at] <= row);
        const int last = hit ? 31 - __clz(hit) : 0;
        lo += last * step;
        n = n - last * step < step ? n - last * step : step;
    }
    return (lo < S && cu[lo] <= row && row < cu[lo + 1]) ? lo : -1;
}

}  // namespace spark
