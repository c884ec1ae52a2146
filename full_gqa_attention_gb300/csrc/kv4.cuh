// kv4.cuh -- keys and values in 4 bits: the format, quantising, reading back,
// and the launch parameters of the calls that use it.
//
// A block of 16 dims x of one token's key (rotated) or value of a KV head is
//     s = e5m3(max |x| / 6),   c_i = e2m1(x_i / s),   x_i ~ c_i s:
// e2m1 are the numbers 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; e5m3 is
// unsigned, 5 bits of exponent and 3 of mantissa, which is a half's bits 7..14,
// so widening a scale is a shift and needs no table, and its range (2^-17 to
// 10240, so values to 61440) needs no further factor per tensor.  Both round to
// nearest, ties to even.  c_i s has six significant bits at most: a half and a
// bf16 hold it exactly.  A block with a value that is not finite gets the scale
// 0xff, a NaN, and reads as NaN.
//
// 4.5 bits a value.  Measured as noise over signal: normal values 0.91 % (0.75 %
// with integers from -7 to 7 in the codes' place), Student's t of 4 degrees 0.85
// (1.16), normal values of log-normal channels 0.85 (1.34): a cache has such
// channels.  Blocks of 32: 1.04, 1.09, 1.17.
//
// A page of a KV head is its slots in groups of 16, 2304 bytes each: 2048 of
// codes, 256 of scales, both in the order in which one warp's matrix
// instructions (m16n8k16, the cache as A) take them, so that a lane reads its
// operands in 16-byte words without a shuffle:
//   K codes  dims 128 h .. 128 h + 127 of slot t: 64 bytes at 1024 h + 64 t, two
//            dims a byte, the even one in the low half
//   K scale  of block b (dims 16 b ..) of slot t: byte
//            2048 + 16 t + 4 (b / 2 % 4) + 2 (b / 8) + b % 2
//   V codes  dim d of slot t: byte 512 (d / 8 % 4) + 64 (d / 32) + 16 (t / 4) +
//            4 (d / 2 % 4) + 2 (t / 2 % 2) + d % 2, low half where t is even
//   V scale  of block b of slot t: byte
//            2048 + 32 (b / 2) + 8 (t / 4) + 4 (b % 2) + 2 (t % 2) + t / 2 % 2
#pragma once

#include <cuda_fp16.h>

#include "paged.cuh"

namespace spark {

constexpr int kKv4Group = 16;                       // slots
constexpr int kKv4Codes = kKv4Group * kHeadDim / 2; // bytes of codes in a group
constexpr int kKv4GroupBytes = kKv4Group * kKv4TokenBytes;
constexpr unsigned kKv4MaxScale = 226;              // 10240: 6 * 10240 is a finite half
constexpr unsigned kKv4NanScale = 0xff;

// Pages in 4 bits: [n_pages][Hkv][page / 16][2304], and the table of the rows.
struct Kv4Pages {
    uint8_t *k, *v;
    const int32_t *table;      // [rows, max_pages]
    int n_pages, page_shift, max_pages;

    // Where a group of 16 slots lies, behind k or v (page id inside the pool).
    __device__ __forceinline__ size_t group(int id, int g, int Hkv, int slot) const {
        const int in = (slot & ((1 << page_shift) - 1)) >> 4;
        return (((static_cast<size_t>(id) * Hkv + g) << (page_shift - 4)) + in) * kKv4GroupBytes;
    }
};

struct Kv4Params {
    const __nv_bfloat16 *qkv;  // [N, (H+2Hkv)*256]
    const float *gate;         // [N, H] (decode)
    const int32_t *pos;        // [N] (decode: [S], -1 idle)
    const int32_t *cu;         // [S + 1] (store)
    const int32_t *begin;      // [S]: first token (store: tokens in the pages; load)
    const int32_t *end;        // [S]: behind the last one (load)
    Kv4Pages pg;
    __nv_bfloat16 *k_pages;    // [n_pages, Hkv, page, 256]: where load writes to
    __nv_bfloat16 *v_pages;
    const int32_t *to_table;   // [S, to_max_pages]
    int to_n_pages, to_page_shift, to_max_pages;
    __nv_bfloat16 *out;        // [S, H*256] (decode)
    unsigned *status;
    float *part_ml;            // decode: states of shared pairs, as PagedParams has them
    float *part_o;
    unsigned *counters;
    int N, S, H, Hkv, G;
    int kind, window, gate_mode;
    int pos_end;               // decode: positions end here
    int heads;                 // store: KV heads of a unit of work
    RopeTable rope;
    double turns[kMaxRopePairs];  // the frequencies in 64 bits
};

// ---------------------------------------------------------------- reading

// Eight codes (dims 0..7 from the lowest four bits up) as halves, two to a word.
__device__ __forceinline__ void kv4_widen(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

__device__ __forceinline__ float kv4_scale(unsigned byte) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// Byte of block b's scale behind a group's codes, slot t.
__device__ __forceinline__ int kv4_key_scale_at(int b, int t) {
    return kKv4Codes + 16 * t + 4 * ((b >> 1) & 3) + 2 * (b >> 3) + (b & 1);
}
// ... of a value's block; slots 4 c .. 4 c + 3 are the bytes 0, 2, 1, 3 behind it.
__device__ __forceinline__ int kv4_value_scale_at(int b, int c) {
    return kKv4Codes + 32 * (b >> 1) + 8 * c + 4 * (b & 1);
}
// The 4 bytes of dims 8 l .. 8 l + 7 of slot t of a key.
__device__ __forceinline__ int kv4_key_at(int l, int t) {
    return 1024 * (l >> 4) + 64 * t + 4 * (l & 15);
}
// The 16 bytes of dims 8 l .. 8 l + 7 of slots 4 c .. 4 c + 3 of a value.
__device__ __forceinline__ int kv4_value_at(int l, int c) {
    return 512 * (l & 3) + 64 * (l >> 2) + 16 * c;
}

// Slots 4 c + t of such a word of values as codes of dims 0..7.
__device__ __forceinline__ uint32_t kv4_value_codes(const uint4 &w, int t) {
    // bytes 2 (t / 2), 2 (t / 2) + 1 of each word: dims 2 i, 2 i + 1
    const int sel = t >> 1 ? 0x7632 : 0x5410;
    uint32_t a = __byte_perm(w.x, w.y, sel), b = __byte_perm(w.z, w.w, sel);
    if (t & 1) {
        a >>= 4;
        b >>= 4;
    }
    a &= 0x0f0f0f0fu;
    b &= 0x0f0f0f0fu;
    a |= a >> 4;
    b |= b >> 4;
    return __byte_perm(a, b, 0x6420);
}

// ---------------------------------------------------------------- quantising

// The scale nearest to t >= 0, in e5m3.
__device__ __forceinline__ unsigned kv4_scale_byte(float t) {
    const unsigned bits = __float_as_uint(t);
    const unsigned normal = ((bits + 0x7ffffu + ((bits >> 20) & 1u)) >> 20) - (112u << 3);
    const unsigned small = static_cast<unsigned>(__float2int_rn(t * 131072.0f));
    const unsigned b = t < 6.103515625e-5f ? small : normal;
    return b < kKv4MaxScale ? b : kKv4MaxScale;
}

// Eight numbers (already divided by the scale) to codes.
__device__ __forceinline__ uint32_t kv4_codes(const float (&y)[8]) {
    uint32_t c;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(c)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return c;
}

// A warp's row of 256 dims, dims 8 lane .. 8 lane + 7 in a lane: two lanes hold
// a block.  The maximum of both, and whether all of both is finite.
__device__ __forceinline__ float kv4_block_max(const float (&x)[8], bool &finite) {
    float a = 0.f, z = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a = fmaxf(a, fabsf(x[i]));
        z += x[i] * 0.f;
    }
    z += __shfl_xor_sync(0xffffffffu, z, 1);
    finite = z == 0.f;
    return fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
}

// A value's row: bf16, so that the quotients round as exact ones would (x / s
// lies on a border between two codes, where 32 bits hold it, or 2^-12 of itself
// away from it; so does max / 6).
__device__ __forceinline__ void kv4_value_row(const uint4 &raw, uint32_t &codes, unsigned &byte) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
    bool finite;
    const float a = kv4_block_max(x, finite);
    byte = kv4_scale_byte(__fdiv_rn(a, 6.f));
    const float s = kv4_scale(byte);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = s > 0.f ? __fdiv_rn(x[i], s) : 0.f;
    codes = kv4_codes(y);
    if (!finite) {
        codes = 0;
        byte = kKv4NanScale;
    }
}

// Dims 8 lane .. of a key: the lane's own values, those they turn with, and
// where in the turn they stand.
struct KeyTurn {
    float x[8], z[8];
    int k0;                    // the first pair
    bool turns, upper;         // upper: the second of each pair
};

__device__ __forceinline__ KeyTurn kv4_key_turn(const uint4 &raw, int rot_dim, int pos, int lane) {
    KeyTurn t;
    const int half = rot_dim >> 4;  // lanes of each half
    t.turns = lane < 2 * half && pos != 0;
    t.upper = lane >= half;
    const int other = !t.turns ? lane : t.upper ? lane - half : lane + half;
    t.k0 = !t.turns ? 0 : (t.upper ? lane - half : lane) * 8;
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t o = __shfl_sync(0xffffffffu, w[i], other);
        t.x[2 * i] = bf16_lo(w[i]);
        t.x[2 * i + 1] = bf16_hi(w[i]);
        t.z[2 * i] = bf16_lo(o);
        t.z[2 * i + 1] = bf16_hi(o);
    }
    return t;
}

// The rotated values in 32 bits; cs: cos and sin of each pair.
__device__ __forceinline__ void kv4_rotate(const KeyTurn &t, const float2 *cs, float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = t.x[i];
        if (t.turns) {
            const float2 c = cs[t.k0 + i];
            y[i] = __fmaf_rn(t.x[i], c.x, t.upper ? __fmul_rn(t.z[i], c.y) : -__fmul_rn(t.z[i], c.y));
        }
    }
}

// Value i of a turned key in 64 bits.
__device__ __noinline__ inline double kv4_exact_turn(float x, float z, bool upper, int pos, double u) {
    const double p = pos * u;
    const double t = (p - rint(p)) + fma(static_cast<double>(pos), u, -p);
    double s, c;
    sincospi(2.0 * t, &s, &c);
    return upper ? x * c + z * s : x * c - z * s;
}

// Settles what 32 bits leave open of a key's row: its scales where `open_scale`,
// and the codes of the dims in `open`, from the rotation in 64 bits.  All lanes
// of the warp; `open_scale` is the same in the two lanes of a block.
__device__ __noinline__ inline void kv4_settle(const KeyTurn &t, int pos, const double *turns,
                                        bool open_scale, unsigned open, uint32_t &codes,
                                        unsigned &byte) {
    auto exact = [&](int i) {
        return t.turns ? kv4_exact_turn(t.x[i], t.z[i], t.upper, pos, turns[t.k0 + i])
                       : static_cast<double>(t.x[i]);
    };
    if (__any_sync(0xffffffffu, open_scale)) {
        double a = 0.0;
        if (open_scale) {
            open = 0xff;
            for (int i = 0; i < 8; ++i) a = fmax(a, fabs(exact(i)));
        }
        a = fmax(a, __shfl_xor_sync(0xffffffffu, a, 1));
        if (open_scale) {
            // the two scales around a / 6, and their middle
            const double want = a / 6.0;
            unsigned lo = kv4_scale_byte(static_cast<float>(want));
            if (lo > 0 && kv4_scale(lo) > want) --lo;
            byte = lo;
            if (lo < kKv4MaxScale) {
                const double mid = 0.5 * (static_cast<double>(kv4_scale(lo)) + kv4_scale(lo + 1));
                if (want > mid || (want == mid && (lo & 1u))) byte = lo + 1;
            }
        }
    }
    const double s = kv4_scale(byte);
    for (int i = 0; i < 8; ++i) {
        if (!(open >> i & 1u)) continue;
        const double v = exact(i), m = fabs(v);
        unsigned c = 0;
        if (s > 0.0)
            c = (m > 0.25 * s) + (m >= 0.75 * s) + (m > 1.25 * s) + (m >= 1.75 * s) +
                (m > 2.5 * s) + (m >= 3.5 * s) + (m > 5.0 * s);
        if (v < 0.0) c |= 8u;
        codes = (codes & ~(15u << (4 * i))) | c << (4 * i);
    }
}

// A key's row, rotated (y, in 32 bits) and quantised.  What the pages hold is
// the nearest to the exact rotation: where 32 bits do not tell on which side of
// a border a value or a scale lies (one row in some hundreds), 64 bits decide.
// |y| is off by 2^-22 (|x| + |z|) at most: cos and sin by 2^-23 each (1 ulp of
// sincospif, and 2^-24 that the frequencies' two parts leave of the angle below
// 2^24 positions), the product and the sum by 2^-24 each.  Twice that is allowed.
// Dims that do not turn are bf16 and lie on borders often; they divide exactly,
// as a value's do.
__device__ __forceinline__ void kv4_key_row(const KeyTurn &t, const float2 *cs, int pos,
                                            const double *turns, float (&y)[8], uint32_t &codes,
                                            unsigned &byte) {
    kv4_rotate(t, cs, y);
    bool finite;
    const float a = kv4_block_max(y, finite);
    float e = 0.f;
    if (t.turns)
#pragma unroll
        for (int i = 0; i < 8; ++i) e = fmaxf(e, fabsf(t.x[i]) + fabsf(t.z[i]));
    e *= 4.76837158e-7f;  // 2^-21
    const float other = __shfl_xor_sync(0xffffffffu, e, 1);  // (a block turns as a whole)
    const float most = t.turns ? fmaf(a, 2.38418579e-7f, fmaxf(e, other)) : 0.f;
    byte = kv4_scale_byte(__fdiv_rn(fmaxf(a - most, 0.f), 6.f));
    const bool open_scale = byte != kv4_scale_byte(__fdiv_rn(a + most, 6.f));
    const float s = kv4_scale(byte);
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = t.turns ? y[i] * r : s > 0.f ? __fdiv_rn(y[i], s) : 0.f;
        const float d = t.turns ? __fmaf_rn(fabsf(q), 2.38418579e-7f, e * r) : 0.f;
        lo[i] = q - d;
        hi[i] = q + d;
    }
    codes = kv4_codes(hi);
    // (a sign that differs beside zero stands for the same value)
    unsigned differ = codes ^ kv4_codes(lo);
    differ = (differ | differ >> 1 | differ >> 2) & 0x11111111u;
    if (!finite) {
        codes = 0;
        byte = kKv4NanScale;
        differ = 0;
    }
    const bool settle = differ != 0 || (open_scale && finite);
    if (__any_sync(0xffffffffu, settle)) {
        unsigned open = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) open |= (differ >> (4 * i) & 1u) << i;
        kv4_settle(t, pos, turns, open_scale && finite, open, codes, byte);
    }
}

}  // namespace spark
