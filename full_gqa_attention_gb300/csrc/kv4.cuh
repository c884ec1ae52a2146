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
constexpr float kKv4LeastNormal = 6.103515625e-5f;  // 2^-14, of a scale

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
    const int32_t *begin;      // [S]: tokens in the pages (store)
    Kv4Pages pg;
    __nv_bfloat16 *out;        // [S, H*256] (decode)
    unsigned *status;
    float *part_ml;            // decode: states of shared pairs, as PagedParams has them
    float *part_o;
    unsigned *counters;        // decode: the header's words behind the status word
    int N, S, H, Hkv, G;
    int kind, window, gate_mode;
    int pos_end;               // decode: positions end here
    RopeTable rope;
    unsigned long long turns[kMaxRopePairs];  // the frequencies, in 2^-64 turns per position
};

struct Kv4LoadParams {
    const int32_t *begin, *end;  // [S]: first token, behind the last one
    Kv4Pages pg;
    __nv_bfloat16 *k_pages;    // [n_pages, Hkv, page, 256]
    __nv_bfloat16 *v_pages;
    const int32_t *to_table;   // [S, to_max_pages]
    int to_n_pages, to_page_shift, to_max_pages;
    unsigned *status;
    int S, Hkv;
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

// The scale nearest to t >= 0, in e5m3: the upper bits of a float, rounded, with
// the exponent moved.  Below 2^-14 the steps stay those of the binade above, which
// adding 2^-14 makes them.
__device__ __forceinline__ unsigned kv4_scale_byte(float t) {
    const bool small = t < kKv4LeastNormal;
    const unsigned bits = __float_as_uint(t + (small ? kKv4LeastNormal : 0.f));
    const unsigned b = ((bits + 0x7ffffu + (bits >> 20 & 1u)) >> 20) - (small ? 904u : 896u);
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
// a block.

__device__ __forceinline__ void kv4_floats(const uint4 &raw, float (&x)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ bool kv4_finite(const uint4 &raw) {
    // an exponent of all ones carries into the sign's place
    const uint32_t c = ((raw.x & 0x7f807f80u) + 0x00800080u) | ((raw.y & 0x7f807f80u) + 0x00800080u) |
                       ((raw.z & 0x7f807f80u) + 0x00800080u) | ((raw.w & 0x7f807f80u) + 0x00800080u);
    return !(c & 0x80008000u);
}

// The largest of three sizes, NaN where one is; the largest of a lane's eight.
__device__ __forceinline__ float kv4_larger(float a, float b, float c = 0.f) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
__device__ __forceinline__ float kv4_largest(const float (&x)[8]) {
    return kv4_larger(kv4_larger(x[0], x[1], x[2]), kv4_larger(x[3], x[4], x[5]),
                      kv4_larger(x[6], x[7]));
}

__device__ __forceinline__ float kv4_reciprocal(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return s > 0.f ? r : 0.f;
}

// What an exact quotient by a scale (or by 6) rounds to is told by one that is
// off by 2^-22, where the number divided is bf16: the quotient lies on a border
// between two codes (or scales), which have few bits, or 2^-9 of itself away
// from it.  So a maximum's sixth keeps sixteen bits, and a quotient, which is 8 at
// most or saturates, what is left of it beside kSnap: multiples of 2^-13.
__device__ __forceinline__ float kv4_snap(float y) {
    return __uint_as_float((__float_as_uint(y) + 0x80u) & 0xffffff00u);
}

constexpr float kSnap = 1536.0f;
constexpr float kSixth = 1.0f / 6.0f;

// N values' rows: their chains interleave.
template <int N>
__device__ __forceinline__ void kv4_value_rows(const uint4 (&raw)[N], uint32_t (&codes)[N],
                                               unsigned (&byte)[N]) {
    bool odd = false;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float x[8];
        kv4_floats(raw[n], x);
        float a = kv4_largest(x);
        a = kv4_larger(a, __shfl_xor_sync(0xffffffffu, a, 1));
        byte[n] = kv4_scale_byte(kv4_snap(a * kSixth));
        const float r = kv4_reciprocal(kv4_scale(byte[n]));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmaf_rn(x[i], r, kSnap), -kSnap);
        codes[n] = kv4_codes(x);
        odd = odd || !(a < INFINITY);
    }
    if (__any_sync(0xffffffffu, odd))
#pragma unroll
        for (int n = 0; n < N; ++n) {
            int bad = !kv4_finite(raw[n]);
            bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
            if (bad) {
                codes[n] = 0;
                byte[n] = kKv4NanScale;
            }
        }
}

// How a lane's dims 8 lane .. of a key turn: y = x cos + z sin, where z are the dims
// of the other end (with the sign changed in the first of each pair).
struct KeyTurn {
    int partner;               // the lane that has the others
    int k0;                    // the first pair
    bool turns;
    uint32_t sign;
};

__device__ __forceinline__ KeyTurn kv4_key_turn(int rot_dim, int pos, int lane) {
    KeyTurn t;
    const int half = rot_dim >> 4;  // lanes of each half
    const bool inside = lane < 2 * half, upper = lane >= half;
    t.turns = inside && pos != 0;
    t.partner = !inside ? lane : upper ? lane - half : lane + half;
    t.k0 = !inside ? 0 : (upper ? lane - half : lane) * 8;
    t.sign = upper ? 0u : 0x80008000u;
    return t;
}

// The lane's dims of a row (512 bytes in shared memory), and the other end's.
__device__ __forceinline__ uint4 kv4_own(const uint8_t *row, int lane) {
    return *reinterpret_cast<const uint4 *>(row + lane * 16);
}
__device__ __forceinline__ uint4 kv4_other(const uint8_t *row, int partner, uint32_t sign) {
    const uint4 z = *reinterpret_cast<const uint4 *>(row + partner * 16);
    return make_uint4(z.x ^ sign, z.y ^ sign, z.z ^ sign, z.w ^ sign);
}

// The rotated values in 32 bits; c, s: cosines and sines of the lane's pairs, 1 and
// 0 for dims that do not turn.
__device__ __forceinline__ void kv4_rotate(const KeyTurn &t, const uint8_t *row, int lane,
                                           const float (&c)[8], const float (&s)[8],
                                           float (&y)[8]) {
    float z[8];
    kv4_floats(kv4_own(row, lane), y);
    kv4_floats(kv4_other(row, t.partner, t.sign), z);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmaf_rn(y[i], c[i], __fmul_rn(z[i], s[i]));
}
// ... from a table of all pairs.
__device__ __forceinline__ void kv4_rotate(const KeyTurn &t, const uint8_t *row, int lane,
                                           const float2 *cs, float (&y)[8]) {
    kv4_floats(kv4_own(row, lane), y);
    if (!t.turns) return;
    float z[8];
    kv4_floats(kv4_other(row, t.partner, t.sign), z);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 c = cs[t.k0 + i];
        y[i] = __fmaf_rn(y[i], c.x, __fmul_rn(z[i], c.y));
    }
}

// The product of two numbers in units of 2^-62.
__device__ __forceinline__ long long kv4_mul62(long long a, long long b) {
    return __mul64hi(a, b) << 2;
}

// A number in units of 2^-62 as the sum of two floats.
__device__ __forceinline__ float2 kv4_two_floats(long long a) {
    const float hi = __ll2float_rn(a);
    const float lo = __ll2float_rn(a - __float2ll_rn(hi));
    return make_float2(hi * 0x1p-62f, lo * 0x1p-62f);
}

// Cosine (x, y) and sine (z, w) of position `pos`'s turn, each as the sum of two
// floats, to 2^-48 for the given `turn`: a position's in units of 2^-64 turns, so
// that a product of 64 bits leaves the part behind whole turns.  (The turn itself is
// the host's 64-bit float: the real number's at position p is p 2^-54 turns off at
// most, 2^-36 at 262,144.  That float is what "exact" means.)  By the series, to the
// 17th power of an angle of an eighth of a turn at most, in whole numbers: 64-bit
// floats are some twenty times slower on this chip.
__device__ __noinline__ inline float4 kv4_exact_turn(int pos, unsigned long long turn) {
    const unsigned long long t = pos * turn;
    const unsigned long long quarter = (t + (1ull << 61)) >> 62;
    const long long r = static_cast<long long>(t - (quarter << 62));
    const long long a = kv4_mul62(r, 7244019458077122842ll);  // half of pi
    const long long a2 = kv4_mul62(a, a);
    long long c = 220414ll;
    c = -52899477ll + kv4_mul62(c, a2);
    c = 9627704831ll + kv4_mul62(c, a2);
    c = -1270857037706ll + kv4_mul62(c, a2);
    c = 114377133393536ll + kv4_mul62(c, a2);
    c = -6405119470038039ll + kv4_mul62(c, a2);
    c = 192153584101141163ll + kv4_mul62(c, a2);
    c = -2305843009213693952ll + kv4_mul62(c, a2);
    long long s = 12966ll;
    s = -3526632ll + kv4_mul62(s, a2);
    s = 740592679ll + kv4_mul62(s, a2);
    s = -115532457973ll + kv4_mul62(s, a2);
    s = 12708570377060ll + kv4_mul62(s, a2);
    s = -915017067148291ll + kv4_mul62(s, a2);
    s = 38430716820228233ll + kv4_mul62(s, a2);
    s = -768614336404564651ll + kv4_mul62(s, a2);
    c = (1ll << 62) + kv4_mul62(c, a2);
    s = a + kv4_mul62(kv4_mul62(s, a2), a);
    const int q = static_cast<int>(quarter) & 3;  // turned on by quarters
    const long long cq = q == 0 ? c : q == 1 ? -s : q == 2 ? -c : s;
    const long long sq = q == 0 ? s : q == 1 ? c : q == 2 ? -s : -c;
    const float2 x = kv4_two_floats(cq), y = kv4_two_floats(sq);
    return make_float4(x.x, x.y, y.x, y.y);
}

__device__ __forceinline__ float kv4_pick(const uint4 &raw, int i) {
    const uint32_t w = i < 4 ? (i < 2 ? raw.x : raw.y) : (i < 6 ? raw.z : raw.w);
    return i & 1 ? bf16_hi(w) : bf16_lo(w);
}

// |x cos + z sin| as the sum of two floats, and its sign.  Where finite numbers turn
// into one past the largest, of which 32 bits have only the half, the first is infinity.
__device__ __forceinline__ float2 kv4_exact_size(float x, float z, int pos,
                                                 unsigned long long turn, bool &negative) {
    const float4 t = kv4_exact_turn(pos, turn);
    const bool large = fmaxf(fabsf(x), fabsf(z)) >= 0x1p126f;
    x = large ? 0.5f * x : x;
    z = large ? 0.5f * z : z;
    const float p = __fmul_rn(x, t.x), q = __fmul_rn(z, t.z);
    const float sum = __fadd_rn(p, q), back = __fadd_rn(sum, -p);
    float rest = __fadd_rn(__fadd_rn(p, -__fadd_rn(sum, -back)), __fadd_rn(q, -back));
    rest += __fmaf_rn(x, t.x, -p) + __fmaf_rn(z, t.z, -q) + __fmaf_rn(x, t.y, z * t.w);
    float hi = __fadd_rn(sum, rest), lo = __fadd_rn(rest, -__fadd_rn(hi, -sum));
    negative = hi < 0.f;
    hi = large ? 2.f * hi : hi;
    lo = large ? 2.f * lo : lo;
    return negative ? make_float2(-hi, -lo) : make_float2(hi, lo);
}

// Settles the scale of the blocks in `open` (the same in a block's two lanes) from
// the exact rotation.  turns: the lane's pairs' (kv4_exact_turn); maybe: bit 4 i,
// dims that can be the largest.  All lanes.
__device__ __forceinline__ unsigned kv4_settle_scale(const uint4 &own, const uint4 &other, int pos,
                                                     const unsigned long long *turns,
                                                     unsigned maybe, bool open, unsigned byte) {
    float2 a = make_float2(0.f, 0.f);
    if (open)
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            if (!(maybe >> (4 * i) & 1u)) continue;
            bool negative;
            const float2 v =
                kv4_exact_size(kv4_pick(own, i), kv4_pick(other, i), pos, turns[i], negative);
            if (v.x > a.x || (v.x == a.x && v.y > a.y)) a = v;
        }
    const float2 b = make_float2(__shfl_xor_sync(0xffffffffu, a.x, 1),
                                 __shfl_xor_sync(0xffffffffu, a.y, 1));
    if (b.x > a.x || (b.x == a.x && b.y > a.y)) a = b;
    if (!open) return byte;
    // the scale below a / 6, the next one, and their middle (a few bits each: exact)
    unsigned lo = kv4_scale_byte(a.x * kSixth);
    if (lo > 0 && 6.f * kv4_scale(lo) > a.x) --lo;
    if (lo == kKv4MaxScale) return lo;
    const float mid = 3.f * (kv4_scale(lo) + kv4_scale(lo + 1));
    const float over = (a.x - mid) + a.y;
    return over > 0.f || (over == 0.f && (lo & 1u)) ? lo + 1 : lo;
}

// Settles the codes of the dims in `open` (bit 4 i) from the exact rotation.
__device__ __forceinline__ uint32_t kv4_settle_codes(const uint4 &own, const uint4 &other, int pos,
                                                     const unsigned long long *turns, float s,
                                                     unsigned open, uint32_t codes) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        if (!(open >> (4 * i) & 1u)) continue;
        bool negative;
        const float2 m =
            kv4_exact_size(kv4_pick(own, i), kv4_pick(other, i), pos, turns[i], negative);
        // (borders have few bits: exact; so is a difference from one nearby)
        auto over = [&](float border) { return __fadd_rn(m.x, -border * s) + m.y; };
        unsigned c = (over(0.25f) > 0.f) + (over(0.75f) >= 0.f) + (over(1.25f) > 0.f) +
                     (over(1.75f) >= 0.f) + (over(2.5f) > 0.f) + (over(3.5f) >= 0.f) +
                     (over(5.f) > 0.f);
        if (negative) c |= 8u;
        codes = (codes & ~(15u << (4 * i))) | c << (4 * i);
    }
    return codes;
}

// A key's row, rotated (y, in 32 bits), quantised.  What the pages hold is the
// nearest to the exact rotation: where 32 bits do not tell on which side of a
// border a value or a scale lies (one row in some hundreds), more bits decide.
// Let N be the larger of the two blocks' largest |y| times 2^(1/2): a turn keeps
// x^2 + z^2, so no (x, z) of the block is longer.  (cos, sin) is off by less than
// 2^-21.2, as a vector: each of two turns put together by 2^-23.5 (1 ulp of
// sincospif, 2^-24, in each component) and 2^-24.5 (its correction's rounding),
// their product by 2^-23.5, and 2^-24 is the angle's, which the frequencies' two
// parts leave below 2^24 positions.  The product and the sum round by 2^-24 N
// each.  In all |y| is off by 2^-20.8 N at most; 2^-20.7 is allowed, and of a
// quotient (7 at most, or it saturates) also 2^-22 of it.  Dims that do not turn
// are bf16: kSnap.
constexpr float kKeyRel = 2.38418579e-7f, kKeyAbs = 8.31e-7f;  // 2^-22, 2^(1/2 - 20.7)

// Does the error e of a block's maximum reach the border between its scale and a
// next one?  top: a sixth of the maximum.
__device__ __forceinline__ bool kv4_scale_open(float top, float e) {
    const float moved = top + (top < kKv4LeastNormal ? kKv4LeastNormal : 0.f);
    const float border = __uint_as_float((__float_as_uint(moved) & 0xfff00000u) | 0x80000u);
    return fabsf(moved - border) <= fmaf(e, kSixth, moved * kKeyRel);
}

// Codes of rotated values under scale s, and which of them (bit 4 i) the values'
// error e leaves open.  kAll: every lane turns.
template <bool kAll>
__device__ __forceinline__ uint32_t kv4_key_codes(const float (&y)[8], float s, float e,
                                                  bool turns_here, unsigned &open) {
    const float r = kv4_reciprocal(s), d = fmaf(e, r, 8.f * kKeyRel);
    float lo[8], hi[8];
    if (kAll) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __fmaf_rn(y[i], r, -d);
            hi[i] = __fmaf_rn(y[i], r, d);
        }
    } else {
        // both ends of what a quotient can be, or itself, snapped
        const float down = turns_here ? -d : kSnap, up = turns_here ? d : kSnap;
        const float back = turns_here ? 0.f : -kSnap;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __fadd_rn(__fmaf_rn(y[i], r, down), back);
            hi[i] = __fadd_rn(__fmaf_rn(y[i], r, up), back);
        }
    }
    const uint32_t codes = kv4_codes(hi);
    // (a sign that differs beside zero stands for the same value; quotients that are
    // known to a quarter only, of rotations that cancel, can be of either sign)
    open = codes ^ kv4_codes(lo);
    open = (open | open >> 1 | open >> 2) & 0x11111111u;
    if (turns_here && d >= 0.25f) open = 0x11111111u;
    return codes;
}

// Codes (x) and scale (y) of a row some block of which is open or not finite.
// (Out of line, arguments by value: nothing of it is held where it is not called.)
__device__ __noinline__ inline uint2 kv4_key_row_settled(KeyTurn t, const uint8_t *row, int lane,
                                                         int pos, const unsigned long long *turns,
                                                         float4 y0, float4 y1, float a, float e,
                                                         bool turns_here, bool open_scale) {
    const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
    const uint4 own = kv4_own(row, lane), other = kv4_other(row, t.partner, t.sign);
    int bad = !kv4_finite(own) || !kv4_finite(other);
    bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
    // A block's lanes may turn with different blocks: what the maximum may be off by, and
    // whether that reaches a border, is the larger of what its lanes say.
    int settle = open_scale;
    settle |= __shfl_xor_sync(0xffffffffu, settle, 1);
    e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, 1));
    const float top = a * kSixth, least = a - 2.f * fmaf(a, kKeyRel, e);
    unsigned byte = kv4_scale_byte(turns_here ? top : kv4_snap(top)), maybe = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) maybe |= fabsf(y[i]) < least ? 0u : 1u << (4 * i);
    byte = kv4_settle_scale(own, other, pos, turns, maybe, turns_here && settle && !bad, byte);
    const float s = kv4_scale(byte);
    unsigned open;
    uint32_t codes = kv4_key_codes<false>(y, s, e, turns_here, open);
    if (bad) return make_uint2(0, kKv4NanScale);
    return make_uint2(kv4_settle_codes(own, other, pos, turns, s, open, codes), byte);
}

// kAll: every lane turns.
template <bool kAll>
__device__ __forceinline__ void kv4_key_row(const KeyTurn &t, const uint8_t *row, int lane,
                                            const float (&y)[8], int pos,
                                            const unsigned long long *turns, uint32_t &codes,
                                            unsigned &byte) {
    const bool turns_here = kAll || t.turns;
    float a = kv4_largest(y);
    a = kv4_larger(a, __shfl_xor_sync(0xffffffffu, a, 1));
    const float a_other = __shfl_sync(0xffffffffu, a, t.partner);
    const float e = fmaxf(a, a_other) * kKeyAbs, top = a * kSixth;
    byte = kv4_scale_byte(turns_here ? top : kv4_snap(top));
    unsigned open;
    codes = kv4_key_codes<kAll>(y, kv4_scale(byte), e, turns_here, open);
    const bool open_scale = (turns_here && kv4_scale_open(top, e)) || !(a < INFINITY);
    if (__any_sync(0xffffffffu, open_scale || open)) {
        const uint2 x = kv4_key_row_settled(t, row, lane, pos, turns + t.k0,
                                            make_float4(y[0], y[1], y[2], y[3]),
                                            make_float4(y[4], y[5], y[6], y[7]), a, e, turns_here,
                                            open_scale);
        codes = x.x;
        byte = x.y;
    }
}

}  // namespace spark
