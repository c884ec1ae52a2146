// decode_kv4.cu -- one decode step over a cache in 4 bits (format: kv4.cuh).
//
// For every row b and KV head g the G query heads of the group attend to the
// cached slots [lo, pos) of the row's pages, as they are held, and to the new
// token itself, as it is:
//     out = sigma(gate) * sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
// with s_j = q.k_j / 16.  The new token's key and value are quantised into
// slot pos.
#include "kv4.cuh"

namespace spark {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

}  // namespace

// One CTA per pair of a row and a KV head, a warp per slot in turn.
__global__ void __launch_bounds__(kThreads) decode_kv4_kernel(const __grid_constant__ Kv4Params P) {
    __shared__ float2 cs[kMaxRopePairs];
    __shared__ float sm_m[kWarps][8], sm_l[kWarps][8];
    __shared__ float sm_o[kWarps][8][kHeadDim];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.y, g = blockIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    const int pos = P.pos[b];
    if (pos < 0 || pos >= P.pos_end) {
        if (g == 0 && tid == 0 && pos != -1) atomicOr(P.status, kErrPosition);
        return;
    }
    const int half = P.rope.rot_dim / 2;
    if (tid < half) rope_cos_sin_fine(pos, P.rope.u[tid], cs[tid].x, cs[tid].y);
    __syncthreads();
    const __nv_bfloat16 *x = P.qkv + static_cast<size_t>(b) * (P.H + 2 * P.Hkv) * kHeadDim;
    float q[8][8];
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        if (h >= P.G) break;
        const uint4 raw = *reinterpret_cast<const uint4 *>(x + (g * P.G + h) * kHeadDim + lane * 8);
        kv4_rotate(kv4_key_turn(raw, P.rope.rot_dim, pos, lane), cs, q[h]);
    }
    const int lo = P.kind == 1 && pos >= P.window ? pos - P.window + 1 : 0;
    const int32_t *table = P.pg.table + static_cast<size_t>(b) * P.pg.max_pages;
    float m[8], l[8], o[8][8];
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[h][i] = 0.f;
    }
    auto add = [&](const float (&k)[8], const float (&v)[8]) {
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            if (h >= P.G) break;
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) d = fmaf(q[h][i], k[i], d);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
            const float s = d * kScaleLog2, n = fmaxf(m[h], s), z = n == -INFINITY ? 0.f : n;
            const float w = fast_exp2(m[h] - z), p = fast_exp2(s - z);
            m[h] = n;
            l[h] = l[h] * w + p;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[h][i] = o[h][i] * w + p * v[i];
        }
    };
    for (int j = lo + warp; j < pos; j += kWarps) {
        const int id = table[j >> P.pg.page_shift], t = j & 15;
        uint32_t kc = 0, vc = 0;
        float ks = 0.f, vs = 0.f;
        if (id >= 0 && id < P.pg.n_pages) {
            const size_t at = P.pg.group(id, g, P.Hkv, j);
            kc = *reinterpret_cast<const uint32_t *>(P.pg.k + at + kv4_key_at(lane, t));
            ks = kv4_scale(P.pg.k[at + kv4_key_scale_at(lane >> 1, t)]);
            vc = kv4_value_codes(
                *reinterpret_cast<const uint4 *>(P.pg.v + at + kv4_value_at(lane, t >> 2)), t & 3);
            vs = kv4_scale(P.pg.v[at + kv4_value_scale_at(lane >> 1, t >> 2) + 2 * (t & 1) +
                                  (t >> 1 & 1)]);
        } else if (lane == 0) {
            atomicOr(P.status, kErrPage);
        }
        uint32_t h[4];
        float k[8], v[8];
        kv4_widen(kc, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            k[2 * i] = f.x * ks;
            k[2 * i + 1] = f.y * ks;
        }
        kv4_widen(vc, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            v[2 * i] = f.x * vs;
            v[2 * i + 1] = f.y * vs;
        }
        add(k, v);
    }
    if (warp == 0) {  // the new token: joined as it is, stored in 4 bits
        const uint4 kr = *reinterpret_cast<const uint4 *>(x + (P.H + g) * kHeadDim + lane * 8);
        const uint4 vr =
            *reinterpret_cast<const uint4 *>(x + (P.H + P.Hkv + g) * kHeadDim + lane * 8);
        float k[8], v[8];
        uint32_t kc, vc;
        unsigned kb, vb;
        kv4_key_row(kv4_key_turn(kr, P.rope.rot_dim, pos, lane), cs, pos, P.turns, k, kc, kb);
        kv4_value_row(vr, vc, vb);
        const uint32_t w[4] = {vr.x, vr.y, vr.z, vr.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
        add(k, v);
        const int id = table[pos >> P.pg.page_shift], t = pos & 15;
        if (id < 0 || id >= P.pg.n_pages) {
            if (lane == 0) atomicOr(P.status, kErrPage);
        } else {
            const size_t at = P.pg.group(id, g, P.Hkv, pos);
            *reinterpret_cast<uint32_t *>(P.pg.k + at + kv4_key_at(lane, t)) = kc;
            uint8_t *dst = P.pg.v + at + kv4_value_at(lane, t >> 2) + 2 * (t >> 1 & 1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint8_t &byte = dst[4 * (i >> 1) + (i & 1)];
                const unsigned c = vc >> (4 * i) & 15u;
                byte = t & 1 ? (byte & 0x0f) | c << 4 : (byte & 0xf0) | c;
            }
            if (!(lane & 1)) {
                P.pg.k[at + kv4_key_scale_at(lane >> 1, t)] = kb;
                P.pg.v[at + kv4_value_scale_at(lane >> 1, t >> 2) + 2 * (t & 1) + (t >> 1 & 1)] =
                    vb;
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        if (h >= P.G) break;
        if (lane == 0) {
            sm_m[warp][h] = m[h];
            sm_l[warp][h] = l[h];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sm_o[warp][h][lane * 8 + i] = o[h][i];
    }
    __syncthreads();
    for (int h = warp; h < P.G; h += kWarps) {
        float M = -INFINITY, L = 0.f, y[8] = {};
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][h]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = fast_exp2(sm_m[w][h] - M);
            L += sm_l[w][h] * f;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] += sm_o[w][h][lane * 8 + i] * f;
        }
        const int head = g * P.G + h;
        const float c = gate_act(P.gate[static_cast<size_t>(b) * P.H + head], P.gate_mode) / L;
        *reinterpret_cast<uint4 *>(P.out + (static_cast<size_t>(b) * P.H + head) * kHeadDim +
                                   lane * 8) =
            make_uint4(pack_bf16x2(y[0] * c, y[1] * c), pack_bf16x2(y[2] * c, y[3] * c),
                       pack_bf16x2(y[4] * c, y[5] * c), pack_bf16x2(y[6] * c, y[7] * c));
    }
}

// ---------------------------------------------------------------- launcher

cudaError_t launch_decode_kv4(const Kv4Params &P, int, cudaStream_t stream) {
    return launch_overlapped(decode_kv4_kernel, dim3(P.Hkv, P.S), dim3(kThreads), 0, stream, P);
}

}  // namespace spark
