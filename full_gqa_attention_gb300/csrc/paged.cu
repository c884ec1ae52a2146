// paged.cu -- packed prompts and a cache in pages: the host side and the
// kernels that are not attention itself.
#include <cstring>

#include "paged.cuh"
#include "spark_attn.h"

namespace spark {

void fill_rope_table(const spark_layer_desc *d, RopeTable *t);
spark_status device_ready(int *sms);
spark_status check_layer_desc(const spark_layer_desc *d, int H, int Hkv);

namespace {

constexpr int kStoreThreads = 256;

// Stores the new tokens' rotated keys and their values in the pages.  One
// thread per (token, group of 8 rotated pairs / 8 copied key dims / 8 value
// dims), looping over the KV heads.
template <bool kDecode>
__global__ void __launch_bounds__(kStoreThreads) paged_store_kernel(
    const __grid_constant__ PagedParams P) {
    grid_dep_wait();
    grid_dep_launch();
    const int r = P.rope.rot_dim, half = r / 2;
    const int n_rot = half / 8, n_kcopy = (kHeadDim - r) / 8, n_v = kHeadDim / 8;
    const int items = n_rot + n_kcopy + n_v;
    const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int row = static_cast<int>(idx / items);
    const int it = static_cast<int>(idx % items);
    if (row >= P.N) return;
    const long long cap = static_cast<long long>(P.max_pages) << P.page_shift;
    long long a;  // index in the sequence
    int seq;
    if (kDecode) {
        seq = row;
        a = P.pos[row];
        if (a == -1) return;
        if (a < 0 || a >= cap) {
            if (it == 0) atomicOr(P.status, kErrPosition);
            return;
        }
    } else {
        seq = find_sequence(P.cu, P.S, row);
        if (seq < 0) return;
        const int t0 = P.cu[seq], t1 = P.cu[seq + 1];
        if (t0 < 0 || t1 > P.N) return;
        const long long st = P.start[seq];
        if (st < 0 || st + (t1 - t0) > cap) {
            if (it == 0) atomicOr(P.status, kErrPosition);
            return;
        }
        a = st + (row - t0);
    }
    const int page = P.table[static_cast<size_t>(seq) * P.max_pages + (a >> P.page_shift)];
    if (page < 0 || page >= P.n_pages) {
        if (it == 0) atomicOr(P.status, kErrPage);
        return;
    }
    const size_t width = static_cast<size_t>(P.H + 2 * P.Hkv) * kHeadDim;
    const __nv_bfloat16 *src_k = P.qkv + row * width + static_cast<size_t>(P.H) * kHeadDim;
    const __nv_bfloat16 *src_v = src_k + static_cast<size_t>(P.Hkv) * kHeadDim;
    const size_t head_stride = static_cast<size_t>(kHeadDim) << P.page_shift;
    const size_t slot = static_cast<size_t>(a & ((1 << P.page_shift) - 1));
    const size_t base = page * (head_stride * P.Hkv) + slot * kHeadDim;
    if (it < n_rot) {
        const int k0 = it * 8;
        const int p = P.pos[row];
        float c[8], s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) rope_cos_sin(p, P.rope.u[k0 + i], c[i], s[i]);
        for (int g = 0; g < P.Hkv; ++g) {
            const uint4 x = *reinterpret_cast<const uint4 *>(src_k + g * kHeadDim + k0);
            const uint4 y = *reinterpret_cast<const uint4 *>(src_k + g * kHeadDim + k0 + half);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
            const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
            uint32_t ya[4], yb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y1l, y2l, y1h, y2h;
                rope_rotate(bf16_lo(xw[i]), bf16_lo(yw[i]), c[2 * i], s[2 * i], y1l, y2l);
                rope_rotate(bf16_hi(xw[i]), bf16_hi(yw[i]), c[2 * i + 1], s[2 * i + 1], y1h, y2h);
                ya[i] = pack_bf16x2(y1l, y1h);
                yb[i] = pack_bf16x2(y2l, y2h);
            }
            __nv_bfloat16 *dst = P.k_pages + base + g * head_stride;
            *reinterpret_cast<uint4 *>(dst + k0) = make_uint4(ya[0], ya[1], ya[2], ya[3]);
            *reinterpret_cast<uint4 *>(dst + k0 + half) = make_uint4(yb[0], yb[1], yb[2], yb[3]);
        }
    } else if (it < n_rot + n_kcopy) {
        const int d0 = r + (it - n_rot) * 8;
        for (int g = 0; g < P.Hkv; ++g)
            *reinterpret_cast<uint4 *>(P.k_pages + base + g * head_stride + d0) =
                *reinterpret_cast<const uint4 *>(src_k + g * kHeadDim + d0);
    } else {
        const int d0 = (it - n_rot - n_kcopy) * 8;
        for (int g = 0; g < P.Hkv; ++g)
            *reinterpret_cast<uint4 *>(P.v_pages + base + g * head_stride + d0) =
                *reinterpret_cast<const uint4 *>(src_v + g * kHeadDim + d0);
    }
}

// The plain attention of every row: one warp per (token, query head), lane l
// holding dims 8l..8l+7, keys one after another with an online softmax.
constexpr int kRowWarps = 8;

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(u[i]);
        x[2 * i + 1] = bf16_hi(u[i]);
    }
}

// Rotates this lane's 8 dims of one head (the partner dims live r/16 lanes
// away) and rounds them to bf16.
__device__ __forceinline__ void rotate_lane(float (&x)[8], int pos, const RopeTable &rope,
                                            int lane) {
    const int r = rope.rot_dim, half = r / 2, d0 = lane * 8;
    const int partner = (d0 >= r) ? lane : (d0 < half ? lane + half / 8 : lane - half / 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(0xffffffffu, x[i], partner);
        if (d0 < r) {
            float c, s, y1, y2;
            rope_cos_sin(pos, rope.u[d0 < half ? d0 + i : d0 + i - half], c, s);
            if (d0 < half)
                rope_rotate(x[i], y, c, s, y1, y2);
            else
                rope_rotate(y, x[i], c, s, y1, y2);
            x[i] = __bfloat162float(__float2bfloat16_rn(d0 < half ? y1 : y2));
        }
    }
}

template <bool kDecode>
__global__ void __launch_bounds__(kRowWarps * 32) rows_attn_kernel(
    const __grid_constant__ PagedParams P) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    if (!kDecode && blockIdx.x == 0)
        for (int i = threadIdx.x; i < P.S; i += kRowWarps * 32)
            if (P.cu[i] < 0 || P.cu[i] > P.cu[i + 1] || P.cu[i + 1] > P.N)
                atomicOr(P.status, kErrSeqlens);
    const long long w = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    const int row = static_cast<int>(w / P.H), h = static_cast<int>(w % P.H);
    if (row >= P.N) return;
    const int g = h / P.G;
    int seq, t0 = 0;
    long long at;
    const long long cap = static_cast<long long>(P.max_pages) << P.page_shift;
    if (kDecode) {
        seq = row;
        at = P.pos[row];
        if (at < 0 || at >= cap) return;
    } else {
        seq = find_sequence(P.cu, P.S, row);
        if (seq < 0) return;
        t0 = P.cu[seq];
        const int t1 = P.cu[seq + 1];
        if (t0 < 0 || t1 > P.N) {
            if (lane == 0 && h == 0) atomicOr(P.status, kErrSeqlens);
            return;
        }
        const long long st = P.start ? P.start[seq] : 0;
        if (st < 0 || (P.k_pages && st + (t1 - t0) > cap)) return;
        at = st + (row - t0);
    }
    const size_t width = static_cast<size_t>(P.H + 2 * P.Hkv) * kHeadDim;
    float q[8], o[8], k[8], v[8];
    unpack8(*reinterpret_cast<const uint4 *>(P.qkv + row * width + h * kHeadDim + lane * 8), q);
    if (P.rope.rot_dim > 0) rotate_lane(q, P.pos[row], P.rope, lane);
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0.f;
    long long j = P.kind == kLayerSliding ? at - P.window + 1 : 0;
    for (j = j > 0 ? j : 0; j <= at; ++j) {
        if (P.k_pages) {
            const int page = P.table[static_cast<size_t>(seq) * P.max_pages + (j >> P.page_shift)];
            if (page < 0 || page >= P.n_pages) {
                if (lane == 0) atomicOr(P.status, kErrPage);
                continue;
            }
            const size_t off = ((static_cast<size_t>(page) * P.Hkv + g) << P.page_shift) * kHeadDim +
                               (j & ((1 << P.page_shift) - 1)) * kHeadDim + lane * 8;
            unpack8(*reinterpret_cast<const uint4 *>(P.k_pages + off), k);
            unpack8(*reinterpret_cast<const uint4 *>(P.v_pages + off), v);
        } else {
            const __nv_bfloat16 *src = P.qkv + (t0 + j) * width + (P.H + g) * kHeadDim + lane * 8;
            unpack8(*reinterpret_cast<const uint4 *>(src), k);
            unpack8(*reinterpret_cast<const uint4 *>(src + P.Hkv * kHeadDim), v);
            if (P.rope.rot_dim > 0) rotate_lane(k, P.pos[t0 + j], P.rope, lane);
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= kScaleLog2;
        const float mn = fmaxf(m, s);
        const float z = mn == -INFINITY ? 0.f : mn;
        const float a = fast_exp2(m - z), p = fast_exp2(s - z);
        l = l * a + p;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = o[i] * a + p * v[i];
        m = mn;
    }
    const float scale = gate_act(P.gate[static_cast<size_t>(row) * P.H + h], P.gate_mode) / l;
    *reinterpret_cast<uint4 *>(P.out + (static_cast<size_t>(row) * P.H + h) * kHeadDim + lane * 8) =
        make_uint4(pack_bf16x2(o[0] * scale, o[1] * scale), pack_bf16x2(o[2] * scale, o[3] * scale),
                   pack_bf16x2(o[4] * scale, o[5] * scale), pack_bf16x2(o[6] * scale, o[7] * scale));
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
    P.window = desc->kind == SPARK_LAYER_SLIDING ? desc->window : 0;
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

template <bool kDecode>
spark_status launch_rows(const PagedParams &P, cudaStream_t s) {
    if (P.k_pages) {
        const int r = P.rope.rot_dim;
        const long long items = r / 16 + (kHeadDim - r) / 8 + kHeadDim / 8;
        const long long blocks = (P.N * items + kStoreThreads - 1) / kStoreThreads;
        const spark_status st =
            done(launch_overlapped(paged_store_kernel<kDecode>, dim3(static_cast<unsigned>(blocks)),
                                   dim3(kStoreThreads), 0, s, P));
        if (st != SPARK_OK) return st;
    }
    const long long warps = static_cast<long long>(P.N) * P.H;
    return done(launch_overlapped(rows_attn_kernel<kDecode>,
                                  dim3(static_cast<unsigned>((warps + kRowWarps - 1) / kRowWarps)),
                                  dim3(kRowWarps * 32), 0, s, P));
}

size_t packed_workspace(int, int, int, int, const spark_layer_desc *, bool) {
    return kWorkspaceHeader;
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
    }
    if (workspace_bytes < packed_workspace(N, S, H, Hkv, desc, paged)) return SPARK_ERR_WORKSPACE;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    PagedParams P = make_params(qkv, gate, pos, desc, N, S, H, Hkv, out, workspace);
    P.cu = cu;
    if (paged) {
        P.start = start;
        set_pages(P, k_pages, v_pages, n_pages, page_size, table, max_pages);
    }
    return launch_rows<false>(P, static_cast<cudaStream_t>(stream));
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
    return kWorkspaceHeader;
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
    if (workspace_bytes < spark_attn_decode_paged_workspace_size(B, H, Hkv, desc))
        return SPARK_ERR_WORKSPACE;
    int sms;
    st = device_ready(&sms);
    if (st != SPARK_OK) return st;
    PagedParams P = make_params(qkv, gate, pos, desc, B, B, H, Hkv, out, workspace);
    set_pages(P, k_pages, v_pages, n_pages, page_size, page_table, max_pages);
    return launch_rows<true>(P, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
