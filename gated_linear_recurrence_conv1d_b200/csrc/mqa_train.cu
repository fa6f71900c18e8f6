// mqa_train.cu -- local sliding-window MQA for training: the forward that keeps what its gradient
// needs, and the backward pass, for packed documents (bf16, head_dim 256).
//
// Row r = t H + h of a batch row is query head h of token t; all H heads share the keys and values,
// so a batch row is one attention of T H queries over T keys.  With c = scale log2 e and lo_t the
// first key token t sees (its window and its document):
//     s_ri = q~_r . k~_i,   L_r = log2 sum_{lo_t <= i <= t} 2^{c s_ri},   P_ri = 2^{c s_ri - L_r},
//     out_r = sum_i P_ri v_i
// and, given dO = dL/dout,
//     dP_ri = dO_r . v_i,   delta_r = sum_i P_ri dP_ri = dO_r . out_r,   dS_ri = P_ri (dP_ri - delta_r),
//     dq~_r = scale sum_i dS_ri k~_i,   dk~_i = scale sum_r dS_ri q~_r,   dv_i = sum_r P_ri dO_r.
// dq, dk are dq~, dk~ turned back by their positions (the rotation is orthogonal).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace rglru {
namespace mt {

constexpr int D = 256;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------- rotary embedding, documents ----
// cosine and sine of position pos0 + t, pair j, angle and reduction in fp64: [T][d/2]
__global__ void __launch_bounds__(D / 2) mqa_angles_kernel(int pos0, float base, float2* cs) {
    const int j = threadIdx.x, t = blockIdx.x;
    const double ang = ((double)pos0 + t) * pow((double)base, -2.0 * j / D);
    double s, c;
    sincos(ang, &s, &c);
    cs[(size_t)t * (D / 2) + j] = make_float2((float)c, (float)s);
}

// lo[b][t] = max(0, t - w + 1, start of t's document): a running maximum along the row
__global__ void __launch_bounds__(1024) mqa_first_key_kernel(int T, int w, const uint8_t* reset, int* lo) {
    __shared__ int warp_max[32];
    const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int carry = 0;
    for (int t0 = 0; t0 < T; t0 += 1024) {
        const int t = t0 + threadIdx.x;
        int v = (t < T && reset && reset[(size_t)b * T + t]) ? t : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = max(v, u);
        }
        if (lane == 31) warp_max[warp] = v;
        __syncthreads();
        int base = carry, all = carry;
        for (int i = 0; i < 32; ++i) {
            if (i < warp) base = max(base, warp_max[i]);
            all = max(all, warp_max[i]);
        }
        if (t < T) lo[(size_t)b * T + t] = max(max(base, v), t - w + 1);
        carry = all;
        __syncthreads();
    }
}

// thread = (row b, token t, pair j) over the H query heads and the key
__global__ void __launch_bounds__(D / 2) mqa_turn_kernel(int T, int H, const float2* cs, const __nv_bfloat16* q,
                                                         const __nv_bfloat16* k, __nv_bfloat16* q_rot,
                                                         __nv_bfloat16* k_rot) {
    const int j = threadIdx.x, t = blockIdx.x, b = blockIdx.y;
    const float2 a = cs[(size_t)t * (D / 2) + j];
    const size_t tok = (size_t)b * T + t;
    for (int h = 0; h <= H; ++h) {
        const __nv_bfloat16* src = h < H ? q + (tok * H + h) * D : k + tok * D;
        __nv_bfloat16* dst = h < H ? q_rot + (tok * H + h) * D : k_rot + tok * D;
        const float x1 = __bfloat162float(src[j]), x2 = __bfloat162float(src[j + D / 2]);
        dst[j] = __float2bfloat16_rn(x1 * a.x - x2 * a.y);
        dst[j + D / 2] = __float2bfloat16_rn(x2 * a.x + x1 * a.y);
    }
}

struct Args {
    int B, T, H;
    float scale, scale_log2;
    const __nv_bfloat16 *q_rot, *k_rot, *v, *dout;
    const float2* cs;
    const int* lo;
    float* lse;                 // [B, T H], log2 domain
    float* delta;
    __nv_bfloat16 *out, *dq, *dk, *dv;
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
// lane l holds elements 8 l .. 8 l + 7; its pair partner (element +- d/2) is lane l ^ 16
__device__ __forceinline__ void turn_back_store(float (&g)[8], const float2* cs, int lane, __nv_bfloat16* p) {
    __align__(16) __nv_bfloat16 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float other = __shfl_xor_sync(0xffffffffu, g[i], 16);
        const float2 a = cs[(8 * lane + i) & (D / 2 - 1)];
        // the inverse turn: (x1, x2) = (y1 c + y2 s, y2 c - y1 s)
        o[i] = __float2bfloat16_rn(g[i] * a.x + (lane < 16 ? other : -other) * a.y);
    }
    *reinterpret_cast<uint4*>(p + 8 * lane) = *reinterpret_cast<const uint4*>(o);
}
__device__ __forceinline__ void store8(const float (&v)[8], __nv_bfloat16* p) {
    __align__(16) __nv_bfloat16 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __float2bfloat16_rn(v[i]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(o);
}

// warp = one query row: one pass over its keys with the running maximum and sum
__global__ void __launch_bounds__(128) mqa_fwd_kernel(Args a) {
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (long long)a.B * a.T * a.H) return;
    const long long tok = row / a.H;
    const long long b = tok / a.T;
    const int t = (int)(tok % a.T);
    float q[8], o[8] = {};
    load8(a.q_rot + row * D + 8 * lane, q);
    float m = -INFINITY, l = 0.f;
    for (int i = a.lo[tok]; i <= t; ++i) {
        float k[8], v[8];
        load8(a.k_rot + (b * a.T + i) * D + 8 * lane, k);
        load8(a.v + (b * a.T + i) * D + 8 * lane, v);
        const float s = dot8(q, k) * a.scale_log2;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = fmaf(l, f, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(o[e], f, p * v[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] /= l;
    store8(o, a.out + row * D + 8 * lane);
    if (lane == 0) a.lse[row] = m + log2f(l);
}

// warp = one query row: delta, then dq
__global__ void __launch_bounds__(128) mqa_dq_kernel(Args a) {
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (long long)a.B * a.T * a.H) return;
    const long long tok = row / a.H;
    const long long b = tok / a.T;
    const int t = (int)(tok % a.T);
    float q[8], od[8], g[8] = {}, x[8];
    load8(a.q_rot + row * D + 8 * lane, q);
    load8(a.dout + row * D + 8 * lane, od);
    load8(a.out + row * D + 8 * lane, x);
    const float delta = dot8(od, x), lse = a.lse[row];
    if (lane == 0) a.delta[row] = delta;
    for (int i = a.lo[tok]; i <= t; ++i) {
        float k[8], v[8];
        load8(a.k_rot + (b * a.T + i) * D + 8 * lane, k);
        load8(a.v + (b * a.T + i) * D + 8 * lane, v);
        const float p = exp2f(dot8(q, k) * a.scale_log2 - lse);
        const float ds = p * (dot8(od, v) - delta);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = fmaf(ds, k[e], g[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] *= a.scale;
    turn_back_store(g, a.cs + (size_t)t * (D / 2), lane, a.dq + row * D);
}

// warp = one key: every query row that sees it (lo_t is non-decreasing in t)
__global__ void __launch_bounds__(128) mqa_dkv_kernel(Args a) {
    const long long key = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (key >= (long long)a.B * a.T) return;
    const long long b = key / a.T;
    const int i = (int)(key % a.T);
    float k[8], v[8], gk[8] = {}, gv[8] = {};
    load8(a.k_rot + key * D + 8 * lane, k);
    load8(a.v + key * D + 8 * lane, v);
    for (int t = i; t < a.T && a.lo[b * a.T + t] <= i; ++t)
        for (int h = 0; h < a.H; ++h) {
            const long long row = (b * a.T + t) * a.H + h;
            float q[8], od[8];
            load8(a.q_rot + row * D + 8 * lane, q);
            load8(a.dout + row * D + 8 * lane, od);
            const float p = exp2f(dot8(q, k) * a.scale_log2 - a.lse[row]);
            const float ds = p * (dot8(od, v) - a.delta[row]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                gk[e] = fmaf(ds, q[e], gk[e]);
                gv[e] = fmaf(p, od[e], gv[e]);
            }
        }
#pragma unroll
    for (int e = 0; e < 8; ++e) gk[e] *= a.scale;
    store8(gv, a.dv + key * D + 8 * lane);
    turn_back_store(gk, a.cs + (size_t)i * (D / 2), lane, a.dk + key * D);
}

// What the forward keeps: lse, first keys, angles, the rotated queries and keys.
struct SaveLayout {
    size_t lse, lo, cs, q_rot, k_rot, total;
};
inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
inline SaveLayout save_layout(const rglru_mqa_dims* d) {
    const size_t tok = (size_t)d->batch * d->seq_len;
    SaveLayout l{};
    size_t o = 0;
    l.lse = o; o = up256(o + tok * d->q_heads * 4);
    l.lo = o; o = up256(o + tok * 4);
    l.cs = o; o = up256(o + (size_t)d->seq_len * (D / 2) * sizeof(float2));
    l.q_rot = o; o = up256(o + tok * d->q_heads * D * 2);
    l.k_rot = o; o = up256(o + tok * D * 2);
    l.total = o;
    return l;
}
struct WsLayout {
    size_t delta, total;
};
inline WsLayout ws_layout(const rglru_mqa_dims* d) {
    WsLayout l{};
    size_t o = 256;                    // the status word
    l.delta = o; o = up256(o + (size_t)d->batch * d->seq_len * d->q_heads * 4);
    l.total = o;
    return l;
}

inline Args make_args(const rglru_mqa_dims* d, void* save) {
    const SaveLayout l = save_layout(d);
    uint8_t* p = static_cast<uint8_t*>(save);
    Args a{};
    a.B = d->batch; a.T = d->seq_len; a.H = d->q_heads;
    a.scale = d->scale; a.scale_log2 = d->scale * kLog2e;
    a.q_rot = reinterpret_cast<const __nv_bfloat16*>(p + l.q_rot);
    a.k_rot = reinterpret_cast<const __nv_bfloat16*>(p + l.k_rot);
    a.cs = reinterpret_cast<const float2*>(p + l.cs);
    a.lo = reinterpret_cast<const int*>(p + l.lo);
    a.lse = reinterpret_cast<float*>(p + l.lse);
    return a;
}

}  // namespace mt

size_t mqa_save_bytes(const rglru_mqa_dims* d) { return mt::save_layout(d).total; }
size_t mqa_train_workspace(const rglru_mqa_dims* d) { return mt::ws_layout(d).total; }

cudaError_t launch_mqa_forward(const rglru_mqa_dims* d, const void* q, const void* k, const void* v,
                               const uint8_t* reset, int pos0, void* out, void* save, void* ws, cudaStream_t s) {
    using namespace mt;
    (void)ws;
    const SaveLayout l = save_layout(d);
    uint8_t* p = static_cast<uint8_t*>(save);
    const int B = d->batch, T = d->seq_len, H = d->q_heads;
    mqa_angles_kernel<<<T, D / 2, 0, s>>>(pos0, d->rope_base, reinterpret_cast<float2*>(p + l.cs));
    mqa_first_key_kernel<<<B, 1024, 0, s>>>(T, d->window, reset, reinterpret_cast<int*>(p + l.lo));
    mqa_turn_kernel<<<dim3(T, B), D / 2, 0, s>>>(T, H, reinterpret_cast<const float2*>(p + l.cs),
                                                 static_cast<const __nv_bfloat16*>(q),
                                                 static_cast<const __nv_bfloat16*>(k),
                                                 reinterpret_cast<__nv_bfloat16*>(p + l.q_rot),
                                                 reinterpret_cast<__nv_bfloat16*>(p + l.k_rot));
    Args a = make_args(d, save);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.out = static_cast<__nv_bfloat16*>(out);
    const long long rows = (long long)B * T * H;
    mqa_fwd_kernel<<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_mqa_backward(const rglru_mqa_dims* d, const void* v, const void* out, const void* dout,
                                const void* save, void* dq, void* dk, void* dv, void* ws, cudaStream_t s) {
    using namespace mt;
    Args a = make_args(d, const_cast<void*>(save));
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out));
    a.dout = static_cast<const __nv_bfloat16*>(dout);
    a.delta = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ws_layout(d).delta);
    a.dq = static_cast<__nv_bfloat16*>(dq);
    a.dk = static_cast<__nv_bfloat16*>(dk);
    a.dv = static_cast<__nv_bfloat16*>(dv);
    const long long rows = (long long)a.B * a.T * a.H, keys = (long long)a.B * a.T;
    mqa_dq_kernel<<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(a);
    mqa_dkv_kernel<<<(unsigned)((keys + 3) / 4), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace rglru
