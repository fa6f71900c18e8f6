// mqa_cache8.cu -- the 8-bit ring cache of local MQA: written as it is quantised, read by the decode
// step, read back as the bf16 ring (head_dim 256).
//
// A slot holds the 256 elements of a rotated key (first half) or a value (second half) as e4m3 codes
// [B][2][w][d] with one fp32 scale each [B][2][w]:
//     scale = max(amax |x|, 448 * 2^-126) / 448,   code = e4m3(x / scale),   value = code * scale
// (448 is e4m3's largest value; the floor keeps the scale of a zero slot a normal number).  The key is
// rotated, and the quotient taken, in fp64 and rounded once to fp32 before the code: a code then does
// not depend on the rounding of a sine or a product next to a border between two codes.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace rglru {
namespace c8 {

constexpr int D = 256;

// e4m3 codes of two fp32 values, lo in the low byte (round to nearest even, saturating)
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float e4m3_value(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// 128 threads (thread j: elements j, j + d/2) quantise one row; x in fp64
__device__ __forceinline__ void quantise_row(double x1, double x2, uint8_t* codes, float* scale, double* red) {
    const int j = threadIdx.x;
    double m = fmax(fabs(x1), fabs(x2));
    // fmax drops a NaN: keep it, so that a slot with one is NaN as a whole
    if (x1 != x1 || x2 != x2) m = x1 + x2;
    for (int o = 16; o > 0; o >>= 1) {
        const double u = __shfl_xor_sync(0xffffffffu, m, o);
        m = (m != m || u != u) ? m + u : fmax(m, u);
    }
    if ((j & 31) == 0) red[j >> 5] = m;
    __syncthreads();
    m = red[0];
    for (int i = 1; i < 4; ++i) m = (m != m || red[i] != red[i]) ? m + red[i] : fmax(m, red[i]);
    if (!(m >= 448.0 * 1.1754943508222875e-38) && m == m) m = 448.0 * 1.1754943508222875e-38;
    const float s = (float)(m / 448.0);
    const uint16_t c = e4m3x2((float)(x1 / (double)s), (float)(x2 / (double)s));
    codes[j] = (uint8_t)(c & 0xff);
    codes[j + D / 2] = (uint8_t)(c >> 8);
    if (j == 0) *scale = s;
    __syncthreads();
}

__device__ __forceinline__ void turn64(double p, float base, int j, double x1, double x2, double& y1, double& y2) {
    double s, c;
    sincos(p * pow((double)base, -2.0 * j / D), &s, &c);
    y1 = x1 * c - x2 * s;
    y2 = x2 * c + x1 * s;
}

// block = (token, row): the last min(len, w) tokens of a row go into their slots
__global__ void __launch_bounds__(D / 2) mqa_cache8_write_kernel(int T, int w, int pos0, float base, const int* lengths,
                                                                 const __nv_bfloat16* k, const __nv_bfloat16* v,
                                                                 uint8_t* codes, float* scales) {
    __shared__ double red[4];
    const int b = blockIdx.y, j = threadIdx.x;
    const int len = lengths ? min(max(lengths[b], 0), T) : T;
    const int t = max(0, len - w) + (int)blockIdx.x;
    if (t >= len) return;
    const size_t e = ((size_t)b * T + t) * D;
    const long long p = (long long)pos0 + t;
    const size_t ks = (size_t)b * 2 * w + (size_t)(p % w), vs = ks + w;
    double y1, y2;
    turn64((double)p, base, j, (double)__bfloat162float(k[e + j]), (double)__bfloat162float(k[e + j + D / 2]), y1, y2);
    quantise_row(y1, y2, codes + ks * D, scales + ks, red);
    quantise_row((double)__bfloat162float(v[e + j]), (double)__bfloat162float(v[e + j + D / 2]), codes + vs * D,
                 scales + vs, red);
}

// block = row: rotated queries (fp32), the new slot
__global__ void __launch_bounds__(D / 2) mqa_decode8_turn_kernel(int H, int w, float base, const int* pos,
                                                                 const __nv_bfloat16* q, const __nv_bfloat16* k,
                                                                 const __nv_bfloat16* v, float* q_rot, uint8_t* codes,
                                                                 float* scales) {
    __shared__ double red[4];
    const int b = blockIdx.x, j = threadIdx.x, p = pos[b];
    if (p < 0) return;
    const size_t ks = (size_t)b * 2 * w + (size_t)(p % w), vs = ks + w;
    double y1, y2, s, c;
    sincos((double)p * pow((double)base, -2.0 * j / D), &s, &c);
    for (int h = 0; h < H; ++h) {
        const size_t e = ((size_t)b * H + h) * D;
        const float x1 = __bfloat162float(q[e + j]), x2 = __bfloat162float(q[e + j + D / 2]);
        q_rot[e + j] = x1 * (float)c - x2 * (float)s;
        q_rot[e + j + D / 2] = x2 * (float)c + x1 * (float)s;
    }
    const double x1 = (double)__bfloat162float(k[(size_t)b * D + j]), x2 = (double)__bfloat162float(k[(size_t)b * D + j + D / 2]);
    y1 = x1 * c - x2 * s;
    y2 = x2 * c + x1 * s;
    quantise_row(y1, y2, codes + ks * D, scales + ks, red);
    quantise_row((double)__bfloat162float(v[(size_t)b * D + j]), (double)__bfloat162float(v[(size_t)b * D + j + D / 2]),
                 codes + vs * D, scales + vs, red);
}

// block = (head, row), 8 warps over the slots, lane = 8 elements; one pass, running maximum and sum
__global__ void __launch_bounds__(256) mqa_decode8_kernel(int H, int w, float scale_log2, const int* pos,
                                                          const float* q_rot, const uint8_t* codes, const float* scales,
                                                          __nv_bfloat16* out) {
    __shared__ float sm[8], sl[8], so[8][D];
    const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int p = pos[b], n = p < 0 ? 0 : min(p, w - 1) + 1;
    const size_t e = ((size_t)b * H + h) * D;
    float q[8], o[8] = {};
    for (int i = 0; i < 8; ++i) q[i] = q_rot[e + 8 * lane + i];
    float m = -INFINITY, l = 0.f;
    for (int i = warp; i < n; i += 8) {
        const size_t ks = (size_t)b * 2 * w + i, vs = ks + w;
        const uint2 kc = *reinterpret_cast<const uint2*>(codes + ks * D + 8 * lane);
        const uint2 vc = *reinterpret_cast<const uint2*>(codes + vs * D + 8 * lane);
        float s = 0.f;
        for (int x = 0; x < 8; ++x) s = fmaf(q[x], e4m3_value((uint8_t)((x < 4 ? kc.x : kc.y) >> (8 * (x & 3)))), s);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= scales[ks] * scale_log2;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), pr = exp2f(s - mn);
        m = mn;
        l = fmaf(l, f, pr);
        const float pv = pr * scales[vs];
        for (int x = 0; x < 8; ++x) o[x] = fmaf(o[x], f, pv * e4m3_value((uint8_t)((x < 4 ? vc.x : vc.y) >> (8 * (x & 3)))));
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    for (int x = 0; x < 8; ++x) so[warp][8 * lane + x] = o[x];
    __syncthreads();
    float mx = -INFINITY, ls = 0.f, v = 0.f;
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, sm[i]);
    for (int i = 0; i < 8; ++i) {
        const float f = sl[i] == 0.f ? 0.f : exp2f(sm[i] - mx);
        ls = fmaf(sl[i], f, ls);
        v = fmaf(so[i][threadIdx.x], f, v);
    }
    out[e + threadIdx.x] = __float2bfloat16_rn(n > 0 ? v / ls : 0.f);
}

// thread = 8 elements of one slot
__global__ void __launch_bounds__(256) mqa_cache8_read_kernel(long long slots, int w, const int* pos,
                                                              const uint8_t* codes, const float* scales,
                                                              __nv_bfloat16* cache) {
    const long long s = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (s >= slots) return;
    if (pos && s % w > pos[s / (2 * (long long)w)]) return;
    const uint2 c = *reinterpret_cast<const uint2*>(codes + s * D + 8 * lane);
    const float f = scales[s];
    __align__(16) __nv_bfloat16 o[8];
    for (int x = 0; x < 8; ++x) o[x] = __float2bfloat16_rn(f * e4m3_value((uint8_t)((x < 4 ? c.x : c.y) >> (8 * (x & 3)))));
    *reinterpret_cast<uint4*>(cache + s * D + 8 * lane) = *reinterpret_cast<const uint4*>(o);
}

}  // namespace c8

size_t mqa_decode8_workspace(const rglru_mqa_dims* d) {
    return 256 + (size_t)d->batch * d->q_heads * c8::D * 4;
}

cudaError_t launch_mqa_cache8_write(const rglru_mqa_dims* d, const void* k, const void* v, const int* lengths, int pos0,
                                    void* codes, float* scales, cudaStream_t s) {
    using namespace c8;
    mqa_cache8_write_kernel<<<dim3(std::min(d->seq_len, d->window), d->batch), D / 2, 0, s>>>(
        d->seq_len, d->window, pos0, d->rope_base, lengths, static_cast<const __nv_bfloat16*>(k),
        static_cast<const __nv_bfloat16*>(v), static_cast<uint8_t*>(codes), scales);
    return cudaGetLastError();
}

cudaError_t launch_mqa_decode8(const rglru_mqa_dims* d, const void* q, const void* k, const void* v, const int* pos,
                               void* codes, float* scales, void* out, void* ws, cudaStream_t s) {
    using namespace c8;
    float* q_rot = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    mqa_decode8_turn_kernel<<<d->batch, D / 2, 0, s>>>(
        d->q_heads, d->window, d->rope_base, pos, static_cast<const __nv_bfloat16*>(q),
        static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), q_rot,
        static_cast<uint8_t*>(codes), scales);
    mqa_decode8_kernel<<<dim3(d->q_heads, d->batch), 256, 0, s>>>(d->q_heads, d->window, d->scale * 1.4426950408889634f,
                                                                  pos, q_rot, static_cast<const uint8_t*>(codes), scales,
                                                                  static_cast<__nv_bfloat16*>(out));
    return cudaGetLastError();
}

cudaError_t launch_mqa_cache8_read(const rglru_mqa_dims* d, const void* codes, const float* scales, const int* pos,
                                   void* cache, cudaStream_t s) {
    using namespace c8;
    const long long slots = 2LL * d->batch * d->window;
    mqa_cache8_read_kernel<<<(unsigned)((slots + 7) / 8), 256, 0, s>>>(slots, d->window, pos,
                                                                       static_cast<const uint8_t*>(codes), scales,
                                                                       static_cast<__nv_bfloat16*>(cache));
    return cudaGetLastError();
}

}  // namespace rglru
