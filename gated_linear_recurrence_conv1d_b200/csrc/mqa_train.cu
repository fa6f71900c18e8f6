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
//
// Rounded to bf16 are the operands of the tensor cores (of the types of this rate fp16 has three bits more, but not
// the range of the bf16 tensors that come in, and both operands of a product have one type), and what is written:
// q~ and k~ once, into the save (in fp32 they would double its largest part and the loads of every tile, and be
// rounded in front of the product all the same), P for P v, P^T dO and dS^T, dS for dS k~ and dS^T q~, and out, dq, dk,
// dv.  Scores, their maxima and sums, dP, delta and all products' sums are fp32.  Together an RMS error of 0.38 %, where
// rounding the results alone leaves 0.17 %; the two parts of each operand that fp32 accuracy takes would cost 3 times
// the products.
#include <algorithm>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "angles.cuh"
#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "tma_maps.h"

namespace rglru {
namespace mt {

using namespace pr;

constexpr int D = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxClusters = 74;       // 2-CTA clusters of 148 SMs

// ---------------------------------------------------------------- rotary embedding, documents ----
constexpr int kAngleStep = 8, kAngleTokens = 64;         // tokens a block of 1024 threads has at a time, and in all
constexpr int kScanThreads = 1024, kScanPer = 8, kScanChunk = kScanThreads * kScanPer;

// The maximum (or minimum) of v over the threads of the block before this one, start for the first, and over all.
template <bool kMax>
__device__ __forceinline__ int better(int a, int b) {
    return kMax ? max(a, b) : min(a, b);
}
template <bool kMax>
__device__ __forceinline__ int scan_before(int v, int start, int* warp_v, int& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = better<kMax>(v, u);
    }
    if (lane == 31) warp_v[warp] = v;
    __syncthreads();
    int w = warp_v[lane];                                // kScanThreads / 32 = 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w = better<kMax>(w, u);
    }
    all = __shfl_sync(0xffffffffu, w, 31);
    const int warps_before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    int before = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) before = start;
    if (warp > 0) before = better<kMax>(before, warps_before);
    __syncthreads();
    return before;
}

// Blocks [0, B): a row's first key of every token, lo = max(0, t - w + 1, start of its document), and the last token
// that sees it, last = min(T - 1, t + w - 1, end of its document): a running maximum forwards and a running
// minimum backwards over the tokens that start a document.  The other blocks: cosine and sine of position
// pos0 + t, pair j, [T][d/2], angle and reduction in fp64.  Bound by latency: 4 us, 9 us at 8 rows of 2048 tokens.
__global__ void __launch_bounds__(kScanThreads) mqa_prepare_kernel(int B, int T, int w, const uint8_t* reset, int* lo, int* last,
                                                                   int pos0, RopeBase base, float2* cs) {
    pdl_launch();
    pdl_wait();
    if (blockIdx.x >= (unsigned)B) {
        int t = (blockIdx.x - B) * kAngleTokens + threadIdx.x / (D / 2);
        const int j = threadIdx.x % (D / 2);
        if (t >= T) return;
        // every kAngleStep-th token by an angle addition (a dozen units of fp64's last place at most)
        double c, s, dc, ds;
        rope_cos_sin(base, j, (double)pos0 + t, c, s);
        rope_cos_sin(base, j, (double)kAngleStep, dc, ds);
#pragma unroll 1
        for (int i = 0; i < kAngleTokens / kAngleStep && t < T; ++i, t += kAngleStep) {
            cs[(size_t)t * (D / 2) + j] = make_float2((float)c, (float)s);
            const double x = c * dc - s * ds;
            s = s * dc + c * ds;
            c = x;
        }
        return;
    }
    __shared__ int warp_v[32];
    const int b = blockIdx.x;
    const uint8_t* rs = reset ? reset + (size_t)b * T : nullptr;
    lo += (size_t)b * T;
    last += (size_t)b * T;
    const int chunks = (T + kScanChunk - 1) / kScanChunk;
    int carry = 0, all;
    for (int c = 0; c < chunks; ++c) {
        const int t0 = c * kScanChunk + threadIdx.x * kScanPer;
        int v[kScanPer], run = 0;
#pragma unroll
        for (int e = 0; e < kScanPer; ++e) v[e] = rs ? rs[min(t0 + e, T - 1)] : 0;      // loads together
#pragma unroll
        for (int e = 0; e < kScanPer; ++e) {
            v[e] = t0 + e < T && v[e] ? t0 + e : 0;
            run = max(run, v[e]);
        }
        run = max(carry, scan_before<true>(run, 0, warp_v, all));
#pragma unroll
        for (int e = 0; e < kScanPer; ++e) {
            run = max(run, v[e]);
            if (t0 + e < T) lo[t0 + e] = max(run, t0 + e - w + 1);
        }
        carry = max(carry, all);
    }
    carry = T;                          // the first document start after the tokens seen so far, going back
    for (int c = chunks - 1; c >= 0; --c) {
        // thread 0 has the chunk's last tokens
        const int t1 = c * kScanChunk + (kScanThreads - (int)threadIdx.x) * kScanPer - 1;
        int v[kScanPer], run = T;
#pragma unroll
        for (int e = 0; e < kScanPer; ++e) v[e] = rs ? rs[min(t1 - e, T - 1)] : 0;
#pragma unroll
        for (int e = 0; e < kScanPer; ++e) {
            v[e] = t1 - e < T && v[e] ? t1 - e : T;
            run = min(run, v[e]);
        }
        run = min(carry, scan_before<false>(run, T, warp_v, all));
#pragma unroll
        for (int e = 0; e < kScanPer; ++e) {
            const int t = t1 - e;
            if (t < T) last[t] = w - 1 < run - 1 - t ? t + w - 1 : run - 1;
            run = min(run, v[e]);
        }
        carry = min(carry, all);
    }
}

// Blocks but the last: 16 threads a token, 8 pairs each, over its H query heads and its key: bound by HBM (q and k in
// and out: 185 MB for 16384 tokens of 10 heads, 43 us), so the rows of a few heads are in flight together.  The
// last block: the line of (key tile, row
// tile) products that the backward cuts into pieces: cum[j] = the row tiles of the key tiles before j, a
// key tile's rows being those from its first key's token to the last token that sees its last key.
constexpr int kTurnRows = 4, kTurnThreads = 256, kKeyTile = 128, kRowTile = 64;
__global__ void __launch_bounds__(kTurnThreads) mqa_turn_kernel(long long tokens, int T, int H, const float2* cs,
                                                                const __nv_bfloat16* q, const __nv_bfloat16* k,
                                                                __nv_bfloat16* q_rot, __nv_bfloat16* k_rot, const int* last_t,
                                                                long long* cum) {
    pdl_launch();
    pdl_wait();
    if (blockIdx.x == gridDim.x - 1) {
        __shared__ long long warp_v[kTurnThreads / 32];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nkt = (T + kKeyTile - 1) / kKeyTile;
        const long long nk = tokens / T * nkt;
        long long carry = 0;
        if (threadIdx.x == 0) cum[0] = 0;
        for (long long j0 = 0; j0 < nk; j0 += kTurnThreads) {
            const long long j = j0 + threadIdx.x;
            long long v = 0;
            if (j < nk) {
                const int key0 = (int)(j % nkt) * kKeyTile, key1 = min(key0 + kKeyTile, T) - 1;
                v = ((long long)(last_t[j / nkt * T + key1] + 1 - key0) * H + kRowTile - 1) / kRowTile;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (lane == 31) warp_v[warp] = v;
            __syncthreads();
            long long before = carry;
#pragma unroll
            for (int i = 0; i < kTurnThreads / 32; ++i) {
                if (i < warp) before += warp_v[i];
                carry += warp_v[i];
            }
            if (j < nk) cum[j + 1] = before + v;
            __syncthreads();
        }
        return;
    }
    const long long tok = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int c = threadIdx.x & 15;
    if (tok >= tokens) return;
    float4 a[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = reinterpret_cast<const float4*>(cs + (size_t)(tok % T) * (D / 2) + 8 * c)[e];
    for (int h0 = 0; h0 <= H; h0 += kTurnRows) {
        uint4 x[kTurnRows], y[kTurnRows];
#pragma unroll
        for (int i = 0; i < kTurnRows; ++i) {
            const int h = h0 + i;
            if (h > H) break;
            const uint4* src = reinterpret_cast<const uint4*>(h < H ? q + (tok * H + h) * D : k + tok * D);
            x[i] = src[c];
            y[i] = src[16 + c];
        }
#pragma unroll
        for (int i = 0; i < kTurnRows; ++i) {
            const int h = h0 + i;
            if (h > H) break;
            const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
            uint32_t o1[4], o2[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = __uint_as_float(xs[e] << 16), x1 = __uint_as_float(xs[e] & 0xffff0000u);
                const float y0 = __uint_as_float(ys[e] << 16), y1 = __uint_as_float(ys[e] & 0xffff0000u);
                o1[e] = bf16x2(x0 * a[e].x - y0 * a[e].y, x1 * a[e].z - y1 * a[e].w);
                o2[e] = bf16x2(y0 * a[e].x + x0 * a[e].y, y1 * a[e].z + x1 * a[e].w);
            }
            uint4* dst = reinterpret_cast<uint4*>(h < H ? q_rot + (tok * H + h) * D : k_rot + tok * D);
            dst[c] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
            dst[16 + c] = make_uint4(o2[0], o2[1], o2[2], o2[3]);
        }
    }
}

// ---------------------------------------------------------------- tensor-core kernels: shared ---------
struct Args {
    int B, T, H, TH, THp;       // TH = T H query rows of a batch row; THp: their pitch in lse, delta
    int ntr;                    // 256-row pair tiles of a batch row
    float scale, scale_log2;
    const int* lo;              // [B, T]
    const float2* cs;           // [T, d/2]
    float* neg_lse;             // [B, THp], -L, log2 domain
    int8_t* low;                // [B, T, H, d]: the bits of out below its bf16, 8 of them
    float* neg_delta;           // [B, THp]
    const long long* cum;       // [B nkt + 1]: 64-row tiles before each key tile
    float* part;                // partial dk, dv of (cluster, key tile)
    int nkt;                    // 128-key tiles of a batch row
    __nv_bfloat16 *out, *dq, *dk, *dv;
    unsigned* delta_there;      // 1 from dq's first CTA on: what dk / dv read is complete (0 from the delta kernel on)
    DeviceStatus* status;
    unsigned long long timeout_ns;
};

// Pair tiles in the order of falling position (the longest rows of a causal window first), dealt to
// the CTA pairs forwards and backwards in turn, so that every pair gets long and short ones alike.
// lo_t is non-decreasing in t, so a tile's keys are [lo of its first token, its last token].
struct QTile {
    int b, r0, lo, t1;          // batch row, first query row of the pair, first key, last token
    // The last key tile may hold no key that a row sees in its second half: then S has 64 columns, 32 keys of each CTA, and
    // the product with V or K half the keys (3 % of the step's products at 1000 keys a row).
    template <int BK>
    __device__ __forceinline__ bool half(int j) const {
        return t1 + 1 - (lo + j * BK) <= BK / 2;
    }
};
// walks a pair's tiles; the load of the next tile's first key is in flight while a tile is worked on
template <int BK>
struct QTiles {
    QTile t, nx;
    int k, n;                   // number of the tile, its key tiles; k = -1 before the first advance()
    bool has;
    int pair, npairs;
    __device__ __forceinline__ void fetch(const Args& a, int i) {
        const int p = i * npairs + ((i & 1) ? npairs - 1 - pair : pair);
        has = p < a.B * a.ntr;
        if (!has) return;
        nx.b = p % a.B;
        nx.r0 = (a.ntr - 1 - p / a.B) * 256;
        nx.t1 = min(nx.r0 + 255, a.TH - 1) / a.H;
        nx.lo = a.lo[(size_t)nx.b * a.T + nx.r0 / a.H];
    }
    __device__ __forceinline__ QTiles(const Args& a, int pair_, int npairs_) : t{}, nx{}, k(-1), n(0), pair(pair_), npairs(npairs_) {
        fetch(a, 0);
    }
    __device__ __forceinline__ bool advance(const Args& a) {
        ++k;
        if (!has) return false;
        t = nx;
        n = (t.t1 + 1 - t.lo + BK - 1) / BK;
        fetch(a, k + 1);
        return true;
    }
};

// ---------------------------------------------------------------- forward -----------------------------
// A CTA pair (cta_group::2) takes 256 query rows, 128 a CTA, and walks the keys that any of them sees in tiles of 128:
//   S = Q K^T   (M 256, N 128, K 256; Q and K from shared memory)      two TMEM buffers of 128 columns
//   O += P V    (M 256, N 256, K 128; P in TMEM over its S, V from shared memory)    256 columns
// Each CTA loads half of every K tile (64 keys) and of every V tile (128 of its columns), so a key tile costs
// an SM 64 KB for 2048 tensor cycles: half of what a CTA alone would pull from L2.  8 softmax warps, thread =
// (row, 64 of the 128 keys): P = 2^(c s - m) with a reference maximum m that moves only when a score
// passes it by 2^8 (then O and the sums are rescaled; the two threads of a row meet for that only).  P is rounded to
// bf16 for the MMA, and O is divided by the sum of the rounded weights; L takes the sum of the fp32 ones.  The S
// of the next tile runs under the softmax of this one.
// Beside out the forward keeps the next 8 bits of each of its elements for delta = dO . out.  Where one key holds nearly
// all of a row's weight, dP of that key and delta cancel: dS is what the small weights leave of the difference,
// and a delta from out in bf16, or from weights that do not sum to one, can be off by more than dS itself (rows of two
// keys: dq of a row off by up to 6 %, over many rows 0.45 % RMS instead of 0.34 %).  The bytes cost 8 us of the 145.
// Bound by the tensor pipe and its hand-overs: 8 rows of 2048 tokens, 10 heads, window 2048 (172 GFLOP) in 145 us,
// 1.18 PFLOP/s.  The exponentials take about half of a key tile's 2048 tensor cycles, in pairs of fp32 operations
// with everything around them.
namespace fw {
// Two fp32 values rounded to bf16 (to nearest, ties away from zero, so that bit 15 of the value alone says whether
// it was rounded up), and bits 8 to 15 of four: as a signed byte, what to add to the rounded value's bits.  A NaN has to
// be quiet_nan(), which stays itself with a byte of zero: the one that arithmetic makes, 0x7fffffff, would be carried
// into the sign and leave as -0.
__device__ __forceinline__ uint32_t bf16x2_away(float a, float b) {
    return __byte_perm(__float_as_uint(a) + 0x8000u, __float_as_uint(b) + 0x8000u, 0x7632);
}
__device__ __forceinline__ uint32_t low_bytes(const float* x) {
    return __byte_perm(__byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x0051),
                       __byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x0051), 0x5410);
}
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7fc00000u); }
constexpr int BK = 128;
constexpr uint32_t SLOT = 32768;
constexpr int NSLOT = 5;
constexpr uint32_t OFF_Q = 0, OFF_SLOT = 65536, OFF_X = OFF_SLOT + NSLOT * SLOT, OFF_BAR = OFF_X + 1536;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 256 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TM_O = 0, TM_S = 256;
constexpr int kThreads = 352, kSoft = 256, kWarpTma = 8, kWarpMma = 9, kWarpQ = 10;
}  // namespace fw

__global__ void __launch_bounds__(fw::kThreads, 1)
mqa_forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const Args a) {
    using namespace fw;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const uint32_t bars = sb + OFF_BAR;
    const uint32_t q_full = bars, q_empty = bars + 8, o_free = bars + 16, mma_done = bars + 24;
    auto s_full = [&](uint32_t i) { return bars + 32 + 8 * i; };
    auto p_full = [&](uint32_t i) { return bars + 48 + 8 * i; };
    auto o_done = [&](uint32_t i) { return bars + 64 + 8 * i; };
    auto full = [&](uint32_t s) { return bars + 80 + 8 * s; };
    auto empty = [&](uint32_t s) { return bars + 80 + 8 * NSLOT + 8 * s; };
    volatile uint32_t* tmem_s = reinterpret_cast<volatile uint32_t*>(smem + OFF_BAR + 80 + 16 * NSLOT);
    float* xch = reinterpret_cast<float*>(smem + OFF_X);
    const Guard g{reinterpret_cast<volatile int*>(smem + OFF_BAR + 96 + 16 * NSLOT), a.status, a.timeout_ns};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(o_free, 16);
        mbar_init(mma_done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 16);
            mbar_init(o_done(i), 1);
        }
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        *g.abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc_pair(smem_u32((const void*)tmem_s), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    pdl_launch();
    pdl_wait();

    if (warp == kWarpTma) {
        if (lane == 0) {
            const uint32_t lead = map_to_rank(bars, 0) - bars;      // this CTA's barrier address -> the leader's
            uint32_t L = 0;
            bool ok = true;
            // key tile j of the values (v) or keys into the next slot
            auto load = [&](bool v, const QTile& q, int j) {
                const uint32_t s = L % NSLOT, u = L / NSLOT;
                if (u > 0 && !wait(empty(s), (u - 1) & 1, g, 1)) return false;
                if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * SLOT);
                const uint32_t dst = sb + OFF_SLOT + s * SLOT, bar = full(s) + lead;
                const int key0 = q.lo + j * BK;
                if (v) {
                    for (int c = 0; c < 2; ++c)
                        tma_load_3d_pair(dst + c * 16384, &map_v, (int)rank * 128 + c * 64, key0, q.b, bar);
                } else {
                    for (int c = 0; c < 4; ++c)
                        tma_load_3d_pair(dst + c * 8192, &map_k, c * 64, key0 + (int)rank * (q.half<BK>(j) ? 32 : 64), q.b, bar);
                }
                ++L;
                return true;
            };
            // in the order of the MMAs: K two key tiles ahead of V, across query tiles
            QTiles<BK> qk(a, pair, npairs), qv = qk;
            int jk = 0, jv = 0, ahead = 0;
            bool ks = qk.advance(a), vs = qv.advance(a);
            while (ok && vs) {
                if (ks && ahead < 2) {
                    if (!(ok = load(false, qk.t, jk))) break;
                    ++ahead;
                    if (++jk == qk.n) {
                        jk = 0;
                        ks = qk.advance(a);
                    }
                    continue;
                }
                if (!(ok = load(true, qv.t, jv))) break;
                --ahead;
                if (++jv == qv.n) {
                    jv = 0;
                    vs = qv.advance(a);
                }
            }
            // no bulk copy may still be writing shared memory at the exit: the leader sees both CTAs' land
            if (rank == 0) {
                const uint64_t t0 = globaltimer_ns();
                for (uint32_t l = L > NSLOT ? L - NSLOT : 0; l < L; ++l)
                    while (!mbar_try_wait_cluster(full(l % NSLOT), (l / NSLOT) & 1) && globaltimer_ns() - t0 < a.timeout_ns) {
                    }
            }
        }
    } else if (warp == kWarpQ) {
        // the query tiles: each as soon as the S before it are through with the buffer
        if (lane == 0) {
            const uint32_t lead = map_to_rank(bars, 0) - bars;
            QTiles<BK> q(a, pair, npairs);
            while (q.advance(a)) {
                if (q.k > 0 && !wait(q_empty, (q.k - 1) & 1, g, 2)) break;
                if (rank == 0) mbar_arrive_expect_tx(q_full, 2 * 65536);
                for (int c = 0; c < 4; ++c)
                    tma_load_3d_pair(sb + OFF_Q + c * 16384, &map_q, c * 64, q.t.r0 + (int)rank * 128, q.t.b, q_full + lead);
            }
            const uint64_t t0 = globaltimer_ns();
            if (rank == 0 && q.k > 0)
                while (!mbar_try_wait_cluster(q_full, (q.k - 1) & 1) && globaltimer_ns() - t0 < a.timeout_ns) {
                }
        }
    } else if (warp == kWarpMma) {
        if (rank == 0) {
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t id_full = idesc_bf16(256, BK, 0), id_half = idesc_bf16(256, BK / 2, 0), id_o = idesc_bf16(256, D, 1);
            // S runs two key tiles ahead of P V, across query tiles
            QTiles<BK> qs(a, pair, npairs), qp = qs;
            int js = 0;
            uint32_t L = 0, gt = 0, gs = 0;                          // slots used; key tiles done, key tiles with S issued
            bool more = qs.advance(a), ok = true;
            auto wait_slot = [&](uint32_t l) { return wait_w(full(l % NSLOT), (l / NSLOT) & 1, g, 4); };
            auto issue_s = [&]() {                                   // S of the next key tile, from the next slot (which is there)
                if (js == 0 && !wait_w(q_full, qs.k & 1, g, 3)) return false;
                tc_fence_after();
                const uint32_t s = L % NSLOT, buf = gs & 1, id_s = qs.t.half<BK>(js) ? id_half : id_full;
                ++L;
                ++gs;
                const bool last = ++js == qs.n;
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_ss_pair(tm + TM_S + buf * BK, desc_k_sw128(sb + OFF_Q + (ks >> 2) * 16384 + (ks & 3) * 32),
                                    desc_k_sw128(sb + OFF_SLOT + s * SLOT + (ks >> 2) * 8192 + (ks & 3) * 32), id_s,
                                    ks > 0 ? 1u : 0u);
                    mma_commit_pair(s_full(buf));
                    mma_commit_pair(empty(s));
                    if (last) mma_commit_pair(q_empty);
                }
                __syncwarp();
                if (last) {
                    js = 0;
                    more = qs.advance(a);
                }
                return true;
            };
            for (int i = 0; ok && more && i < 2; ++i) ok = wait_slot(L) && issue_s();
            while (ok && qp.advance(a))
                for (int j = 0; j < qp.n; ++j, ++gt) {
                    const uint32_t buf = gt & 1, s = L % NSLOT, lk = more ? L + 1 : L;   // the next K behind this V
                    if (j == 0 && qp.k > 0 && !(ok = wait_w(o_free, (qp.k - 1) & 1, g, 5))) break;
                    if (!(ok = wait_w(p_full(buf), (gt >> 1) & 1, full(s), (L / NSLOT) & 1, full(lk % NSLOT), (lk / NSLOT) & 1, g, 6))) break;
                    ++L;
                    tc_fence_after();
                    const int steps = qp.t.half<BK>(j) ? BK / 32 : BK / 16;
                    if (elect_one()) {                               // O += P_j V_j
                        // P of keys [16 ks, 16 ks + 16): the two halves of a row sit 64 columns apart
#pragma unroll
                        for (int ks = 0; ks < BK / 16; ++ks)
                            if (ks < steps)
                                mma_ts_pair(tm + TM_O, tm + TM_S + buf * BK + (ks >> 2) * 64 + (ks & 3) * 8,
                                            desc_mn_sw128(sb + OFF_SLOT + s * SLOT + ks * 2048, 16384), id_o,
                                            (j > 0 || ks > 0) ? 1u : 0u);
                        mma_commit_pair(o_done(buf));
                        mma_commit_pair(empty(s));
                    }
                    __syncwarp();
                    if (more && !(ok = issue_s())) break;
                }
            if (elect_one()) mma_commit_pair(mma_done);              // every MMA is over before TMEM is released
            __syncwarp();
        }
        if (lane == 0) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait_cluster(mma_done, 0) && globaltimer_ns() - t0 < 4 * a.timeout_ns) {
            }
        }
        __syncwarp();
    } else {
        // softmax: row r of this CTA's 128, keys [64 half, 64 half + 64) of each tile
        const int r = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t lead_p = map_to_rank(p_full(0), 0), lead_free = map_to_rank(o_free, 0);
        uint32_t gt = 0;
        bool ok = true, stop = false;
        // out = O / l of the query tile before, its last key tile number `last`, done between the first P of the
        // next query tile and the next: the tensor pipe has that P and two S ahead of it meanwhile
        bool pending = false;
        int p_b = 0, p_row = 0;
        float p_m = 0.f, p_l = 0.f, p_w = 0.f;
        auto finish = [&](uint32_t last) {
            ok = ok && wait_w(o_done(last & 1), (last >> 1) & 1, g, 10);
            bar_or(false, kSoft);                         // xch has been read
            xch[half * 128 + r] = p_w;
            if (half == 1) xch[256 + r] = p_l;
            if (bar_or(!ok, kSoft)) return false;
            const float w = xch[r] + xch[128 + r], l = p_l + xch[256 + r];       // the row's sums (l: of half 0)
            bar_or(false, kSoft);                         // xch is read before its next use
            tc_fence_after();
            const float inv = 1.0f / w;
            const int row0 = p_row & ~3;                  // the quad's rows, of which this lane writes 16 bytes each
            const size_t at = ((size_t)p_b * a.TH + row0) * D + half * 128;
            __nv_bfloat16* dst = a.out + at + 8 * (lane & 3);
            int8_t* low = a.low + at + 16 * (lane & 3);
#pragma unroll 1
            for (int c = 0; c < 128; c += 64) {
                uint32_t lb[16];
#pragma unroll
                for (int h = 0; h < 64; h += 32) {
                    float o[32];
                    uint32_t e[16];
                    tmem_ld32(tl + TM_O + half * 128 + c + h, o);
                    tmem_wait_ld();
                    float2 odd = make_float2(0.f, 0.f);              // stays 0 unless a value is not finite
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 x = mul2(make_float2(o[i], o[i + 1]), make_float2(inv, inv));
                        odd = fma2(x, make_float2(0.f, 0.f), odd);
                        o[i] = x.x;
                        o[i + 1] = x.y;
                    }
                    if (!(odd.x + odd.y == 0.f)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = o[i] == o[i] ? o[i] : quiet_nan();
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) e[i] = bf16x2_away(o[2 * i], o[2 * i + 1]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) lb[h / 4 + i] = low_bytes(o + 4 * i);
                    quad_transpose(e);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (row0 + i < a.TH)
                            *reinterpret_cast<uint4*>(dst + (size_t)i * D + c + h) = make_uint4(e[4 * i], e[4 * i + 1], e[4 * i + 2], e[4 * i + 3]);
                }
                quad_transpose(lb);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (row0 + i < a.TH)
                        *reinterpret_cast<uint4*>(low + (size_t)i * D + c) = make_uint4(lb[4 * i], lb[4 * i + 1], lb[4 * i + 2], lb[4 * i + 3]);
            }
            if (half == 0 && p_row < a.TH) a.neg_lse[(size_t)p_b * a.THp + p_row] = -(p_m + log2f(l));
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(lead_free);
            return true;
        };
        QTiles<BK> q(a, pair, npairs);
        while (!stop && q.advance(a)) {
            const QTile t = q.t;
            const int row0 = t.r0 + (int)rank * 128, row = row0 + r;
            const int tok = min(row, a.TH - 1) / a.H;
            const int lo_row = a.lo[(size_t)t.b * a.T + tok];
            // a tile inside every row's keys needs no mask: [lo of the CTA's last token, its first token]
            const int full_lo = a.lo[(size_t)t.b * a.T + min(row0 + 127, a.TH - 1) / a.H], full_hi = min(row0, a.TH - 1) / a.H;
            float m = -INFINITY, l = 0.f, wsum = 0.f;    // sums of the weights, and of the weights as rounded for P V
            for (int j = 0; j < q.n; ++j) {
                const uint32_t i = gt + j, buf = i & 1;
                ok = ok && wait_w(s_full(buf), (i >> 1) & 1, g, 8);
                tc_fence_after();
                float s[64];
                tmem_ld32(tl + TM_S + buf * BK + half * 64, s);
                tmem_ld32(tl + TM_S + buf * BK + half * 64 + 32, s + 32);
                tmem_wait_ld();
                const int key0 = t.lo + j * BK + half * 64;
                float mx = -INFINITY;
                if (t.lo + j * BK >= full_lo && t.lo + j * BK + BK - 1 <= full_hi) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) mx = fmaxf(mx, s[c]);
                } else {
                    const int c_lo = lo_row - key0, c_hi = tok - key0;
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        s[c] = (c >= c_lo && c <= c_hi) ? s[c] : -INFINITY;
                        mx = fmaxf(mx, s[c]);
                    }
                }
                mx *= a.scale_log2;
                if (bar_or(mx > m + 8.0f || !ok, kSoft)) {           // some row of the CTA moves (or a wait failed)
                    xch[half * 128 + r] = mx;
                    if (bar_or(!ok, kSoft)) {
                        stop = true;
                        break;
                    }
                    mx = fmaxf(xch[r], xch[128 + r]);
                    const bool move = mx > m + 8.0f;
                    const float f = move && m != -INFINITY ? ex2_approx(m - mx) : 1.0f;
                    if (move) m = mx;
                    l *= f;
                    wsum *= f;
                    if (j > 0) {
                        ok = wait_w(o_done((i - 1) & 1), ((i - 1) >> 1) & 1, g, 9);
                        tc_fence_after();
                        if (__any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
                            for (int c = half * 128; c < half * 128 + 128; c += 16) {
                                float o[16];
                                tmem_ld16(tl + TM_O + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] *= f;
                                tmem_st16f(tl + TM_O + c, o);
                            }
                        }
                    }
                }
                const float nm = m == -INFINITY ? 0.f : -m;
                uint32_t p[32];
                const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), nm2 = make_float2(nm, nm);
                float2 l2 = make_float2(0.f, 0.f), w2 = l2;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float2 x = fma2(make_float2(s[2 * c], s[2 * c + 1]), sc2, nm2);
                    const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    l2 = add2(l2, e);
                    p[c] = bf16x2(e.x, e.y);
                    w2 = add2(w2, make_float2(__uint_as_float(p[c] << 16), __uint_as_float(p[c] & 0xffff0000u)));
                }
                l += l2.x + l2.y;
                wsum += w2.x + w2.y;
                tmem_st32(tl + TM_S + buf * BK + half * 64, p);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead_p + 8 * buf);
                if (j == 0 && pending && !finish(gt - 1)) {
                    stop = true;
                    break;
                }
            }
            if (stop) break;
            pending = true;
            p_b = t.b;
            p_row = row;
            p_m = m;
            p_l = l;
            p_w = wsum;
            gt += q.n;
        }
        if (!stop && pending) finish(gt - 1);
        tmem_wait_ld();
        tmem_wait_st();
    }
    // no CTA of the pair leaves while the other may still reach its shared memory or TMEM
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------- backward: dq ------------------------
// A CTA pair takes 256 query rows again and walks their keys in tiles of 128:
//   S = Q K^T,  dP = dO V^T   (M 256, N 128, K 256; all from shared memory)
//   dQ += dS K                (M 256, N 256, K 128; dS in TMEM over its dP)
// TMEM: dQ 256 columns, S 128, dP 128.  A CTA loads 64 keys of every K and V tile and 128 columns of every K tile,
// each into a buffer of its own: S of tile j + 1, dQ of tile j, dP of tile j + 1 follow each other in the tensor
// pipe, so each has the other two's time to arrive, and dS of tile j is formed under S of tile j + 1.
// 8 warps, thread = (row, 64 of the 128 keys): P = 2^(c s - L), dS = P (dP - delta), the row's L and delta in
// registers.  dq of a query tile is written after the first dS of the next.
// (Key tiles of 64 with two buffers of S and dP: 242 us instead of 202.  An MMA of N 64 reads 5 KB of shared memory a
// CTA in the time of 32 cycles, one of N 128 6 KB in 64, and shared memory gives 128 bytes a cycle.)
// Bound by the tensor pipe: 8 x 2048 tokens, 10 heads, window 2048 (258 GFLOP) in 187 us, 1.38 PFLOP/s.
namespace bq {
constexpr int BK = 128;
constexpr uint32_t SLOT = 32768;
constexpr int NSLOT = 3, KS = 0, VS = 1, KD = 2;         // K by keys, V by keys, K by columns
constexpr uint32_t OFF_Q = 0, OFF_DO = 65536, OFF_SLOT = 131072, OFF_BAR = OFF_SLOT + NSLOT * SLOT;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 256 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TM_DQ = 0, TM_S = 256, TM_DP = 384;
constexpr int kThreads = 352, kWarpTma = 8, kWarpMma = 9, kWarpQ = 10;
}  // namespace bq

__global__ void __launch_bounds__(bq::kThreads, 1)
mqa_dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
              const __grid_constant__ CUtensorMap map_ks, const __grid_constant__ CUtensorMap map_vs,
              const __grid_constant__ CUtensorMap map_kd, const Args a) {
    using namespace bq;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const uint32_t bars = sb + OFF_BAR;
    const uint32_t q_full = bars, q_empty = bars + 8, do_full = bars + 16, do_empty = bars + 24, dq_done = bars + 32,
                   dq_free = bars + 40, mma_done = bars + 48, s_full = bars + 56, s_free = bars + 64, dp_full = bars + 72,
                   ds_full = bars + 80;
    auto full = [&](uint32_t s) { return bars + 88 + 8 * s; };
    auto empty = [&](uint32_t s) { return bars + 88 + 8 * NSLOT + 8 * s; };
    volatile uint32_t* tmem_s = reinterpret_cast<volatile uint32_t*>(smem + OFF_BAR + 88 + 16 * NSLOT);
    const Guard g{reinterpret_cast<volatile int*>(smem + OFF_BAR + 96 + 16 * NSLOT), a.status, a.timeout_ns};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(do_full, 1);
        mbar_init(do_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(s_free, 16);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 16);
        mbar_init(dq_done, 1);
        mbar_init(dq_free, 16);
        mbar_init(mma_done, 1);
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        *g.abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc_pair(smem_u32((const void*)tmem_s), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    pdl_wait();
    // mqa_dkv_kernel may run beside this one: all that it reads is complete, and visible here by the wait, so to those
    // that see this flag
    if (blockIdx.x == 0 && threadIdx.x == 0) st_release_gpu(a.delta_there, 1);
    pdl_launch();

    // Number i of the pair's key tiles uses each of the three buffers for the i-th time.
    if (warp == kWarpTma) {
        if (lane == 0) {
            const uint32_t lead = map_to_rank(bars, 0) - bars;
            bool ok = true;
            uint32_t n_loads[NSLOT] = {};
            auto load = [&](uint32_t slot, const CUtensorMap* m, const QTile& q, int j, uint32_t i) {
                if (i > 0 && !wait(empty(slot), (i - 1) & 1, g, 1)) return false;
                n_loads[slot] = i + 1;
                if (rank == 0) mbar_arrive_expect_tx(full(slot), 2 * SLOT);
                const int key0 = q.lo + j * BK;
                if (slot == KD) {                                    // 128 keys, this CTA's 128 columns
                    for (int c = 0; c < 2; ++c)
                        tma_load_3d_pair(sb + OFF_SLOT + slot * SLOT + c * 16384, m, (int)rank * 128 + c * 64, key0, q.b, full(slot) + lead);
                } else {                                             // this CTA's 64 keys, all columns
                    for (int c = 0; c < 4; ++c)
                        tma_load_3d_pair(sb + OFF_SLOT + slot * SLOT + c * 8192, m, c * 64, key0 + (int)rank * (q.half<BK>(j) ? 32 : 64), q.b,
                                         full(slot) + lead);
                }
                return true;
            };
            // the order of the MMAs: K and V of the first tile, then K by keys, K by columns of the tile before, V
            QTiles<BK> qs(a, pair, npairs), qd = qs;
            int js = 0, jd = 0;
            uint32_t i = 0;
            bool more = qs.advance(a);
            qd.advance(a);
            while (ok && (more || i > 0)) {
                if (more) ok = load(KS, &map_ks, qs.t, js, i);
                if (ok && i > 0) {
                    ok = load(KD, &map_kd, qd.t, jd, i - 1);
                    if (++jd == qd.n) {
                        jd = 0;
                        qd.advance(a);
                    }
                }
                if (!more) break;
                ok = ok && load(VS, &map_vs, qs.t, js, i);
                ++i;
                if (++js == qs.n) {
                    js = 0;
                    more = qs.advance(a);
                }
            }
            // no bulk copy may still be writing shared memory at the exit: the leader sees both CTAs' land
            if (rank == 0) {
                const uint64_t t0 = globaltimer_ns();
#pragma unroll
                for (uint32_t s = 0; s < NSLOT; ++s)
                    while (n_loads[s] && !mbar_try_wait_cluster(full(s), (n_loads[s] - 1) & 1) && globaltimer_ns() - t0 < a.timeout_ns) {
                    }
            }
        }
    } else if (warp == kWarpQ) {
        // Q and dO: each as soon as the MMAs before are through with its buffer
        if (lane == 0) {
            const uint32_t lead = map_to_rank(bars, 0) - bars;
            QTiles<BK> q(a, pair, npairs);
            bool ok = true;
            auto load_rows = [&](const CUtensorMap* m, uint32_t off, uint32_t bar, uint32_t freed) {
                if (q.k > 0 && !wait(freed, (q.k - 1) & 1, g, 2)) return false;
                if (rank == 0) mbar_arrive_expect_tx(bar, 2 * 65536);
                for (int c = 0; c < 4; ++c)
                    tma_load_3d_pair(sb + off + c * 16384, m, c * 64, q.t.r0 + (int)rank * 128, q.t.b, bar + lead);
                return true;
            };
            while (ok && q.advance(a))
                ok = load_rows(&map_q, OFF_Q, q_full, q_empty) && load_rows(&map_do, OFF_DO, do_full, do_empty);
            const uint64_t t0 = globaltimer_ns();
            if (rank == 0 && ok && q.k > 0)
                while (!(mbar_try_wait_cluster(q_full, (q.k - 1) & 1) && mbar_try_wait_cluster(do_full, (q.k - 1) & 1)) &&
                       globaltimer_ns() - t0 < a.timeout_ns) {
                }
        }
    } else if (warp == kWarpMma) {
        if (rank == 0) {
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t id_full = idesc_bf16(256, BK, 0), id_half = idesc_bf16(256, BK / 2, 0), id_q = idesc_bf16(256, D, 1);
            QTiles<BK> qs(a, pair, npairs), qd = qs;                 // S and dP run one key tile ahead of dQ, across query tiles
            int js = 0;
            uint32_t i = 0;                                          // the key tile whose dQ is next
            bool more = qs.advance(a), ok = true;
            // 256 rows (at off_a) times the 128 keys in a slot (which are there)
            auto issue = [&](uint32_t off_a, uint32_t d, uint32_t slot, uint32_t done, uint32_t rows_free) {
                const uint32_t id_s = qs.t.half<BK>(js) ? id_half : id_full;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_ss_pair(tm + d, desc_k_sw128(sb + off_a + (ks >> 2) * 16384 + (ks & 3) * 32),
                                    desc_k_sw128(sb + OFF_SLOT + slot * SLOT + (ks >> 2) * 8192 + (ks & 3) * 32), id_s, ks > 0 ? 1u : 0u);
                    mma_commit_pair(done);
                    mma_commit_pair(empty(slot));
                    if (js + 1 == qs.n) mma_commit_pair(rows_free);
                }
                __syncwarp();
            };
            auto issue_s = [&]() {
                if (js == 0 && !wait_w(q_full, qs.k & 1, g, 3)) return false;
                issue(OFF_Q, TM_S, KS, s_full, q_empty);
                return true;
            };
            auto issue_dp = [&]() {
                if (js == 0 && !wait_w(do_full, qs.k & 1, g, 5)) return false;
                issue(OFF_DO, TM_DP, VS, dp_full, do_empty);
                if (++js == qs.n) {
                    js = 0;
                    more = qs.advance(a);
                }
                return true;
            };
            if (more) ok = wait_w(full(KS), 0, full(VS), 0, g, 4) && issue_s() && issue_dp();
            while (ok && qd.advance(a))
                for (int j = 0; j < qd.n; ++j, ++i) {
                    const bool next = more;
                    if (next && !(ok = wait_w(s_free, i & 1, full(KS), (i + 1) & 1, g, 9) && issue_s())) break;
                    if (j == 0 && qd.k > 0 && !(ok = wait_w(dq_free, (qd.k - 1) & 1, g, 8))) break;
                    if (!(ok = wait_w(ds_full, i & 1, full(KD), i & 1, g, 6))) break;
                    tc_fence_after();
                    const int steps = qd.t.half<BK>(j) ? BK / 32 : BK / 16;
                    if (elect_one()) {
                        // dS of keys [16 ks, 16 ks + 16): the two halves of a row sit 64 columns apart
#pragma unroll
                        for (int ks = 0; ks < BK / 16; ++ks)
                            if (ks < steps)
                                mma_ts_pair(tm + TM_DQ, tm + TM_DP + (ks >> 2) * 64 + (ks & 3) * 8,
                                            desc_mn_sw128(sb + OFF_SLOT + KD * SLOT + ks * 2048, 16384), id_q,
                                            (j > 0 || ks > 0) ? 1u : 0u);
                        mma_commit_pair(empty(KD));
                        if (j == qd.n - 1) mma_commit_pair(dq_done);
                    }
                    __syncwarp();
                    if (next && !(ok = wait_w(full(VS), (i + 1) & 1, g, 7) && issue_dp())) break;
                }
            if (elect_one()) mma_commit_pair(mma_done);
            __syncwarp();
        }
        if (lane == 0) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait_cluster(mma_done, 0) && globaltimer_ns() - t0 < 4 * a.timeout_ns) {
            }
        }
        __syncwarp();
    } else {
        const int r = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t lead = map_to_rank(bars, 0) - bars;
        uint32_t gt = 0;
        // dq of query tile k - 1, after the first dS of tile k
        int p_b = 0, p_row = 0;
        auto finish = [&](int kp) {
            if (!wait_w(dq_done, kp & 1, g, 12)) return false;
            tc_fence_after();
            // turn back: columns [64 half, +64) and their partners 128 further; stores as in the forward
            const int row0 = p_row & ~3;
            __nv_bfloat16* dst = a.dq + ((size_t)p_b * a.TH + row0) * D + half * 64 + 8 * (lane & 3);
            const float4* cs = reinterpret_cast<const float4*>(a.cs + (size_t)(min(p_row, a.TH - 1) / a.H) * (D / 2) + half * 64);
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
                uint32_t o1[16], o2[16];
#pragma unroll
                for (int g16 = 0; g16 < 2; ++g16) {
                    float x1[16], x2[16];
                    float4 fs[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) fs[e] = cs[c / 2 + 8 * g16 + e];   // (cos, sin) of two pairs
                    tmem_ld16(tl + TM_DQ + half * 64 + c + 16 * g16, x1);
                    tmem_ld16(tl + TM_DQ + 128 + half * 64 + c + 16 * g16, x2);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 f = fs[e];
                        const float y0 = x1[2 * e] * a.scale, y1 = x1[2 * e + 1] * a.scale;
                        const float z0 = x2[2 * e] * a.scale, z1 = x2[2 * e + 1] * a.scale;
                        o1[8 * g16 + e] = bf16x2(y0 * f.x + z0 * f.y, y1 * f.z + z1 * f.w);
                        o2[8 * g16 + e] = bf16x2(z0 * f.x - y0 * f.y, z1 * f.z - y1 * f.w);
                    }
                }
                quad_transpose(o1);
                quad_transpose(o2);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (row0 + i < a.TH) {
                        *reinterpret_cast<uint4*>(dst + (size_t)i * D + c) = make_uint4(o1[4 * i], o1[4 * i + 1], o1[4 * i + 2], o1[4 * i + 3]);
                        *reinterpret_cast<uint4*>(dst + (size_t)i * D + 128 + c) = make_uint4(o2[4 * i], o2[4 * i + 1], o2[4 * i + 2], o2[4 * i + 3]);
                    }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(dq_free + lead);
            return true;
        };
        bool ok = true;
        QTiles<BK> q(a, pair, npairs);
        while (ok && q.advance(a)) {
            const QTile t = q.t;
            const int row0 = t.r0 + (int)rank * 128, row = row0 + r;
            const bool live = row < a.TH;
            const int tok = min(row, a.TH - 1) / a.H;
            const int lo_row = live ? a.lo[(size_t)t.b * a.T + tok] : 0x7fffffff;   // a row past the end sees no key
            const int full_lo = row0 + 127 < a.TH ? a.lo[(size_t)t.b * a.T + (row0 + 127) / a.H] : 0x7fffffff;
            const int full_hi = min(row0, a.TH - 1) / a.H;
            const float nl = live ? a.neg_lse[(size_t)t.b * a.THp + row] : 0.f;
            const float nd = live ? a.neg_delta[(size_t)t.b * a.THp + row] : 0.f;
            for (int j = 0; j < q.n; ++j) {
                const uint32_t par = (gt + j) & 1;
                if (!(ok = wait_w(s_full, par, g, 10))) break;
                tc_fence_after();
                float s[64];
                tmem_ld32(tl + TM_S + half * 64, s);
                tmem_ld32(tl + TM_S + half * 64 + 32, s + 32);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(s_free + lead);
                const int key0 = t.lo + j * BK;
                const bool whole = key0 >= full_lo && key0 + BK - 1 <= full_hi;
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    const float2 x = fma2(make_float2(s[c], s[c + 1]), make_float2(a.scale_log2, a.scale_log2), make_float2(nl, nl));
                    s[c] = ex2_approx(x.x);
                    s[c + 1] = ex2_approx(x.y);
                }
                if (!whole) {
                    const int c_lo = lo_row - (key0 + half * 64), c_hi = tok - (key0 + half * 64);
#pragma unroll
                    for (int c = 0; c < 64; ++c) s[c] = (c >= c_lo && c <= c_hi) ? s[c] : 0.f;
                }
                if (!(ok = wait_w(dp_full, par, g, 11))) break;
                tc_fence_after();
                float dp[32];
                uint32_t v[32];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    tmem_ld32(tl + TM_DP + half * 64 + 32 * e, dp);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 x = mul2(make_float2(s[32 * e + 2 * c], s[32 * e + 2 * c + 1]),
                                              add2(make_float2(dp[2 * c], dp[2 * c + 1]), make_float2(nd, nd)));
                        v[16 * e + c] = bf16x2(x.x, x.y);
                    }
                }
                tmem_st32(tl + TM_DP + half * 64, v);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(ds_full + lead);
                if (j == 0 && q.k > 0 && !(ok = finish(q.k - 1))) break;
            }
            p_b = t.b;
            p_row = row;
            gt += q.n;
        }
        if (ok && q.k > 0) finish(q.k - 1);
        tmem_wait_ld();
        tmem_wait_st();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------- backward: dk, dv --------------------
// A cluster of two CTAs takes 128 keys and walks the query rows that see them in tiles of 64 rows:
//   CTA 0:  S^T  = K Q^T   (M 128, N 64, K 256; K in TMEM),   dV += P^T dO    (M 128, N 256, K 64)
//   CTA 1:  dP^T = V dO^T  (the same, V in TMEM),             dK += dS^T Q
// The two fp32 accumulators of a key tile are 256 TMEM columns each, a CTA's whole TMEM together; so each CTA
// keeps one, 128 columns of its stationary operand and two buffers of 64 for S^T or dP^T, over which
// P^T or dS^T is written in bf16 as the A operand of the second product.  CTA 0 hands its P^T to CTA 1
// through distributed shared memory (16 KB a tile, two buffers).  Thread = (key, 64 rows); two
// warpgroups take every other tile.
// The (key tile, row tile) products of all key tiles form one line, cut into equal pieces for the clusters
// (cum = the line's length before each key tile), so that every cluster has the same work whatever the
// documents; a piece of a key tile leaves its sums in fp32 as part number (cluster + key tile), and
// mqa_dkv_sum_kernel adds the parts of a key tile in order: the same bits at every run.
// Bound by shared memory and the tensor pipe together (a row tile's operands are read twice, 64 rows at a time):
// 8 x 2048 tokens, 10 heads, window 2048 (344 GFLOP) in 303 us, 1.13 PFLOP/s.  (Row tiles of 128, which need P^T in
// shared memory: 448 us.  Both warpgroups on every row tile: 337 us.)
namespace bk {
constexpr int BR = kRowTile, BKEY = kKeyTile;
constexpr uint32_t SLOT = 32768;
constexpr int NSLOT = 6, NVEC = 4;
constexpr uint32_t OFF_P = NSLOT * SLOT, OFF_VEC = OFF_P + 2 * 16384, OFF_BAR = OFF_VEC + NVEC * 256;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 320 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TM_ACC = 0, TM_A = 256, TM_S = 384;
constexpr int kThreads = 320, kWarpTma = 8, kWarpMma = 9;
constexpr size_t PART_FLOATS = (size_t)BKEY * D;         // of one gradient: [D / 4][128 keys][4]
}  // namespace bk

// where the piece of cluster c of G begins; no piece is empty (clusters past the line's length have none)
__device__ __forceinline__ int pieces(long long total, int G) { return (int)min((long long)G, total); }
__device__ __forceinline__ long long piece(long long total, int c, int G) { return total * c / G; }

struct Seg {
    int j, b, key0, n;              // key tile, its batch row, its first key; row tiles of this piece
    int r0;                         // first row
};
// walks the key tiles of a piece; cum has nk + 1 entries, strictly increasing
struct Segs {
    const long long* cum;
    long long pos, end;
    int j;
    __device__ __forceinline__ Segs(const Args& a, int c, int G) : cum(a.cum) {
        const int nk = a.B * a.nkt;
        const long long total = cum[nk];
        G = pieces(total, G);
        j = 0;
        pos = end = 0;
        if (c >= G) return;
        pos = piece(total, c, G);
        end = piece(total, c + 1, G);
        int lo = 0, hi = nk;                             // the last j with cum[j] <= pos
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cum[mid] <= pos) lo = mid; else hi = mid;
        }
        j = lo;
    }
    __device__ __forceinline__ bool next(const Args& a, Seg& s) {
        if (pos >= end || j >= a.B * a.nkt) return false;
        const long long c0 = cum[j], c1 = cum[j + 1];
        s.j = j;
        s.b = j / a.nkt;
        s.key0 = (j % a.nkt) * bk::BKEY;
        s.r0 = s.key0 * a.H + (int)(pos - c0) * bk::BR;
        s.n = (int)(min(c1, end) - pos);
        pos += s.n;
        ++j;
        return true;
    }
};

__global__ void __launch_bounds__(bk::kThreads, 1)
mqa_dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
               const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const int* __restrict__ last_t, const Args a) {
    using namespace bk;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const uint32_t bars = sb + OFF_BAR;
    auto s_full = [&](uint32_t i) { return bars + 8 * i; };
    auto p_full = [&](uint32_t i) { return bars + 16 + 8 * i; };
    auto p_here = [&](uint32_t i) { return bars + 32 + 8 * i; };     // CTA 1: P^T has arrived
    auto p_free = [&](uint32_t i) { return bars + 48 + 8 * i; };     // CTA 0: CTA 1 has read it
    const uint32_t a_tmem = bars + 64, acc_done = bars + 72, mma_done = bars + 80;
    auto v_full = [&](uint32_t i) { return bars + 96 + 8 * i; };
    auto v_free = [&](uint32_t i) { return bars + 96 + 8 * NVEC + 8 * i; };
    auto full = [&](uint32_t s) { return bars + 96 + 16 * NVEC + 8 * s; };
    auto empty = [&](uint32_t s) { return bars + 96 + 16 * NVEC + 8 * NSLOT + 8 * s; };
    volatile uint32_t* tmem_s = reinterpret_cast<volatile uint32_t*>(smem + OFF_BAR + 96 + 16 * (NVEC + NSLOT));
    const Guard g{reinterpret_cast<volatile int*>(smem + OFF_BAR + 104 + 16 * (NVEC + NSLOT)), a.status, a.timeout_ns};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cl = blockIdx.x >> 1, G = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < NVEC; ++i) {
            mbar_init(v_full(i), 1);
            mbar_init(v_free(i), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 4);
            mbar_init(p_here(i), 1);                     // CTA 1 expects the bytes
            mbar_init(p_free(i), 4);
        }
        mbar_init(a_tmem, 8);
        mbar_init(acc_done, 1);
        mbar_init(mma_done, 1);
        *g.abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32((const void*)tmem_s), 512);
        tmem_relinquish();
    }
    // This kernel starts when mqa_dq_kernel allows it, not at that one's end, and the permission alone orders no memory.
    // dq's flag does: released behind dq's own wait for the kernels before, acquired here ahead of every read.  Should
    // it not be there yet, dq's end does.  (Waiting for that end always: the SMs that dq leaves early stand idle.)
    if (threadIdx.x == 0 && ld_acquire_gpu(a.delta_there) != 1u) pdl_wait();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    pdl_launch();
    Segs segs(a, cl, G);
    Seg sg{};

    // Slots in order, per piece of a key tile: the stationary operand's two column halves, then the first
    // product's rows X_0 and, for every j >= 1, X_j and the second product's rows Y_{j-1}, and Y_{n-1}: the order of
    // the MMAs, which give an X back long before its Y (CTA 0: X = Q, Y = dO; CTA 1: the other way round).
    // The rows' L (CTA 0) or delta (CTA 1) have a ring of their own.
    if (warp == kWarpTma) {
        if (lane == 0) {
            const CUtensorMap *map_a = rank == 0 ? &map_k : &map_v, *map_x = rank == 0 ? &map_q : &map_do,
                              *map_y = rank == 0 ? &map_do : &map_q;
            const float* vec = rank == 0 ? a.neg_lse : a.neg_delta;
            fence_proxy_async_global();                  // the copies below come after the flag, too
            uint32_t L = 0, gi = 0;
            bool ok = true;
            auto load = [&](const CUtensorMap* m, int row, uint32_t box, int c0, int nc) {   // nc boxes from column block c0
                const uint32_t s = L % NSLOT, u = L / NSLOT;
                ++L;
                if (u > 0 && !wait(empty(s), (u - 1) & 1, g, 1)) return false;
                mbar_arrive_expect_tx(full(s), SLOT);
                for (int c = 0; c < nc; ++c) tma_load_3d(sb + s * SLOT + c * box, m, (c0 + c) * 64, row, sg.b, full(s));
                return true;
            };
            while (ok && segs.next(a, sg)) {
                ok = load(map_a, sg.key0, 16384, 0, 2) && load(map_a, sg.key0, 16384, 2, 2);
                for (int j = 0; ok && j <= sg.n; ++j) {
                    if (j < sg.n) {
                        const uint32_t i = gi + j, ve = i % NVEC, u = i / NVEC;
                        const int r = sg.r0 + j * BR;
                        if (!(ok = load(map_x, r, 8192, 0, 4))) break;
                        if (u > 0 && !(ok = wait(v_free(ve), (u - 1) & 1, g, 11))) break;
                        mbar_arrive_expect_tx(v_full(ve), 256);
                        bulk_load(sb + OFF_VEC + ve * 256, vec + (size_t)sg.b * a.THp + r, 256, v_full(ve));
                    }
                    if (j >= 1) ok = load(map_y, sg.r0 + (j - 1) * BR, 8192, 0, 4);
                }
                gi += sg.n;
            }
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t l = L > NSLOT ? L - NSLOT : 0; l < L; ++l)
                while (!mbar_try_wait(full(l % NSLOT), (l / NSLOT) & 1) && globaltimer_ns() - t0 < a.timeout_ns) {
                }
            for (uint32_t l = gi > NVEC ? gi - NVEC : 0; l < gi; ++l)
                while (!mbar_try_wait(v_full(l % NVEC), (l / NVEC) & 1) && globaltimer_ns() - t0 < a.timeout_ns) {
                }
        }
    } else if (warp == kWarpMma) {
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t id_s = idesc_bf16(128, BR, 0), id_a = idesc_bf16(128, D, 1);
        uint32_t L = 0, gi = 0, ns = 0;
        bool ok = true;
        auto wait_slot = [&](uint32_t l) { return wait_w(full(l % NSLOT), (l / NSLOT) & 1, g, 3); };
        for (; ok && segs.next(a, sg); ++ns) {
            if (!(ok = wait_w(a_tmem, ns & 1, g, 2))) break;
            tc_fence_after();
            if (elect_one()) {
                mma_commit(empty(L % NSLOT));
                mma_commit(empty((L + 1) % NSLOT));
            }
            __syncwarp();
            L += 2;
            auto issue_s = [&](int j) {                              // S^T_j from the next slot
                const uint32_t s = L % NSLOT, buf = (gi + j) & 1;
                ++L;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_ts(tm + TM_S + buf * BR, tm + TM_A + ks * 8,
                               desc_k_sw128(sb + s * SLOT + (ks >> 2) * 8192 + (ks & 3) * 32), id_s, ks > 0 ? 1u : 0u);
                    mma_commit(s_full(buf));
                    mma_commit(empty(s));
                }
                __syncwarp();
            };
            for (int j = 0; ok && j < min(2, sg.n); ++j)
                if ((ok = wait_slot(L))) issue_s(j);
            for (int j = 0; ok && j < sg.n; ++j) {
                const uint32_t i = gi + j, buf = i & 1, s = L % NSLOT;
                const bool more = j + 2 < sg.n;
                const uint32_t lx = more ? L + 1 : L;                // X_{j+2} behind Y_j
                if (!(ok = wait_w(p_full(buf), (i >> 1) & 1, full(s), (L / NSLOT) & 1, full(lx % NSLOT), (lx / NSLOT) & 1, g, 4))) break;
                ++L;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < BR / 16; ++ks)
                        mma_ts(tm + TM_ACC, tm + TM_S + buf * BR + ks * 8,
                               desc_mn_sw128(sb + s * SLOT + ks * 2048, 8192), id_a, (j > 0 || ks > 0) ? 1u : 0u);
                    mma_commit(empty(s));
                    if (j == sg.n - 1) mma_commit(acc_done);
                }
                __syncwarp();
                if (more) issue_s(j + 2);
            }
            gi += sg.n;
        }
        if (elect_one()) mma_commit(mma_done);
        __syncwarp();
        if (lane == 0) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(mma_done, 0) && globaltimer_ns() - t0 < a.timeout_ns) {
            }
        }
        __syncwarp();
    } else {
        const int r = (warp & 3) * 32 + lane, wg = warp >> 2;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t peer_p = map_to_rank(sb + OFF_P, 1), peer_here = map_to_rank(p_here(0), 1),
                       peer_free = map_to_rank(p_free(0), 0);
        uint32_t L = 0, gi = 0, ns = 0;
        bool ok = true;
        for (; ok && segs.next(a, sg); ++ns) {
            // the rows that this thread's key sees: [key H, (last + 1) H)
            const int key = sg.key0 + r;
            const int last_key = min(sg.key0 + BKEY, a.T) - 1;
            const int* lt = last_t + (size_t)sg.b * a.T;
            const int row_lo = key < a.T ? key * a.H : 0x7fffffff, row_hi = key < a.T ? (lt[key] + 1) * a.H - 1 : -1;
            // rows that every key of the tile sees
            const int all_lo = sg.key0 + BKEY <= a.T ? last_key * a.H : 0x7fffffff, all_hi = (lt[sg.key0] + 1) * a.H - 1;
            // the stationary operand's columns [128 wg, +128): shared memory (swizzled rows) to TMEM
            const uint32_t la = L + wg;
            if (!(ok = wait_w(full(la % NSLOT), (la / NSLOT) & 1, g, 5))) break;
            for (int c = 2 * wg; c < 2 * wg + 2; ++c) {
                const uint8_t* src = smem + (la % NSLOT) * SLOT + (c & 1) * 16384 + r * 128;
                uint32_t v[32];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    *reinterpret_cast<uint4*>(v + 4 * e) = *reinterpret_cast<const uint4*>(src + ((e ^ (r & 7)) << 4));
                tmem_st32(tl + TM_A + c * 32, v);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(a_tmem);
            L += 2 + 2 * sg.n;
            for (int j = 0; j < sg.n; ++j) {
                const uint32_t i = gi + j, buf = i & 1, u = i >> 1, ve = i % NVEC;
                if ((int)buf != wg) continue;
                if (!(ok = wait_w(v_full(ve), (i / NVEC) & 1, g, 6))) break;   // L or delta
                if (!(ok = wait_w(s_full(buf), u & 1, g, 7))) break;
                tc_fence_after();
                float s[64];
                tmem_ld32(tl + TM_S + buf * BR, s);
                tmem_ld32(tl + TM_S + buf * BR + 32, s + 32);
                const float4* vec = reinterpret_cast<const float4*>(smem + OFF_VEC + ve * 256);
                const int r0 = sg.r0 + j * BR;
                const bool whole = r0 >= all_lo && r0 + BR - 1 <= all_hi;
                const int c_lo = row_lo - r0, c_hi = row_hi - r0;
                uint32_t v[32];
                if (rank == 0) {
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float4 f = vec[c];
                        const float2 k = make_float2(a.scale_log2, a.scale_log2);
                        const float2 x = fma2(make_float2(s[4 * c], s[4 * c + 1]), k, make_float2(f.x, f.y));
                        const float2 y = fma2(make_float2(s[4 * c + 2], s[4 * c + 3]), k, make_float2(f.z, f.w));
                        s[4 * c] = ex2_approx(x.x);
                        s[4 * c + 1] = ex2_approx(x.y);
                        s[4 * c + 2] = ex2_approx(y.x);
                        s[4 * c + 3] = ex2_approx(y.y);
                    }
                    if (!whole) {
#pragma unroll
                        for (int c = 0; c < 64; ++c) s[c] = (c >= c_lo && c <= c_hi) ? s[c] : 0.f;
                    }
#pragma unroll
                    for (int c = 0; c < 32; ++c) v[c] = bf16x2(s[2 * c], s[2 * c + 1]);
                    tmem_st32(tl + TM_S + buf * BR, v);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(p_full(buf));
                        mbar_arrive(v_free(ve));
                    }
                    // the same to CTA 1, 16 bytes of every thread side by side
                    if (u > 0 && !(ok = wait_w(p_free(buf), (u - 1) & 1, g, 8))) break;
                    const uint32_t dst = peer_p + buf * 16384 + r * 16;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        st_async_v4(dst + c * 2048, v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3], peer_here + 8 * buf);
                } else {
                    if ((warp & 3) == 0 && lane == 0) mbar_arrive_expect_tx(p_here(buf), 16384);
                    if (!(ok = wait_w(p_here(buf), u & 1, g, 9))) break;
                    const uint8_t* src = smem + OFF_P + buf * 16384 + r * 16;
#pragma unroll
                    for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(v + 4 * c) = *reinterpret_cast<const uint4*>(src + c * 2048);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float4 f = vec[c];
                        const float2 p = make_float2(__uint_as_float(v[2 * c] << 16), __uint_as_float(v[2 * c] & 0xffff0000u));
                        const float2 q = make_float2(__uint_as_float(v[2 * c + 1] << 16), __uint_as_float(v[2 * c + 1] & 0xffff0000u));
                        const float2 x = mul2(p, add2(make_float2(s[4 * c], s[4 * c + 1]), make_float2(f.x, f.y)));
                        const float2 y = mul2(q, add2(make_float2(s[4 * c + 2], s[4 * c + 3]), make_float2(f.z, f.w)));
                        s[4 * c] = x.x;
                        s[4 * c + 1] = x.y;
                        s[4 * c + 2] = y.x;
                        s[4 * c + 3] = y.y;
                    }
                    if (!whole) {
#pragma unroll
                        for (int c = 0; c < 64; ++c) s[c] = (c >= c_lo && c <= c_hi) ? s[c] : 0.f;
                    }
#pragma unroll
                    for (int c = 0; c < 32; ++c) v[c] = bf16x2(s[2 * c], s[2 * c + 1]);
                    tmem_st32(tl + TM_S + buf * BR, v);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(p_full(buf));
                        mbar_arrive(v_free(ve));
                        mbar_arrive_pair(peer_free + 8 * buf);       // P^T has been used
                    }
                }
            }
            gi += sg.n;
            if (!ok || !(ok = wait_w(acc_done, ns & 1, g, 10))) break;
            tc_fence_after();
            float4* part = reinterpret_cast<float4*>(a.part + ((size_t)(cl + sg.j) * 2 + rank) * PART_FLOATS);
#pragma unroll 1
            for (int c = wg * 128; c < wg * 128 + 128; c += 32) {
                float o[32];
                tmem_ld32(tl + TM_ACC + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    part[(c / 4 + e) * BKEY + r] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
            tc_fence_before();
        }
        tmem_wait_ld();
        tmem_wait_st();
    }
    // the kernel behind this one has to find mqa_dq_kernel complete too
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The sum of a key tile's parts in the clusters' order; dk is scaled and turned back.  Thread = (key, 4 columns of the
// first half and their partners of the second); block = 32 keys x 32 columns twice; z = 0: dv, 1: dk.  Bound by reading the
// parts (128 KB each: 53 MB at 128 key tiles and 74 clusters, mostly still in L2).
__global__ void __launch_bounds__(256) mqa_dkv_sum_kernel(const Args a, int G) {
    using namespace bk;
    pdl_launch();
    const int j = blockIdx.x, z = blockIdx.z, r = (blockIdx.y & 3) * 32 + (threadIdx.x >> 3);
    const int grp = (blockIdx.y >> 2) * 8 + (threadIdx.x & 7);           // columns [4 grp, +4) and 128 further
    const int b = j / a.nkt, key = (j % a.nkt) * BKEY + r;
    pdl_wait();
    const long long total = a.cum[a.B * a.nkt], x0 = a.cum[j], x1 = a.cum[j + 1] - 1;
    G = pieces(total, G);
    auto cluster_of = [&](long long x) {
        int c = (int)(x * G / total);
        while (c + 1 < G && piece(total, c + 1, G) <= x) ++c;
        while (c > 0 && piece(total, c, G) > x) --c;
        return c;
    };
    const int c0 = cluster_of(x0), c1 = cluster_of(x1);
    if (key >= a.T) return;
    const float4* cs = reinterpret_cast<const float4*>(a.cs + (size_t)key * (D / 2) + 4 * grp);
    const float4 f0 = cs[0], f1 = cs[1];
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
        const float4* part = reinterpret_cast<const float4*>(a.part + ((size_t)(c + j) * 2 + z) * PART_FLOATS) + r;
        const float4 u = part[grp * BKEY], v = part[(grp + 32) * BKEY];
        x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
        y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
    }
    if (z == 1) {
        const float4 u = make_float4(x.x * a.scale, x.y * a.scale, x.z * a.scale, x.w * a.scale);
        const float4 v = make_float4(y.x * a.scale, y.y * a.scale, y.z * a.scale, y.w * a.scale);
        x = make_float4(u.x * f0.x + v.x * f0.y, u.y * f0.z + v.y * f0.w, u.z * f1.x + v.z * f1.y, u.w * f1.z + v.w * f1.w);
        y = make_float4(v.x * f0.x - u.x * f0.y, v.y * f0.z - u.y * f0.w, v.z * f1.x - u.z * f1.y, v.w * f1.z - u.w * f1.w);
    }
    __nv_bfloat16* o = (z == 0 ? a.dv : a.dk) + ((size_t)b * a.T + key) * D + 4 * grp;
    *reinterpret_cast<uint2*>(o) = make_uint2(bf16x2(x.x, x.y), bf16x2(x.z, x.w));
    *reinterpret_cast<uint2*>(o + 128) = make_uint2(bf16x2(y.x, y.y), bf16x2(y.z, y.w));
}

// ---------------------------------------------------------------- backward: delta ------------------------
// delta = dO . out per query row, of out in the 16 bits of significand that the forward kept of it.  A warp takes kDeltaRows
// rows, their loads in flight together: bound by HBM (1280 bytes a row; 210 MB for 163840 rows: 32 us).
constexpr int kDeltaRows = 4, kDeltaWarps = 8;
__device__ __forceinline__ float with_low(uint32_t hi, uint32_t byte) {
    return __uint_as_float(hi + (uint32_t)((int)(byte << 24) >> 16));
}
__global__ void __launch_bounds__(32 * kDeltaWarps) mqa_delta_kernel(const Args a, const __nv_bfloat16* dout) {
    pdl_launch();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.delta_there = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row0 = ((long long)blockIdx.x * kDeltaWarps + warp) * kDeltaRows, rows = (long long)a.B * a.TH;
    uint4 x[kDeltaRows], y[kDeltaRows];
    uint2 w[kDeltaRows];
#pragma unroll
    for (int i = 0; i < kDeltaRows; ++i) {
        if (row0 + i >= rows) break;
        x[i] = reinterpret_cast<const uint4*>(dout + (row0 + i) * D)[lane];
        y[i] = reinterpret_cast<const uint4*>(a.out + (row0 + i) * D)[lane];
        w[i] = reinterpret_cast<const uint2*>(a.low + (row0 + i) * D)[lane];
    }
#pragma unroll
    for (int i = 0; i < kDeltaRows; ++i) {
        const long long row = row0 + i;
        if (row >= rows) break;
        const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t two = (e < 2 ? w[i].x : w[i].y) >> (16 * (e & 1));
            s = fmaf(__uint_as_float(xs[e] << 16), with_low(ys[e] << 16, two), s);
            s = fmaf(__uint_as_float(xs[e] & 0xffff0000u), with_low(ys[e] & 0xffff0000u, two >> 8), s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) a.neg_delta[row / a.TH * a.THp + row % a.TH] = -s;
    }
}

// What the forward keeps: lse, first keys and last queries, the backward's line, angles, the rotated queries and keys, the
// low bytes of out.
struct SaveLayout {
    size_t lse, lo, last, cum, cs, q_rot, k_rot, low, total;
};
inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
inline size_t row_pitch(const rglru_mqa_dims* d) { return ((size_t)d->seq_len * d->q_heads + 63) & ~size_t(63); }
inline int key_tiles(const rglru_mqa_dims* d) { return (d->seq_len + kKeyTile - 1) / kKeyTile; }
inline SaveLayout save_layout(const rglru_mqa_dims* d) {
    const size_t tok = (size_t)d->batch * d->seq_len;
    SaveLayout l{};
    size_t o = 0;
    l.lse = o; o = up256(o + d->batch * row_pitch(d) * 4);
    l.lo = o; o = up256(o + tok * 4);
    l.last = o; o = up256(o + tok * 4);
    l.cum = o; o = up256(o + ((size_t)d->batch * key_tiles(d) + 1) * 8);
    l.cs = o; o = up256(o + (size_t)d->seq_len * (D / 2) * sizeof(float2));
    l.q_rot = o; o = up256(o + tok * d->q_heads * D * 2);
    l.k_rot = o; o = up256(o + tok * D * 2);
    l.low = o; o = up256(o + tok * d->q_heads * D);
    l.total = o;
    return l;
}
struct WsLayout {
    size_t delta, part, total;
};
inline WsLayout ws_layout(const rglru_mqa_dims* d) {
    const size_t nk = (size_t)d->batch * key_tiles(d);
    WsLayout l{};
    size_t o = 256;                    // the status word, the flag
    l.delta = o; o = up256(o + d->batch * row_pitch(d) * 4);
    l.part = o; o = up256(o + (nk + kMaxClusters) * 2 * bk::PART_FLOATS * 4);
    l.total = o;
    return l;
}

inline Args make_args(const rglru_mqa_dims* d, void* save, void* ws) {
    const SaveLayout l = save_layout(d);
    const WsLayout wl = ws_layout(d);
    uint8_t *p = static_cast<uint8_t*>(save), *w = static_cast<uint8_t*>(ws);
    Args a{};
    a.B = d->batch; a.T = d->seq_len; a.H = d->q_heads;
    a.TH = a.T * a.H; a.THp = (int)row_pitch(d);
    a.ntr = (a.TH + 255) / 256;
    a.nkt = key_tiles(d);
    a.scale = d->scale; a.scale_log2 = d->scale * kLog2e;
    a.cs = reinterpret_cast<const float2*>(p + l.cs);
    a.lo = reinterpret_cast<const int*>(p + l.lo);
    a.neg_lse = reinterpret_cast<float*>(p + l.lse);
    a.low = reinterpret_cast<int8_t*>(p + l.low);
    a.neg_delta = reinterpret_cast<float*>(w + wl.delta);
    a.cum = reinterpret_cast<const long long*>(p + l.cum);
    a.part = reinterpret_cast<float*>(w + wl.part);
    a.status = static_cast<DeviceStatus*>(ws);
    a.delta_there = reinterpret_cast<unsigned*>(w + 128);
    a.timeout_ns = 1000000000ull;
    return a;
}

// [B][rows][d] bf16, box 64 columns x box_rows, 128-byte swizzle; rows past a batch row's end read as zeros
inline bool map_rows(CUtensorMap* m, const void* base, int rows, int B, int box_rows) {
    return tc::make_map_3d_box_sw128(m, base, D, (uint64_t)rows, (uint64_t)B, 64, (uint32_t)box_rows, 1);
}

// how many 2-CTA clusters of a kernel fit on the device at once (asked once per kernel and device)
template <typename K>
cudaError_t resident_pairs(K kern, int threads, uint32_t smem, int which, int* pairs) {
    static std::mutex mu;
    static int cache[3][64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = set_smem_once(kern, (int)smem)) != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (cache[which][dev] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
        if (n <= 0) return cudaErrorLaunchOutOfResources;
        cache[which][dev] = std::min(n, kMaxClusters);
    }
    *pairs = cache[which][dev];
    return cudaSuccess;
}

// a launch behind the kernel before it on the stream (programmatic dependent), in clusters of `cluster` CTAs
template <typename... KArgs, typename... Given>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, int threads, uint32_t smem, int cluster, cudaStream_t s, const Given&... given) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, given...);
}

}  // namespace mt

size_t mqa_save_bytes(const rglru_mqa_dims* d) { return mt::save_layout(d).total; }
size_t mqa_train_workspace(const rglru_mqa_dims* d) { return mt::ws_layout(d).total; }

cudaError_t launch_mqa_forward(const rglru_mqa_dims* d, const void* q, const void* k, const void* v,
                               const uint8_t* reset, int pos0, void* out, void* save, void* ws, cudaStream_t s) {
    using namespace mt;
    const SaveLayout l = save_layout(d);
    uint8_t* p = static_cast<uint8_t*>(save);
    const int B = d->batch, T = d->seq_len, H = d->q_heads;
    int pairs = 0;
    cudaError_t e = resident_pairs(mqa_forward_kernel, fw::kThreads, fw::SMEM_BYTES, 0, &pairs);
    if (e != cudaSuccess) return e;
    Args a = make_args(d, save, ws);
    a.out = static_cast<__nv_bfloat16*>(out);
    CUtensorMap mq, mk, mv;
    if (!map_rows(&mq, p + l.q_rot, a.TH, B, 128) || !map_rows(&mk, p + l.k_rot, T, B, 64) || !map_rows(&mv, v, T, B, 128))
        return cudaErrorInvalidValue;
    const long long tokens = (long long)B * T;
    e = launch(mqa_prepare_kernel, dim3(B + (T + kAngleTokens - 1) / kAngleTokens), kScanThreads, 0, 1, s, B, T, d->window, reset,
               reinterpret_cast<int*>(p + l.lo), reinterpret_cast<int*>(p + l.last), pos0, rope_base(d->rope_base),
               reinterpret_cast<float2*>(p + l.cs));
    if (e != cudaSuccess) return e;
    e = launch(mqa_turn_kernel, dim3((unsigned)((tokens + 15) / 16 + 1)), kTurnThreads, 0, 1, s, tokens, T, H, a.cs,
               static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
               reinterpret_cast<__nv_bfloat16*>(p + l.q_rot), reinterpret_cast<__nv_bfloat16*>(p + l.k_rot),
               reinterpret_cast<const int*>(p + l.last), reinterpret_cast<long long*>(p + l.cum));
    if (e != cudaSuccess) return e;
    return launch(mqa_forward_kernel, dim3(2 * std::min(pairs, B * a.ntr)), fw::kThreads, fw::SMEM_BYTES, 2, s, mq, mk, mv, a);
}

cudaError_t launch_mqa_backward(const rglru_mqa_dims* d, const void* v, const void* out, const void* dout,
                                const void* save, void* dq, void* dk, void* dv, void* ws, cudaStream_t s) {
    using namespace mt;
    const SaveLayout l = save_layout(d);
    const uint8_t* p = static_cast<const uint8_t*>(save);
    const int B = d->batch, T = d->seq_len;
    int pq = 0, pk = 0;
    cudaError_t e = resident_pairs(mqa_dq_kernel, bq::kThreads, bq::SMEM_BYTES, 1, &pq);
    if (e == cudaSuccess) e = resident_pairs(mqa_dkv_kernel, bk::kThreads, bk::SMEM_BYTES, 2, &pk);
    if (e != cudaSuccess) return e;
    Args a = make_args(d, const_cast<void*>(save), ws);
    a.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out));
    a.dq = static_cast<__nv_bfloat16*>(dq);
    a.dk = static_cast<__nv_bfloat16*>(dk);
    a.dv = static_cast<__nv_bfloat16*>(dv);
    const int* last = reinterpret_cast<const int*>(p + l.last);
    CUtensorMap q128, do128, q64, do64, k64, v64, k128, v128;
    if (!map_rows(&q128, p + l.q_rot, a.TH, B, 128) || !map_rows(&do128, dout, a.TH, B, 128) ||
        !map_rows(&q64, p + l.q_rot, a.TH, B, 64) || !map_rows(&do64, dout, a.TH, B, 64) ||
        !map_rows(&k64, p + l.k_rot, T, B, 64) || !map_rows(&v64, v, T, B, 64) ||
        !map_rows(&k128, p + l.k_rot, T, B, 128) || !map_rows(&v128, v, T, B, 128))
        return cudaErrorInvalidValue;
    const long long rows = (long long)B * a.TH;
    constexpr int per = kDeltaWarps * kDeltaRows;
    e = launch(mqa_delta_kernel, dim3((unsigned)((rows + per - 1) / per)), 32 * kDeltaWarps, 0, 1, s, a,
               static_cast<const __nv_bfloat16*>(dout));
    if (e != cudaSuccess) return e;
    e = launch(mqa_dq_kernel, dim3(2 * std::min(pq, B * a.ntr)), bq::kThreads, bq::SMEM_BYTES, 2, s, q128, do128, k64, v64, k128, a);
    if (e != cudaSuccess) return e;
    e = launch(mqa_dkv_kernel, dim3(2 * pk), bk::kThreads, bk::SMEM_BYTES, 2, s, q64, do64, k128, v128, last, a);
    if (e != cudaSuccess) return e;
    return launch(mqa_dkv_sum_kernel, dim3(B * a.nkt, 16, 2), 256, 0, 1, s, a, pk);
}

}  // namespace rglru
