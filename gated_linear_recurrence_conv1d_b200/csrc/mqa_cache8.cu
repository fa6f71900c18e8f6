// mqa_cache8.cu -- the 8-bit ring cache of local MQA: written as it is quantised, read by the decode
// step, read back as the bf16 ring (head_dim 256).
//
// A slot holds the 256 elements of a rotated key (first half) or a value (second half) as e4m3 codes
// [B][2][w][d] with one fp32 scale each [B][2][w]:
//     scale = max(amax |x|, 448 * 2^-126) / 448,   code = e4m3(x / scale),   value = code * scale
// (448 is e4m3's largest value; the floor keeps the scale of a zero slot a normal number).  The key is
// rotated, and the quotient taken, in fp64 and rounded once to fp32 before the code: a code then does
// not depend on the rounding of a sine or a product next to a border between two codes.  (The quotient is the
// product with the fp64 reciprocal, off by 2^-52: after the rounding to fp32 a quotient that is exactly
// on a border, which has 5 bits, is on it again.)
#include <algorithm>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "angles.cuh"
#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "tma_maps.h"

namespace rglru {
namespace c8 {

using namespace pr;

constexpr int D = 256;
constexpr int kMaxH = 16;
constexpr int kTile = 128;             // slots per tile (the MMA's M)
constexpr int kGroups = 4;             // groups of 4 warps: group g has the heads h = g mod 4
constexpr int kHg = kMaxH / kGroups;
// rows of the queries' and weights' operands, columns of S and O: the heads of group 0, then those of group 1, ...
__host__ __device__ constexpr int head_row(int h) { return (h % kGroups) * kHg + h / kGroups; }
constexpr double kFloor = 448.0 * 1.1754943508222875e-38;

// ---- e4m3 ------------------------------------------------------------------------------------------
// codes of two fp32 values, lo in the low byte (round to nearest even, saturating)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// the same in e5m2 (2 mantissa bits, down to 2^-16: the upper byte of an fp16)
__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 e5m2x2_values(uint32_t c) {
    const uint32_t h = __byte_perm(c, 0, 0x1404);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// the values of two codes (exact in fp16)
__device__ __forceinline__ float2 e4m3x2_values(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// ---- one slot by one warp ------------------------------------------------------------------------------
// lane l holds the pairs j = 4 l .. 4 l + 3: elements j and j + 128
struct Pairs {
    uint2 a, b;                        // bf16
};
__device__ __forceinline__ Pairs load_pairs(const __nv_bfloat16* p, int lane) {
    return Pairs{reinterpret_cast<const uint2*>(p)[lane], reinterpret_cast<const uint2*>(p + D / 2)[lane]};
}
__device__ __forceinline__ void unpack(const Pairs& p, float (&x)[8]) {
    const uint32_t w[4] = {p.a.x, p.a.y, p.b.x, p.b.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
// this lane's codes: 4 of the first half, 4 of the second; every lane has the scale
struct SlotCodes {
    uint32_t a, b;
    float scale;
};
__device__ __forceinline__ SlotCodes quantise_slot(const double (&x)[8]) {
    // the largest |x| by its bits: a NaN is larger than infinity, so the slot is NaN as a whole
    long long m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __double_as_longlong(fabs(x[e])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    // Products with reciprocals off by 2^-52 instead of fp64 divisions, which took half of the fp64 pipe's time: rounded to
    // fp32 they are the quotients unless those are within 2^-51 of the middle of two fp32 numbers.  1 / s from its
    // fp32 value by two Newton steps (2^-22, 2^-44, 2^-52; s is at least 2^-126, so its reciprocal is finite).
    const float s = (float)(__longlong_as_double(max(m, __double_as_longlong(kFloor))) * (1.0 / 448.0));
    const double ds = (double)s;
    double r = (double)__frcp_rn(s);
    r = fma(r, fma(-ds, r, 1.0), r);
    r = fma(r, fma(-ds, r, 1.0), r);
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = (float)(x[e] * r);
    return SlotCodes{e4m3x2(q[0], q[1]) | e4m3x2(q[2], q[3]) << 16, e4m3x2(q[4], q[5]) | e4m3x2(q[6], q[7]) << 16, s};
}
// The same from fp32 (a value: nothing to rotate).  Rounding the quotients of bf16 numbers once to fp32 gives what rounding
// them to fp64 first gives: x / s with 8 bits over 24 is never within 2^-54 of the middle of two fp32 numbers.
__device__ __forceinline__ SlotCodes quantise_slot(const float (&x)[8]) {
    int m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_int(fabsf(x[e])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = __fdiv_rn(__int_as_float(max(m, __float_as_int((float)kFloor))), 448.0f);
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = __fdiv_rn(x[e], s);
    return SlotCodes{e4m3x2(q[0], q[1]) | e4m3x2(q[2], q[3]) << 16, e4m3x2(q[4], q[5]) | e4m3x2(q[6], q[7]) << 16, s};
}
__device__ __forceinline__ void store_slot(const SlotCodes& c, int lane, uint8_t* codes, float* scale) {
    reinterpret_cast<uint32_t*>(codes)[lane] = c.a;
    reinterpret_cast<uint32_t*>(codes + D / 2)[lane] = c.b;
    if (lane == 0) *scale = c.scale;
}
__device__ __forceinline__ void turn64(const float (&x)[8], const double2* cs, int lane, double (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const double2 a = cs[4 * lane + e];
        y[e] = (double)x[e] * a.x - (double)x[4 + e] * a.y;
        y[4 + e] = (double)x[4 + e] * a.x + (double)x[e] * a.y;
    }
}
// ---------------------------------------------------------------- write -------------------------------
// Block = (token, up to kWriteRows batch rows): the angles of the token's position once for all of them (they are
// half of the arithmetic), while the rows' keys and values are on their way; a warp per row.  The last min(len, w)
// tokens of a row go into their slots.  Bound by latency and issue, not by the fp64 pipe (16 % busy; the conversions
// between fp64 and fp32 fill theirs to 45 %): 2048 short blocks, each load -> angles -> barrier -> rotation ->
// maximum over the warp -> store, two and a half rounds of them.  8 rows of 2048 tokens in 12.7 us, of which the
// bytes need 4 (a block a row: 22.6 us, its own angles each time; fp64 divisions: 14.4 us).
constexpr int kWriteRows = 8;
__global__ void __launch_bounds__(32 * kWriteRows, 6)
mqa_cache8_write_kernel(int B, int T, int w, int pos0, RopeBase base, const int* lengths, const __nv_bfloat16* k,
                        const __nv_bfloat16* v, uint8_t* codes, float* scales) {
    __shared__ double2 cs[D / 2];
    const int t = blockIdx.x + (lengths ? 0 : max(0, T - w));
    const int lane = threadIdx.x & 31, b = blockIdx.y * kWriteRows + (threadIdx.x >> 5);
    bool mine = b < B;
    if (mine && lengths) {
        const int len = min(lengths[b], T);
        mine = t < len && t >= len - w;
    }
    if (!__syncthreads_or(mine)) return;
    Pairs pk{}, pv{};
    if (mine) {
        pk = load_pairs(k + ((size_t)b * T + t) * D, lane);
        pv = load_pairs(v + ((size_t)b * T + t) * D, lane);
    }
    const long long p = (long long)pos0 + t;
    if (threadIdx.x < D / 2) rope_cos_sin(base, threadIdx.x, (double)p, cs[threadIdx.x].x, cs[threadIdx.x].y);
    __syncthreads();
    if (!mine) return;
    const size_t s = (size_t)b * 2 * w + (int)(p % w);
    float x[8];
    double y[8];
    unpack(pk, x);
    turn64(x, cs, lane, y);
    store_slot(quantise_slot(y), lane, codes + s * D, scales + s);
    unpack(pv, x);
    store_slot(quantise_slot(x), lane, codes + (s + w) * D, scales + s + w);
}

// ---------------------------------------------------------------- read ---------------------------------
// A warp takes kReadSlots slots, a lane 8 codes of each, their loads in flight together: bound by HBM (64 rings of
// 2048 slots: 34.5 us, 5.9 TB/s; with 4 slots a warp and a division for each 41 us).
constexpr int kReadSlots = 8, kReadBlock = 8 * kReadSlots;           // slots of a block of 8 warps
__global__ void __launch_bounds__(256) mqa_cache8_read_kernel(long long slots, int w, const int* pos,
                                                              const uint8_t* codes, const float* scales,
                                                              __nv_bfloat16* cache) {
    const long long s0 = (long long)blockIdx.x * kReadBlock + (threadIdx.x >> 5) * kReadSlots;
    const int lane = threadIdx.x & 31;
    unsigned half = (unsigned)s0 / (unsigned)w;          // 2 row + (key, value); 2 B w < 2^31
    int slot = (int)((unsigned)s0 - half * (unsigned)w);
    uint2 u[kReadSlots];
    float f[kReadSlots];
    bool have[kReadSlots];
#pragma unroll
    for (int i = 0; i < kReadSlots; ++i) {
        const long long s = s0 + i;
        have[i] = s < slots && (!pos || slot <= pos[half >> 1]);
        if (++slot == w) {
            slot = 0;
            ++half;
        }
        if (have[i]) {
            u[i] = __ldcs(reinterpret_cast<const uint2*>(codes + s * D) + lane);
            f[i] = scales[s];
        }
    }
#pragma unroll
    for (int i = 0; i < kReadSlots; ++i) {
        if (!have[i]) continue;
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 x = e4m3x2_values(((e < 2 ? u[i].x : u[i].y) >> (16 * (e & 1))) & 0xffffu);
            o[e] = bf16x2(f[i] * x.x, f[i] * x.y);
        }
        __stcs(reinterpret_cast<uint4*>(cache + (s0 + i) * D) + lane, make_uint4(o[0], o[1], o[2], o[3]));
    }
}

// ---------------------------------------------------------------- decode: attention --------------------
// The slots of a row are cut into tiles of 128 and the tiles of all rows laid out as one line, of which every
// CTA takes an equal piece (a "segment" is a piece of one row): the rings' bytes are spread evenly
// over the SMs whatever the rows' lengths.  Per tile
//   S^T = K Qp^T   (M 128 slots, N 48 = 16 heads x 3 parts, K 256; e4m3, fp32 sums)
//   O^T += V^T Wp^T (M 128 columns twice, N 48 = 16 heads x 3 parts, K 128 slots)
// straight from the codes in shared memory (V^T is the value tile read MN-major).  Four groups of 4 warps, each
// with every fourth head, thread = slot: s = (S0 + S1 / 16 + S2 / 256) 2^e c scale_k, p = 2^(s - m) for the sum of
// the weights, and for the weighted sum of the codes alpha 2^(u - n), u = s + log2 scale_v, as three e5m2 parts.
// m and n are reference maxima of a head's s and u, which move when one passes them by more than 3 (8 times).  A
// reference of u, not one of s beside a largest scale: the scale of a slot that has no weight to speak of would
// push the others' weights out of e5m2's range.  Parts: what is left of a weight w after each is at most an
// eighth of it or 2^-17, so three (1, 1/8, 1/64) leave max(2^-9 w, 2^-23): 2^-9 of the weight, half of what bf16
// would leave, or 2^-35 of the segment's heaviest, whose w is 2^12 at least (e4m3 parts end at 2^-22 of it, which
// shows).  p adds to the thread's own sum in fp32.  O stays in TMEM for the whole segment, in units of 2^n / alpha;
// when n moves it is rescaled there (each group has its own columns of S, W and O, so within a segment the groups
// never meet).  A row inside one segment is written
// at once; else the segments leave (m, sum, O) and mqa_decode8_merge_kernel adds them up in order.  (The segment
// that finishes last doing that here, by a counter of the row, took longer at the end of the kernel, and its
// registers spilled the softmax's.)
// Before a segment its row's queries are rotated and their parts written as the B operand: with 2^e the power of two that
// brings the head's largest element into (224, 448], q~ = 2^e (x0 + x1 / 16 + x2 / 256) + r, x0 = e4m3(q~ 2^-e),
// x1 = e4m3(16 (q~ 2^-e - x0)), ...: a part is off by at most 2^-4 of itself, so |r| <= 2^-12 |q~| (or
// 2^-18 448 2^e where x2 is below e4m3's normal numbers), less than bf16 would leave.  The segment that holds the
// row's new slot also rotates and quantises the new key and value, writes them to the ring and hands them to the
// MMA warp, which puts them into the tiles that it has (they may have been loaded before the ring was written).
// All softmax warps prepare a CTA's first segment; two warps of their own the next one while a segment is worked on,
// with two buffers for everything prepared.  S runs one tile ahead of the weighted sum, across segments, and a
// segment's output is written after the first weights of the next.
// The step reads every code once: bound by HBM.  256 full rings of 2048 slots, 10 heads: 54.9 us in a graph, 58.6 us
// launched in a loop (272 MB; streaming alone would take 42), of which about 10 us pass at the two ends (the angles,
// the first tile's way through, the merge) and 2.5 us at each change of the row; a tile of 64 KB takes 1.40 us, and
// 1.15 us when the rings are in L2.
constexpr uint32_t TILE_BYTES = kTile * D;            // 32768: 2 boxes of [128 slots x 128 B]
constexpr int kNBuf = 5;
constexpr int kMaxCtas = 148;
constexpr int kQParts = 3, kQRows = kQParts * kMaxH;
constexpr uint32_t Q_BYTES = kQRows * D;              // 12288: 2 boxes of [48 x 128 B]
constexpr int kWParts = 3, kWRows = kWParts * kMaxH;
constexpr uint32_t W_BYTES = kWRows * kTile;          // 6144: [48 x 128 slots]
constexpr uint32_t RED_BYTES = 224;                   // of a group: [4 warps][kHg] of s, of u; a segment's [4 warps][kHg] sums, [kHg] m, [kHg] n
constexpr uint32_t STG_BYTES = 2 * D + 16;            // the new slot: key and value codes, their scales
constexpr uint32_t OFF_Q = kNBuf * TILE_BYTES, OFF_W = OFF_Q + 2 * Q_BYTES, OFF_CS = OFF_W + 2 * W_BYTES;
constexpr uint32_t IN_BYTES = (kMaxH + 2) * D * 2;     // a segment's queries, new key and value
constexpr uint32_t CS_BYTES = D / 2 * (16 + 8);         // cos, sin in fp64 (the new key), then in fp32 (the queries)
constexpr uint32_t OFF_IN = OFF_CS + 2 * CS_BYTES, OFF_STG = OFF_IN + 2 * IN_BYTES;
constexpr uint32_t OFF_QS = OFF_STG + 2 * STG_BYTES, OFF_SEG = OFF_QS + 2 * 64, OFF_SC = OFF_SEG + 2 * 32, OFF_RED = OFF_SC + 2 * 2 * kTile * 4;
constexpr uint32_t OFF_BAR = OFF_RED + kGroups * RED_BYTES;
constexpr uint32_t SMEM_BYTES = OFF_BAR + 256 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TM_S = 0, TM_O = 128, TMEM_COLS = 256;     // S: two buffers, 64 apart; O: two halves, 64 apart
constexpr int kSoftWarps = 4 * kGroups, kSoft = 32 * kSoftWarps, kWarpTma = kSoftWarps, kWarpMma = kSoftWarps + 1;
constexpr int kPrepWarps = 2;          // five warps a scheduler in all, with 96 registers as without them
constexpr int kThreads = kSoft + 64 + 32 * kPrepWarps;

constexpr float kLog2Alpha = 12.0f;                   // weights are held as alpha 2^(u - n): u - n <= 3 keeps them below 57344
// Where a head's n begins: below every log2 scale, and finite, so that slots whose scale is 0 (a ring of zeros that was not
// written there) have weight 2^(-inf - n) = 0 also where there is no other
constexpr float kNoU = -1.0e30f;

struct DecArgs {
    int B, H, w;
    float scale_log2;
    RopeBase base;
    const int* pos;
    const __nv_bfloat16 *q, *k, *v;
    uint8_t* codes;                    // [B][2][w][d]
    float* scales;                     // [B][2][w]
    int2* meta;                        // [B] the first and the last CTA of a row
    float* part;                       // [B + CTAs][part_pitch]: m [16], sum [16] by head_row, O [H][d]
    __nv_bfloat16* out;
    DeviceStatus* status;
    unsigned long long timeout_ns;
};

__host__ __device__ constexpr int part_pitch(int H) { return H * D + 2 * kMaxH; }

// e4m3 x e4m3 (b_e5m2 = 0) or e5m2 (1) -> fp32; A K-major (a_mn = 0) or MN-major (1), B K-major
__device__ __forceinline__ constexpr uint32_t idesc_fp8(int n, int a_mn, int b_e5m2) {
    return (1u << 4) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}
__device__ __forceinline__ void mma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(id), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ int slots_of(const DecArgs& a, int b) {
    const int p = a.pos[b];
    return p < 0 ? 0 : min(p, a.w - 1) + 1;
}
// Tiles of all rows: batch * window <= 2^29, so at most 2^22 + 2^16, and 148 times that fits 32 bits.
struct Walk {
    unsigned pos, end, total, row_beg;   // on the line; row_beg: where the current row begins
    unsigned G;
    int row;
};
struct DecSeg {
    int b, t0, nt, n, c0, c1;            // row, its first tile here, tiles here, slots of the row, the row's CTAs
    int last, slot;                      // the CTA's last one; the row's new slot
};
static_assert(sizeof(DecSeg) == 32, "two int4");
// the CTA whose piece [total c / G, total (c + 1) / G) holds x: the last c with total c < (x + 1) G
__device__ __forceinline__ int owner(unsigned x, unsigned total, unsigned G) { return (int)(((x + 1) * G - 1) / total); }
__device__ __forceinline__ bool next_seg(const DecArgs& a, Walk& k, DecSeg& s) {
    if (k.pos >= k.end) return false;
    int n;
    unsigned tiles;
    for (;;) {                           // rows without tokens have no tiles
        n = slots_of(a, k.row);
        tiles = (unsigned)(n + kTile - 1) / kTile;
        if (k.pos < k.row_beg + tiles) break;
        k.row_beg += tiles;
        if (++k.row >= a.B) return false;
    }
    s.b = k.row;
    s.n = n;
    s.t0 = (int)(k.pos - k.row_beg);
    s.nt = (int)(min(k.end, k.row_beg + tiles) - k.pos);
    const bool whole = s.nt == (int)tiles;
    s.c0 = whole ? (int)blockIdx.x : owner(k.row_beg, k.total, k.G);
    s.c1 = whole ? (int)blockIdx.x : owner(k.row_beg + tiles - 1, k.total, k.G);
    k.pos += s.nt;
    s.last = k.pos >= k.end;
    s.slot = a.pos[s.b] % a.w;
    return true;
}

// the maximum over the warp; NaN only where every lane's is
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// the OR of v over the threads that meet at barrier `id`
__device__ __forceinline__ bool named_or(bool v, int id, int threads) {
    uint32_t o;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(o)
        : "r"((uint32_t)v), "r"(id), "r"(threads)
        : "memory");
    return o != 0;
}

__global__ void __launch_bounds__(kThreads, 1)
mqa_decode8_kernel(const __grid_constant__ CUtensorMap map_kv, const DecArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const uint32_t bars = sb + OFF_BAR;
    auto full = [&](uint32_t i) { return bars + 8 * i; };
    auto empty = [&](uint32_t i) { return bars + 8 * kNBuf + 8 * i; };
    auto s_full = [&](uint32_t i) { return bars + 16 * kNBuf + 8 * i; };
    auto w_full = [&](uint32_t i) { return bars + 16 * kNBuf + 16 + 8 * i; };
    auto o_done = [&](uint32_t i) { return bars + 16 * kNBuf + 32 + 8 * i; };
    const uint32_t o_free = bars + 16 * kNBuf + 48, mma_done = o_free + 8;
    auto q_ready = [&](uint32_t i) { return bars + 16 * kNBuf + 64 + 8 * i; };
    auto q_free = [&](uint32_t i) { return bars + 16 * kNBuf + 80 + 8 * i; };
    auto in_full = [&](uint32_t i) { return bars + 16 * kNBuf + 96 + 8 * i; };
    auto in_free = [&](uint32_t i) { return bars + 16 * kNBuf + 112 + 8 * i; };
    volatile uint32_t* tmem_s = reinterpret_cast<volatile uint32_t*>(smem + OFF_BAR + 16 * kNBuf + 128);
    const Guard g{reinterpret_cast<volatile int*>(smem + OFF_BAR + 16 * kNBuf + 136), a.status, a.timeout_ns};
    unsigned* scan = reinterpret_cast<unsigned*>(smem);            // before the first load: per-warp sums
    Walk* walk_s = reinterpret_cast<Walk*>(smem + OFF_W);            // before the first weights
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kNBuf; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(w_full(i), kSoftWarps);
            mbar_init(o_done(i), 1);
            mbar_init(in_full(i), 1);
            mbar_init(in_free(i), 1);
            mbar_init(q_ready(i), 1);
            mbar_init(q_free(i), 1);
        }
        mbar_init(o_free, kSoftWarps);
        mbar_init(mma_done, 1);
        *g.abort = 0;
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32((const void*)tmem_s), TMEM_COLS);
        tmem_relinquish();
    }
    pdl_launch();
    pdl_wait();
    // this CTA's piece of the line of tiles: every thread counts the tiles of a run of rows
    {
        const int per = (a.B + kThreads - 1) / kThreads, r0 = min(a.B, (int)threadIdx.x * per), r1 = min(a.B, r0 + per);
        unsigned mine = 0;
        for (int b = r0; b < r1; ++b) mine += (slots_of(a, b) + kTile - 1) / kTile;
        unsigned sum = mine;                                        // through this thread, in the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        if (lane == 31) scan[warp] = sum;
        __syncthreads();
        unsigned before = sum - mine, total = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += scan[i];
            total += scan[i];
        }
        Walk k;
        k.total = total;
        k.G = min(gridDim.x, total);
        k.pos = k.end = 0;
        k.row = 0;
        k.row_beg = 0;
        const bool some = blockIdx.x < k.G;
        if (some) {
            k.pos = total * blockIdx.x / k.G;
            k.end = total * (blockIdx.x + 1) / k.G;
        }
        if (some ? (before <= k.pos && k.pos < before + mine) : threadIdx.x == 0) {
            k.row = r0;
            k.row_beg = before;
            *walk_s = k;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    Walk k = *walk_s;
    __syncthreads();                                                 // walk_s and scan give way to the tiles
    DecSeg sg{};

    // Segment n's queries, and its new slot if it holds it, into shared memory (and the ring), by `warps` warps, of which
    // this is number wi
    auto prepare = [&](const DecSeg& x, uint32_t n, int wi, auto num_warps, uint8_t* angles, auto all_or) {
        constexpr int warps = decltype(num_warps)::value;
        double2* cs = reinterpret_cast<double2*>(angles);
        float2* csf = reinterpret_cast<float2*>(angles + D / 2 * 16);
        uint8_t* stg = smem + OFF_STG + (n & 1) * STG_BYTES;
        const int p = a.pos[x.b], slot = x.slot;
        if (wi == 0 && lane == 0) *reinterpret_cast<DecSeg*>(smem + OFF_SEG + (n & 1) * 32) = x;
        const bool fresh = slot >= x.t0 * kTile && slot < (x.t0 + x.nt) * kTile;
        // the scales of the first tile, stored at the end (the new slot's come from elsewhere: these may be read before it is
        // written)
        constexpr int kPer = (kTile + 32 * warps - 1) / (32 * warps);
        float2 sc[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = 32 * (i * warps + wi) + lane, at = x.t0 * kTile + j;
            const float* src = a.scales + (size_t)x.b * 2 * a.w + at;
            sc[i] = j < kTile && at < x.n ? make_float2(src[0], src[a.w]) : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int j0 = 0; j0 < D / 2; j0 += 32 * warps) {
            const int j = j0 + 32 * wi + lane;
            if (j < D / 2) {
                double2 c;
                rope_cos_sin(a.base, j, (double)p, c.x, c.y);
                cs[j] = c;
                csf[j] = make_float2((float)c.x, (float)c.y);
            }
        }
        const __nv_bfloat16* in = reinterpret_cast<const __nv_bfloat16*>(smem + OFF_IN + (n & 1) * IN_BYTES);
        const bool here = wait_w(in_full(n & 1), (n >> 1) & 1, g, 12);
        if (all_or(!here)) return false;             // the angles are there too
#pragma unroll 1
        for (int i = wi; i < a.H + (fresh ? 2 : 0); i += warps) {
            float y[8], z[8];
            if (i >= a.H) {
                const int half = i - a.H;
                unpack(load_pairs(in + (kMaxH + half) * D, lane), z);
                SlotCodes c;
                if (half) {
                    c = quantise_slot(z);
                } else {
                    double d[8];
                    turn64(z, cs, lane, d);
                    c = quantise_slot(d);
                }
                const size_t at = ((size_t)x.b * 2 + half) * a.w + slot;
                store_slot(c, lane, a.codes + at * D, a.scales + at);
                store_slot(c, lane, stg + half * D, reinterpret_cast<float*>(stg + 2 * D) + half);
                continue;
            }
            unpack(load_pairs(in + i * D, lane), z);
            float mq = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float c = csf[4 * lane + e].x, s = csf[4 * lane + e].y;
                y[e] = z[e] * c - z[4 + e] * s;
                y[4 + e] = z[4 + e] * c + z[e] * s;
                mq = fmaxf(mq, fmaxf(fabsf(y[e]), fabsf(y[4 + e])));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, o));
            // mq / 448 rounded up to a power of two (at least 2^-100, so that its reciprocal is finite)
            const float r448 = fminf(fmaxf(mq, 448.0f * 7.9e-31f), 3.0e38f) * (1.0f / 448.0f);
            int e2 = (__float_as_int(r448) >> 23) - 127;
            if (__float_as_int(r448) & 0x7fffff) ++e2;
            const float up = __int_as_float((e2 + 127) << 23), down = __int_as_float((127 - e2) << 23);
            if (lane == 0)                            // a query with an infinity: NaN
                reinterpret_cast<float*>(smem + OFF_QS + (n & 1) * 64)[head_row(i)] = mq < INFINITY ? up : __int_as_float(0x7fffffff);
            uint32_t c[kQParts][2] = {};
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float u = y[e] * down, v = y[e + 1] * down;
#pragma unroll
                for (int part = 0; part < kQParts; ++part) {
                    const uint32_t cc = e4m3x2(u, v);
                    const float2 f = e4m3x2_values(cc);
                    c[part][e >> 2] |= cc << (8 * (e & 2));
                    u = (u - f.x) * 16.0f;
                    v = (v - f.y) * 16.0f;
                }
            }
            // row part * 16 + head_row of the two [48 x 128 bytes] blocks, 16-byte chunks swizzled by the row
#pragma unroll
            for (int part = 0; part < kQParts; ++part) {
                const int row = part * kMaxH + head_row(i);
                uint8_t* dst = smem + OFF_Q + (n & 1) * Q_BYTES + row * 128 + (((lane >> 2) ^ (row & 7)) << 4) + (lane & 3) * 4;
                *reinterpret_cast<uint32_t*>(dst) = c[part][0];
                *reinterpret_cast<uint32_t*>(dst + Q_BYTES / 2) = c[part][1];
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = 32 * (i * warps + wi) + lane;
            if (j < kTile) reinterpret_cast<float2*>(smem + OFF_SC)[(n & 1) * kTile + j] = sc[i];
        }
        fence_proxy_async_smem();
        if (all_or(false)) return false;              // (never: a barrier) every warp's part is there
        if (wi == 0 && lane == 0) {
            mbar_arrive(in_free(n & 1));
            mbar_arrive(q_ready(n & 1));
        }
        return true;
    };

    if (warp == kWarpTma) {
        if (lane == 0) {
            // a segment's inputs behind the first tile of the segment before it
            uint32_t L = 0, ns = 0;
            auto load_in = [&]() {
                if (!next_seg(a, k, sg)) return true;
                const uint32_t e = ns & 1, row_bytes = (uint32_t)a.H * D * 2, in = sb + OFF_IN + e * IN_BYTES;
                if (ns > 1 && !wait(in_free(e), ((ns >> 1) - 1) & 1, g, 11)) return false;
                ++ns;
                mbar_arrive_expect_tx(in_full(e), row_bytes + 2 * D * 2);
                bulk_load(in, a.q + (size_t)sg.b * a.H * D, row_bytes, in_full(e));
                bulk_load(in + kMaxH * D * 2, a.k + (size_t)sg.b * D, D * 2, in_full(e));
                bulk_load(in + kMaxH * D * 2 + D * 2, a.v + (size_t)sg.b * D, D * 2, in_full(e));
                return true;
            };
            bool ok = load_in();
            for (bool on = ns > 0; ok && on;) {
                const DecSeg here = sg;
                on = !here.last;
                for (int t = 0; ok && t < here.nt; ++t) {
                    for (int kv = 0; kv < 2; ++kv, ++L) {
                        const uint32_t s = L % kNBuf, u = L / kNBuf;
                        if (u > 0 && !(ok = wait(empty(s), (u - 1) & 1, g, 1))) break;
                        mbar_arrive_expect_tx(full(s), TILE_BYTES);
                        for (int c = 0; c < 2; ++c)
                            tma_load_2d(sb + s * TILE_BYTES + c * 16384, &map_kv, c * 128, (2 * here.b + kv) * a.w + (here.t0 + t) * kTile,
                                        full(s));
                    }
                    if (t == 0 && ok) ok = load_in();
                }
            }
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t l = L > kNBuf ? L - kNBuf : 0; l < L; ++l)
                while (!mbar_try_wait(full(l % kNBuf), (l / kNBuf) & 1) && globaltimer_ns() - t0 < a.timeout_ns) {
                }
            for (uint32_t l = ns > 2 ? ns - 2 : 0; l < ns; ++l)
                while (!mbar_try_wait(in_full(l & 1), (l >> 1) & 1) && globaltimer_ns() - t0 < a.timeout_ns) {
                }
        }
    } else if (warp == kWarpMma) {
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t id_s = idesc_fp8(kQRows, 0, 0), id_o = idesc_fp8(kWRows, 1, 1);
        // S runs one tile ahead of the weighted sum, across segments
        uint32_t is = 0, ns = 0;                                     // tiles with S issued, segments with S begun
        int ts = 0, slot_s = 0;                                      // the next S: its tile, the segment's new slot from its first
        bool ok = true, more = next_seg(a, k, sg);                   // the segments themselves: as they were prepared
        auto seg = [&](uint32_t n) { return *reinterpret_cast<const DecSeg*>(smem + OFF_SEG + (n & 1) * 32); };
        // segment n's new key's (half 0) or value's (1) codes over row `slot` of the tile in buffer s
        auto put_new = [&](uint32_t n, uint32_t s, int slot, int half) {
            if (lane < 16) {
                const uint4 c = *reinterpret_cast<const uint4*>(smem + OFF_STG + (n & 1) * STG_BYTES + half * D + lane * 16);
                *reinterpret_cast<uint4*>(smem + s * TILE_BYTES + (lane >> 3) * 16384 + slot * 128 + (((lane & 7) ^ (slot & 7)) << 4)) = c;
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        auto issue_s = [&]() {
            if (ts == 0) {
                if (!wait_w(q_ready(ns & 1), (ns >> 1) & 1, g, 10)) return false;
                sg = seg(ns);
                slot_s = sg.slot - sg.t0 * kTile;
            }
            const uint32_t l = 2 * is, s = l % kNBuf, buf = is & 1, e = ns & 1;
            if (!wait_w(full(s), (l / kNBuf) & 1, g, 2)) return false;
            if (slot_s >= ts * kTile && slot_s < (ts + 1) * kTile) put_new(ns, s, slot_s - ts * kTile, 0);
            tc_fence_after();
            const bool last = ts + 1 == sg.nt;
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks)
                    mma_fp8(tm + TM_S + buf * 64, desc_k_sw128(sb + s * TILE_BYTES + (ks >> 2) * 16384 + (ks & 3) * 32),
                             desc_k_sw128(sb + OFF_Q + e * Q_BYTES + (ks >> 2) * (Q_BYTES / 2) + (ks & 3) * 32), id_s, ks > 0 ? 1u : 0u);
                mma_commit(s_full(buf));
                mma_commit(empty(s));
                if (last) mma_commit(q_free(e));
            }
            __syncwarp();
            ++is;
            ++ts;
            if (last) {
                ts = 0;
                ++ns;
                more = !sg.last;
            }
            return true;
        };
        uint32_t i = 0, np = 0;
        bool on = more;
        if (more) ok = issue_s();
        for (; ok && on; ++np) {
            const DecSeg sp = seg(np);
            on = !sp.last;
            const int slot = sp.slot - sp.t0 * kTile;       // the new slot, from the segment's first
            for (int t = 0; t < sp.nt; ++t, ++i) {
                if (more && !(ok = issue_s())) break;
                const uint32_t l = 2 * i + 1, s = l % kNBuf, buf = i & 1;
                if (t == 0 && np > 0 && !(ok = wait_w(o_free, (np - 1) & 1, g, 3))) break;
                if (!(ok = wait_w(full(s), (l / kNBuf) & 1, w_full(buf), (i >> 1) & 1, g, 4))) break;
                if (slot >= t * kTile && slot < (t + 1) * kTile) put_new(np, s, slot - t * kTile, 1);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)                   // columns [128 hh, 128 hh + 128)
#pragma unroll
                        for (int ks = 0; ks < kTile / 32; ++ks)
                            mma_fp8(tm + TM_O + hh * 64, desc_mn_sw128(sb + s * TILE_BYTES + hh * 16384 + ks * 4096, 16384),
                                     desc_k_sw128(sb + OFF_W + buf * W_BYTES + ks * 32), id_o, (t > 0 || ks > 0) ? 1u : 0u);
                    mma_commit(o_done(buf));
                    mma_commit(empty(s));
                }
                __syncwarp();
            }
        }
        if (elect_one()) mma_commit(mma_done);
        __syncwarp();
        if (lane == 0) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(mma_done, 0) && globaltimer_ns() - t0 < a.timeout_ns) {
            }
        }
        __syncwarp();
    } else if (warp > kWarpMma) {
        // the segments after the first, while the one before is worked on: n overwrites the queries, scales and new slot
        // of n - 2, whose S is done (q_free) and whose softmax is (o_free)
        auto prep_or = [&](bool v) { return named_or(v, 6, 32 * kPrepWarps); };
        bool some = next_seg(a, k, sg);
        for (uint32_t n = 1; some && (some = next_seg(a, k, sg)); ++n) {
            bool ok = n < 2 || wait_w(q_free(n & 1), ((n >> 1) - 1) & 1, g, 13);
            ok = ok && (n < 2 || wait_w(o_free, (n - 2) & 1, g, 14));
            if (prep_or(!ok) || !prepare(sg, n, warp - kWarpMma - 1, std::integral_constant<int, kPrepWarps>{}, smem + OFF_CS + CS_BYTES, prep_or)) break;
        }
    } else {
        const int grp = warp >> 2, r = threadIdx.x & 127;            // group; slot of a tile, then column
        const int nh = (a.H + kGroups - 1 - grp) / kGroups;          // this group's heads: kGroups i + grp, i < nh
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + grp * kHg;
        float* red = reinterpret_cast<float*>(smem + OFF_RED + grp * RED_BYTES);
        auto grp_or = [&](bool v) { return named_or(v, 1 + grp, 128); };     // over the group's threads
        float *sums = red + 8 * kHg, *maxima = red + 12 * kHg, *maxima_u = red + 13 * kHg;
        // a segment's output, its last tile number `last`: the row's, or a part of it
        auto finish = [&](uint32_t n, uint32_t last) {
            const DecSeg x = *reinterpret_cast<const DecSeg*>(smem + OFF_SEG + (n & 1) * 32);
            if (grp_or(!wait_w(o_done(last & 1), (last >> 1) & 1, g, 9))) return false;
            tc_fence_after();
            float o[2][kHg], l[kHg];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float y1[kHg], y2[kHg];
                tmem_ld4(tl + TM_O + hh * 64, o[hh]);
                tmem_ld4(tl + TM_O + hh * 64 + 16, y1);
                tmem_ld4(tl + TM_O + hh * 64 + 32, y2);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < kHg; ++h) {          // times 2^(n - m) / alpha, in two steps: it may be past fp32's ends
                    const float e = ex2_approx(0.5f * (maxima_u[h] - maxima[h] - kLog2Alpha));
                    o[hh][h] = fmaf(y2[h], 1.0f / 64.0f, fmaf(y1[h], 1.0f / 8.0f, o[hh][h])) * e * e;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
#pragma unroll
            for (int h = 0; h < kHg; ++h) l[h] = (sums[h] + sums[kHg + h]) + (sums[2 * kHg + h] + sums[3 * kHg + h]);
            if (x.t0 == 0 && r == 0 && grp == 0) a.meta[x.b] = make_int2(x.c0, x.c1);
            if (x.c0 == x.c1) {
#pragma unroll
                for (int h = 0; h < kHg; ++h)
                    if (h < nh) {
                        const float inv = 1.0f / l[h];
                        __nv_bfloat16* row = a.out + ((size_t)x.b * a.H + kGroups * h + grp) * D + r;
                        row[0] = __float2bfloat16_rn(o[0][h] * inv);
                        row[128] = __float2bfloat16_rn(o[1][h] * inv);
                    }
                grp_or(false);                            // red is read before the next use
                return true;
            }
            const int pitch = part_pitch(a.H);
            float* part = a.part + (size_t)(blockIdx.x + x.b) * pitch;
#pragma unroll
            for (int h = 0; h < kHg; ++h)
                if (h < nh) {
                    part[2 * kMaxH + (kGroups * h + grp) * D + r] = o[0][h];
                    part[2 * kMaxH + (kGroups * h + grp) * D + 128 + r] = o[1][h];
                    if (r == 0) {
                        part[grp * kHg + h] = maxima[h];
                        part[kMaxH + grp * kHg + h] = l[h];
                    }
                }
            grp_or(false);                                // sums and maxima are read before the next use
            return true;
        };
        uint32_t gt = 0;
        bool ok = true, stop = true;
        uint32_t ns = 0;
        if (next_seg(a, k, sg)) {                                    // the first segment is prepared by all of these warps
            auto soft_or = [&](bool v) { return named_or(v, 5, kSoft); };
            stop = !prepare(sg, 0, warp, std::integral_constant<int, kSoftWarps>{}, smem + OFF_CS, soft_or);
        }
        for (bool last = false; !stop && !last; ++ns) {
            if (grp_or(!wait_w(q_ready(ns & 1), (ns >> 1) & 1, g, 12))) {
                stop = true;
                break;
            }
            const DecSeg sg = *reinterpret_cast<const DecSeg*>(smem + OFF_SEG + (ns & 1) * 32);
            last = sg.last;
            const float *sk = a.scales + (size_t)sg.b * 2 * a.w, *sv = sk + a.w;
            const float* qs = reinterpret_cast<const float*>(smem + OFF_QS + (ns & 1) * 64) + grp * kHg;
            const float* fresh = reinterpret_cast<const float*>(smem + OFF_STG + (ns & 1) * STG_BYTES + 2 * D);
            float m[kHg], mu[kHg], l[kHg];
#pragma unroll
            for (int h = 0; h < kHg; ++h) {
                m[h] = -INFINITY;
                mu[h] = kNoU;
                l[h] = 0.f;
            }
            int x = sg.t0 * kTile + r;
            const float2 sc0 = reinterpret_cast<const float2*>(smem + OFF_SC)[(ns & 1) * kTile + r];
            float k_next = sc0.x, v_next = sc0.y;
#pragma unroll 1
            for (int t = 0; !stop && t < sg.nt; ++t) {
                const uint32_t i = gt + t, buf = i & 1;
                const bool valid = x < sg.n;
                const bool is_new = x == sg.slot;            // the ring's own scale of it may be read before it is written
                const float ks = (is_new ? fresh[0] : k_next) * a.scale_log2, vs = is_new ? fresh[1] : v_next;
                x += kTile;                               // the next tile's scales while this one is worked on
                k_next = x < sg.n ? sk[x] : 0.f;
                v_next = x < sg.n ? sv[x] : 0.f;
                ok = ok && wait_w(s_full(buf), (i >> 1) & 1, g, 6);
                // a tile's last slots may be past the ring's: their codes could be NaN, weight 0 or not
                if (grp == 0 && sg.n - (sg.t0 + t) * kTile < kTile) {
                    const uint32_t lv = 2 * i + 1;
                    ok = ok && wait_w(full(lv % kNBuf), (lv / kNBuf) & 1, g, 7);
                    if (ok && !valid)
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            *reinterpret_cast<uint4*>(smem + (lv % kNBuf) * TILE_BYTES + (c >> 3) * 16384 + r * 128 + (c & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                }
                tc_fence_after();
                float s[kHg];
                const float lv = __log2f(vs);            // a scale that is not finite: u is not
                bool move = false;
                {
                    float s1[kHg], s2[kHg];
                    tmem_ld4(tl + TM_S + buf * 64, s);
                    tmem_ld4(tl + TM_S + buf * 64 + 16, s1);
                    tmem_ld4(tl + TM_S + buf * 64 + 32, s2);
                    tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < kHg; ++h) {
                        const float d = fmaf(s2[h], 1.0f / 256.0f, fmaf(s1[h], 1.0f / 16.0f, s[h]));
                        s[h] = valid && h < nh ? d * (qs[h] * ks) : -INFINITY;
                        move |= s[h] > m[h] + 3.0f || s[h] + lv > mu[h] + 3.0f;
                    }
                }
                if (grp_or(move || !ok)) {
                    // the new reference values from the 4 warps' maxima; O and the sums follow
#pragma unroll
                    for (int h = 0; h < kHg; ++h) {
                        const float v = warp_max(s[h]), u = warp_max(s[h] + lv);
                        if (lane == 0) {
                            red[(warp & 3) * kHg + h] = v;
                            red[(4 + (warp & 3)) * kHg + h] = u;
                        }
                    }
                    if (grp_or(!ok)) {
                        stop = true;
                        break;
                    }
                    float f[kHg];
                    bool any = false;
#pragma unroll
                    for (int h = 0; h < kHg; ++h) {
                        const float mx = fmaxf(fmaxf(red[h], red[kHg + h]), fmaxf(red[2 * kHg + h], red[3 * kHg + h]));
                        if (mx > m[h] + 3.0f) {
                            l[h] *= m[h] == -INFINITY ? 1.0f : ex2_approx(m[h] - mx);
                            m[h] = mx;
                        }
                        const float ux = fmaxf(fmaxf(red[4 * kHg + h], red[5 * kHg + h]), fmaxf(red[6 * kHg + h], red[7 * kHg + h]));
                        f[h] = 1.0f;
                        if (ux > mu[h] + 3.0f) {
                            f[h] = ex2_approx(mu[h] - ux);
                            mu[h] = ux;
                            any = true;
                        }
                    }
                    if (t > 0 && any) {
                        ok = wait_w(o_done((i - 1) & 1), ((i - 1) >> 1) & 1, g, 8);
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < 2 * kWParts; ++c) {
                            const uint32_t col = tl + TM_O + (c / kWParts) * 64 + (c % kWParts) * 16;
                            float o[kHg];
                            tmem_ld4(col, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int h = 0; h < kHg; ++h) o[h] *= f[h];
                            tmem_st4f(col, o);
                        }
                        tmem_wait_st();
                    }
                    grp_or(false);                        // red is read before the next use
                }
                // weights: row part * 16 + head row, byte = slot, in 128-byte rows swizzled by the row
                uint8_t* wb = smem + OFF_W + buf * W_BYTES + grp * (kHg * kTile) + (r & 15);
                const uint32_t ch = (uint32_t)(r >> 4) ^ (uint32_t)(grp * kHg & 7);   // swizzled by the row, grp * kHg + h
#pragma unroll
                for (int h = 0; h < kHg; h += 2) {
                    uint32_t c[kWParts] = {};
                    if (h < nh) {
                        const bool two = valid && h + 1 < nh;
                        l[h] += valid ? ex2_approx(s[h] - m[h]) : 0.f;
                        l[h + 1] += two ? ex2_approx(s[h + 1] - m[h + 1]) : 0.f;
                        float w0 = valid ? ex2_approx(s[h] + lv - (mu[h] - kLog2Alpha)) : 0.f;
                        float w1 = two ? ex2_approx(s[h + 1] + lv - (mu[h + 1] - kLog2Alpha)) : 0.f;
#pragma unroll
                        for (int part = 0; part < kWParts; ++part) {
                            c[part] = e5m2x2(w0, w1);
                            const float2 y = e5m2x2_values(c[part]);
                            w0 = (w0 - y.x) * 8.0f;
                            w1 = (w1 - y.y) * 8.0f;
                        }
                    }
#pragma unroll
                    for (int part = 0; part < kWParts; ++part) {
                        wb[part * (kMaxH * kTile) + h * 128 + ((ch ^ h) << 4)] = (uint8_t)c[part];
                        wb[part * (kMaxH * kTile) + (h + 1) * 128 + ((ch ^ (h + 1)) << 4)] = (uint8_t)(c[part] >> 8);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(w_full(buf));
                // the segment before, under this one's first products
                if (t == 0 && ns > 0 && !finish(ns - 1, gt - 1)) stop = true;
            }
            if (stop) break;
            gt += sg.nt;
            // sums over the slots: lanes, then (in finish) warps
#pragma unroll
            for (int h = 0; h < kHg; ++h) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
                if (lane == 0) sums[(warp & 3) * kHg + h] = l[h];
                if (r == 0) {
                    maxima[h] = m[h];
                    maxima_u[h] = mu[h];
                }
            }
        }
        if (!stop) finish(ns - 1, gt - 1);
        tmem_wait_ld();
        tmem_wait_st();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// The rows of several segments from their parts, in order: block = (kHeads heads, row), thread = 4 columns, kLoads parts
// in flight.  A row without a token is zero.  Bound by latency (two dependent loads, then the parts of a row together).
// <1, 8> while there are fewer rows than CTAs, so that a row may have many parts (one ring of 2048: 16, two rounds of
// loads).  Else <2, 4>: most rows have one to three parts, and the blocks, half as many, are resident together (in a
// graph, 256 rings of 2048: a step of 55.0 us instead of 55.6; 592 rings of 896, every row in one piece: 57.2
// instead of 59.6, now 56.1).
template <int kHeads, int kLoads>
__global__ void __launch_bounds__(kHeads * D / 4, kHeads == 1 ? 12 : 9)
mqa_decode8_merge_kernel(int H, const int* pos, const int2* meta, const float* part, __nv_bfloat16* out) {
    pdl_launch();
    pdl_wait();
    const int h = blockIdx.x * kHeads + threadIdx.x / (D / 4), b = blockIdx.y, t = threadIdx.x % (D / 4);
    const int pitch = part_pitch(H);
    if (h >= H) return;
    uint2* row = reinterpret_cast<uint2*>(out + ((size_t)b * H + h) * D) + t;
    const int p = pos[b];
    // Not written for a row without a token.  Kept inside the parts, for a pos that was changed under way (a caller's
    // missing dependency between streams): its output is then any, but nothing else is touched.
    const int2 m2 = meta[b], c = make_int2(min(max(m2.x, 0), kMaxCtas - 1), min(max(m2.y, 0), kMaxCtas - 1));
    if (p < 0) {
        *row = make_uint2(0, 0);
        return;
    }
    if (c.x == c.y) return;
    const float* p0 = part + (size_t)(c.x + b) * pitch;
    const int np = c.y - c.x + 1;
    float mx = -INFINITY, l = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c0 = 0; c0 < np; c0 += kLoads) {
        float m[kLoads], s[kLoads];
        float4 z[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            m[i] = -INFINITY;
            if (c0 + i < np) {
                const float* pc = p0 + (size_t)(c0 + i) * pitch;
                m[i] = pc[head_row(h)];
                s[i] = pc[kMaxH + head_row(h)];
                z[i] = reinterpret_cast<const float4*>(pc + 2 * kMaxH + h * D)[t];
            }
        }
        float mn = mx;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) mn = fmaxf(mn, m[i]);
        const float old = mx == -INFINITY ? 0.f : ex2_approx(mx - mn);
        l *= old;
        y = make_float4(y.x * old, y.y * old, y.z * old, y.w * old);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (c0 + i < np) {
                const float f = ex2_approx(m[i] - mn);
                l = fmaf(s[i], f, l);
                y = make_float4(fmaf(z[i].x, f, y.x), fmaf(z[i].y, f, y.y), fmaf(z[i].z, f, y.z), fmaf(z[i].w, f, y.w));
            }
        mx = mn;
    }
    const float inv = 1.0f / l;
    *row = make_uint2(bf16x2(y.x * inv, y.y * inv), bf16x2(y.z * inv, y.w * inv));
}

struct DecLayout {
    size_t meta, part, total;
};
inline DecLayout dec_layout(const rglru_mqa_dims* d) {
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    const size_t B = (size_t)d->batch;
    DecLayout l{};
    size_t o = 256;                    // the status word
    l.meta = o; o = up(o + B * sizeof(int2));
    l.part = o; o = up(o + (B + kMaxCtas) * part_pitch(d->q_heads) * 4);
    l.total = o;
    return l;
}

}  // namespace c8

size_t mqa_decode8_workspace(const rglru_mqa_dims* d) { return c8::dec_layout(d).total; }

cudaError_t launch_mqa_cache8_write(const rglru_mqa_dims* d, const void* k, const void* v, const int* lengths, int pos0,
                                    void* codes, float* scales, cudaStream_t s) {
    using namespace c8;
    // without lengths only the last min(T, w) tokens are written; with them any token may be
    const int tokens = lengths ? d->seq_len : std::min(d->seq_len, d->window);
    mqa_cache8_write_kernel<<<dim3(tokens, (d->batch + kWriteRows - 1) / kWriteRows), 32 * kWriteRows, 0, s>>>(
        d->batch, d->seq_len, d->window, pos0, rope_base(d->rope_base), lengths, static_cast<const __nv_bfloat16*>(k),
        static_cast<const __nv_bfloat16*>(v), static_cast<uint8_t*>(codes), scales);
    return cudaGetLastError();
}

cudaError_t launch_mqa_decode8(const rglru_mqa_dims* d, const void* q, const void* k, const void* v, const int* pos,
                               void* codes, float* scales, void* out, void* ws, cudaStream_t s) {
    using namespace c8;
    const DecLayout l = dec_layout(d);
    uint8_t* p = static_cast<uint8_t*>(ws);
    const int B = d->batch, w = d->window;
    // the ring as [B 2 w slots][256 bytes] (box 128 x 128)
    CUtensorMap mkv;
    if (!tc::make_map_2d_sw128_elem(&mkv, codes, 1, D, (uint64_t)B * 2 * w, D, 128, kTile)) return cudaErrorInvalidValue;
    cudaError_t e = set_smem_once(mqa_decode8_kernel, (int)SMEM_BYTES);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    DecArgs a{};
    a.B = B; a.H = d->q_heads; a.w = w;
    a.scale_log2 = d->scale * 1.4426950408889634f;
    a.pos = pos;
    a.base = rope_base(d->rope_base);
    a.q = static_cast<const __nv_bfloat16*>(q); a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = scales;
    a.meta = reinterpret_cast<int2*>(p + l.meta);
    a.part = reinterpret_cast<float*>(p + l.part);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.status = static_cast<DeviceStatus*>(ws);
    a.timeout_ns = 1000000000ull;
    // both launched behind the kernel before them on the stream, their set-up under that kernel's end
    const long long tiles = (long long)B * ((w + kTile - 1) / kTile);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int ctas = (int)std::min<long long>(tiles, std::min(sms, kMaxCtas));
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, mqa_decode8_kernel, mkv, a)) != cudaSuccess) return e;
    cfg.dynamicSmemBytes = 0;
    auto merge = [&](auto kern, int heads) {
        cfg.gridDim = dim3((d->q_heads + heads - 1) / heads, B);
        cfg.blockDim = dim3(heads * D / 4);
        return cudaLaunchKernelEx(&cfg, kern, d->q_heads, pos, static_cast<const int2*>(a.meta), static_cast<const float*>(a.part),
                                  a.out);
    };
    return B < ctas ? merge(mqa_decode8_merge_kernel<1, 8>, 1) : merge(mqa_decode8_merge_kernel<2, 4>, 2);
}

cudaError_t launch_mqa_cache8_read(const rglru_mqa_dims* d, const void* codes, const float* scales, const int* pos,
                                   void* cache, cudaStream_t s) {
    using namespace c8;
    const long long slots = 2LL * d->batch * d->window;
    mqa_cache8_read_kernel<<<(unsigned)((slots + kReadBlock - 1) / kReadBlock), 256, 0, s>>>(slots, d->window, pos,
                                                                       static_cast<const uint8_t*>(codes), scales,
                                                                       static_cast<__nv_bfloat16*>(cache));
    return cudaGetLastError();
}

}  // namespace rglru
