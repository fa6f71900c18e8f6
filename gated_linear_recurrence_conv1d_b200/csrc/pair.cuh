// pair.cuh -- tcgen05 and TMA wrappers of a CTA pair (cta_group::2), and bounded waits on barriers of a
// cluster, for the attention kernels and the GEMM.  Rank 0 (the leader) issues the MMAs of the pair; each CTA's
// TMEM holds its own 128 of the 256 rows, each CTA's shared memory half of the B operand.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace rglru {
namespace pr {

using namespace sm100;

__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (both CTAs' TMEM) (+)= A (both CTAs' halves, shared memory) B (both CTAs' halves)^T
__device__ __forceinline__ void mma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t id,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(id), "r"(accumulate)
        : "memory");
}
// the same with A in both CTAs' TMEM
__device__ __forceinline__ void mma_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t id,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(id), "r"(accumulate)
        : "memory");
}
// arrive on the mbarrier at this shared address in both CTAs once every prior MMA of this thread completes
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// a tile into this CTA's shared memory, its bytes counted on a barrier of the pair (shared::cluster address)
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
// `bytes` (a multiple of 16, 16-byte aligned) of global memory into this CTA's shared memory
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// asynchronous copies behind this thread's view of global memory (what it has acquired of ordinary stores)
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// MN-major (128-byte swizzle) descriptor: atoms of 64 MN-elements x K rows of 128 B, `atom` bytes apart,
// 8-row K groups 1024 B apart
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t smem_addr, uint32_t atom) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
    d |= (uint64_t)(atom >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// fp32 accumulator, bf16 operands, A K-major (or TMEM), B K-major (b_mn = 0) or MN-major (1)
__device__ __forceinline__ constexpr uint32_t idesc_bf16(int m, int n, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// Arrive on a barrier of either CTA (a shared::cluster address).  What these arrivals hand over is TMEM contents
// (ordered by the tcgen05 fences around them) or a buffer whose reads are complete, so they need no fence of
// the other memories at cluster scope, which would hold the warp for hundreds of cycles.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// 16 bytes into another CTA's shared memory, counted on a barrier there
__device__ __forceinline__ void st_async_v4(uint32_t dst_cluster, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                            uint32_t bar_cluster) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     dst_cluster),
                 "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar_cluster)
                 : "memory");
}

// Programmatic dependent launch: the kernel behind this one may be launched from now on (its set-up overlaps this
// kernel); and the kernels before this one are complete and their writes visible.  Every CTA of every
// kernel of a chain waits, so that "the kernel before" stands for all of them.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Bounded waits: a wait that expires latches TIMEOUT (site, CTA) and makes every later wait of the CTA fail.
struct Guard {
    volatile int* abort;               // shared memory, one per CTA
    DeviceStatus* status;
    unsigned long long timeout_ns;
};
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, const Guard& g, unsigned where) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*g.abort) return false;
        if (it > 64) __nanosleep(100);
        if (globaltimer_ns() - t0 > g.timeout_ns) {
            latch_status(g.status, RGLRU_ERR_TIMEOUT, where, blockIdx.x, parity);
            *g.abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Guard& g, unsigned where) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, g, where);
}
// the whole warp follows one wait
__device__ __forceinline__ bool wait_w(uint32_t bar, uint32_t parity, const Guard& g, unsigned where) {
    return __all_sync(0xffffffffu, wait(bar, parity, g, where));
}
// The whole warp follows two or three waits, asked one behind the other before any answer is looked at: an answer
// takes 80 cycles and more, in which an MMA warp that asks one by one leaves the tensor pipe (whose queue is two
// MMAs deep) idle.
__device__ __forceinline__ bool wait_w(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, const Guard& g, unsigned where) {
    const bool r0 = mbar_try_wait(b0, p0), r1 = mbar_try_wait(b1, p1);
    if (__all_sync(0xffffffffu, r0 & r1)) return true;
    return __all_sync(0xffffffffu, wait(b0, p0, g, where) && wait(b1, p1, g, where + 16));
}
__device__ __forceinline__ bool wait_w(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2,
                                       const Guard& g, unsigned where) {
    const bool r0 = mbar_try_wait(b0, p0), r1 = mbar_try_wait(b1, p1), r2 = mbar_try_wait(b2, p2);
    if (__all_sync(0xffffffffu, r0 & r1 & r2)) return true;
    return __all_sync(0xffffffffu, wait(b0, p0, g, where) && wait(b1, p1, g, where + 16) && wait(b2, p2, g, where + 32));
}
// named barrier 1 over `threads` threads, returning the OR of v over them
__device__ __forceinline__ bool bar_or(bool v, int threads) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.red.or.pred p, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(threads)
        : "memory");
    return r != 0;
}

// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t as_u64(float2 v) {
    return (uint64_t)__float_as_uint(v.x) | (uint64_t)__float_as_uint(v.y) << 32;
}
__device__ __forceinline__ float2 as_float2(uint64_t v) {
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
    return as_float2(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_float2(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_float2(d);
}

// two fp32 as packed bf16 (lo in the low half), round to nearest even
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four lanes with 64 bytes of a row each (four 16-byte pieces e[4 k ..]) hand them round so that lane j has piece j of the
// four rows (row i of the quad in e[4 i ..]): a store of a warp then writes 8 rows of 64 bytes, not 32 of 16.
__device__ __forceinline__ void quad_transpose(uint32_t (&e)[16]) {
#pragma unroll
    for (int step = 1; step < 4; step *= 2) {
        const bool up = threadIdx.x & step;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & step) continue;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t &lo = e[4 * k + w], &hi = e[4 * (k + step) + w];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, step);
                if (up) lo = got; else hi = got;
            }
        }
    }
}
// 32 lanes x 32 bits, 4 consecutive columns per thread
__device__ __forceinline__ void tmem_st4f(uint32_t taddr, const float (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3])
                 : "memory");
}
// 32 lanes x 32 bits, 32 consecutive columns per thread
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

}  // namespace pr
}  // namespace rglru
