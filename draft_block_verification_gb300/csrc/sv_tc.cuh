// sv_tc.cuh -- what the attention kernels share: wrappers of the tensor-core
// instructions (tcgen05), waits that end when another role of the CTA has given
// up, spans of work for the CTAs of one wave, and the cache's tensor maps.
#pragma once

#include <cuda.h>

#include "sv_common.cuh"

namespace sv {

constexpr uint32_t kAtSpin = 1u << 20; // tries of a wait (a tile takes microseconds)

// Quotient of non-negative numbers; 64-bit division costs thousands of cycles.
__device__ __forceinline__ long long div_pos(long long a, long long b)
{
    if (((unsigned long long)(a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// Span of CTA i of `ctas` over `total` tiles, and the CTA that owns a tile.
__device__ __forceinline__ long long span_at(long long total, int ctas, int i)
{
    return div_pos(total * i, ctas);
}
__device__ __forceinline__ int span_owner(long long total, int ctas, long long x)
{
    int i = (int)div_pos(x * ctas, total);
    while (i + 1 < ctas && span_at(total, ctas, i + 1) <= x) ++i;
    while (i > 0 && span_at(total, ctas, i) > x) --i;
    return i;
}

// Product of packed fp32 pairs.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
        " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// ---------------------------------------------------------------------------
// tcgen05 wrappers.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_ld8(uint32_t addr, float *v)
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const float *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                     addr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
                 "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
                 "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}
__device__ __forceinline__ void tc_ld4(uint32_t addr, float *v)
{
    uint32_t r[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
// The registers of the loads before it may be read after it: they pass through.
template <int N>
__device__ __forceinline__ void tc_wait_ld(float (&v)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tc_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory operand descriptors.  layout: 2 = 128-byte swizzle, 4 = 64-byte.
// Operands whose products' dimension is contiguous: stride = 8 rows.  Operands
// whose rows (tokens) are the products' dimension: stride = 8 tokens, lead =
// the next 128 (64) bytes of the other dimension.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lead, uint32_t stride,
                                            uint32_t layout)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)((lead >> 4) & 0x3FFF) << 16) |
           ((uint64_t)((stride >> 4) & 0x3FFF) << 32) | (1ull << 46) | ((uint64_t)layout << 61);
}

__device__ __forceinline__ void fence_async()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Whether one of four e4m3 bytes is NaN (all magnitude bits set).
__device__ __forceinline__ bool has_nan(uint32_t w)
{
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Barrier over `n` threads with an or over a flag.
__device__ __forceinline__ bool bar_or(int id, int n, bool flag)
{
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
        " barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"((uint32_t)flag), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

// Bounded wait that also ends when another role has given up.  (The roles'
// loops share the instruction caches: what is rarely run is marked so, to lie
// outside them.)
__device__ __forceinline__ bool at_wait_on(int *abort, int *err, uint64_t *bar,
                                           uint32_t parity)
{
    for (uint32_t i = 0; i < kAtSpin; ++i) {
        if (mbar_try(bar, parity)) return true;
        if ((i & 63) == 63) {
            if (*(volatile int *)abort) return false;
            __nanosleep(64);
        }
    }
    *(volatile int *)abort = 1;
    latch(err, SV_ERR_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool at_wait(int *abort, int *err, uint64_t *bar, uint32_t parity)
{
    if (__builtin_expect(mbar_try(bar, parity), 1)) return true;
    return at_wait_on(abort, err, bar, parity);
}

// Map of one side of the cache: [pages * H][block][D] bytes, `rows` rows of a
// page's head at a time, in the swizzle that the products read.
bool cache_map(CUtensorMap *m, const uint8_t *cache, int D, int block, int rows, int pages, int H);

}  // namespace sv
