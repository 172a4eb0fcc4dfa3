// sv_kvread.cu -- tokens read back from the paged 8-bit cache:
//   out[cu_b + i, h, :] = e4m3(byte) * scale[page, h]
// for position first_b + i of sequence b, keys and values alike, in fp32 or
// rounded once to bf16 (exactly, where the scale is a power of two).
//
// Bound by DRAM: a byte in, two or four out, nothing is read twice.  A thread
// takes the bytes that make 16 bytes of output, so that both the loads and the
// stores of a warp are whole lines; it has the keys' and the values' loads of
// kAhead items in flight.  A CTA takes a run of rows and looks up where they
// lie once, a thread for each row.  506 MB of reads and writes (82,000 tokens of
// 8 x 128 to bf16) take 81 us, 93 % of the rate of a copy (131,072 tokens 112 us as a
// graph; with scales that need odd_product a fifth more); 17 tokens, as a graph, 2.1 us.
#include "sv_common.cuh"
#include "sv_kv.cuh"

namespace sv {

constexpr int kReadThreads = 256;
constexpr int kReadRows = 16;
constexpr int kAhead = 4;

__device__ __forceinline__ float2 e4m3_pair(uint32_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// A value times its scale, to be rounded to bf16.  Up to 4 times 24 bits: rounded to fp32
// before, as it is where the scale has all of its bits, a product beside the middle of two
// steps would fall into it.  So it is rounded to odd there: cut off, and the last bit set
// where something was.
__device__ __forceinline__ bool whole_products(float scale)
{
    return (__float_as_uint(scale) & 15u) == 0;
}
__device__ __forceinline__ float odd_product(float v, float scale)
{
    const float p = __fmul_rz(v, scale);
    return __uint_as_float(__float_as_uint(p) | (fmaf(v, scale, -p) != 0.f ? 1u : 0u));
}

template <bool F32>
__device__ __forceinline__ void put(char *dst, uint2 raw, float scale)
{
    const float2 a = e4m3_pair(raw.x & 0xFFFFu), b = e4m3_pair(raw.x >> 16);
    if (F32) {
        __stcs(reinterpret_cast<float4 *>(dst),
               make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale));
    } else {
        const float2 c = e4m3_pair(raw.y & 0xFFFFu), d = e4m3_pair(raw.y >> 16);
        auto two = [](float x, float y) {
            uint32_t r;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
            return r;
        };
        uint4 o;
        if (__builtin_expect(whole_products(scale), 1)) {
            o = make_uint4(two(a.x * scale, a.y * scale), two(b.x * scale, b.y * scale),
                           two(c.x * scale, c.y * scale), two(d.x * scale, d.y * scale));
        } else {
            auto odd = [&](float2 v) { return two(odd_product(v.x, scale), odd_product(v.y, scale)); };
            o = make_uint4(odd(a), odd(b), odd(c), odd(d));
        }
        __stcs(reinterpret_cast<uint4 *>(dst), o);
    }
}

// VEC: output rows start on 16 bytes.  (Else elements are stored one by one: 131,072
// tokens of 8 x 128 to bf16 take 568 us, with VEC 112.)
template <bool F32, bool VEC>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadJob j, int rows)
{
    constexpr int kElems = F32 ? 4 : 8;           // of an item
    __shared__ int64_t s_row[kReadRows];          // page * H * block + row in it, or -1
    __shared__ int s_page[kReadRows];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * rows;
    pdl_wait();
    pdl_trigger();
    if (tid < rows) {
        const int64_t t = t0 + tid;
        int64_t row = -1;
        int page = 0;
        if (t < j.T && t < j.cu[j.B]) {
            int lo = 0, hi = j.B;                 // the last b with cu[b] <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (j.cu[mid] <= t) lo = mid; else hi = mid;
            }
            const int64_t i = t - j.cu[lo], f = j.first ? j.first[lo] : 0, p = f + i;
            const int shift = 31 - __clz(j.block);
            bool ok = i >= 0 && t < j.cu[lo + 1] && f >= 0 && (p >> shift) < j.cols;
            if (ok) {
                page = j.table[(int64_t)lo * j.cols + (p >> shift)];
                ok = page >= 0 && page < j.pages;
            }
            if (ok)
                row = (int64_t)page * j.H * j.block + (p & (j.block - 1));
            else
                latch(j.err, SV_ERR_DEVICE_BOUNDS);
        }
        s_row[tid] = row;
        s_page[tid] = page;
    }
    __syncthreads();
    const int per = j.D / kElems, items = rows * j.H * per;
    const int shift = 31 - __clz(per);
    for (int base = tid; base < items; base += kReadThreads * kAhead) {
        uint2 raw[kAhead][2];
        float sc[kAhead][2];
        int r[kAhead], h[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = base + k * kReadThreads;
            const int e = (i & (per - 1)) * kElems, rh = i >> shift;
            r[k] = -1;
            if (i < items) {
                const int rr = rh / j.H;
                h[k] = rh - rr * j.H;
                if (s_row[rr] >= 0) {
                    r[k] = rr;
                    const int64_t at = (s_row[rr] + (int64_t)h[k] * j.block) * j.D + e;
                    const int64_t ph = (int64_t)s_page[rr] * j.H + h[k];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        if (F32)
                            raw[k][n].x = __ldcs(reinterpret_cast<const uint32_t *>(j.cache[n] + at));
                        else
                            raw[k][n] = __ldcs(reinterpret_cast<const uint2 *>(j.cache[n] + at));
                        sc[k][n] = __ldg(j.scale[n] + ph);
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (r[k] < 0) continue;
            const int e = ((base + k * kReadThreads) & (per - 1)) * kElems;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                char *dst = j.dst[n] + (t0 + r[k]) * j.ts[n] + (int64_t)h[k] * j.hs[n] +
                            e * (F32 ? 4 : 2);
                if (VEC) {
                    put<F32>(dst, raw[k][n], sc[k][n]);
                } else {
#pragma unroll
                    for (int q = 0; q < kElems; ++q) {
                        const uint32_t b = ((q < 4 ? raw[k][n].x : raw[k][n].y) >> (8 * (q & 3))) & 255;
                        const float a = e4m3_pair(b).x, s = sc[k][n];
                        if (F32)
                            reinterpret_cast<float *>(dst)[q] = a * s;
                        else
                            reinterpret_cast<uint16_t *>(dst)[q] = __bfloat16_as_ushort(
                                __float2bfloat16_rn(whole_products(s) ? a * s : odd_product(a, s)));
                    }
                }
            }
        }
    }
}

cudaError_t read_launch(const ReadJob &j, int sms, cudaStream_t s)
{
    // fewer rows a CTA where that leaves SMs without one (17 tokens of 8 x 128: 2.0 us, by
    // 16 rows 4.0; 1,088: 3.5 and 4.9)
    int rows = kReadRows;
    while (rows > 1 && (int64_t)j.T < (int64_t)rows * sms * 2) rows /= 2;
    bool vec = true;
    for (int i = 0; i < 2; ++i)
        vec = vec && ((uintptr_t)j.dst[i] | (uintptr_t)j.ts[i] | (uintptr_t)j.hs[i]) % 16 == 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    pdl_config(cfg, at, dim3((unsigned)(((int64_t)j.T + rows - 1) / rows)), dim3(kReadThreads), 0, s);
    if (j.dtype == SV_F32)
        return vec ? cudaLaunchKernelEx(&cfg, read_kernel<true, true>, j, rows)
                   : cudaLaunchKernelEx(&cfg, read_kernel<true, false>, j, rows);
    return vec ? cudaLaunchKernelEx(&cfg, read_kernel<false, true>, j, rows)
               : cudaLaunchKernelEx(&cfg, read_kernel<false, false>, j, rows);
}

}  // namespace sv
