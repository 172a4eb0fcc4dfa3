// sv_kvattn.cu -- attention over the paged 8-bit cache.
//
// Token i of sequence b's new tokens (i = 0 .. n_b - 1, at position
// L_b - n_b + i of the L_b tokens in the cache) attends with query head g to
// the cache's head g / G:
//   z_p = scale * q . (k_p s^k),  w_p = exp(z_p - max z),
//   o = sum_p w_p (v_p s^v) / sum_p w_p
// over the positions it sees: those up to its own, or, with a mask, every
// position before the new tokens and the new tokens whose bit is set.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sv_common.cuh"
#include "sv_kv.cuh"

namespace sv {

__device__ __forceinline__ float e4m3_to_f32(uint8_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    return __low2float(*reinterpret_cast<__half2 *>(&h));
}

constexpr int kAttThreads = 128;

// One warp per token and query head, the head's elements over the lanes.
template <int D>
__global__ void __launch_bounds__(kAttThreads) attend_kernel(const AttendJob j)
{
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kAttThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    const int t = (int)(item / j.Hq), g = (int)(item % j.Hq);
    if (t >= j.T) return;
    int lo = 0, hi = j.B;  // the last b with cu[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (j.cu[mid] <= t) lo = mid; else hi = mid;
    }
    const int b = lo;
    const int n = j.cu[b + 1] - j.cu[b], L = j.kv_len[b], ctx = L - n, i = t - j.cu[b];
    if (i >= n || i < 0) return;
    bool bad = ctx < 0 || (long long)(L + j.block - 1) / j.block > j.cols;
    float q[N], o[N];
    for (int k = 0; k < N; ++k) {
        q[k] = __uint_as_float((uint32_t)j.q[t * j.qts + g * j.qhs + lane + 32 * k] << 16) *
               j.softmax_scale * 1.4426950408889634f;
        o[k] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int h = g / j.G;
    for (int p = 0; p < (bad ? 0 : L); ++p) {
        bool sees = p <= ctx + i;
        if (j.mask && p >= ctx) {
            const int k = p - ctx;
            sees = k < 32 * j.words && ((j.mask[(int64_t)t * j.words + (k >> 5)] >> (k & 31)) & 1);
        }
        if (!sees) continue;
        const int page = j.table[(int64_t)b * j.cols + p / j.block];
        if (page < 0 || page >= j.pages) {
            bad = true;
            break;
        }
        const int64_t ph = (int64_t)page * j.H + h;
        const int64_t at = (ph * j.block + p % j.block) * D + lane;
        float z = 0.f;
        for (int k = 0; k < N; ++k) z += q[k] * e4m3_to_f32(j.cache[0][at + 32 * k]);
        z = warp_sum(z) * j.scale[0][ph];
        const float top = fmaxf(m, z), c = ex2f(m - top), w = ex2f(z - top);
        l = l * c + w;
        m = top;
        const float vs = j.scale[1][ph] * w;
        for (int k = 0; k < N; ++k) o[k] = o[k] * c + vs * e4m3_to_f32(j.cache[1][at + 32 * k]);
    }
    if (bad && lane == 0) latch(j.err, SV_ERR_DEVICE_BOUNDS);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int k = 0; k < N; ++k)
        j.out[((int64_t)t * j.Hq + g) * D + lane + 32 * k] =
            __bfloat16_as_ushort(__float2bfloat16_rn(o[k] * inv));
    if (j.lse && lane == 0)
        j.lse[(int64_t)t * j.Hq + g] =
            l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

cudaError_t attend_launch(const AttendJob &j, int sms, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    const int64_t items = (int64_t)j.T * j.Hq;
    pdl_config(cfg, at, dim3((unsigned)((items + 3) / 4)), dim3(kAttThreads), 0, s);
    return j.D == 64 ? cudaLaunchKernelEx(&cfg, attend_kernel<64>, j)
                     : cudaLaunchKernelEx(&cfg, attend_kernel<128>, j);
}

}  // namespace sv
