// sv_rope.cu -- norms of queries and keys for each head, and the rotation by
// the token's position, in one pass.
//
// For a token at position p and a head's elements x (D of them):
//   x'_d = x_d w_d / sqrt(mean(x^2) + eps)      (where there is a weight)
//   y_a = x'_a cos t_i - x'_b sin t_i,  y_b = x'_b cos t_i + x'_a sin t_i
// with t_i = p inv_freq_i for the pairs i < rot / 2: (a, b) = (i, i + rot / 2),
// or (2i, 2i + 1) where neighbours are paired.  Elements from rot on stay x'.
// All of it in fp32, rounded once to the output's type.
//
// Angles.  What counts is the fraction of a turn: p * (inv_freq / 2 pi) mod 1.
// inv_freq / 2 pi mod 1 is held as a 64-bit fraction, taken from the float's 24
// bits times 65 bits of 1 / 2 pi, so that a 64-bit product with the position
// wraps by itself: for |inv_freq| < 2 the angle is right to 2^-32 of a turn at
// any position, where an fp32 product would be off by p 2^-25 turns.
//
// Bound by DRAM.  A head is D / 16 threads, each with two vectors of eight
// elements: the two halves of its pairs, so that the rotation needs no
// exchange.  A warp takes kGroups times as many heads of one token as fit its
// lanes (D = 128: four at a time); the loads of all are in flight before the
// first angle is computed, and its cosines and sines serve them all.
#include "sv_common.cuh"
#include "sv_kv.cuh"

namespace sv {

constexpr int kRopeWarps = 4;
constexpr int kGroups = 4;

// inv_freq / (2 pi) mod 1, in units of 2^-64.
__device__ __forceinline__ uint64_t turns(float inv_freq)
{
    const uint32_t u = __float_as_uint(inv_freq);
    const int e = (int)((u >> 23) & 255) - 127;
    const uint64_t m = (u & 0x7FFFFFu) | (e > -127 ? 0x800000u : 0u);
    // value = m 2^(e - 23); 1 / 2 pi = kInv 2^-66 (rounded down)
    constexpr uint64_t kInv = 11743562013128004905ull;  // floor(2^66 / 2 pi)
    const uint64_t lo = m * kInv, hi = __umul64hi(m, kInv);  // 88 bits
    const int down = 25 - max(e, -126);           // m kInv 2^-down, mod 2^64
    uint64_t f;
    if (down <= 0)
        f = down > -64 ? lo << -down : 0;
    else if (down < 64)
        f = lo >> down | hi << (64 - down);
    else
        f = down < 128 ? hi >> (down - 64) : 0;
    return u >> 31 ? 0 - f : f;
}

// Cosine and sine of position times inv_freq.
__device__ __forceinline__ float2 turn(float inv_freq, int pos)
{
    const uint64_t f = turns(inv_freq) * (uint64_t)(uint32_t)pos;
    float t = (float)(int64_t)f * 0x1p-63f;       // half turns, [-1, 1]
    if (!(fabsf(inv_freq) < INFINITY)) t = __int_as_float(0x7FC00000);
    float2 cs;
    sincospif(t, &cs.y, &cs.x);
    return cs;
}

template <typename T>
__device__ __forceinline__ float load_one(const char *p);
template <>
__device__ __forceinline__ float load_one<uint16_t>(const char *p)
{
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16);
}
template <>
__device__ __forceinline__ float load_one<float>(const char *p)
{
    return *reinterpret_cast<const float *>(p);
}
__device__ __forceinline__ void store_one(uint16_t *p, float v)
{
    *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }

// Eight elements on a 16-byte boundary.
template <typename In>
struct Octet;
template <>
struct Octet<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void load(const char *p)
    {
        v = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void get(float *f) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Octet<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const char *p)
    {
        a = *reinterpret_cast<const float4 *>(p);
        b = *(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float *f) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(uint16_t *p, const float *f)
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]),
                                               bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float *p, const float *f)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Heads in vectors.  PER: threads of a head, the least power of two that is
// D / 16 or more.  A warp: one token, heads from `part` * kGroups * (32 / PER).
template <typename In, typename Out, int PER, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const RopeJob j, int parts)
{
    constexpr int kHeads = 32 / PER;              // at a time
    __shared__ float s_cos[kRopeWarps][PER * 8], s_sin[kRopeWarps][PER * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t tok = unit / parts;
    if (tok >= j.T) return;                       // (warps do not meet below)
    const int h0 = (int)(unit - tok * parts) * (kGroups * kHeads) + lane / PER;
    const int l = lane % PER, half = j.rot >> 4;  // vectors of half the rotated elements
    const int pos = j.pos[tok];
    if (pos < 0) return;
    const bool live = l < (j.D >> 4);
    // where this thread's two vectors start
    int e0, e1;
    if (INTER) {
        e0 = l * 16;
        e1 = e0 + 8;
    } else if (l < half) {
        e0 = l * 8;
        e1 = e0 + (j.rot >> 1);
    } else {
        e0 = j.rot + (l - half) * 16;
        e1 = e0 + 8;
    }
    Octet<In> raw[kGroups][2];
    int head[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int h = h0 + g * kHeads;
        head[g] = live && h < j.Hq + j.H ? h : -1;
        if (head[g] >= 0) {
            const bool key = h >= j.Hq;
            const char *src = key ? j.src[1] + tok * j.ts[1] + (int64_t)(h - j.Hq) * j.hs[1]
                                  : j.src[0] + tok * j.ts[0] + (int64_t)h * j.hs[0];
            raw[g][0].load(src + e0 * (int)sizeof(In));
            raw[g][1].load(src + e1 * (int)sizeof(In));
        }
    }
    for (int i = lane; i < (j.rot >> 1); i += 32) {
        const float2 cs = turn(j.inv_freq[i], pos);
        s_cos[warp][i] = cs.x;
        s_sin[warp][i] = cs.y;
    }
    __syncwarp();
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = l * 8 + i;
        const bool on = k < (j.rot >> 1);
        c[i] = on ? s_cos[warp][k] : 1.f;
        s[i] = on ? s_sin[warp][k] : 0.f;
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int h = head[g];
        const bool key = h >= j.Hq;
        float x[16];
        if (h >= 0) {
            raw[g][0].get(x);
            raw[g][1].get(x + 8);
        }
        const float *w = key ? j.weight[1] : j.weight[0];
        float sum = 0.f;
        if (h >= 0 && w) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
        }
#pragma unroll
        for (int k = PER / 2; k > 0; k >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
        if (h < 0) continue;
        if (w) {
            const float r = rsqrtf(sum / (float)j.D + j.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] *= r * __ldg(w + e0 + i);
                x[8 + i] *= r * __ldg(w + e1 + i);
            }
        }
        float y[16];
        if (INTER) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
                y[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * s[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] = x[i] * c[i] - x[8 + i] * s[i];
                y[8 + i] = x[8 + i] * c[i] + x[i] * s[i];
            }
        }
        Out *dst = reinterpret_cast<Out *>(
            key ? j.dst[1] + tok * j.ots[1] + (int64_t)(h - j.Hq) * j.ohs[1]
                : j.dst[0] + tok * j.ots[0] + (int64_t)h * j.ohs[0]);
        store8(dst + e0, y);
        store8(dst + e1, y + 8);
    }
}

// Any even D and rot, any alignment: a warp for each token and head, pairs of
// elements dealt to its lanes.
template <typename In, typename Out, int PAIRS, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_any_kernel(const RopeJob j)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int all = j.Hq + j.H;
    const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t tok = unit / all;
    if (tok >= j.T) return;
    const int h = (int)(unit - tok * all);
    const int pos = j.pos[tok];
    if (pos < 0) return;
    const int side = h >= j.Hq, hh = side ? h - j.Hq : h;
    const char *src = (side ? j.src[1] : j.src[0]) + tok * (side ? j.ts[1] : j.ts[0]) +
                      (int64_t)hh * (side ? j.hs[1] : j.hs[0]);
    Out *dst = reinterpret_cast<Out *>((side ? j.dst[1] : j.dst[0]) +
                                       tok * (side ? j.ots[1] : j.ots[0]) +
                                       (int64_t)hh * (side ? j.ohs[1] : j.ohs[0]));
    const float *w = side ? j.weight[1] : j.weight[0];
    const int half = j.rot >> 1;
    float a[PAIRS], b[PAIRS];
    float sum = 0.f;
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
        const int i = lane + 32 * p;
        a[p] = b[p] = 0.f;
        if (2 * i < j.D) {
            const bool near = INTER || i >= half;
            a[p] = load_one<In>(src + (int64_t)(near ? 2 * i : i) * sizeof(In));
            b[p] = load_one<In>(src + (int64_t)(near ? 2 * i + 1 : i + half) * sizeof(In));
        }
        sum = fmaf(a[p], a[p], fmaf(b[p], b[p], sum));
    }
    float r = 1.f;
    if (w) r = rsqrtf(warp_sum(sum) / (float)j.D + j.eps);
    __syncwarp();  // a head is read whole before any of it is written in its place
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
        const int i = lane + 32 * p;
        if (2 * i >= j.D) continue;
        const bool near = INTER || i >= half;
        const int ia = near ? 2 * i : i, ib = near ? 2 * i + 1 : i + half;
        const float x = w ? a[p] * (r * w[ia]) : a[p], z = w ? b[p] * (r * w[ib]) : b[p];
        const float2 cs = i < half ? turn(j.inv_freq[i], pos) : make_float2(1.f, 0.f);
        store_one(dst + ia, x * cs.x - z * cs.y);
        store_one(dst + ib, z * cs.x + x * cs.y);
    }
}

template <typename In, typename Out, bool INTER>
static cudaError_t rope_pick(const RopeJob &j, bool vec, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    int per = 1;
    while (per * 16 < j.D) per *= 2;
    if (!vec) {
        const int64_t units = (int64_t)j.T * (j.Hq + j.H);
        pdl_config(cfg, at, dim3((unsigned)((units + kRopeWarps - 1) / kRopeWarps)),
                   dim3(kRopeWarps * 32), 0, s);
        if (per <= 4) return cudaLaunchKernelEx(&cfg, rope_any_kernel<In, Out, 1, INTER>, j);
        if (per <= 8) return cudaLaunchKernelEx(&cfg, rope_any_kernel<In, Out, 2, INTER>, j);
        if (per <= 16) return cudaLaunchKernelEx(&cfg, rope_any_kernel<In, Out, 4, INTER>, j);
        return cudaLaunchKernelEx(&cfg, rope_any_kernel<In, Out, 8, INTER>, j);
    }
    const int heads = kGroups * (32 / per), parts = (j.Hq + j.H + heads - 1) / heads;
    const int64_t units = (int64_t)j.T * parts;
    pdl_config(cfg, at, dim3((unsigned)((units + kRopeWarps - 1) / kRopeWarps)),
               dim3(kRopeWarps * 32), 0, s);
    switch (per) {
        case 4: return cudaLaunchKernelEx(&cfg, rope_kernel<In, Out, 4, INTER>, j, parts);
        case 8: return cudaLaunchKernelEx(&cfg, rope_kernel<In, Out, 8, INTER>, j, parts);
        case 16: return cudaLaunchKernelEx(&cfg, rope_kernel<In, Out, 16, INTER>, j, parts);
        default: return cudaLaunchKernelEx(&cfg, rope_kernel<In, Out, 32, INTER>, j, parts);
    }
}

template <typename In, typename Out>
static cudaError_t rope_way(const RopeJob &j, bool vec, cudaStream_t s)
{
    return j.inter ? rope_pick<In, Out, true>(j, vec, s) : rope_pick<In, Out, false>(j, vec, s);
}

cudaError_t rope_launch(const RopeJob &j, cudaStream_t s)
{
    // vectors: rows on 16 bytes, and halves of pairs that are whole vectors
    bool vec = j.D > 32 && j.D % 16 == 0 && (j.inter || j.rot % 16 == 0);
    for (int i = 0; i < 2; ++i)
        if (i ? j.H : j.Hq)
            vec = vec && ((uintptr_t)j.src[i] | (uintptr_t)j.ts[i] | (uintptr_t)j.hs[i] |
                          (uintptr_t)j.dst[i] | (uintptr_t)j.ots[i] | (uintptr_t)j.ohs[i]) % 16 == 0;
    if (j.dtype == SV_BF16)
        return j.odtype == SV_BF16 ? rope_way<uint16_t, uint16_t>(j, vec, s)
                                   : rope_way<uint16_t, float>(j, vec, s);
    return j.odtype == SV_BF16 ? rope_way<float, uint16_t>(j, vec, s)
                               : rope_way<float, float>(j, vec, s);
}

}  // namespace sv
