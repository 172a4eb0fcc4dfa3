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
// wraps by itself: for |inv_freq| < 2 the fraction is right to 2^-32 of a turn at
// any position, where an fp32 product would be off by p 2^-25 turns.  It is rounded
// to fp32 once, in half turns: 2^-26 of a turn.
//
// Bound by DRAM.  A head is D / 16 threads, each with two vectors of eight
// elements: the two halves of its pairs, so that the rotation needs no
// exchange.  As many heads of a token as fit a warp's lanes are taken at a time
// (D = 128: four), the next kGroups times as many are in flight; the first ones
// are before the position is there and the angles are.  The weights are
// multiplied into the cosines and sines, once for all heads of a side.  16,384
// tokens of 40 heads of 128, bf16: 60 us, 5.6 TB/s of reads and writes; one of
// kGroups in flight 61, three 71 (fewer warps), with a division and the weights
// in each head 72.
#include "sv_common.cuh"
#include "sv_kv.cuh"
#include "sv_tc.cuh"

namespace sv {

constexpr int kRopeWarps = 4;
constexpr int kGroups = 2;
constexpr int kRopeBusy = 8;           // warps an SM, before a token's heads are cut less

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
        v = __ldcs(reinterpret_cast<const uint4 *>(p));
    }
    __device__ __forceinline__ void get(float2 *f) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
};
template <>
struct Octet<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const char *p)
    {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float2 *f) const
    {
        f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
    }
};
__device__ __forceinline__ uint32_t bf16x2(float2 v)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
    return r;
}
__device__ __forceinline__ void store8(uint16_t *p, const float2 *f)
{
    __stcs(reinterpret_cast<uint4 *>(p),
           make_uint4(bf16x2(f[0]), bf16x2(f[1]), bf16x2(f[2]), bf16x2(f[3])));
}
__device__ __forceinline__ void store8(float *p, const float2 *f)
{
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[2].x, f[2].y, f[3].x, f[3].y));
}

// Heads in vectors.  PER: threads of a head, the least power of two that is
// D / 16 or more.  A warp: one token, `span` heads from part * span.
template <typename In, typename Out, int PER, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const RopeJob j, int parts, int span)
{
    constexpr int kHeads = 32 / PER;              // at a time
    __shared__ float s_cos[kRopeWarps][PER * 8], s_sin[kRopeWarps][PER * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t tok = unit / parts;
    if (tok >= j.T) return;                       // (warps do not meet below)
    const int part = (int)(unit - tok * parts);
    const int hend = min((part + 1) * span, j.Hq + j.H);
    const int l = lane % PER, half = j.rot >> 4;  // vectors of half the rotated elements
    const int pos = j.pos[tok];
    // where this thread's two vectors start, and how many of its pairs are turned
    int e0, e1, turned;
    if (INTER) {
        e0 = l * 16;
        e1 = e0 + 8;
        turned = min(max((j.rot >> 1) - l * 8, 0), 8);
    } else if (l < half) {
        e0 = l * 8;
        e1 = e0 + (j.rot >> 1);
        turned = 8;
    } else {
        e0 = j.rot + (l - half) * 16;
        e1 = e0 + 8;
        turned = 0;
    }
    int h = l < (j.D >> 4) ? part * span + lane / PER : hend;
    // heads of keys are counted on from the queries'
    const char *src0 = j.src[0] + tok * j.ts[0], *src1 = j.src[1] + tok * j.ts[1] - j.Hq * j.hs[1];
    char *dst0 = j.dst[0] + tok * j.ots[0], *dst1 = j.dst[1] + tok * j.ots[1] - j.Hq * j.ohs[1];
    Octet<In> raw[kGroups][2];
    auto fetch = [&](Octet<In> (&r)[2], int g) {
        if (g >= hend) return;
        const char *p = (g >= j.Hq ? src1 : src0) + g * (g >= j.Hq ? j.hs[1] : j.hs[0]);
        r[0].load(p + e0 * (int)sizeof(In));
        r[1].load(p + e1 * (int)sizeof(In));
    };
#pragma unroll
    for (int g = 0; g < kGroups; ++g) fetch(raw[g], h + g * kHeads);
    if (pos < 0) return;
    for (int i = lane; i < (j.rot >> 1); i += 32) {
        const float2 cs = turn(j.inv_freq[i], pos);
        s_cos[warp][i] = cs.x;
        s_sin[warp][i] = cs.y;
    }
    __syncwarp();
    // What the two elements of a pair count in the two of the result, weights in it:
    //   y_a = r (x_a w_a cos - x_b w_b sin),  y_b = r (x_b w_b cos + x_a w_a sin),
    // in fours of a pair of pairs, or (neighbours) of the pair itself.
    float2 one[8], two[8];
    const float *with = nullptr;
    auto factors = [&](const float *w) {
        with = w;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool on = i < turned;
            const float c = on ? s_cos[warp][l * 8 + i] : 1.f, s = on ? s_sin[warp][l * 8 + i] : 0.f;
            const int a = INTER ? e0 + 2 * i : e0 + i, b = INTER ? a + 1 : e1 + i;
            const float wa = w ? __ldg(w + a) : 1.f, wb = w ? __ldg(w + b) : 1.f;
            if (INTER) {
                one[i] = make_float2(wa * c, wb * c);
                two[i] = make_float2(-(wb * s), wa * s);
            } else {  // element i of the first four: a's, of the other four: b's
                float2 &p = one[i / 2], &q = two[i / 2], &x = one[4 + i / 2], &y = two[4 + i / 2];
                (i & 1 ? p.y : p.x) = wa * c;
                (i & 1 ? q.y : q.x) = -(wb * s);
                (i & 1 ? x.y : x.x) = wb * c;
                (i & 1 ? y.y : y.x) = wa * s;
            }
        }
    };
    const bool live = l < (j.D >> 4);
    if (live) factors(h >= j.Hq ? j.weight[1] : j.weight[0]);
    const int rounds = (hend - part * span + kGroups * kHeads - 1) / (kGroups * kHeads);
    for (int n = 0; n < rounds; ++n) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g, h += kHeads) {
            const bool on = h < hend;
            float2 x[8];
            if (on) {
                raw[g][0].get(x);
                raw[g][1].get(x + 4);
            }
            fetch(raw[g], h + kGroups * kHeads);
            const float *w = h >= j.Hq ? j.weight[1] : j.weight[0];
            float r = 1.f;
            if (j.weight[0] || j.weight[1]) {
                float2 sum = make_float2(0.f, 0.f);
                if (on)
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum = fma2(x[i], x[i], sum);
                float all = sum.x + sum.y;
#pragma unroll
                for (int k = PER / 2; k > 0; k >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, k);
                r = w ? rsqrtf(fmaf(all, j.share, j.eps)) : 1.f;
            }
            if (!on) continue;
            if (w != with) factors(w);
            float2 y[8];
            const float2 r2 = make_float2(r, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 z = INTER ? make_float2(x[i].y, x[i].x) : x[i ^ 4];
                y[i] = fma2(x[i], one[i], mul2(z, two[i]));
            }
            if (turned < 8) {  // (0 times what is not finite)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if ((INTER ? i : 0) >= turned) y[i] = mul2(x[i], one[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = mul2(y[i], r2);
            Out *dst = reinterpret_cast<Out *>((h >= j.Hq ? dst1 : dst0) +
                                               h * (h >= j.Hq ? j.ohs[1] : j.ohs[0]));
            store8(dst + e0, y);
            store8(dst + e1, y + 4);
        }
    }
}

// Any even D and rot, any alignment: a warp's lanes are dealt the pairs of one head
// after the other, `span` heads of a token.  (16,384 tokens as above:
// 123 us; twice the vectors' time, for its loads and stores of single elements.)
template <typename In, typename Out, int PAIRS, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32)
rope_any_kernel(const RopeJob j, int parts, int span)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t tok = unit / parts;
    if (tok >= j.T) return;
    const int pos = j.pos[tok];
    if (pos < 0) return;
    const int half = j.rot >> 1;
    int ia[PAIRS], ib[PAIRS];
    float2 cs[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
        const int i = lane + 32 * p;
        const bool near = INTER || i >= half;
        ia[p] = near ? 2 * i : i;
        ib[p] = near ? 2 * i + 1 : i + half;
        cs[p] = i < half ? turn(j.inv_freq[i], pos) : make_float2(1.f, 0.f);
    }
    const int h0 = (int)(unit - tok * parts) * span, hend = min(h0 + span, j.Hq + j.H);
    for (int h = h0; h < hend; ++h) {
        const int side = h >= j.Hq, hh = side ? h - j.Hq : h;
        const char *src = (side ? j.src[1] : j.src[0]) + tok * (side ? j.ts[1] : j.ts[0]) +
                          (int64_t)hh * (side ? j.hs[1] : j.hs[0]);
        Out *dst = reinterpret_cast<Out *>((side ? j.dst[1] : j.dst[0]) +
                                           tok * (side ? j.ots[1] : j.ots[0]) +
                                           (int64_t)hh * (side ? j.ohs[1] : j.ohs[0]));
        const float *w = side ? j.weight[1] : j.weight[0];
        float a[PAIRS], b[PAIRS];
        float sum = 0.f;
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            a[p] = b[p] = 0.f;
            if (2 * (lane + 32 * p) < j.D) {
                a[p] = load_one<In>(src + (int64_t)ia[p] * sizeof(In));
                b[p] = load_one<In>(src + (int64_t)ib[p] * sizeof(In));
            }
            sum = fmaf(a[p], a[p], fmaf(b[p], b[p], sum));
        }
        float r = 1.f;
        if (w) r = rsqrtf(fmaf(warp_sum(sum), j.share, j.eps));
        __syncwarp();  // a head is read whole before any of it is written in its place
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            const int i = lane + 32 * p;
            if (2 * i >= j.D) continue;
            const float x = w ? a[p] * (r * w[ia[p]]) : a[p], z = w ? b[p] * (r * w[ib[p]]) : b[p];
            if (i < half) {
                store_one(dst + ia[p], x * cs[p].x - z * cs[p].y);
                store_one(dst + ib[p], z * cs[p].x + x * cs[p].y);
            } else {
                store_one(dst + ia[p], x);
                store_one(dst + ib[p], z);
            }
        }
    }
}

template <typename In, typename Out, bool INTER>
static cudaError_t rope_pick(const RopeJob &j, bool vec, int sms, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    int per = 1;
    while (per * 16 < j.D) per *= 2;
    // A token's heads are a warp's, where that leaves warps enough: its angles and
    // factors are computed once.  Else they are cut, for about kRopeBusy warps an SM
    // (single elements: twice that, which wait longer).  40 heads of 128, as graphs:
    // 16,384 tokens whole 60 us, cut 82; 1,088 at 4, 8, 16, 32 warps an SM 5.9, 5.4,
    // 7.5, 7.8; 64 at 1, 8, 32 3.3, 2.8, 2.7.
    const int all = j.Hq + j.H, least = vec ? kGroups * (32 / per) : 1;
    const int64_t want = ((int64_t)sms * (vec ? kRopeBusy : 2 * kRopeBusy) + j.T - 1) / j.T;
    const int most = (all + least - 1) / least, cut = (int)(want < most ? want : most);
    const int span = ((all + cut - 1) / cut + least - 1) / least * least;
    const int parts = (all + span - 1) / span;
    const int64_t units = (int64_t)j.T * parts;
    pdl_config(cfg, at, dim3((unsigned)((units + kRopeWarps - 1) / kRopeWarps)),
               dim3(kRopeWarps * 32), 0, s);
    if (!vec) {
        if (per <= 4) return cudaLaunchKernelEx(&cfg, rope_any_kernel<In, Out, 1, INTER>, j, parts, span);
        if (per <= 8) return cudaLaunchKernelEx(&cfg, rope_any_kernel<In, Out, 2, INTER>, j, parts, span);
        if (per <= 16) return cudaLaunchKernelEx(&cfg, rope_any_kernel<In, Out, 4, INTER>, j, parts, span);
        return cudaLaunchKernelEx(&cfg, rope_any_kernel<In, Out, 8, INTER>, j, parts, span);
    }
    switch (per) {
        case 4: return cudaLaunchKernelEx(&cfg, rope_kernel<In, Out, 4, INTER>, j, parts, span);
        case 8: return cudaLaunchKernelEx(&cfg, rope_kernel<In, Out, 8, INTER>, j, parts, span);
        case 16: return cudaLaunchKernelEx(&cfg, rope_kernel<In, Out, 16, INTER>, j, parts, span);
        default: return cudaLaunchKernelEx(&cfg, rope_kernel<In, Out, 32, INTER>, j, parts, span);
    }
}

template <typename In, typename Out>
static cudaError_t rope_way(const RopeJob &j, bool vec, int sms, cudaStream_t s)
{
    return j.inter ? rope_pick<In, Out, true>(j, vec, sms, s) : rope_pick<In, Out, false>(j, vec, sms, s);
}

cudaError_t rope_launch(const RopeJob &j, int sms, cudaStream_t s)
{
    // vectors: rows on 16 bytes, and halves of pairs that are whole vectors
    bool vec = j.D > 32 && j.D % 16 == 0 && (j.inter || j.rot % 16 == 0);
    for (int i = 0; i < 2; ++i)
        if (i ? j.H : j.Hq)
            vec = vec && ((uintptr_t)j.src[i] | (uintptr_t)j.ts[i] | (uintptr_t)j.hs[i] |
                          (uintptr_t)j.dst[i] | (uintptr_t)j.ots[i] | (uintptr_t)j.ohs[i]) % 16 == 0;
    if (j.dtype == SV_BF16)
        return j.odtype == SV_BF16 ? rope_way<uint16_t, uint16_t>(j, vec, sms, s)
                                   : rope_way<uint16_t, float>(j, vec, sms, s);
    return j.odtype == SV_BF16 ? rope_way<float, uint16_t>(j, vec, sms, s)
                               : rope_way<float, float>(j, vec, sms, s);
}

}  // namespace sv
