// sv_kvplan.cu -- the places of new tokens in the paged cache, and the append
// of their keys and values in 8 bits.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sv_common.cuh"
#include "sv_kv.cuh"

namespace sv {

// ---------------------------------------------------------------------------
// Plan.  With c_b tokens in the cache and n_b to come, sequence b wants
// w_b = ceil((c_b + n_b) / block) pages and holds h_b: it takes w_b - h_b from
// the queue of free pages or gives h_b - w_b back, in order of b and then of
// the page's place in the table.  So the e-th page taken is queue entry
// head + e and the e-th given goes to tail + e: three exclusive sums over b
// (tokens, pages taken, pages given) place everything.
//
// The call is bound by latency (a few KB to read for a step of 64 sequences).
// One launch, and no CTA waits for another: every CTA takes the sums over all
// sequences for itself from L2 and keeps them in shared memory, then handles
// its share of the pages and tokens, each of which finds its sequence by
// bisection.  That needs nothing a CTA reads to be written by another one:
// the lengths, counts and queue position come out in arrays of their own, the
// table is written only at entries that no sequence held, and the queue only
// outside [head, tail).  (Three launches of one sum each would pay their gaps:
// 64 sequences take 8 us of the GPU, launch included, 1,024 with 73,221 new
// tokens 10 us.)
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

struct PlanSums {
    long long fresh, take, give;
};

// Exclusive sums over the CTA's threads; returns the totals in `tot`.
__device__ __forceinline__ PlanSums plan_scan(PlanSums v, PlanSums *part, PlanSums &tot)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const PlanSums own = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long a = __shfl_up_sync(0xFFFFFFFFu, v.fresh, d);
        const long long t = __shfl_up_sync(0xFFFFFFFFu, v.take, d);
        const long long g = __shfl_up_sync(0xFFFFFFFFu, v.give, d);
        if (lane >= d) {
            v.fresh += a;
            v.take += t;
            v.give += g;
        }
    }
    __syncthreads();
    if (lane == 31) part[warp] = v;
    __syncthreads();
    PlanSums base = {0, 0, 0};
    tot = {0, 0, 0};
#pragma unroll 8
    for (int i = 0; i < kPlanThreads / 32; ++i) {
        const PlanSums p = part[i];
        if (i < warp) {
            base.fresh += p.fresh;
            base.take += p.take;
            base.give += p.give;
        }
        tot.fresh += p.fresh;
        tot.take += p.take;
        tot.give += p.give;
    }
    return {base.fresh + v.fresh - own.fresh, base.take + v.take - own.take,
            base.give + v.give - own.give};
}

// The last b with first[b] <= e, over B entries that do not decrease.
__device__ __forceinline__ int plan_find(const int32_t *first, int B, int e)
{
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= e)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanJob j)
{
    extern __shared__ int32_t plan_words[];
    __shared__ PlanSums part[kPlanThreads / 32];
    int32_t *s_cu = plan_words, *s_take = s_cu + j.B, *s_give = s_take + j.B;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();

    const int64_t head = j.free_pos[0], tail = j.free_pos[1];
    PlanSums carry = {0, 0, 0};
    int bad = 0;
    for (int b0 = 0; b0 < j.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        PlanSums v = {0, 0, 0};
        if (b < j.B) {
            const int c = j.cached[b], n = j.fresh[b], h = j.held[b];
            const long long total = (long long)c + n;
            const long long want = (total + j.block - 1) / j.block;
            if (c < 0 || n < 0 || h < 0 || h > j.cols || want > j.cols || total > 0x7FFFFFFF) {
                bad = 1;
            } else {
                v.fresh = n;
                v.take = want > h ? want - h : 0;
                v.give = h > want ? h - want : 0;
            }
        }
        PlanSums tot;
        const PlanSums at = plan_scan(v, part, tot);
        if (b < j.B) {
            // sums beyond 32 bits are refused below, before they are used
            s_cu[b] = (int32_t)(carry.fresh + at.fresh);
            s_take[b] = (int32_t)(carry.take + at.take);
            s_give[b] = (int32_t)(carry.give + at.give);
        }
        carry.fresh += tot.fresh;
        carry.take += tot.take;
        carry.give += tot.give;
    }
    // The queue holds tail - head pages; with the pages given back it still
    // fits its ring.
    if (carry.fresh > j.cap || head < 0 || tail < head || tail - head > j.ring ||
        tail + carry.give - head > j.ring)
        bad = 1;
    const int refused = __syncthreads_or(bad) ? SV_ERR_DEVICE_BOUNDS
                        : carry.take > tail - head ? SV_ERR_OOM : 0;
    const int64_t step = (int64_t)gridDim.x * kPlanThreads;
    const int64_t first = (int64_t)blockIdx.x * kPlanThreads + tid;

    if (first == 0) {
        j.free_out[0] = refused ? head : head + carry.take;
        j.free_out[1] = refused ? tail : tail + carry.give;
        j.cu[j.B] = refused ? 0 : (int32_t)carry.fresh;
        if (refused) latch(j.err, refused);
    }
    for (int64_t b = first; b < j.B; b += step) {
        const int c = j.cached[b], n = j.fresh[b];
        j.kv_len[b] = refused ? c : c + n;
        j.cu[b] = refused ? 0 : s_cu[b];
        j.held_out[b] = refused ? j.held[b] : (c + n + j.block - 1) / j.block;
    }
    const int h0 = refused ? 0 : (int)(head % j.ring), t0 = refused ? 0 : (int)(tail % j.ring);
    if (!refused) {
        for (int64_t e = first; e < carry.take; e += step) {
            const int b = plan_find(s_take, j.B, (int)e);
            const int64_t q = h0 + e;
            j.table[(int64_t)b * j.cols + j.held[b] + ((int)e - s_take[b])] =
                j.free_ids[q < j.ring ? q : q - j.ring];
        }
        for (int64_t e = first; e < carry.give; e += step) {
            const int b = plan_find(s_give, j.B, (int)e);
            const int want = (j.cached[b] + j.fresh[b] + j.block - 1) / j.block;
            const int64_t q = t0 + e;
            j.free_ids[q < j.ring ? q : q - j.ring] =
                j.table[(int64_t)b * j.cols + want + ((int)e - s_give[b])];
        }
    }
    const int shift = 31 - __clz(j.block);  // block sizes are powers of two
    for (int64_t t = first; t < j.cap; t += step) {
        int32_t slot = -1, pos = -1;
        if (!refused && t < carry.fresh) {
            const int b = plan_find(s_cu, j.B, (int)t);
            pos = j.cached[b] + ((int)t - s_cu[b]);
            const int col = pos >> shift, h = j.held[b];
            int page;
            if (col < h) {
                page = j.table[(int64_t)b * j.cols + col];
            } else {
                const int64_t q = (int64_t)h0 + s_take[b] + (col - h);
                page = j.free_ids[q < j.ring ? q : q - j.ring];
            }
            slot = (page << shift) + (pos & (j.block - 1));
        }
        j.slot[t] = slot;
        j.pos[t] = pos;
    }
}

constexpr size_t plan_smem(int B) { return (size_t)B * 3 * sizeof(int32_t); }
static_assert(plan_smem(kPlanMaxB) + sizeof(PlanSums) * (kPlanThreads / 32) <= 227 * 1024,
              "a plan's sums fit the shared memory");

cudaError_t plan_setup()
{
    return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)plan_smem(kPlanMaxB));
}

cudaError_t plan_launch(const PlanJob &j, int sms, cudaStream_t s)
{
    // a thread for each token, page or sequence of the largest kind, on one
    // wave at most
    const long long items = std::max(j.B, j.cap);
    const int grid = (int)std::min<long long>(sms, (items + kPlanThreads - 1) / kPlanThreads);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    pdl_config(cfg, at, dim3(std::max(grid, 1)), dim3(kPlanThreads), plan_smem(j.B), s);
    return cudaLaunchKernelEx(&cfg, plan_kernel, j);
}

// ---------------------------------------------------------------------------
// Append.  Tokens with consecutive slots in one page form a run.  For each
// run, head and side (keys, values): the page's scale is the least power of
// two s >= 2^-40 (at most 2^40) with max |x| <= 448 s over the run, and at
// least the scale the page had if the run does not start at its first row.
// Where that scale grows, the rows before the run are rounded again at the new
// scale; a power of two makes that exact except for values that fall below
// the least e4m3 step.  Rows after the run are dead and stay as they are.
//
// Bound by DRAM: each element is read once, kept in registers between the
// maximum and the conversion, and written as one byte.  One CTA handles a
// run's rows of one head and side; it looks at a window of tokens for the
// first tokens of runs, so that neither many CTAs find nothing to do (long
// prompts) nor one CTA works off many runs in turn (single tokens).  CTAs of
// four warps, many on an SM, keep more loads in flight than wider ones: 38,152
// bf16 tokens of 8 heads of 128 in pages of 32 take 44 us (5.4 TB/s, 79% of the
// copy rate; 58 us with eight warps), 64 draft blocks of 9 to 17 tokens 8 us.
// ---------------------------------------------------------------------------
constexpr int kAppThreads = 128;
constexpr int kScaleExp = 40;

// Least e in [-40, 40] with amax <= 448 * 2^e, exactly: amax = f 2^E with
// f in [1, 2), and 448 = 1.75 * 2^8.
__device__ __forceinline__ int needed_exp(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int E = (int)(u >> 23) - 127;  // denormals fall below the clamp
    const int e = (u & 0x7FFFFFu) <= 0x600000u ? E - 8 : E - 7;
    return min(max(e, -kScaleExp), kScaleExp);
}

// Two floats to two e4m3 bytes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    __half2 p = *reinterpret_cast<__half2 *>(&h);
    return __half22float2(p);
}

// Eight consecutive elements of a row.
template <typename In, bool VEC>
struct Eight;
template <bool VEC>
struct Eight<uint16_t, VEC> {
    uint4 v;
    __device__ __forceinline__ void load(const char *p)
    {
        if (VEC) {
            v = __ldcs(reinterpret_cast<const uint4 *>(p));
        } else {
            const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)q[2 * i] | ((uint32_t)q[2 * i + 1] << 16);
            v = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const { VecTraits<uint16_t>::unpack(v, f); }
};
template <bool VEC>
struct Eight<float, VEC> {
    float x[8];
    __device__ __forceinline__ void load(const char *p)
    {
        if (VEC) {
            const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
            const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = reinterpret_cast<const float *>(p)[i];
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = x[i];
    }
};

// PASSES * 128 * 8 elements cover a page's rows of one head.
template <typename In, int D, int PASSES, bool VEC>
__global__ void __launch_bounds__(kAppThreads) append_kernel(const AppendJob j, int window)
{
    constexpr int kLanes = D / 8;                 // threads of a row
    constexpr int kRows = kAppThreads / kLanes;   // rows of a pass
    __shared__ float s_max[kAppThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int head = blockIdx.y >> 1, side = blockIdx.y & 1;
    const int col = (tid % kLanes) * 8, row0 = tid / kLanes;
    const char *const base = (side ? j.src[1] : j.src[0]) +
                             (int64_t)head * (side ? j.hs[1] : j.hs[0]) +
                             (int64_t)col * sizeof(In);
    const int64_t ts = side ? j.ts[1] : j.ts[0];
    uint8_t *const cache = side ? j.cache[1] : j.cache[0];
    float *const scales = side ? j.scale[1] : j.scale[0];
    pdl_wait();
    pdl_trigger();

    const int t0 = blockIdx.x * window;
    // the window's first tokens of runs, found by every warp for itself
    int mine = -1;
    bool start = false;
    if (lane < window && t0 + lane < j.T) {
        mine = j.slot[t0 + lane];
        const int before = t0 + lane > 0 ? j.slot[t0 + lane - 1] : -2;
        start = mine >= 0 && (mine != before + 1 || before < 0 || (mine & (j.block - 1)) == 0);
    }
    unsigned starts = __ballot_sync(0xFFFFFFFFu, start);
    for (; starts; starts &= starts - 1) {
        const int first = __ffs(starts) - 1;
        const int t = t0 + first;
        const int slot = __shfl_sync(0xFFFFFFFFu, mine, first);
        const int off = slot & (j.block - 1), page = slot / j.block;
        if (page >= j.pages) {
            if (tid == 0) latch(j.err, SV_ERR_DEVICE_BOUNDS);
            continue;
        }
        // the run's rows: up to the page's end, while the slots go on
        int n = 1;
        for (int i = 1; off + i < j.block; i += 32) {
            const int k = i + lane;
            const bool on = off + k < j.block && t + k < j.T && j.slot[t + k] == slot + k;
            const unsigned m = __ballot_sync(0xFFFFFFFFu, on);
            n += m == 0xFFFFFFFFu ? 32 : __ffs(~m) - 1;
            if (m != 0xFFFFFFFFu) break;
        }
        const char *src = base + (int64_t)t * ts;
        const int64_t ph = (int64_t)page * j.H + head;
        uint8_t *dst = cache + ph * j.block * D;
        Eight<In, VEC> x[PASSES];
        float amax = 0.f;
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            if (p * kRows + row0 < n) x[p].load(src + (int64_t)(p * kRows + row0) * ts);
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            if (p * kRows + row0 < n) {
                float f[8];
                x[p].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));  // NaN does not count
            }
        const float had = off ? scales[ph] : 0.f;
        amax = warp_max(amax);
        if (lane == 0) s_max[tid >> 5] = amax;
        __syncthreads();  // also: every thread has read the old scale
#pragma unroll
        for (int i = 0; i < kAppThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
        const float need = __int_as_float((needed_exp(amax) + 127) << 23);
        const float scale = fmaxf(need, had);
        if (off && scale > had) {
            const float ratio = had / scale;
            for (int i = tid; i < off * D / 16; i += kAppThreads) {
                uint4 v = reinterpret_cast<uint4 *>(dst)[i];
                uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 a = from_e4m3x2(w[k] & 0xFFFFu), b = from_e4m3x2(w[k] >> 16);
                    w[k] = e4m3x2(a.x * ratio, a.y * ratio) |
                           (e4m3x2(b.x * ratio, b.y * ratio) << 16);
                }
                reinterpret_cast<uint4 *>(dst)[i] = v;
            }
        }
        if (tid == 0) scales[ph] = scale;
        const float inv = 1.f / scale;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * kRows + row0;
            if (r < n) {
                float f[8];
                x[p].get(f);
                uint2 o;
                o.x = e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
                o.y = e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16);
                *reinterpret_cast<uint2 *>(dst + (int64_t)(off + r) * D + col) = o;
            }
        }
        __syncthreads();  // s_max is free again
    }
}

template <typename In, int D, bool VEC>
static cudaError_t append_pick(const AppendJob &j, int window, cudaStream_t s)
{
    constexpr int kRows = kAppThreads / (D / 8);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    pdl_config(cfg, at, dim3((j.T + window - 1) / window, 2 * j.H), dim3(kAppThreads), 0, s);
    const int passes = (j.block + kRows - 1) / kRows;
    if (passes <= 1) return cudaLaunchKernelEx(&cfg, append_kernel<In, D, 1, VEC>, j, window);
    if (passes <= 2) return cudaLaunchKernelEx(&cfg, append_kernel<In, D, 2, VEC>, j, window);
    if (passes <= 4) return cudaLaunchKernelEx(&cfg, append_kernel<In, D, 4, VEC>, j, window);
    if (passes <= 8) return cudaLaunchKernelEx(&cfg, append_kernel<In, D, 8, VEC>, j, window);
    return cudaLaunchKernelEx(&cfg, append_kernel<In, D, 16, VEC>, j, window);
}

template <typename In, bool VEC>
static cudaError_t append_dim(const AppendJob &j, int window, cudaStream_t s)
{
    return j.D == 64 ? append_pick<In, 64, VEC>(j, window, s)
                     : append_pick<In, 128, VEC>(j, window, s);
}

cudaError_t append_launch(const AppendJob &j, int sms, cudaStream_t s)
{
    // the window grows with the tokens until about six CTAs per SM are left
    int window = 1;
    while (window < 32 && (long long)j.T * j.H * 2 > 6LL * sms * window) window *= 2;
    bool vec = true;
    for (int i = 0; i < 2; ++i)
        vec = vec && ((uintptr_t)j.src[i] | (uintptr_t)j.ts[i] | (uintptr_t)j.hs[i]) % 16 == 0;
    if (j.dtype == SV_BF16)
        return vec ? append_dim<uint16_t, true>(j, window, s)
                   : append_dim<uint16_t, false>(j, window, s);
    return vec ? append_dim<float, true>(j, window, s) : append_dim<float, false>(j, window, s);
}

}  // namespace sv
