// sv_rows.cu -- one draw per logit row with temperature, top-k, top-p and
// min-p, from given uniforms.
//
// With the row's logits x and its maximum m, token v has the weight
// w_v = exp((x_v - m) / T).  Order the tokens by logit, the lower id first
// among equals.  Each filter keeps a prefix of that order: top-k its first k;
// top-p the shortest one whose weight reaches p times the weight of the top k;
// min-p the tokens with w_v >= min_p.  The shortest of the three is kept, and
// the draw is the first kept token, by id, whose running weight exceeds
// u times the kept weight.
//
// Decisions are exact.  Ranks are counted in integers.  Masses are sums of
// fixed-point weights (64-bit integers, so that no order of summation changes
// them), each within 2^-44 of its value: exp is taken as 2^(j/64) from a table
// times a Taylor polynomial, in pairs of floats (products split with fma,
// sums by the two-sum of Knuth and Dekker).  Only the mass of a whole row is
// first taken in fp32 with a bound on its error, and taken again in fixed
// point where a decision falls inside the bound.
//
// The boundary of the kept prefix is found by counting, not by sorting: a
// sample of 4096 logits tells about where it lies, one pass over the row
// collects the tokens around it into a shared list (all tokens above it where
// they fit), and bisection over the list's keys finds it exactly.  A row comes
// from DRAM once; the later passes hit L2, since the rows in flight (two a SM)
// take a fraction of it.
#include <float.h>
#include <math.h>

#include "sv_common.cuh"
#include "sv_rows.cuh"

namespace sv {

constexpr int kRwThreads = 512;
constexpr int kRwWarps = kRwThreads / 32;
constexpr int kListCap = 4096;
constexpr int kBins = 1024;        // of 1/16 in log2 of the weight
constexpr float kBinsPer = 16.f;
constexpr int kSampled = kRwThreads * 8;
constexpr int kIdBlock = 256;      // ids of one warp's block: 8 a lane
static_assert(kRowsMaxV / kIdBlock <= kListCap, "block sums share the list's memory");

// Bound on the relative error of the fp32 mass of a row: the argument's
// rounding and that of log2(e)/T weigh a term by its distance below the
// maximum in log2, on average at most log2 V <= 20 (twice 20 * ln2 * 2^-24),
// ex2 2^-22, and 11 additions of 2^-24: under 2^-18.
constexpr double kMassEps = 0x1p-18;

struct RowShared {
    unsigned long long mass[2][kRwWarps];
    unsigned cnt[2][kRwWarps];
    double dred[kRwWarps];
    float fred[kRwWarps];
    unsigned list_n;
    int pick;
    unsigned long long base;
    float ch, cl, xmin;
    float2 exp2_tab[64];
};

struct RowCtx {
    const char *row;
    int V, tid, lane, warp;
    float m;          // maximum
    float ch, cl;     // log2(e) / T as a pair
    int S;            // weights are multiples of 2^-S
    bool top_inf;     // the maximum is +inf: those logits share the mass
    int par;          // buffer of the next reduction
    RowShared *sh;
};

// 8 logits from id v0 on; -inf past the row's end and in place of NaN.
template <typename In, bool VEC>
__device__ __forceinline__ void load8(const RowCtx &c, int v0, float (&f)[8])
{
    if (VEC && v0 + 8 <= c.V) {
        if (sizeof(In) == 2) {
            VecTraits<uint16_t>::unpack(__ldg(reinterpret_cast<const uint4 *>(c.row + (int64_t)v0 * 2)), f);
        } else {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(c.row + (int64_t)v0 * 4));
            const float4 b = __ldg(reinterpret_cast<const float4 *>(c.row + (int64_t)v0 * 4) + 1);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = v0 + i < c.V ? VecTraits<In>::load1(c.row, v0 + i) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fmaxf(f[i], -INFINITY);
    if (c.top_inf) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] == INFINITY ? 0.f : -INFINITY;
    }
}

// The order key of a logit; -0 counts as +0.
__device__ __forceinline__ uint32_t row_key(float x) { return f2ord(x + 0.f); }
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // f2ord(-inf)

// w = exp((x - m) / T) as a multiple of 2^-S, to the nearest within 2^-44 w.
__device__ __forceinline__ unsigned long long row_weight(const RowCtx &c, float x)
{
    if (x == -INFINITY) return 0;
    // x - m = d + dl exactly
    const float d = x - c.m, bb = d - x;
    const float dl = (x - (d - bb)) + (-c.m - bb);
    // log2 w = p + e
    const float p = d * c.ch;
    if (!(p > -100.f)) return 0;
    float e = fmaf(d, c.ch, -p);
    e = fmaf(d, c.cl, e);
    e = fmaf(dl, c.ch, e);
    const float n = rintf(p * 64.f);
    const float f = fmaf(n, -0.015625f, p);  // exact
    // (f + e) ln 2 = rh + rl
    constexpr float kL = 0.693147180559945309417f;
    constexpr float kLl = (float)(0.693147180559945309417 - (double)kL);
    const float rh = f * kL;
    float rl = fmaf(f, kL, -rh);
    rl = fmaf(f, kLl, rl);
    rl = fmaf(e, kL, rl);
    // exp(r) - 1 = r + r^2/2 + r^3/6 + r^4/24 + r^5/120, |r| < 0.0055
    const float s = rh * rh;
    float se = fmaf(rh, rh, -s);
    se = fmaf(2.f * rh, rl, se);
    const float q = s * rh * fmaf(rh, fmaf(rh, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f);
    const float h = fmaf(0.5f, s, rh);
    const float l = ((rh - h) + 0.5f * s) + (fmaf(0.5f, se, rl) + q);
    const int ni = (int)n;
    const float2 t = c.sh->exp2_tab[ni & 63];
    const float ph = t.x * h;
    float pl = fmaf(t.x, h, -ph);
    pl = fmaf(t.x, l, pl);
    pl = fmaf(t.y, h, pl) + t.y;
    const float wh = t.x + ph;
    const float wl = ((t.x - wh) + ph) + pl;
    // 48 fraction bits (wh has at most 24)
    const long long I = ((long long)(int)(wh * 16777216.f) << 24) + (int)rintf(wl * 0x1p48f);
    const int sh = c.S - 48 + (ni >> 6);
    if (sh >= 0) return (unsigned long long)I << sh;
    if (sh < -62) return 0;
    return (unsigned long long)((I + (1ll << (-sh - 1))) >> -sh);
}

// Sum of up to 2^62 over the CTA, in every thread.
__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long v)
{
    const unsigned a = __reduce_add_sync(0xFFFFFFFFu, (unsigned)(v & 0x3FFFFFu));
    const unsigned b = __reduce_add_sync(0xFFFFFFFFu, (unsigned)((v >> 22) & 0x3FFFFFu));
    const unsigned d = __reduce_add_sync(0xFFFFFFFFu, (unsigned)(v >> 44));
    return (unsigned long long)a + ((unsigned long long)b << 22) + ((unsigned long long)d << 44);
}
__device__ __forceinline__ unsigned long long cta_mass(RowCtx &c, unsigned long long v)
{
    v = warp_sum64(v);
    const int par = c.par;
    c.par ^= 1;
    if (c.lane == 0) c.sh->mass[par][c.warp] = v;
    __syncthreads();
    unsigned long long r = 0;
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) r += c.sh->mass[par][i];
    return r;
}
__device__ __forceinline__ unsigned cta_count(RowCtx &c, unsigned v)
{
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    const int par = c.par;
    c.par ^= 1;
    if (c.lane == 0) c.sh->cnt[par][c.warp] = v;
    __syncthreads();
    unsigned r = 0;
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) r += c.sh->cnt[par][i];
    return r;
}

// floor(f * M) and ceil(f * M) for a float f in [0, 1], exactly.
__device__ __forceinline__ unsigned long long scale_mass(float f, unsigned long long M, bool up)
{
    if (f >= 1.f) return M;
    const uint32_t b = __float_as_uint(f);
    const int ex = (int)(b >> 23);
    const unsigned long long mant = ex ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
    const int k = 150 - (ex ? ex : 1);  // f = mant * 2^-k, k >= 24
    const unsigned long long lo = M * mant, hi = __umul64hi(M, mant);
    unsigned long long r, rest;
    if (k < 64) {
        r = (lo >> k) | (hi << (64 - k));
        rest = lo & ((1ull << k) - 1);
    } else if (k < 128) {
        r = k == 64 ? hi : hi >> (k - 64);
        rest = lo | (k == 64 ? 0 : hi & ((1ull << (k - 64)) - 1));
    } else {
        r = 0;
        rest = lo | hi;
    }
    return r + (up && rest ? 1 : 0);
}

// Visit the row in steps of 8 logits a thread: f(v0, logits).
template <typename In, bool VEC, typename F>
__device__ __forceinline__ void each8(const RowCtx &c, F f)
{
    constexpr int kStep = kRwThreads * 8;
    int v0 = c.tid * 8;
    for (; v0 + kStep < c.V; v0 += 2 * kStep) {  // two loads in flight
        float a[8], b[8];
        load8<In, VEC>(c, v0, a);
        load8<In, VEC>(c, v0 + kStep, b);
        f(v0, a);
        f(v0 + kStep, b);
    }
    if (v0 < c.V) {
        float a[8];
        load8<In, VEC>(c, v0, a);
        f(v0, a);
    }
}

__device__ __forceinline__ float max8(const float (&f)[8])
{
    return fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])),
                 fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));
}

// The row's maximum.
template <typename In, bool VEC>
__device__ float row_max(RowCtx &c)
{
    float m = -INFINITY;
    each8<In, VEC>(c, [&](int, const float (&f)[8]) { m = fmaxf(m, max8(f)); });
    m = warp_max(m);
    if (c.lane == 0) c.sh->fred[c.warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) m = fmaxf(m, c.sh->fred[i]);
    return m;
}

// The row's maximum and its mass sum_v 2^((x_v - m) ch) within kMassEps.
template <typename In, bool VEC>
__device__ float row_max_mass(RowCtx &c, double *mass)
{
    // terms against an integer reference e (a multiple of the exponent): a
    // larger reference moves the sum by an exact power of two
    float m = -INFINITY, e = -FLT_MAX, s = 0.f;
    double total = 0.0;
    int n = 0;
    each8<In, VEC>(c, [&](int, const float (&f)[8]) {
        const float top = max8(f);
        m = fmaxf(m, top);
        if (top > -INFINITY && top < INFINITY) {
            const float r = ceilf(top * c.ch);
            if (r > e) {
                const float k = e == -FLT_MAX ? 0.f : pow2_int(fmaxf(e - r, -127.f));
                s *= k;
                total *= (double)k;
                e = r;
            }
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = ex2f(fmaf(f[i], c.ch, -e));
            s += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
            if (++n == 8) {
                total += (double)s;
                s = 0.f;
                n = 0;
            }
        }
    });
    total += (double)s;
    float wm = warp_max(m);
    if (c.lane == 0) c.sh->fred[c.warp] = wm;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) wm = fmaxf(wm, c.sh->fred[i]);
    m = wm;
    // this thread's sum in units of 2^(m ch): e - m ch in fp64, its power in fp32
    const double y = e == -FLT_MAX ? -1000.0 : (double)e - (double)m * (double)c.ch;
    total *= y < -126.0 ? 0.0 : (double)exp2f((float)y);
    total = warp_sumd(total);
    if (c.lane == 0) c.sh->dred[c.warp] = total;
    __syncthreads();
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) z += c.sh->dred[i];
    *mass = z;
    return m;
}

// Exact mass and count of the logits with key >= k.
template <typename In, bool VEC>
__device__ void row_above(RowCtx &c, uint32_t k, bool want_mass, unsigned *cnt,
                          unsigned long long *mass)
{
    const float t = ord2f(k);
    unsigned n = 0;
    unsigned long long w = 0;
    each8<In, VEC>(c, [&](int, const float (&f)[8]) {
        if (max8(f) >= t) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (row_key(f[i]) >= k && f[i] > -INFINITY) {
                    ++n;
                    if (want_mass) w += row_weight(c, f[i]);
                }
        }
    });
    *cnt = cta_count(c, n);
    *mass = want_mass ? cta_mass(c, w) : 0;
}

// Collect the logits with lo <= key < hi (hi = 0: no upper end) as (key, id);
// returns how many there are, of which the first kListCap are listed.
template <typename In, bool VEC>
__device__ unsigned row_collect(RowCtx &c, uint32_t lo, uint32_t hi, uint32_t *key, uint32_t *id)
{
    const float t = ord2f(lo);
    if (c.tid == 0) c.sh->list_n = 0;
    __syncthreads();
    each8<In, VEC>(c, [&](int v0, const float (&f)[8]) {
        if (max8(f) >= t) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t k = row_key(f[i]);
                if (k >= lo && (hi == 0 || k < hi) && f[i] > -INFINITY) {
                    const unsigned at = atomicAdd(&c.sh->list_n, 1u);
                    if (at < (unsigned)kListCap) {
                        key[at] = k;
                        id[at] = (uint32_t)(v0 + i);
                    }
                }
            }
        }
    });
    __syncthreads();
    return c.sh->list_n;
}

// What the kept prefix has to reach: `rank` tokens, or a mass known to lie in
// [lo, hi] (equal once it is exact).
struct Goal {
    bool by_mass;
    unsigned rank;
    unsigned long long lo, hi;
    // 1: reached, 0: not, -1: the bounds on the row's mass do not tell
    __device__ int reached(unsigned cnt, unsigned long long mass) const
    {
        if (!by_mass) return cnt >= rank;
        return mass >= hi ? 1 : mass < lo ? 0 : -1;
    }
};

template <typename In, bool VEC>
__global__ void __launch_bounds__(kRwThreads, 2) rows_kernel(const RowsJob j)
{
    extern __shared__ unsigned long long rows_smem[];
    __shared__ RowShared sh;
    unsigned long long *s_w = rows_smem;                              // [kListCap]
    uint32_t *s_key = reinterpret_cast<uint32_t *>(s_w + kListCap);   // [kListCap]
    uint32_t *s_id = s_key + kListCap;                                // [kListCap]
    unsigned *s_hist = reinterpret_cast<unsigned *>(s_w);             // [kBins], before the list
    float *s_tail = reinterpret_cast<float *>(s_hist + kBins);        // [kBins]

    RowCtx c;
    c.tid = threadIdx.x;
    c.lane = c.tid & 31;
    c.warp = c.tid >> 5;
    c.V = j.V;
    c.par = 0;
    c.top_inf = false;
    c.sh = &sh;
    c.S = 0;
    const int r = blockIdx.x;
    // 2^(j/64) as a pair of floats
    if (c.tid < 64) {
        const double t = exp2((double)c.tid / 64.0);
        const float h = (float)t;
        sh.exp2_tab[c.tid] = make_float2(h, (float)(t - (double)h));
    }
    pdl_wait();
    pdl_trigger();
    c.row = j.x + (int64_t)r * j.rs;
    const float T = j.temp ? j.temp[r] : 1.f, u = j.u[r];
    const float top_p = j.top_p ? j.top_p[r] : 1.f, min_p = j.min_p ? j.min_p[r] : 0.f;
    int top_k = j.top_k ? j.top_k[r] : 0;
    auto answer = [&](int token, float prob, int kept) {
        if (c.tid == 0) {
            j.token[r] = token;
            j.prob[r] = prob;
            j.kept[r] = kept;
        }
    };
    // (a temperature below 2^-20 counts as wrong: log2(e)/T has to stay finite)
    if (!(T == 0.f || (T >= 0x1p-20f && T < INFINITY)) || !(u >= 0.f && u <= 1.f) ||
        !(top_p >= 0.f) || !(min_p >= 0.f && min_p <= 1.f) || top_k < 0) {
        if (c.tid == 0) latch(j.err, SV_ERR_DEVICE_BOUNDS);
        answer(-1, __int_as_float(0x7FC00000), 0);
        return;
    }
    const bool by_k = top_k > 0 && top_k < j.V, by_p = top_p < 1.f;
    if (c.tid == 0) {
        const double C = T > 0.f ? 1.4426950408889634 / (double)T : 1.0;
        sh.ch = (float)C;
        sh.cl = (float)(C - (double)sh.ch);
    }
    __syncthreads();
    c.ch = sh.ch;
    c.cl = sh.cl;

    // ---- the maximum, and the row's mass where a filter or the draw needs it
    const bool need_mass = T > 0.f && !by_k;
    double z = 1.0;
    c.m = need_mass ? row_max_mass<In, VEC>(c, &z) : row_max<In, VEC>(c);
    if (c.m == -INFINITY) {  // nothing is left of the row
        answer(-1, 0.f, 0);
        return;
    }
    if (T == 0.f) {
        int best = 0x7FFFFFFF;
        each8<In, VEC>(c, [&](int v0, const float (&f)[8]) {
#pragma unroll
            for (int i = 7; i >= 0; --i)
                if (f[i] == c.m) best = min(best, v0 + i);
        });
        best = __reduce_min_sync(0xFFFFFFFFu, best);
        if (c.lane == 0) sh.cnt[0][c.warp] = (unsigned)best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRwWarps; ++i) best = min(best, (int)sh.cnt[0][i]);
        answer(best, 1.f, 1);
        return;
    }
    if (c.m == INFINITY) {
        c.top_inf = true;
        c.m = 0.f;
        unsigned n;
        unsigned long long w;
        row_above<In, VEC>(c, kKeyNegInf + 1, false, &n, &w);
        z = (double)n;
    }
    // weights in units of 2^-S: sums stay below 2^62.  (Where products of
    // logits and 1/T leave the fp32 range the fp32 mass says nothing.)
    const bool z_known = z >= 0.5 && z <= 2.0 * (double)j.V;
    {
        const double most = need_mass && z_known ? z * 1.001
                            : (double)(by_k && top_k <= kListCap ? kListCap : j.V);
        int ex;
        frexp(most, &ex);
        c.S = min(61 - ex, 58);
    }
    unsigned long long zlo, zhi;
    {
        const double zs = ldexp(z, c.S);
        zlo = (unsigned long long)(zs * (1.0 - kMassEps));
        zhi = (unsigned long long)(zs * (1.0 + kMassEps)) + 1;
    }
    auto refine = [&]() {  // the row's mass in fixed point
        unsigned n;
        unsigned long long w;
        row_above<In, VEC>(c, kKeyNegInf + 1, true, &n, &w);
        zlo = zhi = w;
    };
    if (!z_known && by_p) refine();
    // the least logit that min-p keeps: m + T log(min_p), rounded up
    uint32_t key_min = kKeyNegInf + 1;
    if (min_p > 0.f) {
        if (c.tid == 0) {
            const double b = (double)c.m + (double)T * log((double)min_p);
            sh.xmin = __double2float_ru(b);
        }
        __syncthreads();
        key_min = row_key(sh.xmin);
    }

    // ---- where the boundary lies, from a sample
    // With both k and p the mass of the top k is needed, whatever min-p keeps.
    uint32_t lo = by_k && by_p ? kKeyNegInf + 1 : key_min;
    uint32_t hi = 0;  // the boundary's key is in [lo, hi); 0: open
    unsigned base_n = 0;            // tokens and mass at or above hi
    unsigned long long base_w = 0;
    unsigned list_n = 0;
    bool listed = false;
    Goal goal;
    goal.by_mass = !by_k && by_p;
    goal.rank = by_k ? (unsigned)top_k : 0xFFFFFFFFu;
    auto set_goal = [&]() {
        goal.lo = scale_mass(top_p, zlo, true);
        goal.hi = scale_mass(top_p, zhi, true);
    };
    set_goal();
    const bool filtered = by_k || by_p || min_p > 0.f;
    uint32_t guess_lo = lo, guess_hi = 0;
    float est = (float)j.V;
    if (filtered && j.V > kListCap) {
        for (int i = c.tid; i < kBins; i += kRwThreads) s_hist[i] = 0;
        __syncthreads();
        {
            // 8 consecutive logits a thread, spread evenly over the row
            const int v0 = (int)((int64_t)c.tid * (j.V / 8) / kRwThreads) * 8;
            float f[8];
            load8<In, VEC>(c, v0, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = (c.m - f[i]) * c.ch * kBinsPer;
                atomicAdd(&s_hist[y < (float)(kBins - 1) ? (int)y : kBins - 1], 1u);
            }
        }
        __syncthreads();
        const float per = (float)j.V / (float)kSampled;  // tokens a sampled one stands for
        // Counts from the top and masses from the bottom, two bins a thread.
        {
            const int b = 2 * c.tid;
            const unsigned n0 = s_hist[b], n1 = s_hist[b + 1];
            const float w0 = (float)n0 * ex2f(-((float)b + 0.5f) / kBinsPer);
            const float w1 = (float)n1 * ex2f(-((float)b + 1.5f) / kBinsPer);
            unsigned cs = n0 + n1;
            float ws = w0 + w1;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned a = __shfl_up_sync(0xFFFFFFFFu, cs, d);
                const float q = __shfl_up_sync(0xFFFFFFFFu, ws, d);
                if (c.lane >= d) {
                    cs += a;
                    ws += q;
                }
            }
            if (c.lane == 31) {
                sh.cnt[0][c.warp] = cs;
                sh.fred[c.warp] = ws;
            }
            __syncthreads();
            float all = 0.f;
            for (int i = 0; i < kRwWarps; ++i) {
                if (i < c.warp) {
                    cs += sh.cnt[0][i];
                    ws += sh.fred[i];
                }
                all += sh.fred[i];
            }
            s_hist[b] = cs - n1;
            s_hist[b + 1] = cs;
            s_tail[b] = all - (ws - w1);      // mass of the bins after b
            s_tail[b + 1] = all - ws;
            __syncthreads();
        }
        // the first bin whose end surely (to several deviations) lies past the boundary
        auto first_bin = [&](auto past) {
            int best = kBins - 1;
            for (int b = 2 * c.tid + 1; b >= 2 * c.tid; --b)
                if (past(b)) best = min(best, b);
            best = __reduce_min_sync(0xFFFFFFFFu, best);
            __syncthreads();
            if (c.lane == 0) sh.cnt[0][c.warp] = (unsigned)best;
            __syncthreads();
            for (int i = 0; i < kRwWarps; ++i) best = min(best, (int)sh.cnt[0][i]);
            return best;
        };
        int bin = kBins - 1, bin_hi = 0;
        if (by_k) {
            const float want = (float)top_k / per;
            const float margin = want + 4.f * sqrtf(want) + 8.f;
            const float under = want - 4.f * sqrtf(want) - 8.f;
            bin = first_bin([&](int b) { return (float)s_hist[b] >= margin; });
            bin_hi = first_bin([&](int b) { return (float)s_hist[b] >= under; });
        } else if (by_p) {
            const float left = (1.f - top_p) * (float)z * 0.85f / per;
            bin = first_bin([&](int b) { return s_tail[b] <= left; });
            bin_hi = first_bin([&](int b) { return s_tail[b] * 0.72f <= left; });
        }
        if (bin < kBins - 1) {
            const uint32_t k = row_key(c.m - (float)(bin + 1) / kBinsPer / c.ch);
            guess_lo = max(k, lo);
            guess_hi = row_key(c.m - (float)bin_hi / kBinsPer / c.ch);
        }
        // tokens in the list, if it starts there (a bin too many is no harm)
        const float yl = (c.m - ord2f(guess_lo)) * c.ch * kBinsPer;
        const int bl = yl < (float)(kBins - 1) ? (int)yl : kBins - 1;
        est = (float)s_hist[bl] * per;
        __syncthreads();
    }
    if (filtered) {
        // ---- small kept sets: list everything from the guess on
        if (est < 0.9f * kListCap || j.V <= kListCap) {
            const uint32_t from = max(guess_lo, lo);
            list_n = row_collect<In, VEC>(c, from, 0, s_key, s_id);
            if (list_n <= (unsigned)kListCap) {
                bool enough = from <= lo;
                if (!enough) {
                    if (by_k) {
                        enough = list_n >= (unsigned)top_k;
                    } else {
                        unsigned long long w = 0;
                        for (int i = c.tid; i < (int)list_n; i += kRwThreads)
                            w += row_weight(c, ord2f(s_key[i]));
                        w = cta_mass(c, w);
                        enough = goal.reached(0, w) == 1;
                    }
                }
                if (enough) {
                    lo = from;
                    listed = true;
                }
            }
        }
        // ---- otherwise narrow [lo, hi) until its tokens fit the list (min-p
        // alone needs no list: its boundary is known)
        if (!listed && (by_k || by_p)) {
            unsigned in_n;  // tokens at or above lo
            unsigned long long w;
            row_above<In, VEC>(c, lo, false, &in_n, &w);
            uint32_t top = row_key(c.m) + 1;
            int tries = 0;
            while (in_n - base_n > (unsigned)kListCap && top - lo > 1) {
                // first around the guess, then by halves of the key range
                uint32_t mid = lo + (top - lo) / 2;
                const uint32_t k = tries == 0 ? guess_hi : guess_lo;
                if (tries < 2 && k > lo && k < top) mid = k;
                ++tries;
                unsigned n;
                row_above<In, VEC>(c, mid, goal.by_mass, &n, &w);
                int got = goal.reached(n, w);
                if (got < 0) {
                    refine();
                    set_goal();
                    got = goal.reached(n, w);
                }
                if (got) {
                    lo = mid;
                    in_n = n;
                } else {
                    top = mid;
                    base_n = n;
                    base_w = w;
                }
            }
            hi = top;
            if (in_n - base_n <= (unsigned)kListCap) {
                list_n = row_collect<In, VEC>(c, lo, hi, s_key, s_id);
            } else {
                list_n = 0;  // more equal logits than fit: one key, known count
            }
            // with top-k beyond the list, the mass above the list is still open
            if (by_k && by_p) row_above<In, VEC>(c, hi, true, &base_n, &base_w);
        }
    }

    // ---- the boundary: key t and how many of its tokens (lowest ids first)
    uint32_t t = kKeyNegInf + 1;
    unsigned ties_kept = 0xFFFFFFFFu, kept = 0;
    int id_cut = 0x7FFFFFFF;
    const bool one_key = (by_k || by_p) && !listed && list_n == 0;
    if (filtered) {
        for (int i = c.tid; i < (int)list_n; i += kRwThreads)
            s_w[i] = row_weight(c, ord2f(s_key[i]));
        __syncthreads();
        auto above = [&](uint32_t k, bool want, unsigned *n, unsigned long long *w) {
            unsigned a = 0;
            unsigned long long b = 0;
            for (int i = c.tid; i < (int)list_n; i += kRwThreads)
                if (s_key[i] >= k) {
                    ++a;
                    if (want) b += s_w[i];
                }
            *n = base_n + cta_count(c, a);
            *w = want ? base_w + cta_mass(c, b) : 0;
        };
        unsigned one_n = 0;
        if (one_key) {
            unsigned long long w;
            row_above<In, VEC>(c, lo, false, &one_n, &w);
        }
        // the largest key whose tokens and those above reach the goal; the
        // list's lowest key where none does
        auto boundary = [&](Goal &g, uint32_t *key, unsigned *n_at, unsigned long long *w_at,
                            unsigned *n_over, unsigned long long *w_over) {
            const bool want = g.by_mass;
            uint32_t a = lo, b = hi ? hi : row_key(c.m) + 1;  // reached at a, not at b
            unsigned n;
            unsigned long long w;
            if (one_key) {
                *key = lo;
                *n_at = one_n;
                *n_over = base_n;
                *w_over = base_w;
                *w_at = base_w + (one_n - base_n) * row_weight(c, ord2f(lo));
                return;
            }
            while (b - a > 1) {
                const uint32_t mid = a + (b - a) / 2;
                above(mid, want, &n, &w);
                int got = g.reached(n, w);
                if (got < 0) {
                    refine();
                    set_goal();
                    g = goal;
                    got = g.reached(n, w);
                }
                if (got)
                    a = mid;
                else
                    b = mid;
            }
            *key = a;
            above(a, true, n_at, w_at);
            above(b, true, n_over, w_over);
        };
        t = lo;
        unsigned n_at = 0, n_over = 0;
        unsigned long long w_at, w_over;
        if (by_k) {
            boundary(goal, &t, &n_at, &w_at, &n_over, &w_over);
            // (fewer than k finite logits: every one of them)
            ties_kept = min((unsigned)top_k, n_at) - n_over;
            if (by_p) {
                const unsigned long long wt = row_weight(c, ord2f(t));
                Goal g;
                g.by_mass = true;
                g.rank = 0;
                const unsigned long long M = w_over + ties_kept * wt;
                g.lo = g.hi = scale_mass(top_p, M, true);
                uint32_t tp;
                unsigned pn_at, pn_over;
                unsigned long long pw_at, pw_over;
                if (g.lo <= base_w && base_n > 0) {
                    // the boundary of p lies above the list: narrow again over the row
                    uint32_t a = hi, b = row_key(c.m) + 1;
                    unsigned n;
                    unsigned long long w;
                    while (b - a > 1) {
                        const uint32_t mid = a + (b - a) / 2;
                        row_above<In, VEC>(c, mid, true, &n, &w);
                        if (w >= g.lo)
                            a = mid;
                        else
                            b = mid;
                    }
                    tp = a;
                    row_above<In, VEC>(c, a, true, &pn_at, &pw_at);
                    row_above<In, VEC>(c, b, true, &pn_over, &pw_over);
                } else {
                    boundary(g, &tp, &pn_at, &pw_at, &pn_over, &pw_over);
                }
                const unsigned long long wp = row_weight(c, ord2f(tp));
                unsigned rp = pn_at - pn_over;
                if (wp) rp = (unsigned)min((unsigned long long)rp,
                                           (g.lo - min(pw_over, g.lo) + wp - 1) / wp);
                rp = max(rp, 1u);
                if (tp > t || (tp == t && rp < ties_kept)) {
                    t = tp;
                    ties_kept = rp;
                    n_over = pn_over;
                    n_at = pn_at;
                }
            }
        } else if (by_p) {
            boundary(goal, &t, &n_at, &w_at, &n_over, &w_over);
            const unsigned long long wt = row_weight(c, ord2f(t));
            unsigned rp = n_at - n_over;
            if (wt) {
                // tokens of this key until the goal is reached: both ends of its bounds
                auto until = [&](unsigned long long g) {
                    return (g - min(w_over, g) + wt - 1) / wt;
                };
                if (until(goal.lo) != until(goal.hi) && until(goal.lo) < rp) {
                    refine();
                    set_goal();
                }
                rp = (unsigned)min((unsigned long long)rp, until(goal.hi));
            }
            ties_kept = max(rp, 1u);
        }
        // min-p cuts at a logit, with all its equals (and never above the maximum)
        if (t < key_min || !(by_k || by_p)) {
            t = key_min;
            ties_kept = 0xFFFFFFFFu;
            unsigned long long w;
            if (listed)
                above(t, false, &n_at, &w);
            else
                row_above<In, VEC>(c, t, false, &n_at, &w);
            n_over = 0;
        }
        const unsigned ties = n_at - n_over;
        kept = n_over + min(ties_kept, ties);
        if (ties_kept < ties) {
            // the id of the ties_kept-th lowest id among the boundary's equals
            int a = -1, b = j.V - 1;
            const bool in_list = list_n && t >= lo && (hi == 0 || t < hi);
            while (b - a > 1) {
                const int mid = a + (b - a) / 2;
                unsigned n = 0;
                if (in_list) {
                    for (int i = c.tid; i < (int)list_n; i += kRwThreads)
                        n += s_key[i] == t && (int)s_id[i] <= mid;
                } else {
                    each8<In, VEC>(c, [&](int v0, const float (&f)[8]) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) n += row_key(f[i]) == t && v0 + i <= mid;
                    });
                }
                if (cta_count(c, n) >= ties_kept)
                    b = mid;
                else
                    a = mid;
            }
            id_cut = b;
        }
    }

    // ---- the draw
    const bool all = !filtered;  // every finite logit is kept
    auto is_kept = [&](float x, int id) {
        const uint32_t k = row_key(x);
        return all ? x > -INFINITY : k > t || (k == t && id <= id_cut);
    };
    auto drawn = [&](int id, float x, unsigned long long M) {
        const double w = exp(((double)x - (double)c.m) / (double)T);
        j.token[r] = id;
        j.prob[r] = (float)(ldexp(w, c.S) / (double)M);
        j.kept[r] = (int)kept;
    };
    // At the ends of u the answer is the first or the last kept token of any
    // weight at all (above the least double), however small.
    int end_id = -1;
    if (u == 0.f || u == 1.f) {
        int best = u == 0.f ? 0x7FFFFFFF : -1;
        each8<In, VEC>(c, [&](int v0, const float (&f)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (is_kept(f[i], v0 + i) &&
                    ((double)f[i] - (double)c.m) / (double)T > -745.0)
                    best = u == 0.f ? min(best, v0 + i) : max(best, v0 + i);
        });
        best = u == 0.f ? __reduce_min_sync(0xFFFFFFFFu, best)
                        : __reduce_max_sync(0xFFFFFFFFu, best);
        __syncthreads();
        if (c.lane == 0) sh.cnt[0][c.warp] = (unsigned)best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRwWarps; ++i)
            best = u == 0.f ? min(best, (int)sh.cnt[0][i]) : max(best, (int)sh.cnt[0][i]);
        end_id = best;
        __syncthreads();
    }
    if (listed) {
        unsigned long long w = 0;
        for (int i = c.tid; i < (int)list_n; i += kRwThreads) {
            const bool on = s_key[i] > t || (s_key[i] == t && (int)s_id[i] <= id_cut);
            if (!on) s_w[i] = 0;
            w += s_w[i];
        }
        const unsigned long long M = cta_mass(c, w);
        const unsigned long long g = min(scale_mass(u, M, false), M - 1);
        // running weight at most g at a, above it at b
        int a = end_id < 0 ? -1 : end_id - 1, b = end_id < 0 ? j.V - 1 : end_id;
        while (b - a > 1) {
            const int mid = a + (b - a) / 2;
            w = 0;
            for (int i = c.tid; i < (int)list_n; i += kRwThreads)
                if ((int)s_id[i] <= mid) w += s_w[i];
            if (cta_mass(c, w) > g)
                b = mid;
            else
                a = mid;
        }
        for (int i = c.tid; i < (int)list_n; i += kRwThreads)
            if ((int)s_id[i] == b) drawn(b, ord2f(s_key[i]), M);
        return;
    }
    // Sums of kept weights over blocks of 256 ids, one warp a block.
    const int blocks = (j.V + kIdBlock - 1) / kIdBlock;
    auto kept_weight = [&](float x, int id) -> unsigned long long {
        return is_kept(x, id) ? row_weight(c, x) : 0;
    };
    if (all) t = kKeyNegInf + 1;
    __syncthreads();
    unsigned finite = 0;
    for (int b = c.warp; b < blocks; b += kRwWarps) {
        float f[8];
        load8<In, VEC>(c, b * kIdBlock + c.lane * 8, f);
        unsigned long long w = 0;
        if (max8(f) >= ord2f(t)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w += kept_weight(f[i], b * kIdBlock + c.lane * 8 + i);
                finite += f[i] > -INFINITY;
            }
        }
        w = warp_sum64(w);
        if (c.lane == 0) s_w[b] = w;
    }
    if (all) kept = cta_count(c, finite);
    __syncthreads();
    // each thread takes consecutive blocks
    const int each = (blocks + kRwThreads - 1) / kRwThreads;
    unsigned long long own = 0;
    for (int i = 0; i < each; ++i) {
        const int b = c.tid * each + i;
        if (b < blocks) own += s_w[b];
    }
    const unsigned long long M = cta_mass(c, own);
    const unsigned long long g = min(scale_mass(u, M, false), M - 1);
    unsigned long long run = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long a = __shfl_up_sync(0xFFFFFFFFu, run, d);
        if (c.lane >= d) run += a;
    }
    if (c.lane == 31) sh.mass[c.par][c.warp] = run;
    __syncthreads();
    for (int i = 0; i < c.warp; ++i) run += sh.mass[c.par][i];
    if (run > g && run - own <= g) {  // exactly one thread
        unsigned long long at = run - own;
        int b = c.tid * each;
        while (at + s_w[b] <= g) at += s_w[b++];
        sh.pick = b;
        sh.base = at;
    }
    __syncthreads();
    if (end_id >= 0) {
        if (c.tid == 0) {
            float f[8];
            load8<In, VEC>(c, end_id & ~7, f);
            float x = f[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) x = (end_id & 7) == i ? f[i] : x;
            drawn(end_id, x, M);
        }
        return;
    }
    if (c.warp == 0) {
        const int v0 = sh.pick * kIdBlock + c.lane * 8;
        float f[8];
        load8<In, VEC>(c, v0, f);
        unsigned long long w[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = kept_weight(f[i], v0 + i);
            sum += w[i];
        }
        unsigned long long before = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long a = __shfl_up_sync(0xFFFFFFFFu, before, d);
            if (c.lane >= d) before += a;
        }
        before += sh.base - sum;
        if (before <= g && before + sum > g) {
            bool done = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                before += w[i];
                if (!done && before > g) {
                    done = true;
                    drawn(v0 + i, f[i], M);
                }
            }
        }
    }
}

constexpr size_t kRowsSmem = (size_t)kListCap * (8 + 4 + 4);

template <typename In, bool VEC>
static cudaError_t rows_attr()
{
    return cudaFuncSetAttribute(rows_kernel<In, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kRowsSmem);
}

cudaError_t rows_setup()
{
    cudaError_t e = rows_attr<uint16_t, true>();
    if (e == cudaSuccess) e = rows_attr<uint16_t, false>();
    if (e == cudaSuccess) e = rows_attr<float, true>();
    if (e == cudaSuccess) e = rows_attr<float, false>();
    return e;
}

cudaError_t rows_launch(const RowsJob &j, int sms, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    pdl_config(cfg, at, dim3(j.R), dim3(kRwThreads), kRowsSmem, s);
    // whole 16-byte vectors where the rows start on one; single elements otherwise
    const bool vec = ((uintptr_t)j.x | (uintptr_t)j.rs) % 16 == 0;
    if (j.dtype == SV_BF16)
        return vec ? cudaLaunchKernelEx(&cfg, rows_kernel<uint16_t, true>, j)
                   : cudaLaunchKernelEx(&cfg, rows_kernel<uint16_t, false>, j);
    return vec ? cudaLaunchKernelEx(&cfg, rows_kernel<float, true>, j)
               : cudaLaunchKernelEx(&cfg, rows_kernel<float, false>, j);
}

}  // namespace sv
