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
// Only the tokens around the boundary of the kept prefix are ordered.  A sample
// of 8192 logits tells about where it lies.  Where the tokens above it should
// fit a shared list, the row's only pass collects them while it takes the
// maximum and the mass.  Otherwise a second pass (in L2: the rows in flight,
// two a SM, take a fraction of it) lists those near the boundary and sums the
// others: those above by blocks of ids, for the draw.  In the list the boundary,
// and later the drawn id, are found by histograms over 9 bits at a time.
//
// A bf16 logit of magnitude 2^-10 to 2^12 is one of 5,632; so a pass that sums
// many weights takes them from a table of the row's, 45 KB, and computes only
// the others (a weight costs some 90 instructions, a look-up 8).  fp32 logits
// are queued, and a warp weighs 32 of them at once.
//
// Measured on 1,088 bf16 rows of 128,256 (41 us at the copy rate): T = 0 62 us
// (4.5 TB/s), k = 50 230 us, p = 0.9 with 28,000 kept tokens 720 us, no filter
// 500 us; a mix of them 410 us.  Filtered rows are bound by the chain of short
// steps after the first pass, of which two rows an SM hide each other's; wide
// ones by the instructions of their weights.
#include <float.h>
#include <math.h>

#include "sv_common.cuh"
#include "sv_rows.cuh"

namespace sv {

constexpr int kRwThreads = 512;
constexpr int kRwWarps = kRwThreads / 32;
constexpr int kListCap = 4096;
constexpr int kBins = 1024;        // of 1/32 in log2 of the weight
constexpr float kBinsPer = 32.f;
constexpr int kSampled = kRwThreads * 16;
constexpr int kIdStep = 256;       // ids of a warp's step: 8 a lane
constexpr int kIdBlock = 1024;     // ids of a block: 4 steps
constexpr int kMaxBlocks = kRowsMaxV / kIdBlock;
constexpr int kTabMag = 117 << 7;  // bits of 2^-10, the table's least magnitude
constexpr int kTabHalf = 22 << 7;  // its magnitudes, up to 2^12
constexpr int kDigits = 512;       // bins of a selection step: 9 bits

// Bound on the relative error of the fp32 mass of a row: the argument's
// rounding and that of log2(e)/T weigh a term by its distance below the
// maximum in log2, on average at most log2 V <= 20 (twice 20 * ln2 * 2^-24),
// ex2 2^-22, and 11 additions of 2^-24: under 2^-18.
constexpr double kMassEps = 0x1p-18;
// The same for the tokens below the bracket alone, whose distances are larger
// (up to 35 in log2; beyond, a row's tokens weigh less than 2^-15 of its maximum).
constexpr double kTailEps = 0x1p-17;

// (key, id) of a listed token: larger pairs come first in the order.
__device__ __forceinline__ unsigned long long pair_of(uint32_t key, int id)
{
    return ((unsigned long long)key << 32) | (uint32_t)~id;
}
__device__ __forceinline__ uint32_t pair_key(unsigned long long p) { return (uint32_t)(p >> 32); }
__device__ __forceinline__ int pair_id(unsigned long long p) { return (int)~(uint32_t)p; }

struct Digits {  // counts and masses (16 bits a word) of a selection step
    unsigned n[kDigits], w[4][kDigits];
};

struct RowShared {
    float queue[kRwWarps][64];
    unsigned long long mass[kRwWarps];
    unsigned cnt[kRwWarps];
    double dred[kRwWarps];
    float fred[kRwWarps];
    unsigned list_n;
    int pick;
    unsigned pick_n, pick_at;
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
    RowShared *sh;
};

// 8 logits from id v0 on; -inf past the row's end and in place of NaN.
template <typename In, bool VEC>
__device__ __forceinline__ void load8(const RowCtx c, int v0, float (&f)[8])
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
// (One copy of it, and one of each pass below: copied into the loops that use
// them they were several times the instruction caches.)
__device__ __noinline__ unsigned long long row_weight(float x, float m, float ch, float cl, int S,
                                                      const float2 *tab)
{
    if (x == -INFINITY) return 0;
    // x - m = d + dl exactly
    const float d = x - m, bb = d - x;
    const float dl = (x - (d - bb)) + (-m - bb);
    // log2 w = p + e
    const float p = d * ch;
    if (!(p > -100.f)) return 0;
    float e = fmaf(d, ch, -p);
    e = fmaf(d, cl, e);
    e = fmaf(dl, ch, e);
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
    const float2 t = tab[ni & 63];
    const float ph = t.x * h;
    float pl = fmaf(t.x, h, -ph);
    pl = fmaf(t.x, l, pl);
    pl = fmaf(t.y, h, pl) + t.y;
    const float wh = t.x + ph;
    const float wl = ((t.x - wh) + ph) + pl;
    // 48 fraction bits (wh has at most 24)
    const long long I = ((long long)(int)(wh * 16777216.f) << 24) + (int)rintf(wl * 0x1p48f);
    const int sh = S - 48 + (ni >> 6);
    if (sh >= 0) return (unsigned long long)I << sh;
    if (sh < -62) return 0;
    return (unsigned long long)((I + (1ll << (-sh - 1))) >> -sh);
}
__device__ __forceinline__ unsigned long long row_weight(const RowCtx c, float x)
{
    return row_weight(x, c.m, c.ch, c.cl, c.S, c.sh->exp2_tab);
}

// Sum of up to 2^62 over the CTA, in every thread.
__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long v)
{
    const unsigned a = __reduce_add_sync(0xFFFFFFFFu, (unsigned)(v & 0x3FFFFFu));
    const unsigned b = __reduce_add_sync(0xFFFFFFFFu, (unsigned)((v >> 22) & 0x3FFFFFu));
    const unsigned d = __reduce_add_sync(0xFFFFFFFFu, (unsigned)(v >> 44));
    return (unsigned long long)a + ((unsigned long long)b << 22) + ((unsigned long long)d << 44);
}
__device__ __forceinline__ unsigned long long cta_mass(const RowCtx c, unsigned long long v)
{
    v = warp_sum64(v);
    __syncthreads();
    if (c.lane == 0) c.sh->mass[c.warp] = v;
    __syncthreads();
    unsigned long long r = 0;
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) r += c.sh->mass[i];
    return r;
}
__device__ __forceinline__ unsigned cta_count(const RowCtx c, unsigned v)
{
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if (c.lane == 0) c.sh->cnt[c.warp] = v;
    __syncthreads();
    unsigned r = 0;
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) r += c.sh->cnt[i];
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

// Visit the row in steps of 8 logits a thread: f(v0, logits).  Every lane of a
// warp takes part in every step (logits past the row's end are -inf).
template <typename In, bool VEC, typename F>
__device__ __forceinline__ void each8(const RowCtx c, F f)
{
    constexpr int kStep = kRwThreads * 8, kDeep = sizeof(In) == 2 ? 4 : 2;  // loads in flight
    int v0 = c.tid * 8;
    for (; v0 - c.lane * 8 + (kDeep - 1) * kStep < c.V; v0 += kDeep * kStep) {
        float a[kDeep][8];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) load8<In, VEC>(c, v0 + i * kStep, a[i]);
#pragma unroll
        for (int i = 0; i < kDeep; ++i) f(v0 + i * kStep, a[i]);
    }
    for (; v0 - c.lane * 8 < c.V; v0 += kStep) {
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

// The row's first pass: its maximum (with the lowest id that has it, where
// `top_id` is given), its mass sum_v 2^((x_v - m) ch) within kMassEps (`mass`),
// and the logits at or above `from` in the list (`list`; counted in
// sh.list_n, which is 0 before).
template <typename In, bool VEC>
__device__ __forceinline__ float row_first(const RowCtx c, double *mass, int *top_id, float from,
                           unsigned long long *list)
{
    // terms against an integer reference e (a multiple of the exponent): a
    // larger reference moves the sum by an exact power of two
    float m = -INFINITY, e = -FLT_MAX, s = 0.f;
    double total = 0.0;
    int n = 0, at = -1;
    each8<In, VEC>(c, [&](int v0, const float (&f)[8]) {
        const float top = max8(f);
        if (top > m) {  // (a thread's ids rise)
            m = top;
            at = v0;
        }
        if (list && top >= from) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (f[i] >= from && f[i] > -INFINITY) {
                    const unsigned k = atomicAdd(&c.sh->list_n, 1u);
                    if (k < (unsigned)kListCap) list[k] = pair_of(row_key(f[i]), v0 + i);
                }
        }
        if (mass && top > -INFINITY && top < INFINITY) {
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
    const float own = m;
    m = warp_max(m);
    if (c.lane == 0) c.sh->fred[c.warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) m = fmaxf(m, c.sh->fred[i]);
    if (top_id) {
        int best = 0x7FFFFFFF;
        if (own == m && at >= 0) {
            float f[8];
            load8<In, VEC>(c, at, f);
#pragma unroll
            for (int i = 7; i >= 0; --i)
                if (f[i] == m) best = at + i;
        }
        best = __reduce_min_sync(0xFFFFFFFFu, best);
        if (c.lane == 0) c.sh->cnt[c.warp] = (unsigned)best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRwWarps; ++i) best = min(best, (int)c.sh->cnt[i]);
        *top_id = best;
    }
    if (mass) {
        total += (double)s;
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
    }
    return m;
}

// A warp's queue of logits whose weights are to be summed: the few lanes of a
// step that have one put it there, and a full warp's worth is weighed at once.
struct WeightQueue {
    float *buf;   // 64 of this warp's
    int n;
    unsigned long long sum;
    __device__ __forceinline__ void init(const RowCtx c)
    {
        buf = c.sh->queue[c.warp];
        n = 0;
        sum = 0;
    }
    __device__ __forceinline__ void put(const RowCtx c, float x, bool on)
    {
        const unsigned m = __ballot_sync(0xFFFFFFFFu, on);
        if (on) buf[n + __popc(m & ((1u << c.lane) - 1))] = x;
        n += __popc(m);
        if (n >= 32) {
            __syncwarp();
            sum += row_weight(c, buf[c.lane]);
            const float rest = buf[32 + c.lane];
            __syncwarp();
            n -= 32;
            if (c.lane < n) buf[c.lane] = rest;
        }
    }
    // the lane's part of everything put so far
    __device__ __forceinline__ unsigned long long take(const RowCtx c)
    {
        __syncwarp();
        if (c.lane < n) sum += row_weight(c, buf[c.lane]);
        __syncwarp();
        const unsigned long long s = sum;
        n = 0;
        sum = 0;
        return s;
    }
};

// Exact mass and count of the logits with key >= k.
template <typename In, bool VEC>
__device__ __noinline__ void row_above(const RowCtx c, uint32_t k, bool want_mass, unsigned *cnt,
                          unsigned long long *mass)
{
    const float t = ord2f(k);
    unsigned n = 0;
    WeightQueue q;
    q.init(c);
    each8<In, VEC>(c, [&](int, const float (&f)[8]) {
        if (__any_sync(0xFFFFFFFFu, max8(f) >= t)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool on = row_key(f[i]) >= k && f[i] > -INFINITY;
                n += on;
                if (want_mass) q.put(c, f[i], on);
            }
        }
    });
    const unsigned long long w = want_mass ? q.take(c) : 0;
    *cnt = cta_count(c, n);
    *mass = want_mass ? cta_mass(c, w) : 0;
}

// Collect the logits with lo <= key < hi (hi = 0: no upper end); returns how
// many there are, of which the first kListCap are listed.
template <typename In, bool VEC>
__device__ __noinline__ unsigned row_collect(const RowCtx c, uint32_t lo, uint32_t hi, unsigned long long *list)
{
    const float t = ord2f(lo);
    __syncthreads();
    if (c.tid == 0) c.sh->list_n = 0;
    __syncthreads();
    each8<In, VEC>(c, [&](int v0, const float (&f)[8]) {
        if (max8(f) >= t) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t k = row_key(f[i]);
                if (k >= lo && (hi == 0 || k < hi) && f[i] > -INFINITY) {
                    const unsigned at = atomicAdd(&c.sh->list_n, 1u);
                    if (at < (unsigned)kListCap) list[at] = pair_of(k, v0 + i);
                }
            }
        }
    });
    __syncthreads();
    return c.sh->list_n;
}

// The row's table of bf16 weights (negative magnitudes in its second half).
__device__ __noinline__ void row_table(const RowCtx c, unsigned long long *tab)
{
    __syncthreads();
    for (int e = c.tid; e < 2 * kTabHalf; e += kRwThreads) {
        const uint32_t bits = e < kTabHalf ? (uint32_t)(kTabMag + e)
                                           : 0x8000u | (uint32_t)(kTabMag + e - kTabHalf);
        const float x = __uint_as_float(bits << 16);
        tab[e] = x <= c.m ? row_weight(c, x) : 0;
    }
    __syncthreads();
}
__device__ __forceinline__ unsigned long long table_weight(const RowCtx c,
                                                           const unsigned long long *tab, float x)
{
    const uint32_t bits = __float_as_uint(x) >> 16;
    const uint32_t off = (bits & 0x7FFFu) - (uint32_t)kTabMag;
    if (off < (uint32_t)kTabHalf) return tab[off + (bits >> 15) * (uint32_t)kTabHalf];
    return row_weight(c, x);
}

// The row in three: from hi on exact masses of blocks of ids (`block`) and the
// count; from lo to hi the list (its length is returned; the first kListCap are
// there); below lo the mass (`tail`): exact for bf16, else in fp32 within
// kTailEps (`ftail`, in units of the maximum's weight).
template <typename In, bool VEC>
__device__ __noinline__ unsigned row_split(const RowCtx c, float lo, float hi, const unsigned long long *tab,
                              unsigned long long *list, unsigned long long *block,
                              unsigned *above, unsigned long long *tail, double *ftail)
{
    constexpr bool kTab = sizeof(In) == 2;
    __syncthreads();
    if (c.tid == 0) c.sh->list_n = 0;
    __syncthreads();
    const int blocks = (c.V + kIdBlock - 1) / kIdBlock;
    WeightQueue q;
    q.init(c);
    unsigned n = 0;
    unsigned long long below = 0;
    double total = 0.0;
    for (int b = c.warp; b < blocks; b += kRwWarps) {
        unsigned long long own = 0;
        float s = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float f[2][8];  // two steps in flight
#pragma unroll
            for (int k = 0; k < 2; ++k)
                load8<In, VEC>(c, b * kIdBlock + (half * 2 + k) * kIdStep + c.lane * 8, f[k]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int v0 = b * kIdBlock + (half * 2 + k) * kIdStep + c.lane * 8;
                float t[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = f[k][i];
                    const bool on = x >= hi;
                    n += on;
                    t[i] = 0.f;
                    if (kTab) {
                        const unsigned long long w = table_weight(c, tab, x);
                        own += on ? w : 0;
                        below += x < lo ? w : 0;
                    } else {
                        q.put(c, x, on);
                        if (x < lo) t[i] = ex2f((x - c.m) * c.ch);
                    }
                    if (x >= lo && !on) {
                        const unsigned at = atomicAdd(&c.sh->list_n, 1u);
                        if (at < (unsigned)kListCap) list[at] = pair_of(row_key(x), v0 + i);
                    }
                }
                if (!kTab) s += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
            }
        }
        const unsigned long long w = warp_sum64(kTab ? own : q.take(c));
        if (c.lane == 0) block[b] = w;
        total += (double)s;
    }
    total = warp_sumd(total);
    if (c.lane == 0) c.sh->dred[c.warp] = total;
    *above = cta_count(c, n);
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) z += c.sh->dred[i];
    *ftail = z;
    *tail = cta_mass(c, below);
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

// What select_step looks at: the keys of the listed tokens (downwards), the ids
// of those with one key, or the ids of the kept ones (both upwards).
enum : int { kByKey, kIdsOfKey, kKeptIds };
enum : int { kFound, kOn, kPast, kAgain };

// One step of finding the value in [from, to) at which counts and masses, on
// top of n and w, reach the goal: 9 bits of it.  Narrows [from, to) to the
// step's bin, with n and w what comes before it and n_at the tokens in it.
// kFound: the bin is one value; kPast: the goal is beyond all; kAgain: bounds
// that do not tell (nothing is changed).
__device__ __noinline__ int select_step(const RowCtx c, Digits *dig, const unsigned long long *list,
                                        const unsigned long long *weight, int len, int what,
                                        uint32_t key, int cut, uint32_t *from, uint32_t *to,
                                        const Goal g, unsigned *n, unsigned long long *w,
                                        unsigned *n_at)
{
    RowShared &sh = *c.sh;
    const uint32_t lo = *from, span = *to - lo;
    const int shift = span <= 1 ? 0 : max(32 - __clz(span - 1) - 9, 0);
    const uint32_t last = span <= 1 ? 0 : (span - 1) >> shift;
    dig->n[c.tid] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) dig->w[k][c.tid] = 0;
    if (c.tid == 0) sh.pick = -1;
    __syncthreads();
    for (int i = c.tid; i < len; i += kRwThreads) {
        const unsigned long long p = list[i];
        const uint32_t x = what == kByKey ? pair_key(p) : (uint32_t)pair_id(p);
        const bool on = what == kByKey || (what == kIdsOfKey && pair_key(p) == key) ||
                        (what == kKeptIds && (pair_key(p) > key ||
                                              (pair_key(p) == key && pair_id(p) <= cut)));
        if (on && x >= lo && x - lo < span) {
            const uint32_t b = (x - lo) >> shift, d = what == kByKey ? last - b : b;
            atomicAdd(&dig->n[d], 1u);
            if (g.by_mass || what == kByKey) {
                const unsigned long long y = weight[i];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    atomicAdd(&dig->w[k][d], (unsigned)(y >> (16 * k)) & 0xFFFFu);
            }
        }
    }
    __syncthreads();
    const unsigned own_n = dig->n[c.tid];
    unsigned long long own_w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) own_w += (unsigned long long)dig->w[k][c.tid] << (16 * k);
    unsigned run_n = own_n;
    unsigned long long run_w = own_w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned a = __shfl_up_sync(0xFFFFFFFFu, run_n, d);
        const unsigned long long b = __shfl_up_sync(0xFFFFFFFFu, run_w, d);
        if (c.lane >= d) {
            run_n += a;
            run_w += b;
        }
    }
    if (c.lane == 31) {
        sh.cnt[c.warp] = run_n;
        sh.mass[c.warp] = run_w;
    }
    __syncthreads();
    run_n += *n;
    run_w += *w;
    for (int i = 0; i < c.warp; ++i) {
        run_n += sh.cnt[i];
        run_w += sh.mass[i];
    }
    const int got = g.reached(run_n, run_w), had = g.reached(run_n - own_n, run_w - own_w);
    // (a goal that needs nothing is reached by the first token)
    if (got == 1 && own_n > 0 && (had == 0 || run_n - own_n == *n)) {
        sh.pick = c.tid;
        sh.pick_n = run_n - own_n;
        sh.base = run_w - own_w;
        sh.pick_at = own_n;
    }
    if (__syncthreads_or(own_n > 0 && (got < 0 || had < 0))) return kAgain;
    const int pick = sh.pick;
    if (pick < 0) return kPast;
    *n = sh.pick_n;
    *w = sh.base;
    *n_at = sh.pick_at;
    const uint32_t b = what == kByKey ? last - (uint32_t)pick : (uint32_t)pick;
    *from = lo + (b << shift);
    *to = *from + min(*to - *from, 1u << shift);
    __syncthreads();
    return shift == 0 ? kFound : kOn;
}

template <typename In, bool VEC>
__global__ void __launch_bounds__(kRwThreads, 2) rows_kernel(const RowsJob j)
{
    extern __shared__ unsigned long long rows_smem[];
    __shared__ RowShared sh;
    unsigned long long *s_w = rows_smem;              // [kListCap] weights of the list
    unsigned long long *s_tab = s_w;                  // [2 kTabHalf] before them: the table
    unsigned long long *s_list = s_w + 2 * kTabHalf;  // [kListCap] pairs
    unsigned long long *s_block = s_list + kListCap;  // [kMaxBlocks] masses of id blocks
    Digits *s_dig = reinterpret_cast<Digits *>(s_block + kMaxBlocks);
    unsigned *s_hist = reinterpret_cast<unsigned *>(s_dig);     // [kBins], before selections
    float *s_tail = reinterpret_cast<float *>(s_hist + kBins);  // [kBins]
    static_assert(sizeof(Digits) >= kBins * 8 && kBins == 2 * kRwThreads, "the sample's bins");

    RowCtx c;
    c.tid = threadIdx.x;
    c.lane = c.tid & 31;
    c.warp = c.tid >> 5;
    c.V = j.V;
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

    if (T == 0.f) {
        int id;
        const float m = row_first<In, VEC>(c, nullptr, &id, 0.f, nullptr);
        answer(m > -INFINITY ? id : -1, m > -INFINITY ? 1.f : 0.f, m > -INFINITY);
        return;
    }

    // ---- where the boundary lies, from a sample: bins of log2 weights below
    // the sample's maximum
    const bool filtered = by_k || by_p || min_p > 0.f;
    const bool sampled = filtered && j.V > kListCap;
    const float per = (float)j.V / (float)kSampled;  // tokens a sampled one stands for
    float s_max = -INFINITY, s_all = 0.f;            // the sample's maximum and mass
    if (sampled) {
        for (int i = c.tid; i < kBins; i += kRwThreads) s_hist[i] = 0;
        // twice 8 consecutive logits a thread, spread evenly over the row
        float f[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            load8<In, VEC>(c, (int)((int64_t)(c.tid + k * kRwThreads) * (j.V / 8) /
                                    (2 * kRwThreads)) * 8, f[k]);
        s_max = warp_max(fmaxf(max8(f[0]), max8(f[1])));
        if (c.lane == 0) sh.fred[c.warp] = s_max;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRwWarps; ++i) s_max = fmaxf(s_max, sh.fred[i]);
        if (s_max > -INFINITY && s_max < INFINITY) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = (s_max - f[k][i]) * c.ch * kBinsPer;
                    atomicAdd(&s_hist[y < (float)(kBins - 1) ? (int)y : kBins - 1], 1u);
                }
        }
        __syncthreads();
        // Counts from the top and masses from the bottom, two bins a thread.
        const int b = 2 * c.tid;
        unsigned n[2];
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            n[i] = s_hist[b + i];
            w[i] = (float)n[i] * ex2f(-((float)(b + i) + 0.5f) / kBinsPer);
        }
        unsigned cs = n[0] + n[1];
        float ws = w[0] + w[1];
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
            sh.cnt[c.warp] = cs;
            sh.fred[c.warp] = ws;
        }
        __syncthreads();
        for (int i = 0; i < kRwWarps; ++i) {
            if (i < c.warp) {
                cs += sh.cnt[i];
                ws += sh.fred[i];
            }
            s_all += sh.fred[i];
        }
#pragma unroll
        for (int i = 1; i >= 0; --i) {
            s_hist[b + i] = cs;
            s_tail[b + i] = s_all - ws;  // mass of the bins after it
            cs -= n[i];
            ws -= w[i];
        }
        __syncthreads();
    }
    // the first bin that is past a limit, by counts or by masses of the rest
    auto first_bin = [&](auto past) {
        int best = kBins - 1;
        for (int b = 2 * c.tid + 1; b >= 2 * c.tid; --b)
            if (past(b)) best = min(best, b);
        best = __reduce_min_sync(0xFFFFFFFFu, best);
        __syncthreads();
        if (c.lane == 0) sh.cnt[c.warp] = (unsigned)best;
        __syncthreads();
        for (int i = 0; i < kRwWarps; ++i) best = min(best, (int)sh.cnt[i]);
        return best;
    };
    const bool bins = sampled && s_max > -INFINITY && s_max < INFINITY;
    auto bin_end = [&](int b) {  // the logit at which bin b - 1 ends and b starts
        return b >= kBins - 1 ? -INFINITY : s_max - (float)b / kBinsPer / c.ch;
    };
    // surely (to several deviations) past the boundary, and surely before it;
    // rest: the mass that top-p leaves out, in the sample's terms
    auto guess = [&](float rest, float margin, float *from, float *to) {
        int lo = kBins - 1, hi = 0;
        if (by_k) {
            const float want = (float)top_k / per, off = 4.f * sqrtf(want) + 6.f;
            lo = first_bin([&](int b) { return (float)s_hist[b] >= want + off; });
            hi = first_bin([&](int b) { return (float)s_hist[b] >= want - off; });
        } else if (by_p) {
            lo = first_bin([&](int b) { return s_tail[b] <= (1.f - margin) * rest; });
            hi = first_bin([&](int b) { return s_tail[b] <= (1.f + margin) * rest; });
        }
        *from = bin_end(lo + 1);
        *to = bin_end(hi);
    };
    auto tokens_from = [&](float x) {  // how many, by the sample
        const float y = (s_max - x) * c.ch * kBinsPer;
        return (float)s_hist[y < (float)(kBins - 1) ? max((int)y, 0) : kBins - 1] * per;
    };
    // With both k and p the mass of the top k is needed, whatever min-p keeps.
    const bool min_cuts = min_p > 0.f && !(by_k && by_p);
    float g_lo = -INFINITY, g_hi = INFINITY;
    bool collect = filtered && !sampled;
    if (bins) {
        guess((1.f - top_p) * s_all, 0.1f, &g_lo, &g_hi);
        // (the sample's maximum and mass are at most the row's: this is early)
        if (min_cuts) g_lo = fmaxf(g_lo, s_max + T * logf(min_p) * 1.0001f - 1e-6f);
        collect = tokens_from(g_lo) < 0.8f * kListCap;
    }

    // ---- the first pass
    const bool need_mass = !by_k;
    double z = 1.0;
    if (c.tid == 0) sh.list_n = 0;
    __syncthreads();
    c.m = row_first<In, VEC>(c, need_mass ? &z : nullptr, nullptr, g_lo,
                             collect ? s_list : nullptr);
    if (c.m == -INFINITY) {  // nothing is left of the row
        answer(-1, 0.f, 0);
        return;
    }
    unsigned list_n = collect ? sh.list_n : 0;
    if (list_n > (unsigned)kListCap) collect = false;
    if (c.m == INFINITY) {
        c.top_inf = true;
        c.m = 0.f;
        collect = false;
        g_lo = -INFINITY;
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
    // The row's mass in fixed point.  (The list's weights are lost: the table
    // takes their place.)
    auto refine = [&]() {
        unsigned n;
        unsigned long long w = 0;
        if (sizeof(In) == 2 && !c.top_inf) {
            unsigned long long none;
            double f;
            row_table(c, s_tab);
            row_split<In, VEC>(c, -FLT_MAX, -FLT_MAX, s_tab, s_list, s_block, &n, &none, &f);
            const int blocks = (j.V + kIdBlock - 1) / kIdBlock;
            for (int i = c.tid; i < blocks; i += kRwThreads) w += s_block[i];
            w = cta_mass(c, w);
        } else {
            row_above<In, VEC>(c, kKeyNegInf + 1, true, &n, &w);
        }
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

    uint32_t lo = min_cuts ? key_min : kKeyNegInf + 1;
    uint32_t hi = 0;  // the boundary's key is in [lo, hi); 0: open
    unsigned base_n = 0;            // tokens and mass at or above hi
    unsigned long long base_w = 0;
    bool listed = false;   // the list holds every kept token
    bool one_key = false, p_exact = false;
    bool have_blocks = false;  // s_block holds the masses above hi
    Goal goal;
    goal.by_mass = !by_k && by_p;
    goal.rank = by_k ? (unsigned)top_k : 0xFFFFFFFFu;
    auto set_goal = [&]() {
        goal.lo = scale_mass(top_p, zlo, true);
        goal.hi = scale_mass(top_p, zhi, true);
    };
    set_goal();
    uint32_t guess_lo = max(row_key(g_lo), lo), guess_hi = 0;

    // ---- otherwise narrow [lo, hi) until its tokens fit the list
    auto narrow = [&](Goal &g) {
        unsigned in_n;  // tokens at or above lo
        unsigned long long w;
        row_above<In, VEC>(c, lo, false, &in_n, &w);
        uint32_t top = row_key(c.m) + 1;
        base_n = 0;
        base_w = 0;
        int tries = 0;
        while (in_n - base_n > (unsigned)kListCap && top - lo > 1) {
            // first around the guess, then by halves of the key range
            uint32_t mid = lo + (top - lo) / 2;
            const uint32_t k = tries == 0 ? guess_hi : guess_lo;
            if (tries < 2 && k > lo && k < top) mid = k;
            ++tries;
            unsigned n;
            row_above<In, VEC>(c, mid, g.by_mass, &n, &w);
            int got = g.reached(n, w);
            if (got < 0) {
                refine();
                set_goal();
                got = g.reached(n, w);
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
        // (more equal logits than the list holds: none is listed)
        list_n = in_n - base_n <= (unsigned)kListCap ? row_collect<In, VEC>(c, lo, hi, s_list) : 0;
        one_key = in_n - base_n > (unsigned)kListCap;
    };
    // Weights of the listed tokens.
    auto weigh = [&]() {
        for (int i = c.tid; i < (int)list_n; i += kRwThreads)
            s_w[i] = row_weight(c, ord2f(pair_key(s_list[i])));
        __syncthreads();
    };
    // select_step with the bounds on the row's mass refined where they do not tell
    auto select = [&](int what, uint32_t from, uint32_t to, Goal &g, uint32_t key, int cut,
                      uint32_t *v, unsigned *n, unsigned long long *w, unsigned *n_at) -> bool {
        for (;;) {
            const int r = select_step(c, s_dig, s_list, s_w, (int)list_n, what, key, cut, &from,
                                      &to, g, n, w, n_at);
            if (r == kAgain) {
                refine();
                set_goal();
                weigh();
                g = goal;
            } else if (r != kOn) {
                *v = from;
                return r == kFound;
            }
        }
    };

    // Token `id` with logit x is drawn, of a kept mass M.
    unsigned kept = 0;
    auto drawn = [&](int id, float x, unsigned long long M) {
        const double w = exp(((double)x - (double)c.m) / (double)T);
        j.token[r] = id;
        j.prob[r] = (float)(ldexp(w, c.S) / (double)M);
        j.kept[r] = (int)kept;
    };

    // ---- the boundary: the last kept token's key t and id (id_cut), and the
    // number of kept tokens
    uint32_t t = key_min;
    int id_cut = j.V;
    if (filtered) {
        unsigned long long list_mass = 0;
        // is what the list starts from past the boundary?
        auto try_list = [&](uint32_t from) {
            bool enough = from <= lo || (by_k && list_n >= (unsigned)top_k);
            if (!enough && goal.by_mass) {
                unsigned long long w = 0;
                for (int i = c.tid; i < (int)list_n; i += kRwThreads)
                    w += row_weight(c, ord2f(pair_key(s_list[i])));
                list_mass = cta_mass(c, w);
                enough = goal.reached(0, list_mass) == 1;
            }
            if (enough) {
                lo = min(from, lo);
                listed = true;
            }
        };
        if (collect) try_list(g_lo == -INFINITY ? kKeyNegInf + 1 : row_key(g_lo));
        // Again, with the row's maximum and mass in place of the sample's.  A pass
        // that misses the boundary has told the exact mass above one logit: the
        // sample's mass below that one, and how far the exact mass is from the
        // goal, say where to look next.
        const float unit =  // a weight's mass in the sample's terms
            exp2f(fminf((c.m - s_max) * c.ch, 100.f)) / per;
        float margin = 0.05f, rest = (1.f - top_p) * (float)z * unit;
        auto learn = [&](float x, unsigned long long above, float step) {
            const float y = (s_max - x) * c.ch * kBinsPer;
            const int b = y < (float)(kBins - 1) ? (int)y - 1 : kBins - 1;
            const double off = (double)above - (double)goal.hi;
            const float at = b < 0 ? s_all : s_tail[b];
            rest = fmaxf(at + (float)ldexp(off, -c.S) * unit * step, 0.3f * at);
            margin = 0.1f;
        };
        for (int time = 0; time < (goal.by_mass ? 8 : 1) && !listed && !have_blocks && bins &&
                           !c.top_inf; ++time) {
            guess(rest, margin, &g_lo, &g_hi);
            guess_lo = max(row_key(g_lo), lo);
            guess_hi = row_key(g_hi);
            const float x = ord2f(guess_lo);
            if (tokens_from(x) < 0.9f * kListCap) {
                list_n = row_collect<In, VEC>(c, guess_lo, 0, s_list);
                if (list_n <= (unsigned)kListCap) {
                    try_list(guess_lo);
                    // (the sample misses heavy tokens: longer and longer steps)
                    if (!listed && goal.by_mass) learn(x, list_mass, 1.f + (float)time);
                } else {
                    margin = 0.02f;
                }
            } else if (goal.by_mass && guess_hi > guess_lo && z_known) {
                double ftail;
                unsigned long long tail;
                unsigned above;
                if (sizeof(In) == 2) row_table(c, s_tab);
                list_n = row_split<In, VEC>(c, ord2f(guess_lo), ord2f(guess_hi), s_tab, s_list,
                                            s_block, &above, &tail, &ftail);
                const int blocks = (j.V + kIdBlock - 1) / kIdBlock;
                unsigned long long a = 0, l = 0;
                for (int i = c.tid; i < blocks; i += kRwThreads) a += s_block[i];
                a = cta_mass(c, a);
                if (list_n > (unsigned)kListCap) {
                    learn(ord2f(guess_hi), a, 1.f);
                    margin = 0.02f;
                } else {
                    weigh();
                    for (int i = c.tid; i < (int)list_n; i += kRwThreads) l += s_w[i];
                    l = cta_mass(c, l);
                    // the row's mass again: at most the tail is not exact
                    const double ts = ldexp(ftail, c.S);
                    const unsigned long long old_lo = zlo, old_hi = zhi;
                    if (sizeof(In) == 2) {
                        zlo = zhi = a + l + tail;
                    } else {
                        zlo = max(old_lo, a + l + (unsigned long long)(ts * (1.0 - kTailEps)));
                        zhi = min(old_hi, a + l + (unsigned long long)(ts * (1.0 + kTailEps)) + 1);
                    }
                    set_goal();
                    if (a < goal.lo && a + l >= goal.hi && guess_lo >= lo) {
                        lo = guess_lo;
                        hi = guess_hi;
                        base_n = above;
                        base_w = a;
                        have_blocks = true;
                    } else if (a >= goal.lo) {
                        learn(ord2f(guess_hi), a, 1.f);
                    } else {
                        learn(x, a + l, 1.f);
                    }
                }
            }
        }
        if (listed && list_n <= (unsigned)kRwThreads) {
            // A list of at most a token a thread: each thread counts the tokens
            // before its own, and their weights; then those of lower ids.
            weigh();
            const bool mine = c.tid < (int)list_n;
            const unsigned long long p = mine ? s_list[c.tid] : 0, w = mine ? s_w[c.tid] : 0;
            unsigned rank = 0;
            unsigned long long before = 0;
            if (c.warp * 32 < (int)list_n)
                for (int i = 0; i < (int)list_n; ++i)
                    if (s_list[i] > p) {
                        ++rank;
                        before += s_w[i];
                    }
            bool on = mine && (!by_k || rank < (unsigned)top_k);
            if (by_k && by_p) {
                const unsigned long long M = cta_mass(c, on ? w : 0);
                on = on && (before < scale_mass(top_p, M, true) || rank == 0);
            } else if (by_p) {
                if (__syncthreads_or(mine && before >= goal.lo && before < goal.hi)) {
                    refine();
                    set_goal();
                    weigh();
                }
                on = on && (before < goal.hi || rank == 0);
            }
            on = on && (pair_key(p) >= key_min || rank == 0);
            kept = cta_count(c, on);
            const unsigned long long M = cta_mass(c, on ? w : 0);
            const int id = pair_id(p);
            const float x = ord2f(pair_key(p));
            if (u == 0.f || u == 1.f) {
                // the first or the last kept token of any weight at all
                const bool any = on && ((double)x - (double)c.m) / (double)T > -745.0;
                int best = any ? id : u == 0.f ? 0x7FFFFFFF : -1;
                best = u == 0.f ? __reduce_min_sync(0xFFFFFFFFu, best)
                                : __reduce_max_sync(0xFFFFFFFFu, best);
                __syncthreads();
                if (c.lane == 0) sh.cnt[c.warp] = (unsigned)best;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kRwWarps; ++i)
                    best = u == 0.f ? min(best, (int)sh.cnt[i]) : max(best, (int)sh.cnt[i]);
                if (any && id == best) drawn(id, x, M);
                return;
            }
            const unsigned long long g = min(scale_mass(u, M, false), M - 1);
            if (mine && !on) s_w[c.tid] = 0;
            __syncthreads();
            if (__any_sync(0xFFFFFFFFu, on)) {
                unsigned long long run = w;
                for (int i = 0; i < (int)list_n; ++i)
                    if (pair_id(s_list[i]) < id) run += s_w[i];
                if (on && run > g && run - w <= g) drawn(id, x, M);
            }
            return;
        }
        // min-p's boundary is known; it needs no list where it comes first
        bool min_first = !listed && !by_k && !by_p;
        if (min_first || (!listed && !have_blocks && goal.by_mass && min_cuts)) {
            unsigned long long w;
            row_above<In, VEC>(c, key_min, by_p, &kept, &w);
            min_first = min_first || goal.reached(kept, w) == 0;
        }
        if (min_first) {
            list_n = 0;
        } else {
            if (!listed && !have_blocks) {
                narrow(goal);
                if (by_k && by_p) {
                    // the mass of the top k, and with it the boundary of p
                    unsigned long long w;
                    row_above<In, VEC>(c, hi, true, &base_n, &w);
                    const unsigned r = (unsigned)top_k - base_n;
                    if (one_key) {
                        w += r * row_weight(c, ord2f(lo));
                    } else {
                        weigh();
                        uint32_t v;
                        unsigned n = base_n, n_at;
                        if (select(kByKey, lo, hi, goal, 0u, 0, &v, &n, &w, &n_at))
                            w += ((unsigned)top_k - n) * row_weight(c, ord2f(v));
                        else
                            for (int i = 0; i < (int)list_n; ++i) w += s_w[i];
                    }
                    goal.by_mass = true;
                    goal.rank = 0;
                    goal.lo = goal.hi = scale_mass(top_p, w, true);
                    // It lies at the k-th token or before it: from the same lo on, only
                    // the top k and the bracket's list are summed, which the weights'
                    // unit has room for (a whole row of them it may not have).
                    guess_lo = guess_hi = 0;
                    p_exact = true;
                    narrow(goal);
                }
            }
            if (one_key) {
                // one logit fills the bracket: how many of its tokens, lowest ids first
                const unsigned long long wt = row_weight(c, ord2f(lo));
                unsigned n_at;
                unsigned long long w;
                row_above<In, VEC>(c, lo, false, &n_at, &w);
                unsigned r = n_at - base_n;
                if (goal.by_mass) {
                    auto until = [&](unsigned long long x) -> unsigned {
                        if (!wt) return r;
                        return (unsigned)min((unsigned long long)r,
                                             (x - min(base_w, x) + wt - 1) / wt);
                    };
                    if (until(goal.lo) != until(goal.hi)) {
                        refine();
                        set_goal();
                    }
                    r = until(goal.hi);
                }
                if (by_k) r = min(r, (unsigned)top_k - base_n);
                r = max(r, 1u);
                t = lo;
                kept = base_n + r;
                if (r < n_at - base_n) {
                    // the id of the r-th lowest among the equals
                    int a = -1, b = j.V - 1;
                    while (b - a > 1) {
                        const int mid = a + (b - a) / 2;
                        unsigned n = 0;
                        each8<In, VEC>(c, [&](int v0, const float (&f)[8]) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) n += row_key(f[i]) == t && v0 + i <= mid;
                        });
                        if (cta_count(c, n) >= r)
                            b = mid;
                        else
                            a = mid;
                    }
                    id_cut = b;
                }
            } else {
                if (!have_blocks) weigh();
                const uint32_t end = hi ? hi : row_key(c.m) + 1;
                unsigned n = base_n, n_at = 0;
                unsigned long long w = base_w;
                t = lo;
                kept = base_n + list_n;
                // tokens of the boundary's key until the goal, lowest ids first
                auto until = [&](const Goal &g, unsigned long long wt) -> unsigned {
                    if (!g.by_mass) return g.rank - n;
                    if (!wt) return n_at;
                    return (unsigned)min((unsigned long long)n_at,
                                         (g.hi - min(w, g.hi) + wt - 1) / wt);
                };
                unsigned r = 0xFFFFFFFFu;
                if (select(kByKey, lo, end, goal, 0u, 0, &t, &n, &w, &n_at)) {
                    const unsigned long long wt = row_weight(c, ord2f(t));
                    if (goal.lo != goal.hi && goal.by_mass && wt &&
                        (goal.lo - min(w, goal.lo) + wt - 1) / wt !=
                            (goal.hi - min(w, goal.hi) + wt - 1) / wt) {
                        refine();
                        set_goal();
                        weigh();
                    }
                    r = max(until(goal, wt), 1u);
                    kept = n + min(r, n_at);
                    if (by_k && p_exact) kept = min(kept, (unsigned)top_k);
                } else {
                    // (the goal is past the list's end: fewer than k finite
                    // logits, or min-p's boundary comes first)
                    n = kept;
                    w = base_w;
                    unsigned long long l = 0;
                    for (int i = c.tid; i < (int)list_n; i += kRwThreads) l += s_w[i];
                    w += cta_mass(c, l);
                    n_at = 0;
                }
                if (by_k && by_p && !p_exact) {
                    // the same over the top k, for p of their mass
                    const unsigned long long wt = n_at ? row_weight(c, ord2f(t)) : 0;
                    const unsigned long long M = w + (n_at ? min(r, n_at) * wt : 0);
                    Goal g;
                    g.by_mass = true;
                    g.rank = 0;
                    g.lo = g.hi = scale_mass(top_p, M, true);
                    uint32_t tp;
                    unsigned pn = 0, p_at;
                    unsigned long long pw = 0;
                    if (select(kByKey, lo, end, g, 0u, 0, &tp, &pn, &pw, &p_at)) {
                        n = pn;
                        w = pw;
                        const unsigned all_at = n_at;
                        n_at = p_at;
                        const unsigned rp = max(until(g, row_weight(c, ord2f(tp))), 1u);
                        if (tp > t || r == 0xFFFFFFFFu || rp < r) {
                            r = rp;
                            kept = pn + min(rp, p_at);
                        } else {
                            n_at = all_at;
                        }
                        t = tp;
                    }
                }
                if (r < n_at) {
                    // the id of the r-th lowest among the boundary's equals
                    Goal g;
                    g.by_mass = false;
                    g.rank = r;
                    g.lo = g.hi = 0;
                    uint32_t id;
                    unsigned in = 0, i_at;
                    unsigned long long iw = 0;
                    select(kIdsOfKey, 0u, (uint32_t)j.V, g, t, 0, &id, &in, &iw, &i_at);
                    id_cut = (int)id;
                }
            }
            // min-p cuts at a logit, with all its equals
            if (t < key_min) {
                unsigned long long w;
                t = key_min;
                id_cut = j.V;
                if (hi && key_min >= hi) have_blocks = false;
                if (listed) {
                    unsigned n = 0;
                    for (int i = c.tid; i < (int)list_n; i += kRwThreads)
                        n += pair_key(s_list[i]) >= t;
                    kept = cta_count(c, n);
                } else {
                    row_above<In, VEC>(c, t, false, &kept, &w);
                }
            }
        }
    }

    // ---- the draw
    const bool all = !filtered;  // every finite logit is kept
    auto is_kept = [&](float x, int id) {
        const uint32_t k = row_key(x);
        return all ? x > -INFINITY : k > t || (k == t && id <= id_cut);
    };
    // At the ends of u the answer is the first or the last kept token of any
    // weight at all (above the least double), however small.
    int end_id = -1;
    if (u == 0.f || u == 1.f) {
        int best = u == 0.f ? 0x7FFFFFFF : -1;
        auto see = [&](float x, int id) {
            if (((double)x - (double)c.m) / (double)T > -745.0)
                best = u == 0.f ? min(best, id) : max(best, id);
        };
        if (listed) {
            for (int i = c.tid; i < (int)list_n; i += kRwThreads) {
                const float x = ord2f(pair_key(s_list[i]));
                if (is_kept(x, pair_id(s_list[i]))) see(x, pair_id(s_list[i]));
            }
        } else {
            each8<In, VEC>(c, [&](int v0, const float (&f)[8]) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (is_kept(f[i], v0 + i)) see(f[i], v0 + i);
            });
        }
        best = u == 0.f ? __reduce_min_sync(0xFFFFFFFFu, best)
                        : __reduce_max_sync(0xFFFFFFFFu, best);
        __syncthreads();
        if (c.lane == 0) sh.cnt[c.warp] = (unsigned)best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRwWarps; ++i)
            best = u == 0.f ? min(best, (int)sh.cnt[i]) : max(best, (int)sh.cnt[i]);
        end_id = best;
        __syncthreads();
    }
    auto kept_at = [&](int i, uint32_t *x) {
        const int id = pair_id(s_list[i]);
        *x = (uint32_t)id;
        return is_kept(ord2f(pair_key(s_list[i])), id);
    };
    if (listed) {
        unsigned long long M = 0;
        uint32_t id;
        for (int i = c.tid; i < (int)list_n; i += kRwThreads)
            if (kept_at(i, &id)) M += s_w[i];
        M = cta_mass(c, M);
        id = (uint32_t)end_id;
        if (end_id < 0) {
            // the first id whose running weight exceeds u M
            Goal g;
            g.by_mass = true;
            g.rank = 0;
            g.lo = g.hi = min(scale_mass(u, M, false), M - 1) + 1;
            unsigned n = 0, n_at;
            unsigned long long w = 0;
            select(kKeptIds, 0u, (uint32_t)j.V, g, t, id_cut, &id, &n, &w, &n_at);
        }
        for (int i = c.tid; i < (int)list_n; i += kRwThreads)
            if ((uint32_t)pair_id(s_list[i]) == id) drawn((int)id, ord2f(pair_key(s_list[i])), M);
        return;
    }
    // Sums of kept weights over blocks of ids, one warp a block.
    const int blocks = (j.V + kIdBlock - 1) / kIdBlock;
    auto kept_weight = [&](float x, int id) -> unsigned long long {
        return is_kept(x, id) ? row_weight(c, x) : 0;
    };
    __syncthreads();
    if (have_blocks) {
        // (the masses above the list are there: the list's own kept tokens are missing)
        uint32_t id;
        for (int i = c.tid; i < (int)list_n; i += kRwThreads)
            if (kept_at(i, &id)) atomicAdd(&s_block[id / kIdBlock], s_w[i]);
    } else if (all && !c.top_inf) {
        unsigned long long none;
        double f;
        if (sizeof(In) == 2) row_table(c, s_tab);
        row_split<In, VEC>(c, -FLT_MAX, -FLT_MAX, s_tab, s_list, s_block, &kept, &none, &f);
    } else {
        unsigned finite = 0;
        WeightQueue q;
        q.init(c);
        for (int b = c.warp; b < blocks; b += kRwWarps) {
            for (int k = 0; k < kIdBlock / kIdStep; ++k) {
                const int v0 = b * kIdBlock + k * kIdStep + c.lane * 8;
                float f[8];
                load8<In, VEC>(c, v0, f);
                if (__any_sync(0xFFFFFFFFu, all || max8(f) >= ord2f(t))) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        q.put(c, f[i], is_kept(f[i], v0 + i));
                        finite += f[i] > -INFINITY;
                    }
                }
            }
            const unsigned long long w = warp_sum64(q.take(c));
            if (c.lane == 0) s_block[b] = w;
        }
        if (all) kept = cta_count(c, finite);
    }
    __syncthreads();
    // each thread takes consecutive blocks
    const int each = (blocks + kRwThreads - 1) / kRwThreads;
    unsigned long long own = 0;
    for (int i = 0; i < each; ++i) {
        const int b = c.tid * each + i;
        if (b < blocks) own += s_block[b];
    }
    const unsigned long long M = cta_mass(c, own);
    const unsigned long long g = min(scale_mass(u, M, false), M - 1);
    unsigned long long run = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long a = __shfl_up_sync(0xFFFFFFFFu, run, d);
        if (c.lane >= d) run += a;
    }
    __syncthreads();
    if (c.lane == 31) sh.mass[c.warp] = run;
    __syncthreads();
    for (int i = 0; i < c.warp; ++i) run += sh.mass[i];
    if (run > g && run - own <= g) {  // exactly one thread
        unsigned long long at = run - own;
        int b = c.tid * each;
        while (at + s_block[b] <= g) at += s_block[b++];
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
        unsigned long long at = sh.base;
        for (int k = 0; k < kIdBlock / kIdStep; ++k) {
            const int v0 = sh.pick * kIdBlock + k * kIdStep + c.lane * 8;
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
            const unsigned long long step = __shfl_sync(0xFFFFFFFFu, before, 31);
            before += at - sum;
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
            at += step;
            if (at > g) break;
        }
    }
}

constexpr size_t kRowsSmem = (size_t)(2 * kTabHalf + kListCap + kMaxBlocks) * 8 + sizeof(Digits);
static_assert(2 * kTabHalf >= kListCap, "the list's weights take the table's place");

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
