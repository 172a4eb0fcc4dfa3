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
// two a SM, take a fraction of it) lists those near the boundary, sums those
// above exactly, by blocks of ids for the draw, and those below in fp32.  The
// list is sorted, and the boundary is an entry of it.
#include <float.h>
#include <math.h>

#include "sv_common.cuh"
#include "sv_rows.cuh"

namespace sv {

constexpr int kRwThreads = 512;
constexpr int kRwWarps = kRwThreads / 32;
constexpr int kListCap = 4096;
constexpr int kBins = 2048;        // of 1/32 in log2 of the weight
constexpr float kBinsPer = 32.f;
constexpr int kSampled = kRwThreads * 16;
constexpr int kIdBlock = 256;      // ids of one warp's block: 8 a lane
static_assert(kRowsMaxV / kIdBlock <= kListCap, "block sums share the list's memory");

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

struct RowShared {
    float queue[kRwWarps][64];
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

// Visit the row in steps of 8 logits a thread: f(v0, logits).  Every lane of a
// warp takes part in every step (logits past the row's end are -inf).
template <typename In, bool VEC, typename F>
__device__ __forceinline__ void each8(const RowCtx &c, F f)
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
__device__ float row_first(RowCtx &c, double *mass, int *top_id, float from,
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
        if (c.lane == 0) c.sh->cnt[0][c.warp] = (unsigned)best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRwWarps; ++i) best = min(best, (int)c.sh->cnt[0][i]);
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
    __device__ __forceinline__ void init(RowCtx &c)
    {
        buf = c.sh->queue[c.warp];
        n = 0;
        sum = 0;
    }
    __device__ __forceinline__ void put(const RowCtx &c, float x, bool on)
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
    __device__ __forceinline__ unsigned long long take(const RowCtx &c)
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
__device__ void row_above(RowCtx &c, uint32_t k, bool want_mass, unsigned *cnt,
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
__device__ unsigned row_collect(RowCtx &c, uint32_t lo, uint32_t hi, unsigned long long *list)
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

// The row in three by key: below lo its mass in fp32 (`tail`, within kTailEps,
// in units of the maximum's weight), from lo to hi the list, from hi on exact
// masses of blocks of 256 ids (`block`) and the count.  Returns the length of
// the list (of which the first kListCap are there).
template <typename In, bool VEC>
__device__ unsigned row_split(RowCtx &c, uint32_t lo, uint32_t hi, unsigned long long *list,
                              unsigned long long *block, unsigned *above, double *tail)
{
    const float flo = ord2f(lo), fhi = ord2f(hi);
    __syncthreads();
    if (c.tid == 0) c.sh->list_n = 0;
    __syncthreads();
    const int blocks = (c.V + kIdBlock - 1) / kIdBlock;
    WeightQueue q;
    q.init(c);
    unsigned n = 0;
    float s = 0.f;
    double total = 0.0;
    int steps = 0;
    constexpr int kDeep = 2;  // blocks in flight
    for (int b0 = c.warp; b0 < blocks; b0 += kDeep * kRwWarps) {
        float f[kDeep][8];
#pragma unroll
        for (int d = 0; d < kDeep; ++d)
            load8<In, VEC>(c, (b0 + d * kRwWarps) * kIdBlock + c.lane * 8, f[d]);
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int b = b0 + d * kRwWarps, v0 = b * kIdBlock + c.lane * 8;
            if (b >= blocks) break;
            const float top = max8(f[d]);
            if (__any_sync(0xFFFFFFFFu, top >= fhi)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool on = f[d][i] >= fhi;
                    n += on;
                    q.put(c, f[d][i], on);
                }
            }
            const unsigned long long w = warp_sum64(q.take(c));
            if (c.lane == 0) block[b] = w;
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = f[d][i];
                if (x >= flo && x < fhi && x > -INFINITY) {
                    const unsigned at = atomicAdd(&c.sh->list_n, 1u);
                    if (at < (unsigned)kListCap) list[at] = pair_of(row_key(x), v0 + i);
                }
                t[i] = x < flo ? ex2f((x - c.m) * c.ch) : 0.f;
            }
            s += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
            if (++steps == 8) {
                total += (double)s;
                s = 0.f;
                steps = 0;
            }
        }
    }
    total = warp_sumd(total + (double)s);
    if (c.lane == 0) c.sh->dred[c.warp] = total;
    *above = cta_count(c, n);
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < kRwWarps; ++i) z += c.sh->dred[i];
    *tail = z;
    __syncthreads();
    return c.sh->list_n;
}

// Sort list[0 .. n) downwards (bitonic; padded to a power of two with zeros).
// Stages of distance 32 and less stay within a warp's 64 entries.
__device__ void list_sort(const RowCtx &c, unsigned long long *list, unsigned n)
{
    unsigned size = 64;
    while (size < n) size *= 2;
    for (unsigned i = n + c.tid; i < size; i += kRwThreads) list[i] = 0;
    __syncthreads();
    for (unsigned k = 2; k <= size; k *= 2) {
        for (unsigned d = k / 2; d > 0; d /= 2) {
            for (unsigned p = c.tid; p < size / 2; p += kRwThreads) {
                const unsigned i = 2 * p - (p & (d - 1)), o = i + d;
                const unsigned long long a = list[i], b = list[o];
                if ((a < b) == ((i & k) == 0)) {
                    list[i] = b;
                    list[o] = a;
                }
            }
            if (d > 32 || (d == 1 && k >= 64))
                __syncthreads();
            else
                __syncwarp();
        }
    }
    __syncthreads();
}

// Running sums of the sorted list's weights, inclusive, to sum[0 .. n).
__device__ void list_sums(RowCtx &c, const unsigned long long *list, unsigned long long *sum,
                          unsigned n)
{
    const unsigned each = (n + kRwThreads - 1) / kRwThreads, from = c.tid * each;
    unsigned long long own = 0;
    for (unsigned i = from; i < min(from + each, n); ++i) {
        own += row_weight(c, ord2f(pair_key(list[i])));
        sum[i] = own;
    }
    unsigned long long run = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long a = __shfl_up_sync(0xFFFFFFFFu, run, d);
        if (c.lane >= d) run += a;
    }
    const int par = c.par;
    c.par ^= 1;
    if (c.lane == 31) c.sh->mass[par][c.warp] = run;
    __syncthreads();
    for (int i = 0; i < c.warp; ++i) run += c.sh->mass[par][i];
    run -= own;
    for (unsigned i = from; i < min(from + each, n); ++i) sum[i] += run;
    __syncthreads();
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
    unsigned long long *s_w = rows_smem;              // [kListCap] running weights
    unsigned long long *s_list = s_w + kListCap;      // [kListCap] pairs
    unsigned long long *s_block = s_list + kListCap;  // [kListCap] masses of id blocks
    unsigned *s_hist = reinterpret_cast<unsigned *>(s_w);       // [kBins], before the list
    float *s_tail = reinterpret_cast<float *>(s_hist + kBins);  // [kBins]

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
        // Counts from the top and masses from the bottom, four bins a thread.
        const int b = 4 * c.tid;
        unsigned n[4];
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            n[i] = s_hist[b + i];
            w[i] = (float)n[i] * ex2f(-((float)(b + i) + 0.5f) / kBinsPer);
        }
        unsigned cs = n[0] + n[1] + n[2] + n[3];
        float ws = (w[0] + w[1]) + (w[2] + w[3]);
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
        for (int i = 0; i < kRwWarps; ++i) {
            if (i < c.warp) {
                cs += sh.cnt[0][i];
                ws += sh.fred[i];
            }
            s_all += sh.fred[i];
        }
#pragma unroll
        for (int i = 3; i >= 0; --i) {
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
        for (int b = 4 * c.tid + 3; b >= 4 * c.tid; --b)
            if (past(b)) best = min(best, b);
        best = __reduce_min_sync(0xFFFFFFFFu, best);
        __syncthreads();
        if (c.lane == 0) sh.cnt[0][c.warp] = (unsigned)best;
        __syncthreads();
        for (int i = 0; i < kRwWarps; ++i) best = min(best, (int)sh.cnt[0][i]);
        return best;
    };
    const bool bins = sampled && s_max > -INFINITY && s_max < INFINITY;
    auto bin_end = [&](int b) {  // the logit at which bin b - 1 ends and b starts
        return b >= kBins - 1 ? -INFINITY : s_max - (float)b / kBinsPer / c.ch;
    };
    // surely (to several deviations) past the boundary, and surely before it;
    // rest: the mass that top-p leaves out, in the sample's terms
    auto guess = [&](float rest, float *from, float *to) {
        int lo = kBins - 1, hi = 0;
        if (by_k) {
            const float want = (float)top_k / per, off = 4.f * sqrtf(want) + 8.f;
            lo = first_bin([&](int b) { return (float)s_hist[b] >= want + off; });
            hi = first_bin([&](int b) { return (float)s_hist[b] >= want - off; });
        } else if (by_p) {
            lo = first_bin([&](int b) { return s_tail[b] <= 0.95f * rest; });
            hi = first_bin([&](int b) { return s_tail[b] <= 1.05f * rest; });
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
        guess((1.f - top_p) * s_all, &g_lo, &g_hi);
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
    // entries of the list whose running weight, with the mass above, is below x
    auto below = [&](unsigned long long x) {
        unsigned n = 0;
        for (int i = c.tid; i < (int)list_n; i += kRwThreads) n += base_w + s_w[i] < x;
        return cta_count(c, n);
    };

    // ---- the boundary: the last kept token's key t and id (id_cut), and the
    // number of kept tokens
    uint32_t t = key_min;
    int id_cut = j.V;
    unsigned kept = 0, kept_list = 0;  // all; those in the list, its first ones
    if (filtered) {
        // is what the list starts from past the boundary?
        auto try_list = [&](uint32_t from) {
            bool enough = from <= lo || (by_k && list_n >= (unsigned)top_k);
            if (!enough && goal.by_mass) {
                unsigned long long w = 0;
                for (int i = c.tid; i < (int)list_n; i += kRwThreads)
                    w += row_weight(c, ord2f(pair_key(s_list[i])));
                enough = goal.reached(0, cta_mass(c, w)) == 1;
            }
            if (enough) {
                lo = min(from, lo);
                listed = true;
            }
        };
        if (collect) try_list(g_lo == -INFINITY ? kKeyNegInf + 1 : row_key(g_lo));
        if (!listed && bins && !c.top_inf) {
            // again, with the row's maximum and mass in place of the sample's
            const float up = exp2f(fminf((c.m - s_max) * c.ch, 100.f));
            guess((1.f - top_p) * (float)z * up / per, &g_lo, &g_hi);
            guess_lo = max(row_key(g_lo), lo);
            guess_hi = row_key(g_hi);
            const float x = ord2f(guess_lo);
            if (tokens_from(x) < 0.9f * kListCap) {
                list_n = row_collect<In, VEC>(c, guess_lo, 0, s_list);
                if (list_n <= (unsigned)kListCap) try_list(guess_lo);
            } else if (goal.by_mass && guess_hi > guess_lo && z_known) {
                double tail;
                unsigned above;
                list_n = row_split<In, VEC>(c, guess_lo, guess_hi, s_list, s_block, &above, &tail);
                if (list_n <= (unsigned)kListCap) {
                    const int blocks = (j.V + kIdBlock - 1) / kIdBlock;
                    unsigned long long a = 0, l = 0;
                    for (int i = c.tid; i < blocks; i += kRwThreads) a += s_block[i];
                    for (int i = c.tid; i < (int)list_n; i += kRwThreads)
                        l += row_weight(c, ord2f(pair_key(s_list[i])));
                    a = cta_mass(c, a);
                    l = cta_mass(c, l);
                    // the row's mass again: only the tail is not exact
                    const double ts = ldexp(tail, c.S);
                    const unsigned long long old_lo = zlo, old_hi = zhi;
                    zlo = a + l + (unsigned long long)(ts * (1.0 - kTailEps));
                    zhi = a + l + (unsigned long long)(ts * (1.0 + kTailEps)) + 1;
                    set_goal();
                    if (a < goal.lo && a + l >= goal.hi && guess_lo >= lo) {
                        lo = guess_lo;
                        hi = guess_hi;
                        base_n = above;
                        base_w = a;
                        have_blocks = true;
                    } else {
                        zlo = max(zlo, old_lo);
                        zhi = min(zhi, old_hi);
                        set_goal();
                    }
                }
            }
        }
        if (!listed && !by_k && !by_p) {
            // min-p alone needs no list: its boundary is known
            unsigned long long w;
            list_n = 0;
            row_above<In, VEC>(c, key_min, false, &kept, &w);
        } else {
            if (!listed && !have_blocks) {
                narrow(goal);
                if (by_k && by_p) {
                    // the mass of the top k, and with it the boundary of p
                    unsigned long long w;
                    row_above<In, VEC>(c, hi, true, &base_n, &w);
                    const unsigned r = (unsigned)min(top_k, 0x7FFFFFFF) - base_n;
                    unsigned long long M;
                    if (one_key) {
                        M = w + r * row_weight(c, ord2f(lo));
                    } else {
                        list_sort(c, s_list, list_n);
                        list_sums(c, s_list, s_w, list_n);
                        const unsigned at = min(r, list_n);
                        M = w + (at ? s_w[at - 1] : 0);
                    }
                    Goal g;
                    g.by_mass = true;
                    g.rank = 0;
                    g.lo = g.hi = scale_mass(top_p, M, true);
                    goal = g;
                    lo = kKeyNegInf + 1;
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
                list_sort(c, s_list, list_n);
                list_sums(c, s_list, s_w, list_n);
                unsigned n = list_n;
                if (by_k) n = min(n, (unsigned)top_k - base_n);
                if (by_k && by_p && !p_exact) {
                    // (the list starts at the maximum here)
                    n = min(n, below(scale_mass(top_p, s_w[n - 1], true)) + 1);
                } else if (by_p) {
                    if (below(goal.lo) != below(goal.hi)) {
                        refine();
                        set_goal();
                    }
                    n = min(n, below(goal.hi) + 1);
                }
                // min-p cuts at a logit, with all its equals
                unsigned m = 0;
                for (int i = c.tid; i < (int)list_n; i += kRwThreads)
                    m += pair_key(s_list[i]) >= key_min;
                m = cta_count(c, m);
                if (m < n && min_p > 0.f) {
                    n = m;
                    if (n == 0 && base_n > 0) {
                        // its boundary lies above the list
                        unsigned long long w;
                        row_above<In, VEC>(c, key_min, false, &kept, &w);
                    }
                }
                kept_list = n;
                if (n > 0) {
                    kept = base_n + n;
                    t = pair_key(s_list[n - 1]);
                    id_cut = pair_id(s_list[n - 1]);
                }
            }
            // (a bracket of one key below min-p's boundary)
            if (t < key_min) {
                unsigned long long w;
                t = key_min;
                id_cut = j.V;
                row_above<In, VEC>(c, t, false, &kept, &w);
            }
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
        auto see = [&](float x, int id) {
            if (((double)x - (double)c.m) / (double)T > -745.0)
                best = u == 0.f ? min(best, id) : max(best, id);
        };
        if (listed) {
            for (int i = c.tid; i < (int)kept_list; i += kRwThreads)
                see(ord2f(pair_key(s_list[i])), pair_id(s_list[i]));
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
        if (c.lane == 0) sh.cnt[0][c.warp] = (unsigned)best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRwWarps; ++i)
            best = u == 0.f ? min(best, (int)sh.cnt[0][i]) : max(best, (int)sh.cnt[0][i]);
        end_id = best;
        __syncthreads();
    }
    if (listed) {
        const unsigned long long M = s_w[kept_list - 1];
        const unsigned long long g = min(scale_mass(u, M, false), M - 1);
        auto weight = [&](unsigned i) { return s_w[i] - (i ? s_w[i - 1] : 0ull); };
        if (end_id < 0 && kept_list <= 512u) {
            // each kept token's running weight by id
            const unsigned i = c.tid;
            if (i < kept_list) {
                const int id = pair_id(s_list[i]);
                unsigned long long run = 0, last = 0;
                for (unsigned k = 0; k < kept_list; ++k) {
                    const unsigned long long next = s_w[k];
                    if (pair_id(s_list[k]) <= id) run += next - last;
                    last = next;
                }
                if (run > g && run - weight(i) <= g) drawn(id, ord2f(pair_key(s_list[i])), M);
            }
            return;
        }
        // running weight at most g at a, above it at b
        int a = end_id < 0 ? -1 : end_id - 1, b = end_id < 0 ? j.V - 1 : end_id;
        while (b - a > 1) {
            const int mid = a + (b - a) / 2;
            unsigned long long w = 0;
            for (unsigned i = c.tid; i < kept_list; i += kRwThreads)
                if (pair_id(s_list[i]) <= mid) w += weight(i);
            if (cta_mass(c, w) > g)
                b = mid;
            else
                a = mid;
        }
        for (unsigned i = c.tid; i < kept_list; i += kRwThreads)
            if (pair_id(s_list[i]) == b) drawn(b, ord2f(pair_key(s_list[i])), M);
        return;
    }
    // Sums of kept weights over blocks of 256 ids, one warp a block.
    const int blocks = (j.V + kIdBlock - 1) / kIdBlock;
    auto kept_weight = [&](float x, int id) -> unsigned long long {
        return is_kept(x, id) ? row_weight(c, x) : 0;
    };
    if (all) t = kKeyNegInf + 1;
    __syncthreads();
    // (the masses above the list are there already: its own tokens are missing)
    if (have_blocks && kept_list > 0) {
        for (unsigned i = c.tid; i < kept_list; i += kRwThreads)
            atomicAdd(&s_block[pair_id(s_list[i]) / kIdBlock], s_w[i] - (i ? s_w[i - 1] : 0ull));
    } else {
        unsigned finite = 0;
        WeightQueue q;
        q.init(c);
        for (int b = c.warp; b < blocks; b += kRwWarps) {
            float f[8];
            load8<In, VEC>(c, b * kIdBlock + c.lane * 8, f);
            if (__any_sync(0xFFFFFFFFu, max8(f) >= ord2f(t))) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    q.put(c, f[i], is_kept(f[i], b * kIdBlock + c.lane * 8 + i));
                    finite += f[i] > -INFINITY;
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
    if (c.lane == 31) sh.mass[c.par][c.warp] = run;
    __syncthreads();
    for (int i = 0; i < c.warp; ++i) run += sh.mass[c.par][i];
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

constexpr size_t kRowsSmem = (size_t)kListCap * 24;

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
