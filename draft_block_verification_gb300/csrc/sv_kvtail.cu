// sv_kvtail.cu -- attention over what each sequence has behind its group's shared
// pages (all of it where nothing is shared), and the join with what the prefix
// kernel left.
//
// Few query rows read many tokens here: a sequence's new tokens times the heads
// that share a cache head, 4 to some hundreds.  Up to about 16 rows reading the
// cache bounds it, if only work starts and ends quickly and there is enough of it
// at once.  So the work is cut into tasks of one warp, which share nothing: a
// sequence's cache head, up to 16 of its query rows, a range of its tokens.  Products
// are warp-wide (mma.sync): a task starts with the load of its queries and ends with
// a store, with no tensor memory to fill and drain between (the kernel of
// sv_kvattn.cu, on tcgen05, takes 7 to 20 us a unit for that, one CTA an SM).
//
//   S^T [16 tokens x 8 rows] += K Q^T
//   O^T [16 elements x 8 rows] += V^T P^T    (m16n8k16, fp16 both)
// An e4m3 byte is exact in fp16, and so is a query's element down to 2^-32 of the
// row's largest (which is brought to 2^14); a weight is rounded to fp16.  (Products of
// e4m3 by itself are converted to these by the compiler, every operand each time.)
// Rows are the products' columns: a single token pays for eight, and what it takes to
// fetch and convert is shared by up to twice eight.  A product's place in the head is
// free to choose, the same for both operands; so a lane's queries are D / 4
// consecutive elements, its outputs D / 8, and only the weights cross the warp
// between the products (a transposition of 8 x 8, movmatrix).
//
// Weights are 2^(y - M + 8), M within 2^3 of the running maximum, times the value
// scale against a power of two of the warp's, which stays within 2^3 of the scale;
// where it would not, O moves to the new scale, in fp32.  So a weight reaches 2^15
// at most, has fp16's 11 bits down to 2^-19 of the largest, and steps of 2^-30 of it
// below; value scales may lie any distance apart.  A score is not rounded before M is
// taken from it, but beyond kTlFar it is, as M has been: the difference of a maximum
// from itself would else be anything within half a step (16 at 2^28).
//
// What bounds it: one warp's chain of steps, some 435 instructions for 16 tokens and 16
// rows, three warps to a scheduler.  128 sequences of a token, 32 heads, 320 tokens of
// their own each, with the join of 16 pieces' sums: 43 of the call's 107 us as a graph;
// four of one token over 1,088: 17 of 33.
//
// A warp fetches its own stages of 32 tokens (TMA), two in flight.  Ranges are cut
// so that every warp of a wave has a task; ranges of the same rows join in the
// workspace, by the last to arrive, in their order.
#include <cuda_fp16.h>

#include "sv_common.cuh"
#include "sv_kv.cuh"
#include "sv_tc.cuh"

namespace sv {

constexpr int kTlTile = kTailTile;     // tokens of a stage
constexpr int kTlStages = 2;
constexpr int kTlWarps = 4;            // of a CTA, three CTAs an SM
constexpr uint32_t kTlTries = 1u << 20;
constexpr float kTlNone = -1e30f;      // maximum of no tokens
constexpr float kTlUnit = 8.f;         // log2 of the weight at M
constexpr float kTlLazy = 3.f;         // log2 of how far a weight may pass it
constexpr float kTlFar = 0x1p14f;      // maxima from which on scores are rounded first
constexpr int kTlNear = 3;             // of how far a value scale may lie from the warp's

struct TailWarp {
    uint64_t full[kTlStages];
    float2 scale[kTlStages][2];        // key's and value's, of each 16 tokens
};

// A task: sequence, cache head, rows, stages.
struct TailTask {
    int b, h, row0, rows, first, n, L, skip, z, nz;
    bool own;                          // the sequence's own tokens are read here
    int s0, s1;                        // stages of 32 tokens behind the skipped pages
    int part0;                         // counter and parts of its rows: their first
};

// The sequence that task u belongs to: the last b with unit0[b] <= u.
__device__ __forceinline__ int tail_seq(const PrefixJob &j, int u, int lane)
{
    int lo = 0, n = j.B;               // among [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) >> 5, at = lo + lane * step;
        const bool on = at < lo + n && __ldcg(j.unit0 + at) <= u;
        const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, on));  // (lane 0 is on)
        n = min(step, n - k * step);
        lo += k * step;
    }
    return lo;
}

__device__ __forceinline__ TailTask tail_task(const PrefixJob &j, int u, int lane)
{
    TailTask t;
    t.b = tail_seq(j, u, lane);
    t.first = __ldcg(j.cu + t.b);
    t.n = __ldcg(j.cu + t.b + 1) - t.first;
    t.L = __ldcg(j.kv_len + t.b);
    t.skip = __ldcg(j.skip + t.b);
    const int c = __ldcg(j.tail_stages), rows = t.n * j.G;
    const TailBlocks rb(rows);
    t.own = rows <= kTailMax;
    const int own = t.L - t.skip * j.block, all = t.own ? (own + kTlTile - 1) / kTlTile : 1;
    t.nz = (all + c - 1) / c;
    const int i = u - __ldcg(j.unit0 + t.b), q = i / t.nz;
    t.z = i - q * t.nz;
    t.h = q / rb.blocks;
    t.row0 = (q - t.h * rb.blocks) * rb.rows;
    t.rows = min(rb.rows, rows - t.row0);
    // without a mask no row sees past its own token
    const int sees = j.mask ? own : own - t.n + (t.row0 + t.rows - 1) / j.G + 1;
    const int seen = t.own ? (sees + kTlTile - 1) / kTlTile : 0;
    t.s0 = min(t.z * c, seen);
    t.s1 = min(t.s0 + c, seen);
    t.part0 = __ldcg(j.part0 + t.b) + q * t.nz;
    return t;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The low and the high two e4m3 bytes of w to fp16.
__device__ __forceinline__ void f16_of(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
        " cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ bool nan_byte(uint32_t w)
{
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// What a warp holds of 8 NT rows; a lane (g = lane / 4, c = lane % 4) of rows 2 c and
// 2 c + 1 of each eight, elements [D / 8 * g, + D / 8): o[n][i] are element 2 i of both
// rows, then element 2 i + 1.
template <int D, int NT>
struct TailSums {
    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];          // l: of this lane's tokens
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][i][k] = 0.f;
            m[n][0] = m[n][1] = kTlNone;
            l[n][0] = l[n][1] = 0.f;
        }
    }
    __device__ __forceinline__ void scale(int n, float a, float b)
    {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            o[n][i][0] *= a;
            o[n][i][1] *= b;
            o[n][i][2] *= a;
            o[n][i][3] *= b;
        }
    }
    // another's sums of eight rows, its o by get(x)
    template <typename Get>
    __device__ __forceinline__ void add(int n, float m0, float m1, float l0, float l1, Get get)
    {
        float4 x[D / 16];
        get(x);
        const float t0 = fmaxf(m[n][0], m0), t1 = fmaxf(m[n][1], m1);
        const float f0 = ex2f(m[n][0] - t0), f1 = ex2f(m[n][1] - t1);
        const float g0 = ex2f(m0 - t0), g1 = ex2f(m1 - t1);
        m[n][0] = t0;
        m[n][1] = t1;
        l[n][0] = fmaf(l[n][0], f0, l0 * g0);
        l[n][1] = fmaf(l[n][1], f1, l1 * g1);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            o[n][i][0] = fmaf(o[n][i][0], f0, x[i].x * g0);
            o[n][i][1] = fmaf(o[n][i][1], f1, x[i].y * g1);
            o[n][i][2] = fmaf(o[n][i][2], f0, x[i].z * g0);
            o[n][i][3] = fmaf(o[n][i][3], f1, x[i].w * g1);
        }
    }
};

// A lane's queries: elements [D / 4 * c, + D / 4) of row g of each eight; f: the factors
// from S to log2 units of rows 2 c and 2 c + 1.
template <int D, int NT>
__device__ __forceinline__ void tail_queries(const PrefixJob &j, const TailTask &t, int lane,
                                             uint32_t (&x)[NT][D / 8], float (&f)[NT][2])
{
    constexpr int E = D / 4;
    const int g = lane >> 2, c = lane & 3;
    const bool vec = (((uintptr_t)j.q | (uintptr_t)(j.qts * 2) | (uintptr_t)(j.qhs * 2)) & 15) == 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = n * 8 + g;
        uint32_t raw[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) raw[i] = 0u;
        if (r < t.rows) {
            const int at = t.row0 + r, tok = at / j.G;
            const uint16_t *q = j.q + (int64_t)(t.first + tok) * j.qts +
                                (int64_t)(t.h * j.G + at - tok * j.G) * j.qhs + c * E;
            if (vec) {
#pragma unroll
                for (int i = 0; i < E / 8; ++i) {
                    const uint4 v = reinterpret_cast<const uint4 *>(q)[i];
                    raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) raw[i] = q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
            }
        }
        // (as integers NaN is above infinity, and above the rest)
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            top = max(top, max((raw[i] << 16) & 0x7FFFFFFFu, raw[i] & 0x7FFF0000u));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const bool odd = top >= 0x7F800000u;    // NaN or an infinity
        // 2^e brings the largest element to [2^14, 2^15)
        const int e = top > 0 && !odd ? min(141 - (int)(top >> 23), 126) : 0;
        const float up = __int_as_float((127 + e) << 23);
        const float own = r >= t.rows ? 0.f
                          : odd       ? __int_as_float(0x7FC00000)
                                      : j.softmax_scale * 1.4426950408889634f / up;
        f[n][0] = __shfl_sync(0xFFFFFFFFu, own, 8 * c);
        f[n][1] = __shfl_sync(0xFFFFFFFFu, own, 8 * c + 4);
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                : "=r"(x[n][i])
                : "f"(__uint_as_float(raw[i] & 0xFFFF0000u) * up), "f"(__uint_as_float(raw[i] << 16) * up));
    }
}

// Which of a lane's scores count, where not every row sees every token; values of
// tokens that must not be read are cleared.  A token's value may be NaN: it is
// cleared too (0 times NaN is NaN), and its score made NaN for the rows that see it.
// Returns the hidden scores, four bits for each eight rows.
template <int D, int NT>
__device__ __forceinline__ uint32_t tail_edge(const PrefixJob &j, const TailTask &t, int pos, int lane,
                                           uint32_t (&v)[4][D / 32], float (&y)[NT][4])
{
    const int g = lane >> 2, c = lane & 3, ctx = t.L - t.n;
    uint32_t lost = 0;                          // tokens of the 16, a bit each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tk = 2 * c + (i & 1) + (i >> 1) * 8;
        bool nan = false;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) nan |= nan_byte(v[i][q]);
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, nan);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (who >> k & 0x11111111u) lost |= 1u << (2 * k + (i & 1) + (i >> 1) * 8);
        if (who >> c & 0x11111111u || pos + tk >= t.L) {
#pragma unroll
            for (int q = 0; q < D / 32; ++q) v[i][q] = 0u;
        }
    }
    uint32_t hide = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int tk = g + (k >> 1) * 8, p = pos + tk, q = p - ctx;
            const int row = n * 8 + 2 * c + (k & 1), i = (t.row0 + row) / j.G;  // its token
            bool sees = p < t.L && (q <= i || j.mask);
            if (sees && q >= 0 && j.mask && row < t.rows)
                sees = (q >> 5) < j.words &&
                       (j.mask[(int64_t)(t.first + i) * j.words + (q >> 5)] >> (q & 31) & 1);
            if (!sees)
                hide |= 1u << (4 * n + k);
            else if (lost >> tk & 1)
                y[n][k] = __int_as_float(0x7FC00000);
        }
    return hide;
}

// 16 tokens.
template <int D, int NT>
__device__ __forceinline__ void tail_step(const PrefixJob &j, const TailTask &t, const char *s_k,
                                          const char *s_v, int tok0, int pos, float2 scale, int lane,
                                          const uint32_t (&x)[NT][D / 8], const float (&cf)[NT][2],
                                          int &ref, TailSums<D, NT> &s)
{
    const int g = lane >> 2, c = lane & 3;
    constexpr int C = D / 64;                   // 16-byte pieces of a key a lane
    float y[NT][4];
    {
        uint4 k0[C], k1[C];                     // of tokens g and g + 8
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int tk = tok0 + g, chunk = c * C + i;
            const int sw = D == 128 ? tk & 7 : (tk >> 1) & 3;  // (alike for token g + 8)
            k0[i] = *reinterpret_cast<const uint4 *>(s_k + tk * D + ((chunk ^ sw) << 4));
            k1[i] = *reinterpret_cast<const uint4 *>(s_k + (tk + 8) * D + ((chunk ^ sw) << 4));
        }
        float a[2][NT][4];                      // (two chains)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) a[0][n][i] = a[1][n][i] = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * C; ++i) {
            const uint4 &p = k0[i >> 2], &q = k1[i >> 2];
            uint32_t r[4];
            f16_of(i % 4 == 0 ? p.x : i % 4 == 1 ? p.y : i % 4 == 2 ? p.z : p.w, r[0], r[2]);
            f16_of(i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w, r[1], r[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(a[i & 1][n], r, x[n][2 * i], x[n][2 * i + 1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[n][i] = a[0][n][i] + a[1][n][i];
    }
    // the values: of tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9, D / 8 elements
    uint32_t v[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tk = tok0 + 2 * c + (i & 1) + (i >> 1) * 8;
        if (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(s_v + tk * D + ((g ^ (tk & 7)) << 4));
            v[i][0] = w.x; v[i][1] = w.y; v[i][D / 32 - 2] = w.z; v[i][D / 32 - 1] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(
                s_v + tk * D + (((g >> 1) ^ ((tk >> 1) & 3)) << 4) + (g & 1) * 8);
            v[i][0] = w.x; v[i][1] = w.y;
        }
    }
    uint32_t hide = 0;
    if (__builtin_expect(pos + 16 > t.L - t.n, 0)) hide = tail_edge<D, NT>(j, t, pos, lane, v, y);
    // the value scale against the warp's
    const uint32_t bits = __float_as_uint(scale.y);
    const int e = (int)(bits >> 23) - 127;
    const float fr = __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);
    // (votes: rare branches, not predicates)
    if (__any_sync(0xFFFFFFFFu, ref - e > kTlNear || e - ref > kTlNear)) {
        // (no two scales are 2^127 apart)
        const float by = __int_as_float((127 + ref - e) << 23);
#pragma unroll
        for (int n = 0; n < NT; ++n) s.scale(n, by, by);
        ref = e;
    }
    float lv = kTlUnit + (float)(e - ref);
    float inv = __int_as_float((127 - (int)kTlUnit + ref - e) << 23);
    if (__any_sync(0xFFFFFFFFu, fr != 1.f)) {
        lv += log2f(fr);
        inv /= fr;
    }
    float z[NT][4];
    // (rounded: the scores before the maximum is taken from them, as it has been)
    auto scores = [&](bool rounded) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float u0 = cf[n][0] * scale.x, u1 = cf[n][1] * scale.x;
            const float a0 = lv - s.m[n][0], a1 = lv - s.m[n][1];
#pragma unroll
            for (int i = 0; i < 4; ++i) z[n][i] = fmaf(y[n][i], i & 1 ? u1 : u0, i & 1 ? a1 : a0);
            if (rounded)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    z[n][i] = __fsub_rn(__fmul_rn(y[n][i], i & 1 ? u1 : u0), s.m[n][i & 1]) + lv;
        }
        if (__any_sync(0xFFFFFFFFu, hide != 0))
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (hide >> (4 * n + i) & 1) z[n][i] = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            top = fmaxf(top, fmaxf(fmaxf(z[n][0], z[n][1]), fmaxf(z[n][2], z[n][3])));
        return top;
    };
    auto far = [&] {
        float m = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) m = fmaxf(m, fmaxf(fabsf(s.m[n][0]), fabsf(s.m[n][1])));
        return m >= kTlFar;
    };
    if (__builtin_expect(__any_sync(0xFFFFFFFFu, scores(false) > lv + kTlLazy || far()), 0)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float u = cf[n][r] * scale.x;
                float m = hide >> (4 * n + r) & 1 ? -INFINITY : __fmul_rn(y[n][r], u);
                if (!(hide >> (4 * n + r + 2) & 1)) m = fmaxf(m, __fmul_rn(y[n][r + 2], u));
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
                const float to = m > s.m[n][r] + kTlLazy ? m : s.m[n][r];
                f[r] = ex2f(s.m[n][r] - to);
                s.m[n][r] = to;
                s.l[n][r] *= f[r];
            }
            s.scale(n, f[0], f[1]);
        }
        scores(far());
    }
    uint32_t p[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ex2f(z[n][i]);
        s.l[n][0] = fmaf(w[0] + w[2], inv, s.l[n][0]);
        s.l[n][1] = fmaf(w[1] + w[3], inv, s.l[n][1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t pair;
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pair) : "f"(w[2 * k + 1]), "f"(w[2 * k]));
            p[n][k] = transpose8(pair);
        }
    }
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362 : 0x5140;
            uint32_t a[4];
            f16_of(__byte_perm(v[0][q], v[1][q], sel), a[0], a[1]);
            f16_of(__byte_perm(v[2][q], v[3][q], sel), a[2], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(s.o[n][2 * q + half], a, p[n][0], p[n][1]);
        }
    }
}

// Where a warp's fetches are: the pages of its task, 32 and the next 32.
struct TailFetch {
    int w0, page, npage;
    float ks, vs, nks, nvs;
    __device__ __forceinline__ void window(const PrefixJob &j, const TailTask &t, int w, int lane,
                                           int &pg, float &a, float &b)
    {
        const int last = (t.L + j.block - 1) >> (31 - __clz(j.block));
        pg = w + lane < last ? j.table[(int64_t)t.b * j.cols + w + lane] : -1;
        if (w + lane < last && (pg < 0 || pg >= j.pages)) {
            latch(j.err, SV_ERR_DEVICE_BOUNDS);
            pg = -1;
        }
        a = b = 1.f;
        if (pg >= 0) {
            const int64_t ph = (int64_t)pg * j.H + t.h;
            a = j.scale[0][ph];
            b = fminf(fmaxf(j.scale[1][ph], 0x1p-60f), 0x1p60f);
        }
    }
    __device__ __forceinline__ void start(const PrefixJob &j, const TailTask &t, int lane)
    {
        w0 = (t.skip + ((t.s0 * kTlTile) >> (31 - __clz(j.block)))) & ~31;
        window(j, t, w0, lane, page, ks, vs);
        window(j, t, w0 + 32, lane, npage, nks, nvs);
    }
    // stage s of the task to place `st`
    template <int D>
    __device__ __forceinline__ void fetch(const PrefixJob &j, const TailTask &t, int s, int st,
                                          TailWarp *sh, char *ring, const CUtensorMap &map_k,
                                          const CUtensorMap &map_v, int lane)
    {
        const int shift = 31 - __clz(j.block), at = s * kTlTile;
        const int p0 = t.skip + (at >> shift), off = at & (j.block - 1);
        if (p0 >= w0 + 32) {
            w0 += 32;
            page = npage;
            ks = nks;
            vs = nvs;
            window(j, t, w0 + 32, lane, npage, nks, nvs);
        }
        // lanes 0 and 1: 16 tokens each; pages of 16 are fetched by both
        const int i = p0 - w0 + (j.block == 16 ? lane & 1 : 0);
        const int a = __shfl_sync(0xFFFFFFFFu, page, i & 31), b = __shfl_sync(0xFFFFFFFFu, npage, i & 31);
        const float ka = __shfl_sync(0xFFFFFFFFu, ks, i & 31), kb = __shfl_sync(0xFFFFFFFFu, nks, i & 31);
        const float va = __shfl_sync(0xFFFFFFFFu, vs, i & 31), vb = __shfl_sync(0xFFFFFFFFu, nvs, i & 31);
        const int pg = i < 32 ? a : b;
        const int box = min(j.block, kTlTile);
        if (lane < 2) sh->scale[st][lane] = make_float2(i < 32 ? ka : kb, i < 32 ? va : vb);
        const bool copy = lane < (j.block == 16 ? 2 : 1) && pg >= 0;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, copy)) * box * D * 2;
        if (lane == 0) mbar_arrive_tx(&sh->full[st], bytes);
        __syncwarp();
        if (copy) {
            char *to = ring + st * (2 * kTlTile * D) + lane * box * D;
            auto get = [&](const CUtensorMap *map, char *dst) {
                asm volatile(
                    "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::"
                    "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
                    "l"(map), "r"(0), "r"(off), "r"(pg * j.H + t.h), "r"(smem_u32(&sh->full[st]))
                    : "memory");
            };
            get(&map_k, to);
            get(&map_v, to + kTlTile * D);
        }
        __syncwarp();
    }
};

// A task of up to 8 NT rows.  it: the warp's stages so far.
template <int D, int NT>
__device__ __forceinline__ bool tail_run(const PrefixJob &j, const TailTask &t, TailWarp *sh,
                                         char *ring, const CUtensorMap &map_k,
                                         const CUtensorMap &map_v, int lane, uint32_t &it)
{
    const int g = lane >> 2, c = lane & 3;
    TailFetch f;
    if (t.s0 < t.s1) {
        f.start(j, t, lane);
        for (int k = 0; k < kTlStages && t.s0 + k < t.s1; ++k)
            f.fetch<D>(j, t, t.s0 + k, (it + k) % kTlStages, sh, ring, map_k, map_v, lane);
    }
    TailSums<D, NT> s;
    s.clear();
    int ref = 0;
    if (t.s0 < t.s1) {
        uint32_t x[NT][D / 8];
        float cf[NT][2];
        tail_queries<D, NT>(j, t, lane, x, cf);
        for (int k = t.s0; k < t.s1; ++k, ++it) {
            const int st = it % kTlStages;
            bool ok = mbar_wait_n(&sh->full[st], (it / kTlStages) & 1, kTlTries);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) {
                latch(j.err, SV_ERR_TIMEOUT);
                return false;
            }
            const char *s_k = ring + st * (2 * kTlTile * D);
#pragma unroll 1
            for (int q = 0; q < kTlTile / 16; ++q) {
                const int pos = t.skip * j.block + k * kTlTile + q * 16;
                if (pos < t.L)
                    tail_step<D, NT>(j, t, s_k, s_k + kTlTile * D, q * 16, pos, sh->scale[st][q], lane,
                                     x, cf, ref, s);
            }
            __syncwarp();
            if (k + kTlStages < t.s1)
                f.fetch<D>(j, t, k + kTlStages, st, sh, ring, map_k, map_v, lane);
        }
    }
    const float out = __int_as_float((127 + ref - (int)kTlUnit) << 23);
#pragma unroll
    for (int n = 0; n < NT; ++n) s.scale(n, out, out);
    // ---- what the prefix kernel left of these rows, its pieces dealt to the ranges: of
    // the group's span and of the sequence's
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        if (which ? t.own : t.skip == 0) continue;
        const PrefixSpan gr = j.span[which ? j.groups + t.b : j.seq_group[t.b]];
        const int blocks = (gr.rows + gr.block - 1) / gr.block;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            // (rows 2 c and 2 c + 1 may lie in different units)
            const int row = n * 8 + 2 * c, at = (t.first - gr.first) * j.G + t.row0 + row;
            const int2 none = make_int2(0, -1);
            int unit[2];
            int2 cc[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bool live = row + r < t.rows;
                unit[r] = gr.unit0 + t.h * blocks + (live ? (at + r) / gr.block : 0);
                cc[r] = live ? __ldcg(j.unit_ctas + unit[r]) : none;
                if (!unit_known(cc[r].x, cc[r].y, j.prefix_ctas)) cc[r] = none;
            }
            const int most = max(cc[0].y - cc[0].x, cc[1].y - cc[1].x);
#pragma unroll 2
            for (int k = t.z; k <= most; k += t.nz) {
                // (every load at once, of parts that do not count too)
                const float *p[2];
                float m1[2], l1[2];
                bool on[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int cta = min(cc[r].x + k, j.prefix_ctas - 1), slot = 2 * cta + (k == 0 ? 1 : 0);
                    const bool whole = cc[r].x == cc[r].y;
                    const size_t i = whole ? (size_t)2 * j.prefix_ctas + unit[r] : (size_t)slot;
                    const int in = (at + r) & (gr.block - 1);
                    p[r] = j.part + i * ((size_t)kPrefixRows * (D + 2));
                    on[r] = (__ldcg(j.part_unit + slot) == unit[r] || whole) && cc[r].x + k <= cc[r].y;
                    m1[r] = __ldcg(p[r] + (size_t)D * kPrefixRows + in);
                    l1[r] = __ldcg(p[r] + (size_t)(D + 1) * kPrefixRows + in);
                    p[r] += 4 * in + (size_t)g * (D / 8) * kPrefixRows;
                }
                s.add(n, on[0] ? m1[0] : kTlNone, on[1] ? m1[1] : kTlNone, on[0] && g == 0 ? l1[0] : 0.f,
                      on[1] && g == 0 ? l1[1] : 0.f, [&](float4 (&x)[D / 16]) {
#pragma unroll
                          for (int i = 0; i < D / 32; ++i) {
                              const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
                              float4 a = __ldcg(reinterpret_cast<const float4 *>(p[0]) + i * kPrefixRows);
                              float4 b = __ldcg(reinterpret_cast<const float4 *>(p[1]) + i * kPrefixRows);
                              if (!on[0]) a = zero;
                              if (!on[1]) b = zero;
                              x[2 * i] = make_float4(a.x, b.x, a.y, b.y);
                              x[2 * i + 1] = make_float4(a.z, b.z, a.w, b.w);
                          }
                      });
            }
            __syncwarp();
        }
    }
    // ---- ranges of the same rows: the last to arrive joins them
    if (t.nz > 1) {
        constexpr int kStride = (D / 16 + 1) * 32;  // of eight rows, in float4
        float4 *part = reinterpret_cast<float4 *>(j.tail_part) +
                       (size_t)t.part0 * (kTailTiles * kStride) + lane;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float4 *to = part + (size_t)t.z * (kTailTiles * kStride) + n * kStride;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                to[i * 32] = make_float4(s.o[n][i][0], s.o[n][i][1], s.o[n][i][2], s.o[n][i][3]);
            to[D / 16 * 32] = make_float4(s.m[n][0], s.m[n][1], s.l[n][0], s.l[n][1]);
        }
        __threadfence();
        __syncwarp();
        unsigned seen = 0;
        if (lane == 0) seen = atomicAdd(j.tail_arrived + t.part0, 1u);
        seen = __shfl_sync(0xFFFFFFFFu, seen, 0);
        if (seen != (unsigned)(t.nz - 1)) return true;
        __threadfence();
        s.clear();
#pragma unroll 1
        for (int z = 0; z < t.nz; ++z)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4 *from = part + (size_t)z * (kTailTiles * kStride) + n * kStride;
                const float4 x = __ldcg(from + D / 16 * 32);
                s.add(n, x.x, x.y, x.z, x.w, [&](float4 (&o)[D / 16]) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) o[i] = __ldcg(from + i * 32);
                });
            }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float l = s.l[n][r];
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, k);
            const int row = n * 8 + 2 * c + r;
            if (row >= t.rows) continue;
            const int at = t.row0 + row, tok = at / j.G;
            const int64_t to = (int64_t)(t.first + tok) * j.Hq + t.h * j.G + (at - tok * j.G);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint32_t w[D / 16];
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                    : "=r"(w[i]) : "f"(s.o[n][i][2 + r] * inv), "f"(s.o[n][i][r] * inv));
            uint4 *dst = reinterpret_cast<uint4 *>(j.out + to * D + g * (D / 8));
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            if (j.lse && g == 0)
                j.lse[to] = l == 0.f ? -INFINITY : (s.m[n][r] + log2f(l)) * 0.6931471805599453f;
        }
    return true;
}

template <int D>
__global__ void __launch_bounds__(kTlWarps * 32, 3)
tail_kernel(const __grid_constant__ PrefixJob j, const __grid_constant__ CUtensorMap map_k,
            const __grid_constant__ CUtensorMap map_v)
{
    extern __shared__ char tl_raw[];
    __shared__ TailWarp shared[kTlWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    TailWarp *sh = &shared[warp];
    char *ring = tl_raw + ((1024 - (smem_u32(tl_raw) & 1023)) & 1023) +
                 warp * (kTlStages * 2 * kTlTile * D);
    if (lane == 0) {
        for (int i = 0; i < kTlStages; ++i) mbar_init(&sh->full[i], 1);
        mbar_fence_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    const int tasks = __ldcg(j.unit0 + j.B), step = gridDim.x * kTlWarps;
    uint32_t it = 0;
    bool ok = true;
    // (neighbours in the list, which share a cache head, run side by side)
    for (int u = blockIdx.x * kTlWarps + warp; u < tasks && ok; u += step) {
        const TailTask t = tail_task(j, u, lane);
        if (t.rows <= 8)
            ok = tail_run<D, 1>(j, t, sh, ring, map_k, map_v, lane, it);
        else
            ok = tail_run<D, 2>(j, t, sh, ring, map_k, map_v, lane, it);
    }
    // after a wait that ran out: copies still in flight land before the exit
    if (!ok)
        for (int i = 0; i < kTlStages; ++i)
            mbar_wait_n(&sh->full[(it + i) % kTlStages], ((it + i) / kTlStages) & 1, 1u << 12);
}

constexpr size_t tail_smem(int D)
{
    return 1024 + (size_t)kTlWarps * kTlStages * 2 * kTlTile * D;
}

size_t tail_part_bytes(int sms, int D)
{
    return (size_t)kTailParts * tail_warps(sms) * kTailTiles * (D / 16 + 1) * 128 * sizeof(float);
}

cudaError_t tail_setup()
{
    cudaError_t e = cudaFuncSetAttribute(tail_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)tail_smem(64));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(tail_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)tail_smem(128));
    return e;
}

cudaError_t tail_launch(const PrefixJob &j, int sms, cudaStream_t s)
{
    CUtensorMap mk, mv;
    const int box = j.block < kTlTile ? j.block : kTlTile;
    if (!cache_map(&mk, j.cache[0], j.D, j.block, box, j.pages, j.H) ||
        !cache_map(&mv, j.cache[1], j.D, j.block, box, j.pages, j.H))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    pdl_config(cfg, at, dim3(tail_warps(sms) / kTlWarps), dim3(kTlWarps * 32), tail_smem(j.D), s);
    return j.D == 64 ? cudaLaunchKernelEx(&cfg, tail_kernel<64>, j, mk, mv)
                     : cudaLaunchKernelEx(&cfg, tail_kernel<128>, j, mk, mv);
}

}  // namespace sv
