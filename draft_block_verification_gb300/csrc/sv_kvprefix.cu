// sv_kvprefix.cu -- attention over the paged 8-bit cache for sequences that
// share a prefix: the pages that all sequences of a group have in common are
// read once, for the query rows of the whole group.
//
// The result is that of the attention over each sequence by itself (z, w, o as
// in sv_attend.cuh).  A row's positions are cut in two, the shared pages and the
// rest; each part leaves its maximum m, its sum of weights l = sum 2^(y - m) and
// its sum of weighted values o = sum 2^(y - m) v, and
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,  M = max m_i.
//
// Four kernels:
//   prep     which pages are shared: the leading entries of the group's table
//            rows that are equal, no further than the caller's bound and the
//            tokens before each sequence's new ones.  So a bound that is too
//            large changes nothing.
//   attend   (sv_kvfar.cu) the rest of each sequence.
//   prefix   the shared pages, below.
//   combine  the join.
//
// Shape of the prefix.  All rows see all of it, so there is nothing to mask but
// the end of the last tile.  A unit is a cache head's block of up to 256 query
// rows, two times 128 (slots); a tile is 128 tokens.  Queries are the 128 rows
// of the products, a row's scores lie in one thread's registers, and maxima and
// sums need no exchange:
//   S [128 rows x 128 tokens] = Q K^T    in 8 bits: the cache's bytes as they
//       lie, the query exactly in two e4m3 parts (as in sv_attend.cuh), added up
//   O [128 rows x D]         += P V      in bf16: P from tensor memory, V's bytes
//       brought to bf16 in shared memory
// A weight is rounded to bf16, within 2^-8 of itself at any size, and a value
// times the power of two in its page's scale is exact in bf16; what the scale
// has beside that power goes into the exponent and out of the sum again (as log2
// and 1 / x).  So the scales' range needs no care.
//
// The products of a slot's tile run under the other slot's softmax:
//   tensor  S0 . . PV0 S0' PV1 S1' ...
//   slot 0    softmax     softmax
// A unit of up to 128 rows gives both slots the same queries and every other
// tile each, and joins the two at its end.  Each softmax thread holds its row's
// 128 scores; four more warps bring the values to bf16, one fetches, one issues.
//
// The running maximum moves lazily: only where a tile's maximum passes it by
// 2^8 are a row's sums rescaled.
//
// Split.  Tiles of all units laid end to end are cut into equal spans, one a
// CTA.  A unit's piece leaves its sums in the workspace, [D][256] fp32 with rows
// contiguous; the combine kernel adds a unit's pieces in the order of the CTAs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_common.cuh"
#include "sv_kv.cuh"
#include "sv_tc.cuh"

namespace sv {

constexpr int kPxTile = 128;           // tokens of a tile
constexpr int kPxRows = kPrefixRows;   // query rows of a unit, two slots of 128
constexpr int kPxK = 3, kPxV = 2;      // tiles of keys and of values in flight
constexpr int kPxRing = 8;             // tiles whose scales are kept
constexpr int kPxSoft = 8;             // softmax warps, four a slot
constexpr int kPxThreads = 512;        // + 4 converting warps, producer, issuer, 2 idle
// Registers: 128 a thread at launch; the softmax warps, which hold a row's 128
// scores, take what the others leave (256 * 184 + 256 * 72 = 512 * 128).
constexpr int kPxRegs = 128, kPxSoftRegs = 184, kPxSideRegs = 72;
static_assert(256 * kPxSoftRegs + 256 * kPxSideRegs <= kPxThreads * kPxRegs, "registers");
constexpr float kPxLazy = 8.f;         // log2 of how far a weight may pass 1
constexpr float kPxNone = -1e30f;      // maximum of no tokens

// ---------------------------------------------------------------------------
// Which pages are shared.
// ---------------------------------------------------------------------------
constexpr int kPrepCtas = 8, kPrepThreads = 512;

struct RowBlocks {
    int blocks, last;                  // row blocks of a head; the last one's cost
    __device__ __forceinline__ explicit RowBlocks(int rows)
    {
        blocks = (rows + kPxRows - 1) / kPxRows;
        const int rest = rows - (blocks - 1) * kPxRows;
        last = rest > 128 ? 2 : 1;     // one slot's tiles cost half
    }
    // of all blocks, in slots' tiles a tile
    __device__ __forceinline__ int cost() const { return 2 * (blocks - 1) + last; }
};

// One cluster: its warps take the sequences, its first CTA's the groups.
__global__ void __cluster_dims__(kPrepCtas, 1, 1) __launch_bounds__(kPrepThreads)
prefix_prep_kernel(const PrefixJob j, unsigned *counters, int n_counters)
{
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kPrepThreads / 32;
    const int shift = 31 - __clz(j.block);
    pdl_wait();
    pdl_trigger();
    if (tid == 0) s_bad = 0;
    if (blockIdx.x == 0)
        for (int i = tid; i < n_counters; i += kPrepThreads) counters[i] = 0;
    auto edge = [&](int g) { return j.cu_group ? j.cu_group[g] : g ? j.B : 0; };
    auto tokens = [&](int b, int &n, int &L) {  // false: lengths out of range
        const int first = j.cu[b], end = j.cu[b + 1];
        L = j.kv_len[b];
        n = end - first;
        return first >= 0 && end <= j.T && n >= 0 && L >= n &&
               ((L + (long long)j.block - 1) >> shift) <= j.cols;
    };
    // leading pages that sequence b has in common with its group's first
    for (int b = blockIdx.x * kWarps + warp; b < j.B; b += kPrepCtas * kWarps) {
        int lo = 0, hi = j.groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (edge(mid) <= b) lo = mid; else hi = mid;
        }
        const int b0 = max(edge(lo), 0), b1 = min(edge(lo + 1), j.B);
        int n = 0, L = 0, same = 0;
        if (b >= b0 && b < b1 && tokens(b, n, L) && n > 0) {
            int lead = b;
            for (int i = b0; i < b; i += 32) {
                const int k = i + lane;
                const bool on = k < b && j.cu[k + 1] - j.cu[k] > 0;
                const unsigned m = __ballot_sync(0xFFFFFFFFu, on);
                if (m) {
                    lead = i + __ffs(m) - 1;
                    break;
                }
            }
            int most = L - n;
            if (j.prefix_len) most = min(most, max(j.prefix_len[lo], 0));
            most >>= shift;
            int nl = 0, Ll = 0;
            if (!tokens(lead, nl, Ll)) most = 0;
            same = most;
            const int32_t *a = j.table + (int64_t)b * j.cols, *c = j.table + (int64_t)lead * j.cols;
            if (lead != b) {
                for (int i = 0; i < most; i += 128) {
                    int x[4], y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int p = i + k * 32 + lane;
                        x[k] = y[k] = 0;
                        if (p < most) {
                            x[k] = a[p];
                            y[k] = c[p];
                        }
                    }
                    int at = -1;
#pragma unroll
                    for (int k = 3; k >= 0; --k) {
                        const unsigned m = __ballot_sync(0xFFFFFFFFu, x[k] != y[k]);
                        if (m) at = i + k * 32 + __ffs(m) - 1;
                    }
                    if (at >= 0) {
                        same = at;
                        break;
                    }
                }
            }
        }
        if (lane == 0) j.skip[b] = same;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (blockIdx.x != 0) return;
    for (int g = tid; g < j.groups; g += kPrepThreads) {
        const int lo = edge(g), hi = edge(g + 1);
        if (lo < 0 || hi < lo || hi > j.B) s_bad = 1;
    }
    __syncthreads();
    const bool bad = s_bad;
    if (bad && tid == 0) latch(j.err, SV_ERR_DEVICE_BOUNDS);
    if (bad)
        for (int b = tid; b < j.B; b += kPrepThreads) j.skip[b] = 0;
    for (int g = warp; g < j.groups; g += kWarps) {
        PrefixGroup r = {0, 0, 0, 0, 0, 0, 0};
        if (!bad) {
            const int lo = edge(g), hi = edge(g + 1);
            int pages = 0x7FFFFFFF, lead = 0x7FFFFFFF, live = 0;
            for (int b = lo + lane; b < hi; b += 32) {
                int n, L;
                if (!tokens(b, n, L)) pages = 0;
                if (n != 0) {
                    pages = min(pages, __ldcg(j.skip + b));
                    lead = min(lead, b);
                    ++live;
                }
            }
            pages = __reduce_min_sync(0xFFFFFFFFu, pages);
            lead = __reduce_min_sync(0xFFFFFFFFu, lead);
            live = __reduce_add_sync(0xFFFFFFFFu, live);
            if (live < 2) pages = 0;  // nothing is shared
            const int first = pages ? j.cu[lo] : 0;
            const long long rows = pages ? (long long)(j.cu[hi] - first) * j.G : 0;
            for (int b = lo + lane; b < hi; b += 32) {
                int n, L;
                j.skip[b] = tokens(b, n, L) && n > 0 ? pages : 0;
            }
            if (rows > 0) {
                r.first = first;
                r.rows = (int)rows;
                r.pages = pages;
                r.lead = lead;
            }
        }
        if (lane == 0) j.group[g] = r;
    }
    __syncthreads();
    if (warp != 0) return;
    // where each group's work and units start
    long long at = 0;
    int unit = 0;
    for (int g0 = 0; g0 < j.groups; g0 += 32) {
        const int g = g0 + lane;
        long long w = 0;
        int u = 0;
        if (g < j.groups) {
            const PrefixGroup *r = j.group + g;
            const int pages = __ldcg(&r->pages), rows = __ldcg(&r->rows);
            if (pages) {
                const RowBlocks rb(rows);
                const long long tiles = (((long long)pages << shift) + kPxTile - 1) / kPxTile;
                w = tiles * rb.cost() * j.H;
                u = rb.blocks * j.H;
            }
        }
        long long ws = w;
        int us = u;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const long long a = __shfl_up_sync(0xFFFFFFFFu, ws, k);
            const int c = __shfl_up_sync(0xFFFFFFFFu, us, k);
            if (lane >= k) {
                ws += a;
                us += c;
            }
        }
        if (g < j.groups) {
            j.group[g].start = at + ws - w;
            j.group[g].unit0 = unit + us - u;
        }
        at += __shfl_sync(0xFFFFFFFFu, ws, 31);
        unit += __shfl_sync(0xFFFFFFFFu, us, 31);
    }
    if (lane == 0) {
        PrefixGroup r = {0, 0, 0, 0, 0, 0, 0};
        r.start = at;
        r.unit0 = unit;
        j.group[j.groups] = r;
    }
}

// ---------------------------------------------------------------------------
// Units and pieces.
// ---------------------------------------------------------------------------
struct PxPiece {
    int g, h, row0, rows;              // group, cache head, rows of the group
    int t0, t1, tiles;                 // tiles [t0, t1) of the unit's
    int unit;                          // of the call
    int first, lead, pages;
    __device__ __forceinline__ bool wide() const { return rows > 128; }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};
// A tile belongs to the span that its first unit of cost lies in.
struct PxWalk {
    long long pos, end;
    int g;
    __device__ __forceinline__ void start(const PrefixJob &j, long long from, long long to)
    {
        pos = from;
        end = to;
        int lo = 0, hi = j.groups;     // the last group that starts at pos or before
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (j.group[mid].start <= pos) lo = mid; else hi = mid;
        }
        g = lo;
    }
    __device__ __forceinline__ bool next(const PrefixJob &j, PxPiece &p)
    {
        for (;;) {
            if (pos >= end) return false;
            while (g < j.groups && j.group[g + 1].start <= pos) ++g;
            if (g >= j.groups) return false;
            const PrefixGroup r = j.group[g];
            const RowBlocks rb(r.rows);
            const int tiles = (int)((((long long)r.pages * j.block) + kPxTile - 1) / kPxTile);
            const long long head = (long long)tiles * rb.cost(), wide = (long long)tiles * 2;
            long long x = pos - r.start;
            const int h = (int)div_pos(x, head);
            x -= h * head;
            const int block = min((int)div_pos(x, wide), rb.blocks - 1);
            x -= block * wide;
            const int cost = block == rb.blocks - 1 ? rb.last : 2;
            const int t = (int)div_pos(x + cost - 1, cost);
            pos += (long long)t * cost - x;
            if (t >= tiles) continue;  // (the unit's last tile starts before the span)
            if (pos >= end) return false;
            const int n = (int)min((long long)(tiles - t), div_pos(end - pos + cost - 1, cost));
            pos += (long long)n * cost;
            p.g = g;
            p.h = h;
            p.row0 = block * kPxRows;
            p.rows = min(kPxRows, r.rows - p.row0);
            p.t0 = t;
            p.t1 = t + n;
            p.tiles = tiles;
            p.unit = r.unit0 + h * rb.blocks + block;
            p.first = r.first;
            p.lead = r.lead;
            p.pages = r.pages;
            return true;
        }
    }
};

// A piece's sums: [D][256] of values, then 256 maxima and 256 sums of weights.
// CTA i has parts 2 i (its first unit, begun by another CTA) and 2 i + 1 (one that
// another CTA goes on with); whole units come behind those.
__host__ __device__ constexpr size_t px_part_floats(int D) { return (size_t)kPxRows * (D + 2); }
__device__ __forceinline__ float *px_part(const PrefixJob &j, int ctas, int cta, int t0, bool whole,
                                          int unit)
{
    const size_t i = whole ? (size_t)2 * ctas + unit : (size_t)2 * cta + (t0 == 0 ? 1 : 0);
    return j.part + i * px_part_floats(j.D);
}

struct PxShared {
    uint64_t full_k[kPxK], empty_k[kPxK], full_v[kPxV], empty_v[kPxV], full_b[2], empty_b[2];
    uint64_t s_full[2], p_full[2], pv_done[2], q_full, scales[kPxRing], drained;
    uint32_t tmem;
    int abort;
    // for each 16 tokens: the key's scale, log2 of the value scale's fraction (1 to 2)
    // and its inverse; the scale's power of two, as two factors after the bytes'
    // exponents
    float4 sc[kPxRing][8];
    uint32_t up[kPxRing][8];
    float c[kPxRows];                  // factor from S to log2 units, per row
    float m[2][128], l[2][128];        // of the two slots, where they share rows
};

__device__ __forceinline__ void tc_ld32(uint32_t addr, float *v)
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st8u(uint32_t addr, const uint32_t *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                     addr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                 "r"(v[7])
                 : "memory");
}
// A from tensor memory, 16-bit.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four e4m3 bytes to bf16 pairs.  The byte's exponent and fraction, moved to
// bf16's places, are the value times 2^-120 (subnormals too: both formats count
// the same steps); `up` holds 2^(60 + e) and 2^60 in its halves, e the exponent
// of the scale: the factor is taken in two steps, which stay within the range.
__device__ __forceinline__ void e4m3_to_bf16(uint32_t w, uint32_t up, uint32_t &lo, uint32_t &hi)
{
    const uint32_t head = ((w >> 4) & 0x07070707u) | (w & 0x80808080u);
    const uint32_t tail = (w << 4) & 0xF0F0F0F0u;
    constexpr uint32_t k60 = 0x5D805D80u;       // 2^60, twice
    lo = mul_bf16x2(mul_bf16x2(__byte_perm(tail, head, 0x5140), k60), up);
    hi = mul_bf16x2(mul_bf16x2(__byte_perm(tail, head, 0x7362), k60), up);
}

// The piece's queries: hi and lo parts to shared memory, rows of D bytes in the
// swizzle of the keys; D / 8 lanes a row, eight rows or more a warp in flight.
template <int D>
__device__ __forceinline__ void px_queries(const PrefixJob &j, PxShared *sh, char *smem_q,
                                           const PxPiece &pc)
{
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = 8;
    constexpr int kSide = 128 * D;              // bytes of a slot's part
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % kLanes, all = pc.wide() ? kPxRows : 128;
    const bool vec = (((uintptr_t)j.q | (uintptr_t)(j.qts * 2) | (uintptr_t)(j.qhs * 2)) & 15) == 0;
    const bool minus = j.softmax_scale < 0.f;   // (maxima are taken of scores that grow)
#pragma unroll 1
    for (int n0 = warp * kRows * kBatch; n0 < all; n0 += kPxSoft * kRows * kBatch) {
        uint4 raw[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int n = n0 + k * kRows + lane / kLanes;
            raw[k] = make_uint4(0u, 0u, 0u, 0u);
            if (n < pc.rows) {
                const int row = pc.row0 + n, tok = row / j.G;
                const uint16_t *q = j.q + (int64_t)(pc.first + tok) * j.qts +
                                    (int64_t)(pc.h * j.G + row - tok * j.G) * j.qhs + l * 8;
                if (vec) {
                    raw[k] = *reinterpret_cast<const uint4 *>(q);
                } else {
                    raw[k].x = q[0] | (uint32_t)q[1] << 16;
                    raw[k].y = q[2] | (uint32_t)q[3] << 16;
                    raw[k].z = q[4] | (uint32_t)q[5] << 16;
                    raw[k].w = q[6] | (uint32_t)q[7] << 16;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int n = n0 + k * kRows + lane / kLanes;
            float x[8];
            VecTraits<uint16_t>::unpack(raw[k], x);
            float amax = 0.f;
            bool odd = false;                   // NaN or an infinity
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                amax = fmaxf(amax, fabsf(x[i]));
                odd |= !(fabsf(x[i]) < INFINITY);
            }
#pragma unroll
            for (int i = kLanes / 2; i > 0; i >>= 1) {
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, i));
                odd |= __shfl_xor_sync(0xFFFFFFFFu, (int)odd, i) != 0;
            }
            // 2^e brings the largest element to [128, 256)
            const int e = amax > 0.f && !odd ? min(134 - (int)(__float_as_uint(amax) >> 23), 126) : 0;
            const float up = __int_as_float((127 + e) << 23);
            if (l == 0 && n < all)
                sh->c[n] = n >= pc.rows ? 0.f
                           : odd        ? __int_as_float(0x7FC00000)
                                        : fabsf(j.softmax_scale) * 1.4426950408889634f / up;
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                uint16_t h8, l8;
                const float a = minus ? -x[i] * up : x[i] * up;
                const float b = minus ? -x[i + 1] * up : x[i + 1] * up;
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h8) : "f"(b), "f"(a));
                uint32_t h16;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h16) : "h"(h8));
                const float2 h = __half22float2(*reinterpret_cast<__half2 *>(&h16));
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                    : "=h"(l8)
                    : "f"(b - h.y), "f"(a - h.x));
                if (i & 2) {
                    hi[i >> 2] |= (uint32_t)h8 << 16;
                    lo[i >> 2] |= (uint32_t)l8 << 16;
                } else {
                    hi[i >> 2] = h8;
                    lo[i >> 2] = l8;
                }
            }
            if (n < all) {
                const int r = n & 127, sw = D == 128 ? r & 7 : (r >> 1) & 3;
                char *at = smem_q + (n >> 7) * (2 * kSide) + r * D + (((l >> 1) ^ sw) << 4) + (l & 1) * 8;
                *reinterpret_cast<uint2 *>(at) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2 *>(at + kSide) = make_uint2(lo[0], lo[1]);
            }
        }
    }
}

// One tile of a softmax thread: a row's 128 scores to weights.
// M, l: the row's running maximum and sum of weights.
template <int D>
__device__ __forceinline__ bool px_soft_tile(PxShared *sh, int *err, uint32_t s_at, uint32_t o_at,
                                             uint64_t *pv_done, uint32_t count, bool first, int ring,
                                             int chunks, float c, float &M, float &l)
{
    float s[128];
#pragma unroll
    for (int i = 0; i < 4; ++i) tc_ld32(s_at + i * 32, s + i * 32);
    tc_wait_ld(s);
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k >= chunks) break;
        const float4 f = sh->sc[ring][k];
        float a = s[16 * k], b = s[16 * k + 1];
#pragma unroll
        for (int i = 2; i < 16; i += 4) {
            a = max3(a, s[16 * k + i], s[16 * k + i + 1]);
            if (i + 3 < 16) b = max3(b, s[16 * k + i + 2], s[16 * k + i + 3]);
        }
        m = fmaxf(m, fmaf(fmaxf(a, b), c * f.x, f.y));
    }
    bool ok = true;
    if (first) {
        M = m > -INFINITY ? m : 0.f;
        l = 0.f;
    } else if (__any_sync(0xFFFFFFFFu, m > M + kPxLazy)) {
        const float to = m > M + kPxLazy ? m : M, f = ex2f(M - to);
        M = to;
        l *= f;
        ok = at_wait(&sh->abort, err, pv_done, (count - 1) & 1);
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < D; i += 8) {
            float o[8];
            tc_ld8(o_at + i, o);
            tc_wait_ld(o);
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] *= f;
            tc_st8(o_at + i, o);
        }
        tc_wait_st();
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t p[8];
        if (k < chunks) {
            const float4 f = sh->sc[ring][k];
            const float2 u = make_float2(c * f.x, c * f.x), v = make_float2(f.y - M, f.y - M);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 y = fma2(make_float2(s[16 * k + 2 * i], s[16 * k + 2 * i + 1]), u, v);
                const float2 w = make_float2(ex2f(y.x), ex2f(y.y));
                sum = add2(sum, w);
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[i]) : "f"(w.y), "f"(w.x));
            }
            l = fmaf(sum.x + sum.y, f.z, l);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = 0u;
        }
        tc_st8u(s_at + k * 8, p);
    }
    tc_wait_st();
    return ok;
}

template <int D>
__global__ void __launch_bounds__(kPxThreads, 1)
prefix_kernel(const __grid_constant__ PrefixJob j, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v)
{
    constexpr int kSide = kPxTile * D;          // bytes of a tile's keys (or values)
    constexpr int kWideV = kPxTile * D * 2;     // in bf16
    constexpr uint32_t kSwz = D == 128 ? 2 : 4;
    extern __shared__ char px_raw[];
    __shared__ PxShared shared;
    PxShared *sh = &shared;
    char *s_q = px_raw + ((1024 - (smem_u32(px_raw) & 1023)) & 1023);
    char *s_k = s_q + 4 * kSide, *s_v = s_k + kPxK * kSide, *s_b = s_v + kPxV * kSide;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < kPxK; ++i) {
            mbar_init(&sh->full_k[i], 1);
            mbar_init(&sh->empty_k[i], 1);
        }
        for (int i = 0; i < kPxV; ++i) {
            mbar_init(&sh->full_v[i], 1);
            mbar_init(&sh->empty_v[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->full_b[i], 4);
            mbar_init(&sh->empty_b[i], 1);
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->p_full[i], 4);
            mbar_init(&sh->pv_done[i], 1);
        }
        for (int i = 0; i < kPxRing; ++i) mbar_init(&sh->scales[i], 1);
        mbar_init(&sh->q_full, kPxSoft);
        mbar_init(&sh->drained, 1);
        mbar_fence_init();
        sh->abort = 0;
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&sh->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    const int ctas = gridDim.x;
    const long long total = j.group[j.groups].start;
    PxWalk walk;
    walk.start(j, span_at(total, ctas, blockIdx.x), span_at(total, ctas, blockIdx.x + 1));
    PxPiece pc;
    uint32_t it = 0;                            // tiles of this CTA so far
    bool ok = true;

    if (warp < kPxSoft) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPxSoftRegs));
        const int slot = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_at = lanes + slot * 128, o_at = lanes + 256 + slot * 128;
        uint32_t count = 0;                     // this slot's tiles so far
        while (ok && walk.next(j, pc)) {
            const bool wide = pc.wide();
            px_queries<D>(j, sh, s_q, pc);
            fence_async();
            bar_or(1, kPxSoft * 32, false);     // the rows' factors are there
            if (lane == 0) mbar_arrive(&sh->q_full);
            const float c = sh->c[wide ? slot * 128 + r : r];
            const int step = wide ? 1 : 2, from = wide ? 0 : slot, n = pc.t1 - pc.t0;
            float M = kPxNone, l = 0.f;
            for (int i = from; i < n && ok; i += step, ++count) {
                const int ring = (int)((it + i) % kPxRing);
                ok = at_wait(&sh->abort, j.err, &sh->scales[ring], ((it + i) / kPxRing) & 1);
                ok = ok && at_wait(&sh->abort, j.err, &sh->s_full[slot], count & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const long long left = (long long)pc.pages * j.block - (long long)(pc.t0 + i) * kPxTile;
                const int chunks = left >= kPxTile ? 8 : (int)(left >> 4);
                ok = px_soft_tile<D>(sh, j.err, s_at, o_at, &sh->pv_done[slot], count, i == from,
                                     ring, chunks, c, M, l);
                ok = __all_sync(0xFFFFFFFFu, ok);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full[slot]);
            }
            const bool had = from < n;
            if (had && ok) ok = at_wait(&sh->abort, j.err, &sh->pv_done[slot], (count - 1) & 1);
            if (!wide) {
                sh->m[slot][r] = M;
                sh->l[slot][r] = l;
            }
            if (bar_or(1, kPxSoft * 32, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // ---- the piece's sums
            float *part = px_part(j, ctas, blockIdx.x, pc.t0, pc.whole(), pc.unit);
            if (wide) {
                float *at = part + slot * 128 + r;
#pragma unroll 1
                for (int i = 0; i < D; i += 16) {
                    float o[16];
                    tc_ld8(o_at + i, o);
                    tc_ld8(o_at + i + 8, o + 8);
                    tc_wait_ld(o);
#pragma unroll
                    for (int q = 0; q < 16; ++q) at[(size_t)(i + q) * kPxRows] = o[q];
                }
                at[(size_t)D * kPxRows] = M;
                at[(size_t)(D + 1) * kPxRows] = l;
            } else {
                // both slots' sums of a row; half of its elements each
                const float m0 = sh->m[0][r], m1 = n > 1 ? sh->m[1][r] : kPxNone;
                const float m = fmaxf(m0, m1), f0 = ex2f(m0 - m), f1 = n > 1 ? ex2f(m1 - m) : 0.f;
                float *at = part + r;
#pragma unroll 1
                for (int i = slot * (D / 2); i < (slot + 1) * (D / 2); i += 8) {
                    float a[8], b[8];
                    tc_ld8(lanes + 256 + i, a);
                    tc_wait_ld(a);
                    if (n > 1) {
                        tc_ld8(lanes + 384 + i, b);
                        tc_wait_ld(b);
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        at[(size_t)(i + q) * kPxRows] = n > 1 ? fmaf(b[q], f1, a[q] * f0) : a[q];
                }
                if (slot == 0) {
                    at[(size_t)D * kPxRows] = m;
                    at[(size_t)(D + 1) * kPxRows] = n > 1 ? fmaf(sh->l[1][r], f1, sh->l[0][r] * f0)
                                                          : sh->l[0][r];
                }
            }
            tc_fence_before();
            bar_or(1, kPxSoft * 32, false);     // queries and sums may be overwritten
            it += n;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPxSideRegs));
        if (warp < 12) {
            // ---- the values to bf16, a token a thread
            const int tk = tid - kPxSoft * 32;
            while (ok && walk.next(j, pc)) {
                for (int t = pc.t0; t < pc.t1; ++t, ++it) {
                    const int st = it % kPxV, sb = it & 1, ring = it % kPxRing;
                    ok = at_wait(&sh->abort, j.err, &sh->scales[ring], (it / kPxRing) & 1);
                    ok = ok && at_wait(&sh->abort, j.err, &sh->full_v[st], (it / kPxV) & 1);
                    ok = ok && at_wait(&sh->abort, j.err, &sh->empty_b[sb], ((it >> 1) & 1) ^ 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const bool live = (long long)t * kPxTile + tk < (long long)pc.pages * j.block;
                    const uint32_t up = sh->up[ring][tk >> 4];
                    const char *src = s_v + st * kSide + tk * D;
                    char *dst = s_b + sb * kWideV + tk * 128;
                    const int sw = D == 128 ? tk & 7 : (tk >> 1) & 3;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint4 w = *reinterpret_cast<const uint4 *>(src + ((i ^ sw) << 4));
                        if (!live) w = make_uint4(0u, 0u, 0u, 0u);
                        uint4 a, b;
                        e4m3_to_bf16(w.x, up, a.x, a.y);
                        e4m3_to_bf16(w.y, up, a.z, a.w);
                        e4m3_to_bf16(w.z, up, b.x, b.y);
                        e4m3_to_bf16(w.w, up, b.z, b.w);
                        char *at = dst + (i >> 2) * (kPxTile * 128);
                        const int q = (i & 3) * 2;
                        *reinterpret_cast<uint4 *>(at + ((q ^ (tk & 7)) << 4)) = a;
                        *reinterpret_cast<uint4 *>(at + (((q + 1) ^ (tk & 7)) << 4)) = b;
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh->full_b[sb]);
                        mbar_arrive(&sh->empty_v[st]);
                    }
                }
            }
        } else if (warp == 12) {
            // ---- producer: the pages of each tile, looked up 32 at a time
            const int shift = 31 - __clz(j.block), per_tile = kPxTile >> shift;
            const int inner = lane & (per_tile - 1);
            while (ok && walk.next(j, pc)) {
                const int32_t *tab = j.table + (int64_t)pc.lead * j.cols;
                auto window = [&](int w0, int &page, float &ks, float &vs) {
                    page = w0 + lane < pc.pages ? tab[w0 + lane] : -1;
                    if (w0 + lane < pc.pages && (page < 0 || page >= j.pages)) {
                        latch(j.err, SV_ERR_DEVICE_BOUNDS);
                        page = -1;
                    }
                    ks = vs = 1.f;
                    if (page >= 0) {
                        const int64_t ph = (int64_t)page * j.H + pc.h;
                        ks = j.scale[0][ph];
                        vs = fminf(fmaxf(j.scale[1][ph], 0x1p-60f), 0x1p60f);
                    }
                };
                int w0 = (pc.t0 * per_tile) & ~31, page, npage;
                float ks, vs, nks, nvs;
                window(w0, page, ks, vs);
                window(w0 + 32, npage, nks, nvs);
                for (int t = pc.t0; t < pc.t1; ++t, ++it) {
                    const int p0 = t * per_tile;
                    if (p0 >= w0 + 32) {
                        w0 += 32;
                        page = npage;
                        ks = nks;
                        vs = nvs;
                        window(w0 + 32, npage, nks, nvs);
                    }
                    const bool mine = lane - (p0 - w0) >= 0 && lane - (p0 - w0) < per_tile;
                    const bool copy = mine && page >= 0;
                    const uint32_t bytes =
                        (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, copy)) * j.block * D;
                    const int64_t row = (int64_t)page * j.H + pc.h;
                    auto fetch = [&](const CUtensorMap *map, char *dst, uint64_t *bar) {
                        asm volatile(
                            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::"
                            "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
                            "l"(map), "r"(0), "r"(0), "r"((int)row), "r"(smem_u32(bar))
                            : "memory");
                    };
                    const int sk = it % kPxK, sv = it % kPxV, ring = it % kPxRing;
                    ok = at_wait(&sh->abort, j.err, &sh->empty_k[sk], ((it / kPxK) & 1) ^ 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_tx(&sh->full_k[sk], bytes);
                    __syncwarp();
                    if (copy) fetch(&map_k, s_k + sk * kSide + inner * j.block * D, &sh->full_k[sk]);
                    // (the tile that had these places is behind the scores of all
                    // but the last tiles)
                    if (mine) {
                        const uint32_t u = __float_as_uint(vs);
                        const int e = (int)(u >> 23) - 127;
                        const float f = __uint_as_float((u & 0x7FFFFFu) | 0x3F800000u);
                        const float4 sc = make_float4(ks, f == 1.f ? 0.f : log2f(f), 1.f / f, 0.f);
                        const uint32_t up = (uint32_t)(127 + 60 + e) << 7;  // bf16
                        for (int i = 0; i < j.block >> 4; ++i) {
                            sh->sc[ring][inner * (j.block >> 4) + i] = sc;
                            sh->up[ring][inner * (j.block >> 4) + i] = up | up << 16;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->scales[ring]);
                    ok = at_wait(&sh->abort, j.err, &sh->empty_v[sv], ((it / kPxV) & 1) ^ 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_tx(&sh->full_v[sv], bytes);
                    __syncwarp();
                    if (copy) fetch(&map_v, s_v + sv * kSide + inner * j.block * D, &sh->full_v[sv]);
                }
            }
            // after a wait that ran out: copies still in flight land before the exit
            if (!ok) {
                for (int i = 0; i < kPxK; ++i) mbar_wait_n(&sh->full_k[i], (it / kPxK) & 1, 1u << 12);
                for (int i = 0; i < kPxV; ++i) mbar_wait_n(&sh->full_v[i], (it / kPxV) & 1, 1u << 12);
            }
        } else if (warp == 13 && lane == 0) {
            // ---- issuer of the products
            constexpr uint32_t kSums = 1u << 4, kM = 128u >> 4 << 24;  // fp32 sums, M = 128
            constexpr uint32_t kIdS = kSums | (128u >> 3 << 17) | kM;
            // bf16 both; B with its rows (tokens) as the products' dimension
            constexpr uint32_t kIdO = kSums | 1u << 7 | 1u << 10 | 1u << 16 | ((uint32_t)D >> 3 << 17) | kM;
            const uint64_t dk0 = tc_desc(smem_u32(s_k), 16, 8 * D, kSwz);
            const uint64_t dq0 = tc_desc(smem_u32(s_q), 16, 8 * D, kSwz);
            const uint64_t db0 = tc_desc(smem_u32(s_b), kPxTile * 128, 1024, 2);
            uint32_t count[2] = {0, 0}, pieces = 0;
            auto scores = [&](int slot, bool wide, uint32_t i) {
                const int st = i % kPxK;
                ok = ok && at_wait(&sh->abort, j.err, &sh->full_k[st], (i / kPxK) & 1);
                if (!ok) return;
                tc_fence_after();
                const uint64_t dk = dk0 + st * (kSide >> 4);
                const uint64_t dq = dq0 + (wide ? slot : 0) * (2 * kSide >> 4);
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    tc_mma(tmem + slot * 128, dq + 2 * k, dk + 2 * k, kIdS, k);
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    tc_mma(tmem + slot * 128, dq + (kSide >> 4) + 2 * k, dk + 2 * k, kIdS, 1);
                tc_commit(&sh->s_full[slot]);
            };
            auto values = [&](int slot, uint32_t i, bool add) {
                const int sb = i & 1;
                ok = ok && at_wait(&sh->abort, j.err, &sh->full_b[sb], (i >> 1) & 1);
                ok = ok && at_wait(&sh->abort, j.err, &sh->p_full[slot], count[slot]++ & 1);
                if (!ok) return;
                tc_fence_after();
                const uint64_t db = db0 + sb * (kWideV >> 4);
#pragma unroll
                for (int k = 0; k < kPxTile / 16; ++k)
                    tc_mma_ts(tmem + 256 + slot * 128, tmem + slot * 128 + 8 * k, db + 128 * k, kIdO,
                              add || k);
                tc_commit(&sh->pv_done[slot]);
            };
            while (ok && walk.next(j, pc)) {
                const bool wide = pc.wide();
                const int n = pc.t1 - pc.t0;
                ok = at_wait(&sh->abort, j.err, &sh->q_full, pieces++ & 1);
                tc_fence_after();
                if (wide) {
                    scores(0, true, it);
                    scores(1, true, it);
                    if (ok) tc_commit(&sh->empty_k[it % kPxK]);
                    for (int i = 0; i < n && ok; ++i, ++it) {
                        values(0, it, i > 0);
                        if (i + 1 < n) scores(0, true, it + 1);
                        values(1, it, i > 0);
                        if (ok) tc_commit(&sh->empty_b[it & 1]);
                        if (i + 1 < n) {
                            scores(1, true, it + 1);
                            if (ok) tc_commit(&sh->empty_k[(it + 1) % kPxK]);
                        }
                    }
                } else {
                    for (int i = 0; i < 2 && i < n; ++i) {
                        scores(i, false, it + i);
                        if (ok) tc_commit(&sh->empty_k[(it + i) % kPxK]);
                    }
                    for (int i = 0; i < n && ok; ++i, ++it) {
                        values(i & 1, it, i > 1);
                        if (ok) tc_commit(&sh->empty_b[it & 1]);
                        if (i + 2 < n) {
                            scores(i & 1, false, it + 2);
                            if (ok) tc_commit(&sh->empty_k[(it + 2) % kPxK]);
                        }
                    }
                }
            }
            // after a wait that ran out: products still in flight end before the exit
            if (!ok) {
                tc_commit(&sh->drained);
                mbar_wait_n(&sh->drained, 0, 1u << 12);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// ---------------------------------------------------------------------------
// The join: a unit's pieces and what attend left of its rows.  A CTA has 32
// rows (lanes) and 32 elements of them: two warps with 16 each, times four that
// share the pieces.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256, kJoinWays = 4;

__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixJob j, int ctas)
{
    __shared__ float s_sum[kJoinWays][2][16][32], s_m[kJoinWays][2][32], s_l[kJoinWays][2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, way = warp >> 1, half = warp & 1;
    pdl_wait();
    pdl_trigger();
    const int unit = blockIdx.x >> 3, n = (blockIdx.x & 7) * 32 + lane;
    if (unit >= j.group[j.groups].unit0) return;
    int lo = 0, hi = j.groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (j.group[mid].unit0 <= unit) lo = mid; else hi = mid;
    }
    while (j.group[lo + 1].unit0 <= unit) ++lo;   // (groups without units)
    const PrefixGroup r = j.group[lo];
    const RowBlocks rb(r.rows);
    const int u = unit - r.unit0, h = u / rb.blocks, block = u - h * rb.blocks;
    const int rows = min(kPxRows, r.rows - block * kPxRows);
    if ((int)(blockIdx.x & 7) * 32 >= rows) return;
    const int tiles = (int)((((long long)r.pages * j.block) + kPxTile - 1) / kPxTile);
    const int cost = block == rb.blocks - 1 ? rb.last : 2;
    const long long total = j.group[j.groups].start;
    const long long at = r.start + (long long)tiles * ((long long)h * rb.cost() + 2LL * block);
    const int c0 = span_owner(total, ctas, at);
    const int c1 = span_owner(total, ctas, at + (long long)(tiles - 1) * cost);
    const int e0 = blockIdx.y * 32 + half * 16;
    float m = kPxNone, l = 0.f, o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
    for (int c = c0 + way; c <= c1; c += kJoinWays) {
        // the CTA's first tile of the unit, if it has one
        const long long from = span_at(total, ctas, c), to = span_at(total, ctas, c + 1);
        const int t = from > at ? (int)div_pos(from - at + cost - 1, cost) : 0;
        if (t >= tiles || at + (long long)t * cost >= to) continue;
        const float *p = px_part(j, ctas, c, t, c0 == c1, unit) + n;
        const float mc = __ldcg(p + (size_t)j.D * kPxRows);
        const float lc = __ldcg(p + (size_t)(j.D + 1) * kPxRows);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __ldcg(p + (size_t)(e0 + i) * kPxRows);
        const float top = fmaxf(m, mc), f = ex2f(m - top), g = ex2f(mc - top);
        m = top;
        l = fmaf(l, f, lc * g);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = fmaf(o[i], f, x[i] * g);
    }
    const int row = block * kPxRows + n, tok = row / j.G;
    const int64_t to = (int64_t)(r.first + tok) * j.Hq + h * j.G + (row - tok * j.G);
    if (way == 1 && n < rows) {
        // what attend left
        const float2 ms = __ldcg(j.far_ms + to);
        const float4 *p = reinterpret_cast<const float4 *>(j.far_o + to * j.D + e0);
        const float top = fmaxf(m, ms.x), f = ex2f(m - top), g = ex2f(ms.x - top);
        m = top;
        l = fmaf(l, f, ms.y * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = __ldcg(p + i);
            o[4 * i] = fmaf(o[4 * i], f, x.x * g);
            o[4 * i + 1] = fmaf(o[4 * i + 1], f, x.y * g);
            o[4 * i + 2] = fmaf(o[4 * i + 2], f, x.z * g);
            o[4 * i + 3] = fmaf(o[4 * i + 3], f, x.w * g);
        }
    }
    if (way > 0) {
        s_m[way][half][lane] = m;
        s_l[way][half][lane] = l;
#pragma unroll
        for (int i = 0; i < 16; ++i) s_sum[way][half][i][lane] = o[i];
    }
    __syncthreads();
    if (way > 0 || n >= rows) return;
#pragma unroll
    for (int w = 1; w < kJoinWays; ++w) {
        const float mc = s_m[w][half][lane], top = fmaxf(m, mc), f = ex2f(m - top), g = ex2f(mc - top);
        m = top;
        l = fmaf(l, f, s_l[w][half][lane] * g);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = fmaf(o[i], f, s_sum[w][half][i][lane] * g);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
            : "=r"(w[i]) : "f"(o[2 * i + 1] * inv), "f"(o[2 * i] * inv));
    uint4 *dst = reinterpret_cast<uint4 *>(j.out + to * j.D + e0);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (j.lse && e0 == 0) j.lse[to] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

constexpr size_t prefix_smem(int D)
{
    return 1024 + (size_t)(4 + kPxK + kPxV) * kPxTile * D + 2 * kPxTile * D * 2;
}
static_assert(prefix_smem(128) + sizeof(PxShared) <= 227 * 1024, "shared memory of a CTA");

size_t prefix_part_bytes(int sms, int64_t units, int D)
{
    return ((size_t)2 * sms + units) * px_part_floats(D) * sizeof(float);
}

cudaError_t prefix_setup()
{
    // the softmax warps' registers come out of what the launch gives the others
    cudaError_t e = cudaSuccess;
    const void *const f[2] = {(const void *)prefix_kernel<64>, (const void *)prefix_kernel<128>};
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, f[i]);
        if (e == cudaSuccess && a.numRegs != kPxRegs) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f[i], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)prefix_smem(128));
    }
    return e;
}

cudaError_t prefix_prep_launch(const PrefixJob &j, unsigned *counters, int n, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    pdl_config(cfg, at, dim3(kPrepCtas), dim3(kPrepThreads), 0, s);
    return cudaLaunchKernelEx(&cfg, prefix_prep_kernel, j, counters, n);
}

cudaError_t prefix_launch(const PrefixJob &j, int sms, int64_t units, cudaStream_t s)
{
    CUtensorMap mk, mv;
    if (!cache_map(&mk, j.cache[0], j.D, j.block, j.pages, j.H) ||
        !cache_map(&mv, j.cache[1], j.D, j.block, j.pages, j.H))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    // (one CTA an SM, also at D = 64: each holds all of the SM's tensor memory)
    pdl_config(cfg, at, dim3(sms), dim3(kPxThreads), prefix_smem(128), s);
    cudaError_t e = j.D == 64 ? cudaLaunchKernelEx(&cfg, prefix_kernel<64>, j, mk, mv)
                              : cudaLaunchKernelEx(&cfg, prefix_kernel<128>, j, mk, mv);
    if (e != cudaSuccess) return e;
    pdl_config(cfg, at, dim3((unsigned)(units * 8), j.D / 32), dim3(kJoinThreads), 0, s);
    return cudaLaunchKernelEx(&cfg, prefix_join_kernel, j, sms);
}

}  // namespace sv
