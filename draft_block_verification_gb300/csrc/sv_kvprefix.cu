// sv_kvprefix.cu -- attention over the paged 8-bit cache for sequences that
// share a prefix: the pages that all sequences of a group have in common are
// read once, for the query rows of the whole group.
//
// The result is that of the attention over each sequence by itself (z, w, o as
// in sv_kvattn.cu).  A row's positions are cut in two, the shared pages and the
// rest; each part leaves its maximum m, its sum of weights l = sum 2^(y - m) and
// its sum of weighted values o = sum 2^(y - m) v, and
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,  M = max m_i.
//
// Three kernels:
//   prep     which pages are shared: the leading entries of the group's table
//            rows that are equal, no further than the caller's bound and the
//            tokens before each sequence's new ones.  So a bound that is too
//            large changes nothing.  And how the work is cut.
//   prefix   below: the shared pages, and what sequences of many rows have of
//            their own.
//   tail     (sv_kvtail.cu) what sequences of few rows have, and the join.
//
// Shape of the prefix kernel.  A span is a run of pages that a run of query rows reads:
// a group's shared pages, which all of its rows see whole, or a sequence's own ones,
// where the new tokens are masked.  A unit is a cache head's block of up to 256 rows
// of a span, two times 128 (slots); a tile is 128 tokens.  Queries are the 128 rows
// of the products, a row's scores lie in one thread's registers, and maxima and
// sums need no exchange:
//   S [128 rows x 128 tokens] = Q K^T    in 8 bits: the cache's bytes as they
//       lie, the query in two e4m3 parts, added up (exact from 2^-9 of the row's
//       largest element on, within 2^-17 of it below)
//   O [128 rows x D]         += P V      in fp16: P from tensor memory, V's bytes
//       brought to fp16 in shared memory
// Weights are 2^(y - M) with M 2^6 below the maximum that it was taken from, 2^15 at
// most: fp16's 11 bits down to 2^-19 of the largest, steps of 2^-29 of it below.  Their
// sum is that of the weights before the rounding.  A value times the power of two in its
// page's scale, by a power that the piece has in common (the largest of its first pages),
// is exact in fp16; what the scale has beside the power goes into the exponent
// and out of the sum again (as log2 and 1 / x).  A tile with a page whose scale lies
// more than 2^3 above the common one or 2^5 below it would lose small weights' bits to
// large scales: it is taken in bf16, values and weights, where a weight is within 2^-8
// of itself at any size.  (All in bf16: the same time, and a weight's 2^-8 in every row.)
//
// The products of a slot's tile run under the other slot's softmax:
//   tensor  S0 . . PV0 S0' PV1 S1' ...
//   slot 0    softmax     softmax
// A unit of up to 128 rows gives both slots the same queries and every other
// tile each, and joins the two at its end.  A softmax thread has a row, and takes
// its 128 scores 64 at a time; four more warps bring the values to fp16, one
// fetches, two issue (a slot each, taking turns).
//
// The running maximum moves lazily: only where a tile's maximum passes it by
// 2^8 are a row's sums rescaled.
//
// Split.  Tiles of all large units laid end to end are cut into equal shares, one a
// CTA (fewer where units are few: their pieces are added in turn); small units are
// taken whole, by the CTAs whose shares are done.  A unit's piece leaves its sums in
// the workspace, fp32, four elements of 256 rows after the other; the tail kernel
// adds a unit's pieces.
//
// What bounds it.  A slot's tile is a chain: its softmax (1,400 to 2,000 cycles), the
// products with its weights, the next scores (1,024 of the tensor cores), and what
// passes between them; two slots, which is what tensor memory holds at D = 128 (at 64 a
// quarter of it is not used), make it 3,400 cycles a tile of 256 rows at best, of which
// the tensor cores work 2,048.  A unit takes some 18,000 beside its tiles.  64 sequences
// of 13 tokens of 32 heads behind 8,192 shared ones and 330 of their own: 180 us of the
// call's 238; 24 of 4 behind three prefixes of up to 131,072, D = 64: 344 of 409 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_common.cuh"
#include "sv_kv.cuh"
#include "sv_tc.cuh"

namespace sv {

constexpr int kPxTile = 128;           // tokens of a tile
constexpr int kPxRows = kPrefixRows;   // query rows of a unit, two slots of 128
constexpr int kPxK = 3, kPxV = 2;      // tiles of keys and of values in flight
constexpr int kPxPieces = 4;           // pieces known ahead
constexpr int kPxReaders = 14;         // warps that read them
constexpr int kPxRing = 8;             // tiles whose scales are kept
constexpr int kPxSoft = 8;             // softmax warps, four a slot
constexpr int kPxThreads = 512;        // + 4 converting warps, producer, 2 issuers, 1 idle
// Registers: 128 a thread at launch; the softmax warps, which hold 64 of a row's
// scores, take what the others leave (256 * 184 + 256 * 72 = 512 * 128).
constexpr int kPxRegs = 128, kPxSoftRegs = 184, kPxSideRegs = 72;
static_assert(256 * kPxSoftRegs + 256 * kPxSideRegs <= kPxThreads * kPxRegs, "registers");
constexpr float kPxUnit = 6.f;         // log2 of the weight of a maximum that M was taken from
constexpr float kPxMost = 14.f;        // of the largest weight before M moves
constexpr int kPxAbove = 3, kPxBelow = 5;  // of a value scale about the piece's
constexpr uint32_t kPxTries = 1u << 16; // of a wait
constexpr float kPxNone = -1e30f;      // maximum of no tokens
constexpr float kPxFar = 0x1p14f;      // maxima from which on scores are rounded first
constexpr float kPxMark = -3e38f;      // stands for one of those: every weight passes it

// ---------------------------------------------------------------------------
// Which pages are shared.
// ---------------------------------------------------------------------------
constexpr int kPrepCtas = 8, kPrepThreads = 512;

// What little is shared the tail reads sooner for each sequence by itself: 16 tokens
// of eight rows of a head take it 1 to 2 ns in all, a run of the prefix kernel some
// 15 us more than one without work, and the tail waits for it.  (Single tokens of 32
// heads, 8 of the cache, as graphs: 16 to 64 behind 1,024 to 256 shared ones 35 to 37 us
// against 45 to 47; behind twice as many 39 against 47 for 16, 57 against 49 for 64;
// behind four times as many 48 against 55, and 72 against 51.)
constexpr unsigned long long kPxLeast = 16384;

// Row blocks of a head, and costs, in 400 cycles: a tile of up to 256 rows, one of up
// to 128, and what a unit takes beside its tiles (queries, first scores, sums), which
// is counted at its front.  (64 draft blocks / three long documents: 239 / 409 us; units
// at a ninth of that 239 / 535, narrow tiles at 6 241 / 418.)
constexpr int kPxWide = 9, kPxNarrow = 5, kPxUnitCost = 45;
constexpr int kPxWhole = 130;          // of a unit that is not cut (90 to 250: equal)
struct RowBlocks {
    int blocks, full, last;            // blocks; a tile's cost, in all blocks and in the last
    __device__ __forceinline__ RowBlocks(int rows, int block)
    {
        blocks = (rows + block - 1) / block;
        full = block > 128 ? kPxWide : kPxNarrow;
        last = rows - (blocks - 1) * block > 128 ? kPxWide : kPxNarrow;
    }
    __device__ __forceinline__ long long unit(int tiles) const
    {
        return kPxUnitCost + (long long)tiles * full;
    }
    __device__ __forceinline__ long long head(int tiles) const
    {
        return (blocks - 1) * unit(tiles) + kPxUnitCost + (long long)tiles * last;
    }
};
__device__ __forceinline__ int px_tiles(int end) { return (int)(((long long)end + kPxTile - 1) / kPxTile); }

// One cluster: its warps take the sequences, its first CTA's the groups.
__global__ void __cluster_dims__(kPrepCtas, 1, 1) __launch_bounds__(kPrepThreads)
prefix_prep_kernel(const PrefixJob j, int warps)
{
    __shared__ int s_bad, s_many, s_lost;
    __shared__ unsigned long long s_shared;
    __shared__ longlong2 s_sum[kPrepThreads / 32];
    __shared__ int2 s_scan[kPrepThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kPrepThreads / 32;
    const int shift = 31 - __clz(j.block);
    pdl_wait();
    pdl_trigger();
    if (tid == 0) s_bad = s_many = s_lost = 0, s_shared = 0;
    if (blockIdx.x == 0)
        for (int i = tid; i < kTailParts * warps; i += kPrepThreads) j.tail_arrived[i] = 0;
    auto edge = [&](int g) { return j.cu_group ? j.cu_group[g] : g ? j.B : 0; };
    bool lost = false;
    auto tokens = [&](int b, int &n, int &L) {  // false: lengths out of range
        const int first = j.cu[b], end = j.cu[b + 1];
        L = j.kv_len[b];
        n = end - first;
        return !lost && first >= 0 && end <= j.T && n >= 0 && L >= n &&
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
        // (of no group: 0 already)
        if (lane == 0) j.skip[b] = same;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (blockIdx.x != 0) return;
    for (int g = tid; g < j.groups; g += kPrepThreads) {
        const int lo = edge(g), hi = edge(g + 1);
        if (lo < 0 || hi < lo || hi > j.B) s_bad = 1;
    }
    // Rows of sequences out of order may be more than there are, and than the
    // workspace has units for: then none is taken.
    for (int b = tid; b < j.B; b += kPrepThreads)
        if (j.cu[b + 1] < j.cu[b]) s_lost = 1;
    __syncthreads();
    const bool bad = s_bad;
    lost = s_lost;
    if (bad && tid == 0) latch(j.err, SV_ERR_DEVICE_BOUNDS);
    if (bad)
        for (int b = tid; b < j.B; b += kPrepThreads) j.skip[b] = j.seq_group[b] = 0;
    for (int g = warp; g < j.groups; g += kWarps) {
        PrefixSpan r = {};
        if (!bad) {
            const int lo = edge(g), hi = edge(g + 1);
            int pages = 0x7FFFFFFF, lead = 0x7FFFFFFF, live = 0;
            long long eights = 0;
            bool many = false;
            for (int b = lo + lane; b < hi; b += 32) {
                int n, L;
                if (!tokens(b, n, L)) pages = 0;
                if (n != 0) {
                    pages = min(pages, __ldcg(j.skip + b));
                    lead = min(lead, b);
                    ++live;
                    eights += (n * j.G + 7) >> 3;
                    many |= n * j.G > kTailMax;
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
                j.seq_group[b] = g;
            }
            if (many) s_many = 1;
            if (pages)
                atomicAdd(&s_shared, (unsigned long long)(eights * j.H * ((pages << shift) >> 4)));
            if (rows > 0) {
                r.first = first;
                r.rows = (int)rows;
                r.lead = lead;
                r.end = r.ctx = pages << shift;
            }
        }
        if (lane == 0) j.span[g] = r;
    }
    __syncthreads();
    if (!s_many && s_shared < kPxLeast) {
        for (int b = tid; b < j.B; b += kPrepThreads) j.skip[b] = 0;
        for (int g = tid; g < j.groups; g += kPrepThreads) j.span[g] = PrefixSpan{};
        __syncthreads();
    }
    // the tail's tasks: what is left of each sequence, cut into ranges of `c` stages
    auto left = [&](int b, long long &blocks, int &stages) {
        int n, L;
        const bool fine = tokens(b, n, L);
        if (!fine) latch(j.err, SV_ERR_DEVICE_BOUNDS);
        blocks = fine && n > 0 ? (long long)TailBlocks(n * j.G).blocks * j.H : 0;
        const int own = L - __ldcg(j.skip + b) * j.block;
        // (rows that the prefix kernel takes are only joined)
        stages = !blocks ? 0 : n * j.G > kTailMax ? 1 : (own + kTailTile - 1) / kTailTile;
    };
    for (int b = tid; b < j.B; b += kPrepThreads) {
        int n, L;
        PrefixSpan r = {};
        if (tokens(b, n, L) && n * j.G > kTailMax) {
            const int skip = __ldcg(j.skip + b);
            r.first = j.cu[b];
            r.rows = n * j.G;
            r.lead = b;
            r.page0 = skip;
            r.end = L - (skip << shift);
            r.ctx = r.end - n;
        }
        j.span[j.groups + b] = r;
    }
    long long all = 0, many = 0;
    for (int b = tid; b < j.B; b += kPrepThreads) {
        long long blocks;
        int stages;
        left(b, blocks, stages);
        all += blocks * stages;
        many += blocks;
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        all += __shfl_xor_sync(0xFFFFFFFFu, all, k);
        many += __shfl_xor_sync(0xFFFFFFFFu, many, k);
    }
    if (lane == 0) s_sum[warp] = make_longlong2(all, many);
    __syncthreads();
    all = many = 0;
    for (int w = 0; w < kWarps; ++w) {
        all += s_sum[w].x;
        many += s_sum[w].y;
    }
    __syncthreads();
    // a task a warp, of 128 tokens at least (four sequences of 1,024, as a graph: 33 us;
    // of 192 35, of 256 39); where there are about as many as warps
    // before any is cut, only those of twice the mean
    const long long mean = (all + warps - 1) / warps;
    const int c = (int)max(4LL, 2 * many >= warps ? 2 * mean : mean);
    if (tid == 0) *j.tail_stages = c;
    int units = 0, parts = 0;
    for (int b0 = 0; b0 < j.B; b0 += kPrepThreads) {
        const int b = b0 + tid;
        int mine = 0, part = 0;
        if (b < j.B) {
            long long blocks;
            int stages;
            left(b, blocks, stages);
            const int nz = (stages + c - 1) / c;
            mine = (int)(blocks * nz);
            part = nz > 1 ? mine : 0;
        }
        int ms = mine, ps = part;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, ms, k), y = __shfl_up_sync(0xFFFFFFFFu, ps, k);
            if (lane >= k) {
                ms += x;
                ps += y;
            }
        }
        if (lane == 31) s_scan[warp] = make_int2(ms, ps);
        __syncthreads();
        int um = 0, pm = 0, ua = 0, pa = 0;
        for (int w = 0; w < kWarps; ++w) {
            const int2 x = s_scan[w];
            if (w < warp) {
                um += x.x;
                pm += x.y;
            }
            ua += x.x;
            pa += x.y;
        }
        if (b < j.B) {
            j.unit0[b] = units + um + ms - mine;
            j.part0[b] = parts + pm + ps - part;
        }
        units += ua;
        parts += pa;
        __syncthreads();
    }
    if (tid == 0) j.unit0[j.B] = units;
    if (warp != 0) return;
    // Rows of a unit.  A piece's sums are as many as its rows, whatever its tokens; so
    // where CTAs by far outnumber the units, units of half the rows halve what the
    // tail has to read (128 single tokens of 32 heads: 107 us against 115; with as many
    // units as CTAs the halves would only have values converted twice).
    const int spans = j.groups + j.B;
    int big = 0, small = 0;
    for (int g = lane; g < spans; g += 32) {
        const int rows = __ldcg(&j.span[g].rows);
        if (!rows) continue;
        const RowBlocks rb(rows, kPxRows);
        big += rb.blocks * j.H;
        if (rb.head(px_tiles(__ldcg(&j.span[g].end))) <= kPxWhole * (long long)rb.blocks)
            small += rb.blocks * j.H;
    }
    big = __reduce_add_sync(0xFFFFFFFFu, big);
    small = __reduce_add_sync(0xFFFFFFFFu, small);
    const int block = 4 * big < j.prefix_ctas ? 128 : kPxRows;
    // Small units, if there are at least as many as CTAs, are not cut: CTAs take them one
    // by one when their shares of the rest are done.  (CTAs take 240,000 to 330,000
    // cycles for the same 66 tiles.)
    const int whole = small >= j.prefix_ctas ? kPxWhole : 0;
    // where each span's work and units start
    long long at = 0;
    int unit = 0, loose = 0;
    float most = 0.f;                  // of a unit that is cut
    for (int g0 = 0; g0 < spans; g0 += 32) {
        const int g = g0 + lane;
        long long w = 0;
        int u = 0, v = 0;
        if (g < spans) {
            const int rows = __ldcg(&j.span[g].rows);
            if (rows) {
                const RowBlocks rb(rows, block);
                const int tiles = px_tiles(__ldcg(&j.span[g].end));
                u = rb.blocks * j.H;
                w = rb.head(tiles);
                if (w <= whole * (long long)rb.blocks) {
                    v = u;
                    w = 0;
                } else {
                    most = fmaxf(most, (float)w / (float)rb.blocks);
                    w *= j.H;
                }
            }
        }
        long long ws = w;
        int us = u, vs = v;
#pragma unroll 1
        for (int k = 1; k < 32; k <<= 1) {
            const long long a = __shfl_up_sync(0xFFFFFFFFu, ws, k);
            const int c = __shfl_up_sync(0xFFFFFFFFu, us, k), d = __shfl_up_sync(0xFFFFFFFFu, vs, k);
            if (lane >= k) {
                ws += a;
                us += c;
                vs += d;
            }
        }
        if (g < spans) {
            j.span[g].start = at + ws - w;
            j.span[g].unit0 = unit + us - u;
            j.span[g].loose0 = loose + vs - v;
            j.span[g].block = block;
        }
        at += __shfl_sync(0xFFFFFFFFu, ws, 31);
        unit += __shfl_sync(0xFFFFFFFFu, us, 31);
        loose += __shfl_sync(0xFFFFFFFFu, vs, 31);
    }
#pragma unroll 1
    for (int k = 16; k > 0; k >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, k));
    if (lane == 0) {
        PrefixSpan r = {};
        r.start = at;
        r.unit0 = unit;
        r.loose0 = loose;
        // A unit's pieces are added one after the other, 0.7 us each (what 3.25 of cost
        // take): beyond sqrt(cost / 3.25) of them that takes longer than a piece saves.
        // (One unit of 36 rows over 38,272 tokens: 81 us, in 152 pieces 154;
        // over 131,072 104 and 178.)
        const long long least = max(1LL, (long long)sqrtf(3.25f * most));
        r.rows = (int)min((long long)j.prefix_ctas, max(1LL, at / least));
        j.span[spans] = r;
        *j.next = 0;
    }
}

// ---------------------------------------------------------------------------
// Units and pieces.
// ---------------------------------------------------------------------------
struct PxPiece {
    int h, row0, rows;                 // cache head, rows of the span (0: no more pieces)
    int t0, t1, tiles;                 // tiles [t0, t1) of the unit's
    int unit;                          // of the call
    int first, lead, page0, end, ctx;  // of the span
    __device__ __forceinline__ bool wide() const { return rows > 128; }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};
// A CTA's pieces, found by its producer.  First its share of the units that are cut: a
// tile belongs to the share that its first unit of cost lies in.  Then of the others
// the next one, until none is left.  (Which CTA takes it is not seen in the result.)
struct PxWalk {
    long long pos, end;
    int loose;                         // units that are not cut
    __device__ __forceinline__ bool next(const PrefixJob &j, PxPiece &p, int lane)
    {
        for (;;) {
            const bool cut = pos < end;
            int u = 0;
            if (!cut) {
                if (loose == 0) return false;
                if (lane == 0) u = atomicAdd(j.next, 1);
                u = __shfl_sync(0xFFFFFFFFu, u, 0);
                if (u >= loose) return false;
            }
            // the last span that starts at pos (or u) or before
            int lo = 0, n = j.groups + j.B;
            while (n > 1) {
                const int step = (n + 31) >> 5, at = lo + lane * step;
                const bool on = at < lo + n && (cut ? j.span[at].start <= pos : j.span[at].loose0 <= u);
                const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, on));  // (lane 0 is on)
                n = min(step, n - k * step);
                lo += k * step;
            }
            const PrefixSpan r = j.span[lo];
            const RowBlocks rb(r.rows, r.block);
            const int tiles = px_tiles(r.end);
            int h, block, t = 0, m = tiles;
            if (cut) {
                const long long head = rb.head(tiles), unit = rb.unit(tiles);
                long long x = pos - r.start;
                h = (int)div_pos(x, head);
                x -= h * head;
                block = min((int)div_pos(x, unit), rb.blocks - 1);
                x -= block * unit;
                const int cost = block == rb.blocks - 1 ? rb.last : rb.full;
                // a tile lies behind its unit's front
                const long long front = pos - x + kPxUnitCost;
                t = x <= kPxUnitCost ? 0 : (int)div_pos(x - kPxUnitCost + cost - 1, cost);
                pos = front + (long long)min(t, tiles) * cost;
                if (t >= tiles) continue;  // (the unit's last tile starts before the share)
                if (pos >= end) continue;
                m = (int)min((long long)(tiles - t), div_pos(end - pos + cost - 1, cost));
                pos += (long long)m * cost;
            } else {
                h = (u - r.loose0) / rb.blocks;
                block = u - r.loose0 - h * rb.blocks;
            }
            p.h = h;
            p.row0 = block * r.block;
            p.rows = min(r.block, r.rows - p.row0);
            p.t0 = t;
            p.t1 = t + m;
            p.tiles = tiles;
            p.unit = r.unit0 + h * rb.blocks + block;
            p.first = r.first;
            p.lead = r.lead;
            p.page0 = r.page0;
            p.end = r.end;
            p.ctx = r.ctx;
            return true;
        }
    }
};

// A piece's sums: [D / 4][256][4] of values, then 256 maxima and 256 sums of weights.
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
    uint64_t s_full[2], p_full[2], pv_done[2], q_full, turn[2], scales[kPxRing], drained[2];
    uint32_t tmem;
    int abort;
    // for each 16 tokens: the key's scale, log2 of the value scale's fraction (1 to 2),
    // its inverse, and the log2 once more (the first is infinite where the tile is taken
    // in bf16); the scale's power of two by the piece's, as two factors
    float4 sc[kPxRing][8];
    uint32_t up[kPxRing][8], more[kPxRing][8];
    int kind[kPxRing];                 // kPxApart: in bf16; the rest, less 64: the piece's exponent
    PxPiece piece[kPxPieces];          // handed from the producer to the other roles
    uint64_t piece_full[kPxPieces], piece_empty[kPxPieces];
    uint32_t lost[2][4];               // tokens of a tile with NaN in their value, a bit each
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
__device__ __forceinline__ void tc_st32u(uint32_t addr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
        "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31])
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
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Bytes of w by selector; a selector's bit 3 takes the byte's sign, eight times.
__device__ __forceinline__ uint32_t sign_pairs(uint32_t w, uint32_t sel)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(d) : "r"(w), "r"(sel));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Two weights, the first in the lower half.
__device__ __forceinline__ uint32_t weights_f16(float a, float b)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}
__device__ __forceinline__ uint32_t weights_bf16(float a, float b)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}
__device__ __forceinline__ uint32_t scaled_f16(uint32_t w, float by)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return weights_f16(f.x * by, f.y * by);
}

// Bounded wait that also ends when another role has given up.  A try lets the
// warp sleep until the phase completes or some 10 us have passed: polling warps
// would take a quarter of the instruction slots.
__device__ __forceinline__ bool px_wait(PxShared *sh, int *err, uint64_t *bar, uint32_t parity)
{
    for (uint32_t i = 0; i < kPxTries; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(10000)
            : "memory");
        if (ok) return true;
        if (*(volatile int *)&sh->abort) return false;
    }
    *(volatile int *)&sh->abort = 1;
    latch(err, SV_ERR_TIMEOUT);
    return false;
}

// Four e4m3 bytes to bf16 pairs.  A byte with its sign in the byte above it, moved
// up by four bits, has sign, exponent and fraction in bf16's places (once the bits
// between are cleared) and stands for its value times 2^-120: both formats count the
// same steps, subnormals too.  up: 2^(120 + e), twice, e the scale's exponent, of
// which more than 7 would leave the range (kPxTop).
constexpr int kPxTop = 7;
constexpr int kPxApart = 1 << 8;
__device__ __forceinline__ void e4m3_to_bf16(uint32_t w, uint32_t up, uint32_t &lo, uint32_t &hi)
{
    constexpr uint32_t kKeep = 0x87F087F0u;
    lo = mul_bf16x2((sign_pairs(w, 0x9180) << 4) & kKeep, up);
    hi = mul_bf16x2((sign_pairs(w, 0xB3A2) << 4) & kKeep, up);
}

// To fp16 pairs, exactly, NaN too.  up: 2^d, twice.
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t up, uint32_t &lo, uint32_t &hi)
{
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
        " cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    lo = mul_f16x2(lo, up);
    hi = mul_f16x2(hi, up);
}

// The piece's queries: hi and lo parts to shared memory, rows of D bytes in the
// swizzle of the keys; D / 16 lanes a row, kAhead rows a lane in flight.  (Kept
// short: code that runs once a piece comes from far, some 300 cycles for every
// eight instructions.)
template <int D>
__device__ __forceinline__ void px_queries(const PrefixJob &j, PxShared *sh, char *smem_q,
                                           const PxPiece &pc)
{
    constexpr int kLanes = D / 16, kRows = 32 / kLanes, kAhead = 4;
    constexpr int kStep = kPxSoft * kRows;      // rows of a load of all warps
    constexpr int kSide = 128 * D;              // bytes of a slot's part
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % kLanes, all = pc.wide() ? kPxRows : 128;
    const bool vec = (((uintptr_t)j.q | (uintptr_t)(j.qts * 2) | (uintptr_t)(j.qhs * 2)) & 15) == 0;
    const float sign = j.softmax_scale < 0.f ? -1.f : 1.f;  // (maxima are of scores that grow)
    const int mine = warp * kRows + lane / kLanes;
    // the token and head of the next row to fetch
    const int row0 = pc.row0 + mine, tok_step = kStep / j.G, head_step = kStep - tok_step * j.G;
    int tok = row0 / j.G, head = row0 - tok * j.G, at = mine;
    auto fetch = [&](uint4 (&v)[2]) {
        v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u);
        if (at < pc.rows) {
            const uint16_t *q = j.q + (int64_t)(pc.first + tok) * j.qts +
                                (int64_t)(pc.h * j.G + head) * j.qhs + l * 16;
            if (vec) {
                v[0] = reinterpret_cast<const uint4 *>(q)[0];
                v[1] = reinterpret_cast<const uint4 *>(q)[1];
            } else {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
                v[0] = make_uint4(w[0], w[1], w[2], w[3]);
                v[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
        at += kStep;
        tok += tok_step;
        head += head_step;
        if (head >= j.G) {
            head -= j.G;
            ++tok;
        }
    };
    uint4 raw[kAhead][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(raw[k]);
#pragma unroll 1
    for (int n = mine; n < all; n += kStep) {
        const uint32_t x[8] = {raw[0][0].x, raw[0][0].y, raw[0][0].z, raw[0][0].w,
                               raw[0][1].x, raw[0][1].y, raw[0][1].z, raw[0][1].w};
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) {
            raw[k][0] = raw[k + 1][0];
            raw[k][1] = raw[k + 1][1];
        }
        fetch(raw[kAhead - 1]);
        // (as integers NaN is above infinity, and above the rest)
        uint32_t two = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) two = __vmaxu2(two, x[i] & 0x7FFF7FFFu);
        uint32_t top = max(two << 16, two & 0xFFFF0000u);
#pragma unroll
        for (int i = kLanes / 2; i > 0; i >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
        const bool odd = top >= 0x7F800000u;    // NaN or an infinity
        // 2^e brings the largest element to [128, 256); fp16 holds the rest as it is, down
        // to steps of 2^-24
        const int e = top > 0 && !odd ? min(134 - (int)(top >> 23), 126) : 0;
        const float up = __int_as_float((127 + e) << 23);
        if (l == 0)
            sh->c[n] = n >= pc.rows ? 0.f
                       : odd        ? __int_as_float(0x7FC00000)
                                    : fabsf(j.softmax_scale) * 1.4426950408889634f / up;
        uint32_t hi[4], lo[4];
        const float by = sign * up;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint16_t h8[2], l8[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t w = x[2 * i + k];
                uint32_t v, back;
                asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                    : "=r"(v)
                    : "f"(__uint_as_float(w & 0xFFFF0000u) * by), "f"(__uint_as_float(w << 16) * by));
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h8[k]) : "r"(v));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(h8[k]));
                const __half2 d = __hsub2(*reinterpret_cast<__half2 *>(&v), *reinterpret_cast<__half2 *>(&back));
                asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
                    : "=h"(l8[k]) : "r"(*reinterpret_cast<const uint32_t *>(&d)));
            }
            hi[i] = h8[0] | (uint32_t)h8[1] << 16;
            lo[i] = l8[0] | (uint32_t)l8[1] << 16;
        }
        const int r = n & 127, sw = D == 128 ? r & 7 : (r >> 1) & 3;
        char *to = smem_q + (n >> 7) * (2 * kSide) + r * D + ((l ^ sw) << 4);
        *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(to + kSide) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// The next piece, for a warp that is not the producer; false: no more.
__device__ __forceinline__ bool px_next(PxShared *sh, int *err, uint32_t &pieces, PxPiece &p, int lane)
{
    const int i = pieces % kPxPieces;
    bool ok = px_wait(sh, err, &sh->piece_full[i], pieces / kPxPieces & 1);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok) p = sh->piece[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->piece_empty[i]);
    ++pieces;
    return ok && p.rows > 0;
}

// Which of a tile's 128 tokens a row sees, a bit each: its token is new token i of the
// sequence, `at` the tile's first token.
struct PxSees {
    uint32_t w[4];
    __device__ __forceinline__ PxSees(const PrefixJob &j, const PxPiece &pc, int i, bool live, int at)
    {
        const uint32_t *m = j.mask && live ? j.mask + (int64_t)(pc.first + i) * j.words : nullptr;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int p = at + 32 * k, q = p - pc.ctx;  // of the word's first token
            // tokens before the new ones, and before the end
            auto first = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; };
            uint32_t see;
            if (j.mask) {
                see = first(-q);
                if (m && q > -32) {
                    // bits q to q + 31 of the row's mask
                    const int a = q >> 5, s = q & 31;
                    const uint32_t lo = a >= 0 && a < j.words ? m[a] : 0u;
                    const uint32_t hi = a + 1 >= 0 && a + 1 < j.words ? m[a + 1] : 0u;
                    see |= __funnelshift_r(lo, hi, s);
                }
            } else {
                see = first(i + 1 - q);
            }
            w[k] = see & first(pc.end - p);
        }
    }
};

__device__ __forceinline__ bool px_far(float M) { return fabsf(M) >= kPxFar && M != kPxNone; }

// A tile whose value scales lie apart (bf: values and weights are bf16), or of rows whose
// maxima are far from 0, from its half `q` on, 16 scores at a time (what runs seldom is
// short).  A score s u is not rounded before M is taken from it, which is right while M's
// own steps are small.  Beyond kPxFar it is rounded first, as M has been: the difference
// of a maximum from itself would else be anything within half a step (16 at 2^28).
// sees, lost: as below, null where all tokens count.
struct PxRow {
    float M, l;
    bool ok;
};
template <int D>
__device__ __forceinline__ PxRow px_soft_far(PxShared *sh, int *err, uint32_t s_at, uint32_t o_at,
                                             uint64_t *pv_done, uint32_t count, bool first, int q,
                                             const float4 *sc, bool bf, float c, float M, float l,
                                             const uint32_t *sees, const uint32_t *lost)
{
    bool ok = true;
#pragma unroll 1
    for (; q < 2; ++q) {
        // 16 scores, and which of them count
        auto scores = [&](int k, float (&x)[16]) {
            float a[8], b[8];
            tc_ld8(s_at + q * 64 + 16 * k, a);
            tc_ld8(s_at + q * 64 + 16 * k + 8, b);
            tc_wait_ld(a);
            tc_wait_ld(b);
            const int at = 2 * q + (k >> 1), up = 16 * (k & 1);
            const uint32_t gone = lost ? lost[at] >> up : 0u;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] = i < 8 ? a[i & 7] : b[i & 7];
                if (gone >> i & 1) x[i] = __int_as_float(0x7FC00000);
            }
            return sees ? sees[at] >> up : ~0u;
        };
        float m = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            float x[16], a = -INFINITY;
            const uint32_t see = scores(k, x);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (see >> i & 1) a = fmaxf(a, x[i]);
            const float4 f = sc[4 * q + k];
            if (a > -INFINITY && f.w > -INFINITY) m = fmaxf(m, __fmul_rn(a, c * f.x));
        }
        float to = M, scale = 1.f;
        if (M == kPxNone) {
            if (m > -INFINITY) to = ceilf(m) - kPxUnit;
        } else if (m - M > kPxMost) {
            to = ceilf(m) - kPxUnit;
            scale = pow2_int(M - to);
        }
        M = to;
        l *= scale;
        if (__any_sync(0xFFFFFFFFu, scale != 1.f)) {
            if (!first) {
                ok = ok && px_wait(sh, err, pv_done, (count - 1) & 1);
                tc_fence_after();
#pragma unroll 1
                for (int i = 0; i < D; i += 8) {
                    float o[8];
                    tc_ld8(o_at + i, o);
                    tc_wait_ld(o);
#pragma unroll
                    for (int n = 0; n < 8; ++n) o[n] *= scale;
                    tc_st8(o_at + i, o);
                }
            }
            if (q) {
                tc_wait_st();
                const uint32_t two = weights_bf16(scale, scale);
#pragma unroll 1
                for (int i = 0; i < 32; i += 8) {
                    float o[8];
                    tc_ld8(s_at + i, o);
                    tc_wait_ld(o);
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const uint32_t w = __float_as_uint(o[n]);
                        o[n] = __uint_as_float(bf ? mul_bf16x2(w, two) : scaled_f16(w, scale));
                    }
                    tc_st8(s_at + i, o);
                }
            }
        }
        const bool far = px_far(M);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            float x[16], sum = 0.f, p[8];
            const uint32_t see = scores(k, x);
            const float4 f = sc[4 * q + k];
            const float u = c * f.x, v = f.w - M;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                float w[2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float y = fmaf(x[i + n], u, v);
                    if (far) y = __fsub_rn(__fmul_rn(x[i + n], u), M) + f.w;
                    w[n] = see >> (i + n) & 1 ? ex2f(y) : 0.f;
                    sum += w[n];
                }
                p[i / 2] = __uint_as_float(bf ? weights_bf16(w[0], w[1]) : weights_f16(w[0], w[1]));
            }
            l = fmaf(sum, f.z, l);
            tc_st8(s_at + q * 32 + 8 * k, p);   // (over scores that have been taken)
        }
        tc_wait_st();
    }
    return {M, l, ok};
}

// One tile of a softmax thread: a row's 128 scores to weights, 64 at a time.
// M (a whole number), l: the row's running maximum and sum of weights.  Weights are
// taken against the maximum in use before it is known whether one passes it by too
// much; where one does, M moves, what there is of the row (sums, values, the tile's
// first 64 weights) is scaled by the power of two, and the 64 weights are taken once
// more, which is the last time: they do not pass 2^(kPxUnit + 1) against the new M.
// Returns the half from which on a row's maximum is far from 0 (px_soft_far's), or 2.
// same: pages of 64 tokens or more, one scale for the 64.  EDGE: only the tokens of
// `sees` count, and those of `lost` are NaN.
// (The factors are taken before the scores, the weights stored after them: loads
// and stores between would keep the scores' chains from overlapping.)
template <int D, bool EDGE>
__device__ __forceinline__ int px_soft_tile(PxShared *sh, int *err, uint32_t s_at, uint32_t o_at,
                                            uint64_t *pv_done, uint32_t count, bool first,
                                            const float4 *sc, bool same, float c, float &M, float &l,
                                            const uint32_t *sees, const uint32_t *lost, bool &ok)
{
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
        float s[64];
        tc_ld32(s_at + q * 64, s);
        tc_ld32(s_at + q * 64 + 32, s + 32);
        float4 f[4];
        f[0] = sc[4 * q];
#pragma unroll
        for (int k = 1; k < 4; ++k) {
            f[k] = f[0];
            if (!same) f[k] = sc[4 * q + k];
        }
        tc_wait_ld(s);
        if (EDGE) {
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                const uint32_t see = sees[2 * q + (i >> 5)], gone = lost[2 * q + (i >> 5)];
                if (!(see >> (i & 31) & 1))
                    s[i] = -INFINITY;
                else if (gone >> (i & 31) & 1)
                    s[i] = __int_as_float(0x7FC00000);
            }
        }
        // (a score that is hidden, -inf, keeps its sign against a factor of 0)
        float by[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            by[k] = c * f[k].x;
            if (EDGE && by[k] == 0.f) by[k] = 0x1p-126f;
        }
        uint32_t p[32];
        float add;
#pragma unroll 1
        for (bool again = false;; again = true) {
            float top = -INFINITY;
            add = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 u = make_float2(by[k], by[k]);
                const float2 v = make_float2(f[k].y - M, f[k].y - M);
                float2 sum;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 y = fma2(make_float2(s[16 * k + 2 * i], s[16 * k + 2 * i + 1]), u, v);
                    top = max3(top, y.x, y.y);
                    const float2 w = make_float2(ex2f(y.x), ex2f(y.y));
                    sum = i ? add2(sum, w) : w;
                    p[8 * k + i] = weights_f16(w.x, w.y);
                }
                add = fmaf(sum.x + sum.y, f[k].z, add);
            }
            // (M is unset, at kPxNone, before a row's first token)
            if (again || !__any_sync(0xFFFFFFFFu, top > kPxMost)) break;
            float to = top > kPxMost ? M + (ceilf(top) - kPxUnit) : M;
            float scale = pow2_int(M - to);
            if (M == kPxNone) {
                // no sum was taken against it: from the scores themselves (it stays where
                // there are none)
                float m = -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float a = s[16 * k], b = s[16 * k + 1];
#pragma unroll
                    for (int i = 2; i < 16; i += 2) a = max3(a, s[16 * k + i], s[16 * k + i + 1]);
                    m = fmaxf(m, fmaf(fmaxf(a, b), by[k], f[k].y));
                }
                to = m > -INFINITY ? ceilf(m) - kPxUnit : M;
                scale = 1.f;
            }
            if (__any_sync(0xFFFFFFFFu, px_far(M) || px_far(to))) {
                tc_wait_st();
                return q;
            }
            M = to;
            l *= scale;
            if (!first) {
                ok = ok && px_wait(sh, err, pv_done, (count - 1) & 1);
                tc_fence_after();
#pragma unroll 1
                for (int i = 0; i < D; i += 8) {
                    float o[8];
                    tc_ld8(o_at + i, o);
                    tc_wait_ld(o);
#pragma unroll
                    for (int n = 0; n < 8; ++n) o[n] *= scale;
                    tc_st8(o_at + i, o);
                }
            }
            if (q) {
                tc_wait_st();
#pragma unroll 1
                for (int i = 0; i < 32; i += 8) {
                    float o[8];
                    tc_ld8(s_at + i, o);
                    tc_wait_ld(o);
#pragma unroll
                    for (int n = 0; n < 8; ++n)
                        o[n] = __uint_as_float(scaled_f16(__float_as_uint(o[n]), scale));
                    tc_st8(s_at + i, o);
                }
            }
            tc_wait_st();
        }
        l += add;
        // (over scores that have been taken)
        tc_st32u(s_at + q * 32, p);
    }
    tc_wait_st();
    return 2;
}

template <int D>
__global__ void __launch_bounds__(kPxThreads, 1)
prefix_kernel(const __grid_constant__ PrefixJob j, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v)
{
    constexpr int kSide = kPxTile * D;          // bytes of a tile's keys (or values)
    constexpr int kWideV = kPxTile * D * 2;     // in 16 bits
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
            mbar_init(&sh->empty_k[i], 2);
        }
        for (int i = 0; i < kPxV; ++i) {
            mbar_init(&sh->full_v[i], 1);
            mbar_init(&sh->empty_v[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->full_b[i], 4);
            mbar_init(&sh->empty_b[i], 2);
            mbar_init(&sh->drained[i], 1);
            mbar_init(&sh->turn[i], 1);
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->p_full[i], 4);
            mbar_init(&sh->pv_done[i], 1);
        }
        for (int i = 0; i < kPxRing; ++i) mbar_init(&sh->scales[i], 1);
        for (int i = 0; i < kPxPieces; ++i) {
            mbar_init(&sh->piece_full[i], 1);
            mbar_init(&sh->piece_empty[i], kPxReaders);
        }
        mbar_init(&sh->q_full, kPxSoft);
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
    PxPiece pc;
    uint32_t it = 0, pieces = 0;                // tiles and pieces of this CTA so far
    bool ok = true;

    if (warp < kPxSoft) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPxSoftRegs));
        const int slot = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_at = lanes + slot * 128, o_at = lanes + 256 + slot * 128;
        uint32_t count = 0;                     // this slot's tiles so far
        if (tid == 0) j.part_unit[2 * blockIdx.x] = j.part_unit[2 * blockIdx.x + 1] = -1;
        for (;;) {
            // (all of them go on, or none)
            const bool go = px_next(sh, j.err, pieces, pc, lane);
            if (bar_or(1, kPxSoft * 32, !go)) break;
            const bool wide = pc.wide();
            px_queries<D>(j, sh, s_q, pc);
            fence_async();
            bar_or(1, kPxSoft * 32, false);     // the rows' factors are there
            if (lane == 0) mbar_arrive(&sh->q_full);
            const int row = wide ? slot * 128 + r : r;
            const float c = sh->c[row];
            const int token = (pc.row0 + row) / j.G;  // of the span's
            const int step = wide ? 1 : 2, from = wide ? 0 : slot, n = pc.t1 - pc.t0;
            float M = kPxNone, l = 0.f, far = 0.f;
            for (int i = from; i < n && ok; i += step, ++count) {
                const int ring = (int)((it + i) % kPxRing);
                ok = px_wait(sh, j.err, &sh->scales[ring], ((it + i) / kPxRing) & 1);
                ok = ok && px_wait(sh, j.err, &sh->s_full[slot], count & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const int at = (pc.t0 + i) * kPxTile;
                const bool edge = at + kPxTile > pc.ctx;
                uint32_t seen[4], lost[4];
                // which tokens a row sees, and are lost (known once the values are converted)
                auto look = [&] {
                    const uint32_t sb = (it + i) & 1;
                    ok = ok && px_wait(sh, j.err, &sh->full_b[sb], ((it + i) >> 1) & 1);
                    const PxSees sees(j, pc, token, row < pc.rows, at);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        seen[k] = sees.w[k];
                        lost[k] = sh->lost[sb][k];
                    }
                    ok = __all_sync(0xFFFFFFFFu, ok);
                };
                int half = 0;
                if (__builtin_expect(!edge, 1)) {
                    half = px_soft_tile<D, false>(sh, j.err, s_at, o_at, &sh->pv_done[slot], count,
                                                  i == from, sh->sc[ring], j.block >= 64, c, M, l,
                                                  nullptr, nullptr, ok);
                } else {
                    look();
                    if (ok && !(sh->kind[ring] & kPxApart))
                        half = px_soft_tile<D, true>(sh, j.err, s_at, o_at, &sh->pv_done[slot], count,
                                                     i == from, sh->sc[ring], j.block >= 64, c, M, l,
                                                     seen, lost, ok);
                }
                // (value scales apart, and maxima far from 0, have a way of their own)
                if (__builtin_expect(half < 2, 0)) {
                    const bool bf = sh->kind[ring] & kPxApart;
                    if (bf && !edge) look();
                    const PxRow r = px_soft_far<D>(sh, j.err, s_at, o_at, &sh->pv_done[slot], count,
                                                   i == from, half, sh->sc[ring], bf, c,
                                                   M == kPxMark ? far : M, l, edge || bf ? seen : nullptr,
                                                   edge || bf ? lost : nullptr);
                    far = r.M;
                    M = px_far(far) ? kPxMark : far;
                    l = r.l;
                    ok = ok && r.ok;
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full[slot]);
            }
            if (M == kPxMark) M = far;
            const bool had = from < n;
            if (had && ok) ok = px_wait(sh, j.err, &sh->pv_done[slot], (count - 1) & 1);
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
            if (tid == 0) {
                if (pc.t0 == 0) j.unit_ctas[pc.unit].x = blockIdx.x;
                if (pc.t1 == pc.tiles) j.unit_ctas[pc.unit].y = blockIdx.x;
                if (!pc.whole()) j.part_unit[2 * blockIdx.x + (pc.t0 == 0 ? 1 : 0)] = pc.unit;
            }
            // (the values' unit, the piece's power of two)
            const int e = (sh->kind[(it + n - 1) % kPxRing] & (kPxApart - 1)) - 64;
            const float unit = __int_as_float((127 + e) << 23);
            float *part = px_part(j, ctas, blockIdx.x, pc.t0, pc.whole(), pc.unit);
            float4 *to = reinterpret_cast<float4 *>(part) + row;
            float *ml = part + (size_t)D * kPxRows + row;
            if (wide) {
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    float o[32];
                    tc_ld32(o_at + i, o);
                    tc_wait_ld(o);
#pragma unroll
                    for (int q = 0; q < 32; ++q) o[q] *= unit;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        to[(i / 4 + q) * kPxRows] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
                ml[0] = M;
                ml[kPxRows] = l;
            } else {
                // both slots' sums of a row; half of its elements each
                const float m0 = sh->m[0][r], m1 = n > 1 ? sh->m[1][r] : kPxNone;
                const float m = fmaxf(m0, m1), f0 = ex2f(m0 - m), f1 = n > 1 ? ex2f(m1 - m) : 0.f;
                const float u0 = f0 * unit, u1 = f1 * unit;
#pragma unroll 1
                for (int i = slot * (D / 2); i < (slot + 1) * (D / 2); i += 16) {
                    float a[16], b[16];
                    tc_ld8(lanes + 256 + i, a);
                    tc_ld8(lanes + 256 + i + 8, a + 8);
                    if (n > 1) {
                        tc_ld8(lanes + 384 + i, b);
                        tc_ld8(lanes + 384 + i + 8, b + 8);
                    }
                    tc_wait_ld(a);
                    if (n > 1) tc_wait_ld(b);
#pragma unroll
                    for (int q = 0; q < 16; ++q) a[q] = n > 1 ? fmaf(b[q], u1, a[q] * u0) : a[q] * unit;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        to[(i / 4 + q) * kPxRows] = make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
                }
                if (slot == 0) {
                    ml[0] = m;
                    ml[kPxRows] = n > 1 ? fmaf(sh->l[1][r], f1, sh->l[0][r] * f0) : sh->l[0][r];
                }
            }
            tc_fence_before();
            bar_or(1, kPxSoft * 32, false);     // queries and sums may be overwritten
            it += n;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPxSideRegs));
        if (warp < 12) {
            // ---- the values to fp16 or bf16, a token a thread
            const int tk = tid - kPxSoft * 32;
            while (ok && px_next(sh, j.err, pieces, pc, lane)) {
                for (int t = pc.t0; t < pc.t1; ++t, ++it) {
                    const int st = it % kPxV, sb = it & 1, ring = it % kPxRing;
                    ok = px_wait(sh, j.err, &sh->scales[ring], (it / kPxRing) & 1);
                    ok = ok && px_wait(sh, j.err, &sh->full_v[st], (it / kPxV) & 1);
                    ok = ok && px_wait(sh, j.err, &sh->empty_b[sb], ((it >> 1) & 1) ^ 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const uint32_t up = sh->up[ring][tk >> 4], more = sh->more[ring][tk >> 4];
                    const bool bf = sh->kind[ring] & kPxApart;
                    char *src = s_v + st * kSide + tk * D;
                    char *dst = s_b + sb * kWideV + tk * 128;
                    const int sw = D == 128 ? tk & 7 : (tk >> 1) & 3;
                    // New tokens may be NaN, which rows that do not see them would get (0 times
                    // NaN): cleared, as is what lies behind the last token.  In bf16 NaN would
                    // become a number.
                    if (__builtin_expect(bf || (t + 1) * kPxTile > pc.ctx, 0)) {
                        bool nan = false;
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(src + (i << 4));
                            nan |= has_nan(w.x) | has_nan(w.y) | has_nan(w.z) | has_nan(w.w);
                        }
                        const uint32_t m = __ballot_sync(0xFFFFFFFFu, nan);
                        if (lane == 0) sh->lost[sb][warp - kPxSoft] = m;
#pragma unroll 1
                        for (int i = 0; nan && i < D / 16; ++i)
                            *reinterpret_cast<uint4 *>(src + (i << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    auto bring = [&](auto convert) {
#pragma unroll 2
                        for (int i = 0; i < D / 16; ++i) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(src + ((i ^ sw) << 4));
                            uint4 a, b;
                            convert(w.x, a.x, a.y);
                            convert(w.y, a.z, a.w);
                            convert(w.z, b.x, b.y);
                            convert(w.w, b.z, b.w);
                            char *at = dst + (i >> 2) * (kPxTile * 128);
                            const int q = (i & 3) * 2;
                            *reinterpret_cast<uint4 *>(at + ((q ^ (tk & 7)) << 4)) = a;
                            *reinterpret_cast<uint4 *>(at + (((q + 1) ^ (tk & 7)) << 4)) = b;
                        }
                    };
                    if (__builtin_expect(!bf, 1))
                        bring([&](uint32_t w, uint32_t &lo, uint32_t &hi) { e4m3_to_f16(w, up, lo, hi); });
                    else
                        bring([&](uint32_t w, uint32_t &lo, uint32_t &hi) {
                            e4m3_to_bf16(w, up, lo, hi);
                            lo = mul_bf16x2(lo, more);
                            hi = mul_bf16x2(hi, more);
                        });
                    fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh->full_b[sb]);
                        mbar_arrive(&sh->empty_v[st]);
                    }
                }
            }
        } else if (warp == 12) {
            // ---- producer: the pieces, and the pages of each tile, looked up 32 at a time
            const int shift = 31 - __clz(j.block), per_tile = kPxTile >> shift;
            const int inner = lane & (per_tile - 1);
            const PrefixSpan all = j.span[j.groups + j.B];
            const int mine = min((int)blockIdx.x, all.rows), next = min(mine + 1, all.rows);
            PxWalk walk = {span_at(all.start, all.rows, mine), span_at(all.start, all.rows, next),
                           all.loose0};
            for (bool more = true; ok && more;) {
                more = walk.next(j, pc, lane);
                if (!more) pc.rows = 0;
                const int slot = pieces % kPxPieces;
                ok = px_wait(sh, j.err, &sh->piece_empty[slot], (pieces / kPxPieces & 1) ^ 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (lane == 0) {
                    sh->piece[slot] = pc;
                    mbar_arrive(&sh->piece_full[slot]);
                }
                ++pieces;
                if (!ok || !more) break;
                const int pages = (int)(((long long)pc.end + j.block - 1) >> shift);
                const int32_t *tab = j.table + (int64_t)pc.lead * j.cols + pc.page0;
                auto window = [&](int w0, int &page, float &ks, float &vs) {
                    page = w0 + lane < pages ? tab[w0 + lane] : -1;
                    if (w0 + lane < pages && (page < 0 || page >= j.pages)) {
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
                // The piece's power of two: of the largest scale here.
                auto power = [](float v) { return (int)(__float_as_uint(v) >> 23) - 127; };
                const int unit = max(__reduce_max_sync(0xFFFFFFFFu, page >= 0 ? power(vs) : -64), -40);
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
                    const bool live = w0 + lane < pages;
                    // (behind the last page the tile's first one once more: tokens
                    // of weight 0, but no NaN)
                    const int begin = __shfl_sync(0xFFFFFFFFu, page, p0 - w0);
                    const int row = max(live ? page : begin, 0) * j.H + pc.h;
                    auto fetch = [&](const CUtensorMap *map, char *dst, uint64_t *bar) {
                        asm volatile(
                            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::"
                            "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
                            "l"(map), "r"(0), "r"(0), "r"(row), "r"(smem_u32(bar))
                            : "memory");
                    };
                    const int sk = it % kPxK, sv = it % kPxV, ring = it % kPxRing;
                    ok = px_wait(sh, j.err, &sh->empty_k[sk], ((it / kPxK) & 1) ^ 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_tx(&sh->full_k[sk], kSide);
                    __syncwarp();
                    if (mine) fetch(&map_k, s_k + sk * kSide + inner * j.block * D, &sh->full_k[sk]);
                    // (the tile that had these places is behind the scores of all
                    // but the last tiles)
                    const int e = live ? power(vs) - unit : 0;
                    const bool bf = __any_sync(0xFFFFFFFFu, mine && (e > kPxAbove || e < -kPxBelow));
                    if (lane == 0) sh->kind[ring] = unit + 64 + (bf ? kPxApart : 0);
                    if (mine) {
                        const float f = __uint_as_float((__float_as_uint(vs) & 0x7FFFFFu) | 0x3F800000u);
                        const float lg = f == 1.f ? 0.f : log2f(f);
                        const float4 sc = live ? make_float4(ks, bf ? INFINITY : lg, 1.f / f, lg)
                                               : make_float4(1.f, -INFINITY, 0.f, -INFINITY);
                        const uint32_t up = bf ? (uint32_t)(127 + 120 + min(e, kPxTop)) << 7
                                               : (uint32_t)(15 + e) << 10;
                        const uint32_t more = (uint32_t)(127 + max(e - kPxTop, 0)) << 7;
                        for (int i = 0; i < j.block >> 4; ++i) {
                            sh->sc[ring][inner * (j.block >> 4) + i] = sc;
                            sh->up[ring][inner * (j.block >> 4) + i] = up | up << 16;
                            sh->more[ring][inner * (j.block >> 4) + i] = more | more << 16;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->scales[ring]);
                    ok = px_wait(sh, j.err, &sh->empty_v[sv], ((it / kPxV) & 1) ^ 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_tx(&sh->full_v[sv], kSide);
                    __syncwarp();
                    if (mine) fetch(&map_v, s_v + sv * kSide + inner * j.block * D, &sh->full_v[sv]);
                }
            }
            // after a wait that ran out: copies still in flight land before the exit
            if (!ok) {
                for (int i = 0; i < kPxK; ++i) mbar_wait_n(&sh->full_k[i], (it / kPxK) & 1, 1u << 12);
                for (int i = 0; i < kPxV; ++i) mbar_wait_n(&sh->full_v[i], (it / kPxV) & 1, 1u << 12);
            }
        } else if (warp < 15) {
            // ---- issuers of the products, one a slot.  A step: the product of the slot's
            // weights with the tile's values, then the scores of its next tile, whose
            // place the weights have held.  (The whole warp walks along, so that
            // descriptors lie in uniform registers; one thread issues.)
            constexpr uint32_t kSums = 1u << 4, kM = 128u >> 4 << 24;  // fp32 sums, M = 128
            constexpr uint32_t kIdS = kSums | (128u >> 3 << 17) | kM;
            // fp16 both, or bf16; B with its rows (tokens) as the products' dimension
            constexpr uint32_t kIdO = kSums | 1u << 16 | ((uint32_t)D >> 3 << 17) | kM;
            constexpr uint32_t kBf16 = 1u << 7 | 1u << 10;
            const int slot = __shfl_sync(0xFFFFFFFFu, warp - 13, 0);
            const uint32_t col = tmem + slot * 128;
            const uint64_t dk0 = tc_desc(smem_u32(s_k), 16, 8 * D, kSwz);
            const uint64_t dq0 = tc_desc(smem_u32(s_q), 16, 8 * D, kSwz);
            const uint64_t db0 = tc_desc(smem_u32(s_b), kPxTile * 128, 1024, 2);
            const bool one = elect_one();
            uint32_t count = 0, wides = 0;
            while (ok && px_next(sh, j.err, pieces, pc, lane)) {
                const bool wide = pc.wide();
                const int n = pc.t1 - pc.t0, step = wide ? 1 : 2;
                const uint64_t dq = dq0 + (wide ? slot : 0) * (2 * kSide >> 4);
                ok = px_wait(sh, j.err, &sh->q_full, (pieces - 1) & 1);
                // tiles of this slot, its own first one ahead
#pragma unroll 1
                for (int i = (wide ? 0 : slot) - step; i < n && ok; i += step) {
                    const bool now = i >= 0, next = i + step < n;
                    const uint32_t t = it + i, sb = t & 1;
                    const uint32_t tn = t + step, st = tn % kPxK;
                    // (the weights last: from then on nothing is in the way)
                    if (next) ok = px_wait(sh, j.err, &sh->full_k[st], (tn / kPxK) & 1);
                    uint32_t id = kIdO;
                    if (now) {
                        ok = ok && px_wait(sh, j.err, &sh->full_b[sb], (t >> 1) & 1);
                        if (sh->kind[t % kPxRing] & kPxApart) id |= kBf16;
                        // the slots take turns: one's softmax runs under the other's
                        // products (side by side, both wait for the products, then the
                        // products for both; free to run, one gets a tile ahead and
                        // waits for values that the other holds)
                        if (wide && (slot || wides))
                            ok = ok && px_wait(sh, j.err, &sh->turn[slot ^ 1], (wides + slot + 1) & 1);
                        ok = ok && px_wait(sh, j.err, &sh->p_full[slot], count++ & 1);
                    }
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (now && one) {
                        const uint64_t db = db0 + sb * (kWideV >> 4);
#pragma unroll
                        for (int k = 0; k < kPxTile / 16; ++k)
                            tc_mma_ts(col + 256, col + 8 * k, db + 128 * k, id, k || i >= step);
                        tc_commit(&sh->pv_done[slot]);
                        // (both slots release a tile)
                        tc_commit(&sh->empty_b[sb]);
                        if (!wide) tc_commit(&sh->empty_b[sb]);
                    }
                    if (next && one) {
                        const uint64_t dk = dk0 + st * (kSide >> 4);
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            tc_mma(col, dq + 2 * k, dk + 2 * k, kIdS, k);
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            tc_mma(col, dq + (kSide >> 4) + 2 * k, dk + 2 * k, kIdS, 1);
                        tc_commit(&sh->s_full[slot]);
                        tc_commit(&sh->empty_k[st]);
                        if (!wide) tc_commit(&sh->empty_k[st]);
                    }
                    if (now && wide) {
                        ++wides;
                        if (one) mbar_arrive(&sh->turn[slot]);
                    }
                    __syncwarp();
                }
                it += n;
            }
            // after a wait that ran out: products still in flight end before the exit
            if (!ok && one) {
                tc_commit(&sh->drained[slot]);
                mbar_wait_n(&sh->drained[slot], 0, 1u << 12);
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

cudaError_t prefix_prep_launch(const PrefixJob &j, int sms, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    pdl_config(cfg, at, dim3(kPrepCtas), dim3(kPrepThreads), 0, s);
    return cudaLaunchKernelEx(&cfg, prefix_prep_kernel, j, tail_warps(sms));
}

cudaError_t prefix_launch(const PrefixJob &j, int sms, cudaStream_t s)
{
    CUtensorMap mk, mv;
    if (!cache_map(&mk, j.cache[0], j.D, j.block, j.block, j.pages, j.H) ||
        !cache_map(&mv, j.cache[1], j.D, j.block, j.block, j.pages, j.H))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    // (one CTA an SM, also at D = 64: each holds all of the SM's tensor memory)
    pdl_config(cfg, at, dim3(sms), dim3(kPxThreads), prefix_smem(128), s);
    return j.D == 64 ? cudaLaunchKernelEx(&cfg, prefix_kernel<64>, j, mk, mv)
                     : cudaLaunchKernelEx(&cfg, prefix_kernel<128>, j, mk, mv);
}

}  // namespace sv
