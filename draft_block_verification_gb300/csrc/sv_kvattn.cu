// sv_kvattn.cu -- attention over the paged 8-bit cache.
//
// Token i of sequence b's new tokens (i = 0 .. n_b - 1, at position
// L_b - n_b + i of the L_b tokens in the cache) attends with query head g to
// the cache's head g / G:
//   z_p = scale * q . (k_p s^k),  w_p = exp(z_p - max z),
//   o = sum_p w_p (v_p s^v) / sum_p w_p
// over the positions it sees: those up to its own, or, with a mask, every
// position before the new tokens and the new tokens whose bit is set.
//
// Shape of the work.  A sequence's n_b G query rows of one cache head read the
// same keys and values, so they are handled together, up to 128 at a time.
// Reading the cache bounds the call up to about 64 rows a head (256 bytes a
// token and head at D = 128); the tensor cores take both products:
//   S^T [128 tokens x N rows] = K Q^T     (K is the A operand, as it lies)
//   O^T [D x N rows]         += V^T P^T   (V is the A operand, as it lies)
// With tokens and head elements on the 128 rows of the product, N is the number
// of query rows rounded to 16: a single token pays for 16 rows, not for 128.
//
// The cache's bytes go from TMA to the tensor cores untouched (e4m3); so the
// other operand is e4m3 as well, in two parts.  A bf16 query (8 significant
// bits, scaled by a power of two per row) is the sum of two e4m3 values (4 bits
// each): q = hi + lo exactly, up to 2^-17 of the row's largest element (which is
// brought to [128, 256); the least step of e4m3 is 2^-9).  A weight p is rounded
// to hi + lo with a relative error of 2^-8 and the 2^-11 of fp16 at most (2^-10.5
// in the mean square, under the output's own rounding to bf16), down to a step
// of 2^-16.5 of the weight at the running maximum; lo carries a scale of its own
// and accumulates apart.  Sums, maxima and the rescaling are fp32.
//
// Scales of pages differ from token to token, which is a row of S^T: the key's
// scale multiplies there, and the value's scale goes into the exponent,
//   w'_p = 2^(z_p log2 e + log2 s^v_p - M),  M = max over the same sum,
// so that O needs no scale; the sum of weights takes w'_p / s^v_p.
//
// That makes a weight's step one of the largest w', so a page of a large scale
// would take the others' bits: 2^12 apart cost 1.6% of an output that came from
// the small one, 2^18 all of it.  A piece of work whose pages' value scales lie
// 2^6 apart or more is therefore taken in rounds, one for each class of scales
// (six exponents), with weights and a running maximum of its own, added up in
// fp32.  A CTA begins with loops that know no rounds and goes over to ones that
// do at the first piece that needs them.  (One set of loops for both took 7% to
// 13% longer on calls without rounds: what they keep takes registers from the
// loops over tiles.)
//
// Split.  The tiles (128 tokens of one unit: sequence, head, row block) of the
// whole call, laid end to end by their cost, are cut into equal spans, one per
// CTA of one wave.  A unit that several CTAs share leaves partial sums in the
// workspace; the last of them to finish joins them in the order of the CTAs, so
// the result does not depend on who that is.
//
// Measured at D = 128, 8 cache heads, 4 query heads each, equal lengths: a tile
// of 32 KB takes 0.76 us on an SM for up to 32 rows (6.5 TB/s over all), 0.85 for
// 48, 0.90 for 64, 1.31 for 96, 1.65 for 128, where the softmax warps bound it; a
// unit 7 to 10 us more up to 32 rows, 12 to 20 above (queries, the first tiles'
// maxima, new tokens, the output), and a call some 12.  128 single tokens over
// 4,096 to 8,192 take 314 us (5.2 TB/s, 76% of the copy rate), 64 draft blocks of
// 9 to 17 over 2,048 to 4,096 208 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "sv_common.cuh"
#include "sv_kv.cuh"
#include "sv_tc.cuh"

namespace sv {

constexpr int kTile = 128;             // tokens of a tile (>> 7 below)
constexpr int kRowsMax = 128;          // query rows of a unit
constexpr int kAtStages = 4;           // tiles in flight
constexpr int kSoftWarps = 16;         // four warpgroups
// + a producer, two issuers, and an idle warp that makes up a warpgroup with them
constexpr int kAtThreads = kSoftWarps * 32 + 128;
// Registers: the launch gives each thread 96 of the SM's 65,536; the softmax
// warps hold up to 32 scores and 32 sums each and take what the others leave
// (128 * 56 + 512 * 104 <= 640 * 96).
constexpr int kAtRegs = 96, kSideRegs = 56, kSoftRegs = 104;
static_assert(128 * kSideRegs + kSoftWarps * 32 * kSoftRegs <= kAtThreads * kAtRegs, "registers");
constexpr float kNone = -1e30f;        // running maximum before any token
constexpr int kClass = 6;              // value scales of a class: less than 2^6 apart
// Rounds that the producer may be ahead of a reader of `more`: a tile each, at
// most those in flight and one.
constexpr int kRounds = 8;
static_assert(kRounds > kAtStages + 1, "rounds");
constexpr int kGaveUp = 2;             // AttnShared::abort: roles without rounds end

// ---------------------------------------------------------------------------
// The units of a call.
// ---------------------------------------------------------------------------
struct SeqWork {
    int n, L, first;         // new tokens, tokens, first row of q
    int tiles, blocks, rows; // tiles of a unit, row blocks, rows of a block
    int cost;                // of a tile
    long long work;          // cost of the sequence
    bool bad;
};
// Rows of the products for this many query rows: the two (up to 64) or four
// warpgroups of a tile have 8 rows each, or 16, 24, 32.
__device__ __forceinline__ int round_rows(int rows)
{
    return rows <= 64 ? (rows + 15) & ~15 : (rows + 31) & ~31;
}
// Time of a tile by its rows, as measured: even spans of it are even in time.
__device__ __forceinline__ int tile_cost(int N)
{
    // in units of 0.04 us (152 units of 4,096 and 16,384 tokens, D = 128; a unit's
    // start and end, 7 to 20 us, are not in it)
    return N <= 32 ? 18 : N <= 48 ? 20 : N <= 64 ? 22 : N <= 96 ? 34 : 42;
}

__device__ __forceinline__ SeqWork seq_work(const AttendJob &j, int b)
{
    SeqWork s;
    s.first = j.cu[b];
    const int end = j.cu[b + 1];
    s.L = j.kv_len[b];
    s.n = end - s.first;
    s.bad = s.first < 0 || end > j.T || s.n < 0 || s.L < s.n ||
            ((s.L + (long long)j.block - 1) >> (31 - __clz(j.block))) > j.cols;
    if (s.bad) s.n = 0;
    const long long all = (long long)s.n * j.G;
    s.tiles = (int)(((long long)s.L + kTile - 1) >> 7);
    s.blocks = (int)((all + kRowsMax - 1) >> 7);
    s.rows = s.blocks <= 1 ? (int)all : (int)div_pos(all + s.blocks - 1, s.blocks);
    s.cost = tile_cost(round_rows(s.rows));
    s.work = (long long)s.tiles * s.blocks * j.H * s.cost;
    return s;
}

// A CTA's share of one unit, walked alike by every role.  Costs of tiles, laid
// end to end, are cut into equal spans; a tile belongs to the span that its
// first unit of cost lies in.
struct Piece {
    int b, h, row0, rows;    // sequence, cache head, first row (of n G) and rows
    int t0, t1, tiles;       // tiles [t0, t1) of the unit's
    int cost;                // of a tile
    long long unit0;         // where the unit starts in the call's cost
    int L, n, first;
};
struct PieceWalk {
    long long pos, end;      // the next tile's start, the span's end
    int b, h, block, tile;   // the next tile
    SeqWork s;
    // first, x: the sequence that `from` lies in, and where
    __device__ __forceinline__ void start(const AttendJob &j, int first, long long x,
                                          long long from, long long to)
    {
        pos = from;
        end = to;
        b = first;
        h = block = tile = 0;
        if (pos < end) {
            s = seq_work(j, b);
            // on to the first tile that starts within the span
            long long t = div_pos(x + s.cost - 1, s.cost);
            pos += t * s.cost - x;
            const long long u = div_pos(t, s.tiles);
            tile = (int)(t - u * s.tiles);
            h = (int)div_pos(u, s.blocks);
            block = (int)(u - (long long)h * s.blocks);
        }
    }
    __device__ __forceinline__ bool next(const AttendJob &j, Piece &p)
    {
        if (pos >= end) return false;
        while (h >= j.H || s.work == 0) {
            s = seq_work(j, ++b);
            h = 0;
        }
        const long long left = end - pos, all = (long long)(s.tiles - tile) * s.cost;
        const int n = left >= all ? s.tiles - tile : (int)div_pos(left + s.cost - 1, s.cost);
        p.t0 = tile;
        p.t1 = tile + n;
        p.b = b;
        p.h = h;
        p.row0 = block * s.rows;
        p.rows = min(s.rows, s.n * j.G - p.row0);
        p.tiles = s.tiles;
        p.cost = s.cost;
        p.unit0 = pos - (long long)tile * s.cost;
        p.L = s.L;
        p.n = s.n;
        p.first = s.first;
        pos += (long long)n * s.cost;
        tile += n;
        if (tile == s.tiles) {
            tile = 0;
            if (++block == s.blocks) {
                block = 0;
                ++h;
            }
        }
        return true;
    }
};

// For value scales that lie far apart (a round is a class of them, below).
struct AttnRounds {
    Piece piece;                       // the softmax warps', for its further rounds
    // where the roles without rounds give up: the tiles so far (0 where they do
    // not), the pieces so far, and the piece's start
    uint32_t it, pieces;
    int b;
    long long x, pos;
    uint32_t classes[4];               // exponents of the piece's value scales: of rounds to come
    int more[kRounds];                 // the round's piece needs another one after it
    uint64_t told[kRounds];            // that is known
    uint32_t round[kSoftWarps];        // twice the round, and 1 after a piece's first, per warp
    float old_f[kRowsMax];             // factors of the sums of the rounds before
};

struct AttnShared {
    uint64_t full_k[kAtStages], full_v[kAtStages], empty_k[kAtStages], empty_v[kAtStages];
    uint64_t s_full[2], s_empty[2], p_full[2], pv_done[2], q_full, drained[2];
    // values of a tile with new tokens have been looked over: a pair's tile, or an
    // even or odd one of all four warpgroups
    uint64_t clean[4];
    uint32_t tmem;
    int abort;
    int last;                          // this CTA joins the unit's parts
    int first_b;
    long long first_x, total;          // where the span starts in sequence first_b; the call's cost
    float ks[kAtStages][8], vs[kAtStages][8];  // scales of the tile's pages
    uint32_t looks[kSoftWarps];        // parities of `clean`, a copy per warp
    uint32_t lost[2][4];               // tokens of the tile with NaN in their value, a bit each
    int at[kRowsMax];                  // output row (token * Hq + head), per row
    alignas(16) float c[kRowsMax];     // factor from S to log2 units, per row
    float wmax[kSoftWarps][32];        // tile maxima per warp and row
    alignas(16) float mu[kSoftWarps][32];    // running maximum in use, a copy per warp
    alignas(16) float fac[kSoftWarps][32];   // factor of its last move
    float sum[2][4][kRowsMax];         // sums of weights: warpgroup, quarter of a tile, row
    float top[2][kRowsMax];            // maximum that they are against
    float out_f[2][kRowsMax];          // factors of the output's sums
    short owner[256];                  // CTAs of a shared unit's tiles (spans below a tile)
    long long scan[kAtThreads / 32];
    AttnRounds far;
};

// Workspace of a CTA: two parts (its first and its last unit), each kRowsMax
// rows of D sums, then the rows' maxima and sums of weights.
__host__ __device__ constexpr size_t part_floats(int D) { return (size_t)kRowsMax * (D + 2); }

// ---------------------------------------------------------------------------
// Softmax side of one piece.  Thread: one token of the tile (TMEM lane) for
// the weights, one head element for the output.
//
// Four warpgroups.  Up to 64 rows (turns) two of them take the even tiles and
// two the odd ones, each pair with sums and a running maximum of its own, so
// that one tile's chain (scores, maximum, weights, products) runs under the
// other's; a warpgroup of a pair has half of the rows.  Above, all four share
// each tile, a quarter of the rows each (a second set of sums would not fit the
// tensor memory).  So a thread holds 8 to 32 rows, and four warps hide each
// other's latencies on every scheduler: two warpgroups with up to 64 rows a
// thread took 1.4 to 1.9 times as long.
//
// The running maximum M moves lazily: weights are taken as 2^(y - M + 3.5), and
// M moves only when one would pass 2^8.5 (e4m3 ends at 448).  So most tiles
// need no maximum at all, only a vote of the warpgroup that nothing passes;
// a tile that does is looked at again from its scores.
// ---------------------------------------------------------------------------
constexpr float kUnit = 3.5f;  // log2 of the weight at the running maximum
constexpr float kMost = 8.5f;  // log2 of the largest weight

// Sum v[0 .. N) over the warp's lanes: three halvings leave each lane N / 8
// rows, those from index (lane / 4) * N / 8 on (a quarter of the shuffles of
// whole sums).
template <int N>
__device__ __forceinline__ void warp_sum_rows(float (&v)[N], int lane)
{
#pragma unroll
    for (int level = 0; level < 3; ++level) {
        const int half = N >> (level + 1), bit = 16 >> level;
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if (i >= half) break;
            const float give = up ? v[i] : v[i + half];
            const float keep = up ? v[i + half] : v[i];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, bit);
        }
    }
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], 2);
        v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], 1);
    }
}

// Queries' two parts.  Up to 32 rows they stand side by side in one product:
// with few rows a product's time is that of reading the keys from shared memory
// (64 bytes a cycle), whatever its rows.  Above, the second part's product adds
// to the first's, which saves the softmax warps reading and adding it.
__host__ __device__ constexpr bool stacked(int N) { return N <= 32; }

// R scores of this token; with stacked queries the sum of both parts' products,
// 2 R columns apart.
template <int C8>
__device__ __forceinline__ void load_scores(float (&y)[C8 * 8], uint32_t col)
{
    constexpr int R = C8 * 8;
#pragma unroll
    for (int n = 0; n < R; n += 8) tc_ld8(col + n, y + n);
    if (stacked(2 * R)) {
        float l[R];
#pragma unroll
        for (int n = 0; n < R; n += 8) tc_ld8(col + 2 * R + n, l + n);
        tc_wait_ld(y);
        tc_wait_ld(l);
#pragma unroll
        for (int n = 0; n < R; n += 2) {
            const float2 s = add2(make_float2(y[n], y[n + 1]), make_float2(l[n], l[n + 1]));
            y[n] = s.x;
            y[n + 1] = s.y;
        }
    } else {
        tc_wait_ld(y);
    }
}

template <int D, int C8, bool ROUNDS>
__device__ __forceinline__ bool soft_piece(const AttendJob &j, AttnShared *sh, char *smem_v,
                                           char *smem_p, const Piece &pc, uint32_t &it,
                                           int stage_bytes, int ctas, bool turns, bool ok)
{
    constexpr int R = C8 * 8;                   // rows of this warpgroup
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = warp >> 2, quarter = warp & 3;
    const int part_no = turns ? g & 1 : g, par = turns ? g >> 1 : 0;
    const int tk = quarter * 32 + lane;
    const int r0 = part_no * R;                 // first row of this warpgroup
    const uint32_t lanes = sh->tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t o_own = lanes + 256 + par * 128 + r0 * 2;  // R hi columns, then R lo
    const uint32_t arrivals = turns ? 2 : 1;    // of a warp: 16 a tile
    const int ctx = pc.L - pc.n;
    const int page_in = tk >> (31 - __clz(j.block));
    char *p_row = smem_p + par * (kTile * 128) + tk * 128;
    float *mu = sh->mu[warp];

    float l[R];
#pragma unroll
    for (int n = 0; n < R; ++n) l[n] = 0.f;
    mu[lane] = 0.f;                             // (kept less kUnit)
    __syncwarp();
    uint32_t mine = 0;                          // tiles this warpgroup has taken
    bool none = lane < R;                       // row `lane` has seen no token yet
    bool unset = true;                          // some row has not
    const uint32_t it0 = it;

    bool stop = false;                          // alike in the whole warpgroup
    // The loop over tiles, in a copy for those that every row sees whole and
    // one for the last ones, which reach the new tokens.  (The code between the
    // hot instructions of a loop costs instruction cache.)
    auto tiles = [&](auto is_edge, int from, int to) {
    constexpr bool edge = decltype(is_edge)::value;
#pragma unroll 1
    for (int t = from; t < to && !stop; t += turns ? 2 : 1) {
        const uint32_t it = it0 + (uint32_t)(t - pc.t0);
        const uint32_t st = it % kAtStages, sb = it & 1;
        ok = ok && at_wait(&sh->abort, j.err, &sh->full_v[st], (it / kAtStages) & 1);
        ok = ok && at_wait(&sh->abort, j.err, &sh->s_full[sb], (it >> 1) & 1);
        tc_fence_after();
        const int p0 = t * kTile, pos = p0 + tk;
        const float ks = sh->ks[st][page_in], vs = sh->vs[st][page_in];
        float vl, ivs;
        asm("lg2.approx.f32 %0, %1;" : "=f"(vl) : "f"(vs));  // (-inf: another round's)
        asm("rcp.approx.f32 %0, %1;" : "=f"(ivs) : "f"(ROUNDS ? fmaxf(vs, 0x1p-60f) : vs));
        uint32_t sees = ~0u;  // which rows see this token
        if (edge) {
            const int c = turns ? par : 2 + (int)sb;
            const uint32_t looks = sh->looks[warp];
            ok = ok && at_wait(&sh->abort, j.err, &sh->clean[c], (looks >> c) & 1);
            __syncwarp();
            sh->looks[warp] = looks ^ 1u << c;
            // (its value is cleared: its weight brings NaN to the rows that see it)
            if ((sh->lost[sb][quarter] >> lane) & 1) vl = __int_as_float(0x7FC00000);
            sees = 0;
            if (pos < pc.L) {
                if (pos < ctx) {
                    sees = ~0u;
                } else if (!j.mask) {
                    // rows (row0 + n) / G >= pos - ctx
                    const long long from = (long long)(pos - ctx) * j.G - pc.row0 - r0;
                    sees = from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << (int)from;
                } else {
                    const int k = pos - ctx;
                    if ((k >> 5) < j.words) {
                        const int rows = min(R, pc.rows - r0);
#pragma unroll 1
                        for (int n = 0; n < rows; ++n) {
                            const int64_t tok = pc.first + (pc.row0 + r0 + n) / j.G;
                            const uint32_t m = j.mask[tok * j.words + (k >> 5)];
                            sees |= ((m >> (k & 31)) & 1u) << n;
                        }
                    }
                }
            }
        }
        // Scores in log2 units, the value's scale included, against the maximum
        // in use; again, where that has to move.
        float y[R];
#pragma unroll 1
        for (bool again = false;; again = true) {
            load_scores<C8>(y, lanes + sb * 128 + r0);
            const float2 a2 = make_float2(ks, ks), v2 = make_float2(vl, vl);
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < R; n += 4) {
                const float4 c4 = *reinterpret_cast<const float4 *>(&sh->c[r0 + n]);
                const float4 m4 = *reinterpret_cast<const float4 *>(&mu[n]);
                float2 u = mul2(make_float2(y[n], y[n + 1]), make_float2(c4.x, c4.y));
                float2 w = mul2(make_float2(y[n + 2], y[n + 3]), make_float2(c4.z, c4.w));
                u = add2(fma2(u, a2, v2), make_float2(-m4.x, -m4.y));
                w = add2(fma2(w, a2, v2), make_float2(-m4.z, -m4.w));
                y[n] = u.x; y[n + 1] = u.y; y[n + 2] = w.x; y[n + 3] = w.y;
            }
            if (edge) {
#pragma unroll
                for (int n = 0; n < R; ++n)
                    if (!(sees & (1u << n))) y[n] = -INFINITY;
            }
            if (again) break;
#pragma unroll
            for (int n = 0; n < R; ++n) top = fmaxf(top, y[n]);
            if (__builtin_expect(!bar_or(1 + g, 128, !ok || unset || top > kMost), 1)) break;

            // the tile's maximum of each row: over the warp's tokens, then four warps
            float keep = -INFINITY;
#pragma unroll
            for (int n = 0; n < R; ++n) {
                float m;
                asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(y[n]));
                if (lane == n) keep = m;
            }
            sh->wmax[warp][lane] = keep;
            if (bar_or(1 + g, 128, !ok)) {
                ok = false;
                stop = true;
                break;
            }
            float *fac = sh->fac[warp];
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) m = fmaxf(m, sh->wmax[g * 4 + w][lane]);
            // a row's first maximum is taken as it is; later ones only rise.
            // (Lanes from R on: padding of the arrays, not used.)
            float move = none ? (m > -INFINITY ? m - kUnit : 0.f) : fmaxf(m - kUnit, 0.f);
            const float f = none ? 1.f : ex2f(-move);
            none = none && !(m > -INFINITY);
            if (lane >= R) move = 0.f;
            mu[lane] += move;
            fac[lane] = f;
            unset = __any_sync(0xFFFFFFFFu, none);
            const unsigned moved = __ballot_sync(0xFFFFFFFFu, lane < R && f != 1.f);
            __syncwarp();
            if (!moved) continue;
#pragma unroll
            for (int n = 0; n < R; n += 4) {
                const float4 f4 = *reinterpret_cast<const float4 *>(&fac[n]);
                l[n] *= f4.x; l[n + 1] *= f4.y; l[n + 2] *= f4.z; l[n + 3] *= f4.w;
            }
            if (mine > 0) {
                const uint32_t before = turns ? it - 2 : it - 1;
                ok = at_wait(&sh->abort, j.err, &sh->pv_done[before & 1], (before >> 1) & 1);
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 2 * C8; ++c) {
                    const int n = (c < C8 ? c : c - C8) * 8;
                    if (!((moved >> n) & 0xFFu)) continue;
                    float o[8];
                    tc_ld8(o_own + c * 8, o);
                    tc_wait_ld(o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] *= fac[n + i];
                    tc_st8(o_own + c * 8, o);
                }
                tc_wait_st();
            }
        }
        if (stop) break;
        tc_fence_before();
        __syncwarp();
        if (lane < arrivals) mbar_arrive(&sh->s_empty[sb]);
        // the weights' place is free once the products before have read it
        if (mine > 0) {
            const uint32_t before = turns ? it - 2 : it - 1;
            ok = ok && at_wait(&sh->abort, j.err, &sh->pv_done[before & 1], (before >> 1) & 1);
        }
        ++mine;
        {
            const float2 i2 = make_float2(ivs, ivs);
            constexpr int kStep = C8 % 2 ? 8 : 16;  // rows of a store
#pragma unroll
            for (int c = 0; c < R; c += kStep) {
                uint32_t hi[kStep / 4], lo[kStep / 4];
#pragma unroll
                for (int k = 0; k < kStep / 4; ++k) {
                    uint16_t h8[2], l8[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = c + k * 4 + i * 2;
                        const float2 p = make_float2(ex2f(y[n]), ex2f(y[n + 1]));
                        const float2 s = fma2(p, i2, make_float2(l[n], l[n + 1]));
                        l[n] = s.x;
                        l[n + 1] = s.y;
                        uint32_t h16, p16;
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                            : "=h"(h8[i]) : "f"(p.y), "f"(p.x));
                        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h16) : "h"(h8[i]));
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p16) : "f"(p.y), "f"(p.x));
                        // (p - hi) * 16: exact in fp16
                        __half2 d = __hsub2(*reinterpret_cast<__half2 *>(&p16),
                                            *reinterpret_cast<__half2 *>(&h16));
                        d = __hmul2(d, __floats2half2_rn(16.f, 16.f));
                        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
                            : "=h"(l8[i])
                            : "r"(*reinterpret_cast<uint32_t *>(&d)));
                    }
                    hi[k] = h8[0] | ((uint32_t)h8[1] << 16);
                    lo[k] = l8[0] | ((uint32_t)l8[1] << 16);
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t *v = half ? lo : hi;
                    const int col = r0 * 2 + half * R + c;
                    char *at = p_row + (col >> 7) * (kTile * 128) +
                               ((((col & 127) >> 4) ^ (tk & 7)) << 4) + (col & 15);
                    if (kStep == 16)
                        *reinterpret_cast<uint4 *>(at) = make_uint4(v[0], v[1], v[kStep / 8], v[kStep / 4 - 1]);
                    else
                        *reinterpret_cast<uint2 *>(at) = make_uint2(v[0], v[1]);
                }
            }
        }
        // values past the sequence's end may be anything (NaN times a weight of
        // 0 would stay): clear them
        const int valid = pc.L - p0;
        if (edge && valid < kTile) {
            char *v = smem_v + (size_t)st * stage_bytes;
            const int at = turns ? part_no * 128 + tk : tid;
            for (int i = valid * (D / 16) + at; i < kTile * (D / 16); i += turns ? 256 : 512)
                reinterpret_cast<uint4 *>(v)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async();
        __syncwarp();
        if (lane < arrivals) mbar_arrive(&sh->p_full[sb]);
    }
    };
    {
        // (it0 and t0 may differ in parity: a pair's tiles are those of its it)
        const int own = pc.t0 + (turns ? (int)((par ^ it0) & 1) : 0);
        const int reach = min(max(ctx >> 7, pc.t0), pc.t1);  // first tile that reaches them
        const int on = reach > own ? (turns ? own + ((reach - own + 1) & ~1) : reach) : own;
        tiles(std::false_type{}, own, reach);
        tiles(std::true_type{}, on, pc.t1);
    }

    // ---- the piece's sums
    it = it0 + (uint32_t)(pc.t1 - pc.t0);
    if (mine > 0 && ok) {
        // the last tile of this warpgroup
        const uint32_t last = turns && ((it - 1) & 1) != (uint32_t)par ? it - 2 : it - 1;
        ok = at_wait(&sh->abort, j.err, &sh->pv_done[last & 1], (last >> 1) & 1);
    }
    const uint32_t r2 = ROUNDS ? sh->far.round[warp] : 0, round = r2 >> 1;
    if (ROUNDS)
        ok = ok && at_wait(&sh->abort, j.err, &sh->far.told[round % kRounds], round / kRounds & 1);
    else
        ok = ok && sh->far.it != it;            // (a piece that needs rounds is given up)
    warp_sum_rows(l, lane);
    if ((lane & 3) == 0) {
#pragma unroll
        for (int i = 0; i < C8; ++i) {
            // which row the halvings left here: bits 4, 3, 2 of the lane
            const int n = ((lane >> 4) & 1) * (R / 2) + ((lane >> 3) & 1) * (R / 4) +
                          ((lane >> 2) & 1) * (R / 8) + i;
            sh->sum[par][quarter][r0 + n] = l[i];
        }
    }
    // (a row that saw nothing here has no maximum: one of 0 would flush the
    // sums that it has elsewhere against scores far below it)
    if (quarter == 0 && lane < R) sh->top[par][r0 + lane] = none ? kNone : mu[lane];
    if (bar_or(5, kSoftWarps * 32, !ok)) return false;
    tc_fence_after();

    // Rounds of a piece after its first add to the sums that these left in the
    // workspace (of a whole unit in the part of the CTA's last unit, which comes
    // after it); a thread reads what it wrote itself.
    const bool first = !ROUNDS || !(r2 & 1), more = ROUNDS && sh->far.more[round % kRounds];
    const bool whole = pc.t0 == 0 && pc.t1 == pc.tiles;
    const bool ends = whole && !more;           // the output follows
    int c0 = 0, c1 = 0, owners = 0;  // the CTAs that share the unit
    bool each = false;
    float *part = nullptr;
    if (!whole) {
        c0 = span_owner(sh->total, ctas, pc.unit0);
        c1 = span_owner(sh->total, ctas, pc.unit0 + (long long)(pc.tiles - 1) * pc.cost);
        // Spans at least a tile long leave no CTA between c0 and c1 without a
        // tile; in shorter ones every tile has a CTA of its own.
        each = pc.cost > div_pos(sh->total, ctas);
        owners = each ? pc.tiles : c1 - c0 + 1;
        // a unit that starts before this CTA's span is its first, else its last
        part = j.part + ((size_t)blockIdx.x * 2 + ((int)blockIdx.x == c0 ? 1 : 0)) * part_floats(D);
    } else if (more || !first) {
        part = j.part + ((size_t)blockIdx.x * 2 + 1) * part_floats(D);
    }
    const int d = tk;  // head element of this lane (D = 64: lanes 64.. hold copies)
    // (a pair that had no tile has no sums)
    const int nt = pc.t1 - pc.t0;
    const bool has0 = !turns || nt > 1 || (it0 & 1) == 0;
    const bool has1 = turns && (nt > 1 || (it0 & 1) == 1);
    // a thread for each row: the factors that its sums of the two pairs get
    if (tid < (turns ? 2 : 4) * R) {
        const int n = tid;
        float m = turns ? fmaxf(sh->top[0][n], sh->top[1][n]) : sh->top[0][n];
        float f0 = 0.f, f1 = 0.f, s = 0.f;
        if (has0) {
            f0 = turns ? ex2f(sh->top[0][n] - m) : 1.f;
            s = f0 * ((sh->sum[0][0][n] + sh->sum[0][1][n]) + (sh->sum[0][2][n] + sh->sum[0][3][n]));
        }
        if (has1) {
            f1 = ex2f(sh->top[1][n] - m);
            s = fmaf(f1, (sh->sum[1][0][n] + sh->sum[1][1][n]) +
                             (sh->sum[1][2][n] + sh->sum[1][3][n]), s);
        }
        float fo = 0.f;
        if (!first && n < pc.rows) {
            const float mo = part[(size_t)kRowsMax * D + n];
            const float so = part[(size_t)kRowsMax * (D + 1) + n];
            const float top = fmaxf(m, mo), fn = ex2f(m - top);
            fo = ex2f(mo - top);
            s = fmaf(so, fo, s * fn);
            f0 *= fn;
            f1 *= fn;
            m = top;
        }
        // (a sum of NaN is no sum of nothing: it goes into the output)
        const float inv = !ends ? 1.f : s == 0.f ? 0.f : 1.f / s;
        sh->out_f[0][n] = f0 * inv;
        sh->out_f[1][n] = f1 * inv;
        if (ROUNDS) sh->far.old_f[n] = fo * inv;
        if (n < pc.rows) {
            if (ends) {
                if (j.lse)
                    j.lse[sh->at[n]] =
                        s == 0.f ? -INFINITY : (m + log2f(s)) * 0.6931471805599453f;
            } else {
                part[(size_t)kRowsMax * D + n] = m;
                part[(size_t)kRowsMax * (D + 1) + n] = s;
            }
        }
    }
    bar_or(5, kSoftWarps * 32, false);
    // rows this warpgroup writes: all of its own, or half of those that it
    // shares with the other pair
    const int w0 = r0 + (turns ? par * (R / 2) : 0), w1 = w0 + (turns ? R / 2 : R);
#pragma unroll 1
    for (int w = w0; w < w1; w += 4) {
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int way = has0 ? 0 : 1; way < (has1 ? 2 : 1); ++way) {
            float v[8];  // hi and lo
            const uint32_t col = lanes + 256 + way * 128 + r0 * 2 + (w - r0);
            tc_ld4(col, v);
            tc_ld4(col + R, v + 4);
            tc_wait_ld(v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = fmaf(sh->out_f[way][w + i], fmaf(v[4 + i], 0.0625f, v[i]), o[i]);
        }
        if (d < D) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (w + i >= pc.rows) break;
                if (!first)
                    o[i] = fmaf(sh->far.old_f[w + i], part[(size_t)(w + i) * D + d], o[i]);
                if (ends)
                    j.out[(int64_t)sh->at[w + i] * D + d] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(o[i]));
                else
                    part[(size_t)(w + i) * D + d] = o[i];
            }
        }
    }
    tc_fence_before();
    if (whole || more) {
        bar_or(5, kSoftWarps * 32, false);  // sum and top are free again
        return true;
    }
    // ---- a shared unit: the last CTA to arrive joins the parts
    __threadfence();
    bar_or(5, kSoftWarps * 32, false);
    if (tid == 0) {
        const unsigned seen = atomicAdd(&j.arrived[c0], 1u);
        sh->last = seen == (unsigned)(owners - 1);
        if (sh->last) j.arrived[c0] = 0;
        __threadfence();
    }
    if (each)
        for (int k = tid; k < owners; k += kSoftWarps * 32)
            sh->owner[k] = (short)span_owner(sh->total, ctas, pc.unit0 + (long long)k * pc.cost);
    bar_or(5, kSoftWarps * 32, false);
    if (!sh->last) return true;
#pragma unroll 1
    for (int i = tid; i < pc.rows * D; i += kSoftWarps * 32) {
        const int n = i / D, e = i - n * D;
        float m = kNone, s = 0.f, o = 0.f;
        for (int k = 0; k < owners; ++k) {
            const int c = each ? sh->owner[k] : c0 + k;
            const float *q = j.part + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * part_floats(D);
            const float mc = __ldcg(q + (size_t)kRowsMax * D + n);
            const float sc = __ldcg(q + (size_t)kRowsMax * (D + 1) + n);
            const float oc = __ldcg(q + (size_t)n * D + e);
            const float top = fmaxf(m, mc), fo = ex2f(m - top), fc = ex2f(mc - top);
            s = s * fo + sc * fc;
            o = o * fo + oc * fc;
            m = top;
        }
        const int64_t at = sh->at[n];
        j.out[at * D + e] = __bfloat16_as_ushort(__float2bfloat16_rn(s == 0.f ? 0.f : o / s));
        if (e == 0 && j.lse)
            j.lse[at] = s == 0.f ? -INFINITY : (m + log2f(s)) * 0.6931471805599453f;
    }
    bar_or(5, kSoftWarps * 32, false);  // the next piece's rows go where these are read from
    return true;
}

// The piece's queries: hi and lo parts to shared memory, rows of D bytes in the
// swizzle of the keys; one row a warp at a time.
template <int D>
__device__ __forceinline__ void load_queries(const AttendJob &j, AttnShared *sh, char *smem_q,
                                             const Piece &pc, int N)
{
    constexpr int E = D / 32;  // elements a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int n0 = warp; n0 < N; n0 += 2 * kSoftWarps) {
        uint16_t raw[2][E];  // two rows in flight
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int n = n0 + k * kSoftWarps, row = pc.row0 + n;
#pragma unroll
            for (int i = 0; i < E; ++i) raw[k][i] = 0;
            if (n < pc.rows) {
                const int tok = pc.first + row / j.G, head = pc.h * j.G + row % j.G;
                if (lane == 0) sh->at[n] = tok * j.Hq + head;
                const uint16_t *q = j.q + (int64_t)tok * j.qts + (int64_t)head * j.qhs + lane * E;
#pragma unroll
                for (int i = 0; i < E; ++i) raw[k][i] = q[i];
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int n = n0 + k * kSoftWarps;
            if (n >= N) break;
            float x[E];
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                x[i] = __uint_as_float((uint32_t)raw[k][i] << 16);
                amax = fmaxf(amax, fabsf(x[i]));
            }
            amax = warp_max(amax);
            // 2^e brings the largest element to [128, 256)
            const int e = amax > 0.f ? min(134 - (int)(__float_as_uint(amax) >> 23), 126) : 0;
            const float up = __int_as_float((127 + e) << 23);
            // (an infinity would saturate as if it were a number)
            if (lane == 0)
                sh->c[n] = n >= pc.rows      ? 0.f
                           : amax < INFINITY ? j.softmax_scale * 1.4426950408889634f / up
                                             : __int_as_float(0x7FC00000);
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                uint16_t h8, l8;
                const float a = x[i] * up, b = x[i + 1] * up;
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h8) : "f"(b), "f"(a));
                uint32_t h16;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h16) : "h"(h8));
                const float2 h = __half22float2(*reinterpret_cast<__half2 *>(&h16));
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                    : "=h"(l8)
                    : "f"(b - h.y), "f"(a - h.x));
                hi |= (uint32_t)h8 << (8 * i);
                lo |= (uint32_t)l8 << (8 * i);
            }
            const int byte = lane * E;
            const int sw = D == 128 ? n & 7 : (n >> 1) & 3;
            char *at = smem_q + n * D + (((byte >> 4) ^ sw) << 4) + (byte & 15);
            if (E == 4) {
                *reinterpret_cast<uint32_t *>(at) = hi;
                *reinterpret_cast<uint32_t *>(at + N * D) = lo;
            } else {
                *reinterpret_cast<uint16_t *>(at) = (uint16_t)hi;
                *reinterpret_cast<uint16_t *>(at + N * D) = (uint16_t)lo;
            }
        }
    }
}

// The roles' loops over the pieces of a span: without rounds (up to a piece that
// needs them) or with them (from that piece on).
template <int D, bool ROUNDS>
__device__ __forceinline__ void attend_roles(const AttendJob &j, const CUtensorMap &map_k,
                                             const CUtensorMap &map_v, AttnShared *sh, char *base,
                                             int first, long long x, long long from, long long to,
                                             uint32_t pieces)
{
    constexpr int kSide = kTile * D;            // bytes of a tile's keys (or values)
    constexpr uint32_t kSwz = D == 128 ? 2 : 4;
    char *s_k = base, *s_v = base + kSide, *s_q = base + 2 * kAtStages * kSide;
    char *s_p = s_q + 2 * kRowsMax * D;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = gridDim.x;
    PieceWalk walk;
    Piece pc;
    uint32_t it = ROUNDS ? sh->far.it : 0, round = 0;
    walk.start(j, first, x, from, to);
    if (warp < kSoftWarps) {
        if (!ROUNDS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        bool ok = true;
        if (ROUNDS)
            sh->far.round[warp] = 0;
        else
            sh->looks[warp] = 0;
        bool more = false;  // the piece has another round
        while (ok) {
            if (ROUNDS && more) {
                pc = sh->far.piece;
            } else {
                if (!walk.next(j, pc)) break;
                if (tid == 0) ++sh->far.pieces;
                if (ROUNDS && tid == 0) sh->far.piece = pc;
                load_queries<D>(j, sh, s_q, pc, round_rows(pc.rows));
                fence_async();
                bar_or(5, kSoftWarps * 32, false);  // the rows' factors are there
                if (lane == 0) mbar_arrive(&sh->q_full);
            }
            const int N = round_rows(pc.rows);
            const bool turns = N <= 64;
#define SV_SOFT(C)                                                                              \
    case C:                                                                                     \
        ok = soft_piece<D, C, ROUNDS>(j, sh, s_v, s_p, pc, it, 2 * kSide, ctas, turns, ok);      \
        break;
            switch (N / (turns ? 16 : 32)) {
                SV_SOFT(1) SV_SOFT(2) SV_SOFT(3) SV_SOFT(4)
            }
#undef SV_SOFT
            if (ROUNDS) {
                const uint32_t r = sh->far.round[warp] >> 1;
                more = sh->far.more[r % kRounds] != 0;
                __syncwarp();
                sh->far.round[warp] = (r + 1) * 2 + more;
                __syncwarp();
            }
        }
        // (the issuers are waiting for the next piece)
        if (!ROUNDS && !ok && tid == 0 && sh->abort == 0) *(volatile int *)&sh->abort = kGaveUp;
    } else if (warp >= kSoftWarps) {
        if (!ROUNDS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSideRegs));
    }
    if (warp == kSoftWarps) {
        // ---- producer: the pages of each tile, looked up 32 at a time
        const int shift = 31 - __clz(j.block), per_tile = kTile >> shift;
        const int inner = lane & (per_tile - 1);
        bool ok = true, more = false;
        while (ok && walk.next(j, pc)) {
            const int last = (int)((pc.L + (long long)j.block - 1) >> shift);  // pages of the sequence
            const int32_t *tab = j.table + (int64_t)pc.b * j.cols;
            auto window = [&](int w0, int &page, float &ks, float &vs) {
                page = w0 + lane < last ? tab[w0 + lane] : -1;
                if (w0 + lane < last && (page < 0 || page >= j.pages)) {
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
            const int first_p = pc.t0 * per_tile, end_p = min(pc.t1 * per_tile, last);
            auto exponent = [](float vs) { return (int)(__float_as_uint(vs) >> 23) - 64; };
            if (ROUNDS && lane < 4) sh->far.classes[lane] = 0;
            // without rounds: the lane's extreme exponents; with them: those of the
            // round's class, and the last of the first round's
            int top = 0, bottom = 127, top0 = 0;
            auto own = [&](int w0) { return w0 + lane >= first_p && w0 + lane < end_p; };
            auto note = [&](int w0, float vs) {
                top = max(top, own(w0) ? exponent(vs) : 0);
                bottom = min(bottom, own(w0) ? exponent(vs) : 127);
            };
            more = false;
            do {
                int w0 = first_p & ~31, page, npage;
                float ks, vs, nks, nvs;
                window(w0, page, ks, vs);
                window(w0 + 32, npage, nks, nvs);
                bool fresh = true;  // the window's value scales have not been looked at
                if (more) {
                    const uint32_t w = sh->far.classes[lane & 3];
                    top = __reduce_max_sync(0xFFFFFFFFu, w ? (lane & 3) * 32 + 31 - __clz(w) : 0);
                    bottom = top > top0 ? max(top - kClass, top0) + 1 : top - kClass + 1;
                }
                for (int t = pc.t0; t < pc.t1; ++t, ++it) {
                    const int st = it % kAtStages;
                    const uint32_t ph = ((it / kAtStages) & 1) ^ 1;
                    const int p0 = t * per_tile;
                    if (p0 >= w0 + 32) {
                        if (!ROUNDS) note(w0, vs);
                        w0 += 32;
                        page = npage;
                        ks = nks;
                        vs = nvs;
                        window(w0 + 32, npage, nks, nvs);
                        fresh = true;
                    }
                    const bool mine = lane - (p0 - w0) >= 0 && lane - (p0 - w0) < per_tile;
                    const bool copy = mine && page >= 0;
                    const uint32_t bytes =
                        (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, copy)) * j.block * D;
                    ok = at_wait(&sh->abort, j.err, &sh->empty_k[st], ph);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_tx(&sh->full_k[st], bytes);
                    __syncwarp();
                    const int64_t row = (int64_t)page * j.H + pc.h;
                    auto fetch = [&](const CUtensorMap *map, char *dst, uint64_t *bar) {
                        asm volatile(
                            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::"
                            "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
                            "l"(map), "r"(0), "r"(0), "r"((int)row), "r"(smem_u32(bar))
                            : "memory");
                    };
                    if (copy)
                        fetch(&map_k, s_k + (size_t)st * 2 * kSide + inner * j.block * D,
                              &sh->full_k[st]);
                    if (ROUNDS && fresh) {
                        fresh = false;
                        const int e = exponent(vs);
                        if (!more && t == pc.t0) {
                            // the first class ends at the largest scale of the pages looked
                            // up, or one above it where there are more
                            const int f = w0 + 32 + lane < end_p ? exponent(nvs) : 0;
                            top = top0 = __reduce_max_sync(0xFFFFFFFFu, max(own(w0) ? e : 0, f)) +
                                         (w0 + 64 < end_p ? 1 : 0);
                            bottom = top - kClass + 1;
                        }
                        if (!more && own(w0)) atomicOr(&sh->far.classes[e >> 5], 1u << (e & 31));
                        if (e < bottom || e > top) vs = 0.f;
                    }
                    ok = at_wait(&sh->abort, j.err, &sh->empty_v[st], ph);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (!ROUNDS && t == pc.t1 - 1) {
                        // (told before the last tile's values)
                        note(w0, vs);
                        more = __reduce_max_sync(0xFFFFFFFFu, top) -
                                   __reduce_min_sync(0xFFFFFFFFu, bottom) >= kClass;
                        if (more && lane == 0) {
                            const SeqWork &s = walk.s;
                            const long long unit = (long long)pc.h * s.blocks + pc.row0 / s.rows;
                            sh->far.b = pc.b;
                            sh->far.x = (unit * s.tiles + pc.t0) * s.cost;
                            sh->far.pos = pc.unit0 + (long long)pc.t0 * pc.cost;
                            sh->far.it = it + 1;
                        }
                    }
                    if (mine) {
                        sh->ks[st][inner] = ks;
                        sh->vs[st][inner] = vs;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_tx(&sh->full_v[st], bytes);
                    __syncwarp();
                    if (copy)
                        fetch(&map_v, s_v + (size_t)st * 2 * kSide + inner * j.block * D,
                              &sh->full_v[st]);
                }
                if (ROUNDS) {
                    // what the round leaves
                    __syncwarp();
                    const int base = (lane & 3) * 32;
                    const int lo = max(bottom - base, 0), hi = min(top - base, 31);
                    uint32_t w = sh->far.classes[lane & 3];
                    if (lo <= hi) w &= ~((~0u << lo) & (~0u >> (31 - hi)));
                    __syncwarp();
                    if (lane < 4) sh->far.classes[lane] = w;
                    more = __any_sync(0xFFFFFFFFu, w != 0);
                    if (lane == 0) {
                        sh->far.more[round % kRounds] = more;
                        mbar_arrive(&sh->far.told[round % kRounds]);
                    }
                    ++round;
                    __syncwarp();
                }
            } while (ROUNDS && ok && more);
            if (!ROUNDS && more) break;
        }
        // after a wait that ran out: copies still in flight land before the exit
        if (!ok)
            for (int i = 0; i < kAtStages; ++i) {
                mbar_wait_n(&sh->full_k[i], (it / kAtStages) & 1, 1u << 12);
                mbar_wait_n(&sh->full_v[i], (it / kAtStages) & 1, 1u << 12);
            }
    } else if (warp == kSoftWarps + 1) {
        // ---- issuer of the scores.  (One thread for both products would wait
        // with each for the other's inputs; issuing a product takes it some
        // seventy cycles, a commit almost as many.)
        constexpr uint32_t kKinds = (1u << 4) | ((uint32_t)(kTile >> 4) << 24);  // fp32 sums, M = 128
        const uint32_t tmem = sh->tmem;
        const uint64_t dk0 = tc_desc(smem_u32(s_k), 16, 8 * D, kSwz);
        const uint64_t dq = tc_desc(smem_u32(s_q), 16, 8 * D, kSwz);
        bool ok = true;
        bool more = false;  // the piece has another round
        while (ok && ((ROUNDS && more) || walk.next(j, pc))) {
            const int N = round_rows(pc.rows);
            const bool one = stacked(N);
            const uint32_t id_s = kKinds | ((uint32_t)((one ? 2 * N : N) >> 3) << 17);
            const uint64_t dlo = dq + (uint32_t)(N * D >> 4);
            if (!ROUNDS || !more) {
                ok = at_wait(&sh->abort, j.err, &sh->q_full, pieces & 1);
                ++pieces;
            }
            const int ctx = pc.L - pc.n;
            const int reach = min(max(ctx >> 7, pc.t0), pc.t1);  // first tile of new tokens
            auto tiles = [&](auto is_one, int from, int to) {
#pragma unroll 1
                for (int t = from; t < to; ++t, ++it) {
                    const uint32_t st = it % kAtStages, sb = it & 1;
                    ok = ok && at_wait(&sh->abort, j.err, &sh->full_k[st], (it / kAtStages) & 1);
                    ok = ok && at_wait(&sh->abort, j.err, &sh->s_empty[sb], ((it >> 1) & 1) ^ 1);
                    if (__builtin_expect(!ok, 0)) break;
                    tc_fence_after();
                    const uint64_t dk = dk0 + st * (2 * kSide >> 4);
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        tc_mma(tmem + sb * 128, dk + 2 * k, dq + 2 * k, id_s, k);
                    if (!decltype(is_one)::value)
#pragma unroll
                        for (int k = 0; k < D / 32; ++k)
                            tc_mma(tmem + sb * 128, dk + 2 * k, dlo + 2 * k, id_s, 1);
                    tc_commit(&sh->s_full[sb]);
                    tc_commit(&sh->empty_k[st]);
                }
            };
            // (up to the new tokens without a stop; then a tile at a time)
#pragma unroll 1
            for (int t = pc.t0; t < pc.t1;) {
                const int to = t < reach ? reach : t + 1;
                if (lane == 0) {
                    if (one)
                        tiles(std::true_type{}, t, to);
                    else
                        tiles(std::false_type{}, t, to);
                }
                const bool look = t >= reach;
                t = to;
                it = __shfl_sync(0xFFFFFFFFu, it, 0);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (!look) continue;
                // A new token's value may hold NaN, which a row that does not see it
                // would get all the same (NaN times 0): the warp looks them over, 512
                // bytes at a time, and clears such tokens' values.
                const uint32_t st = (it - 1) % kAtStages, sb = (it - 1) & 1;
                ok = at_wait(&sh->abort, j.err, &sh->full_v[st], ((it - 1) / kAtStages) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                constexpr int kParts = D / 16, kRows = 32 / kParts;
                const int p0 = (t - 1) * kTile, end = min(pc.L - p0, kTile);
                if (lane < 4) sh->lost[sb][lane] = 0;
                __syncwarp();
#pragma unroll 1
                for (int r0 = max(ctx - p0, 0); r0 < end; r0 += kRows) {
                    const int r = r0 + lane / kParts;
                    uint4 *at = reinterpret_cast<uint4 *>(s_v + (size_t)st * 2 * kSide + r0 * D) +
                                lane;
                    bool nan = false;
                    if (r < end) {
                        const uint4 x = *at;
                        nan = has_nan(x.x) | has_nan(x.y) | has_nan(x.z) | has_nan(x.w);
                    }
                    const uint32_t m = __ballot_sync(0xFFFFFFFFu, nan);
                    if ((m >> (lane & ~(kParts - 1))) & ((1u << kParts) - 1)) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                        if (lane % kParts == 0) atomicOr(&sh->lost[sb][r >> 5], 1u << (r & 31));
                    }
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->clean[N <= 64 ? sb : 2 + sb]);
            }
            if (ROUNDS) {
                ok = ok && at_wait(&sh->abort, j.err, &sh->far.told[round % kRounds], round / kRounds & 1);
                more = sh->far.more[round++ % kRounds] != 0;
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        // after a wait that ran out: products still in flight end before the exit
        if (!ok && lane == 0) {
            tc_commit(&sh->drained[0]);
            mbar_wait_n(&sh->drained[0], 0, 1u << 12);
        }
    } else if (warp == kSoftWarps + 2 && lane == 0) {
        // ---- issuer of the outputs
        constexpr uint32_t kKinds = (1u << 4) | ((uint32_t)(kTile >> 4) << 24) | (3u << 15);
        const uint32_t tmem = sh->tmem;
        // D = 64: the second 64 rows read the same values again
        const uint64_t dv0 = tc_desc(smem_u32(s_v), 0, 8 * D, kSwz);
        const uint64_t dp0 = tc_desc(smem_u32(s_p), kTile * 128, 1024, 2);
        bool ok = true, more = false;  // the piece has another round
        while (ok && ((ROUNDS && more) || walk.next(j, pc))) {
            const int N = round_rows(pc.rows);
            const bool turns = N <= 64;
            const uint32_t id_o = kKinds | ((uint32_t)(2 * N >> 3) << 17);
            uint32_t done = 0;
#pragma unroll 1
            for (int t = pc.t0; t < pc.t1; ++t, ++it, ++done) {
                const uint32_t st = it % kAtStages, sb = it & 1;
                ok = ok && at_wait(&sh->abort, j.err, &sh->full_v[st], (it / kAtStages) & 1);
                ok = ok && at_wait(&sh->abort, j.err, &sh->p_full[sb], (it >> 1) & 1);
                if (__builtin_expect(!ok, 0)) break;
                tc_fence_after();
                const uint64_t dv = dv0 + st * (2 * kSide >> 4);
                const uint64_t dp = dp0 + (turns ? sb * (kTile * 128 >> 4) : 0u);
                const uint32_t o = tmem + 256 + (turns ? sb * 128 : 0);
                const bool sum = done > (turns ? 1u : 0u);
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k)
                    tc_mma(o, dv + 2 * D * k, dp + 256 * k, id_o, sum || k);
                tc_commit(&sh->pv_done[sb]);
                tc_commit(&sh->empty_v[st]);
            }
            if (ROUNDS) {
                ok = ok && at_wait(&sh->abort, j.err, &sh->far.told[round % kRounds], round / kRounds & 1);
                more = sh->far.more[round++ % kRounds] != 0;
            }
        }
        if (!ok) {
            tc_commit(&sh->drained[1]);
            mbar_wait_n(&sh->drained[1], 0, 1u << 12);
        }
    }
}

// With rounds.  (A call, which has its own registers.)
template <int D>
__device__ __noinline__ void attend_rounds(const AttendJob *j, const CUtensorMap *map_k,
                                           const CUtensorMap *map_v, AttnShared *sh, char *base,
                                           long long to, uint32_t pieces)
{
    attend_roles<D, true>(*j, *map_k, *map_v, sh, base, sh->far.b, sh->far.x, sh->far.pos, to, pieces);
}

template <int D>
__global__ void __launch_bounds__(kAtThreads, 1)
attend_kernel(const __grid_constant__ AttendJob j, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v)
{
    extern __shared__ char attn_raw[];
    __shared__ AttnShared shared;
    AttnShared *sh = &shared;
    char *base = attn_raw + ((1024 - (smem_u32(attn_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < kAtStages; ++i) {
            mbar_init(&sh->full_k[i], 1);
            mbar_init(&sh->full_v[i], 1);
            mbar_init(&sh->empty_k[i], 1);
            mbar_init(&sh->empty_v[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->s_full[i], 1);
            // (a warp arrives twice where two warpgroups have a tile)
            mbar_init(&sh->s_empty[i], kSoftWarps);
            mbar_init(&sh->p_full[i], kSoftWarps);
            mbar_init(&sh->pv_done[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&sh->clean[i], 1);
        for (int i = 0; i < kRounds; ++i) mbar_init(&sh->far.told[i], 1);
        mbar_init(&sh->q_full, kSoftWarps);
        mbar_init(&sh->drained[0], 1);
        mbar_init(&sh->drained[1], 1);
        mbar_fence_init();
        sh->abort = 0;
        sh->far.it = sh->far.pieces = 0;
        sh->first_b = 0;
        sh->first_x = 0;
    }
    if (warp == kSoftWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&sh->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's span: each thread sums a run of sequences
    const int per = (j.B + kAtThreads - 1) / kAtThreads;
    const int b0 = min(tid * per, j.B), b1 = min(b0 + per, j.B);
    long long own = 0;
    for (int b = b0; b < b1; ++b) {
        const SeqWork s = seq_work(j, b);
        own += s.work;
        if (s.bad && blockIdx.x == 0) latch(j.err, SV_ERR_DEVICE_BOUNDS);
    }
    long long run = own;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const long long a = __shfl_up_sync(0xFFFFFFFFu, run, k);
        if (lane >= k) run += a;
    }
    if (lane == 31) sh->scan[warp] = run;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kAtThreads / 32; ++w) {
        if (w < warp) run += sh->scan[w];
        total += sh->scan[w];
    }
    const int ctas = gridDim.x;
    const int me = blockIdx.x;
    const long long from = span_at(total, ctas, me), to = span_at(total, ctas, me + 1);
    if (from < to && run > from && run - own <= from) {
        long long x = from - (run - own);
        int b = b0;
        for (;; ++b) {
            const long long w = seq_work(j, b).work;
            if (x < w) break;
            x -= w;
        }
        sh->first_b = b;
        sh->first_x = x;
    }
    if (tid == 0) sh->total = total;
    __syncthreads();

    attend_roles<D, false>(j, map_k, map_v, sh, base, sh->first_b, sh->first_x, from, to, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (__builtin_expect(sh->abort == kGaveUp, 0)) {
        const uint32_t pieces = sh->far.pieces;
        __syncthreads();
        if (tid == 0) sh->abort = 0;
        __syncthreads();
        if (warp < kSoftWarps)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtRegs));
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtRegs));
        attend_rounds<D>(&j, &map_k, &map_v, sh, base, to, pieces);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh->tmem));
    }
}

constexpr size_t attend_smem(int D)
{
    return 1024 + (size_t)2 * kAtStages * kTile * D + 2 * kRowsMax * D + 2 * kTile * 128;
}

size_t attend_ws_bytes(int sms) { return (size_t)sms * 2 * part_floats(128) * sizeof(float); }
size_t attend_counter_bytes(int sms) { return ((size_t)sms * sizeof(unsigned) + 255) & ~(size_t)255; }

cudaError_t attend_setup()
{
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<64>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)attend_smem(128));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attend_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)attend_smem(128));
    return e;
}

bool cache_map(CUtensorMap *m, const uint8_t *cache, int D, int block, int rows, int pages,
               int H)
{
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                               const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                               const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &r) != cudaSuccess)
            f = nullptr;
        return (Encode)f;
    }();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)block, (cuuint64_t)pages * H};
    const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * block};
    const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)rows, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, (void *)cache, dims, strides, box,
                  step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t attend_launch(const AttendJob &j, int sms, cudaStream_t s)
{
    sms = sms < 256 ? sms : 256;  // (AttnShared::owner)
    CUtensorMap mk, mv;
    if (!cache_map(&mk, j.cache[0], j.D, j.block, j.block, j.pages, j.H) ||
        !cache_map(&mv, j.cache[1], j.D, j.block, j.block, j.pages, j.H))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    // (one CTA an SM, also where the shared memory of D = 64 would allow two:
    // each holds all of the SM's tensor memory)
    pdl_config(cfg, at, dim3(sms), dim3(kAtThreads), attend_smem(128), s);
    return j.D == 64 ? cudaLaunchKernelEx(&cfg, attend_kernel<64>, j, mk, mv)
                     : cudaLaunchKernelEx(&cfg, attend_kernel<128>, j, mk, mv);
}

}  // namespace sv
