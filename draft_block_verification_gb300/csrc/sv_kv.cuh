// sv_kv.cuh -- jobs of the paged 8-bit key/value cache: the plan that gives
// new tokens their places, the append that writes them, the attention that
// reads the cache, alone or for a batch that shares a prefix, and reading it
// back; and of the norms and rotation of queries and keys before them.
//
// The cache.  Keys and values are held apart, each as [pages, Hkv, block, D]
// bytes (e4m3) with one fp32 scale for each page and head, [pages, Hkv]: the
// value of a byte is its e4m3 value times the scale.  A sequence's token at
// position p lives in page table[b, p / block], row p % block.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace sv {

constexpr int kPlanMaxB = 16384;  // sequences of one plan (three shared words each)

struct PlanJob {
    int B, block, cols, ring, cap;
    const int32_t *cached, *fresh, *held;
    const int64_t *free_pos;   // [2] head, tail of the queue of free pages
    int32_t *free_ids;         // [ring]
    int32_t *table;            // [B, cols]
    int32_t *kv_len, *cu, *held_out;
    int64_t *free_out;
    int32_t *slot, *pos;       // [cap]
    int *err;
};
cudaError_t plan_setup();
cudaError_t plan_launch(const PlanJob &j, int sms, cudaStream_t s);

struct AppendJob {
    const char *src[2];        // keys, values: [T, H, D]
    int64_t ts[2], hs[2];      // token and head strides, bytes
    int dtype, T, H, D, block, pages;
    const int32_t *slot;
    uint8_t *cache[2];
    float *scale[2];
    int *err;
};
cudaError_t append_launch(const AppendJob &j, int sms, cudaStream_t s);

struct AttendJob {
    const uint16_t *q;         // [T, Hq, D] bf16
    int64_t qts, qhs;          // strides, elements
    const uint8_t *cache[2];
    const float *scale[2];
    const int32_t *table, *kv_len, *cu;
    const uint32_t *mask;      // [T, words] or null
    int B, T, Hq, H, G, D, block, pages, cols, words;
    float softmax_scale;
    uint16_t *out;             // [T, Hq, D]
    float *lse;                // [T, Hq] or null
    float *part;               // partial sums of shared units (workspace)
    unsigned *arrived;         // a counter a CTA, zero between calls
    int *err;
};
size_t attend_ws_bytes(int sms);       // partial sums
size_t attend_counter_bytes(int sms);  // counters, before them
cudaError_t attend_setup();
cudaError_t attend_launch(const AttendJob &j, int sms, cudaStream_t s);

// Attention over a shared prefix: prep finds what is shared and cuts the work, the
// prefix kernel reads the shared pages, the tail kernel the rest, and joins.
// A span: pages that query rows read, a group's shared ones or a sequence's own.
// First the groups', then the sequences', then an entry with the totals (rows: the
// shares that the units are cut into).
struct PrefixSpan {
    int first, rows;           // first row of q, query rows a cache head (0: no work)
    int lead, page0;           // the table row, and its first page
    int end, ctx;              // tokens from there on, and those that every row sees
    long long start;           // where its work starts, if its units are cut
    int unit0, block;          // its first unit, rows of a unit
    int loose0, unused;        // units before it that are not cut
};
struct PrefixJob {
    const uint16_t *q;         // [T, Hq, D] bf16
    int64_t qts, qhs;          // strides, elements
    const uint8_t *cache[2];
    const float *scale[2];
    const int32_t *table, *kv_len, *cu;
    const int32_t *prefix_len; // [groups] or null
    const int32_t *cu_group;   // [groups + 1], or null: one group
    const uint32_t *mask;      // [T, words] or null
    int B, T, Hq, H, G, D, block, pages, cols, groups, words;
    float softmax_scale;
    uint16_t *out;             // [T, Hq, D]
    float *lse;                // [T, Hq] or null
    // from prep
    int32_t *skip, *seq_group; // [B] shared pages, and of which group
    int32_t *unit0;            // [B + 1] the tail's tasks of the sequences before
    int32_t *part0;            // [B] its parts
    int32_t *tail_stages;      // of a task, at most
    int32_t *next;             // of the units that are not cut
    PrefixSpan *span;          // [groups + B + 1]
    unsigned *tail_arrived;    // a counter a part
    // from the prefix kernel
    int prefix_ctas;
    int2 *unit_ctas;           // the first and the last CTA with a piece of a unit
    int32_t *part_unit;        // [2 CTAs] the unit of a part
    float *part;               // pieces' sums
    float *tail_part;          // sums of ranges
    int *err;
};
// Whether a unit's entry tells CTAs.  A CTA of the prefix kernel whose wait ran out leaves
// no entry of the units it did not get to: there stands what was in the workspace.
inline __host__ __device__ bool unit_known(int first, int last, int ctas)
{
    return first >= 0 && first <= last && last < ctas;
}
constexpr int kPrefixRows = 256;                             // query rows of a unit
constexpr int64_t kPrefixMaxUnits = 1 << 24;
size_t prefix_part_bytes(int sms, int64_t units, int D);
cudaError_t prefix_setup();
cudaError_t prefix_prep_launch(const PrefixJob &j, int sms, cudaStream_t s);
cudaError_t prefix_launch(const PrefixJob &j, int sms, cudaStream_t s);
// Rows a cache head that the tail reads for, at most.  (64 draft blocks of 36 to 68 rows /
// three long documents of 21 to 35, us: 32 239 / 409, 64 281 / 452.)
constexpr int kTailMax = 32;
constexpr int kTailTiles = 2;                                // eights of rows of a task
constexpr int kTailTile = 32;                                // tokens of a stage
constexpr int kTailParts = 2;                                // ranges that join, a warp
inline __host__ __device__ int tail_warps(int sms) { return 12 * sms; }
// A sequence's rows of a cache head, cut evenly into blocks of eights.
struct TailBlocks {
    int blocks, rows;
    __host__ __device__ explicit TailBlocks(int all)
    {
        const int eights = (all + 7) / 8;
        blocks = (eights + kTailTiles - 1) / kTailTiles;
        rows = blocks ? (eights + blocks - 1) / blocks * 8 : 0;
        blocks = rows ? (all + rows - 1) / rows : 0;
    }
};
size_t tail_part_bytes(int sms, int D);
cudaError_t tail_setup();
cudaError_t tail_launch(const PrefixJob &j, int sms, cudaStream_t s);

struct RopeJob {
    const char *src[2];        // queries [T, Hq, D], keys [T, H, D]
    char *dst[2];
    int64_t ts[2], hs[2], ots[2], ohs[2];  // token and head strides, bytes
    int dtype, odtype, T, Hq, H, D, rot, inter;
    const float *weight[2];    // [D] or null
    const float *inv_freq;     // [rot / 2]
    float eps, share;          // share: 1 / D
    const int32_t *pos;        // [T], negative: skipped
};
constexpr int kRopeMaxD = 512;
cudaError_t rope_launch(const RopeJob &j, int sms, cudaStream_t s);

struct ReadJob {
    const uint8_t *cache[2];
    const float *scale[2];
    const int32_t *table, *first, *cu;  // first: null for 0
    int B, T, H, D, block, pages, cols, dtype;
    char *dst[2];              // [T, H, D]
    int64_t ts[2], hs[2];      // strides, bytes
    int *err;
};
cudaError_t read_launch(const ReadJob &j, int sms, cudaStream_t s);

}  // namespace sv
