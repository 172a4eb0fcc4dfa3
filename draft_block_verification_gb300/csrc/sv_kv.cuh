// sv_kv.cuh -- jobs of the paged 8-bit key/value cache: the plan that gives
// new tokens their places, the append that writes them, and the attention
// that reads the cache.
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

}  // namespace sv
