// sv_rows.cuh -- job of the filtered draw from logit rows.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace sv {

constexpr int kRowsMaxV = 1 << 20;  // ids of a row (1,024 blocks of 1,024 in shared memory)

struct RowsJob {
    const char *x;             // logits, rs bytes from row to row
    int64_t rs;
    int dtype, R, V;
    const float *u;            // [R]
    const float *temp;         // [R] or null (1)
    const int32_t *top_k;      // [R] or null (off)
    const float *top_p, *min_p;  // [R] or null (off)
    int32_t *token, *kept;     // [R]
    float *prob;               // [R]
    int *err;
};
cudaError_t rows_setup();
cudaError_t rows_launch(const RowsJob &j, int sms, cudaStream_t s);

}  // namespace sv
