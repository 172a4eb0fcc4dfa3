// sv_kvattn.cu -- attention over the paged 8-bit cache, for whole sequences.
#include "sv_attend.cuh"

namespace sv {

size_t attend_ws_bytes(int sms) { return (size_t)sms * 2 * part_floats(128) * sizeof(float); }
size_t attend_counter_bytes(int sms) { return ((size_t)sms * sizeof(unsigned) + 255) & ~(size_t)255; }


cudaError_t attend_setup() { return attend_attributes<false>(); }
cudaError_t attend_launch(const AttendJob &j, int sms, cudaStream_t s)
{
    return attend_start<false>(j, sms, s);
}

bool cache_map(CUtensorMap *m, const uint8_t *cache, int D, int block, int pages, int H)
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
    const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)block, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, (void *)cache, dims, strides, box,
                  step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sv
