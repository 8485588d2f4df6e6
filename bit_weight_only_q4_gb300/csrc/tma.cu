// Tensor maps (see tma.h).
#include "tma.h"

#include <mutex>

namespace q4 {

EncodeTiledFn tma_encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

static q4_status encode(CUtensorMap &map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                        const cuuint32_t *box)
{
    const EncodeTiledFn enc = tma_encode_fn();
    if (!enc)
        return fail(Q4_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = enc(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims, strides,
                           box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? Q4_OK : fail(Q4_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

q4_status tma_heads(CUtensorMap &map, const void *base, int D, int heads, uint64_t tokens, int64_t token_stride,
                    int box_heads, int box_tokens)
{
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)token_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    return encode(map, base, 3, dims, strides, box);
}

q4_status tma_rows(CUtensorMap &map, const void *base, uint64_t columns, uint64_t rows, int64_t stride, int box_rows)
{
    const cuuint64_t dims[2] = {columns, rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    return encode(map, base, 2, dims, strides, box);
}

}  // namespace q4
