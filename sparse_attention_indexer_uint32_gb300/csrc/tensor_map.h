// tensor_map.h -- host side of tiled copies: tensor maps of two-byte tensors
// with tiles of 64 values (128 bytes, 128-byte swizzle) by some rows.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace topkidx {

// dims / strides: values and bytes, innermost first (strides of dims 1..);
// box_rows: rows of dimension `row_dim` per copy, one of the others.  An
// extent of 0 becomes 1 with nothing read of it (the caller copies no tile).
inline CUresult encode_map(CUtensorMap* map, bool bf16, const void* base, int rank, const int64_t* dims,
                           const int64_t* strides, int row_dim, int box_rows) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    if (!encode) return CUDA_ERROR_NOT_FOUND;
    cuuint64_t size[4], step[3];
    cuuint32_t box[4], unit[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        size[i] = static_cast<cuuint64_t>(dims[i] > 0 ? dims[i] : 1);
        box[i] = i == 0 ? 64 : i == row_dim ? static_cast<cuuint32_t>(box_rows) : 1;
    }
    for (int i = 0; i + 1 < rank; ++i) step[i] = static_cast<cuuint64_t>(strides[i]);
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  static_cast<cuuint32_t>(rank), const_cast<void*>(base), size, step, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace topkidx
