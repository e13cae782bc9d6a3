// Host helper: tensor maps for TMA tiled loads of the attention operators.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

using TmapEncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline TmapEncodeFn tmap_encode_fn() {
    static TmapEncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<TmapEncodeFn>(p) : nullptr;
    }();
    return fn;
}

// Rows of `width` bytes (a multiple of block_bytes), row_bytes apart, as a
// 3-D view (byte within a block, row, block): a box is box_rows rows of
// box_blocks blocks, each block swizzled over its block_bytes (64 or 128).
// Rows outside the tensor load as zeros.
inline bool make_row_blocks_map(CUtensorMap* m, const void* base, int64_t rows, int64_t row_bytes, int64_t width,
                                int block_bytes, int box_rows, int box_blocks) {
    TmapEncodeFn enc = tmap_encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)block_bytes, (cuuint64_t)rows, (cuuint64_t)(width / block_bytes)};
    const cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)block_bytes};
    const cuuint32_t box[3] = {(cuuint32_t)block_bytes, (cuuint32_t)box_rows, (cuuint32_t)box_blocks};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               block_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
