// Tensor maps of the dense products' row-major bf16 matrices.  A box's rows are 128 bytes
// (operands) or 64 bytes (results, residuals) and swizzled over as many.
#pragma once

#include <cuda.h>

#include <cstdint>
#include <string>

#include "band_common.cuh"
#include "internal.h"

namespace dfs {

inline int encode_bf16_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
                           const cuuint64_t* strides, const cuuint32_t* box) {
    auto fn = band::tensor_map_encoder();
    if (!fn) return fail(DIFFUSER_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    const cuuint32_t es[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          box[0] * 2 == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(DIFFUSER_ERR_CUDA, "cuTensorMapEncodeTiled failed: " + std::to_string((int)r));
    return DIFFUSER_OK;
}

// [rows][width], boxes of box_rows x box_width (64 or 32)
inline int map_matrix(CUtensorMap* m, const void* base, int64_t width, int64_t rows, int box_width, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)width * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_width, (cuuint32_t)box_rows};
    return encode_bf16_map(m, base, 2, dims, strides, box);
}

// [2][rows][width] (the gate's rows, then the up rows), boxes of box_halves x box_rows x
// box_width: a box that passes the end of one half reads zeros, not the other half
inline int map_halves(CUtensorMap* m, const void* base, int64_t width, int64_t rows, int box_width, int box_rows,
                      int box_halves) {
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, 2};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)width * 2 * (cuuint64_t)rows};
    const cuuint32_t box[3] = {(cuuint32_t)box_width, (cuuint32_t)box_rows, (cuuint32_t)box_halves};
    return encode_bf16_map(m, base, 3, dims, strides, box);
}

// [rows][2][width] (a row's gate columns, then its up columns), boxes of box_rows x 1 x
// box_width: a box that passes the end of the gate's columns is cut there
inline int map_column_halves(CUtensorMap* m, const void* base, int64_t width, int64_t rows, int box_width, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)width, 2, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)width * 4};
    const cuuint32_t box[3] = {(cuuint32_t)box_width, 1, (cuuint32_t)box_rows};
    return encode_bf16_map(m, base, 3, dims, strides, box);
}

}  // namespace dfs
