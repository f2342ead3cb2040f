// Argument checks shared by the entry points of the grouped products and the
// adapters.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "tiled_gemm.h"

namespace tmmo {

inline bool valid_size(int64_t n) { return n >= 0 && n <= GEMM_MAX_DIM; }
inline bool valid_dtype(int t) { return t == GEMM_F32 || t == GEMM_F16 || t == GEMM_BF16; }

// Whether `count` matrices of rows x cols (pitch ld >= cols), `stride` elements after
// each other, do not overlap: one behind the other, or interleaved row by row.
inline bool apart(int64_t count, int64_t stride, int64_t rows, int64_t ld, int64_t cols)
{
    const __int128 step = stride;
    return count <= 1 || step >= static_cast<__int128>(rows - 1) * ld + cols ||
           (step >= cols && ld >= (count - 1) * step + cols);
}

// Whether `need` bytes of workspace are not there.
inline bool bad_workspace(const void* ws, size_t have, size_t need)
{
    return need > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || have < need);
}

inline int status_of(cudaError_t err)
{
    if (err == cudaErrorNotSupported)
        return GEMM_ERR_UNSUPPORTED;
    return err == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

}  // namespace tmmo
