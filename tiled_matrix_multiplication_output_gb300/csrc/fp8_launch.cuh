// Tensor maps of quantised operands, for the translation units that launch
// products of them.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "device.h"
#include "fp8.h"
#include "fp8_gemm.cuh"
#include "launch.h"

namespace tmmo {
namespace {

inline int out_bytes(int dt) { return dt == DT_F32 ? 4 : 2; }

// Whether the product can be stored by TMA: nothing to add to, rows on
// 16-byte boundaries.
inline bool tma_output(const Fp8Launch& l)
{
    return l.beta == 0.0f && aligned16(l.C) && (l.ldc * out_bytes(l.out_dtype)) % 16 == 0;
}

// The stored matrix of an operand (outer x K, or K x outer when MN-major) in
// boxes of box_outer x 128 of K, swizzled over the length of a box row.  The
// row pitch is a multiple of 16 bytes; the matrix itself may end anywhere.
inline bool encode_operand(CUtensorMap* map, const Fp8Operand& o, int64_t outer, int64_t K,
                    uint32_t box_outer)
{
    auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(o.mn_major ? outer : K),
                                static_cast<cuuint64_t>(o.mn_major ? K : outer)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(o.ld)};
    const cuuint32_t row = o.mn_major ? box_outer : F8_BK;  // bytes of a box row
    const cuuint32_t box[2] = {o.mn_major ? box_outer : F8_BK, o.mn_major ? F8_BK : box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(o.data), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              row == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
              : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                          : CU_TENSOR_MAP_SWIZZLE_32B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace tmmo
