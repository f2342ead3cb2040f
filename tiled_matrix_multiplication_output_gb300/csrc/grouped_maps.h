// Tensor maps of the row-grouped products and the adapters (host side).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device.h"
#include "launch.h"

namespace tmmo {

inline int type_bytes(int dt) { return dt == DT_F32 ? 4 : 2; }

// A tensor of up to three dimensions, innermost first, in boxes whose rows are
// 128, 64 or 32 bytes, swizzled over that length; strides in elements.
inline bool encode_map(CUtensorMap* map, int dt, const void* base, int rank, const int64_t (&dims)[3],
                       const int64_t (&strides)[2], const uint32_t (&box)[3])
{
    auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (!fn)
        return false;
    const CUtensorMapDataType type = dt == DT_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dt == DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    cuuint64_t d[3], s[2];
    for (int i = 0; i < 3; ++i)
        d[i] = static_cast<cuuint64_t>(dims[i]);
    for (int i = 0; i < 2; ++i)
        s[i] = static_cast<cuuint64_t>(strides[i]) * type_bytes(dt);
    const cuuint32_t step[3] = {1, 1, 1};
    const uint32_t row = box[0] * static_cast<uint32_t>(type_bytes(dt));
    return fn(map, type, rank, const_cast<void*>(base), d, s, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              row == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
              : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                          : CU_TENSOR_MAP_SWIZZLE_32B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensor maps of one call, each encoded once (0.5 us of host time): its kernels
// read some matrices in the same boxes.
class TensorMaps {
public:
    bool get(CUtensorMap* map, int dt, const void* base, int rank, const int64_t (&dims)[3],
             const int64_t (&strides)[2], const uint32_t (&box)[3])
    {
        const Key key{base, {dims[0], dims[1], dims[2]}, {strides[0], strides[1]}, {box[0], box[1], box[2]},
                      dt, rank};
        for (int i = 0; i < n_; ++i)
            if (key == keys_[i]) {
                *map = maps_[i];
                return true;
            }
        if (!encode_map(map, dt, base, rank, dims, strides, box))
            return false;
        if (n_ < kMost) {
            keys_[n_] = key;
            maps_[n_++] = *map;
        }
        return true;
    }

private:
    struct Key {
        const void* base;
        int64_t dims[3], strides[2];
        uint32_t box[3];
        int dt, rank;
        bool operator==(const Key& k) const
        {
            return base == k.base && dt == k.dt && rank == k.rank && box[0] == k.box[0] && box[1] == k.box[1] &&
                   box[2] == k.box[2] && dims[0] == k.dims[0] && dims[1] == k.dims[1] && dims[2] == k.dims[2] &&
                   strides[0] == k.strides[0] && strides[1] == k.strides[1];
        }
    };
    static constexpr int kMost = 16;
    int n_ = 0;
    Key keys_[kMost];
    CUtensorMap maps_[kMost];
};

// Whether TMA can address rows of this pitch (elements).
inline bool aligned_rows(const void* p, int64_t ld, int dt)
{
    return aligned16(p) && (ld * type_bytes(dt)) % 16 == 0;
}

}  // namespace tmmo
