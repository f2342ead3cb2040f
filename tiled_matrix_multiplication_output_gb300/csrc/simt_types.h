// Host side of the FP32-unit kernels: their instances by type, their grids.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "launch.h"

namespace tmmo {

// Calls f with a value of the type a DT_* code names.
template <typename F>
cudaError_t with_type(int dtype, F f)
{
    switch (dtype) {
    case DT_F32:
        return f(float{});
    case DT_F16:
        return f(__half{});
    default:
        return f(__nv_bfloat16{});
    }
}

// Two blocks for each SM, one hiding the other's latencies.
inline unsigned simt_blocks(int64_t tiles, int num_sms)
{
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(tiles, 2ll * num_sms)));
}

}  // namespace tmmo
