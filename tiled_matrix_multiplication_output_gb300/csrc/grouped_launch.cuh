// Host side of the row-grouped tensor-core kernel: its launch.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>

#include "grouped_maps.h"
#include "grouped_tc.cuh"
#include "launch.h"
#include "persistent.cuh"

namespace tmmo {

// Lanes' side; the other side in boxes of 128 rows and fewer; stored gradients.
struct GroupedMaps {
    CUtensorMap a, b, b64, b32, b16, c;
};

template <int MODE, typename OutT>
cudaError_t launch_grouped_tc(const GroupedMaps& m, const GroupedTcParams& p, int64_t most_work,
                              int num_sms, cudaStream_t stream)
{
    using L = GroupedLayout<MODE>;
    static ClusterCaps caps;
    int cap = 0;
    const cudaError_t err = cluster_cap(grouped_tc_kernel<MODE, OutT>, caps, 2, L::THREADS,
                                        L::SMEM_ALLOC, num_sms, &cap);
    if (err != cudaSuccess)
        return err;
    const int64_t units = std::min<int64_t>(std::max(cap, 1), std::max<int64_t>(most_work, 1));
    ClusterLaunch l(static_cast<unsigned>(2 * units), 2, L::THREADS, L::SMEM_ALLOC, stream);
    return l.run(grouped_tc_kernel<MODE, OutT>, m.a, m.b, m.b64, m.b32, m.b16, m.c, p);
}

template <int MODE>
cudaError_t launch_grouped_tc(int out_dtype, const GroupedMaps& m, const GroupedTcParams& p,
                              int64_t most_work, int num_sms, cudaStream_t stream)
{
    switch (out_dtype) {
    case DT_F32:
        return launch_grouped_tc<MODE, float>(m, p, most_work, num_sms, stream);
    case DT_F16:
        return launch_grouped_tc<MODE, __half>(m, p, most_work, num_sms, stream);
    default:
        return launch_grouped_tc<MODE, __nv_bfloat16>(m, p, most_work, num_sms, stream);
    }
}

}  // namespace tmmo
