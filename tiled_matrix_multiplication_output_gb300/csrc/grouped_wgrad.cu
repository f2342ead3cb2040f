// Launch of the grouped weight gradient on the tensor cores (grouped_tc.cuh).
#include "grouped_launch.cuh"

namespace tmmo {

cudaError_t grouped_wgrad_tc_launch(const GroupedWgradLaunch& l, cudaStream_t stream)
{
    GroupedTcParams p{};
    p.by = l.by;
    p.C = l.C;
    p.ldc = l.ldc;
    p.stride_c = l.stride_c;
    p.N = l.N;
    p.K = l.K;
    p.tiles_f = (l.N + 255) / 256;
    p.tiles_c = (l.K + GT_N - 1) / GT_N;
    p.alpha = l.alpha;
    p.beta = l.beta;
    p.idesc = tc_idesc(l.in_dtype == DT_BF16, 256, 0, true, true);
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip_kblock = l.fault_skip_kblock;
    const int64_t rows = l.by.rows, groups = l.by.groups;
    GroupedMaps m;
    if (!encode_map(&m.a, l.in_dtype, l.D, 2, {l.N, rows, 1}, {l.ldd, 0}, {64, TC_BK, 1}) ||
        !encode_map(&m.b, l.in_dtype, l.X, 2, {l.K, rows, 1}, {l.ldx, 0}, {64, TC_BK, 1}))
        return cudaErrorNotSupported;
    m.b64 = m.b32 = m.b16 = m.c = m.b;
    const int64_t size = type_bytes(l.out_dtype);
    p.unit = row_unit(l.C, l.ldc * size, groups > 1 ? l.stride_c * size : 0);
    const int64_t stride = groups > 1 ? l.stride_c : l.N * l.ldc;
    p.tma_out = l.beta == 0.0f && p.unit != 0 && stride >= l.ldc &&  // (not interleaved row by row)
                encode_map(&m.c, l.out_dtype, l.C, 3, {l.K, l.N, groups}, {l.ldc, stride},
                           {static_cast<uint32_t>(64 / size), 32, 1});
    const int64_t most = groups * p.tiles_f * p.tiles_c;
    return launch_grouped_tc<GROUPED_WGRAD>(l.out_dtype, m, p, most, l.num_sms, stream);
}

}  // namespace tmmo
