// The row-grouped products on the FP32 units, of FP32 operands: 32 x 64 tiles,
// each of one group.
#include "grouped.cuh"
#include "launch.h"
#include "simt_tile.cuh"
#include "simt_types.h"

namespace tmmo {
namespace {

template <typename OutT>
__global__ void __launch_bounds__(ST_THREADS) grouped_simt_kernel(const GroupedLaunch l)
{
    __shared__ int table[GroupTable::BYTES / sizeof(int)];
    __shared__ SimtSmem s;
    const GroupTable groups = load_groups(table, l.by, ST_M, [](const GroupTable&, int) { return ST_M; }, [] {});
    OutT* Y = static_cast<OutT*>(l.Y);
    if (l.zero_rest)
        zero_rest_rows(groups, l.by, Y, l.ldy, l.N,
                       static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                       static_cast<int64_t>(gridDim.x) * blockDim.x);
    const int tiles_n = (l.N + ST_N - 1) / ST_N;
    const int64_t total = static_cast<int64_t>(groups.tile[l.by.groups]) * tiles_n;
    for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
        const int rt = static_cast<int>(t / tiles_n), n0 = static_cast<int>(t % tiles_n) * ST_N;
        const int g = groups.group_of(rt, l.by.groups);
        const int row0 = groups.first[g] + (rt - groups.tile[g]) * ST_M;
        const int rows = min(groups.first[g + 1] - row0, ST_M), cols = min(l.N - n0, ST_N);
        const View x{static_cast<const float*>(l.X) + row0 * l.ldx, l.ldx, 1};
        const float* w = static_cast<const float*>(l.W) + g * l.stride_w;
        const View v = l.w_t ? View{w + n0 * l.ldw, l.ldw, 1} : View{w + n0, 1, l.ldw};
        SimtValues acc = {};
        simt_accumulate(acc, s, x, v, 0, l.K, [&](int i, int) { return i < rows; },
                        [&](int j, int) { return j < cols; });
        simt_store(acc, Y + row0 * l.ldy + n0, l.ldy, rows, cols, l.alpha, l.beta);
    }
}

template <typename OutT>
__global__ void __launch_bounds__(ST_THREADS) grouped_wgrad_simt_kernel(const GroupedWgradLaunch l)
{
    __shared__ int table[GroupTable::BYTES / sizeof(int)];
    __shared__ SimtSmem s;
    const GroupTable groups = load_groups(table, l.by, 0, [](const GroupTable&, int) { return 0; }, [] {});
    const int tiles_n = (l.N + ST_M - 1) / ST_M, tiles_k = (l.K + ST_N - 1) / ST_N;
    const int64_t per_group = static_cast<int64_t>(tiles_n) * tiles_k;
    for (int64_t t = blockIdx.x; t < per_group * l.by.groups; t += gridDim.x) {
        const int g = static_cast<int>(t / per_group), u = static_cast<int>(t % per_group);
        const int n0 = u / tiles_k * ST_M, k0 = u % tiles_k * ST_N;
        const int rows = min(l.N - n0, ST_M), cols = min(l.K - k0, ST_N);
        const View d{static_cast<const float*>(l.D) + n0, 1, l.ldd};
        const View x{static_cast<const float*>(l.X) + k0, 1, l.ldx};
        SimtValues acc = {};
        simt_accumulate(acc, s, d, x, groups.first[g], groups.first[g + 1],
                        [&](int i, int) { return i < rows; }, [&](int j, int) { return j < cols; });
        simt_store(acc, static_cast<OutT*>(l.C) + g * l.stride_c + n0 * l.ldc + k0, l.ldc, rows,
                   cols, l.alpha, l.beta);
    }
}

}  // namespace

cudaError_t grouped_simt_launch(const GroupedLaunch& l, cudaStream_t stream)
{
    const int64_t tiles = (l.by.rows / ST_M + static_cast<int64_t>(l.by.groups)) * ((l.N + ST_N - 1) / ST_N);
    return with_type(l.out_dtype, [&](auto out) {
        note_launch();
        grouped_simt_kernel<decltype(out)>
            <<<simt_blocks(tiles, l.num_sms), ST_THREADS, 0, stream>>>(l);
        return cudaGetLastError();
    });
}

cudaError_t grouped_wgrad_simt_launch(const GroupedWgradLaunch& l, cudaStream_t stream)
{
    const int64_t tiles = static_cast<int64_t>(l.by.groups) * ((l.N + ST_M - 1) / ST_M) * ((l.K + ST_N - 1) / ST_N);
    return with_type(l.out_dtype, [&](auto out) {
        note_launch();
        grouped_wgrad_simt_kernel<decltype(out)>
            <<<simt_blocks(tiles, l.num_sms), ST_THREADS, 0, stream>>>(l);
        return cudaGetLastError();
    });
}

}  // namespace tmmo
