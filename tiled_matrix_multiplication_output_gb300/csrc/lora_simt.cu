// Low-rank adapters on the FP32 units, of FP32 operands: 32 x 64 tiles of the shared product,
// and of each adapter's among the tile's rows.
#include "launch.h"
#include "lora.h"
#include "simt_tile.cuh"
#include "simt_types.h"

namespace tmmo {
namespace {

// The adapters of a tile's rows (-1: none, or behind the last row).
__device__ __forceinline__ void load_adapters(int (&s)[ST_M], const int32_t* adapter, int row0, int rows,
                                              int adapters)
{
    __syncthreads();
    if (threadIdx.x < ST_M) {
        const int i = row0 + threadIdx.x;
        const int g = adapters > 0 && i < rows ? adapter[i] : -1;
        s[threadIdx.x] = g >= 0 && g < adapters ? g : -1;
    }
    __syncthreads();
}

// Calls f(g) once for each adapter among the tile's rows.
template <typename F>
__device__ __forceinline__ void each_adapter(const int (&s)[ST_M], F f)
{
    for (int i = 0; i < ST_M; ++i) {
        const int g = s[i];
        bool seen = g < 0;
        for (int j = 0; j < i && !seen; ++j)
            seen = s[j] == g;
        if (!seen)
            f(g);
    }
}

__global__ void __launch_bounds__(ST_THREADS) lora_shrink_kernel(const LoraLaunch l)
{
    __shared__ SimtSmem s;
    __shared__ int of[ST_M];
    const int tiles_r = (l.rank + ST_N - 1) / ST_N;
    const int64_t total = static_cast<int64_t>((l.rows + ST_M - 1) / ST_M) * tiles_r;
    const int r0 = simt_row(), c0 = simt_col();
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const int row0 = static_cast<int>(tile / tiles_r) * ST_M, j0 = static_cast<int>(tile % tiles_r) * ST_N;
        const int cols = min(l.rank - j0, ST_N);
        load_adapters(of, l.adapter, row0, l.rows, l.adapters);
        const View x{static_cast<const float*>(l.X) + row0 * l.ldx, l.ldx, 1};
        each_adapter(of, [&](int g) {
            const float* f = static_cast<const float*>(l.F) + g * l.stride_f;
            const View v = l.across ? View{f + j0, 1, l.ldf} : View{f + j0 * l.ldf, l.ldf, 1};
            SimtValues acc = {};
            simt_accumulate(acc, s, x, v, 0, l.K, [&](int i, int) { return of[i] == g; },
                            [&](int j, int) { return j < cols; });
            const float scale = l.scale ? l.scale[g] : 1.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (of[r0 + i] == g && c0 + j < cols)
                        static_cast<float*>(l.t)[static_cast<int64_t>(row0 + r0 + i) * l.rank + j0 + c0 + j] =
                            scale * acc[i][j];
        });
    }
}

template <typename OutT>
__global__ void __launch_bounds__(ST_THREADS) lora_expand_kernel(const LoraLaunch l)
{
    __shared__ SimtSmem s;
    __shared__ int of[ST_M];
    const int tiles_n = (l.N + ST_N - 1) / ST_N;
    const int64_t total = static_cast<int64_t>((l.rows + ST_M - 1) / ST_M) * tiles_n;
    const int r0 = simt_row();
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const int row0 = static_cast<int>(tile / tiles_n) * ST_M, n0 = static_cast<int>(tile % tiles_n) * ST_N;
        const int rows = min(l.rows - row0, ST_M), cols = min(l.N - n0, ST_N);
        load_adapters(of, l.adapter, row0, l.rows, l.adapters);
        const View x{static_cast<const float*>(l.X) + row0 * l.ldx, l.ldx, 1};
        auto columns = [&](const void* base, int64_t off, int64_t ld) {
            const float* p = static_cast<const float*>(base) + off;
            return l.across ? View{p + n0, 1, ld} : View{p + n0 * ld, ld, 1};
        };
        auto in_cols = [&](int j, int) { return j < cols; };
        SimtValues acc = {};
        simt_accumulate(acc, s, x, columns(l.W, 0, l.ldw), 0, l.K, [&](int i, int) { return i < rows; },
                        in_cols);
        const View t{static_cast<const float*>(l.t) + static_cast<int64_t>(row0) * l.rank, l.rank, 1};
        each_adapter(of, [&](int g) {
            SimtValues add = {};
            simt_accumulate(add, s, t, columns(l.E, g * l.stride_e, l.lde), 0, l.rank,
                            [&](int i, int) { return of[i] == g; }, in_cols);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (of[r0 + i] == g)  // rows of other adapters see nothing of this one
                        acc[i][j] += add[i][j];
        });
        simt_store(acc, static_cast<OutT*>(l.Y) + row0 * l.ldy + n0, l.ldy, rows, cols, 1.0f, 0.0f);
    }
}

// Sixteen rows at a time, so that rows of other adapters between cost a look only: no
// copy is ahead of its use here, and the warps' sums are added for every sixteen.
// (1000 rows of four adapters by 1024 and 768 columns, rank 16: the backward pass 270
// us, the forward one 131.)
template <typename OutT>
__global__ void __launch_bounds__(ST_THREADS) lora_grad_kernel(const LoraGradLaunch l)
{
    __shared__ SimtSmem s;
    const int tiles_c = (l.cols + ST_M - 1) / ST_M, tiles_r = (l.rank + ST_N - 1) / ST_N;
    const int64_t per = static_cast<int64_t>(tiles_c) * tiles_r;
    const int r0 = simt_row(), c0 = simt_col();
    for (int64_t tile = blockIdx.x; tile < per * l.adapters; tile += gridDim.x) {
        const int g = static_cast<int>(tile / per), u = static_cast<int>(tile % per);
        const int p0 = u / tiles_r * ST_M, j0 = u % tiles_r * ST_N;
        const int rows = min(l.cols - p0, ST_M), cols = min(l.rank - j0, ST_N);
        const View p{static_cast<const float*>(l.P) + p0, 1, l.ldp};
        const View t{static_cast<const float*>(l.t) + j0, 1, l.rank};
        SimtValues acc = {};
        for (int k = 0; k < l.rows; k += ST_K) {
            const int i = k + static_cast<int>(threadIdx.x);
            if (!__syncthreads_or(threadIdx.x < ST_K && i < l.rows && l.adapter[i] == g))
                continue;
            simt_accumulate(acc, s, p, t, k, min(k + ST_K, l.rows),
                            [&](int c, int row) { return c < rows && l.adapter[row] == g; },
                            [&](int j, int row) { return j < cols && l.adapter[row] == g; });
        }
        OutT* out = static_cast<OutT*>(l.G) + g * l.stride_g;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r0 + i < rows && c0 + j < cols)
                    put(out + (p0 + r0 + i) * l.step_c + (j0 + c0 + j) * l.step_j, acc[i][j]);
    }
}

}  // namespace

cudaError_t lora_simt_shrink(const LoraLaunch& l, cudaStream_t stream)
{
    const int64_t tiles = static_cast<int64_t>((l.rows + ST_M - 1) / ST_M) * ((l.rank + ST_N - 1) / ST_N);
    note_launch();
    lora_shrink_kernel<<<simt_blocks(tiles, l.num_sms), ST_THREADS, 0, stream>>>(l);
    return cudaGetLastError();
}

cudaError_t lora_simt_expand(const LoraLaunch& l, cudaStream_t stream)
{
    const int64_t tiles = static_cast<int64_t>((l.rows + ST_M - 1) / ST_M) * ((l.N + ST_N - 1) / ST_N);
    return with_type(l.out_dtype, [&](auto out) {
        note_launch();
        lora_expand_kernel<decltype(out)>
            <<<simt_blocks(tiles, l.num_sms), ST_THREADS, 0, stream>>>(l);
        return cudaGetLastError();
    });
}

cudaError_t lora_simt_grad(const LoraGradLaunch& l, cudaStream_t stream)
{
    const int64_t tiles = static_cast<int64_t>(l.adapters) * ((l.cols + ST_M - 1) / ST_M) *
                          ((l.rank + ST_N - 1) / ST_N);
    return with_type(l.out_dtype, [&](auto out) {
        note_launch();
        lora_grad_kernel<decltype(out)>
            <<<simt_blocks(tiles, l.num_sms), ST_THREADS, 0, stream>>>(l);
        return cudaGetLastError();
    });
}

}  // namespace tmmo
