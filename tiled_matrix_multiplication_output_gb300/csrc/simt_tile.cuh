// A 64 x 64 output tile on the FP32 units, for the row-grouped products and
// the adapters: operands with any strides, ragged in every extent.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace tmmo {

constexpr int ST = 64;            // rows and columns of a tile
constexpr int ST_K = 16;          // depth of a step
constexpr int ST_THREADS = 256;   // 16 x 16 threads of 4 x 4 values

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Element (i, k) of an operand at p[i * outer + k * inner].
struct View {
    const float* p;
    int64_t outer, inner;
    __device__ float at(int i, int k) const { return p[i * outer + k * inner]; }
};

struct alignas(16) SimtSmem {  // read as float4
    float a[ST_K][ST + 4];
    float b[ST_K][ST + 4];
};

// Fills one operand's step: keep(i, k) says which elements exist; others are
// zero.  Threads run along whichever axis is contiguous.
template <typename Keep>
__device__ __forceinline__ void simt_fill(float (&s)[ST_K][ST + 4], const View& v, int k0, Keep keep)
{
    const int tid = threadIdx.x;
#pragma unroll
    for (int j = 0; j < ST * ST_K / ST_THREADS; ++j) {
        const int i = v.inner == 1 ? tid / ST_K + 16 * j : tid % ST;
        const int k = v.inner == 1 ? tid % ST_K : tid / ST + 4 * j;
        s[k][i] = keep(i, k0 + k) ? v.at(i, k0 + k) : 0.0f;
    }
}

// acc += A B^T over [k0, k1) of the operands' inner axis, this thread's
// values: rows 4 * (tid / 16) + i, columns 4 * (tid % 16) + j.
template <typename KeepA, typename KeepB>
__device__ __forceinline__ void simt_accumulate(float (&acc)[4][4], SimtSmem& s, const View& a,
                                                const View& b, int k0, int k1, KeepA keep_a,
                                                KeepB keep_b)
{
    const int r0 = 4 * (threadIdx.x / 16), c0 = 4 * (threadIdx.x % 16);
    for (int k = k0; k < k1; k += ST_K) {
        __syncthreads();
        simt_fill(s.a, a, k, [&](int i, int kk) { return kk < k1 && keep_a(i, kk); });
        simt_fill(s.b, b, k, [&](int i, int kk) { return kk < k1 && keep_b(i, kk); });
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < ST_K; ++kk) {
            const float4 x = *reinterpret_cast<const float4*>(&s.a[kk][r0]);
            const float4 y = *reinterpret_cast<const float4*>(&s.b[kk][c0]);
            const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
        }
    }
}

// C = alpha * acc + beta * C for the tile's rows and columns that exist.
template <typename OutT>
__device__ __forceinline__ void simt_store(const float (&acc)[4][4], OutT* C, int64_t ldc, int rows,
                                           int cols, float alpha, float beta)
{
    const int r0 = 4 * (threadIdx.x / 16), c0 = 4 * (threadIdx.x % 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r0 + i < rows && c0 + j < cols) {
                OutT* p = C + (r0 + i) * ldc + c0 + j;
                put(p, beta != 0.0f ? fmaf(beta, to_f32(*p), alpha * acc[i][j])
                                    : alpha * acc[i][j]);
            }
}

}  // namespace tmmo
