// A 32 x 64 output tile on the FP32 units, for the row-grouped products and
// the adapters: operands with any strides, ragged in every extent.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace tmmo {

constexpr int ST_M = 32;          // rows of a tile
constexpr int ST_N = 64;          // columns
constexpr int ST_K = 16;          // depth of a step
constexpr int ST_THREADS = 256;
constexpr int ST_STAGES = 4;      // steps in shared memory, three of them on their way
constexpr int ST_PAD = 4;         // values between rows in shared memory

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
};

struct alignas(16) SimtStep {  // read as float4
    float a[ST_K][ST_M + ST_PAD];
    float b[ST_K][ST_N + ST_PAD];
};
struct SimtSmem {
    SimtStep step[ST_STAGES];
};

// Asynchronous copy of a value, or (not `there`) a zero.
__device__ __forceinline__ void cp_async_4_or_zero(uint32_t dst, const float* src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0)
                 : "memory");
}

// Copies this thread's elements of the steps of an operand of W rows (columns), in
// order.  Threads run along whichever axis is contiguous; keep(i, k) says which
// elements exist, others are zero.
template <int W>
class SimtLoader {
public:
    __device__ SimtLoader(const View& v, int k0) : along_(v.inner == 1), step_(ST_K * v.inner), base_(v.p)
    {
        const int tid = threadIdx.x;
        i_ = along_ ? tid / ST_K : tid % W;
        k_ = along_ ? tid % ST_K : tid / W;
        p_ = v.p + i_ * v.outer + (k0 + k_) * v.inner;
        next_ = along_ ? I_STEP * v.outer : K_STEP * v.inner;
    }
    // The step that starts at k0, the next one of the sequence.
    template <typename Keep>
    __device__ void load(float (&s)[ST_K][W + ST_PAD], int k0, Keep keep)
    {
        const float* p = p_;
        uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&s[k_][i_]));
        const uint32_t step = (along_ ? I_STEP : K_STEP * (W + ST_PAD)) * 4;
#pragma unroll
        for (int j = 0; j < EACH; ++j, p += next_, to += step) {
            const bool there = keep(i_ + (along_ ? I_STEP * j : 0), k0 + k_ + (along_ ? 0 : K_STEP * j));
            cp_async_4_or_zero(to, there ? p : base_, there);
        }
        p_ += step_;
    }

private:
    static constexpr int EACH = W * ST_K / ST_THREADS;
    static constexpr int I_STEP = ST_THREADS / ST_K, K_STEP = ST_THREADS / W;
    bool along_;
    int i_, k_;
    int64_t step_, next_;
    const float *base_, *p_;
};

// This thread's values of a tile: rows simt_row() + i, columns simt_col() + j.
using SimtValues = float[2][4];
__device__ __forceinline__ int simt_row() { return 2 * (threadIdx.x / 16); }
__device__ __forceinline__ int simt_col() { return 4 * (threadIdx.x % 16); }

// acc += A B^T over [k0, k1) of the operands' inner axis.  Three steps are on
// their way while one is multiplied.  The eight warps share a step's depth, each
// thread with 8 x 8 values, and their sums are added at the end: with few
// values a thread the loads from shared memory, not the multiply-adds, set the
// pace.  The tile is small because an SM that gets one more than others takes as
// much longer: 999 rows of eight groups by 512 x 768 took 63 us in 160 tiles of
// 64 x 64, three of which met on one SM, and take 33 so (24 TFLOP/s; 8192 rows of eight
// by 2048 x 2048, where a larger tile would do better, 33).
template <typename KeepA, typename KeepB>
__device__ __forceinline__ void simt_accumulate(SimtValues& acc, SimtSmem& smem, const View& a, const View& b,
                                                int k0, int k1, KeepA keep_a, KeepB keep_b)
{
    constexpr int WARPS = ST_THREADS / 32, DEPTH = ST_K / WARPS;
    const int warp = threadIdx.x / 32;
    // a thread's rows r4 .. r4 + 3 and 16 behind, its columns c4 .. c4 + 3 and 32 behind:
    // eight threads read 128 contiguous bytes
    const int r4 = 4 * (threadIdx.x % 32 / 8), c4 = 4 * (threadIdx.x % 8);
    SimtLoader<ST_M> la(a, k0);
    SimtLoader<ST_N> lb(b, k0);
    auto load = [&](int stage, int k) {
        if (k < k1) {
            la.load(smem.step[stage].a, k, [&](int i, int kk) { return kk < k1 && keep_a(i, kk); });
            lb.load(smem.step[stage].b, k, [&](int i, int kk) { return kk < k1 && keep_b(i, kk); });
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();  // whoever used the stages before is done
    for (int i = 0; i < ST_STAGES - 1; ++i)
        load(i, k0 + i * ST_K);
    float part[8][8] = {};
    int stage = 0;
    for (int k = k0; k < k1; k += ST_K) {
        asm volatile("cp.async.wait_group %0;" ::"n"(ST_STAGES - 2) : "memory");
        __syncthreads();
        load((stage + ST_STAGES - 1) % ST_STAGES, k + (ST_STAGES - 1) * ST_K);
        const SimtStep& s = smem.step[stage];
        stage = (stage + 1) % ST_STAGES;
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int kk = warp * DEPTH + d;
            float x[8], y[8];
#pragma unroll
            for (int h = 0; h < 8; h += 4) {
                *reinterpret_cast<float4*>(x + h) = *reinterpret_cast<const float4*>(&s.a[kk][r4 + 4 * h]);
                *reinterpret_cast<float4*>(y + h) = *reinterpret_cast<const float4*>(&s.b[kk][c4 + 8 * h]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    part[i][j] = fmaf(x[i], y[j], part[i][j]);
        }
    }
    // the warps' sums, two at a time through the stages' memory, in their order
    constexpr int PITCH = ST_N + ST_PAD;
    static_assert(sizeof(SimtSmem) >= 2 * ST_M * PITCH * sizeof(float), "two sums of a tile");
    float* const sums = reinterpret_cast<float*>(&smem);
#pragma unroll 1
    for (int w = 0; w < WARPS; w += 2) {
        __syncthreads();
        if (warp == w || warp == w + 1) {
            float* to = sums + (warp - w) * ST_M * PITCH + r4 * PITCH + c4;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int h = 0; h < 8; h += 4)
                    *reinterpret_cast<float4*>(to + (i % 4 + i / 4 * 16) * PITCH + 8 * h) =
                        make_float4(part[i][h], part[i][h + 1], part[i][h + 2], part[i][h + 3]);
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(sums + q * ST_M * PITCH +
                                                                  (simt_row() + i) * PITCH + simt_col());
                acc[i][0] += v.x;
                acc[i][1] += v.y;
                acc[i][2] += v.z;
                acc[i][3] += v.w;
            }
    }
}

// C = alpha * acc + beta * C for the tile's rows and columns that exist.
template <typename OutT>
__device__ __forceinline__ void simt_store(const SimtValues& acc, OutT* C, int64_t ldc, int rows, int cols,
                                           float alpha, float beta)
{
    const int r0 = simt_row(), c0 = simt_col();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r0 + i < rows && c0 + j < cols) {
                OutT* p = C + (r0 + i) * ldc + c0 + j;
                put(p, beta != 0.0f ? fmaf(beta, to_f32(*p), alpha * acc[i][j])
                                    : alpha * acc[i][j]);
            }
}

}  // namespace tmmo
