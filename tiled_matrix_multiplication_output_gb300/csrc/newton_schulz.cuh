// Pieces shared by the kernels of the Newton-Schulz orthogonalisation: the
// scales of stored values, FP16 pairs, loads and stores of matrix elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.h"
#include "load8.cuh"
#include "ops.cuh"

namespace tmmo {

// Stored value = scale * value.
constexpr float NS_SX = 4096.0f, NS_SA = 4096.0f, NS_SB = 2048.0f;

__device__ __forceinline__ float ns_value(const float* p) { return *p; }
__device__ __forceinline__ float ns_value(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float ns_value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ float2 ns_unpack(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ uint32_t ns_pack(float lo, float hi)
{
    return pack2(lo, hi, static_cast<__half*>(nullptr));
}

template <typename OutT>
__device__ __forceinline__ OutT ns_to_out(float v)
{
    if constexpr (sizeof(OutT) == 4) {
        return v;
    } else {
        const uint32_t u = pack2(v, 0.0f, static_cast<OutT*>(nullptr));
        return *reinterpret_cast<const OutT*>(&u);
    }
}

// A warp's 32 rows x 32 columns of the result, a row a lane, at `o` with row
// pitch ld; `rows` and `n` columns of them lie inside.  vec: rows are on
// 16-byte boundaries and a thread stores its own; otherwise the values go
// through 4 KiB of shared memory and are stored a row at a time, a column a
// lane.  Called by the whole warp.
template <typename OutT>
__device__ __forceinline__ void ns_store_result(OutT* o, long long ld, int rows, int n, bool vec,
                                                uint32_t stg, uint32_t lane, const float (&v)[32])
{
    if (vec && n == 32) {
        if (static_cast<int>(lane) >= rows)
            return;
        OutT* dst = o + static_cast<long long>(lane) * ld;
        constexpr int PER = 16 / static_cast<int>(sizeof(OutT));
#pragma unroll
        for (int c = 0; c < 32 / PER; ++c) {
            uint4 u;
            if constexpr (sizeof(OutT) == 4) {
                u = make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                               __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
            } else {
                OutT* tag = nullptr;
                u = make_uint4(pack2(v[8 * c], v[8 * c + 1], tag), pack2(v[8 * c + 2], v[8 * c + 3], tag),
                               pack2(v[8 * c + 4], v[8 * c + 5], tag),
                               pack2(v[8 * c + 6], v[8 * c + 7], tag));
            }
            *reinterpret_cast<uint4*>(dst + c * PER) = u;
        }
        return;
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c)
        st_shared_v4(stg + lane * 128 + ((c ^ (lane & 7)) << 4), __float_as_uint(v[4 * c]),
                     __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                     __float_as_uint(v[4 * c + 3]));
    __syncwarp();
    if (static_cast<int>(lane) < n) {
        o += lane;
#pragma unroll 8
        for (int r = 0; r < rows; ++r, o += ld)
            *o = ns_to_out<OutT>(ld_shared_f32(
                stg + r * 128 + ((((lane >> 2) ^ (r & 7)) << 4) | ((lane & 3) << 2))));
    }
}

// Eight consecutive values of a row, `n` of them inside it (zeros beyond).
template <typename InT>
__device__ __forceinline__ void ns_load8(const InT* src, int n, float (&v)[8])
{
    uint32_t w[2 * sizeof(InT)];
    load8(src, n, w);
    const InT* e = reinterpret_cast<const InT*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = ns_value(e + i);
}

template <typename T>
__device__ __forceinline__ T ns_block_sum(T s)
{
    __shared__ T part[32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, d);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i)
        s += part[i];
    return s;
}

// Squares are summed in FP32.  Below 2^-90 a sum may have lost squares to
// underflow (each loses at most 2^-150), above FP32 it is infinite: then it is
// taken again in FP64, which holds every square of an FP32 value.  (FP64 is two
// operations a cycle and SM here, too few for every call.)
__device__ __forceinline__ bool ns_squares_fit(float s) { return s >= 0x1p-90f && s <= 3.402823466e38f; }

// What the values of G are multiplied by, NS_SX / (norm + eps), from the sum of
// squares where that fits FP32 -- the first factor -- and otherwise in two
// factors, as their product may not fit.
__device__ __forceinline__ float2 ns_factors(float sum, float eps)
{
    return make_float2(NS_SX / (sqrtf(sum) + eps), 1.0f);
}
// Where the norm is not finite in FP32 the result is NaN throughout.
static __device__ __noinline__ float2 ns_factors_wide(double sum, float eps)
{
    const double norm = sqrt(sum);
    if (!(norm <= 3.402823466e38))
        return make_float2(__int_as_float(0x7fffffff), 1.0f);
    const double d = norm + eps;
    const double first = d < 0x1p-100 ? 0x1p100 : 1.0;
    return make_float2(static_cast<float>(first), static_cast<float>(NS_SX / (d * first)));
}

}  // namespace tmmo
