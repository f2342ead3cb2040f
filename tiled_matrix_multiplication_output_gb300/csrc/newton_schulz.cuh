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
constexpr float NS_LO = 2048.0f;  // lo holds (X - hi) * NS_LO

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
__device__ __forceinline__ void ns_store_result(OutT* dst, int n, const float (&v)[32])
{
    const bool vec = (reinterpret_cast<uintptr_t>(dst) & 15u) == 0;
    constexpr int PER = 16 / static_cast<int>(sizeof(OutT));
#pragma unroll
    for (int c = 0; c < 32 / PER; ++c) {
        if (vec && (c + 1) * PER <= n) {
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
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (c * PER + i < n) {
                    if constexpr (sizeof(OutT) == 4) {
                        dst[c * PER + i] = v[c * PER + i];
                    } else {
                        OutT* tag = nullptr;
                        const uint32_t u = pack2(v[c * PER + i], 0.0f, tag);
                        dst[c * PER + i] = *reinterpret_cast<const OutT*>(&u);
                    }
                }
            }
        }
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

__device__ __forceinline__ float ns_block_sum(float s)
{
    __shared__ float part[32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, d);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i)
        s += part[i];
    return s;
}

}  // namespace tmmo
