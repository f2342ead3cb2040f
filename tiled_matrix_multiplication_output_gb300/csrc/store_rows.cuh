// From an accumulator in tensor memory to rows in global memory, for tiles of
// any extent.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

#include "ops.cuh"
#include "simt_tile.cuh"

namespace tmmo {

// p[r * ld] = alpha * v[r] + beta * p[r * ld] for r < rows: what is added to is
// loaded before anything is stored, so that the loads overlap.
template <int R, typename OutT>
__device__ __forceinline__ void put_column(OutT* p, int64_t ld, int rows, const float (&v)[R], float alpha,
                                           float beta)
{
    float old[R];
    if (beta != 0.0f) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            old[r] = r < rows ? to_f32(p[r * ld]) : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r < rows)
            put(p + r * ld, beta != 0.0f ? fmaf(beta, old[r], alpha * v[r]) : alpha * v[r]);
}

// Strip of 32 rows x 32 FP32 values (this thread holds a row) to C, through 2 KiB
// of shared memory, in whole sectors whatever the alignment.  A whole warp calls it.
template <typename OutT>
__device__ __forceinline__ void put_strip(const uint32_t (&v)[32], uint32_t staging, OutT* c, int64_t ldc,
                                          int rows, int cols, float alpha, float beta)
{
    const uint32_t lane = lane_id(), col = lane & 15, odd = lane >> 4;
#pragma unroll
    for (int h = 0; h < 32; h += 16) {  // 16 columns at a time, two rows a load
#pragma unroll
        for (int j = 0; j < 16; ++j)  // column j of row `lane` at j ^ (lane / 2) % 16
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(staging + lane * 64 + ((j ^ ((lane >> 1) & 15)) << 2)),
                         "r"(v[h + j])
                         : "memory");
        __syncwarp();
        if (h + static_cast<int>(col) < cols)
#pragma unroll 1
            for (int r = 0; r < rows; r += 16) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t row = r + 2 * i + odd;
                    f[i] = ld_shared_f32(staging + row * 64 + ((col ^ ((row >> 1) & 15)) << 2));
                }
                put_column(c + (r + odd) * ldc + h + col, 2 * ldc, (rows - r - static_cast<int>(odd) + 1) / 2, f,
                           alpha, beta);
            }
        __syncwarp();
    }
}

// The widest stores that rows allow: 32 or 16 bytes, or 0 for single values.
inline int row_unit(const void* p, int64_t row_bytes, int64_t matrix_bytes)
{
    const uintptr_t low = (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(row_bytes) |
                           static_cast<uintptr_t>(matrix_bytes)) & 31u;
    return low == 0 ? 32 : low == 16 ? 16 : 0;
}

// p[0 .. n) = alpha * v + beta * p of a row on a boundary of `unit` bytes, at most 32
// values: each thread its own row.
template <typename OutT>
__device__ __forceinline__ void put_row(OutT* p, const uint32_t (&v)[32], int n, int unit, float alpha,
                                        float beta)
{
    constexpr int EACH = 32 / sizeof(OutT);  // values of a store
#pragma unroll
    for (int i = 0; i < 32; i += EACH) {
        if (i + EACH <= n) {
            alignas(16) OutT h[EACH];
            uint4 q[2];
            if (beta != 0.0f) {
                q[0] = reinterpret_cast<const uint4*>(p + i)[0];
                q[1] = reinterpret_cast<const uint4*>(p + i)[1];
                memcpy(h, q, 32);
            }
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                const float f = alpha * __uint_as_float(v[i + k]);
                put(&h[k], beta != 0.0f ? fmaf(beta, to_f32(h[k]), f) : f);
            }
            if (unit == 32) {
                uint32_t w[8];
                memcpy(w, h, 32);
                st_global_v8(p + i, w);
            } else {
                memcpy(q, h, 32);
                reinterpret_cast<uint4*>(p + i)[0] = q[0];
                reinterpret_cast<uint4*>(p + i)[1] = q[1];
            }
        } else {
#pragma unroll
            for (int k = 0; k < EACH; ++k)
                if (i + k < n) {
                    const float f = alpha * __uint_as_float(v[i + k]);
                    put(p + i + k, beta != 0.0f ? fmaf(beta, to_f32(p[i + k]), f) : f);
                }
        }
    }
}

// The 16-byte unit u of row t of a 64-byte wide strip in shared memory, of which
// rows rows and cols values a row exist, to its place in rows of c on 16-byte
// boundaries.
template <typename OutT>
__device__ __forceinline__ void put_unit(uint32_t at, OutT* c, int64_t ldc, int t, int u, int rows, int cols)
{
    constexpr int EACH = 16 / sizeof(OutT);
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    OutT* p = c + t * ldc + EACH * u;
    const int left = cols - EACH * u;
    if (t < rows && left >= EACH) {
        *reinterpret_cast<uint4*>(p) = v;
    } else if (t < rows) {
        OutT h[EACH];
        memcpy(h, &v, 16);
#pragma unroll
        for (int k = 0; k < EACH; ++k)
            if (k < left)
                p[k] = h[k];
    }
}

// alpha * v of 32 rows (this thread holds one), 64 bytes of columns (part: which 16 of
// the values, for FP32), to shared memory as a TMA store of such boxes expects it,
// 64-byte swizzled: 16-byte unit u of row r at u ^ (r / 2) % 4, without bank conflicts.
// A whole warp calls it.
template <typename OutT>
__device__ __forceinline__ void strip_to_smem(const uint32_t (&v)[32], int part, uint32_t staging, float alpha)
{
    const uint32_t lane = lane_id(), turn = (lane >> 1) & 3;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        uint32_t w[4];
        if constexpr (sizeof(OutT) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = __float_as_uint(alpha * __uint_as_float(v[16 * part + 4 * u + i]));
        } else {
            OutT* tag = nullptr;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = pack2(alpha * __uint_as_float(v[8 * u + 2 * i]),
                             alpha * __uint_as_float(v[8 * u + 2 * i + 1]), tag);
        }
        st_shared_v4(staging + lane * 64 + ((u ^ turn) << 4), w[0], w[1], w[2], w[3]);
    }
}

// The same to rows of c on 16-byte boundaries: a store covers 64 bytes of eight rows.
template <typename OutT>
__device__ __forceinline__ void put_rows(const uint32_t (&v)[32], int part, uint32_t staging, OutT* c,
                                         int64_t ldc, int rows, int cols, float alpha)
{
    const uint32_t lane = lane_id();
    strip_to_smem<OutT>(v, part, staging, alpha);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 8 * i + static_cast<int>(lane >> 2), u = lane & 3;
        put_unit(staging + t * 64 + ((u ^ ((t >> 1) & 3)) << 4), c, ldc, t, u, rows, cols);
    }
    __syncwarp();
}

// ------------------------------------------- tiles that are stored turned

// 16 lanes x 32 columns of 32 bits in the layout of a matrix fragment: for each
// eight columns 8 i, r[4 i] and r[4 i + 1] are lane l / 4, columns
// 8 i + 2 (l % 4) and the next one; r[4 i + 2], r[4 i + 3] the same of lane l / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane 8 m + j gives the address
// of the 16 bytes of column j of matrix m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
                 "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// 32 lanes x 32 columns, as tmem_ld_16x256b_x4 gives lanes 0 to 15 and 16 to 31, as 32
// rows (the columns) of 32 16-bit values (the lanes) to y, through 2 KiB of shared
// memory; rows of y are on 16-byte boundaries.  n rows and m values of each exist.  A
// whole warp calls it.
template <typename OutT>
__device__ __forceinline__ void put_turned(const float (&v)[32], uint32_t staging, OutT* y, int64_t ldy,
                                           int n, int m, float alpha)
{
    const uint32_t lane = lane_id();
    OutT* tag = nullptr;
    // 16-byte unit u of row t at u ^ (t / 2) % 4: no bank conflicts either way
    const uint32_t at = staging + lane * 64, turn = (lane >> 1) & 3;
#pragma unroll
    for (int u = 0; u < 4; ++u) {  // eight lanes of the accumulator
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = 16 * (u >> 1) + 4 * i + 2 * (u & 1);
            w[i] = pack2(alpha * v[k], alpha * v[k + 1], tag);
        }
        stmatrix_x4_trans(at + ((u ^ turn) << 4), w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 8 * i + static_cast<int>(lane >> 2), k = lane & 3;
        put_unit(staging + t * 64 + ((k ^ ((t >> 1) & 3)) << 4), y, ldy, t, k, n, m);
    }
    __syncwarp();
}

}  // namespace tmmo
