// Low-rank adapters on the tensor cores: what the kernels share.
//
// The rows of a 128-row tile may have different adapters.  One matrix
// instruction multiplies all 128 rows by one adapter's factor, and its mask of
// lanes keeps the result away from the rows of others: their accumulators are
// not touched, whatever the factor holds.  A tile's plan lists its adapters,
// ascending, with the rows of each.
//
// The rank values t are FP32 sums that enter a second product as operands of 16
// bits, in parts: t = p0 + p1 (+ p2), each the rounding of what the ones before
// leave, multiplied by the same factor.  Two parts hold 16 bits of a BF16 value
// and 22 of an FP16 one, three hold 24.  An FP16 part is no finer than 2^-24, which
// a product may leave out beside the shared one, but not a gradient that is nothing
// but rank values times rows (its values may be 1e-6): its third part is of 2^20
// times what the two leave, and has an accumulator of its own.  They lie in chunks of
// `chunk` rank values, 64 columns (128 bytes, a swizzle row) a chunk: part p of value
// j at column (j / chunk) * 64 + p * chunk + j % chunk.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "launch.h"
#include "lora.h"
#include "ops.cuh"
#include "simt_tile.cuh"
#include "warp_roles.cuh"

namespace tmmo {

constexpr int LT_ROWS = 128;  // rows of a tile, the lanes of a CTA
constexpr float LT_FINE = 1048576.0f;  // 2^20: a remainder of 2^-8 at most stays below 65504

struct alignas(16) LoraPlan {
    int count;                  // adapters among the tile's rows
    int pad[3];
    int ids[LT_ROWS];           // ascending
    uint32_t rows[LT_ROWS][4];  // bit i of the i-th: row i has this adapter
};
static_assert(sizeof(LoraPlan) == LORA_PLAN_BYTES, "size of a plan in the workspace");

// The adapter of a row, or -1.
__device__ __forceinline__ int row_adapter(const int32_t* adapter, int row, int rows, int adapters)
{
    const int g = row < rows ? adapter[row] : -1;
    return g >= 0 && g < adapters ? g : -1;
}

struct PlanScratch {
    int4 of[LT_ROWS / 4];     // each row's adapter
    int4 first[LT_ROWS / 4];  // the same of its adapter's first row, else INT_MAX
};

// The plan of a tile's rows: 128 threads call it, each (i) with its row's adapter g,
// with a barrier sync() of theirs, in which it ends.  Returns the row's place in the
// plan, or -1.
template <typename Sync>
__device__ __forceinline__ int make_plan(LoraPlan& plan, PlanScratch& s, int g, int i, Sync sync)
{
    int* first = reinterpret_cast<int*>(s.first);
    reinterpret_cast<int*>(s.of)[i] = g;
    *reinterpret_cast<uint4*>(plan.rows[i]) = make_uint4(0, 0, 0, 0);
    if (i == 0)
        plan.count = 0;
    sync();
    int before = 0;  // earlier rows with the same adapter
#pragma unroll 4
    for (int j = 0; j < LT_ROWS / 4; ++j) {
        const int4 v = s.of[j];
        before |= (v.x == g & 4 * j < i) | (v.y == g & 4 * j + 1 < i) | (v.z == g & 4 * j + 2 < i) |
                  (v.w == g & 4 * j + 3 < i);
    }
    first[i] = g >= 0 && !before ? g : 0x7fffffff;
    sync();
    int place = -1;
    if (g >= 0) {
        place = 0;
#pragma unroll 4
        for (int j = 0; j < LT_ROWS / 4; ++j) {
            const int4 v = s.first[j];
            place += (v.x < g) + (v.y < g) + (v.z < g) + (v.w < g);
        }
        if (!before) {
            plan.ids[place] = g;
            atomicAdd(&plan.count, 1);
        }
        atomicOr(&plan.rows[place][i >> 5], 1u << (i & 31));
    }
    sync();
    return place;
}

// D[tmem] (+)= A B for the lanes whose bit of `off` is clear.
__device__ __forceinline__ void tc_mma_f16_lanes(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate,
                                                 const uint32_t (&off)[4])
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(off[0]), "r"(off[1]), "r"(off[2]),
        "r"(off[3])
        : "memory");
}
// The same on a CTA pair: the leader's lanes, then its peer's.
__device__ __forceinline__ void tc_mma_f16_lanes(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate,
                                                 const uint32_t (&off)[8])
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%5, %6, %7, %8, %9, %10, %11, %12}, "
        "p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(off[0]), "r"(off[1]), "r"(off[2]),
        "r"(off[3]), "r"(off[4]), "r"(off[5]), "r"(off[6]), "r"(off[7])
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                            int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// How the rank values are laid out.
struct LoraParts {
    int parts, chunk, chunks;
    int plain;    // parts to the scale of 1; one behind them is to that of LT_FINE
    __host__ __device__ int columns() const { return 64 * chunks; }
    // 16-deep instructions of each part in chunk c
    __host__ __device__ int deep(int c, int rank) const
    {
        const int left = rank - c * chunk;
        return ((left < chunk ? left : chunk) + 15) / 16;
    }
};
inline LoraParts lora_parts(int rank, int parts, int dtype)
{
    const int chunk = rank <= 16 || parts == 3 ? 16 : 32;
    return {parts, chunk, (rank + chunk - 1) / chunk, dtype == DT_F16 ? 2 : parts};
}

// Eight rank values in parts: store(part, its eight values).
template <typename T, typename Store>
__device__ __forceinline__ void each_part(float (&left)[8], const LoraParts& lay, Store store)
{
#pragma unroll 1
    for (int part = 0; part < lay.parts; ++part) {
        T h[8];
        if (part == lay.plain) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                left[i] *= LT_FINE;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            put(&h[i], left[i]);
            const float f = to_f32(h[i]);
            left[i] = isfinite(f) ? left[i] - f : 0.0f;  // an infinity has no remainder
        }
        uint4 w;
        memcpy(&w, h, 16);
        store(part, w);
    }
}

}  // namespace tmmo
