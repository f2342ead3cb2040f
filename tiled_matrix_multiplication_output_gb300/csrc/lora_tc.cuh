// Low-rank adapters on the tensor cores: what the kernels share.
//
// The rows of a 128-row tile may have different adapters.  One matrix
// instruction multiplies all 128 rows by one adapter's factor, and its mask of
// lanes keeps the result away from the rows of others: their accumulators are
// not touched, whatever the factor holds.  A tile's plan lists its adapters,
// ascending, with the rows of each.
//
// The rank values t are FP32 sums that enter a second product as operands of 16
// bits, in BF16 parts, which have FP32's range: t = p0 + p1 (+ p2), each the rounding
// of what the ones before leave, multiplied by the same factor.  Two parts hold 16
// bits, three 24.  A matrix instruction takes both operands in one type: a factor
// in FP16 is split in shared memory into two BF16 values, which hold all of
// its 11 bits.  (FP16 parts would lose what is below 2^-25, 1e-6 of a young
// adapter's gradients being 3 % off, and turn what is above 65504 into infinities.)
//
// The gradients multiply rank values by rows instead, which in FP16 are not worth
// splitting: there the parts are FP16, each to a scale and with an accumulator of its own:
// t = 2^22 h0 + 2^11 h1 + h2 + 2^-20 h3, from 2^-45 to 2.7e11.
//
// Parts lie in chunks of `chunk` rank values, 64 columns (128 bytes, a swizzle row) a
// chunk: part p of value j at column (j / chunk) * 64 + p * chunk + j % chunk.
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
constexpr int LT_F16_PARTS = 4;

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

// 32 lanes x 16 columns of 32 bits to tensor memory, and the wait for such stores.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// K steps that one accumulator adds up, at most: 64 instructions (see grouped_tc.cuh).
// Where a CTA has more, the accumulators are added to FP32 sums, with rounding, and begin
// anew; the sums lie in tensor memory.
constexpr int LT_SEGMENT = 16;

// Adds `chains` accumulators of cols columns (a multiple of 16), one behind the other from
// acc, to the sums of this warp's lanes: of those lanes that are mine, whose first addition
// it may be.
__device__ __forceinline__ void add_to_sums(uint32_t acc, int chains, uint32_t sums, int cols, bool first,
                                            bool mine)
{
#pragma unroll 1
    for (int j = 0; j < cols; j += 16) {
        uint32_t v[16], o[16];
        tmem_ld_32x32b_x16(acc + j, v);
        tmem_wait_ld(v);
#pragma unroll 1
        for (int c = 1; c < chains; ++c) {
            tmem_ld_32x32b_x16(acc + c * cols + j, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(o[i]));
        }
        tmem_ld_32x32b_x16(sums + j, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (!first)
                v[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(v[i]));
            v[i] = mine ? v[i] : o[i];
        }
        tmem_st_32x32b_x16(sums + j, v);
    }
    tmem_wait_st();
}

// How the rank values are laid out.
struct LoraParts {
    int parts, chunk, chunks;
    __host__ __device__ int columns() const { return 64 * chunks; }
    // 16-deep instructions of each part in chunk c
    __host__ __device__ int deep(int c, int rank) const
    {
        const int left = rank - c * chunk;
        return ((left < chunk ? left : chunk) + 15) / 16;
    }
};
inline LoraParts lora_parts(int rank, int parts)
{
    const int chunk = rank <= 16 || parts > 2 ? 16 : 32;
    return {parts, chunk, (rank + chunk - 1) / chunk};
}

// The rounding of eight values; what it leaves of them stays.
template <typename T>
__device__ __forceinline__ uint4 take_part(float (&left)[8])
{
    T h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        put(&h[i], left[i]);
        const float f = to_f32(h[i]);
        left[i] = isfinite(f) ? left[i] - f : 0.0f;  // an infinity has no remainder
    }
    uint4 w;
    memcpy(&w, h, 16);
    return w;
}

// Eight rank values in BF16 parts: store(part, its eight values).
template <typename Store>
__device__ __forceinline__ void each_part(float (&left)[8], int parts, Store store)
{
#pragma unroll 1
    for (int part = 0; part < parts; ++part)
        store(part, take_part<__nv_bfloat16>(left));
}

// What an FP16 part counts for.
__device__ __forceinline__ float f16_part_scale(int part)
{
    return part == 0 ? 0x1p22f : part == 1 ? 0x1p11f : part == 2 ? 1.0f : 0x1p-20f;
}
// The same in FP16 parts, for the gradients.  A part of 2^11 or 2^22 takes what is too
// large to leave less than 2^-5 to the parts of 1 and of 2^-20: rank values below 2^7 have
// the last two, those below 2^26 two or three, 23 bits at least.
template <typename Store>
__device__ __forceinline__ void each_f16_part(float (&left)[8], Store store)
{
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        const float least = part == 0 ? 0x1p26f : 0x1p7f, scale = f16_part_scale(part);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = fabsf(left[i]) >= least ? left[i] * (1.0f / scale) : 0.0f;
        float rest[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            rest[i] = v[i];
        store(part, take_part<__half>(rest));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            left[i] = v[i] != 0.0f ? rest[i] * scale : left[i];
    }
    store(2, take_part<__half>(left));
#pragma unroll
    for (int i = 0; i < 8; ++i)  // (more is left of rank values above 2^19 alone: 2^-23 of them at most)
        left[i] = fabsf(left[i]) <= 0x1p-5f ? left[i] * 0x1p20f : 0.0f;
    store(3, take_part<__half>(left));
}

// Eight FP16 values at `at` in shared memory as pairs of BF16 ones: the first of each in
// their place, the second at `rest`.
__device__ __forceinline__ void split_eight(uint32_t at, uint32_t rest)
{
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(at)
                 : "memory");
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t first[4], second[4];
    __nv_bfloat16* const tag = nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 h;
        memcpy(&h, &in[i], 4);
        const float2 f = __half22float2(h);
        first[i] = pack2(f.x, f.y, tag);
        second[i] = pack2(f.x - __uint_as_float(first[i] << 16), f.y - __uint_as_float(first[i] & 0xffff0000u), tag);
    }
    st_shared_v4(at, first[0], first[1], first[2], first[3]);
    st_shared_v4(rest, second[0], second[1], second[2], second[3]);
}

// Splits a factor's tile of one chunk (16 rank values), a whole warp's work.  K-major: n
// rows of 64 or 128 bytes, swizzled over them; the second values lie in the 16 columns
// behind the first.
__device__ __forceinline__ void split_rows(uint32_t tile, int n, uint32_t width)
{
#pragma unroll 8
    for (int i = lane_id(); i < 2 * n; i += 32) {
        const uint32_t r = i >> 1, u = i & 1, turn = width == 128 ? r & 7 : (r >> 1) & 3;
        const uint32_t row = tile + r * width;
        split_eight(row + ((u ^ turn) << 4), row + (((u + 2) ^ turn) << 4));
    }
}
// Across: boxes of 64 outputs, a row of 128 bytes for each rank value; the second values
// lie in the 16 rows behind the first (with the same swizzle).
__device__ __forceinline__ void split_across(uint32_t tile, int boxes)
{
#pragma unroll 8
    for (int i = lane_id(); i < 128 * boxes; i += 32) {
        const uint32_t at = tile + (i >> 7) * 8192 + (i & 127) * 16;
        split_eight(at, at + 2048);
    }
}

// The products of a chunk's parts: multiply(part, pair, k) for each 16-deep instruction,
// pair being 1 for the second values of a factor in two (of which the third part's
// product is below 2^-24 of the sum).
template <typename Multiply>
__device__ __forceinline__ void each_product(const LoraParts& lay, int deep, bool split, Multiply multiply)
{
    for (int part = 0; part < lay.parts; ++part)
        for (int pair = 0; pair <= static_cast<int>(split && part < 2); ++pair)
            for (int k = 0; k < deep; ++k)
                multiply(part, pair, k);
}

}  // namespace tmmo
