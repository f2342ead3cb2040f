// Orthogonalisation of a matrix (or a batch of them) by Newton-Schulz
// products, the step that turns a gradient's running mean into the update of
// the Muon optimiser:
//
//     X <- G / (|G|_F + eps)
//     `steps` times:  A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// on the side that is shorter (A = X^T X and X <- a X + X B for a matrix
// with more rows than columns), so A and B are m x m with m = min(rows,
// cols).  The polynomial a s + b s^3 + c s^5 is applied to every singular
// value s; the vectors stay.
//
// Work: with n = max(rows, cols), a step is m^2 n + m^3 + 2 m^2 n operations:
// A and A A are symmetric, so only tiles on and above the diagonal are
// computed and each is written twice, once mirrored.  Nothing is transposed
// in memory: the tensor core takes X with either axis contiguous.
//
// Matrices with a short side of up to 128 are held on chip by a cluster, in
// one launch (ns_resident.cu).  For the others every product is a launch,
// and the launches are programmatic dependents of each other.  Large ones are
// bound by the tensor pipe: 4096 x 4096 BF16 takes 1.09 ms for five steps (1.04
// in shorter runs, before the power cap sets in), 1260 TFLOP/s, where whole
// waves of tiles would take 0.73 (the two symmetric products run 136 tiles of
// 256 x 256 in two waves of 76 pairs, the update 256 in four).  Small ones are
// bound by the latency of a product, about 5.5 us whatever its size (0.95 from
// the end of one grid to the start of the next, 1.45 to the first operands, 1
// to 2 of MMAs, 0.6 to 1.1 of epilogue): 8 x 1000 x 200 takes 104 us.  With
// operands of two halves (FP32 results) 4096 x 4096 takes 2.8 ms,
// 8 x 1000 x 200 163 us.
//
// Numbers.  A singular value may start at 1e-4 of the norm and grow by
// a factor of 3.4 a step, and so do rounding errors in its direction, so
// plain 16-bit storage loses the small directions: against 64 bits, BF16
// throughout is off by 1-3 % for matrices with a flat spectrum and up to
// 18 % for a few strong directions over a noise floor, FP16 by 0.2-2 %.
// Here X is kept in FP32, which is where small directions grow (along a X),
// and only the products' operands are FP16: B acts only on directions in which
// A = X X^T is not small, so an operand's rounding is not amplified.  How many
// bits the operands have goes by what the result can show:
//
//   * BF16 results: one FP16 value an element (A, which is also added, B, and
//     X as an operand).  At most 2e-3 off exact arithmetic for every spectrum
//     tried, 1.3e-3 for a few strong directions over a noise floor, before the
//     result's own rounding, which is 1.66e-3 over all elements;
//   * FP32 and FP16 results, and those with a short side of up to 128, where
//     one value would be up to 7e-3 off: two FP16 values, hi + lo, 22 bits, and
//     three products (hi hi + hi lo + lo hi) in one accumulator, for three
//     times the MMAs.  1e-6 to 5e-5 off for sides of up to 4096, growing with
//     the length of the contractions, whose sums the tensor core truncates to
//     FP32 every 16 of K.
//     The next rounding down, TF32, has FP16's ten bits at half its rate.
//
// FP16 rather than BF16 for its three more bits at the same rate;
// power-of-two scales (NS_SX, NS_SA, NS_SB) keep its range away from
// subnormals: entries of X up to 16 in magnitude, A up to 16, B up to 32, with
// 24 binary orders below.  All sums (norm, products, a X + B X) are FP32.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "newton_schulz.cuh"
#include "newton_schulz.h"
#include "persistent.cuh"

namespace tmmo {
namespace {

constexpr int NS_THREADS = 320;   // warp 0: copies, 1: MMA, 2-9: epilogue
constexpr int NS_EPI_WARP0 = 2;
constexpr int NS_EPI_WARPS = 8;
constexpr int NS_BK = 64;
constexpr int NS_BOX = 128 * NS_BK * 2;  // bytes of one operand box per CTA
constexpr int NS_NORM_BLOCKS = 512;      // partial sums of squares per matrix, at most: one a thread

enum NsMode {
    NS_GRAM = 0,    // A = X X^T: symmetric
    NS_POLY = 1,    // B = b A + c A A: symmetric, addend A
    NS_UPDATE = 2,  // X' = a X + B X, stored as hi and lo
    NS_LAST = 3     // the same, stored as the result
};

struct NsParams {
    int batch, M, N, K;            // of one product
    int tiles_m, tiles_n, tiles;   // per matrix; symmetric: tiles on and above the diagonal
    int num_tiles;                 // all
    int k_blocks;
    bool a_mn, b_mn;
    uint32_t idesc;
    long long ld, batch_pitch;     // of the addend and of the output in the workspace
    float* x;                      // X in FP32, read as the addend and written (updates)
    void* result;                  // NS_LAST
    long long ld_res, batch_res;
    bool vec_res;                  // its rows are on 16-byte boundaries
    int out_dtype;
    int* gave_up;                  // set by a product that did not finish; then no result is stored
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

// An operand of a product, in one or two FP16 halves.
struct NsOperand {
    __half *hi, *lo;               // lo: the rest hi leaves (two halves)
};

// What differs from step to step: acc * alpha + beta * addend -> out.
struct NsOperands {
    float alpha, beta;
    NsOperand add;                 // of B = b A + c A A
    NsOperand out;
};

// One orthogonalisation: the products' parameters by mode (an update's serve
// its last step as well) and where the operands are.
struct NsPlan {
    NsParams p[3];
    NsOperand X[2], A, B;          // X: read from one, written to the other
    float coefficients[3 * NS_MAX_STEPS];
};

__host__ __device__ inline NsOperands ns_operands(const NsPlan& f, int mode, int step)
{
    const float a = f.coefficients[3 * step], b = f.coefficients[3 * step + 1],
                c = f.coefficients[3 * step + 2];
    switch (mode) {
    case NS_GRAM:
        return {NS_SA / (NS_SX * NS_SX), 0.0f, {}, f.A};
    case NS_POLY:
        return {c * (NS_SB / (NS_SA * NS_SA)), b * (NS_SB / NS_SA), f.A, f.B};
    default:
        return {1.0f / NS_SB, a, {}, f.X[(step & 1) ^ 1]};
    }
}

// The last product of a call stages its output, which need not be aligned; the
// others leave that shared memory to the L1 cache, through which the addends
// come (with it, 8 x 545 x 552 took 1.1 times as long).
template <int CG, int BN, bool SPLIT, bool STAGED>
struct NsLayout {
    static constexpr int STAGE = (SPLIT ? 4 : 2) * NS_BOX;  // A, B and with two halves A lo, B lo
    static constexpr int STAGES = SPLIT ? 3 : STAGED ? 5 : 6;
    static constexpr int OFF_STAGING = STAGES * STAGE;  // 4 KiB of output per epilogue warp
    static constexpr int OFF_BAR = OFF_STAGING + (STAGED ? NS_EPI_WARPS * TC_STAGING_BYTES : 0);
    static constexpr int NUM_BARS = 2 * STAGES + 5;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NUM_BARS;
    static constexpr int BYTES = OFF_MISC + 16;
    static constexpr int SMEM_ALLOC = BYTES + 1024;
    static constexpr uint32_t TMEM_COLS = 2 * BN;
    static_assert(BN / CG == 128, "each CTA holds 128 rows of B");
    static_assert(SMEM_ALLOC <= 232448, "exceeds 227 KiB of dynamic shared memory");
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Tile t of the batch: its matrix and block coordinates.  Symmetric products
// enumerate the blocks (i, j), i <= j, column by column of the triangle.
__device__ __forceinline__ void ns_tile(int t, const NsParams& p, bool symmetric, int& z, int& mb,
                                        int& nb)
{
    z = t / p.tiles;
    const int r = t - z * p.tiles;
    if (symmetric) {
        nb = static_cast<int>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
        while ((nb + 1) * (nb + 2) / 2 <= r)
            ++nb;
        while (nb * (nb + 1) / 2 > r)
            --nb;
        mb = r - nb * (nb + 1) / 2;
    } else {
        constexpr int GROUP = 8;
        const int per = GROUP * p.tiles_n;
        const int g = r / per;
        const int gm = min(p.tiles_m - g * GROUP, GROUP);
        const int s = r - g * per;
        mb = g * GROUP + s % gm;
        nb = s / gm;
    }
}

// 32 values of one row, FP16 (16 words) or FP32, `n` of them inside the matrix.
// Rows start on 32-byte boundaries and are padded to whole 16-value groups.
template <int WORDS>
__device__ __forceinline__ void ns_load_row(const void* src, int n, uint32_t (&w)[WORDS])
{
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (i * (128 / WORDS) < n)
            u = static_cast<const uint4*>(src)[i];
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
    }
}

template <int WORDS>
__device__ __forceinline__ void ns_store_row(void* dst, int n, const uint32_t (&w)[WORDS])
{
#pragma unroll
    for (int i = 0; i < WORDS / 8; ++i) {
        if (i * (256 / WORDS) < n) {
            uint32_t u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                u[k] = w[8 * i + k];
            st_global_v8(static_cast<uint32_t*>(dst) + 8 * i, u);
        }
    }
}

// Column `at` of `n` rows (pitch ld) from a row of FP16 values: the mirrored
// part of a symmetric product.
__device__ __forceinline__ void ns_store_column(__half* at, long long ld, int n, const uint32_t (&w)[16])
{
    unsigned short* dst = reinterpret_cast<unsigned short*>(at);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (i < n)
            dst[i * ld] = static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1)));
    }
}

// Descriptor constants of an operand box (128 outer x 64 of K).  K-major: one
// box of 128-byte rows; MN-major: two atoms of 64 outer values, 64 K rows of
// 128 bytes each.
__device__ __forceinline__ uint64_t ns_desc_hi(bool mn)
{
    return (1ull << 46) | (2ull << 61) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (static_cast<uint64_t>((mn ? NS_BOX / 2 : 16) >> 4) << 16);
}

// One warp's part of a finished tile: rows `row` (one a lane), COLS columns
// from col0 in chunks of 32.  The addend is fetched two chunks ahead, the
// first two before `wait`, which returns once the accumulator at taddr is
// complete (false: given up).
template <int MODE, int COLS, bool SPLIT, typename Wait>
__device__ __forceinline__ void ns_epilogue(const NsParams& p, const NsOperands& o, int z, bool mirror,
                                            int row, int col0, uint32_t taddr, uint32_t stg, Wait&& wait)
{
    const bool inside = row < p.M;
    const bool stored = MODE != NS_LAST || *p.gave_up == 0;  // (asked for ahead of the wait)
    const long long at0 = z * p.batch_pitch + row * p.ld + col0;
    uint32_t add[2][32];  // FP32; of A 16 words of hi, then of lo
    auto fetch = [&](int c, int b) {  // the addend of chunk c
        const int n = inside ? p.N - col0 - c * 32 : 0;
        const long long at = at0 + c * 32;
        if constexpr (MODE == NS_POLY) {
            uint32_t w[16];
            ns_load_row(o.add.hi + at, n, w);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                add[b][i] = w[i];
            if constexpr (SPLIT) {
                ns_load_row(o.add.lo + at, n, w);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    add[b][16 + i] = w[i];
            }
        } else if constexpr (MODE >= NS_UPDATE) {
            ns_load_row(p.x + at, n, add[b]);
        }
    };
    fetch(0, 0);
    fetch(1, 1);
    if (!wait() || !stored)
        return;
    tc_fence_after();
#pragma unroll 1
    for (int c0 = 0; c0 < COLS / 32; c0 += 2)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int c = c0 + b;
        const int col = col0 + c * 32;
        const int n = min(p.N - col, 32);
        if (n <= 0)
            break;
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c * 32, v);
        tmem_wait_ld(v);
        float f[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            f[i] = o.alpha * __uint_as_float(v[i]);
            if constexpr (MODE >= NS_UPDATE)
                f[i] = fmaf(o.beta, __uint_as_float(add[b][i]), f[i]);
        }
        if constexpr (MODE == NS_POLY) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float2 a = ns_unpack(add[b][i]);
                if constexpr (SPLIT) {
                    const float2 l = ns_unpack(add[b][16 + i]);
                    a.x += l.x;
                    a.y += l.y;
                }
                f[2 * i] = fmaf(o.beta, a.x, f[2 * i]);
                f[2 * i + 1] = fmaf(o.beta, a.y, f[2 * i + 1]);
            }
        }
        if (c + 2 < COLS / 32)
            fetch(c + 2, b);
        if constexpr (MODE == NS_LAST) {
            const uint32_t lane = threadIdx.x & 31;
            const int row0 = row - static_cast<int>(lane), rows = min(p.M - row0, 32);
            const long long at = z * p.batch_res + row0 * p.ld_res + col;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                f[i] *= 1.0f / NS_SX;
            if (p.out_dtype == DT_F32)
                ns_store_result(static_cast<float*>(p.result) + at, p.ld_res, rows, n, p.vec_res, stg, lane, f);
            else if (p.out_dtype == DT_F16)
                ns_store_result(static_cast<__half*>(p.result) + at, p.ld_res, rows, n, p.vec_res, stg, lane, f);
            else
                ns_store_result(static_cast<__nv_bfloat16*>(p.result) + at, p.ld_res, rows, n, p.vec_res, stg,
                                lane, f);
        } else if (inside) {
            const long long at = at0 + c * 32;
            // the mirrored tile: lane l writes column `row` of the rows col .. col + 31
            const long long at_mirror = z * p.batch_pitch + col * p.ld + row;
            if constexpr (MODE == NS_UPDATE) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] = __float_as_uint(f[i]);
                ns_store_row(p.x + at, n, v);
            }
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i] = ns_pack(f[2 * i], f[2 * i + 1]);
            ns_store_row(o.out.hi + at, n, w);
            if (MODE != NS_UPDATE && mirror)
                ns_store_column(o.out.hi + at_mirror, p.ld, n, w);
            if constexpr (SPLIT) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 h = ns_unpack(w[i]);
                    w[i] = ns_pack(f[2 * i] - h.x, f[2 * i + 1] - h.y);
                }
                ns_store_row(o.out.lo + at, n, w);
                if (MODE != NS_UPDATE && mirror)
                    ns_store_column(o.out.lo + at_mirror, p.ld, n, w);
            }
        }
    }
}

// One product of the iteration over a batch.  Roles and barriers as in
// tc_gemm_kernel: a persistent grid, TMA into a ring of 128-byte-swizzled
// boxes, tcgen05 into two accumulators in tensor memory so that a tile's
// epilogue overlaps the next tile's main loop, every wait bounded.
// SPLIT: operands of two halves, three products of halves into one
// accumulator (lo lo, 2^-22 of the whole, is left out).
template <int CG, int BN, int MODE, bool SPLIT>
__global__ void __launch_bounds__(NS_THREADS, 1)
    ns_product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmAlo, const __grid_constant__ CUtensorMap tmBlo,
                      const NsParams p, const NsOperands o)
{
    using L = NsLayout<CG, BN, SPLIT, MODE == NS_LAST>;
    constexpr int STAGES = L::STAGES;
    constexpr bool SYMMETRIC = MODE == NS_GRAM || MODE == NS_POLY;
    constexpr int TILE_M = TC_BM * CG;
    constexpr int COLS = BN / 2;  // columns of the tile per epilogue warp
    static_assert(!SYMMETRIC || TILE_M == BN, "mirrored tiles are square");

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::OFF_BAR;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);

    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = (CG == 2) ? cluster_ctarank() : 0;
    const bool leader = (rank == 0);
    const int unit = (CG == 2) ? (blockIdx.x >> 1) : blockIdx.x;
    const int num_units = (CG == 2) ? (gridDim.x >> 1) : gridDim.x;
    const TcWatch watch{abort_flag, p.status, p.wait_budget};
    // The next product's blocks may take the SMs that this one leaves idle
    // and set themselves up; they wait for this grid to complete before they
    // touch global memory.
    grid_dep_launch_dependents();

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), NS_EPI_WARPS * CG);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if constexpr (SPLIT) {
            tma_prefetch_desc(&tmAlo);
            tma_prefetch_desc(&tmBlo);
        }
    }
    if (warp == 1) {
        tmem_alloc<CG>(smem_u32(tmem_slot), L::TMEM_COLS);
        tmem_relinquish<CG>();
    }
    tc_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dep_wait();

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0;
            uint32_t phase = 0;
            int issued[STAGES];
#pragma unroll
            for (int s = 0; s < STAGES; ++s)
                issued[s] = 0;
            bool ok = true;
            for (int t = unit; ok && t < p.num_tiles; t += num_units) {
                int z, mb, nb;
                ns_tile(t, p, SYMMETRIC, z, mb, nb);
                const int a_row = mb * TILE_M + static_cast<int>(rank) * 128;
                const int b_row = nb * BN + static_cast<int>(rank) * 128;
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!tc_wait(empty_bar(stage), phase ^ 1, watch)) {
                        ok = false;
                        break;
                    }
                    if (p.fault_skip_kblock != kb) {  // test hook, -1 in normal use
                        if (leader)
                            mbar_arrive_expect_tx(full_bar(stage), CG * L::STAGE);
                        const uint32_t fb = (CG == 2) ? mapa_shared(full_bar(stage), 0) : full_bar(stage);
                        const uint32_t dst = sbase + stage * L::STAGE;
                        const int k0 = kb * NS_BK;
                        auto load = [&](uint32_t to, const CUtensorMap* map, int x, int y) {
                            if constexpr (CG == 2)
                                tma_load_3d_pair(to, map, fb, x, y, z);
                            else
                                tma_load_3d(to, map, fb, x, y, z);
                        };
                        // K-major: one box of 128 rows x 64 of K; MN-major:
                        // two boxes of 64 of K x 64 outer values.
                        auto load_box = [&](uint32_t to, const CUtensorMap* map, bool mn, int outer) {
                            if (mn) {
                                load(to, map, outer, k0);
                                load(to + NS_BOX / 2, map, outer + 64, k0);
                            } else {
                                load(to, map, k0, outer);
                            }
                        };
                        load_box(dst, &tmA, p.a_mn, a_row);
                        load_box(dst + NS_BOX, &tmB, p.b_mn, b_row);
                        if constexpr (SPLIT) {
                            load_box(dst + 2 * NS_BOX, &tmAlo, p.a_mn, a_row);
                            load_box(dst + 3 * NS_BOX, &tmBlo, p.b_mn, b_row);
                        }
#pragma unroll
                        for (int s = 0; s < STAGES; ++s)
                            issued[s] += (s == stage);
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok && leader) {
                // Drain (bounded): the copies already issued land before
                // shared memory goes away.
#pragma unroll
                for (int s = 0; s < STAGES; ++s) {
                    if (issued[s] == 0)
                        continue;
                    const uint32_t par = static_cast<uint32_t>(issued[s] - 1) & 1u;
                    const long long t0 = clock64();
                    while (!mbar_try_wait(full_bar(s), par) && clock64() - t0 < p.wait_budget) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // ------------------------------------------------ MMA issuer (a
            // uniform loop, one elected lane issues)
            int stage = 0, local = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint64_t a_hi = ns_desc_hi(p.a_mn), b_hi = ns_desc_hi(p.b_mn);
            const uint32_t a_step = (p.a_mn ? 2048 : 32) >> 4;
            const uint32_t b_step = (p.b_mn ? 2048 : 32) >> 4;
            for (int t = unit; ok && t < p.num_tiles; t += num_units, ++local) {
                const int acc = local & 1;
                ok = tc_wait_warp(tempty_bar(acc), ((local >> 1) & 1) ^ 1, watch);
                if (!ok)
                    break;
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
#pragma unroll 1
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    ok = tc_wait_warp(full_bar(stage), phase, watch);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t a0 = (sbase + stage * L::STAGE) >> 4;
                    const uint32_t b0 = a0 + (NS_BOX >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int part = 0; part < (SPLIT ? 3 : 1); ++part) {  // hi hi, hi lo, lo hi
                            const uint32_t a = a0 + (part == 2 ? 2 * NS_BOX >> 4 : 0);
                            const uint32_t b = b0 + (part == 1 ? 2 * NS_BOX >> 4 : 0);
#pragma unroll
                            for (int k = 0; k < NS_BK / TC_UMMA_K; ++k)
                                tc_mma_f16<CG>(d, a_hi | ((a + k * a_step) & 0x3FFF),
                                               b_hi | ((b + k * b_step) & 0x3FFF), p.idesc,
                                               kb != 0 || part != 0 || k != 0);
                        }
                        if constexpr (CG == 2)
                            tc_commit_pair(empty_bar(stage), 0x3);
                        else
                            tc_commit(empty_bar(stage));
                        if (kb + 1 == p.k_blocks) {
                            if constexpr (CG == 2)
                                tc_commit_pair(tfull_bar(acc), 0x3);
                            else
                                tc_commit(tfull_bar(acc));
                        }
                    }
                    __syncwarp();
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // every MMA issued has completed before TMEM is released (bounded)
            if (elect_one())
                tc_commit_self<CG>(drain_bar);
            __syncwarp();
            const long long t0 = clock64();
            while (!__all_sync(0xffffffffu, mbar_test_wait(drain_bar, 0))) {
                if (__any_sync(0xffffffffu, clock64() - t0 > p.wait_budget))
                    break;
            }
        }
    } else {
        // ---------------------------------------------------- epilogue
        const int q = warp & 3;  // TMEM lane quarter
        const int half = (warp - NS_EPI_WARP0) >> 2;
        const uint32_t tempty0 = (CG == 2) ? mapa_shared(tempty_bar(0), 0) : tempty_bar(0);
        int local = 0;
        for (int t = unit; t < p.num_tiles; t += num_units, ++local) {
            int z, mb, nb;
            ns_tile(t, p, SYMMETRIC, z, mb, nb);
            const int acc = local & 1;
            const int row = mb * TILE_M + static_cast<int>(rank) * TC_BM + q * 32 + static_cast<int>(lane);
            const int col0 = nb * BN + half * COLS;
            bool ok = true;
            ns_epilogue<MODE, COLS, SPLIT>(p, o, z, mb != nb, row, col0,
                                    tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                        static_cast<uint32_t>(acc * BN + half * COLS),
                                    sbase + L::OFF_STAGING + (warp - NS_EPI_WARP0) * TC_STAGING_BYTES,
                                    [&]() {
                                        ok = tc_wait_warp(tfull_bar(acc), (local >> 1) & 1, watch);
                                        return ok;
                                    });
            if (!ok)
                break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2)
                    mbar_arrive_cluster_relaxed(tempty0 + 8u * acc);
                else
                    mbar_arrive(tempty0 + 8u * acc);
            }
        }
    }

    // ---------------------------------------------------- teardown
    __syncwarp();
    tc_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<CG>(tmem_base, L::TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag)
        *p.gave_up = 1;
}

// ------------------------------------------------------------ normalisation

struct NsNorm {
    const void* G;
    long long ldg, batch_g;
    int rows, cols, groups;        // groups of 8 columns per row
    float* partial;                // [batch][blocks]
    double* wide;                  // the same, for the sums that FP32 does not hold
    int* gave_up;                  // cleared here
    int blocks;
    float eps;
    float* x;
    __half *hi, *lo;               // lo: null without split operands
    long long ld, batch_x;
};

// A thread's sum of squares, in FP32 or FP64, over the groups first, first +
// step, ... of matrix z.
template <typename InT, typename SumT>
__device__ __forceinline__ SumT ns_square_sum(const NsNorm& p, long long z, long long first,
                                               long long step)
{
    const InT* g = static_cast<const InT*>(p.G) + z * p.batch_g;
    const long long total = static_cast<long long>(p.rows) * p.groups;
    SumT s = 0;
    for (long long i = first; i < total; i += step) {
        const int row = static_cast<int>(i / p.groups), c = static_cast<int>(i % p.groups) * 8;
        float v[8];
        ns_load8(g + row * p.ldg + c, min(p.cols - c, 8), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const SumT x = v[k];
            s = fma(x, x, s);
        }
    }
    return s;
}

// X = G / (norm + eps) over the same groups, in FP32 and as an operand.
template <typename InT>
__device__ __forceinline__ void ns_scale(const NsNorm& p, long long z, long long first,
                                         long long step, float2 factors)
{
    const InT* g = static_cast<const InT*>(p.G) + z * p.batch_g;
    const long long total = static_cast<long long>(p.rows) * p.groups;
    for (long long i = first; i < total; i += step) {
        const int row = static_cast<int>(i / p.groups), c = static_cast<int>(i % p.groups) * 8;
        float v[8];
        ns_load8(g + row * p.ldg + c, min(p.cols - c, 8), v);
        uint32_t h[4], l[4];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = v[k] * factors.x * factors.y;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = ns_pack(v[2 * k], v[2 * k + 1]);
            const float2 r = ns_unpack(h[k]);
            l[k] = ns_pack(v[2 * k] - r.x, v[2 * k + 1] - r.y);
        }
        const long long at = z * p.batch_x + row * p.ld + c;
        float4* x = reinterpret_cast<float4*>(p.x + at);
        x[0] = make_float4(v[0], v[1], v[2], v[3]);
        x[1] = make_float4(v[4], v[5], v[6], v[7]);
        *reinterpret_cast<uint4*>(p.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
        if (p.lo)
            *reinterpret_cast<uint4*>(p.lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// Partial sums of squares, a fixed set of elements per block.
template <typename InT>
__global__ void __launch_bounds__(512) ns_norm_kernel(const NsNorm p)
{
    grid_dep_launch_dependents();
    grid_dep_wait();
    const long long first = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
    const long long at = static_cast<long long>(blockIdx.y) * p.blocks + blockIdx.x;
    const float s = ns_block_sum(ns_square_sum<InT, float>(p, blockIdx.y, first, step));
    if (threadIdx.x == 0) {
        p.partial[at] = s;
        if (at == 0)
            *p.gave_up = 0;
    }
    if (!ns_squares_fit(s)) {  // (the same for the whole block)
        const double wide = ns_block_sum(ns_square_sum<InT, double>(p, blockIdx.y, first, step));
        if (threadIdx.x == 0)
            p.wide[at] = wide;
    }
}

// Every block adds the partial sums in the same order.
template <typename InT>
__global__ void __launch_bounds__(512) ns_scale_kernel(const NsNorm p)
{
    grid_dep_launch_dependents();
    grid_dep_wait();
    const int i = static_cast<int>(threadIdx.x);
    const long long at = static_cast<long long>(blockIdx.y) * p.blocks + i;
    const float part = i < p.blocks ? p.partial[at] : 0.0f;
    const float sum = ns_block_sum(part);
    float2 factors;
    if (ns_squares_fit(sum)) {
        factors = ns_factors(sum, p.eps);
    } else {
        double wide = part;
        if (i < p.blocks && !ns_squares_fit(part))
            wide = p.wide[at];
        factors = ns_factors_wide(ns_block_sum(wide), p.eps);
    }
    const long long first = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    ns_scale<InT>(p, blockIdx.y, first, static_cast<long long>(gridDim.x) * blockDim.x, factors);
}

// ------------------------------------------------------------------- host

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Workspace: X in FP32, X as an operand twice (a product reads one and writes
// the other), A, B, each in two halves, and partial sums.  Rows are padded to
// 16 values (32 bytes of FP16).
struct NsSpace {
    int64_t m, ld_x, ld_a;
    int64_t x, a;                   // elements of one matrix
    size_t off_x, off_hi[2], off_lo[2], off_a[2], off_b[2], off_partial, off_wide, off_gave_up, bytes;
};

NsSpace ns_space(int64_t batch, int64_t rows, int64_t cols)
{
    NsSpace s{};
    s.m = std::min(rows, cols);
    s.ld_x = round_up(cols, 16);
    s.ld_a = round_up(s.m, 16);
    s.x = rows * s.ld_x;
    s.a = s.m * s.ld_a;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += static_cast<size_t>(round_up(bytes, 256));
        return here;
    };
    s.off_x = take(batch * s.x * 4);
    for (int i = 0; i < 2; ++i) {
        s.off_hi[i] = take(batch * s.x * 2);
        s.off_lo[i] = take(batch * s.x * 2);
        s.off_a[i] = take(batch * s.a * 2);
        s.off_b[i] = take(batch * s.a * 2);
    }
    s.off_partial = take(batch * NS_NORM_BLOCKS * 4);
    s.off_wide = take(batch * NS_NORM_BLOCKS * 8);
    s.off_gave_up = take(4);
    s.bytes = at;
    return s;
}

// A batch of FP16 matrices of rows x cols, in boxes of 64 columns x box_rows.
bool ns_encode(CUtensorMap* map, const __half* base, int64_t rows, int64_t cols, int64_t ld,
               int64_t batch, int64_t batch_pitch, uint32_t box_rows)
{
    auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2,
                                   static_cast<cuuint64_t>(batch_pitch) * 2};
    const cuuint32_t box[3] = {64, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensor maps of an operand's halves.
struct NsMaps {
    CUtensorMap hi, lo;
};

template <int CG, int BN, int MODE, bool SPLIT>
cudaError_t ns_run(const NsMaps& a, const NsMaps& b, NsParams p, const NsOperands& o, int num_sms,
                   cudaStream_t stream)
{
    using L = NsLayout<CG, BN, SPLIT, MODE == NS_LAST>;
    auto kern = ns_product_kernel<CG, BN, MODE, SPLIT>;
    static ClusterCaps caps;
    int units_cap = 0;
    const cudaError_t err = cluster_cap(kern, caps, CG, NS_THREADS, L::SMEM_ALLOC, num_sms, &units_cap);
    if (err != cudaSuccess)
        return err;
    p.tiles_m = (p.M + TC_BM * CG - 1) / (TC_BM * CG);
    p.tiles_n = (p.N + BN - 1) / BN;
    const bool symmetric = MODE == NS_GRAM || MODE == NS_POLY;
    const long long tiles = symmetric ? static_cast<long long>(p.tiles_n) * (p.tiles_n + 1) / 2
                                      : static_cast<long long>(p.tiles_m) * p.tiles_n;
    if (tiles * p.batch > 0x1fffffffLL)
        return cudaErrorNotSupported;
    p.tiles = static_cast<int>(tiles);
    p.num_tiles = static_cast<int>(tiles * p.batch);
    p.k_blocks = (p.K + NS_BK - 1) / NS_BK;
    p.idesc = tc_idesc(false, TC_BM * CG, BN, p.a_mn, p.b_mn);
    const int units = std::max(1, std::min(p.num_tiles, units_cap));
    ClusterLaunch launch(static_cast<unsigned>(units * CG), CG, NS_THREADS, L::SMEM_ALLOC, stream, true);
    return launch.run(kern, a.hi, b.hi, a.lo, b.lo, p, o);
}

// 256 x 256 pair tiles once they fill half of the CTA pairs, 128 x 128 tiles
// below that and where the pairs' last wave would be so empty that the smaller
// tiles need clearly fewer waves, a wave of pairs counted as two: by a factor
// of 1.4, or of 1.2 for a K of up to 512, where a tile's fixed costs outweigh
// its operands' traffic.  Measured on GB300, us, pairs / 128 x 128:
// 8 x 256 x 2400 193 / 158, 8 x 545 x 552 163 / 139, 8 x 300 x 1800 187 / 163,
// 3000 x 3000 598 / 552; not taken: 2300 x 2300 (a factor of 1.33) 375 / 390.
template <int MODE, bool SPLIT>
cudaError_t ns_product_tiles(const NsMaps& a, const NsMaps& b, const NsParams& p, const NsOperands& o,
                             int num_sms, cudaStream_t stream)
{
    const long long tm = (p.M + 255) / 256, tn = (p.N + 255) / 256;
    const bool symmetric = MODE == NS_GRAM || MODE == NS_POLY;
    const long long pairs = p.batch * (symmetric ? tn * (tn + 1) / 2 : tm * tn);
    const long long m1 = (p.M + 127) / 128, n1 = (p.N + 127) / 128;
    const long long singles = p.batch * (symmetric ? n1 * (n1 + 1) / 2 : m1 * n1);
    const long long pair_waves = 2 * ((2 * pairs + num_sms - 1) / num_sms);
    const long long single_waves = (singles + num_sms - 1) / num_sms;
    const bool empty = single_waves * (p.K <= 512 ? 12 : 14) <= pair_waves * 10;
    if (pairs * 4 >= num_sms && !empty)
        return ns_run<2, 256, MODE, SPLIT>(a, b, p, o, num_sms, stream);
    return ns_run<1, 128, MODE, SPLIT>(a, b, p, o, num_sms, stream);
}

template <int MODE>
cudaError_t ns_product(const NsMaps& a, const NsMaps& b, const NsParams& p, const NsOperands& o, bool split,
                       int num_sms, cudaStream_t stream)
{
    return split ? ns_product_tiles<MODE, true>(a, b, p, o, num_sms, stream)
                 : ns_product_tiles<MODE, false>(a, b, p, o, num_sms, stream);
}

template <typename InT>
cudaError_t ns_normalise(const NsNorm& n, int batch, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(n.blocks, batch);
    cfg.blockDim = dim3(512, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    note_launch();
    cudaError_t err = cudaLaunchKernelEx(&cfg, ns_norm_kernel<InT>, n);
    if (err != cudaSuccess)
        return err;
    note_launch();
    err = cudaLaunchKernelEx(&cfg, ns_scale_kernel<InT>, n);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

size_t ns_workspace_bytes(int64_t batch, int64_t rows, int64_t cols)
{
    return ns_space(batch, rows, cols).bytes;
}

cudaError_t ns_launch(const NsLaunch& l, cudaStream_t stream)
{
    if (ns_resident_takes(l))
        return ns_resident_launch(l, stream);
    const NsSpace s = ns_space(l.batch, l.rows, l.cols);
    char* ws = static_cast<char*>(l.workspace);
    const bool tall = l.rows > l.cols;
    const int m = static_cast<int>(s.m), wide = std::max(l.rows, l.cols);
    const bool split = ns_split(l);
    auto half = [&](size_t offset) { return reinterpret_cast<__half*>(ws + offset); };
    NsPlan plan{};
    for (int i = 0; i < 2; ++i)
        plan.X[i] = {half(s.off_hi[i]), half(s.off_lo[i])};
    plan.A = {half(s.off_a[0]), half(s.off_a[1])};
    plan.B = {half(s.off_b[0]), half(s.off_b[1])};
    std::copy(l.coefficients, l.coefficients + 3 * l.steps, plan.coefficients);
    for (int mode = 0; mode < 3; ++mode) {
        NsParams& p = plan.p[mode];
        const bool update = mode == NS_UPDATE;
        p.batch = l.batch;
        p.M = update ? l.rows : m;
        p.N = update ? l.cols : m;
        p.K = mode == NS_GRAM ? wide : m;
        p.a_mn = mode == NS_GRAM && tall;
        p.b_mn = mode == NS_GRAM ? tall : update && !tall;
        p.ld = update ? s.ld_x : s.ld_a;
        p.batch_pitch = update ? s.x : s.a;
        p.x = reinterpret_cast<float*>(ws + s.off_x);
        p.result = l.O;
        p.ld_res = l.ldo;
        p.batch_res = l.batch_o;
        p.vec_res = ns_vec_rows(l);
        p.out_dtype = l.out_dtype;
        p.gave_up = reinterpret_cast<int*>(ws + s.off_gave_up);
        p.status = l.status;
        p.wait_budget = l.wait_budget;
        p.fault_skip_kblock = l.fault_skip_kblock;
    }

    NsNorm n{};
    n.G = l.G;
    n.ldg = l.ldg;
    n.batch_g = l.batch_g;
    n.rows = l.rows;
    n.cols = l.cols;
    n.groups = (l.cols + 7) / 8;
    n.partial = reinterpret_cast<float*>(ws + s.off_partial);
    n.wide = reinterpret_cast<double*>(ws + s.off_wide);
    n.gave_up = reinterpret_cast<int*>(ws + s.off_gave_up);
    // one group of 8 values a thread, more from NS_NORM_BLOCKS blocks on (with
    // four: 1024^2 151 us in all instead of 143; with at most 64 blocks 4096^2
    // 1059 instead of 969; measured with X in two FP16 values)
    const int64_t groups = static_cast<int64_t>(l.rows) * n.groups;
    n.blocks = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(NS_NORM_BLOCKS, (groups + 511) / 512)));
    n.eps = l.eps;
    n.x = reinterpret_cast<float*>(ws + s.off_x);
    n.hi = plan.X[0].hi;
    n.lo = split ? plan.X[0].lo : nullptr;
    n.ld = s.ld_x;
    n.batch_x = s.x;

    // Tensor maps: X with K (128-row boxes) or the outer axis (64-row boxes)
    // contiguous, A and B.
    NsMaps x_rows[2], x_cols[2], ta, tb;
    auto encode = [&](NsMaps* maps, const NsOperand& o, int64_t rows, int64_t cols, int64_t ld, int64_t pitch,
                      uint32_t box_rows) {
        return ns_encode(&maps->hi, o.hi, rows, cols, ld, l.batch, pitch, box_rows) &&
               ns_encode(&maps->lo, o.lo, rows, cols, ld, l.batch, pitch, box_rows);
    };
    for (int i = 0; i < 2; ++i)
        if (!encode(&x_rows[i], plan.X[i], l.rows, l.cols, s.ld_x, s.x, 128) ||
            !encode(&x_cols[i], plan.X[i], l.rows, l.cols, s.ld_x, s.x, 64))
            return cudaErrorNotSupported;
    if (!encode(&ta, plan.A, m, m, s.ld_a, s.a, 128) || !encode(&tb, plan.B, m, m, s.ld_a, s.a, 128))
        return cudaErrorNotSupported;

    cudaError_t err = l.in_dtype == DT_F32   ? ns_normalise<float>(n, l.batch, stream)
                      : l.in_dtype == DT_F16 ? ns_normalise<__half>(n, l.batch, stream)
                                             : ns_normalise<__nv_bfloat16>(n, l.batch, stream);
    if (err != cudaSuccess)
        return err;
    for (int i = 0; i < l.steps; ++i) {
        const int cur = i & 1;
        const NsOperands gram = ns_operands(plan, NS_GRAM, i), poly = ns_operands(plan, NS_POLY, i),
                         update = ns_operands(plan, NS_UPDATE, i);
        const NsMaps& tx = tall ? x_cols[cur] : x_rows[cur];
        const NsMaps& t1 = tall ? x_rows[cur] : tb;
        const NsMaps& t2 = tall ? tb : x_cols[cur];
        const int sms = l.num_sms;
        if ((err = ns_product<NS_GRAM>(tx, tx, plan.p[NS_GRAM], gram, split, sms, stream)) != cudaSuccess ||
            (err = ns_product<NS_POLY>(ta, ta, plan.p[NS_POLY], poly, split, sms, stream)) != cudaSuccess)
            return err;
        err = i + 1 < l.steps ? ns_product<NS_UPDATE>(t1, t2, plan.p[NS_UPDATE], update, split, sms, stream)
                              : ns_product<NS_LAST>(t1, t2, plan.p[NS_UPDATE], update, split, sms, stream);
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

}  // namespace tmmo
