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
// bound by the tensor pipe: 4096 x 4096 BF16 takes 1.01 ms for five steps,
// 1360 TFLOP/s, where whole waves of tiles would take 0.73 (the two symmetric
// products run 136 tiles of 256 x 256 in two waves of 76 pairs, the update
// 256 in four).  Small ones are bound by the latency of a product, about
// 5.5 us whatever its size (0.95 from the end of one grid to the start of
// the next, 1.45 to the first operands, 1 to 2 of MMAs, 0.6 to 1.1 of
// epilogue): 8 x 1000 x 200 takes 104 us.
//
// Numbers.  A singular value may start at 1e-4 of the norm and grow by
// a factor of 3.4 a step, and so do rounding errors in its direction, so
// plain 16-bit storage loses the small directions: against 64 bits, BF16
// throughout is off by 1-3 % for matrices with a flat spectrum and up to
// 18 % for a few strong directions over a noise floor, FP16 by 0.2-2 %.
// Here X is kept as a pair of FP16 values (hi + lo, 22 bits) along the path
// a X, which is where small directions grow, and the products take FP16
// operands: B acts only on directions in which A = X X^T is not small, so
// the operand's rounding is not amplified.  Simulated, 0.2 % or less for
// every spectrum tried, about BF16's own rounding.  FP16 rather than BF16
// for its three more bits at the same rate; power-of-two scales (NS_SX,
// NS_SA, NS_SB) keep its range away from subnormals: entries of X up to
// 16 in magnitude, A up to 16, B up to 32, with 24 binary orders below.
// All sums (norm, products, a X + B X) are FP32.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "launch.h"
#include "newton_schulz.cuh"
#include "newton_schulz.h"

namespace tmmo {
namespace {

constexpr int kMaxDevices = 64;

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
    // pitches of the FP16 addend and output; X's low half has X's
    long long ld_add, batch_add;
    __half* lo;                    // X's low half, read as part of the addend and written
    long long ld_out, batch_out;
    void* result;                  // NS_LAST
    long long ld_res, batch_res;
    bool vec_res;                  // its rows are on 16-byte boundaries
    int out_dtype;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

// What differs from step to step: acc * alpha + beta * add -> out.
struct NsOperands {
    float alpha, beta;
    const __half* add;
    __half* out;
};

// One orthogonalisation: the products' parameters by mode (an update's serve
// its last step as well) and where the operands are.
struct NsPlan {
    NsParams p[3];
    __half *hi[2], *A, *B;         // X (read from one, written to the other), A, B
    float coefficients[3 * NS_MAX_STEPS];
};

__host__ __device__ inline NsOperands ns_operands(const NsPlan& f, int mode, int step)
{
    const float a = f.coefficients[3 * step], b = f.coefficients[3 * step + 1],
                c = f.coefficients[3 * step + 2];
    switch (mode) {
    case NS_GRAM:
        return {NS_SA / (NS_SX * NS_SX), 0.0f, nullptr, f.A};
    case NS_POLY:
        return {c * (NS_SB / (NS_SA * NS_SA)), b * (NS_SB / NS_SA), f.A, f.B};
    default:
        return {1.0f / NS_SB, a, f.hi[step & 1], f.hi[(step & 1) ^ 1]};
    }
}

// The last product of a call stages its output, which need not be aligned; the
// others leave that shared memory to the L1 cache, through which the addends
// come (with it, 8 x 545 x 552 took 1.1 times as long).
template <int CG, int BN, int STAGES, bool STAGED>
struct NsLayout {
    static constexpr int STAGE = 2 * NS_BOX;
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

// 32 FP16 values of one row, `n` of them inside the matrix.  Rows start on
// 32-byte boundaries and are padded to whole 16-value groups.
__device__ __forceinline__ void ns_load_row(const __half* src, int n, uint32_t (&w)[16])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (8 * i < n)
            u = *reinterpret_cast<const uint4*>(src + 8 * i);
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
    }
}

__device__ __forceinline__ void ns_store_row(__half* dst, int n, const uint32_t (&w)[16])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (16 * i < n) {
            uint32_t u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                u[k] = w[8 * i + k];
            st_global_v8(dst + 16 * i, u);
        }
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
template <int MODE, int COLS, typename Wait>
__device__ __forceinline__ void ns_epilogue(const NsParams& p, const NsOperands& o, int z, bool mirror,
                                            int row, int col0, uint32_t taddr, uint32_t stg, Wait&& wait)
{
    const bool inside = row < p.M;
    const long long at_add = z * p.batch_add + row * p.ld_add + col0;
    uint32_t ah[2][16], al[2][16];
    auto fetch = [&](int c, int b) {  // the addend of chunk c
        const int n = inside ? p.N - col0 - c * 32 : 0;
        if constexpr (MODE != NS_GRAM)
            ns_load_row(o.add + at_add + c * 32, n, ah[b]);
        if constexpr (MODE >= NS_UPDATE)
            ns_load_row(p.lo + at_add + c * 32, n, al[b]);
    };
    fetch(0, 0);
    fetch(1, 1);
    if (!wait())
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
        for (int i = 0; i < 16; ++i) {
            f[2 * i] = o.alpha * __uint_as_float(v[2 * i]);
            f[2 * i + 1] = o.alpha * __uint_as_float(v[2 * i + 1]);
            if constexpr (MODE != NS_GRAM) {
                float2 a = ns_unpack(ah[b][i]);
                if constexpr (MODE >= NS_UPDATE) {
                    const float2 l = ns_unpack(al[b][i]);
                    a.x = fmaf(l.x, 1.0f / NS_LO, a.x);
                    a.y = fmaf(l.y, 1.0f / NS_LO, a.y);
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
        } else {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i] = ns_pack(f[2 * i], f[2 * i + 1]);
            const long long at = z * p.batch_out + row * p.ld_out + col;
            if (inside)
                ns_store_row(o.out + at, n, w);
            if constexpr (MODE == NS_UPDATE) {
                uint32_t lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 h = ns_unpack(w[i]);
                    lo[i] = ns_pack((f[2 * i] - h.x) * NS_LO, (f[2 * i + 1] - h.y) * NS_LO);
                }
                if (inside)
                    ns_store_row(p.lo + at, n, lo);
            } else if (mirror) {
                // the mirrored tile: lane l writes column `row` of the rows
                // col .. col + 31
                unsigned short* dst = reinterpret_cast<unsigned short*>(o.out) + z * p.batch_out +
                                      col * p.ld_out + row;
                if (inside) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (i < n)
                            dst[i * p.ld_out] = static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1)));
                    }
                }
            }
        }
    }
}

// One product of the iteration over a batch.  Roles and barriers as in
// tc_gemm_kernel: a persistent grid, TMA into a ring of 128-byte-swizzled
// boxes, tcgen05 into two accumulators in tensor memory so that a tile's
// epilogue overlaps the next tile's main loop, every wait bounded.
template <int CG, int BN, int STAGES, int MODE>
__global__ void __launch_bounds__(NS_THREADS, 1)
    ns_product_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB, const NsParams p,
                      const NsOperands o)
{
    using L = NsLayout<CG, BN, STAGES, MODE == NS_LAST>;
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
                        const uint32_t dA = sbase + stage * L::STAGE, dB = dA + NS_BOX;
                        const int k0 = kb * NS_BK;
                        // K-major: one box of 128 rows x 64 of K; MN-major:
                        // two boxes of 64 of K x 64 outer values.
                        auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y) {
                            if constexpr (CG == 2)
                                tma_load_3d_pair(dst, map, fb, x, y, z);
                            else
                                tma_load_3d(dst, map, fb, x, y, z);
                        };
                        if (p.a_mn) {
                            load(dA, &tmA, a_row, k0);
                            load(dA + NS_BOX / 2, &tmA, a_row + 64, k0);
                        } else {
                            load(dA, &tmA, k0, a_row);
                        }
                        if (p.b_mn) {
                            load(dB, &tmB, b_row, k0);
                            load(dB + NS_BOX / 2, &tmB, b_row + 64, k0);
                        } else {
                            load(dB, &tmB, k0, b_row);
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
                        for (int k = 0; k < NS_BK / TC_UMMA_K; ++k)
                            tc_mma_f16<CG>(d, a_hi | ((a0 + k * a_step) & 0x3FFF),
                                           b_hi | ((b0 + k * b_step) & 0x3FFF), p.idesc, kb != 0 || k != 0);
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
            ns_epilogue<MODE, COLS>(p, o, z, mb != nb, row, col0,
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
}

// ------------------------------------------------------------ normalisation

struct NsNorm {
    const void* G;
    long long ldg, batch_g;
    int rows, cols, groups;        // groups of 8 columns per row
    float* partial;                // [batch][blocks]
    double* wide;                  // the same, for the sums that FP32 does not hold
    int blocks;
    float eps;
    __half *hi, *lo;
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

// X = G / (norm + eps) as hi and lo over the same groups.
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
        for (int k = 0; k < 4; ++k) {
            const float x = v[2 * k] * factors.x * factors.y, y = v[2 * k + 1] * factors.x * factors.y;
            h[k] = ns_pack(x, y);
            const float2 r = ns_unpack(h[k]);
            l[k] = ns_pack((x - r.x) * NS_LO, (y - r.y) * NS_LO);
        }
        const long long at = z * p.batch_x + row * p.ld + c;
        *reinterpret_cast<uint4*>(p.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
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
    if (threadIdx.x == 0)
        p.partial[at] = s;
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

// Workspace: X hi twice (a product reads one and writes the other), X lo, A,
// B, partial sums.  Rows are padded to 16 values (32 bytes).
struct NsSpace {
    int64_t m, ld_x, ld_a;
    int64_t x, a;                   // elements of one matrix
    size_t off_hi[2], off_lo, off_a, off_b, off_partial, off_wide, bytes;
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
    s.off_hi[0] = take(batch * s.x * 2);
    s.off_hi[1] = take(batch * s.x * 2);
    s.off_lo = take(batch * s.x * 2);
    s.off_a = take(batch * s.a * 2);
    s.off_b = take(batch * s.a * 2);
    s.off_partial = take(batch * NS_NORM_BLOCKS * 4);
    s.off_wide = take(batch * NS_NORM_BLOCKS * 8);
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

template <int CG, int BN, int STAGES, int MODE>
cudaError_t ns_run(const CUtensorMap& ta, const CUtensorMap& tb, NsParams p, const NsOperands& o,
                   int num_sms, cudaStream_t stream)
{
    using L = NsLayout<CG, BN, STAGES, MODE == NS_LAST>;
    auto kern = ns_product_kernel<CG, BN, STAGES, MODE>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    static int max_units[kMaxDevices] = {};
    static std::mutex mu;
    int units_cap = 0;
    {
        std::lock_guard<std::mutex> g(mu);
        if (max_units[dev] == 0) {
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       L::SMEM_ALLOC);
            if (err != cudaSuccess)
                return err;
            int cap = num_sms;
            if (CG == 2) {
                cudaLaunchConfig_t cfg{};
                cudaLaunchAttribute attr[1];
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = 2;
                attr[0].val.clusterDim.y = 1;
                attr[0].val.clusterDim.z = 1;
                cfg.gridDim = dim3(2 * std::max(1, num_sms / 2), 1, 1);
                cfg.blockDim = dim3(NS_THREADS, 1, 1);
                cfg.dynamicSmemBytes = L::SMEM_ALLOC;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                int clusters = 0;
                err = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
                if (err != cudaSuccess)
                    return err;
                cap = std::max(1, clusters);
            }
            max_units[dev] = cap;
        }
        units_cap = max_units[dev];
    }
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
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(units * CG, 1, 1);
    cfg.blockDim = dim3(NS_THREADS, 1, 1);
    cfg.dynamicSmemBytes = L::SMEM_ALLOC;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    note_launch();
    err = cudaLaunchKernelEx(&cfg, kern, ta, tb, p, o);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// 256 x 256 pair tiles once they fill half of the CTA pairs, 128 x 128 tiles
// below that and where the pairs' last wave would be so empty that the smaller
// tiles need clearly fewer waves, a wave of pairs counted as two: by a factor
// of 1.4, or of 1.2 for a K of up to 512, where a tile's fixed costs outweigh
// its operands' traffic.  Measured on GB300, us, pairs / 128 x 128:
// 8 x 256 x 2400 193 / 158, 8 x 545 x 552 163 / 139, 8 x 300 x 1800 187 / 163,
// 3000 x 3000 598 / 552; not taken: 2300 x 2300 (a factor of 1.33) 375 / 390.
template <int MODE>
cudaError_t ns_product(const CUtensorMap& ta, const CUtensorMap& tb, const NsParams& p,
                       const NsOperands& o, int num_sms, cudaStream_t stream)
{
    const long long tm = (p.M + 255) / 256, tn = (p.N + 255) / 256;
    const bool symmetric = MODE == NS_GRAM || MODE == NS_POLY;
    const long long pairs = p.batch * (symmetric ? tn * (tn + 1) / 2 : tm * tn);
    constexpr int STAGES = MODE == NS_LAST ? 5 : 6;
    const long long m1 = (p.M + 127) / 128, n1 = (p.N + 127) / 128;
    const long long singles = p.batch * (symmetric ? n1 * (n1 + 1) / 2 : m1 * n1);
    const long long pair_waves = 2 * ((2 * pairs + num_sms - 1) / num_sms);
    const long long single_waves = (singles + num_sms - 1) / num_sms;
    const bool empty = single_waves * (p.K <= 512 ? 12 : 14) <= pair_waves * 10;
    if (pairs * 4 >= num_sms && !empty)
        return ns_run<2, 256, STAGES, MODE>(ta, tb, p, o, num_sms, stream);
    return ns_run<1, 128, STAGES, MODE>(ta, tb, p, o, num_sms, stream);
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
    NsPlan plan{};
    plan.hi[0] = reinterpret_cast<__half*>(ws + s.off_hi[0]);
    plan.hi[1] = reinterpret_cast<__half*>(ws + s.off_hi[1]);
    plan.A = reinterpret_cast<__half*>(ws + s.off_a);
    plan.B = reinterpret_cast<__half*>(ws + s.off_b);
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
        p.ld_add = p.ld_out = update ? s.ld_x : s.ld_a;
        p.batch_add = p.batch_out = update ? s.x : s.a;
        p.lo = reinterpret_cast<__half*>(ws + s.off_lo);
        p.result = l.O;
        p.ld_res = l.ldo;
        p.batch_res = l.batch_o;
        p.vec_res = ns_vec_rows(l);
        p.out_dtype = l.out_dtype;
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
    // one group of 8 values a thread, more from NS_NORM_BLOCKS blocks on (with
    // four: 1024^2 151 us in all instead of 143; with at most 64 blocks 4096^2
    // 1059 instead of 969)
    const int64_t groups = static_cast<int64_t>(l.rows) * n.groups;
    n.blocks = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(NS_NORM_BLOCKS, (groups + 511) / 512)));
    n.eps = l.eps;
    n.hi = plan.hi[0];
    n.lo = reinterpret_cast<__half*>(ws + s.off_lo);
    n.ld = s.ld_x;
    n.batch_x = s.x;

    // Tensor maps: X with K (128-row boxes) or the outer axis (64-row boxes)
    // contiguous, A and B.
    CUtensorMap x_rows[2], x_cols[2], ta, tb;
    for (int i = 0; i < 2; ++i)
        if (!ns_encode(&x_rows[i], plan.hi[i], l.rows, l.cols, s.ld_x, l.batch, s.x, 128) ||
            !ns_encode(&x_cols[i], plan.hi[i], l.rows, l.cols, s.ld_x, l.batch, s.x, 64))
            return cudaErrorNotSupported;
    if (!ns_encode(&ta, plan.A, m, m, s.ld_a, l.batch, s.a, 128) ||
        !ns_encode(&tb, plan.B, m, m, s.ld_a, l.batch, s.a, 128))
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
        const CUtensorMap& tx = tall ? x_cols[cur] : x_rows[cur];
        const CUtensorMap& t1 = tall ? x_rows[cur] : tb;
        const CUtensorMap& t2 = tall ? tb : x_cols[cur];
        if ((err = ns_product<NS_GRAM>(tx, tx, plan.p[NS_GRAM], gram, l.num_sms, stream)) != cudaSuccess ||
            (err = ns_product<NS_POLY>(ta, ta, plan.p[NS_POLY], poly, l.num_sms, stream)) != cudaSuccess)
            return err;
        err = i + 1 < l.steps
                  ? ns_product<NS_UPDATE>(t1, t2, plan.p[NS_UPDATE], update, l.num_sms, stream)
                  : ns_product<NS_LAST>(t1, t2, plan.p[NS_UPDATE], update, l.num_sms, stream);
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

}  // namespace tmmo
