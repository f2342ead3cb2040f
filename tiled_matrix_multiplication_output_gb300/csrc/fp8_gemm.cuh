// Block-scaled 8-bit matrix product on the 5th-generation tensor cores:
//
//   C[m, n] = alpha * sum_kb sA[m, kb] * sB[n, kb] * P_kb[m, n] + beta * C[m, n],
//   P_kb[m, n] = sum over the 128 k of block kb of a[m, k] * b[n, k],
//
// a and b in e4m3 or e5m2, the scales in FP32, one for each outer index (or
// for 128 of them) and K block.
//
// The scales are arbitrary FP32 numbers, so a K block's product has to be
// scaled before it joins the sum: P_kb is accumulated by the tensor core
// (FP32, in tensor memory), read back, and added to the running sum in
// registers, FP32, as acc += (sA * sB) * P_kb.  For a CTA pair's 256 x 256
// tile a K block is 512 cycles of MMA, against 128 x 256 values a CTA that
// have to cross from tensor memory and one multiply-add each, 256 cycles of
// the FP32 pipe.  So:
//
//   * eight epilogue warps, two per SM partition, hold the running sums: 128
//     registers a thread for 256-column tiles.  setmaxnreg moves registers
//     from the copying and issuing warps to them.  (Sixteen warps with half
//     the columns took 1.16 times the time.);
//   * several partial buffers in tensor memory (512 columns in all), so the
//     tensor core works on the next K blocks while one is promoted; a pair's
//     K block is issued as two groups of 128 columns with barriers of their
//     own, so that its first half is promoted during the second's MMAs;
//   * multiply-adds in pairs (fma.rn.f32x2), half the instructions;
//   * little synchronisation on the critical path, where every K block waits
//     on it twice.  A herald warp polls the mbarriers for the epilogue and
//     releases it through a hardware barrier (a poll costs some 300 cycles,
//     a barrier that the herald has reached about 40); the arrivals that
//     free a buffer carry no memory ordering; the MMA warp runs a uniform
//     loop with an elected issuer, which keeps descriptors in uniform
//     registers; one commit a group serves copies and epilogue.  Together
//     these took 8192 x 8192 x 16384 from 2055 us to 780;
//   * one warp copies the scales of each K block into a ring in shared
//     memory, twelve K blocks ahead (asynchronous 4-byte copies, which take
//     any alignment).  Loads by the epilogue warps themselves, two K blocks
//     ahead, waited for the memory system: 1.2 times the time.
//
// What bounds it.  Measured on GB300, BF16 out, one vector of scales and one
// of tiles: 8192 x 8192 x 4096 200 us (198 to 214 by card; 2.7 PFLOP/s, 0.72 of
// twice the measured 16-bit burst rate), x 16384 771 us (2.9).  A K block takes 714
// cycles at the 1.8 GHz that the chip holds at this power: the shared memory
// of an SM moves 80 KiB for it (32 written by TMA, A read once a group, B
// once), 640 cycles.  A tile's end, when the sums go out and the MMAs wait
// for free buffers, adds about 3000.  With two vectors of scales a thread
// needs the scales of all its columns, 256 broadcast loads a K block and one
// multiplication more a value: 1200 cycles (4096 x 4096 x 8192 141 to
// 156 us against 106 to 113).  There the FP32 pipe and the registers' read ports count for
// most: a packed multiplication and a multiply-add of three different
// operands take 5.3 cycles (one with a shared factor 2.7), 680 a K block and
// partition; without any load of scales it would still be 1130.
//
// Waves.  A last wave that would fill at most half of the CTA pairs has its
// tiles split into parts of 128 columns, one group of MMAs a K block, which
// all epilogue warps share; a pair has at most one, after its whole tiles.
//
// One K step is one 128-byte swizzle row: a 128 x 128 block of either
// operand is 16 KiB, one TMA box, whether K or the outer axis is contiguous
// in memory (K-major or MN-major operand), so the same stored bytes serve
// the forward product and both gradients.  TMA fills what lies outside the
// matrix with zeros, which add nothing.
//
// CG = 2 runs on a CTA pair (M = 256 MMAs, each CTA loading its 128 rows of A
// and half of B's columns), as tc_gemm_kernel does.  Every wait is bounded in
// the same way.
#pragma once

#include <type_traits>

#include "fp8.h"
#include "launch.h"
#include "ops.cuh"

namespace tmmo {

constexpr int F8_BK = 128;       // K per step and per scale block
constexpr int F8_THREADS = 384;  // warps 0-3: copies, MMA, scales, herald; 4-11: epilogue
constexpr int F8_EPI_WARP0 = 4;
constexpr int F8_EPI_WARPS = 8;
constexpr int F8_HERALD_BAR = 1;  // hardware barriers of the herald and the epilogue warps
constexpr int F8_BOX = 128 * F8_BK;  // bytes of one operand box
// Registers: 384 threads are launched with 168 each (64,512 in all); the
// first warpgroup keeps 72 and the two epilogue warpgroups get 216 each:
// 128 * 72 + 256 * 216 = 64,512.
constexpr int F8_REGS_LAUNCH = 168;
constexpr int F8_REGS_FEW = 72;
constexpr int F8_REGS_EPI = 216;
static_assert(128 * F8_REGS_FEW + 256 * F8_REGS_EPI <= F8_THREADS * F8_REGS_LAUNCH, "register split");

struct Fp8Params {
    int M, N;
    int tiles_m, tiles_n;
    int whole;                     // tiles computed whole, an item each
    int items;                     // those and the parts: two for each further tile
    int k_blocks;
    int group_m;
    uint32_t idesc;
    bool a_mn, b_mn;               // operands stored with the outer axis contiguous
    const float *sa, *sb;          // scales, see Fp8Operand
    long long sa_k, sa_o, sb_k, sb_o;
    int sa_shift, sb_shift;
    void* C;
    long long ldc;
    int out_dtype;                 // DT_*
    bool tma_out;                  // the output goes through a tensor map (beta == 0)
    float alpha, beta;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

template <int CG, int BN, int STAGES>
struct Fp8Layout {
    static constexpr int STAGE = 2 * F8_BOX;           // one box of A, one of B per CTA
    static constexpr int NBUF = 512 / BN < 4 ? 512 / BN : 4;
    // Scale ring: per K block, 128 row scales and BN column scales (or two);
    // a slot, with one pair of barriers, holds GROUP K blocks.
    static constexpr int SLOTS = 3;
    static constexpr int GROUP = 4;
    static constexpr int BLOCK_BYTES = (128 + BN) * 4;
    static constexpr int SLOT_BYTES = GROUP * BLOCK_BYTES;
    // Two output buffers of 4 KiB per epilogue warp.
    static constexpr int OFF_STAGING = STAGES * STAGE;
    static constexpr int OFF_SCALE = OFF_STAGING + F8_EPI_WARPS * 2 * TC_STAGING_BYTES;
    static constexpr int OFF_BAR = OFF_SCALE + SLOTS * SLOT_BYTES;
    // A K block's MMAs are issued as SUB groups of BN / SUB columns, each
    // with its own barriers.
    static constexpr int SUB = CG;
    static constexpr int NUM_BARS = STAGES * (1 + SUB) + NBUF * SUB + 2 * SLOTS + 1;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NUM_BARS;
    static constexpr int BYTES = OFF_MISC + 16;
    static constexpr int SMEM_ALLOC = BYTES + 1024;
    static constexpr uint32_t TMEM_COLS = NBUF * BN;
    static_assert(BN / CG == 128, "each CTA holds 128 rows of B");
    static_assert(SMEM_ALLOC <= 232448, "exceeds 227 KiB of dynamic shared memory");
};

// Instruction descriptor of tcgen05.mma kind::f8f6f4: as kind::f16, with the
// types e4m3 = 0 and e5m2 = 1.
__host__ __device__ constexpr uint32_t fp8_idesc(int a_type, int b_type, int m, int n, bool a_mn,
                                                 bool b_mn)
{
    return (1u << 4) | (static_cast<uint32_t>(a_type) << 7) | (static_cast<uint32_t>(b_type) << 10) |
           ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The constant part of an operand box's shared-memory descriptor: offsets,
// version, and the swizzle mode (128, 64 or 32 bytes, the length of a row).
__device__ __forceinline__ uint64_t fp8_desc_hi(uint32_t row_bytes, bool mn)
{
    const uint64_t lbo = mn ? F8_BOX : 16, sbo = 8 * row_bytes;
    return ((lbo >> 4) << 16) | ((sbo >> 4) << 32) | (1ull << 46) |
           (static_cast<uint64_t>(row_bytes == 128 ? 2 : row_bytes == 64 ? 4 : 6) << 61);
}

template <typename OutT>
__device__ __forceinline__ OutT fp8_to_out(float v)
{
    if constexpr (sizeof(OutT) == 4)
        return v;
    else if constexpr (std::is_same<OutT, __half>::value)
        return __float2half_rn(v);
    else
        return __float2bfloat16_rn(v);
}

// A warp's 32 x COLS part of a finished tile through its staging buffer, in
// strips of 32 rows x 128 bytes: swizzled, conflict-free stores to shared
// memory and one TMA store each, which clips at C's edges.  Straight from
// registers, a thread holding a row, the stores scatter over 32 lines each.
template <typename OutT, int COLS>
__device__ __forceinline__ void fp8_store_tile(const uint64_t (&acc)[COLS / 2], uint32_t stg,
                                               const CUtensorMap* map, int row0, int col0, uint32_t lane,
                                               const Fp8Params& p)
{
    constexpr int STRIP = TcOut<OutT>::STRIP;
    const uint32_t sw = lane & 7;
#pragma unroll
    for (int s = 0; s < COLS / STRIP; ++s) {
        if (row0 >= p.M || col0 + s * STRIP >= p.N)
            break;
        // Two buffers in turn.  Both are free at a tile's first strip (the
        // last tile's left long before); later the strip before the last has
        // to have left this one.
        if (lane == 0) {
            if (s == 0)
                bulk_wait_group_read<0>();
            else
                bulk_wait_group_read<1>();
        }
        __syncwarp();
        const uint32_t buf = stg + (s & 1) * TC_STAGING_BYTES, base = buf + lane * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // 16-byte chunks
            uint32_t w[4];
            if constexpr (sizeof(OutT) == 4) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    unpack_f32x2(acc[s * 16 + c * 2 + i], w[2 * i], w[2 * i + 1]);
                if (p.alpha != 1.0f) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = __float_as_uint(p.alpha * __uint_as_float(w[i]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t lo, hi;
                    unpack_f32x2(acc[s * 32 + c * 4 + i], lo, hi);
                    w[i] = pack2(p.alpha * __uint_as_float(lo), p.alpha * __uint_as_float(hi),
                                 static_cast<OutT*>(nullptr));
                }
            }
            st_shared_v4(base + ((c ^ sw) << 4), w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(map, buf, col0 + s * STRIP, row0);
            bulk_commit_group();
        }
    }
}

// The same for an output without a tensor map (rows that are not 16-byte
// aligned, or beta != 0): strips of 32 FP32 columns, stored and, for beta,
// read a row at a time, a column a lane.  A thread writing its own row
// element by element took ten times as long.
template <typename OutT, int COLS>
__device__ __forceinline__ void fp8_store_rows(const uint64_t (&acc)[COLS / 2], uint32_t stg, int row0,
                                               int col0, uint32_t lane, const Fp8Params& p)
{
    const uint32_t base = stg + lane * 128, sw = lane & 7;
    const int rows = min(p.M - row0, 32);
#pragma unroll
    for (int s = 0; s < COLS / 32; ++s) {
        if (rows <= 0 || col0 + s * 32 >= p.N)
            break;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t w[4];
            unpack_f32x2(acc[s * 16 + 2 * c], w[0], w[1]);
            unpack_f32x2(acc[s * 16 + 2 * c + 1], w[2], w[3]);
            st_shared_v4(base + ((c ^ sw) << 4), w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        const int col = col0 + s * 32 + static_cast<int>(lane);
        if (col < p.N) {
            OutT* c = static_cast<OutT*>(p.C) + static_cast<long long>(row0) * p.ldc + col;
#pragma unroll 8
            for (int r = 0; r < rows; ++r, c += p.ldc) {
                float v = p.alpha * ld_shared_f32(stg + r * 128 + ((((lane >> 2) ^ (r & 7)) << 4) |
                                                                  ((lane & 3) << 2)));
                if (p.beta != 0.0f)
                    v = fmaf(p.beta, out_to_f32(*c), v);
                *c = fp8_to_out<OutT>(v);
            }
        }
    }
}

// COLV: the column operand has a scale for each column (a vector along the
// tile's columns); otherwise one for 128 columns, the same for all of a
// thread's columns.
template <int CG, int BN, int STAGES, bool COLV>
__global__ void __launch_bounds__(F8_THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmC, const Fp8Params p)
{
    using L = Fp8Layout<CG, BN, STAGES>;
    constexpr int TILE_M = TC_BM * CG;
    constexpr int NBUF = L::NBUF;
    constexpr int SUB = L::SUB;
    constexpr int COLS = BN / 2;  // columns of the tile per epilogue thread
    constexpr int HERALD_THREADS = 32 * (F8_EPI_WARPS / SUB + 1);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::OFF_BAR;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    // Group j of the MMAs on stage s has completed (and with the last group
    // all of them): its product can be read, the stage overwritten.
    auto done_bar = [&](int s, int j) { return bar0 + 8u * (STAGES + s * SUB + j); };
    auto tempty_bar = [&](int b, int j) { return bar0 + 8u * (STAGES * (1 + SUB) + b * SUB + j); };
    const uint32_t sbar0 = bar0 + 8u * (STAGES * (1 + SUB) + NBUF * SUB);
    auto sfull_bar = [&](int i) { return sbar0 + 8u * i; };
    auto sempty_bar = [&](int i) { return sbar0 + 8u * (L::SLOTS + i); };
    const uint32_t drain_bar = sbar0 + 8u * (2 * L::SLOTS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);

    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = (CG == 2) ? cluster_ctarank() : 0;
    const bool leader = (rank == 0);
    const int unit = (CG == 2) ? (blockIdx.x >> 1) : blockIdx.x;
    const int num_units = (CG == 2) ? (gridDim.x >> 1) : gridDim.x;
    const TcWatch watch{abort_flag, p.status, p.wait_budget};
    // Item t: its tile, whether it is a part of one only, and the first of its
    // columns in the tile.  A unit has at most one part, its last item.
    auto item_coords = [&](int t, int& mb, int& nb, bool& part, int& first) {
        part = false;
        first = 0;
        if (SUB == 2 && t >= p.whole) {
            part = true;
            first = ((t - p.whole) & 1) * (BN / 2);
            t = p.whole + ((t - p.whole) >> 1);
        }
        const int per_group = p.group_m * p.tiles_n;
        const int g = t / per_group;
        const int first_m = g * p.group_m;
        const int gm = min(p.tiles_m - first_m, p.group_m);
        const int r = t - g * per_group;
        mb = first_m + r % gm;
        nb = r / gm;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            for (int j = 0; j < SUB; ++j)
                mbar_init(done_bar(s, j), 1);
        }
        for (int b = 0; b < NBUF; ++b)
            for (int j = 0; j < SUB; ++j)
                mbar_init(tempty_bar(b, j), F8_EPI_WARPS / SUB * CG);
        for (int i = 0; i < L::SLOTS; ++i) {
            mbar_init(sfull_bar(i), 32);
            mbar_init(sempty_bar(i), F8_EPI_WARPS);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if (p.tma_out)
            tma_prefetch_desc(&tmC);
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

    if (warp < F8_EPI_WARP0) {
        set_max_regs_dec<F8_REGS_FEW>();
        if (warp == 0 && lane == 0) {
            // -------------------------------------------- TMA producer
            int stage = 0;
            uint32_t phase = 0;
            int issued[STAGES];
#pragma unroll
            for (int s = 0; s < STAGES; ++s)
                issued[s] = 0;
            bool ok = true;
            for (int t = unit; ok && t < p.items; t += num_units) {
                int mb, nb, first;
                bool part;
                item_coords(t, mb, nb, part, first);
                const int a_row = mb * TILE_M + static_cast<int>(rank) * TC_BM;
                // Group j of the columns takes 128 / SUB rows of B from each CTA.
                const int b_row = nb * BN + first + static_cast<int>(rank) * (128 / SUB);
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (!tc_wait(done_bar(stage, SUB - 1), phase ^ 1, watch)) {
                        ok = false;
                        break;
                    }
                    if (p.fault_skip_kblock != kb) {  // test hook, -1 in normal use
                        if (leader)
                            mbar_arrive_expect_tx(full_bar(stage),
                                                  CG * (part ? F8_BOX + F8_BOX / SUB : L::STAGE));
                        const uint32_t fb = (CG == 2) ? mapa_shared(full_bar(stage), 0) : full_bar(stage);
                        const uint32_t dA = sbase + stage * L::STAGE;
                        auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y) {
                            if constexpr (CG == 2)
                                tma_load_2d_pair(dst, map, fb, x, y);
                            else
                                tma_load_2d(dst, map, fb, x, y);
                        };
                        const int k0 = kb * F8_BK;
                        if (p.a_mn)
                            load(dA, &tmA, a_row, k0);
                        else
                            load(dA, &tmA, k0, a_row);
#pragma unroll
                        for (int j = 0; j < SUB; ++j) {
                            if (part && j > 0)
                                break;
                            const uint32_t dB = dA + F8_BOX + j * (F8_BOX / SUB);
                            const int o = b_row + j * 128;
                            if (p.b_mn)
                                load(dB, &tmB, o, k0);
                            else
                                load(dB, &tmB, k0, o);
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
                // Drain (bounded): the copies already issued into each stage
                // land before shared memory goes away.
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
        } else if (warp == 1 && leader) {
            // -------------------------------------------- MMA issuer
            // The whole warp runs the loop and one elected lane issues: the
            // descriptors then live in uniform registers, where the
            // instruction takes them from.
            // Descriptor of a 32-wide K slice of an operand box.  K-major:
            // 128-byte rows, 8-row groups 1024 bytes apart, 32 bytes along
            // the row per slice.  MN-major: a row holds the box's 128 (or,
            // in groups, 64) outer values, one swizzle atom of as many
            // bytes, so the leading offset is unused; 8-row K groups follow
            // each other, 32 rows per slice.
            constexpr uint32_t B_ROW = 128 / SUB;  // bytes of an MN-major row of B
            const uint64_t a_hi = fp8_desc_hi(128, p.a_mn);
            const uint64_t b_hi = fp8_desc_hi(p.b_mn ? B_ROW : 128, p.b_mn);
            const uint32_t a_step = (p.a_mn ? 32 * 128 : 32) >> 4;
            const uint32_t b_step = (p.b_mn ? 32 * B_ROW : 32) >> 4;
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool ok = true;
            // The K loop of an item.  PART: one group, issued when both halves of
            // the buffer are free, and shared by all epilogue warps.
            auto issue_item = [&](auto is_part) {
                constexpr bool PART = decltype(is_part)::value;
#pragma unroll 1
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    ok = tc_wait_warp(full_bar(stage), phase, watch);
                    const uint32_t a0 = (sbase + stage * L::STAGE) >> 4;
                    const uint32_t b0 = a0 + (F8_BOX >> 4);
                    const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
#pragma unroll
                    for (int j = 0; j < SUB; ++j) {
                        ok = ok && tc_wait_warp(tempty_bar(buf, j), buf_phase ^ 1, watch);
                        if (!ok)
                            break;
                        if (PART && j + 1 < SUB)
                            continue;
                        const int g = PART ? 0 : j;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < F8_BK / 32; ++k)
                                tc_mma_f8<CG>(d + g * (BN / SUB), a_hi | ((a0 + k * a_step) & 0x3FFF),
                                              b_hi | ((b0 + g * (F8_BOX / SUB >> 4) + k * b_step) & 0x3FFF),
                                              p.idesc, k != 0);
#pragma unroll
                            for (int i = g; i <= j; ++i) {
                                if constexpr (CG == 2)
                                    tc_commit_pair(done_bar(stage, i), 0x3);
                                else
                                    tc_commit(done_bar(stage, i));
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok)
                        break;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                    if (++buf == NBUF) {
                        buf = 0;
                        buf_phase ^= 1;
                    }
                }
            };
            for (int t = unit; ok && t < p.items; t += num_units) {
                if (SUB == 2 && t >= p.whole)
                    issue_item(std::true_type{});
                else
                    issue_item(std::false_type{});
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
        } else if (warp == 2) {
            // -------------------------------------------- scales
            int slot = 0;
            uint32_t slot_phase = 0;
            bool ok = true;
            for (int t = unit; ok && t < p.items; t += num_units) {
                int mb, nb, first;
                bool part;
                item_coords(t, mb, nb, part, first);
                // Rows and columns beyond the matrix take the last one's
                // scale (their products are never stored).
                const int row0 = mb * TILE_M + static_cast<int>(rank) * TC_BM + static_cast<int>(lane);
                const int col0 = nb * BN + static_cast<int>(lane) * (COLV ? 1 : COLS);
                const float* ra[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ra[i] = p.sa + (static_cast<long long>(min(row0 + 32 * i, p.M - 1)) >> p.sa_shift) *
                                       p.sa_o;
                constexpr int NC = COLV ? BN / 32 : 1;
                const float* cb[NC];
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    cb[i] = p.sb + (static_cast<long long>(min(col0 + 32 * i, p.N - 1)) >> p.sb_shift) *
                                       p.sb_o;
                for (int kb0 = 0; kb0 < p.k_blocks; kb0 += L::GROUP) {
                    int w = 1;
                    if (lane == 0)
                        w = tc_wait(sempty_bar(slot), slot_phase ^ 1, watch) ? 1 : 0;
                    if (!__shfl_sync(0xffffffffu, w, 0)) {
                        ok = false;
                        break;
                    }
                    uint32_t dst = sbase + L::OFF_SCALE + slot * L::SLOT_BYTES + lane * 4;
                    const int kb1 = min(kb0 + L::GROUP, p.k_blocks);
#pragma unroll 1
                    for (int kb = kb0; kb < kb1; ++kb, dst += L::BLOCK_BYTES) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            cp_async_4(dst + 128 * i, ra[i] + kb * p.sa_k);
                        if (COLV || lane < 2) {
#pragma unroll
                            for (int i = 0; i < NC; ++i)
                                cp_async_4(dst + 512 + 128 * i, cb[i] + kb * p.sb_k);
                        }
                    }
                    cp_async_mbar_arrive(sfull_bar(slot));
                    if (++slot == L::SLOTS) {
                        slot = 0;
                        slot_phase ^= 1;
                    }
                }
            }
            cp_async_wait_all();
        } else if (warp == 3) {
            // -------------------------------------------- herald
            // Waits on the barriers of each K block for the epilogue warps and
            // lets them go on through a hardware barrier.  After a wait that
            // ran out it goes through the barriers without waiting, so that
            // every warp reaches the end.
            int stage = 0, slot = 0;
            uint32_t phase = 0, slot_phase = 0;
            bool ok = true;
            for (int t = unit; t < p.items; t += num_units) {
#pragma unroll 1
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    if (kb % L::GROUP == 0) {
                        ok = ok && tc_wait_warp(sfull_bar(slot), slot_phase, watch);
                        if (++slot == L::SLOTS) {
                            slot = 0;
                            slot_phase ^= 1;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < SUB; ++j) {
                        ok = ok && tc_wait_warp(done_bar(stage, j), phase, watch);
                        bar_sync(F8_HERALD_BAR + j, HERALD_THREADS);
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------ promotion, epilogue
        set_max_regs_inc<F8_REGS_EPI>();
        const int ew = warp - F8_EPI_WARP0;
        const int q = warp & 3;        // TMEM lane quarter
        const int half = ew >> 2;      // column half of the tile
        const int group = SUB == 2 ? half : 0;  // the MMA group that fills this warp's columns
        const uint32_t tempty0 =
            (CG == 2) ? mapa_shared(tempty_bar(0, group), 0) : tempty_bar(0, group);
        int buf = 0, slot = 0;
        // Item t, WIDTH columns a warp.  (Whole tiles have a loop of their own,
        // which a choice in it makes 1 to 3 % slower; so has the MMA warp, 5 %.)
        auto run_item = [&](auto width, int t) {
            constexpr int WIDTH = decltype(width)::value;
            const uint32_t t_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                    static_cast<uint32_t>(half * WIDTH);
            // the warp's first column in the tile
            const int cfirst = half * WIDTH + (WIDTH < COLS ? ((t - p.whole) & 1) * (BN / 2) : 0);
            int mb, nb, first;
            bool part;
            item_coords(t, mb, nb, part, first);
            const int row0 = mb * TILE_M + static_cast<int>(rank) * TC_BM + q * 32;
            const int col0 = nb * BN + first + half * WIDTH;
            uint64_t acc[WIDTH / 2];
#pragma unroll
            for (int i = 0; i < WIDTH / 2; ++i)
                acc[i] = 0;
            // Tensor memory is read in chunks of 32 columns, each load issued
            // before the arithmetic of the chunk before it, across K blocks
            // as well: the next block's first chunk and scales are fetched
            // before the last chunk's arithmetic.
            constexpr int NCH = WIDTH / 32;
            uint32_t v[2][32];
            float rs = 0.0f;
            uint32_t caddr = 0;
            auto begin = [&](int kb) {
                bar_sync(F8_HERALD_BAR + group, HERALD_THREADS);
                tc_fence_after();
                tmem_ld_32x32b_x32(t_base + static_cast<uint32_t>(buf * BN), v[0]);
                const uint32_t saddr =
                    sbase + L::OFF_SCALE + slot * L::SLOT_BYTES + (kb % L::GROUP) * L::BLOCK_BYTES;
                caddr = saddr + 512 + (COLV ? cfirst : cfirst / COLS) * 4;
                rs = ld_shared_f32(saddr + (q * 32 + lane) * 4);
                if constexpr (!COLV)
                    rs *= ld_shared_f32(caddr);
            };
            begin(0);
#pragma unroll 1
            for (int kb = 0; kb < p.k_blocks; ++kb) {
                const uint64_t rs2 = pack_f32x2(__float_as_uint(rs), __float_as_uint(rs));
                const uint32_t taddr = t_base + static_cast<uint32_t>(buf * BN);
                const bool more = kb + 1 < p.k_blocks;
                const bool slot_end = (kb + 1) % L::GROUP == 0 || !more;
                const uint32_t sempty = sempty_bar(slot);
                // the block has been read: its partial buffer may be refilled
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 2)
                            mbar_arrive_cluster_relaxed(tempty0 + 8u * SUB * buf);
                        else
                            mbar_arrive(tempty0 + 8u * SUB * buf);
                    }
                    if (++buf == NBUF)
                        buf = 0;
                    if (slot_end && ++slot == L::SLOTS)
                        slot = 0;
                };
                if constexpr (COLV) {
                    const uint32_t cols = caddr;
                    // The products of the scales are formed while the chunk
                    // is on its way from tensor memory, in the registers of a
                    // second chunk.
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        uint64_t f[16];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            uint32_t w[4];
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                         : "r"(cols + (c * 32 + 2 * i) * 4));
                            f[i] = fmul2(rs2, pack_f32x2(w[0], w[1]));
                            f[i + 1] = fmul2(rs2, pack_f32x2(w[2], w[3]));
                        }
                        tmem_wait_ld(v[0]);
                        if (c + 1 == NCH)
                            release();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            ffma2(acc[c * 16 + i], pack_f32x2(v[0][2 * i], v[0][2 * i + 1]), f[i]);
                        if (c + 1 < NCH)
                            tmem_ld_32x32b_x32(taddr + (c + 1) * 32, v[0]);
                        else if (more)
                            begin(kb + 1);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < NCH; ++c) {
                        tmem_wait_ld(v[c & 1]);
                        if (c + 1 < NCH) {
                            tmem_ld_32x32b_x32(taddr + (c + 1) * 32, v[(c + 1) & 1]);
                        } else {
                            release();
                            if (more)
                                begin(kb + 1);
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            ffma2(acc[c * 16 + i], pack_f32x2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), rs2);
                    }
                }
                if (slot_end) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(sempty);
                }
            }
            const bool stored = !*abort_flag;  // an unfinished tile is not written
            // ---- the finished tile: alpha, beta, rounding to the output type
            const uint32_t stg = sbase + L::OFF_STAGING + ew * 2 * TC_STAGING_BYTES;
            if (stored && p.tma_out) {
                if (p.out_dtype == DT_F32)
                    fp8_store_tile<float, WIDTH>(acc, stg, &tmC, row0, col0, lane, p);
                else if (p.out_dtype == DT_F16)
                    fp8_store_tile<__half, WIDTH>(acc, stg, &tmC, row0, col0, lane, p);
                else
                    fp8_store_tile<__nv_bfloat16, WIDTH>(acc, stg, &tmC, row0, col0, lane, p);
            } else if (stored) {
                if (p.out_dtype == DT_F32)
                    fp8_store_rows<float, WIDTH>(acc, stg, row0, col0, lane, p);
                else if (p.out_dtype == DT_F16)
                    fp8_store_rows<__half, WIDTH>(acc, stg, row0, col0, lane, p);
                else
                    fp8_store_rows<__nv_bfloat16, WIDTH>(acc, stg, row0, col0, lane, p);
            }
        };
        int t = unit;
        for (; t < p.whole; t += num_units)
            run_item(std::integral_constant<int, COLS>{}, t);
        if (SUB == 2 && t < p.items)
            run_item(std::integral_constant<int, COLS / SUB>{}, t);
    }

    // ---------------------------------------------------- teardown
    if (warp >= F8_EPI_WARP0 && lane == 0)
        bulk_wait_group_read<0>();  // the output copies have read shared memory
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

}  // namespace tmmo
