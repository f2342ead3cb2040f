// The row-grouped products on the 5th-generation tensor cores: one persistent
// kernel on CTA pairs (cta_group::2, M = 256) for the products and for their
// weight gradient.
//
// Products (GROUPED_T, GROUPED_N).  A group may have one row or thousands, so
// the rows are the tensor core's N side, which can be any multiple of 32 up to
// 256, and the weight's outputs are the 256 lanes of the pair: a tile of n rows
// costs n / 256 of a full one, and no tile is padded beyond 31 rows.
// (With the rows as lanes, groups of 200 rows would cost 256 each.)  A group's
// rows are cut into tiles of equal size.  The accumulator comes out
// transposed, lanes along the outputs, so that the 32 lanes of a warp store
// consecutive elements of a row of Y.
//
// Weight gradient (GROUPED_WGRAD).  D^T X of a group's rows: both operands lie
// across the contraction (MN-major), and the contraction is ragged.  The last
// 64 rows of a group hold rows of the next one; those among the last 16 that
// the tensor core reads are zeroed in shared memory by a warp of each CTA,
// in both operands (a zero against an infinity of another group would be a
// NaN), before they count as loaded.
//
// The tensor core drops what does not fit when it adds to its accumulator, half a unit in
// the last place an instruction on average (3e-6 of a sum over 2000 products of one
// sign, 3e-5 over 8000).  So every 768 rows of the gradient, every 1024 inputs of a
// product, the accumulator is added, with rounding, to sums in the epilogue warps'
// registers.
//
// Both are bound by the operands' way from L2 (a K step of a full tile takes 630
// cycles, its MMAs 512) or, with few rows, by reading the weights from HBM.  BF16, on the
// device, GPU not power-capped: 16384 rows of 16 groups by 4096 x 4096 319 us (1.72
// PFLOP/s; one accumulator for all of K 316), 256 rows of 64 groups by 4096 x 2048 153
// us (6.5 TB/s), the gradient of 16384 rows of 8 groups, 4096 x 2048, FP32, 180 us (1.53
// PFLOP/s).  Capped, the large ones take up to 370 and 205.
//
// Warps: 0 TMA producer, 1 MMA issuer (of the leader CTA), 2 for the gradient one that
// zeroes, 4 to 11 epilogue (with four, 4148 rows of 17 groups by 1360 x 152 took
// 13.7 us, with eight 12.4; 16384 of 16 by 4096 x 4096 300 and 303).  A ring of K
// steps, bounded waits and two accumulators in tensor memory, as in tc_gemm_kernel.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "grouped.cuh"
#include "ops.cuh"
#include "store_rows.cuh"
#include "warp_roles.cuh"

namespace tmmo {

enum { GROUPED_T = 0, GROUPED_N = 1, GROUPED_WGRAD = 2 };

constexpr int GT_RING = 192 * 1024;
constexpr int GT_MAX_STAGES = 10;
constexpr int GT_A_BYTES = TC_BM * TC_BK * 2;  // a K step of the lanes' side
constexpr int GT_N = 256;        // the N side of a full tile
constexpr int GT_SORTED = 256;   // groups, at most, that the gradient sorts
constexpr int GT_SEGMENT = 12;   // K steps of the gradient that one accumulator adds up
constexpr int GT_SEGMENT_PRODUCT = 16;  // the same of a product, at most

struct GroupedTcParams {
    Grouping by;
    void* C;              // Y, or the gradients
    int64_t ldc, stride_c;
    int N, K;             // outputs and inputs of a weight
    int segments, segment;  // products: how many parts of K, and their K steps
    int tiles_f, tiles_c; // 256-wide tiles of the lanes' axis; gradient: of the other one
    float alpha, beta;
    bool zero_rest;
    bool swap;            // the weights' map has its outer dimensions exchanged
    bool one_weight;
    int unit;             // row_unit of the output
    bool tma_out;         // gradient: stored by TMA
    uint32_t idesc;       // with N = 0
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

template <int MODE>
struct GroupedLayout {
    static constexpr bool WGRAD = MODE == GROUPED_WGRAD;
    static constexpr int EPI_WARPS = 8;
    static constexpr int EPI_WARP0 = 4;
    static constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
    // Of the 168 registers a thread that the block is launched with, the first warps
    // need few and the epilogue's sums many.
    static constexpr int REGS_FEW = 88, REGS_EPI = 208;
    static_assert(4 * REGS_FEW + EPI_WARPS * REGS_EPI <= (4 + EPI_WARPS) * 168, "of the block's registers");
    static constexpr int OFF_STAGING = GT_RING;
    static constexpr int STAGING = 2048;  // of an epilogue warp
    static constexpr int OFF_TABLE = OFF_STAGING + EPI_WARPS * STAGING;
    static constexpr int OFF_BAR = OFF_TABLE + (GroupTable::BYTES + 15) / 16 * 16;
    static constexpr int NUM_BARS = 2 * GT_MAX_STAGES + 5 + (WGRAD ? GT_MAX_STAGES : 0);
    static constexpr int OFF_MISC = OFF_BAR + 8 * NUM_BARS;
    static constexpr int BYTES = OFF_MISC + 16;
    static constexpr int SMEM_ALLOC = BYTES + 1024;
    static constexpr uint32_t TMEM_COLS = 2 * GT_N;
    static_assert(SMEM_ALLOC <= 232448, "exceeds 227 KiB of dynamic shared memory");
};

// One tile: its group, first lane-side index (of the pair), the other side's
// first index and extent (rounded up to what the tensor core takes), and the K
// steps.
struct GroupedWork {
    int g, f0, c0, count, n, k_blocks, row0, rows;
};

template <int MODE>
__device__ __forceinline__ GroupedWork grouped_work(int t, const GroupTable& table, const GroupedTcParams& p)
{
    GroupedWork w;
    if constexpr (MODE == GROUPED_WGRAD) {
        const int per = p.tiles_f * p.tiles_c;
        const int place = t / per;
        w.g = p.by.groups <= GT_SORTED ? table.tile[place] : place;
        const int u = t - place * per;
        w.f0 = u / p.tiles_c * 256;
        w.c0 = u % p.tiles_c * GT_N;
        w.count = min(GT_N, p.K - w.c0);
        w.n = w.count > 128 ? 256 : 128;
        w.row0 = table.first[w.g];
        w.rows = table.first[w.g + 1] - w.row0;
        w.k_blocks = (w.rows + TC_BK - 1) / TC_BK;
    } else {
        w.g = table.group_of(t / p.tiles_f, p.by.groups);
        const int tiles = table.tile[w.g + 1] - table.tile[w.g];
        const int begin = table.first[w.g], rows = table.first[w.g + 1] - begin;
        // (rounded up to 32; rows + tiles may not fit 32 bits)
        const int each = ((rows - 1) / tiles + 32) / 32 * 32;
        // row tiles eight at a time, and within those down the rows first: the
        // tiles that run together share weights and rows in L2
        int u = t - table.tile[w.g] * p.tiles_f;
        const int band = u / (8 * p.tiles_f) * 8;
        const int high = min(tiles - band, 8);
        u -= band * p.tiles_f;
        w.f0 = u / high * 256;
        w.c0 = begin + (band + u % high) * each;
        w.count = min(each, begin + rows - w.c0);
        w.n = (w.count + 31) / 32 * 32;
        w.row0 = 0;
        w.rows = 0;
        w.k_blocks = (p.K + TC_BK - 1) / TC_BK;
    }
    return w;
}

// How many rows a tile of the products has at most: what is quickest, by the waves
// of tiles on the pairs and the time of a tile.  A K step of n rows takes about
// 315 + 1.23 n cycles (630 at 256: operands from L2 set the pace).  5000 rows of 12
// groups by 1000 outputs are 104 tiles of 256 rows, two waves on 76 pairs, and 132
// of 192.  One warp calls it.
// largest: receives the rows that a tile then has at most.
__device__ __forceinline__ int tile_rows(const GroupTable& table, int groups, int tiles, int tiles_f,
                                         int pairs, int* largest)
{
    constexpr int KINDS = 5;  // 256, 224 .. 128 rows
    int best = GT_N;
    if (tiles * static_cast<int64_t>(tiles_f) > pairs) {  // (else smaller tiles win nothing)
        int n[KINDS] = {};
        for (int g = threadIdx.x; g < groups; g += 32) {
            const int rows = table.first[g + 1] - table.first[g];
#pragma unroll
            for (int k = 0; k < KINDS; ++k)
                n[k] += (rows + GT_N - 32 * k - 1) / (GT_N - 32 * k);
        }
        float least = 0.0f;
#pragma unroll
        for (int k = 0; k < KINDS; ++k) {
            const float work = static_cast<float>(__reduce_add_sync(0xffffffffu, n[k])) * tiles_f;
            const float time = ceilf(__fdividef(work, static_cast<float>(pairs))) * (315 + 1.23f * (GT_N - 32 * k));
            if (k == 0 || time < least) {
                best = GT_N - 32 * k;
                least = time;
            }
        }
    }
    int most = 0;
    for (int g = threadIdx.x; g < groups; g += 32)
        most = max(most, table.first[g + 1] - table.first[g]);
    most = __reduce_max_sync(0xffffffffu, min(most, best));
    if (threadIdx.x == 0)
        *largest = max(32, (most + 31) / 32 * 32);
    return best;
}

// Puts the groups into table.tile with the longest first (the gradient has no use
// for the tiles): the last tiles to start are then the short ones.  Every thread
// of the block calls it; it ends in a block barrier.
__device__ __forceinline__ void sort_groups(const GroupTable& table, int groups)
{
    for (int g = threadIdx.x; g < groups; g += blockDim.x) {
        const int rows = table.first[g + 1] - table.first[g];
        int place = 0;
        for (int h = 0; h < groups; ++h) {
            const int other = table.first[h + 1] - table.first[h];
            place += other > rows || (other == rows && h < g);
        }
        table.tile[place] = g;
    }
    __syncthreads();
}

template <int MODE, typename OutT>
__global__ void __launch_bounds__(GroupedLayout<MODE>::THREADS, 1)
    grouped_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmB64, const __grid_constant__ CUtensorMap tmB32,
                      const __grid_constant__ CUtensorMap tmB16, const __grid_constant__ CUtensorMap tmC,
                      const __grid_constant__ GroupedTcParams p)
{
    using L = GroupedLayout<MODE>;
    constexpr bool WGRAD = L::WGRAD;
    constexpr bool A_MN = MODE != GROUPED_T;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::OFF_BAR;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (GT_MAX_STAGES + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * GT_MAX_STAGES + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * GT_MAX_STAGES + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * GT_MAX_STAGES + 4);
    // gradient: a group's last K step lands on this CTA's own barrier first
    auto tail_bar = [&](int s) { return bar0 + 8u * (2 * GT_MAX_STAGES + 5 + s); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
    int* largest = reinterpret_cast<int*>(smem + L::OFF_MISC + 8);
    volatile int* progress = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 12);  // K steps copied

    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int unit = blockIdx.x >> 1, num_units = gridDim.x >> 1;
    const TcWatch watch{abort_flag, p.status, p.wait_budget};

    if (threadIdx.x == 32) {
        for (int s = 0; s < GT_MAX_STAGES; ++s) {
            // gradient: an arrival for each CTA, as either may have to zero
            mbar_init(full_bar(s), WGRAD ? 2 : 1);
            mbar_init(empty_bar(s), 1);
            if (WGRAD)
                mbar_init(tail_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 2 * L::EPI_WARPS);  // of the pair
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        *progress = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    // (the first warp makes the table meanwhile)
    const GroupTable table = load_groups(
        reinterpret_cast<int*>(smem + L::OFF_TABLE), p.by, WGRAD ? 0 : GT_N,
        [&](const GroupTable& t, int tiles) { return tile_rows(t, p.by.groups, tiles, p.tiles_f, num_units, largest); },
        [&] {
            if (warp == 1) {
                tmem_alloc<2>(smem_u32(tmem_slot), L::TMEM_COLS);
                tmem_relinquish<2>();
            }
        });
    if (WGRAD && p.by.groups <= GT_SORTED)
        sort_groups(table, p.by.groups);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // The ring: a stage is a K step of both operands, of as many rows as the
    // largest tile has, so that small tiles have more steps on their way.
    const int stage_bytes = GT_A_BYTES + (WGRAD ? GT_N : *largest) / 2 * TC_BK * 2;
    const int stages = min(GT_RING / stage_bytes, GT_MAX_STAGES);
    const int num_work = (WGRAD ? p.by.groups * p.tiles_c : table.tile[p.by.groups]) * p.tiles_f;
    // rows of a group's last K step that the tensor core reads beyond the group
    auto is_ragged = [&](const GroupedWork& w, int kb) {
        return WGRAD && kb == w.k_blocks - 1 && (w.rows & 15) != 0;
    };

    if (warp < L::EPI_WARP0) {
        set_max_regs_dec<L::REGS_FEW>();
        if (warp == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0, steps = 0;
            uint32_t phase = 0;
            uint32_t ragged = 0, ragged_parity = 0;  // of the stages' tail barriers: used, and how often
            bool ok = true;
            for (int t = unit; ok && t < num_work; t += num_units) {
                const GroupedWork w = grouped_work<MODE>(t, table, p);
                const int f = w.f0 + static_cast<int>(rank) * TC_BM;
                const int half = w.n / 2;
                const int c = w.c0 + static_cast<int>(rank) * half;
                const int z = p.one_weight ? 0 : w.g;
                const uint32_t bytes = GT_A_BYTES + half * TC_BK * 2;
                for (int kb = 0; kb < w.k_blocks; ++kb) {
                    ok = warp_wait(empty_bar(stage), phase ^ 1, watch);
                    if (!ok)
                        break;
                    const bool tail = is_ragged(w, kb);
                    ++steps;
                    if (WGRAD && lane == 0)
                        *progress = steps;
                    if (kb != p.fault_skip_kblock) {  // (test hook, -1 in normal use)
                        if (elect_one()) {
                            if (tail) {
                                mbar_arrive_expect_tx(tail_bar(stage), bytes);
                            } else if (leader) {
                                if (WGRAD)
                                    mbar_arrive(full_bar(stage));
                                mbar_arrive_expect_tx(full_bar(stage), 2 * bytes);
                            }
                            const uint32_t bar = tail ? mapa_shared(tail_bar(stage), rank)
                                                      : mapa_shared(full_bar(stage), 0);
                            const uint32_t dA = sbase + stage * stage_bytes, dB = dA + GT_A_BYTES;
                            if constexpr (WGRAD) {
                                const int row = w.row0 + kb * TC_BK;
                                tma_load_2d_pair(dA, &tmA, bar, f, row);
                                tma_load_2d_pair(dA + 8192, &tmA, bar, f + 64, row);
                                tma_load_2d_pair(dB, &tmB, bar, c, row);
                                if (half > 64)
                                    tma_load_2d_pair(dB + 8192, &tmB, bar, c + 64, row);
                            } else {
                                const int k = kb * TC_BK;
                                auto weights = [&](uint32_t dst, int x, int y) {
                                    tma_load_3d_pair(dst, &tmA, bar, x, p.swap ? z : y, p.swap ? y : z);
                                };
                                if (A_MN) {
                                    weights(dA, f, k);
                                    weights(dA + 8192, f + 64, k);
                                } else {
                                    weights(dA, k, f);
                                }
                                // the tile's rows in boxes of 128, 64, 32 and 16
                                if (half == 128) {
                                    tma_load_2d_pair(dB, &tmB, bar, k, c);
                                } else {
                                    int b = 0;
                                    if (half & 64) {
                                        tma_load_2d_pair(dB, &tmB64, bar, k, c);
                                        b = 64;
                                    }
                                    if (half & 32) {
                                        tma_load_2d_pair(dB + b * 128, &tmB32, bar, k, c + b);
                                        b += 32;
                                    }
                                    if (half & 16)
                                        tma_load_2d_pair(dB + b * 128, &tmB16, bar, k, c + b);
                                }
                            }
                        }
                        __syncwarp();
                        if (tail) {
                            ragged |= 1u << stage;
                            ragged_parity ^= 1u << stage;
                        }
                    }
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok && lane == 0) {
                // Wait (bounded) for the loads already issued before shared
                // memory goes away: the leader's barriers cover both CTAs.
                auto drain = [&](uint32_t bar, uint32_t parity) {
                    const long long t0 = clock64();
                    while (!mbar_try_wait(bar, parity) && clock64() - t0 < p.wait_budget) {
                    }
                };
                for (int s = 0; s < stages; ++s) {
                    const int uses = steps / stages + (s < steps % stages);
                    if (leader && uses > 0)
                        drain(full_bar(s), (uses - 1) & 1);
                    if (WGRAD && ((ragged >> s) & 1))
                        drain(tail_bar(s), ((ragged_parity >> s) & 1) ^ 1);
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issuer
            if (leader) {
                int stage = 0;
                uint32_t phase = 0;
                int local = 0;
                bool ok = true;
                for (int t = unit; ok && t < num_work; t += num_units) {
                    const GroupedWork w = grouped_work<MODE>(t, table, p);
                    if (w.k_blocks == 0)
                        continue;
                    const uint32_t idesc = p.idesc | static_cast<uint32_t>(w.n >> 3) << 17;
                    for (int kb = 0; ok && kb < w.k_blocks;) {  // by segments: a loop with one accumulator
                        ok = warp_wait<true>(tempty_bar(local & 1), ((local >> 1) & 1) ^ 1, watch);
                        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>((local & 1) * GT_N);
                        const int begin = kb, end = min(kb + (WGRAD ? GT_SEGMENT : p.segment), w.k_blocks);
                        for (; ok && kb < end; ++kb) {
                            ok = warp_wait<WGRAD>(full_bar(stage), phase, watch);
                            if (!ok)
                                break;
                            tc_fence_after();
                            const uint32_t a0 = sbase + stage * stage_bytes, b0 = a0 + GT_A_BYTES;
                            // 16-deep instructions; gradient: as many as there are rows
                            const int deep = WGRAD ? min(4, (w.rows - kb * TC_BK + 15) / 16) : 4;
                            if (elect_one()) {
#pragma unroll
                                for (int k = 0; k < TC_BK / TC_UMMA_K; ++k) {
                                    if (WGRAD && k >= deep)
                                        break;
                                    const uint64_t adesc = A_MN ? smem_desc_sw128(a0 + k * 2048, 8192, 1024)
                                                                : smem_desc_sw128(a0 + k * 32, 16, 1024);
                                    const uint64_t bdesc = WGRAD ? smem_desc_sw128(b0 + k * 2048, 8192, 1024)
                                                                 : smem_desc_sw128(b0 + k * 32, 16, 1024);
                                    tc_mma_f16<2>(d_tmem, adesc, bdesc, idesc, kb != begin || k != 0);
                                }
                                tc_commit_pair(empty_bar(stage), 0x3);
                                if (kb == end - 1)
                                    tc_commit_pair(tfull_bar(local & 1), 0x3);
                            }
                            __syncwarp();
                            if (++stage == stages) {
                                stage = 0;
                                phase ^= 1;
                            }
                        }
                        ++local;
                    }
                }
                // Wait (bounded) until every MMA issued so far has completed, so
                // TMEM and the input stages are no longer in use.
                if (elect_one())
                    tc_commit_self<2>(drain_bar);
                __syncwarp();
                const long long t0 = clock64();
                while (!mbar_try_wait(drain_bar, 0) && clock64() - t0 < p.wait_budget) {
                }
            }
        } else if (WGRAD && warp == 2) {
            // ------------------------- rows of other groups in a group's last K step
            int stage = 0;
            uint32_t parity = 0;  // a bit for each step's barrier
            for (int t = unit; t < num_work; t += num_units) {
                const GroupedWork w = grouped_work<MODE>(t, table, p);
                if (w.k_blocks == 0)
                    continue;
                const int last = w.k_blocks - 1;
                const int s = (stage + last) % stages;
                stage = (s + 1) % stages;
                if (!is_ragged(w, last))
                    continue;
                // (the steps before, of this tile and of ones that end evenly, are not waited for)
                if (!warp_wait_behind(tail_bar(s), (parity >> s) & 1, watch, progress))
                    break;
                parity ^= 1u << s;
                // a row of 64 values is 128 contiguous bytes (its swizzle stays within)
                const int from = w.rows - last * TC_BK, to = (from + 15) / 16 * 16;
                const int boxes = 2 + w.n / 128;
                for (int b = 0; b < boxes; ++b) {  // (A's two boxes, then B's)
                    const uint32_t box = sbase + s * stage_bytes + b * 8192;
                    for (int i = from * 8 + static_cast<int>(lane); i < to * 8; i += 32)
                        st_shared_v4(box + i * 16, 0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(mapa_shared(full_bar(s), 0));
            }
        }
    } else {
        set_max_regs_inc<L::REGS_EPI>();
        // ------------------------------------------------ epilogue
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const uint32_t leader_tempty0 = mapa_shared(tempty_bar(0), 0);
        const uint32_t leader_tempty1 = mapa_shared(tempty_bar(1), 0);
        OutT* const out = static_cast<OutT*>(p.C);
        const uint32_t staging = sbase + L::OFF_STAGING + (warp - L::EPI_WARP0) * L::STAGING;
        // waits for the next accumulator, of a segment; gives it back
        int local = 0;
        auto take = [&] {
            int ok = 1;
            if (lane == 0)
                ok = tc_wait(tfull_bar(local & 1), (local >> 1) & 1, watch) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            tc_fence_after();
            return ok != 0;
        };
        auto give = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(local & 1 ? leader_tempty1 : leader_tempty0);
            ++local;
        };
        const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        if constexpr (!WGRAD) {
            if (p.zero_rest)
                zero_rest_rows(table, p.by, out, p.ldc, p.N,
                               static_cast<int64_t>(blockIdx.x) * (32 * L::EPI_WARPS) + threadIdx.x -
                                   32 * L::EPI_WARP0,
                               static_cast<int64_t>(gridDim.x) * (32 * L::EPI_WARPS));
            const int half = (warp - L::EPI_WARP0) / 4;  // these warps' strips: every other one
            constexpr int STRIPS = GT_N / 64;
            const bool turned = sizeof(OutT) == 2 && p.unit && p.beta == 0.0f;
            bool ok = true;
            for (int t = unit; t < num_work; t += num_units) {
                const GroupedWork w = grouped_work<MODE>(t, table, p);
                const int f = w.f0 + static_cast<int>(rank) * TC_BM + q * 32;
                auto store = [&](const auto& v, int s) {
                    OutT* c = out + (w.c0 + s) * p.ldc + f;
                    if constexpr (sizeof(OutT) == 2) {
                        if (turned) {
                            put_turned(v, staging, c, p.ldc, w.count - s, p.N - f, p.alpha);
                            return;
                        }
                    }
                    if (f + static_cast<int>(lane) < p.N)
                        put_column(c + lane, p.ldc, w.count - s, v, p.alpha, p.beta);
                };
                // 16 of the lanes (turned: see put_turned()) or columns of a strip
                auto load = [&](uint32_t from, int h, uint32_t (&v)[16]) {
                    if (turned)
                        tmem_ld_16x256b_x4(from + (static_cast<uint32_t>(h) << 16), v);
                    else
                        tmem_ld_32x32b_x16(from + h, v);
                    tmem_wait_ld(v);
                };
                if (p.segments == 1) {
                    ok = take();
                    if (!ok)
                        break;
                    const uint32_t from = t_lane + static_cast<uint32_t>((local & 1) * GT_N);
#pragma unroll 1
                    for (int s = 32 * half; s < w.count; s += 64) {
                        float x[32];
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            uint32_t v[16];
                            load(from + s, h, v);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                x[h + i] = __uint_as_float(v[i]);
                        }
                        store(x, s);
                    }
                    give();
                    continue;
                }
                float sum[STRIPS][32] = {};
#pragma unroll 1
                for (int segment = 0; segment < p.segments; ++segment) {
                    ok = take();
                    if (!ok)
                        break;
                    const uint32_t from = t_lane + static_cast<uint32_t>((local & 1) * GT_N + 32 * half);
#pragma unroll
                    for (int j = 0; j < STRIPS; ++j)
                        if (32 * half + 64 * j < w.count) {
#pragma unroll
                            for (int h = 0; h < 32; h += 16) {
                                uint32_t v[16];
                                load(from + 64 * j, h, v);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    sum[j][h + i] += __uint_as_float(v[i]);
                            }
                        }
                    give();  // (before the stores: the next tile's segments take both accumulators)
                }
                if (!ok)
                    break;
#pragma unroll
                for (int j = 0; j < STRIPS; ++j)
                    if (32 * half + 64 * j < w.count)
                        store(sum[j], 32 * half + 64 * j);
            }
        } else {
            constexpr int HALF = GT_N / 2, CHUNKS = HALF / 32;
            const int half = (warp - L::EPI_WARP0) / 4;  // of the tile's columns
            bool ok = true;
            for (int t = unit; t < num_work; t += num_units) {
                const GroupedWork w = grouped_work<MODE>(t, table, p);
                float sum[CHUNKS][32] = {};
                for (int kb = 0; kb < w.k_blocks; kb += GT_SEGMENT) {
                    ok = take();
                    if (!ok)
                        break;
                    const uint32_t from = t_lane + static_cast<uint32_t>((local & 1) * GT_N + half * HALF);
#pragma unroll
                    for (int j = 0; j < CHUNKS; ++j)
                        if (half * HALF + 32 * j < w.count) {
#pragma unroll
                            for (int h = 0; h < 32; h += 16) {
                                uint32_t v[16];
                                tmem_ld_32x32b_x16(from + 32 * j + h, v);
                                tmem_wait_ld(v);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    sum[j][h + i] += __uint_as_float(v[i]);
                            }
                        }
                    give();
                }
                if (!ok)
                    break;
                const int f = w.f0 + static_cast<int>(rank) * TC_BM + q * 32, row = f + static_cast<int>(lane);
                if (f >= p.N)
                    continue;
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) {
                    const int s = half * HALF + 32 * j, left = w.count - s;
                    if (left <= 0)
                        break;
                    uint32_t v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = __float_as_uint(sum[j][i]);
                    OutT* c = out + w.g * p.stride_c + row * p.ldc + w.c0 + s;
                    if (p.tma_out) {
#pragma unroll
                        for (int part = 0; part < static_cast<int>(sizeof(OutT)) / 2; ++part) {
                            if (lane == 0)
                                bulk_wait_group_read<0>();
                            __syncwarp();
                            strip_to_smem<OutT>(v, part, staging, p.alpha);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                tma_store_3d(&tmC, staging, w.c0 + s + 16 * part, f, w.g);
                                bulk_commit_group();
                            }
                        }
                    } else if (p.unit && p.beta == 0.0f) {
#pragma unroll
                        for (int part = 0; part < static_cast<int>(sizeof(OutT)) / 2; ++part)
                            put_rows(v, part, staging, c - lane * p.ldc + 16 * part, p.ldc, p.N - f,
                                     left - 16 * part, p.alpha);
                    } else if (p.unit) {
                        if (row < p.N)
                            put_row(c, v, left, p.unit, p.alpha, p.beta);
                    } else {
                        put_strip(v, staging, c - lane * p.ldc, p.ldc, min(32, p.N - f), left, p.alpha, p.beta);
                    }
                }
            }
            if (lane == 0)
                bulk_wait_group_read<0>();
            __syncwarp();
        }
    }

    // ---------------------------------------------------- teardown
    __syncwarp();  // reconverge each warp after its role's divergent loop
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<2>(tmem_base, L::TMEM_COLS);
    }
}

}  // namespace tmmo
