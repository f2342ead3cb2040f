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
// Warps: 0 TMA producer, 1 MMA issuer (of the leader CTA), 2-5 epilogue, and for
// the gradient 6, which zeroes.  The ring of two 64-deep K steps per stage with a
// barrier each, the bounded waits and the two accumulators in tensor memory
// are those of tc_gemm_kernel.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "grouped.cuh"
#include "ops.cuh"
#include "simt_tile.cuh"
#include "warp_roles.cuh"

namespace tmmo {

enum { GROUPED_T = 0, GROUPED_N = 1, GROUPED_WGRAD = 2 };

constexpr int GT_STAGES = 3;
constexpr int GT_KSUB = 2;
constexpr int GT_N = 256;        // the N side of a full tile
constexpr int GT_SORTED = 256;   // groups, at most, that the gradient sorts

struct GroupedTcParams {
    Grouping by;
    void* C;              // Y, or the gradients
    int64_t ldc, stride_c;
    int N, K;             // outputs and inputs of a weight
    int tiles_f, tiles_c; // 256-wide tiles of the lanes' axis; gradient: of the other one
    float alpha, beta;
    bool zero_rest;
    bool swap;            // the weights' map has its outer dimensions exchanged
    bool one_weight;
    bool tma_out;         // gradient: stored by TMA
    uint32_t idesc;       // with N = 0
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

template <int MODE>
struct GroupedLayout {
    static constexpr bool WGRAD = MODE == GROUPED_WGRAD;
    static constexpr int THREADS = WGRAD ? 224 : 192;
    static constexpr int SUB = TC_BM * TC_BK * 2;  // 16 KiB: an operand's K step
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + GT_STAGES * GT_KSUB * SUB;
    static constexpr int OFF_STAGING = OFF_B + GT_STAGES * GT_KSUB * SUB;
    static constexpr int OFF_TABLE = OFF_STAGING + (WGRAD ? 4 * TC_STAGING_BYTES : 0);
    static constexpr int OFF_BAR = OFF_TABLE + (GroupTable::BYTES + 15) / 16 * 16;
    static constexpr int STEPS = GT_STAGES * GT_KSUB;
    static constexpr int NUM_BARS = STEPS + GT_STAGES + 5 + (WGRAD ? STEPS : 0);
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
        const int each = ((rows + tiles - 1) / tiles + 31) / 32 * 32;
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

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// p[r * ld] = alpha * v[r] + beta * p[r * ld] for r < rows: what is added to is
// loaded before anything is stored, so that the loads overlap.
template <int R, typename OutT>
__device__ __forceinline__ void grouped_put(OutT* p, int64_t ld, int rows, const float (&v)[R],
                                            const GroupedTcParams& q)
{
    float old[R];
    if (q.beta != 0.0f) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            old[r] = r < rows ? to_f32(p[r * ld]) : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r < rows)
            put(p + r * ld, q.beta != 0.0f ? fmaf(q.beta, old[r], q.alpha * v[r]) : q.alpha * v[r]);
}

// Strip of 32 rows x 32 FP32 values of a lane-major accumulator (this thread
// holds a row) to C, through `staging`, in whole lines: any alignment, and
// with the addition to C.
template <typename OutT>
__device__ __forceinline__ void grouped_strip(const uint32_t (&v)[32], uint32_t staging, uint32_t lane,
                                              OutT* c, int64_t ldc, int rows, int cols,
                                              const GroupedTcParams& p)
{
    const uint32_t at = staging + lane * 128;
#pragma unroll
    for (int j = 0; j < 32; ++j)  // column j of row `lane` at j ^ lane: no bank conflicts
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + ((j ^ lane) << 2)), "r"(v[j]) : "memory");
    __syncwarp();
    if (static_cast<int>(lane) < cols)
        for (int r = 0; r < rows; r += 8) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = ld_shared_f32(staging + (r + i) * 128 + ((lane ^ (r + i)) << 2));
            grouped_put(c + r * ldc + lane, ldc, rows - r, f, p);
        }
    __syncwarp();
}

// How many rows a tile of the products has at most: what is quickest, by the waves
// of tiles on the pairs and the time of a tile.  A K step of n rows takes about
// 315 + 1.23 n cycles (630 at 256: operands from L2 set the pace).  5000 rows of 12
// groups by 1000 outputs are 104 tiles of 256 rows, two waves on 76 pairs, and 132
// of 192.  One warp calls it.
__device__ __forceinline__ int tile_rows(const GroupTable& table, int groups, int tiles_f, int pairs)
{
    int best = GT_N, least = 0;
#pragma unroll 1
    for (int rows = GT_N; rows >= 128; rows -= 32) {
        const int tiles = __reduce_add_sync(0xffffffffu, lane_tiles(table, groups, rows));
        const int waves = static_cast<int>((static_cast<int64_t>(tiles) * tiles_f + pairs - 1) / pairs);
        const int time = min(waves, 1 << 18) * (315 + rows * 5 / 4);
        if (rows == GT_N || time < least) {
            best = rows;
            least = time;
        }
        if (waves <= 1)
            break;  // smaller tiles win nothing
    }
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
    auto full_bar = [&](int s, int j) { return bar0 + 8u * (s * GT_KSUB + j); };
    auto empty_bar = [&](int s) { return bar0 + 8u * (L::STEPS + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (L::STEPS + GT_STAGES + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (L::STEPS + GT_STAGES + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (L::STEPS + GT_STAGES + 4);
    // gradient: a group's last K step lands on this CTA's own barrier first
    auto tail_bar = [&](int s, int j) {
        return bar0 + 8u * (L::STEPS + GT_STAGES + 5 + s * GT_KSUB + j);
    };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);

    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int unit = blockIdx.x >> 1, num_units = gridDim.x >> 1;
    const TcWatch watch{abort_flag, p.status, p.wait_budget};

    if (threadIdx.x == 0) {
        for (int s = 0; s < GT_STAGES; ++s) {
            for (int j = 0; j < GT_KSUB; ++j) {
                // gradient: an arrival for each CTA, as either may have to zero
                mbar_init(full_bar(s, j), WGRAD ? 2 : 1);
                if (WGRAD)
                    mbar_init(tail_bar(s, j), 1);
            }
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 8);  // every epilogue warp of the pair
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmC);
    }
    if (warp == 1) {
        tmem_alloc<2>(smem_u32(tmem_slot), L::TMEM_COLS);
        tmem_relinquish<2>();
    }
    const GroupTable table = load_groups(reinterpret_cast<int*>(smem + L::OFF_TABLE), p.by);
    if (!WGRAD)
        count_tiles(table, p.by.groups, [&] { return tile_rows(table, p.by.groups, p.tiles_f, num_units); });
    else if (p.by.groups <= GT_SORTED)
        sort_groups(table, p.by.groups);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int num_work = (WGRAD ? p.by.groups * p.tiles_c : table.tile[p.by.groups]) * p.tiles_f;
    // rows of a group's last K step that the tensor core reads beyond the group
    auto is_ragged = [&](const GroupedWork& w, int kb) {
        return WGRAD && kb == w.k_blocks - 1 && (w.rows & 15) != 0;
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        const uint32_t sA = sbase + L::OFF_A;
        const uint32_t sB = sbase + L::OFF_B;
        int stage = 0;
        uint32_t phase = 0;
        int issued[GT_STAGES], ragged[L::STEPS];
#pragma unroll
        for (int s = 0; s < GT_STAGES; ++s)
            issued[s] = 0;
#pragma unroll
        for (int s = 0; s < L::STEPS; ++s)
            ragged[s] = 0;
        bool ok = true;
        for (int t = unit; ok && t < num_work; t += num_units) {
            const GroupedWork w = grouped_work<MODE>(t, table, p);
            const int f = w.f0 + static_cast<int>(rank) * TC_BM;
            const int half = w.n / 2;
            const int c = w.c0 + static_cast<int>(rank) * half;
            const int z = p.one_weight ? 0 : w.g;
            const uint32_t bytes = L::SUB + half * TC_BK * 2;
            for (int kb0 = 0; kb0 < w.k_blocks; kb0 += GT_KSUB) {
                const int nsub = min(GT_KSUB, w.k_blocks - kb0);
                ok = warp_wait(empty_bar(stage), phase ^ 1, watch);
                if (!ok)
                    break;
                // test hook (-1 in normal use): skip the stage holding that K step
                if (p.fault_skip_kblock < kb0 || p.fault_skip_kblock >= kb0 + nsub) {
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < GT_KSUB; ++j) {
                            if (j < nsub && is_ragged(w, kb0 + j)) {
                                mbar_arrive_expect_tx(tail_bar(stage, j), bytes);
                            } else if (leader) {
                                if (WGRAD)
                                    mbar_arrive(full_bar(stage, j));
                                if (j < nsub)
                                    mbar_arrive_expect_tx(full_bar(stage, j), 2 * bytes);
                                else
                                    mbar_arrive(full_bar(stage, j));  // unused: complete its phase
                            }
                        }
#pragma unroll
                        for (int j = 0; j < GT_KSUB; ++j) {
                            if (j >= nsub)
                                break;
                            const int kb = kb0 + j;
                            const uint32_t bar = is_ragged(w, kb) ? mapa_shared(tail_bar(stage, j), rank)
                                                                  : mapa_shared(full_bar(stage, j), 0);
                            const uint32_t dA = sA + (stage * GT_KSUB + j) * L::SUB;
                            const uint32_t dB = sB + (stage * GT_KSUB + j) * L::SUB;
                            if constexpr (WGRAD) {
                                const int row = w.row0 + kb * TC_BK;
#pragma unroll
                                for (int b = 0; b < 2; ++b)
                                    tma_load_2d_pair(dA + b * 8192, &tmA, bar, f + 64 * b, row);
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
                    }
                    __syncwarp();
#pragma unroll
                    for (int s = 0; s < GT_STAGES; ++s) {  // (registers: no indexing)
                        issued[s] += s == stage;
#pragma unroll
                        for (int j = 0; j < GT_KSUB; ++j)
                            ragged[s * GT_KSUB + j] += s == stage && j < nsub && is_ragged(w, kb0 + j);
                    }
                }
                if (++stage == GT_STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) {
            // Wait (bounded) for the loads already issued before shared
            // memory goes away: the leader's barriers cover both CTAs.
            auto drain = [&](uint32_t bar, int uses) {
                const long long t0 = clock64();
                while (!mbar_try_wait(bar, static_cast<uint32_t>(uses - 1) & 1u) &&
                       clock64() - t0 < p.wait_budget) {
                }
            };
            for (int s = 0; s < GT_STAGES; ++s)
                for (int j = 0; j < GT_KSUB; ++j) {
                    if (leader && issued[s] > 0)
                        drain(full_bar(s, j), issued[s]);
                    if (WGRAD && ragged[s * GT_KSUB + j] > 0)
                        drain(tail_bar(s, j), ragged[s * GT_KSUB + j]);
                }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (leader) {
            const uint32_t sA = sbase + L::OFF_A;
            const uint32_t sB = sbase + L::OFF_B;
            int stage = 0;
            uint32_t phase = 0;
            int local = 0;
            bool ok = true;
            for (int t = unit; ok && t < num_work; t += num_units) {
                const GroupedWork w = grouped_work<MODE>(t, table, p);
                if (w.k_blocks == 0)
                    continue;
                const int acc = local & 1;
                const uint32_t acc_phase = (local >> 1) & 1;
                ++local;
                ok = warp_wait<true>(tempty_bar(acc), acc_phase ^ 1, watch);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * GT_N);
                const uint32_t idesc = p.idesc | static_cast<uint32_t>(w.n >> 3) << 17;
                for (int kb0 = 0; kb0 < w.k_blocks; kb0 += GT_KSUB) {
                    const int nsub = min(GT_KSUB, w.k_blocks - kb0);
#pragma unroll
                    for (int j = 0; j < GT_KSUB; ++j) {
                        if (j >= nsub)
                            break;
                        ok = warp_wait<WGRAD>(full_bar(stage, j), phase, watch);
                        if (!ok)
                            break;
                        tc_fence_after();
                        const uint32_t a0 = sA + (stage * GT_KSUB + j) * L::SUB;
                        const uint32_t b0 = sB + (stage * GT_KSUB + j) * L::SUB;
                        // 16-deep instructions; gradient: as many as there are rows
                        const int deep = WGRAD ? min(4, (w.rows - (kb0 + j) * TC_BK + 15) / 16) : 4;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < TC_BK / TC_UMMA_K; ++k) {
                                if (WGRAD && k >= deep)
                                    break;
                                const uint64_t adesc = A_MN ? smem_desc_sw128(a0 + k * 2048, 8192, 1024)
                                                            : smem_desc_sw128(a0 + k * 32, 16, 1024);
                                const uint64_t bdesc = WGRAD ? smem_desc_sw128(b0 + k * 2048, 8192, 1024)
                                                             : smem_desc_sw128(b0 + k * 32, 16, 1024);
                                tc_mma_f16<2>(d_tmem, adesc, bdesc, idesc, kb0 != 0 || j != 0 || k != 0);
                            }
                            if (j == nsub - 1) {
                                tc_commit_pair(empty_bar(stage), 0x3);
                                if (kb0 + GT_KSUB >= w.k_blocks)
                                    tc_commit_pair(tfull_bar(acc), 0x3);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok)
                        break;
                    if (++stage == GT_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
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
    } else if (warp < 6) {
        // ------------------------------------------------ epilogue
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const uint32_t leader_tempty0 = mapa_shared(tempty_bar(0), 0);
        const uint32_t leader_tempty1 = mapa_shared(tempty_bar(1), 0);
        OutT* const out = static_cast<OutT*>(p.C);
        if (!WGRAD && p.zero_rest)
            zero_rest_rows(table, p.by, out, p.ldc, p.N,
                           static_cast<int64_t>(blockIdx.x) * 128 + (threadIdx.x - 64),
                           static_cast<int64_t>(gridDim.x) * 128);
        int local = 0;
        for (int t = unit; t < num_work; t += num_units) {
            const GroupedWork w = grouped_work<MODE>(t, table, p);
            const int acc = local & 1;
            const bool any = w.k_blocks > 0;
            if (any) {
                int ok = 1;
                if (lane == 0)
                    ok = tc_wait(tfull_bar(acc), (local >> 1) & 1, watch) ? 1 : 0;
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok)
                    break;
                ++local;
                tc_fence_after();
            }
            const int f = w.f0 + static_cast<int>(rank) * TC_BM + q * 32;
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                   static_cast<uint32_t>(acc * GT_N);
            if constexpr (WGRAD) {
                const uint32_t staging = sbase + L::OFF_STAGING + q * TC_STAGING_BYTES;
                if (any && p.tma_out) {
                    constexpr int STRIP = TcOut<OutT>::STRIP;
                    TcParams scale{};
                    scale.alpha = p.alpha;
#pragma unroll 1
                    for (int s = 0; s < w.n / STRIP; ++s) {
                        const int col = w.c0 + s * STRIP;
                        if (f >= p.N || col >= p.K)
                            break;
                        if (lane == 0)
                            bulk_wait_group_read<0>();
                        __syncwarp();
                        tc_strip_to_smem<OutT>(t_row + s * STRIP, staging, lane, scale, 0, 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_3d(&tmC, staging, col, f, w.g);
                            bulk_commit_group();
                        }
                    }
                } else if (p.tma_out) {
                    // no rows: one strip of zeros, stored again and again
                    if (lane == 0)
                        bulk_wait_group_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_shared_v4(staging + lane * 128 + i * 16, 0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && f < p.N) {
                        for (int col = w.c0; col < min(p.K, w.c0 + GT_N); col += TcOut<OutT>::STRIP)
                            tma_store_3d(&tmC, staging, col, f, w.g);
                        bulk_commit_group();
                    }
                } else {
                    if (lane == 0)
                        bulk_wait_group_read<0>();
                    __syncwarp();
#pragma unroll 1
                    for (int s = 0; s < w.count; s += 32) {
                        uint32_t v[32] = {};
                        if (any) {
                            tmem_ld_32x32b_x32(t_row + s, v);
                            tmem_wait_ld(v);
                        }
                        if (f < p.N)
                            grouped_strip(v, staging, lane,
                                          out + w.g * p.stride_c + f * p.ldc + w.c0 + s, p.ldc,
                                          min(32, p.N - f), w.count - s, p);
                    }
                }
            } else {
                const bool mine = f + static_cast<int>(lane) < p.N;
                OutT* c = out + w.c0 * p.ldc + f + lane;
#pragma unroll 1
                for (int s = 0; s < w.count; s += 32, c += 32 * p.ldc) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(t_row + s, v);
                    tmem_wait_ld(v);
                    const int rows = w.count - s;
                    if (mine) {
                        float x[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            x[j] = __uint_as_float(v[j]);
                        grouped_put(c, p.ldc, rows, x, p);
                    }
                }
            }
            if (any) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(acc ? leader_tempty1 : leader_tempty0);
            }
        }
        if (WGRAD && lane == 0)
            bulk_wait_group_read<0>();
        __syncwarp();
    } else if constexpr (WGRAD) {
        // ------------------------- rows of other groups in a group's last K step
        int stage = 0;
        uint32_t parity = 0;  // a bit for each step's barrier
        for (int t = unit; t < num_work; t += num_units) {
            const GroupedWork w = grouped_work<MODE>(t, table, p);
            if (w.k_blocks == 0)
                continue;
            const int last = w.k_blocks - 1;
            const int s = (stage + last / GT_KSUB) % GT_STAGES, j = last % GT_KSUB;
            stage = (s + 1) % GT_STAGES;
            if (!is_ragged(w, last))
                continue;
            const int step = s * GT_KSUB + j;
            int ok = 1;
            if (lane == 0)
                ok = tc_wait(tail_bar(s, j), (parity >> step) & 1, watch) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok)
                break;
            parity ^= 1u << step;
            // a row of 64 values is 128 contiguous bytes (its swizzle stays within)
            const int from = w.rows - last * TC_BK, to = (from + 15) / 16 * 16;
            const int boxes = 2 + w.n / 128;
            for (int b = 0; b < boxes; ++b) {
                const uint32_t box = sbase + (b < 2 ? L::OFF_A + b * 8192 : L::OFF_B + (b - 2) * 8192) +
                                     step * L::SUB;
                for (int i = from * 8 + static_cast<int>(lane); i < to * 8; i += 32)
                    st_shared_v4(box + i * 16, 0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(mapa_shared(full_bar(s, j), 0));
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
