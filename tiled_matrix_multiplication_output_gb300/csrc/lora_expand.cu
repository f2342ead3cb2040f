// Y = X W^T + t E^T on the tensor cores, for products with many output tiles: the
// shared product and every adapter's in one accumulator.
//
// The kernel is the CTA-pair GEMM (256 x 256 tiles, two 64-deep K steps per
// stage) whose contraction goes on, for each adapter among the tile's rows, over
// its rank values: A is then t in parts, B the adapter's factor, and the lanes
// of other adapters' rows are masked out.  An adapter of rank 64 costs two more
// K steps (of 64 at K = 4096; four with rank values in three parts) in the tiles that
// have it, and Y is written once.  Every 1024 inputs the accumulator is added to sums in
// the epilogue's registers (see grouped_tc.cuh; 171 us without, 174 so, rank values
// included).  Bound by the tensor cores as the shared product alone: 8192 rows of 12
// adapters of rank 64 by 4096 x 4096, BF16, not power-capped, 159 us (1.77 PFLOP/s).
//
// Of FP16 operands, a warp of each CTA splits its half of a factor in two in shared
// memory (lora_tc.cuh) before the step counts as loaded: 210 us for the same call of
// 174 (five instructions for 16 rank values instead of two, and four steps of rank 64
// instead of two).
//
// Launched as a programmatic dependent of the kernel that makes the rank values: it
// waits for them only when the first tile's shared product has been issued.
#include <algorithm>

#include "grouped_maps.h"
#include "lora_tc.cuh"
#include "persistent.cuh"
#include "store_rows.cuh"

namespace tmmo {
namespace {

constexpr int LE_STAGES = 3;
constexpr int LE_KSUB = 2;
// Warps 0: copies, 1: MMA, 2: FP16 factors in two, 4 to 11: epilogue, to which the first
// ones leave registers of the 168 that a thread is launched with.
constexpr int LE_EPI_WARP0 = 4;
constexpr int LE_EPI_WARPS = 8;
constexpr int LE_THREADS = 32 * (LE_EPI_WARP0 + LE_EPI_WARPS);
constexpr int LE_REGS_FEW = 88, LE_REGS_EPI = 208;
static_assert(LE_EPI_WARP0 * LE_REGS_FEW + LE_EPI_WARPS * LE_REGS_EPI <= LE_THREADS / 32 * 168,
              "of the block's registers");
constexpr int LE_SEGMENT = 16;  // K steps that one accumulator adds up, at most (see grouped_tc.cuh)

struct ExpandParams {
    int M, N, k_blocks, rank;
    int segments, segment;  // parts of K, and their K steps
    int tiles_m, tiles_n;
    int whole, items;     // tiles of 256 columns first, the others in halves
    bool adapters;        // there are any: plans and rank values are made
    bool one;             // one factor for every adapter
    LoraParts lay;
    const LoraPlan* plan;
    void* C;
    int64_t ldc;
    int unit;             // row_unit of the output
    uint32_t idesc;       // with N = 0
    bool split;           // FP16 factors, split in two
    uint32_t idesc_e;     // of the adapters' products: BF16
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

struct ExpandLayout {
    static constexpr int SUB = 16384;
    static constexpr int STEPS = LE_STAGES * LE_KSUB;
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = STEPS * SUB;
    static constexpr int OFF_STAGING = OFF_B + STEPS * SUB;
    static constexpr int OFF_BAR = OFF_STAGING + LE_EPI_WARPS * 2048;
    static constexpr int NUM_BARS = 2 * STEPS + LE_STAGES + 5;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NUM_BARS;
    static constexpr int SMEM_ALLOC = OFF_MISC + 16 + 1024;
    static_assert(SMEM_ALLOC <= 232448, "exceeds 227 KiB of dynamic shared memory");
};

// The adapters of a pair's 256 rows, ascending, from the plans of its halves.
// What comes next is loaded ahead, so that the tile's shared product hides it.
class PairAdapters {
public:
    __device__ void begin(const ExpandParams& p, int mb)
    {
        const int plans = (p.M + LT_ROWS - 1) / LT_ROWS;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            half_[h] = p.plan + 2 * mb + h;
            count_[h] = 2 * mb + h < plans ? half_[h]->count : 0;
            at_[h] = 0;
            // (the first entry lies in memory even if it is not one)
            id_[h] = 2 * mb + h < plans ? half_[h]->ids[0] : 0;
            rows_[h] = 2 * mb + h < plans ? *reinterpret_cast<const uint4*>(half_[h]->rows[0])
                                          : make_uint4(0, 0, 0, 0);
        }
    }
    // The next adapter, or -1, and (off) the lanes that do not have it.
    __device__ int next(uint32_t (&off)[8])
    {
        int g[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            g[h] = at_[h] < count_[h] ? id_[h] : 0x7fffffff;
        const int least = min(g[0], g[1]);
        if (least == 0x7fffffff)
            return -1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool has = g[h] == least;
            off[4 * h] = has ? ~rows_[h].x : ~0u;
            off[4 * h + 1] = has ? ~rows_[h].y : ~0u;
            off[4 * h + 2] = has ? ~rows_[h].z : ~0u;
            off[4 * h + 3] = has ? ~rows_[h].w : ~0u;
            at_[h] += has;
            if (has && at_[h] < count_[h]) {
                id_[h] = half_[h]->ids[at_[h]];
                rows_[h] = *reinterpret_cast<const uint4*>(half_[h]->rows[at_[h]]);
            }
        }
        return least;
    }

private:
    const LoraPlan* half_[2];
    int count_[2], at_[2], id_[2];
    uint4 rows_[2];
};

// An output tile, or half of one.
struct Item {
    int mb, col, n;
};
__device__ __forceinline__ Item item(int t, const ExpandParams& p)
{
    const int half = t < p.whole ? 0 : (t - p.whole) & 1;
    const int n = t < p.whole ? 256 : 128;
    if (t >= p.whole)
        t = p.whole + (t - p.whole) / 2;
    // row tiles eight at a time, and within those down the rows first
    const int band = t / (8 * p.tiles_n) * 8;
    const int high = min(p.tiles_m - band, 8);
    const int u = t - band * p.tiles_n;
    return {band + u % high, u / high * 256 + half * 128, n};
}

template <bool ACROSS, typename OutT>
__global__ void __launch_bounds__(LE_THREADS, 1)
    lora_expand_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmT, const __grid_constant__ CUtensorMap tmE,
                       const __grid_constant__ CUtensorMap tmW64, const __grid_constant__ CUtensorMap tmE64,
                       const __grid_constant__ ExpandParams p)
{
    using L = ExpandLayout;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::OFF_BAR;
    auto full_bar = [&](int s, int j) { return bar0 + 8u * (s * LE_KSUB + j); };
    auto empty_bar = [&](int s) { return bar0 + 8u * (L::STEPS + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (L::STEPS + LE_STAGES + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (L::STEPS + LE_STAGES + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (L::STEPS + LE_STAGES + 4);
    // a step whose factor is to be split lands on this CTA's own barrier first
    auto landed_bar = [&](int at) { return bar0 + 8u * (L::STEPS + LE_STAGES + 5 + at); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
    volatile int* progress = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 8);  // steps copied

    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int unit = blockIdx.x >> 1, num_units = gridDim.x >> 1;
    const TcWatch watch{abort_flag, p.status, p.wait_budget};

    if (threadIdx.x == 0) {
        for (int s = 0; s < LE_STAGES; ++s) {
            for (int j = 0; j < LE_KSUB; ++j)
                mbar_init(full_bar(s, j), p.split ? 2 : 1);  // (either CTA's factor)
            mbar_init(empty_bar(s), 1);
        }
        for (int at = 0; at < L::STEPS; ++at)
            mbar_init(landed_bar(at), 1);
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 2 * LE_EPI_WARPS);  // of the pair
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        *progress = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmT);
        tma_prefetch_desc(&tmE);
    }
    if (warp == 1) {
        tmem_alloc<2>(smem_u32(tmem_slot), 512);
        tmem_relinquish<2>();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp < LE_EPI_WARP0) {
        set_max_regs_dec<LE_REGS_FEW>();
        if (warp == 0) {
            // ------------------------------------------------ TMA producer
            const uint32_t sA = sbase + L::OFF_A, sB = sbase + L::OFF_B;
            int stage = 0, sub = 0;
            uint32_t phase = 0;
            int issued[L::STEPS];
#pragma unroll
            for (int s = 0; s < L::STEPS; ++s)
                issued[s] = 0;
            uint32_t to_split = 0, parity = 0;  // steps that last landed on their own barrier; how often
            int steps = 0;
            bool ok = true, waited = false;
            auto next_stage = [&] {
                sub = 0;
                if (++stage == LE_STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            };
            auto count = [&](int at) {
#pragma unroll
                for (int s = 0; s < L::STEPS; ++s)  // (registers: no indexing)
                    issued[s] += s == at;
            };
            // One K step: load(A's place, B's place, barrier); split: its factor is to be split.
            auto step = [&](bool skip, bool split, uint32_t bytes, auto load) {
                if (sub == 0 && !warp_wait(empty_bar(stage), phase ^ 1, watch))
                    return false;
                ++steps;
                if (p.split && lane == 0)
                    *progress = steps;
                if (!skip) {
                    const int at = stage * LE_KSUB + sub;
                    if (elect_one()) {
                        if (split) {
                            mbar_arrive_expect_tx(landed_bar(at), bytes / 2);
                        } else if (leader) {
                            if (p.split)
                                mbar_arrive(full_bar(stage, sub));
                            mbar_arrive_expect_tx(full_bar(stage, sub), bytes);
                        }
                        load(sA + at * L::SUB, sB + at * L::SUB,
                             split ? mapa_shared(landed_bar(at), rank) : mapa_shared(full_bar(stage, sub), 0));
                    }
                    __syncwarp();
                    count(at);
                    to_split = split ? to_split | 1u << at : to_split & ~(1u << at);
                    parity ^= static_cast<uint32_t>(split) << at;
                }
                if (++sub == LE_KSUB)
                    next_stage();
                return true;
            };
            for (int t = unit; ok && t < p.items; t += num_units) {
                const Item w = item(t, p);
                const int row = w.mb * 256 + static_cast<int>(rank) * TC_BM;
                const int col = w.col + static_cast<int>(rank) * w.n / 2;
                const uint32_t bytes = 2 * (L::SUB + w.n * 64);
                PairAdapters list;
                if (waited)
                    list.begin(p, w.mb);
                // W's or a factor's outputs: boxes of 64 (x) or 128 and 64 (y)
                auto outputs = [&](auto box, auto box64, uint32_t dB) {
                    if (ACROSS) {
                        box(dB, col);
                        if (w.n > 128)
                            box(dB + 8192, col + 64);
                    } else if (w.n > 128) {
                        box(dB, col);
                    } else {
                        box64(dB, col);
                    }
                };
                for (int kb = 0; ok && kb < p.k_blocks; ++kb) {
                    const int k = kb * TC_BK;
                    ok = step(kb == p.fault_skip_kblock, false, bytes, [&](uint32_t dA, uint32_t dB, uint32_t bar) {
                        tma_load_2d_pair(dA, &tmX, bar, k, row);
                        auto load = [&](const CUtensorMap* map) {
                            return [=](uint32_t to, int c) {
                                tma_load_2d_pair(to, map, bar, ACROSS ? c : k, ACROSS ? k : c);
                            };
                        };
                        outputs(load(&tmW), load(&tmW64), dB);
                    });
                }
                if (!ok)
                    break;
                if (p.adapters) {
                    if (!waited) {
                        grid_dep_wait();
                        grid_dep_launch_dependents();  // the rank values are there for others, too
                        list.begin(p, w.mb);
                    }
                    waited = true;
                    uint32_t off[8];
                    for (int g = list.next(off); ok && g >= 0; g = list.next(off)) {
                        const int z = p.one ? 0 : g;
                        for (int c = 0; ok && c < p.lay.chunks; ++c) {
                            const int j = c * p.lay.chunk;
                            ok = step(false, p.split, bytes, [&](uint32_t dA, uint32_t dB, uint32_t bar) {
                                tma_load_2d_pair(dA, &tmT, bar, c * 64, row);
                                auto load = [&](const CUtensorMap* map) {
                                    return [=](uint32_t to, int o) {
                                        tma_load_3d_pair(to, map, bar, ACROSS ? o : j, ACROSS ? j : o, z);
                                    };
                                };
                                outputs(load(&tmE), load(&tmE64), dB);
                            });
                        }
                    }
                }
                if (ok && sub != 0) {
                    if (leader && elect_one()) {  // the stage's unused step
                        mbar_arrive(full_bar(stage, 1));
                        if (p.split)
                            mbar_arrive(full_bar(stage, 1));
                    }
                    __syncwarp();
                    count(stage * LE_KSUB + 1);
                    to_split &= ~(1u << (stage * LE_KSUB + 1));
                    next_stage();
                }
            }
            if (!ok && lane == 0) {
                // wait (bounded) for the loads already issued (those of both CTAs, but each CTA
                // its own factors to be split) before shared memory goes away
                for (int s = 0; s < L::STEPS; ++s) {
                    const bool own = (to_split >> s) & 1;
                    const uint32_t bar = own ? landed_bar(s) : bar0 + 8u * s;
                    const uint32_t phase_of = own ? ((parity >> s) & 1) ^ 1 : (issued[s] - 1) & 1;
                    const long long t0 = clock64();
                    while ((own || (leader && issued[s] > 0)) && !mbar_try_wait(bar, phase_of) &&
                           clock64() - t0 < p.wait_budget) {
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issuer
            if (leader) {
                const uint32_t sA = sbase + L::OFF_A, sB = sbase + L::OFF_B;
                int stage = 0, sub = 0, local = 0;
                uint32_t phase = 0;
                bool ok = true, waited = false;
                auto next_stage = [&] {
                    if (elect_one())
                        tc_commit_pair(empty_bar(stage), 0x3);
                    __syncwarp();
                    sub = 0;
                    if (++stage == LE_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                };
                auto step = [&](auto multiply) {
                    if (!(p.split ? warp_wait<true>(full_bar(stage, sub), phase, watch)
                                  : warp_wait(full_bar(stage, sub), phase, watch)))
                        return false;
                    tc_fence_after();
                    const int at = stage * LE_KSUB + sub;
                    if (elect_one())
                        multiply(sA + at * L::SUB, sB + at * L::SUB);
                    __syncwarp();
                    if (++sub == LE_KSUB)
                        next_stage();
                    return true;
                };
                for (int t = unit; ok && t < p.items; t += num_units) {
                    const Item w = item(t, p);
                    uint32_t d_tmem = 0;
                    const uint32_t idesc = p.idesc | static_cast<uint32_t>(w.n >> 3) << 17;
                    PairAdapters list;
                    if (waited)
                        list.begin(p, w.mb);
                    for (int kb = 0; ok && kb < p.k_blocks;) {
                        ok = warp_wait<true>(tempty_bar(local & 1), ((local >> 1) & 1) ^ 1, watch);
                        if (!ok)
                            break;
                        tc_fence_after();
                        d_tmem = tmem_base + static_cast<uint32_t>((local & 1) * 256);
                        const int begin = kb, end = min(kb + p.segment, p.k_blocks);
                        for (; ok && kb < end; ++kb)
                            ok = step([&](uint32_t a0, uint32_t b0) {
#pragma unroll
                                for (int k = 0; k < TC_BK / TC_UMMA_K; ++k)
                                    tc_mma_f16<2>(d_tmem, smem_desc_sw128(a0 + k * 32, 16, 1024),
                                                  ACROSS ? smem_desc_sw128(b0 + k * 2048, 8192, 1024)
                                                         : smem_desc_sw128(b0 + k * 32, 16, 1024),
                                                  idesc, kb != begin || k != 0);
                            });
                        if (ok && kb < p.k_blocks) {
                            if (elect_one())
                                tc_commit_pair(tfull_bar(local & 1), 0x3);
                            __syncwarp();
                            ++local;
                        }
                    }
                    if (!ok)
                        break;
                    if (p.adapters) {  // (of the last segment)
                        if (!waited) {
                            grid_dep_wait();
                            list.begin(p, w.mb);
                        }
                        waited = true;
                        uint32_t off[8];
                        for (int g = list.next(off); ok && g >= 0; g = list.next(off))
                            for (int c = 0; ok && c < p.lay.chunks; ++c)
                                ok = step([&](uint32_t a0, uint32_t b0) {
                                    const uint32_t idesc_e = p.idesc_e | static_cast<uint32_t>(w.n >> 3) << 17;
                                    each_product(p.lay, p.lay.deep(c, p.rank), p.split, [&](int part, int pair, int k) {
                                        const int b = pair * p.lay.chunk / 16 + k;
                                        tc_mma_f16_lanes(
                                            d_tmem, smem_desc_sw128(a0 + part * p.lay.chunk * 2 + k * 32, 16, 1024),
                                            ACROSS ? smem_desc_sw128(b0 + b * 2048, 8192, 1024)
                                                   : smem_desc_sw128(b0 + b * 32, 16, 1024),
                                            idesc_e, 1, off);
                                    });
                                });
                    }
                    if (!ok)
                        break;
                    if (sub != 0)
                        next_stage();
                    if (elect_one())
                        tc_commit_pair(tfull_bar(local & 1), 0x3);
                    __syncwarp();
                    ++local;
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
        } else if (warp == 2) {
            // ------------------------------------------------ factors in two
            if (p.split && p.adapters) {
                grid_dep_wait();
                int at = 0;           // the step's place
                uint32_t parity = 0;  // a bit for each
                bool ok = true;
                for (int t = unit; ok && t < p.items; t += num_units) {
                    const Item w = item(t, p);
                    PairAdapters list;
                    list.begin(p, w.mb);
                    at = (at + p.k_blocks) % L::STEPS;
                    uint32_t off[8];
                    for (int g = list.next(off); ok && g >= 0; g = list.next(off))
                        for (int c = 0; ok && c < p.lay.chunks; ++c) {
                            // (the steps of the shared product are not waited for)
                            ok = warp_wait_behind(landed_bar(at), (parity >> at) & 1, watch, progress);
                            if (!ok)
                                break;
                            parity ^= 1u << at;
                            const uint32_t tile = sbase + L::OFF_B + at * L::SUB;
                            if (ACROSS)
                                split_across(tile, w.n / 128);
                            else
                                split_rows(tile, w.n / 2, 128);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive_cluster(mapa_shared(bar0 + 8u * at, 0));
                            at = (at + 1) % L::STEPS;
                        }
                    at = (at + at % LE_KSUB) % L::STEPS;  // (behind a stage's unused step)
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue
        set_max_regs_inc<LE_REGS_EPI>();
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const int half = (warp - LE_EPI_WARP0) / 4;  // of the tile's columns
        const uint32_t staging = sbase + L::OFF_STAGING + (warp - LE_EPI_WARP0) * 2048;
        const uint32_t leader_tempty0 = mapa_shared(tempty_bar(0), 0);
        const uint32_t leader_tempty1 = mapa_shared(tempty_bar(1), 0);
        OutT* const out = static_cast<OutT*>(p.C);
        const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        constexpr int STRIPS = 128 / 32;
        int local = 0;
        // waits for the next accumulator, of a segment (whether of a tile's last one); gives it back
        bool waited = !p.adapters;
        auto take = [&](bool last) {
            if (last && !waited) {
                grid_dep_wait();  // (the first tile ends no sooner: its wait begins here)
                waited = true;
            }
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
        bool ok = true;
        for (int t = unit; t < p.items; t += num_units) {
            const Item w = item(t, p);
            const int row = w.mb * 256 + static_cast<int>(rank) * TC_BM + q * 32;
            const int first = half * w.n / 2;  // of these warps' columns, and behind the last
            const int cols = row < p.M ? min(first + w.n / 2, p.N - w.col) : 0;
            OutT* c = out + row * p.ldc + w.col;
            auto store = [&](const uint32_t (&v)[32], int s) {
                if (p.unit) {
#pragma unroll
                    for (int part = 0; part < static_cast<int>(sizeof(OutT)) / 2; ++part)
                        put_rows(v, part, staging, c + s + 16 * part, p.ldc, p.M - row, cols - s - 16 * part, 1.0f);
                } else {
                    put_strip(v, staging, c + s, p.ldc, min(32, p.M - row), cols - s, 1.0f, 0.0f);
                }
            };
            if (p.segments == 1) {
                ok = take(true);
                if (!ok)
                    break;
                const uint32_t from = t_lane + static_cast<uint32_t>((local & 1) * 256);
#pragma unroll 1
                for (int s = first; s < cols; s += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(from + s, v);
                    tmem_wait_ld(v);
                    store(v, s);
                }
                give();
                continue;
            }
            float sum[STRIPS][32] = {};
#pragma unroll 1
            for (int segment = 0; segment < p.segments; ++segment) {
                ok = take(segment == p.segments - 1);
                if (!ok)
                    break;
                const uint32_t from = t_lane + static_cast<uint32_t>((local & 1) * 256 + first);
#pragma unroll
                for (int j = 0; j < STRIPS; ++j)
                    if (first + 32 * j < cols) {
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
                give();  // (before the stores: the next tile's segments take both accumulators)
            }
            if (!ok)
                break;
#pragma unroll
            for (int j = 0; j < STRIPS; ++j)
                if (first + 32 * j < cols) {
                    uint32_t v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = __float_as_uint(sum[j][i]);
                    store(v, first + 32 * j);
                }
        }
    }

    // ---------------------------------------------------- teardown
    __syncwarp();  // reconverge each warp after its role's divergent loop
    if (p.adapters)
        grid_dep_wait();  // this grid must not end before the one it depends on
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<2>(tmem_base, 512);
    }
}

template <bool ACROSS, typename OutT>
cudaError_t launch(const CUtensorMap (&m)[6], ExpandParams& p, int num_sms, cudaStream_t stream)
{
    using L = ExpandLayout;
    static ClusterCaps caps;
    int cap = 0;
    const cudaError_t err =
        cluster_cap(lora_expand_kernel<ACROSS, OutT>, caps, 2, LE_THREADS, L::SMEM_ALLOC, num_sms, &cap);
    if (err != cudaSuccess)
        return err;
    // The tiles of a last wave that leaves at least half of the pairs idle are
    // cut in halves: 3.4 waves of tiles take 3.5 instead of 4.
    const int tiles = p.tiles_m * p.tiles_n, pairs = std::max(cap, 1), rest = tiles % pairs;
    p.whole = rest > 0 && 2 * rest <= pairs ? tiles - rest : tiles;
    p.items = p.whole + 2 * (tiles - p.whole);
    const int units = std::min(pairs, p.items);
    ClusterLaunch l(static_cast<unsigned>(2 * units), 2, LE_THREADS, L::SMEM_ALLOC, stream, p.adapters);
    return l.run(lora_expand_kernel<ACROSS, OutT>, m[0], m[1], m[2], m[3], m[4], m[5], p);
}

template <bool ACROSS>
cudaError_t launch(int out_dtype, const CUtensorMap (&m)[6], ExpandParams& p, int num_sms,
                   cudaStream_t stream)
{
    switch (out_dtype) {
    case DT_F32:
        return launch<ACROSS, float>(m, p, num_sms, stream);
    case DT_F16:
        return launch<ACROSS, __half>(m, p, num_sms, stream);
    default:
        return launch<ACROSS, __nv_bfloat16>(m, p, num_sms, stream);
    }
}

}  // namespace

int lora_parts_bytes(int rank, int parts) { return 2 * lora_parts(rank, parts).columns(); }

cudaError_t lora_expand_tc_launch(const LoraLaunch& l, cudaStream_t stream)
{
    if (lora_small_takes(l))
        return lora_small_tc_launch(l, stream);
    ExpandParams p{};
    p.M = l.rows;
    p.N = l.N;
    p.k_blocks = (l.K + TC_BK - 1) / TC_BK;
    p.segments = (p.k_blocks + LE_SEGMENT - 1) / LE_SEGMENT;
    p.segment = (p.k_blocks + p.segments - 1) / p.segments;
    p.segments = (p.k_blocks + p.segment - 1) / p.segment;
    p.rank = l.rank;
    p.tiles_m = (l.rows + 255) / 256;
    p.tiles_n = (l.N + 255) / 256;
    p.adapters = l.adapters > 0;
    p.one = l.adapters == 1 || l.stride_e == 0;
    p.lay = lora_parts(l.rank, l.parts);
    p.plan = static_cast<const LoraPlan*>(l.plan);
    p.C = l.Y;
    p.ldc = l.ldy;
    p.split = l.in_dtype == DT_F16;
    p.idesc = tc_idesc(!p.split, 256, 0, false, l.across);
    p.idesc_e = tc_idesc(true, 256, 0, false, l.across);
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip_kblock = l.fault_skip_kblock;
    CUtensorMap m[6];
    const int dt = l.in_dtype;
    auto weights = [&](CUtensorMap* map, uint32_t outputs) {
        return l.across ? l.maps->get(map, dt, l.W, 2, {l.N, l.K, 1}, {l.ldw, 0}, {64, TC_BK, 1})
                        : l.maps->get(map, dt, l.W, 2, {l.K, l.N, 1}, {l.ldw, 0}, {64, outputs, 1});
    };
    const int64_t stacked = p.one ? 1 : l.adapters, stride = p.one ? l.lde : l.stride_e;
    auto factors = [&](CUtensorMap* map, uint32_t outputs) {
        return l.across ? l.maps->get(map, dt, l.E, 3, {l.N, l.rank, stacked}, {l.lde, stride}, {64, TC_BK, 1})
                        : l.maps->get(map, dt, l.E, 3, {l.rank, l.N, stacked}, {l.lde, stride}, {64, outputs, 1});
    };
    bool ok = l.maps->get(&m[0], dt, l.X, 2, {l.K, l.rows, 1}, {l.ldx, 0}, {64, TC_BM, 1}) &&
              weights(&m[1], TC_BM) && weights(&m[4], 64);
    m[2] = m[3] = m[5] = m[0];
    if (ok && p.adapters)
        ok = l.maps->get(&m[2], DT_BF16, l.t, 2, {p.lay.columns(), l.rows, 1}, {p.lay.columns(), 0}, {64, TC_BM, 1}) &&
             factors(&m[3], TC_BM) && factors(&m[5], 64);
    if (!ok)
        return cudaErrorNotSupported;
    p.unit = row_unit(l.Y, l.ldy * type_bytes(l.out_dtype), 0);
    return l.across ? launch<true>(l.out_dtype, m, p, l.num_sms, stream)
                    : launch<false>(l.out_dtype, m, p, l.num_sms, stream);
}

}  // namespace tmmo
