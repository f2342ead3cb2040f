// Y = X W^T + t E^T on the tensor cores, for few output tiles: a decoding batch
// against a layer, or a small layer.
//
// Up to a few hundred rows the bound is reading the weights from HBM, and the
// adapters' factors where every row has its own.  One tile is 128 rows by 128
// outputs; its contraction is split over a cluster of up to eight CTAs, so that
// every SM has weights in flight, and the tile's adapters are dealt out among
// them as further K steps (with the lanes of other rows masked out).  The
// FP32 sums are added through distributed shared memory in rank order.
//
// For many adapters it is launched as a programmatic dependent of the kernel that
// makes the rank values, and small enough to share an SM with it: the shared
// product's weights are read while the rank values are still being summed, and so
// are the adapters' factors, as each CTA makes its tile's plan itself.  64 rows of
// 64 adapters (4096 x 4096, rank 16, BF16): 22 us for both, 16 of them this kernel,
// for 43 MB (FP16, whose factors a warp splits in two: 26 to 29).
//
// For few it makes the rank values itself (OWN): the first factors F of up to eight
// adapters come with the K steps of W, and X is multiplied by both; the shares of a
// cluster are added by the CTA to which a row's adapter is dealt, the only one that
// needs them.  Every column tile then sums the same rank values, so the choice goes by
// adapters x K steps of a CTA.  Measured, two kernels against one (BF16, us): 4
// adapters x 4 steps 12.0 and 12.0, 3 x 8 17.2 and 18.1, 16 x 2 13.1 and 14.7, 8 x 8
// 14.9 and 19.6, 16 x 8 16.5 and 27; but a call from Python takes 24 us of
// the host's time with two and 17 with one, which needs no workspace either.  Up to
// 32 take one kernel.
#include <algorithm>
#include <cstring>

#include "grouped_maps.h"
#include "lora_tc.cuh"
#include "persistent.cuh"

namespace tmmo {
namespace {

// warps 0: copies, 1: MMA, 2: rank values, 3: FP16 factors in two, 4-7: plan, accumulators
constexpr int LM_THREADS = 256;
constexpr int LM_MAX_STAGES = 8;
constexpr int LM_RING = 200 * 1024;
constexpr int LM_RING_SHARED = 120 * 1024;  // leaves room for the shrink's kernel on the SM
constexpr int LM_PITCH = 132;    // of the sums in shared memory: rows 16 bytes apart in the banks
constexpr int LM_HELD = 16384;   // a tile's rank values in parts, of one chunk
constexpr int LM_FACTORS = 16384;  // factors of F beside a K step of W, at most
constexpr int LM_OWN_STEPS = 32;
static_assert(LM_OWN_STEPS <= 2 * LT_SEGMENT, "two accumulators");
constexpr int LM_OWN_SECOND = 384;  // OWN: tensor memory of a second accumulator
constexpr int LM_THIN = LT_ROWS * (32 + 4) * 4;  // a CTA's share of their sums

struct SmallParams {
    int M, N, k_blocks, rank;
    int segment;             // K steps that one accumulator adds up
    int tmem_cols;
    int tiles_n;
    bool one;
    int adapters;
    LoraParts lay;
    const int32_t* adapter;
    void* C;
    int64_t ldc;
    uint32_t idesc;
    int box_rows;            // rows of X that a copy brings
    int stages, stage_bytes, ring;
    bool words;              // 16-byte stores
    int out_dtype;
    // Adapters of one chunk of rank values: the tile's rank values stay in shared
    // memory (behind the ring), and a stage holds the factors of several adapters,
    // rows of 32 or 64 bytes (width); 0: an adapter a stage, with the rank values.
    int beside;
    uint32_t width;
    bool split;              // FP16 factors, split in two (lora_tc.cuh)
    uint32_t idesc_e;        // of the adapters' products: BF16
    // Where the kernel makes the rank values: rows of X times the factors F
    const float* scale;
    bool one_f;
    int together;            // adapters whose factors come with a K step of W
    int extra;               // further ones share a stage of X and factors
    int w_bytes;             // of a stage before X: W, factors
    int chains;              // accumulators that K steps take in turn (see lora_shrink.cu)
    uint32_t idesc_t;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

struct SmallSmem {
    uint64_t full[LM_MAX_STAGES], empty[LM_MAX_STAGES], planned, held, done, thin, thin_all;
    uint64_t landed[LM_MAX_STAGES];  // of steps whose factors are to be split
    uint64_t segment, taken;         // a segment's sums are there, are added
    uint32_t tmem;
    int abort_flag;
    int progress;  // steps copied
    PlanScratch scratch;
    LoraPlan plan;
};

// Eight values of a row, of which the first n exist; words: p is on a 16-byte
// boundary.
template <typename T>
__device__ __forceinline__ void store_eight(T* p, const float (&v)[8], int n, bool words)
{
    alignas(16) T h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        put(&h[i], v[i]);
    if (words && n >= 8) {
        uint4 w[sizeof(T) / 2];
        memcpy(w, h, sizeof h);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
            reinterpret_cast<uint4*>(p)[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = h[i];
    }
}

// Descriptor of a K-major operand whose rows are 32, 64 or 128 bytes.
__device__ __forceinline__ uint64_t smem_desc_rows(uint32_t addr, uint32_t width)
{
    const uint64_t mode = width == 128 ? 2 : width == 64 ? 4 : 6;
    return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | 1ull << 16 |
           static_cast<uint64_t>(8 * width >> 4) << 32 | 1ull << 46 | mode << 61;
}

// store(C) with C as a pointer to the output's type.
template <typename Store>
__device__ __forceinline__ void with_output(const SmallParams& p, Store&& store)
{
    if (p.out_dtype == DT_F32)
        store(static_cast<float*>(p.C));
    else if (p.out_dtype == DT_F16)
        store(static_cast<__half*>(p.C));
    else
        store(static_cast<__nv_bfloat16*>(p.C));
}

// OWN: the rank values are made here, tmT being the map of the factors F.
template <bool ACROSS, int SPLITS, bool OWN>
__global__ void __launch_bounds__(LM_THREADS, 1)
    lora_small_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmT, const __grid_constant__ CUtensorMap tmE,
                      const __grid_constant__ SmallParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                     ~static_cast<uintptr_t>(1023));
    const uint32_t ring = smem_u32(base);
    __shared__ SmallSmem s;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const int split = SPLITS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tile = blockIdx.x / SPLITS;
    const int mb = tile / p.tiles_n, nb = tile % p.tiles_n;
    const int row0 = mb * LT_ROWS, col0 = nb * 128;
    const int per = (p.k_blocks + SPLITS - 1) / SPLITS;
    const int kb0 = split * per, kb1 = min(kb0 + per, p.k_blocks);
    const TcWatch watch{&s.abort_flag, p.status, p.wait_budget};
    // each row's adapter, asked for before anything else
    const int g = warp >= 4 && p.adapters > 0
                      ? row_adapter(p.adapter, row0 + static_cast<int>(threadIdx.x) - 128, p.M, p.adapters)
                      : -1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(smem_u32(&s.full[i]), OWN ? 2 : 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
            mbar_init(smem_u32(&s.landed[i]), 1);
        }
        mbar_init(smem_u32(&s.planned), 128);
        mbar_init(smem_u32(&s.held), OWN ? 4 : 1);
        mbar_init(smem_u32(&s.done), 1);
        mbar_init(smem_u32(&s.segment), 1);
        mbar_init(smem_u32(&s.taken), 4);
        mbar_init(smem_u32(&s.thin), 1);
        mbar_init(smem_u32(&s.thin_all), 4 * SPLITS);
        s.abort_flag = 0;
        s.progress = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmT);
        tma_prefetch_desc(&tmE);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&s.tmem), p.tmem_cols);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (OWN && SPLITS > 1)
        cluster_arrive();  // (waited for before another CTA's barrier is touched)
    const uint32_t tmem = s.tmem;
    const uint32_t a_bytes = p.box_rows * 128;
    // The contraction goes in segments.  Their sums are added in tensor memory, behind
    // the accumulator; the kernel that makes the rank values too, whose warps are not free for
    // that, has two at most, in accumulators of their own.
    const int segments = (kb1 - kb0 + p.segment - 1) / p.segment;
    const uint32_t second = tmem + (OWN ? LM_OWN_SECOND : 128);
    const uint32_t held = ring + p.ring;  // the tile's rank values
    float* const thin = reinterpret_cast<float*>(base + p.ring + LM_HELD);  // shares of their sums
    volatile int* const progress = &s.progress;

    if (warp == 0) {
        int stage = 0, n = 0;
        uint32_t phase = 0;
        uint32_t to_split = 0, parity = 0;  // stages that last landed on their own barrier; how often
        // split_e: the step's factors are to be split
        auto step = [&](bool skip, bool split_e, uint32_t bytes, auto load) {
            if (!warp_wait(smem_u32(&s.empty[stage]), phase ^ 1, watch))
                return false;
            if (p.split && lane == 0)
                *progress = n + 1;
            to_split = split_e ? to_split | 1u << stage : to_split & ~(1u << stage);
            parity ^= static_cast<uint32_t>(split_e) << stage;
            if (!skip) {
                const uint32_t bar = smem_u32(split_e ? &s.landed[stage] : &s.full[stage]);
                if (elect_one()) {
                    if (OWN && !split_e)
                        mbar_arrive(bar);
                    mbar_arrive_expect_tx(bar, bytes);
                    load(ring + stage * p.stage_bytes + p.w_bytes, ring + stage * p.stage_bytes, bar);
                }
                __syncwarp();
            }
            ++n;
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1;
            }
            return true;
        };
        bool ok = true;
        auto shared_product = [&](int kb, uint32_t dA, uint32_t dB, uint32_t bar) {
            if (ACROSS) {
                tma_load_2d(dB, &tmW, bar, col0, kb * TC_BK);
                tma_load_2d(dB + 8192, &tmW, bar, col0 + 64, kb * TC_BK);
            } else {
                tma_load_2d(dB, &tmW, bar, kb * TC_BK, col0);
            }
            tma_load_2d(dA, &tmX, bar, kb * TC_BK, row0);
        };
        if constexpr (OWN) {
            // W and X need no plan: the first steps' factors follow when it is there.
            const uint32_t each = p.lay.chunk * 128;
            const int ahead = min(p.stages, kb1 - kb0);
            auto factors = [&](int a, int some, int kb, uint32_t to, uint32_t bar) {
                for (int i = 0; i < some; ++i)
                    tma_load_3d(to + i * each, &tmT, bar, kb * TC_BK, 0, p.one_f ? 0 : s.plan.ids[a + i]);
            };
            if (elect_one())
                for (int i = 0; i < ahead; ++i) {
                    if (kb0 + i == p.fault_skip_kblock)
                        continue;
                    const uint32_t bar = smem_u32(&s.full[i]), dB = ring + i * p.stage_bytes;
                    mbar_arrive_expect_tx(bar, a_bytes + 16384);
                    shared_product(kb0 + i, dB + p.w_bytes, dB, bar);
                }
            __syncwarp();
            ok = warp_wait(smem_u32(&s.planned), 0, watch);
            const int some = ok ? min(p.together, s.plan.count) : 0;
            if (elect_one())
                for (int i = 0; i < ahead; ++i) {
                    if (kb0 + i == p.fault_skip_kblock)
                        continue;
                    const uint32_t bar = smem_u32(&s.full[i]);
                    mbar_arrive_expect_tx(bar, some * each);
                    factors(0, some, kb0 + i, ring + i * p.stage_bytes + 16384, bar);
                }
            __syncwarp();
            n = ahead;
            stage = ahead % p.stages;
            phase = ahead / p.stages;
            for (int kb = kb0 + ahead; ok && kb < kb1; ++kb)
                ok = step(kb == p.fault_skip_kblock, false, a_bytes + 16384 + some * each,
                          [&](uint32_t dA, uint32_t dB, uint32_t bar) {
                              shared_product(kb, dA, dB, bar);
                              factors(0, some, kb, dB + 16384, bar);
                          });
            for (int a = p.together; ok && a < s.plan.count; a += p.extra) {
                const int more = min(p.extra, s.plan.count - a);
                for (int kb = kb0; ok && kb < kb1; ++kb)
                    ok = step(false, false, a_bytes + more * each, [&](uint32_t dA, uint32_t dB, uint32_t bar) {
                        tma_load_2d(dA, &tmX, bar, kb * TC_BK, row0);
                        factors(a, more, kb, dB, bar);
                    });
            }
        } else {
            for (int kb = kb0; ok && kb < kb1; ++kb)
                ok = step(kb == p.fault_skip_kblock, false, a_bytes + 16384,
                          [&](uint32_t dA, uint32_t dB, uint32_t bar) { shared_product(kb, dA, dB, bar); });
        }
        if (ok && p.adapters > 0) {
            ok = warp_wait(smem_u32(&s.planned), 0, watch);
            if (!ACROSS && p.beside > 0) {
                for (int a = split; ok && a < s.plan.count; a += p.beside * SPLITS) {
                    const int some = min(p.beside, (s.plan.count - a + SPLITS - 1) / SPLITS);
                    const uint32_t each = p.width * 128;
                    ok = step(false, p.split, some * each, [&](uint32_t, uint32_t dB, uint32_t bar) {
                        for (int i = 0; i < some; ++i)
                            tma_load_3d(dB + i * each, &tmE, bar, 0, col0,
                                        p.one ? 0 : s.plan.ids[a + i * SPLITS]);
                    });
                }
            } else {
                grid_dep_wait();  // the rank values come with the factors
                for (int a = split; ok && a < s.plan.count; a += SPLITS) {
                    const int z = p.one ? 0 : s.plan.ids[a];
                    for (int c = 0; ok && c < p.lay.chunks; ++c) {
                        const int j = c * p.lay.chunk;
                        ok = step(false, p.split, a_bytes + 16384, [&](uint32_t dA, uint32_t dB, uint32_t bar) {
                            if (ACROSS) {
                                tma_load_3d(dB, &tmE, bar, col0, j, z);
                                tma_load_3d(dB + 8192, &tmE, bar, col0 + 64, j, z);
                            } else {
                                tma_load_3d(dB, &tmE, bar, j, col0, z);
                            }
                            tma_load_2d(dA, &tmT, bar, c * 64, row0);
                        });
                    }
                }
            }
        }
        if (!ok && lane == 0) {  // wait (bounded) for the copies in flight before shared memory goes away
            for (int i = 0; i < p.stages; ++i) {
                const int uses = n / p.stages + (i < n % p.stages);
                const bool own = (to_split >> i) & 1;
                const uint32_t bar = smem_u32(own ? &s.landed[i] : &s.full[i]);
                const uint32_t phase_of = own ? ((parity >> i) & 1) ^ 1 : (uses - 1) & 1;
                const long long t0 = clock64();
                while (uses > 0 && !mbar_try_wait(bar, phase_of) && clock64() - t0 < p.wait_budget) {
                }
            }
        }
    } else if (warp == 1) {
        int stage = 0;
        uint32_t phase = 0;
        auto step = [&](auto multiply) {
            if (!warp_wait(smem_u32(&s.full[stage]), phase, watch))
                return false;
            tc_fence_after();
            if (elect_one()) {
                multiply(ring + stage * p.stage_bytes + p.w_bytes, ring + stage * p.stage_bytes);
                tc_commit(smem_u32(&s.empty[stage]));
            }
            __syncwarp();
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1;
            }
            return true;
        };
        bool ok = true;
        auto others = [&](int a, uint32_t (&off)[4]) {
            const uint4 rows = *reinterpret_cast<const uint4*>(s.plan.rows[a]);
            off[0] = ~rows.x;
            off[1] = ~rows.y;
            off[2] = ~rows.z;
            off[3] = ~rows.w;
        };
        // rows of X times the factors of adapters a .. a + some - 1
        auto rank_values = [&](int a, int some, int kb, uint32_t a0, uint32_t b0) {
            const uint32_t to = tmem + 128 + (kb - kb0) % p.chains * p.lay.chunk;
            for (int i = 0; i < some; ++i, b0 += p.lay.chunk * 128) {
                uint32_t off[4];
                others(a + i, off);
#pragma unroll
                for (int k = 0; k < TC_BK / TC_UMMA_K; ++k)
                    tc_mma_f16_lanes(to, smem_desc_sw128(a0 + k * 32, 16, 1024),
                                     smem_desc_sw128(b0 + k * 32, 16, 1024), p.idesc_t,
                                     kb - kb0 >= p.chains || k != 0, off);
            }
        };
        int some = 0;  // adapters whose factors come with W
        if constexpr (OWN) {
            ok = warp_wait(smem_u32(&s.planned), 0, watch);
            some = min(p.together, s.plan.count);
        }
        uint32_t acc = tmem;
        for (int n = 0; ok && n < segments; ++n) {
            if (OWN && n > 0)
                acc = second;
            if (!OWN && n > 0) {
                if (elect_one())
                    tc_commit(smem_u32(&s.segment));
                __syncwarp();
                ok = warp_wait(smem_u32(&s.taken), (n - 1) & 1, watch);
                tc_fence_after();
            }
            const int begin = kb0 + n * p.segment, end = min(begin + p.segment, kb1);
            for (int kb = begin; ok && kb < end; ++kb)
                ok = step([&](uint32_t a0, uint32_t b0) {
#pragma unroll
                    for (int k = 0; k < TC_BK / TC_UMMA_K; ++k)
                        tc_mma_f16<1>(acc, smem_desc_sw128(a0 + k * 32, 16, 1024),
                                      ACROSS ? smem_desc_sw128(b0 + k * 2048, 8192, 1024)
                                             : smem_desc_sw128(b0 + k * 32, 16, 1024),
                                      p.idesc, kb != begin || k != 0);
                    if constexpr (OWN)
                        rank_values(0, some, kb, a0, b0 + 16384);
                });
        }
        if constexpr (OWN) {
            for (int a = p.together; ok && a < s.plan.count; a += p.extra)
                for (int kb = kb0; ok && kb < kb1; ++kb)
                    ok = step([&](uint32_t a0, uint32_t b0) {
                        rank_values(a, min(p.extra, s.plan.count - a), kb, a0, b0);
                    });
            if (elect_one())
                tc_commit(smem_u32(&s.thin));
            __syncwarp();
        }
        if (ok && p.adapters > 0) {
            ok = warp_wait(smem_u32(&s.planned), 0, watch);
            if (!ACROSS && p.beside > 0) {
                const int deep = p.lay.deep(0, p.rank);
                grid_dep_wait();  // (so that no wait spans the kernel before)
                ok = ok && warp_wait(smem_u32(&s.held), 0, watch);
                for (int a = split; ok && a < s.plan.count; a += p.beside * SPLITS)
                    ok = step([&](uint32_t, uint32_t b0) {
                        const int some = min(p.beside, (s.plan.count - a + SPLITS - 1) / SPLITS);
                        for (int i = 0; i < some; ++i, b0 += p.width * 128) {
                            uint32_t off[4];
                            others(a + i * SPLITS, off);
                            each_product(p.lay, deep, p.split, [&](int part, int pair, int k) {
                                const int b = pair * p.lay.chunk / 16 + k;
                                tc_mma_f16_lanes(
                                    acc, smem_desc_sw128(held + part * p.lay.chunk * 2 + k * 32, 16, 1024),
                                    smem_desc_rows(b0 + b * 32, p.width), p.idesc_e, 1, off);
                            });
                        }
                    });
            } else {
                grid_dep_wait();
                for (int a = split; ok && a < s.plan.count; a += SPLITS) {
                    uint32_t off[4];
                    others(a, off);
                    for (int c = 0; ok && c < p.lay.chunks; ++c)
                        ok = step([&](uint32_t a0, uint32_t b0) {
                            each_product(p.lay, p.lay.deep(c, p.rank), p.split, [&](int part, int pair, int k) {
                                const int b = pair * p.lay.chunk / 16 + k;
                                tc_mma_f16_lanes(
                                    acc, smem_desc_sw128(a0 + part * p.lay.chunk * 2 + k * 32, 16, 1024),
                                    ACROSS ? smem_desc_sw128(b0 + b * 2048, 8192, 1024)
                                           : smem_desc_sw128(b0 + b * 32, 16, 1024),
                                    p.idesc_e, 1, off);
                            });
                        });
                }
            }
        }
        if (elect_one())
            tc_commit(smem_u32(&s.done));  // also after giving up: nothing may run on
        __syncwarp();
        const long long t0 = clock64();
        while (!mbar_try_wait(smem_u32(&s.done), 0) && clock64() - t0 < p.wait_budget) {
        }
    } else if (warp == 2 && p.adapters > 0 && !OWN) {
        grid_dep_wait();
        grid_dep_launch_dependents();  // the rank values are there for others, too
        if (!ACROSS && p.beside > 0) {
            if (elect_one()) {
                mbar_arrive_expect_tx(smem_u32(&s.held), a_bytes);
                tma_load_2d(held, &tmT, smem_u32(&s.held), 0, row0);
            }
            __syncwarp();
            // (also after the others gave up: nothing may land when this CTA is gone)
            warp_wait(smem_u32(&s.held), 0, watch);
        }
    } else if (warp == 3 && p.adapters > 0 && p.split) {
        grid_dep_wait();  // (so that no wait spans the kernel before)
        bool ok = warp_wait(smem_u32(&s.planned), 0, watch);
        const int count = ok ? s.plan.count : 0;
        int n = kb1 - kb0;  // steps before
        if (OWN && count > p.together)
            n += (count - p.together + p.extra - 1) / p.extra * (kb1 - kb0);
        uint32_t parity = 0;  // a bit for each stage
        // split(tile) of the next step's factors
        auto step = [&](auto split_tile) {
            const int stage = n++ % p.stages;
            // (the steps before are not waited for)
            if (!warp_wait_behind(smem_u32(&s.landed[stage]), (parity >> stage) & 1, watch, progress))
                return false;
            parity ^= 1u << stage;
            split_tile(ring + stage * p.stage_bytes);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&s.full[stage]));
                if (OWN)
                    mbar_arrive(smem_u32(&s.full[stage]));
            }
            return true;
        };
        if (!ACROSS && p.beside > 0) {
            for (int a = split; ok && a < count; a += p.beside * SPLITS)
                ok = step([&](uint32_t tile) {
                    split_rows(tile, 128 * min(p.beside, (count - a + SPLITS - 1) / SPLITS), p.width);
                });
        } else {
            for (int a = split; a < count; a += SPLITS)
                for (int c = 0; ok && c < p.lay.chunks; ++c)
                    ok = step([&](uint32_t tile) {
                        if (ACROSS)
                            split_across(tile, 2);
                        else
                            split_rows(tile, 128, 128);
                    });
        }
    } else if (warp >= 4 && p.adapters > 0) {
        const int place = make_plan(s.plan, s.scratch, g, threadIdx.x - 128, [] { bar_sync(1, 128); });
        mbar_arrive(smem_u32(&s.planned));
        if constexpr (OWN) {
            // This CTA's share of its rows' sums, and then the whole ones of the rows
            // whose adapters are dealt to it: each thread one row.
            const int row = threadIdx.x - 128, pitch = p.lay.chunk + 4;
            const float scale = p.scale && g >= 0 ? p.scale[g] : 1.0f;
            const uint32_t mine = smem_u32(thin + row * pitch);
            int ok = 1;
            if (lane == 0)
                ok = tc_wait(smem_u32(&s.thin), 0, patient(watch, p.k_blocks)) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (ok) {
                tc_fence_after();
                const int chains = min(p.chains, kb1 - kb0);
#pragma unroll 1
                for (int j = 0; j < p.lay.chunk; j += 16) {
                    const uint32_t from = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128 + j;
                    float v[16] = {};
#pragma unroll 1
                    for (int c = 0; c < chains; ++c) {
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(from + c * p.lay.chunk, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[i] += __uint_as_float(o[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        st_shared_v4(mine + (j + i) * 4, __float_as_uint(v[i]), __float_as_uint(v[i + 1]),
                                     __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
                }
            }
            __syncwarp();
            if constexpr (SPLITS > 1) {  // (also after giving up: the others need not wait)
                cluster_wait();
                if (static_cast<int>(lane) < SPLITS)
                    mbar_arrive_cluster(mapa_shared(smem_u32(&s.thin_all), lane));
                __syncwarp();
                warp_wait<true>(smem_u32(&s.thin_all), 0, watch);
            }
            if (place >= 0 && place % SPLITS == split) {
                uint32_t peer[SPLITS];
#pragma unroll
                for (int k = 0; k < SPLITS; ++k)
                    peer[k] = SPLITS > 1 ? mapa_shared(mine, k) : mine;
#pragma unroll 1
                for (int j = 0; j < p.lay.chunk; j += 8) {
                    float sum[8] = {};
                    float4 v[SPLITS][2];
#pragma unroll
                    for (int k = 0; k < SPLITS; ++k)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            v[k][h] = ld_cluster_v4(peer[k] + j * 4 + 16 * h);
#pragma unroll
                    for (int k = 0; k < SPLITS; ++k)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            sum[4 * h] += v[k][h].x;
                            sum[4 * h + 1] += v[k][h].y;
                            sum[4 * h + 2] += v[k][h].z;
                            sum[4 * h + 3] += v[k][h].w;
                        }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sum[i] = j + i < p.rank ? scale * sum[i] : 0.0f;
                    auto store = [&](int part, const uint4& w) {  // 128-byte rows, swizzled
                        const uint32_t at = (part * p.lay.chunk + j) / 8;
                        st_shared_v4(held + row * 128 + ((at ^ (row & 7)) << 4), w.x, w.y, w.z, w.w);
                    };
                    each_part(sum, p.lay.parts, store);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&s.held));
        }
    }
    // The sums to shared memory; the ring holds nothing any more.
    __syncwarp();
    const int rows = min(LT_ROWS, p.M - row0);
    float* sums = reinterpret_cast<float*>(base);
    if (warp >= 4) {
        const int q = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        int ok = 1;
        for (int n = 0; !OWN && n + 1 < segments; ++n) {
            if (!warp_wait(smem_u32(&s.segment), n & 1, watch))
                break;
            tc_fence_after();
            add_to_sums(tmem + lanes, 1, second + lanes, 128, n == 0, true);
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&s.taken));
        }
        if (p.adapters > 0)
            grid_dep_wait();  // (so that no wait spans the kernel before)
        if (lane == 0)
            ok = tc_wait(smem_u32(&s.done), 0, patient(watch, p.k_blocks)) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (ok && q * 32 < rows) {
            tc_fence_after();
            const uint32_t to = smem_u32(sums + (q * 32 + lane) * LM_PITCH);
#pragma unroll 1
            for (int j = 0; j < 128; j += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + lanes + j, v);
                tmem_wait_ld(v);
                if (segments > 1) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(second + lanes + j, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(v[i]));
                }
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    st_shared_v4(to + (j + i) * 4, v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
        }
        tc_fence_before();
    }
    if (p.adapters > 0)
        grid_dep_wait();  // this grid must not end before the one it depends on
    if constexpr (OWN && SPLITS > 1)
        if (warp < 4)
            cluster_wait();
    if constexpr (SPLITS > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc<1>(tmem, p.tmem_cols);
    // (a lane asks each CTA: a loop would wait for one answer after another)
    int gave_up = s.abort_flag;
    if (SPLITS > 1 && static_cast<int>(lane) < SPLITS)
        gave_up = __float_as_int(ld_cluster_f32(mapa_shared(smem_u32(&s.abort_flag), lane)));
    // Each CTA adds up and stores its share: sixteen rows at a time, eight columns a
    // thread.
    const int col = (threadIdx.x & 15) * 8, cols = p.N - col0 - col;
    uint32_t peer[SPLITS];
#pragma unroll
    for (int k = 0; k < SPLITS; ++k) {
        const uint32_t at = smem_u32(sums + col);
        peer[k] = SPLITS > 1 ? mapa_shared(at, k) : at;
    }
#pragma unroll 1
    for (int r0 = 16 * split; r0 < rows; r0 += 16 * SPLITS) {
        const int r = r0 + (threadIdx.x >> 4);  // (rows behind the last: whatever is there)
        float4 v[SPLITS][2];
#pragma unroll
        for (int k = 0; k < SPLITS; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                v[k][h] = ld_cluster_v4(peer[k] + r * LM_PITCH * 4 + 16 * h);
        if (__any_sync(0xffffffffu, gave_up))
            break;
        float sum[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 a = v[0][h];
#pragma unroll
            for (int k = 1; k < SPLITS; ++k) {
                a.x += v[k][h].x;
                a.y += v[k][h].y;
                a.z += v[k][h].z;
                a.w += v[k][h].w;
            }
            sum[4 * h] = a.x;
            sum[4 * h + 1] = a.y;
            sum[4 * h + 2] = a.z;
            sum[4 * h + 3] = a.w;
        }
        if (r < rows && cols > 0)
            with_output(p, [&](auto* c) { store_eight(c + (row0 + r) * p.ldc + col0 + col, sum, cols, p.words); });
    }
    if constexpr (SPLITS > 1) {
        __syncwarp();
        cluster_sync();  // nobody leaves while others read its sums
    }
}

// Sets the kernel up, once; how many of its clusters run at a time.
template <bool ACROSS, bool OWN, int SPLITS>
cudaError_t most_clusters(int num_sms, int* cap)
{
    static ClusterCaps caps;
    return cluster_cap(lora_small_kernel<ACROSS, SPLITS, OWN>, caps, SPLITS, LM_THREADS, LM_RING + 1024,
                       num_sms, cap);
}

template <bool ACROSS, bool OWN, int SPLITS>
cudaError_t launch(const CUtensorMap (&m)[4], const SmallParams& p, int tiles, cudaStream_t stream)
{
    ClusterLaunch l(static_cast<unsigned>(tiles * SPLITS), SPLITS, LM_THREADS,
                    p.ring + (p.beside ? LM_HELD : 0) + (OWN ? LM_THIN : 0) + 1024, stream,
                    p.adapters > 0 && !OWN);
    return l.run(lora_small_kernel<ACROSS, SPLITS, OWN>, m[0], m[1], m[2], m[3], p);
}

template <bool ACROSS, bool OWN>
cudaError_t launch(const CUtensorMap (&m)[4], const SmallParams& p, int tiles, int splits, cudaStream_t stream)
{
    switch (splits) {
    case 1:
        return launch<ACROSS, OWN, 1>(m, p, tiles, stream);
    case 2:
        return launch<ACROSS, OWN, 2>(m, p, tiles, stream);
    case 4:
        return launch<ACROSS, OWN, 4>(m, p, tiles, stream);
    default:
        return launch<ACROSS, OWN, 8>(m, p, tiles, stream);
    }
}

int64_t small_tiles(int64_t rows, int64_t N)
{
    return (rows + LT_ROWS - 1) / LT_ROWS * ((N + 127) / 128);
}

// CTAs for every SM, none without a K step, in clusters that run all at once: 15 of
// eight CTAs fit the 152 SMs (a cluster's lie in one GPC), 36 of four.  128 rows
// by 2048 outputs (16 tiles, K = 1024) took 24 us in eights, and take 13 in fours.
template <bool ACROSS, bool OWN>
cudaError_t small_splits(int64_t tiles, int64_t k_blocks, int num_sms, int* splits)
{
    static SplitCaps known;
    const int* cap = nullptr;
    const cudaError_t err = split_caps(known, [&](int i, int* n) {
        return i == 0   ? most_clusters<ACROSS, OWN, 1>(num_sms, n)
               : i == 1 ? most_clusters<ACROSS, OWN, 2>(num_sms, n)
               : i == 2 ? most_clusters<ACROSS, OWN, 4>(num_sms, n)
                        : most_clusters<ACROSS, OWN, 8>(num_sms, n);
    }, &cap);
    if (err != cudaSuccess)
        return err;
    *splits = 1;
    for (int i = 1; i < 4; ++i) {
        const int64_t n = 1 << i, per = (k_blocks + n - 1) / n;
        if (tiles > cap[i] || (n - 1) * per >= k_blocks)
            break;
        *splits = 1 << i;
    }
    return cudaSuccess;
}

// own: with rank values made by the kernel
cudaError_t launch_small(const LoraLaunch& l, bool own, cudaStream_t stream)
{
    SmallParams p{};
    p.M = l.rows;
    p.N = l.N;
    p.k_blocks = (l.K + TC_BK - 1) / TC_BK;
    p.rank = l.rank;
    p.tiles_n = (l.N + 127) / 128;
    p.adapters = l.adapters;
    p.one = l.adapters == 1 || l.stride_e == 0;
    p.lay = lora_parts(l.rank, l.parts);
    p.adapter = l.adapter;
    p.C = l.Y;
    p.ldc = l.ldy;
    p.out_dtype = l.out_dtype;
    p.words = aligned_rows(l.Y, l.ldy, l.out_dtype);
    const bool bf16 = l.in_dtype == DT_BF16;
    p.idesc = tc_idesc(bf16, LT_ROWS, 128, false, l.across);
    p.box_rows = std::min(LT_ROWS, (l.rows + 7) / 8 * 8);
    p.split = !bf16;
    p.idesc_e = tc_idesc(true, LT_ROWS, 128, false, l.across);
    p.width = static_cast<uint32_t>(p.lay.chunk * (p.split ? 4 : 2));
    p.beside = p.adapters && !l.across && p.lay.chunks == 1 ? static_cast<int>(16384 / (p.width * 128)) : 0;
    p.w_bytes = 16384;
    if (own) {
        const int each = p.lay.chunk * 128;
        p.scale = l.scale;
        p.one_f = l.adapters == 1 || l.stride_f == 0;
        p.together = std::min(std::min(l.adapters, l.rows), LM_FACTORS / each);
        p.w_bytes += p.together * each;
        p.extra = p.w_bytes / each;
        p.chains = 8;
        p.idesc_t = tc_idesc(bf16, LT_ROWS, p.lay.chunk, false, false);
    }
    p.stage_bytes = p.w_bytes + (p.box_rows * 128 + 1023) / 1024 * 1024;
    p.ring = !l.across && !own && lora_shrink_shares(l) ? LM_RING_SHARED : LM_RING;
    p.ring -= (p.beside ? LM_HELD : 0) + (own ? LM_THIN : 0);
    // The tensor core reads 128 rows of A whatever a copy brings: what follows
    // lies within the ring too (those lanes are not used).
    p.stages = std::min(LM_MAX_STAGES, (p.ring - p.w_bytes - 16384) / p.stage_bytes + 1);
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip_kblock = l.fault_skip_kblock;
    CUtensorMap m[4];
    const int dt = l.in_dtype;
    const uint32_t box = static_cast<uint32_t>(p.box_rows), chunk = static_cast<uint32_t>(p.lay.chunk);
    bool ok = l.maps->get(&m[0], dt, l.X, 2, {l.K, l.rows, 1}, {l.ldx, 0}, {64, box, 1}) &&
              (l.across ? l.maps->get(&m[1], dt, l.W, 2, {l.N, l.K, 1}, {l.ldw, 0}, {64, TC_BK, 1})
                        : l.maps->get(&m[1], dt, l.W, 2, {l.K, l.N, 1}, {l.ldw, 0}, {64, 128, 1}));
    m[2] = m[3] = m[0];
    if (ok && p.adapters > 0) {
        const int64_t stacked = p.one ? 1 : l.adapters, stride = p.one ? l.lde : l.stride_e;
        ok = (own ? l.maps->get(&m[2], dt, l.F, 3, {l.K, l.rank, p.one_f ? 1 : l.adapters},
                                {l.ldf, p.one_f ? l.ldf : l.stride_f}, {64, chunk, 1})
                  : l.maps->get(&m[2], DT_BF16, l.t, 2, {p.lay.columns(), l.rows, 1}, {p.lay.columns(), 0},
                                {64, box, 1})) &&
             (l.across ? l.maps->get(&m[3], dt, l.E, 3, {l.N, l.rank, stacked}, {l.lde, stride}, {64, TC_BK, 1})
                       : l.maps->get(&m[3], dt, l.E, 3, {l.rank, l.N, stacked}, {l.lde, stride},
                                    {p.beside ? p.width / 2 : 64u, 128, 1}));
    }
    if (!ok)
        return cudaErrorNotSupported;
    const int tiles = static_cast<int>(small_tiles(l.rows, l.N));
    int splits = 1;
    const cudaError_t err = l.across ? small_splits<true, false>(tiles, p.k_blocks, l.num_sms, &splits)
                            : own    ? small_splits<false, true>(tiles, p.k_blocks, l.num_sms, &splits)
                                     : small_splits<false, false>(tiles, p.k_blocks, l.num_sms, &splits);
    if (err != cudaSuccess)
        return err;
    const int per = (p.k_blocks + splits - 1) / splits, segments = (per + LT_SEGMENT - 1) / LT_SEGMENT;
    p.segment = (per + segments - 1) / segments;
    p.tmem_cols = own ? 512 : segments > 1 ? 256 : 128;
    return l.across ? launch<true, false>(m, p, tiles, splits, stream)
           : own    ? launch<false, true>(m, p, tiles, splits, stream)
                    : launch<false, false>(m, p, tiles, splits, stream);
}

}  // namespace

bool lora_small_takes(const LoraLaunch& l) { return small_tiles(l.rows, l.N) <= l.num_sms; }

bool lora_alone_takes(int64_t rows, int64_t N, int64_t K, int64_t adapters, int rank, int parts, int num_sms)
{
    const int64_t tiles = small_tiles(rows, N), k_blocks = (K + TC_BK - 1) / TC_BK;
    if (adapters == 0 || tiles > num_sms || lora_parts(rank, parts).chunks > 1)
        return false;
    int splits = 1;
    if (small_splits<false, true>(tiles, k_blocks, num_sms, &splits) != cudaSuccess)
        return false;
    const int64_t most = std::min(std::min(adapters, rows), static_cast<int64_t>(LT_ROWS));
    return most * ((k_blocks + splits - 1) / splits) <= LM_OWN_STEPS;
}

cudaError_t lora_small_tc_launch(const LoraLaunch& l, cudaStream_t stream) { return launch_small(l, false, stream); }
cudaError_t lora_alone_tc_launch(const LoraLaunch& l, cudaStream_t stream) { return launch_small(l, true, stream); }

}  // namespace tmmo
