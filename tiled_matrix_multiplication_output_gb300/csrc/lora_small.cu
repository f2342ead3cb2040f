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
// Launched as a programmatic dependent of the kernel that makes the rank values,
// and small enough to share an SM with it: the shared product's weights are read
// while the rank values are still being summed.
#include <algorithm>

#include "grouped_maps.h"
#include "lora_tc.cuh"
#include "persistent.cuh"

namespace tmmo {
namespace {

constexpr int LM_THREADS = 256;  // warps 0: copies, 1: MMA, 4-7: accumulator
constexpr int LM_MAX_STAGES = 8;
constexpr int LM_RING = 112 * 1024;
constexpr int LM_PITCH = 129;    // of the sums in shared memory

struct SmallParams {
    int M, N, k_blocks, rank;
    int tiles_n;
    bool adapters, one;
    LoraParts lay;
    const LoraPlan* plan;
    void* C;
    int64_t ldc;
    uint32_t idesc;
    int box_rows;            // rows of X that a copy brings
    int stages, stage_bytes;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

struct SmallSmem {
    uint64_t full[LM_MAX_STAGES], empty[LM_MAX_STAGES], done;
    uint32_t tmem;
    int abort_flag;
};

template <bool ACROSS, typename OutT>
__global__ void __launch_bounds__(LM_THREADS, 2)
    lora_small_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmT, const __grid_constant__ CUtensorMap tmE,
                      const __grid_constant__ SmallParams p, int splits)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                     ~static_cast<uintptr_t>(1023));
    const uint32_t ring = smem_u32(base);
    __shared__ SmallSmem s;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const int split = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tile = blockIdx.x / splits;
    const int mb = tile / p.tiles_n, nb = tile % p.tiles_n;
    const int row0 = mb * LT_ROWS, col0 = nb * 128;
    const int per = (p.k_blocks + splits - 1) / splits;
    const int kb0 = split * per, kb1 = min(kb0 + per, p.k_blocks);
    const TcWatch watch{&s.abort_flag, p.status, p.wait_budget};
    const LoraPlan& plan = p.plan[mb];

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(smem_u32(&s.full[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
        }
        mbar_init(smem_u32(&s.done), 1);
        s.abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmT);
        tma_prefetch_desc(&tmE);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&s.tmem), 128);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    const uint32_t a_bytes = p.box_rows * 128;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, n = 0;
            uint32_t phase = 0;
            auto step = [&](bool skip, auto load) {
                if (!tc_wait(smem_u32(&s.empty[stage]), phase ^ 1, watch))
                    return false;
                if (!skip) {
                    const uint32_t bar = smem_u32(&s.full[stage]);
                    mbar_arrive_expect_tx(bar, a_bytes + 16384);
                    load(ring + stage * p.stage_bytes + 16384, ring + stage * p.stage_bytes, bar);
                    ++n;
                }
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
                return true;
            };
            bool ok = true;
            for (int kb = kb0; ok && kb < kb1; ++kb)
                ok = step(kb == p.fault_skip_kblock, [&](uint32_t dA, uint32_t dB, uint32_t bar) {
                    if (ACROSS) {
                        tma_load_2d(dB, &tmW, bar, col0, kb * TC_BK);
                        tma_load_2d(dB + 8192, &tmW, bar, col0 + 64, kb * TC_BK);
                    } else {
                        tma_load_2d(dB, &tmW, bar, kb * TC_BK, col0);
                    }
                    tma_load_2d(dA, &tmX, bar, kb * TC_BK, row0);
                });
            if (ok && p.adapters) {
                grid_dep_wait();
                for (int a = split; ok && a < plan.count; a += splits) {
                    const int z = p.one ? 0 : plan.ids[a];
                    for (int c = 0; ok && c < p.lay.chunks; ++c) {
                        const int j = c * p.lay.chunk;
                        ok = step(false, [&](uint32_t dA, uint32_t dB, uint32_t bar) {
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
            if (!ok) {  // wait (bounded) for the copies in flight before shared memory goes away
                for (int i = 0; i < p.stages; ++i) {
                    const int uses = n / p.stages + (i < n % p.stages);
                    const long long t0 = clock64();
                    while (uses > 0 && !mbar_try_wait(smem_u32(&s.full[i]), (uses - 1) & 1) &&
                           clock64() - t0 < p.wait_budget) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            auto step = [&](auto multiply) {
                if (!tc_wait(smem_u32(&s.full[stage]), phase, watch))
                    return false;
                tc_fence_after();
                multiply(ring + stage * p.stage_bytes + 16384, ring + stage * p.stage_bytes);
                tc_commit(smem_u32(&s.empty[stage]));
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
                return true;
            };
            bool ok = true;
            for (int kb = kb0; ok && kb < kb1; ++kb)
                ok = step([&](uint32_t a0, uint32_t b0) {
#pragma unroll
                    for (int k = 0; k < TC_BK / TC_UMMA_K; ++k)
                        tc_mma_f16<1>(tmem, smem_desc_sw128(a0 + k * 32, 16, 1024),
                                      ACROSS ? smem_desc_sw128(b0 + k * 2048, 8192, 1024)
                                             : smem_desc_sw128(b0 + k * 32, 16, 1024),
                                      p.idesc, kb != kb0 || k != 0);
                });
            if (ok && p.adapters) {
                grid_dep_wait();
                for (int a = split; ok && a < plan.count; a += splits) {
                    uint32_t off[4];
                    for (int w = 0; w < 4; ++w)
                        off[w] = ~plan.rows[a][w];
                    for (int c = 0; ok && c < p.lay.chunks; ++c)
                        ok = step([&](uint32_t a0, uint32_t b0) {
                            const int deep = p.lay.deep(c, p.rank);
                            for (int part = 0; part < p.lay.parts; ++part)
                                for (int k = 0; k < deep; ++k)
                                    tc_mma_f16_lanes(
                                        tmem, smem_desc_sw128(a0 + part * p.lay.chunk * 2 + k * 32, 16, 1024),
                                        ACROSS ? smem_desc_sw128(b0 + k * 2048, 8192, 1024)
                                               : smem_desc_sw128(b0 + k * 32, 16, 1024),
                                        p.idesc, 1, off);
                        });
                }
            }
            tc_commit(smem_u32(&s.done));  // also after giving up: nothing may run on
            const long long t0 = clock64();
            while (!mbar_try_wait(smem_u32(&s.done), 0) && clock64() - t0 < p.wait_budget) {
            }
        }
    }
    // The sums to shared memory; the ring holds nothing any more.
    __syncwarp();
    const int rows = min(LT_ROWS, p.M - row0);
    float* sums = reinterpret_cast<float*>(base);
    if (warp >= 4) {
        const int q = warp & 3;
        int ok = 1;
        if (lane == 0)
            ok = tc_wait(smem_u32(&s.done), 0, watch) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (ok && q * 32 < rows) {
            tc_fence_after();
            float* to = sums + (q * 32 + lane) * LM_PITCH;
#pragma unroll 1
            for (int j = 0; j < 128; j += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + j, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    to[j + i] = __uint_as_float(v[i]);
            }
        }
        tc_fence_before();
    }
    if (p.adapters)
        grid_dep_wait();  // this grid must not end before the one it depends on
    if (splits > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc<1>(tmem, 128);
    int gave_up = s.abort_flag;
    for (int k = 0; k < splits && splits > 1; ++k)
        gave_up |= __float_as_int(ld_cluster_f32(mapa_shared(smem_u32(&s.abort_flag), k)));
    // Each CTA adds up and stores its share: two rows at a time, with the
    // columns along the threads.
    const int col = threadIdx.x & 127;
    OutT* out = static_cast<OutT*>(p.C) + row0 * p.ldc + col0 + col;
    if (!gave_up && col0 + col < p.N)
        for (int r = 2 * split + (threadIdx.x >> 7); r < rows; r += 2 * splits) {
            float sum = 0.0f;
            if (splits == 1) {
                sum = sums[r * LM_PITCH + col];
            } else {
                const uint32_t at = smem_u32(&sums[r * LM_PITCH + col]);
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = k < splits ? ld_cluster_f32(mapa_shared(at, k)) : 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    sum += v[k];
            }
            put(out + r * p.ldc, sum);
        }
    if (splits > 1) {
        __syncwarp();
        cluster_sync();  // nobody leaves while others read its sums
    }
}

template <bool ACROSS, typename OutT>
cudaError_t launch(const CUtensorMap (&m)[4], const SmallParams& p, int tiles, int splits,
                   cudaStream_t stream)
{
    static ClusterCaps caps;
    int cap = 0;
    const cudaError_t err =
        cluster_cap(lora_small_kernel<ACROSS, OutT>, caps, 1, LM_THREADS, LM_RING + 1024, 1, &cap);
    if (err != cudaSuccess)
        return err;
    ClusterLaunch l(static_cast<unsigned>(tiles * splits), splits, LM_THREADS, LM_RING + 1024, stream,
                    p.adapters);
    return l.run(lora_small_kernel<ACROSS, OutT>, m[0], m[1], m[2], m[3], p, splits);
}

template <bool ACROSS>
cudaError_t launch(int out_dtype, const CUtensorMap (&m)[4], const SmallParams& p, int tiles, int splits,
                   cudaStream_t stream)
{
    switch (out_dtype) {
    case DT_F32:
        return launch<ACROSS, float>(m, p, tiles, splits, stream);
    case DT_F16:
        return launch<ACROSS, __half>(m, p, tiles, splits, stream);
    default:
        return launch<ACROSS, __nv_bfloat16>(m, p, tiles, splits, stream);
    }
}

int64_t small_tiles(const LoraLaunch& l)
{
    return (static_cast<int64_t>(l.rows) + LT_ROWS - 1) / LT_ROWS * ((l.N + 127) / 128);
}

}  // namespace

bool lora_small_takes(const LoraLaunch& l) { return small_tiles(l) <= l.num_sms; }

cudaError_t lora_small_tc_launch(const LoraLaunch& l, cudaStream_t stream)
{
    SmallParams p{};
    p.M = l.rows;
    p.N = l.N;
    p.k_blocks = (l.K + TC_BK - 1) / TC_BK;
    p.rank = l.rank;
    p.tiles_n = (l.N + 127) / 128;
    p.adapters = l.adapters > 0;
    p.one = l.adapters == 1 || l.stride_e == 0;
    p.lay = lora_parts(l.rank, l.parts);
    p.plan = static_cast<const LoraPlan*>(l.plan);
    p.C = l.Y;
    p.ldc = l.ldy;
    p.idesc = tc_idesc(l.in_dtype == DT_BF16, LT_ROWS, 128, false, l.across);
    p.box_rows = std::min(LT_ROWS, (l.rows + 7) / 8 * 8);
    p.stage_bytes = 16384 + (p.box_rows * 128 + 1023) / 1024 * 1024;
    // The tensor core reads 128 rows of A whatever a copy brings: what follows
    // lies within the ring too (those lanes are not used).
    p.stages = std::min(LM_MAX_STAGES, (LM_RING - 32768) / p.stage_bytes + 1);
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip_kblock = l.fault_skip_kblock;
    CUtensorMap m[4];
    const int dt = l.in_dtype;
    const uint32_t box = static_cast<uint32_t>(p.box_rows);
    bool ok = encode_map(&m[0], dt, l.X, 2, {l.K, l.rows, 1}, {l.ldx, 0}, {64, box, 1}) &&
              (l.across ? encode_map(&m[1], dt, l.W, 2, {l.N, l.K, 1}, {l.ldw, 0}, {64, TC_BK, 1})
                        : encode_map(&m[1], dt, l.W, 2, {l.K, l.N, 1}, {l.ldw, 0}, {64, 128, 1}));
    m[2] = m[3] = m[0];
    if (ok && p.adapters) {
        const int64_t stacked = p.one ? 1 : l.adapters, stride = p.one ? l.lde : l.stride_e;
        ok = encode_map(&m[2], dt, l.t, 2, {p.lay.columns(), l.rows, 1}, {p.lay.columns(), 0}, {64, box, 1}) &&
             (l.across ? encode_map(&m[3], dt, l.E, 3, {l.N, l.rank, stacked}, {l.lde, stride}, {64, TC_BK, 1})
                       : encode_map(&m[3], dt, l.E, 3, {l.rank, l.N, stacked}, {l.lde, stride}, {64, 128, 1}));
    }
    if (!ok)
        return cudaErrorNotSupported;
    // a CTA for every SM, none without a K step
    const int tiles = static_cast<int>(small_tiles(l));
    int splits = 1;
    auto fits = [&](int n) {
        const int per = (p.k_blocks + n - 1) / n;
        return n <= 8 && tiles * n <= l.num_sms && (n - 1) * per < p.k_blocks;
    };
    while (fits(2 * splits))
        splits *= 2;
    return l.across ? launch<true>(l.out_dtype, m, p, tiles, splits, stream)
                    : launch<false>(l.out_dtype, m, p, tiles, splits, stream);
}

}  // namespace tmmo
