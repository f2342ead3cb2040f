// The block-scaled 8-bit product for few output tiles: a few tokens against
// a weight matrix, or a small product of any form.
//
// With M tokens every byte of the weights is used for 2 M operations, so up
// to a few hundred tokens the bound is reading the weights from HBM, and for
// small weights the latency of a launch.  So:
//
//   * the longer outer axis (usually the weights' rows) is the tensor core's
//     128-row side and the shorter one its columns, 16, 32 or 64 of them: no
//     128-row tile is filled with padding for one token.  C is then written
//     transposed, which is coalesced, as a thread holds a row of the tile;
//   * a tile's K range is divided over a cluster of up to eight blocks, so
//     that every SM has weights in flight; each block keeps its FP32 sum in
//     registers, and the cluster adds the sums through distributed shared
//     memory in a fixed order -- one launch, no workspace, the same result
//     every run;
//   * a block's first copies are issued before anything else is set up, and
//     its ring holds 80 to 100 KiB, so that two blocks fit on an SM.
//
// The scaling of each K block's product is fp8_gemm_kernel's.  Measured on
// GB300, BF16 out: one token against 8192 x 8192 weights 14.0 us (4.8 TB/s
// with the launch, 0.71 of the measured copy bandwidth), 64 tokens 17.9; one
// against 4096 x 4096 6.0 to 6.3 (7.1 to 7.4 with weights that are not in L2),
// of which a launch alone is about 4.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fp8_gemm.cuh"
#include "fp8_launch.cuh"
#include "persistent.cuh"

namespace tmmo {
namespace {

constexpr int FS_THREADS = 256;  // warps 0: copies, 1: MMA, 2: scales, 3: herald, 4-7: epilogue
constexpr int FS_EPI_WARP0 = 4;
constexpr int FS_MAX_SPLITS = 8;

struct Fp8SmallParams {
    int rows, cols;                // of the tile's axes: rows of P, rows of Q
    int tiles_c;
    int k_blocks;
    uint32_t idesc;
    bool p_mn, q_mn;
    const float *sp, *sq;
    long long sp_k, sp_o, sq_k, sq_o;
    int sp_shift, sq_shift;
    void* C;
    long long c_row, c_col;        // elements from one row / column of the tile to the next in C
    bool by_row;                   // rows of the tile are rows of C
    int out_dtype;
    float alpha, beta;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

template <int BN>
struct Fp8SmallLayout {
    static constexpr int STAGES = BN == 64 ? 4 : 5;
    static constexpr int Q_BYTES = BN * F8_BK;
    static constexpr int STAGE = F8_BOX + Q_BYTES;
    static constexpr int NBUF = 4;
    static constexpr int GROUP = 4;                  // K blocks per scale slot
    static constexpr int SLOTS = 3;
    static constexpr int BLOCK_BYTES = (128 + BN) * 4;
    static constexpr int OFF_SCALE = STAGES * STAGE;
    static constexpr int OFF_BAR = OFF_SCALE + SLOTS * GROUP * BLOCK_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES + NBUF + 2 * SLOTS + 1;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NUM_BARS;
    static constexpr int BYTES = OFF_MISC + 16;
    static constexpr int SMEM_ALLOC = BYTES + 1024;
    static constexpr uint32_t TMEM_COLS = NBUF * BN;
    static_assert(STAGE % 1024 == 0, "boxes start on whole swizzle atoms");
    static_assert(128 * (BN + 1) * 4 <= STAGES * STAGE, "the partial sums fit into the ring");
    static_assert(SMEM_ALLOC <= 113 * 1024, "two blocks fit on an SM");
};

template <typename OutT>
__device__ __forceinline__ void fs_store(const Fp8SmallParams& p, OutT* c, float v)
{
    v *= p.alpha;
    if (p.beta != 0.0f)
        v = fmaf(p.beta, out_to_f32(*c), v);
    *c = fp8_to_out<OutT>(v);
}

// store(C) with C as a pointer to the output's type.
template <typename Store>
__device__ __forceinline__ void fs_with_output(const Fp8SmallParams& p, Store&& store)
{
    if (p.out_dtype == DT_F32)
        store(static_cast<float*>(p.C));
    else if (p.out_dtype == DT_F16)
        store(static_cast<__half*>(p.C));
    else
        store(static_cast<__nv_bfloat16*>(p.C));
}

// The end of a tile: the blocks' sums through shared memory (at `base`, whose
// ring holds nothing any more), added up over the cluster in rank order and
// stored, with rows (BY_ROW) or columns of the tile contiguous as they are in
// C.  `full`: this thread holds a row of sums.  Each block adds up a share,
// 128 / SPLITS rows or BN / SPLITS columns, with all its threads.
template <int BN, int SPLITS, bool BY_ROW>
__device__ __forceinline__ void fs_finish(const Fp8SmallParams& p, const uint64_t (&acc)[BN / 2], bool full,
                                          uint32_t base, int split, int row0, int col0,
                                          volatile int* abort_flag)
{
    // rows with a word between them, against bank conflicts
    constexpr int STEP_R = BY_ROW ? BN + 1 : 1, STEP_C = BY_ROW ? 1 : 128;
    const int t = static_cast<int>(threadIdx.x);
    if (full) {
        const uint32_t at = base + (t & 127) * STEP_R * 4;
#pragma unroll
        for (int j = 0; j < BN; ++j) {
            uint32_t w[2];
            unpack_f32x2(acc[j / 2], w[0], w[1]);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + j * STEP_C * 4), "r"(w[j & 1]) : "memory");
        }
    }
    __syncwarp();
    if constexpr (SPLITS > 1)
        cluster_sync();
    else
        __syncthreads();
    constexpr int MINE = 128 * BN / SPLITS / FS_THREADS;
    constexpr int BATCH = MINE * SPLITS > 64 ? 64 / SPLITS : MINE;  // loads in flight
    // this thread's first element; the next ones are FS_THREADS / BN rows, or
    // two columns, further
    const int r0 = BY_ROW ? split * (128 / SPLITS) + t / BN : t & 127;
    const int c0 = BY_ROW ? t % BN : split * (BN / SPLITS) + (t >> 7);
    constexpr int DR = BY_ROW ? FS_THREADS / BN : 0, DC = BY_ROW ? 0 : 2;
    const uint32_t at = base + (r0 * STEP_R + c0 * STEP_C) * 4;
    uint32_t peer[SPLITS];
#pragma unroll
    for (int k = 0; k < SPLITS; ++k)
        peer[k] = SPLITS > 1 ? mapa_shared(at, k) : at;
    // A block that gave up has no sum: then no block of the cluster stores.
    // (The question costs 0.1 us; asked after the first sums are on their way,
    // the same.)
    int gave_up = *abort_flag;
    if constexpr (SPLITS > 1) {
        const uint32_t flag = smem_u32(const_cast<int*>(abort_flag));
        const int lane = t & 31;
        if (lane < SPLITS)
            gave_up |= __float_as_int(ld_cluster_f32(mapa_shared(flag, lane)));
    }
    const bool store = !__any_sync(0xffffffffu, gave_up);
#pragma unroll
    for (int j0 = 0; j0 < MINE; j0 += BATCH) {
        float v[BATCH][SPLITS];
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
#pragma unroll
            for (int k = 0; k < SPLITS; ++k) {
                const uint32_t from = peer[k] + (j0 + j) * (DR * STEP_R + DC * STEP_C) * 4;
                v[j][k] = SPLITS > 1 ? ld_cluster_f32(from) : ld_shared_f32(from);
            }
        const int row = row0 + r0 + j0 * DR, col = col0 + c0 + j0 * DC;
        fs_with_output(p, [&](auto* out) {
            auto* c = out + row * p.c_row + col * p.c_col;
#pragma unroll
            for (int j = 0; j < BATCH; ++j, c += DR * p.c_row + DC * p.c_col) {
                float sum = v[j][0];
#pragma unroll
                for (int k = 1; k < SPLITS; ++k)
                    sum += v[j][k];
                if (store && row + j * DR < p.rows && col + j * DC < p.cols)
                    fs_store(p, c, sum);
            }
        });
    }
    if constexpr (SPLITS > 1) {
        __syncwarp();
        cluster_sync();
    }
}

template <int BN, int SPLITS>
__global__ void __launch_bounds__(FS_THREADS, 2)
    fp8_small_kernel(const __grid_constant__ CUtensorMap tmP,
                     const __grid_constant__ CUtensorMap tmQ, const Fp8SmallParams p)
{
    using L = Fp8SmallLayout<BN>;
    constexpr int STAGES = L::STAGES;
    constexpr int NBUF = L::NBUF;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::OFF_BAR;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto done_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    auto sfull_bar = [&](int i) { return bar0 + 8u * (2 * STAGES + NBUF + i); };
    auto sempty_bar = [&](int i) { return bar0 + 8u * (2 * STAGES + NBUF + L::SLOTS + i); };
    const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + NBUF + 2 * L::SLOTS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);

    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const int tile = blockIdx.x / SPLITS;
    const int split = SPLITS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int row0 = (tile / p.tiles_c) * 128;
    const int col0 = (tile % p.tiles_c) * BN;
    const int kb0 = static_cast<int>(static_cast<long long>(p.k_blocks) * split / SPLITS);
    const int kb1 = static_cast<int>(static_cast<long long>(p.k_blocks) * (split + 1) / SPLITS);
    const int nkb = kb1 - kb0;
    const TcWatch watch{abort_flag, p.status, p.wait_budget};

    auto issue = [&](int i) {  // the copies of this block's K block i
        const int s = i % STAGES, kb = kb0 + i;
        if (p.fault_skip_kblock == kb)
            return;  // test hook, -1 in normal use
        const uint32_t dP = sbase + s * L::STAGE;
        mbar_arrive_expect_tx(full_bar(s), L::STAGE);
        if (p.p_mn)
            tma_load_2d(dP, &tmP, full_bar(s), row0, kb * F8_BK);
        else
            tma_load_2d(dP, &tmP, full_bar(s), kb * F8_BK, row0);
        if (p.q_mn)
            tma_load_2d(dP + F8_BOX, &tmQ, full_bar(s), col0, kb * F8_BK);
        else
            tma_load_2d(dP + F8_BOX, &tmQ, full_bar(s), kb * F8_BK, col0);
    };
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmP);
        tma_prefetch_desc(&tmQ);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(done_bar(s), 1);
        }
        for (int b = 0; b < NBUF; ++b)
            mbar_init(tempty_bar(b), 4);
        for (int i = 0; i < L::SLOTS; ++i) {
            mbar_init(sfull_bar(i), 32);
            mbar_init(sempty_bar(i), 4);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        for (int i = 0; i < STAGES && i < nkb; ++i)
            issue(i);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(tmem_slot), L::TMEM_COLS);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    uint64_t acc[BN / 2];  // pairs of columns
    bool ok = true;
    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            int last = min(STAGES, nkb) - 1;
            for (int i = STAGES; i < nkb; ++i) {
                if (!tc_wait(done_bar(i % STAGES), static_cast<uint32_t>((i / STAGES - 1) & 1), watch)) {
                    ok = false;
                    break;
                }
                issue(i);
                last = i;
            }
            if (!ok) {
                // Drain (bounded): the copies of the last blocks issued land
                // before shared memory goes away.
                for (int i = max(0, last - STAGES + 1); i <= last; ++i) {
                    const long long t0 = clock64();
                    while (!mbar_try_wait(full_bar(i % STAGES), static_cast<uint32_t>((i / STAGES) & 1)) &&
                           clock64() - t0 < p.wait_budget) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        const uint64_t p_hi = fp8_desc_hi(128, p.p_mn);
        const uint64_t q_hi = fp8_desc_hi(p.q_mn ? BN : 128, p.q_mn);
        const uint32_t p_step = (p.p_mn ? 32 * 128 : 32) >> 4;
        const uint32_t q_step = (p.q_mn ? 32 * BN : 32) >> 4;
        for (int i = 0; i < nkb; ++i) {
            const int s = i % STAGES, b = i % NBUF;
            ok = tc_wait_warp(full_bar(s), static_cast<uint32_t>((i / STAGES) & 1), watch) &&
                 tc_wait_warp(tempty_bar(b), static_cast<uint32_t>(((i / NBUF) & 1) ^ 1), watch);
            if (!ok)
                break;
            tc_fence_after();
            const uint32_t p0 = (sbase + s * L::STAGE) >> 4;
            const uint32_t q0 = p0 + (F8_BOX >> 4);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < F8_BK / 32; ++k)
                    tc_mma_f8<1>(tmem_base + static_cast<uint32_t>(b * BN),
                                 p_hi | ((p0 + k * p_step) & 0x3FFF), q_hi | ((q0 + k * q_step) & 0x3FFF),
                                 p.idesc, k != 0);
                tc_commit(done_bar(s));
            }
            __syncwarp();
        }
        // every MMA issued has completed before TMEM is released (bounded)
        if (elect_one())
            tc_commit(drain_bar);
        __syncwarp();
        const long long t0 = clock64();
        while (!__all_sync(0xffffffffu, mbar_test_wait(drain_bar, 0))) {
            if (__any_sync(0xffffffffu, clock64() - t0 > p.wait_budget))
                break;
        }
    } else if (warp == 2) {
        // ------------------------------------------------ scales
        const float* rp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            rp[i] = p.sp + (static_cast<long long>(min(row0 + 32 * i + static_cast<int>(lane), p.rows - 1)) >>
                            p.sp_shift) * p.sp_o;
        constexpr int NC = (BN + 31) / 32;
        const float* cq[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i)
            cq[i] = p.sq + (static_cast<long long>(min(col0 + 32 * i + static_cast<int>(lane), p.cols - 1)) >>
                            p.sq_shift) * p.sq_o;
        for (int g = 0; g * L::GROUP < nkb; ++g) {
            const int slot = g % L::SLOTS;
            ok = tc_wait_warp(sempty_bar(slot), static_cast<uint32_t>(((g / L::SLOTS) & 1) ^ 1), watch);
            if (!ok)
                break;
            const int end = min((g + 1) * L::GROUP, nkb);
            uint32_t dst = sbase + L::OFF_SCALE + slot * L::GROUP * L::BLOCK_BYTES + lane * 4;
            for (int i = g * L::GROUP; i < end; ++i, dst += L::BLOCK_BYTES) {
                const long long kb = kb0 + i;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    cp_async_4(dst + 128 * k, rp[k] + kb * p.sp_k);
                if (BN >= 32 || lane < BN) {
#pragma unroll
                    for (int k = 0; k < NC; ++k)
                        cp_async_4(dst + 512 + 128 * k, cq[k] + kb * p.sq_k);
                }
            }
            cp_async_mbar_arrive(sfull_bar(slot));
        }
        cp_async_wait_all();
    } else if (warp == 3) {
        // ------------------------------------------------ herald, as in
        // fp8_gemm_kernel: a poll of an mbarrier takes about 300 cycles even
        // when it succeeds, a hardware barrier that the herald has already
        // reached about 40
        for (int i = 0; i < nkb; ++i) {
            const int g = i / L::GROUP;
            if (i % L::GROUP == 0)
                ok = ok && tc_wait_warp(sfull_bar(g % L::SLOTS),
                                        static_cast<uint32_t>((g / L::SLOTS) & 1), watch);
            ok = ok && tc_wait_warp(done_bar(i % STAGES), static_cast<uint32_t>((i / STAGES) & 1), watch);
            bar_sync(F8_HERALD_BAR, 160);
        }
    } else {
        // ------------------------------------------------ promotion
        const int q = warp & 3;
#pragma unroll
        for (int j = 0; j < BN / 2; ++j)
            acc[j] = 0;
#pragma unroll 1
        for (int i = 0; i < nkb; ++i) {
            const int b = i % NBUF, slot = i / L::GROUP % L::SLOTS;
            bar_sync(F8_HERALD_BAR, 160);
            tc_fence_after();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                   static_cast<uint32_t>(b * BN);
            const uint32_t saddr = sbase + L::OFF_SCALE +
                                   (slot * L::GROUP + i % L::GROUP) * L::BLOCK_BYTES;
            const uint32_t rs = __float_as_uint(ld_shared_f32(saddr + (q * 32 + lane) * 4));
            const uint64_t rs2 = pack_f32x2(rs, rs);
            constexpr int CH = BN < 32 ? BN : 32;
#pragma unroll
            for (int c = 0; c < BN / CH; ++c) {
                uint32_t v[CH];
                if constexpr (CH == 16)
                    tmem_ld_32x32b_x16(taddr, v);
                else
                    tmem_ld_32x32b_x32(taddr + c * 32, v);
                tmem_wait_ld(v);
                if (c + 1 == BN / CH) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(tempty_bar(b));
                }
#pragma unroll
                for (int j = 0; j < CH; j += 4) {
                    uint32_t f[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
                                 : "r"(saddr + 512 + (c * CH + j) * 4));
                    uint64_t* t = &acc[(c * CH + j) / 2];
                    ffma2(t[0], pack_f32x2(v[j], v[j + 1]), fmul2(rs2, pack_f32x2(f[0], f[1])));
                    ffma2(t[1], pack_f32x2(v[j + 2], v[j + 3]), fmul2(rs2, pack_f32x2(f[2], f[3])));
                }
            }
            if (i % L::GROUP == L::GROUP - 1) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(sempty_bar(slot));
            }
        }
        ok = !*abort_flag;  // an unfinished sum is not used
    }

    // ------------------------------------------------ sums of the cluster, output
    if (SPLITS == 1 && !p.by_row) {
        // a thread's values lie next to its neighbours' in C
        const int r = static_cast<int>(threadIdx.x) & 127;
        if (warp >= FS_EPI_WARP0 && ok && row0 + r < p.rows) {
            fs_with_output(p, [&](auto* out) {
                auto* c = out + (row0 + r) * p.c_row + col0 * p.c_col;
#pragma unroll
                for (int j = 0; j < BN; ++j, c += p.c_col) {
                    uint32_t w[2];
                    unpack_f32x2(acc[j / 2], w[0], w[1]);
                    if (col0 + j < p.cols)
                        fs_store(p, c, __uint_as_float(w[j & 1]));
                }
            });
        }
    } else if (p.by_row) {
        fs_finish<BN, SPLITS, true>(p, acc, warp >= FS_EPI_WARP0 && ok, sbase, split, row0, col0, abort_flag);
    } else {
        fs_finish<BN, SPLITS, false>(p, acc, warp >= FS_EPI_WARP0 && ok, sbase, split, row0, col0, abort_flag);
    }

    // ---------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<1>(tmem_base, L::TMEM_COLS);
    }
}

template <int BN, int SPLITS>
cudaError_t launch_small(const Fp8Launch& l, bool swapped, cudaStream_t stream)
{
    using L = Fp8SmallLayout<BN>;
    auto kern = fp8_small_kernel<BN, SPLITS>;
    static ClusterCaps caps;
    int cap = 0;
    const cudaError_t err = cluster_cap(kern, caps, SPLITS, FS_THREADS, L::SMEM_ALLOC, l.num_sms, &cap);
    if (err != cudaSuccess)
        return err;
    const Fp8Operand& P = swapped ? l.b : l.a;
    const Fp8Operand& Q = swapped ? l.a : l.b;
    Fp8SmallParams p{};
    p.rows = swapped ? l.N : l.M;
    p.cols = swapped ? l.M : l.N;
    CUtensorMap tp, tq;
    if (!encode_operand(&tp, P, p.rows, l.K, 128) || !encode_operand(&tq, Q, p.cols, l.K, BN))
        return cudaErrorNotSupported;
    p.tiles_c = (p.cols + BN - 1) / BN;
    p.k_blocks = (l.K + F8_BK - 1) / F8_BK;
    p.idesc = fp8_idesc(P.type, Q.type, 128, BN, P.mn_major, Q.mn_major);
    p.p_mn = P.mn_major;
    p.q_mn = Q.mn_major;
    p.sp = P.scale;
    p.sp_k = P.stride_k;
    p.sp_o = P.stride_o;
    p.sp_shift = P.shift;
    p.sq = Q.scale;
    p.sq_k = Q.stride_k;
    p.sq_o = Q.stride_o;
    p.sq_shift = Q.shift;
    p.C = l.C;
    p.c_row = swapped ? 1 : l.ldc;
    p.c_col = swapped ? l.ldc : 1;
    p.by_row = !swapped;
    p.out_dtype = l.out_dtype;
    p.alpha = l.alpha;
    p.beta = l.beta;
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip_kblock = l.fault_skip_kblock;
    const long long tiles = static_cast<long long>((p.rows + 127) / 128) * p.tiles_c;
    if (tiles * SPLITS > 0x7fffffffLL)
        return cudaErrorNotSupported;
    ClusterLaunch launch(static_cast<unsigned>(tiles * SPLITS), SPLITS, FS_THREADS, L::SMEM_ALLOC, stream);
    return launch.run(kern, tp, tq, p);
}

template <int BN>
cudaError_t launch_splits(const Fp8Launch& l, bool swapped, int splits, cudaStream_t stream)
{
    switch (splits) {
    case 8:
        return launch_small<BN, 8>(l, swapped, stream);
    case 4:
        return launch_small<BN, 4>(l, swapped, stream);
    case 2:
        return launch_small<BN, 2>(l, swapped, stream);
    default:
        return launch_small<BN, 1>(l, swapped, stream);
    }
}

// Columns of a tile for `cols` of the shorter axis.  An MN-major box of 16
// would be a 16-byte row, below the least swizzle.
int tile_cols(int cols, bool mn_major)
{
    return cols <= 16 && !mn_major ? 16 : cols <= 32 ? 32 : 64;
}

}  // namespace

// Up to 64 columns the long operand is read once, in one column of tiles.
// Beyond that this kernel pays while the persistent kernels' 128 x 128 tiles
// would leave three SMs in four idle.  Measured on GB300, BF16 out, us, this
// kernel / the persistent ones: 1 x 4096 x 4096 6.1 / 13.6, 64 x 8192 x 8192
// 17.7 / 22.9, 96 x 200 x 1000 6.0 / 18.3, 128 x 4096 x 4096 (32 tiles) 12.2 /
// 13.2, 512 x 512 x 4096 (16) 9.7 / 12.7; not taken: 256 x 4096 x 4096 (64)
// 17.3 / 13.3, 1024^3 (64) 8.9 / 6.7.
//
// With few K blocks there is nothing to divide over a cluster, and the
// persistent kernels' stores by TMA are the faster end: 64 x 4096 x 256 6.5 /
// 4.4, 256 x 2048 x 512 6.4 / 5.3, 64 x 8192 x 768 6.9 / 5.7, 24 x 4096 x 256
// 4.7 / 4.3, 32 x 8192 x 768 5.5 / 5.6, 16 x 4096 x 256 3.9 / 4.0; without
// them 100 x 300 x 500 6.0 / 6.8.
bool fp8_small_takes(const Fp8Launch& l)
{
    const int least = std::min(l.M, l.N);
    const int k_blocks = (l.K + F8_BK - 1) / F8_BK;
    if (least > 16 && k_blocks <= (least > 32 ? 6 : 4) && tma_output(l))
        return false;
    if (least <= 64)
        return true;
    const long long tiles =
        static_cast<long long>((l.M + 127) / 128) * ((l.N + 127) / 128);
    return tiles * 4 <= l.num_sms;
}

cudaError_t fp8_small_launch(const Fp8Launch& l, cudaStream_t stream)
{
    const bool swapped = l.M <= l.N;
    const int cols = std::min(l.M, l.N), rows = std::max(l.M, l.N);
    const int bn = tile_cols(cols, swapped ? l.a.mn_major : l.b.mn_major);
    const long long tiles = static_cast<long long>((rows + 127) / 128) * ((cols + bn - 1) / bn);
    // Splits of K: up to one block an SM, each with at least two K blocks, or
    // up to two with eight or more each.  (With two of fewer the exchange
    // costs more than the overlap gives: 64 x 4096 x 4096 10.3 us instead of
    // 9.4, 1 x 4096 x 4096 7.3 instead of 6.8, 16 x 4096 x 2048 6.2 instead of
    // 5.6.  With one of more, 16 x 5120 x 5120 takes 10.0 instead of 9.4.)
    const int k_blocks = (l.K + F8_BK - 1) / F8_BK;
    int splits = 1;
    while (splits < FS_MAX_SPLITS && k_blocks >= 4 * splits &&
           tiles * splits * 2 <= (k_blocks >= 16 * splits ? 2LL : 1LL) * l.num_sms)
        splits *= 2;
    if (bn == 16)
        return launch_splits<16>(l, swapped, splits, stream);
    if (bn == 32)
        return launch_splits<32>(l, swapped, splits, stream);
    return launch_splits<64>(l, swapped, splits, stream);
}

}  // namespace tmmo
