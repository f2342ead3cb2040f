// Rank values t = scale * X F^T of every row's adapter on the tensor cores, and
// the plans of the row tiles.
//
// With rank r, a row tile of X (128 rows) is read once for 2 * 128 * r
// operations a column: the bound is reading X from HBM, and for few rows the
// adapters' factors.  So a tile's contraction is split over a cluster of up to
// eight CTAs, and where that still leaves SMs idle its adapters are dealt out to
// several clusters (their rows are disjoint): 8192 rows are 64 tiles on 2
// CTAs each, 64 rows of 64 adapters one tile on 8 x 15.  The FP32 sums of a
// cluster are added through distributed shared memory in rank order.  8192 rows of
// 4096, 12 adapters of rank 64, BF16: 20 us, 10 of them HBM's, the others launch, plan,
// first copies and the sums.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "grouped_maps.h"
#include "lora_tc.cuh"
#include "persistent.cuh"

namespace tmmo {
namespace {

constexpr int LS_THREADS = 256;  // warps 0: copies, 1: MMA, 4-7: accumulator
constexpr int LS_MAX_STAGES = 8;
constexpr int LS_RING = 192 * 1024;
constexpr int LS_RING_SHARED = 88 * 1024;  // leaves room for the product's kernel on the SM

struct ShrinkSide {
    int k_blocks;
    int across;
    int one;  // one factor for every adapter
    uint32_t idesc;
    void* t;       // BF16 parts, rows x columns()
    void* t_grad;  // FP16 parts, laid out the same (either may be null)
};

struct ShrinkParams {
    ShrinkSide side[2];
    const int32_t* adapter;
    const float* scale;
    LoraPlan* plan;
    int rows, adapters, rank, cols;  // cols: rank rounded up to 16
    LoraParts lay;
    int tiles, deal;                 // row tiles; clusters that share a tile's adapters
    int stages, stage_bytes, a_offset, b_bytes[2];
    int together;                    // adapters whose factors share a stage
    int box_rows;                    // rows of X that a copy brings
    int chains;                      // accumulators that K steps take in turn; behind them, sums
    uint32_t tmem_cols;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

struct ShrinkSmem {
    uint64_t full[LS_MAX_STAGES], empty[LS_MAX_STAGES], done;
    uint64_t segment, taken;  // accumulators are to be added to the sums, are added
    uint32_t tmem;
    int abort_flag;
    PlanScratch scratch;
    int place[LT_ROWS];        // each row's place in the plan
    float scale[LT_ROWS];      // of each place
    LoraPlan plan;
};

// The place of rank values j .. j + 7 (a multiple of 8) of a row in parts: that of the
// first part, and how far each next one lies behind (16-byte words).
__device__ __forceinline__ uint4* parts_at(void* t, int64_t row, const LoraParts& lay, int j)
{
    return static_cast<uint4*>(t) + (row * lay.columns() + j / lay.chunk * 64 + j % lay.chunk) / 8;
}

template <int SPLITS>
__global__ void __launch_bounds__(LS_THREADS, 1)
    lora_shrink_tc_kernel(const __grid_constant__ CUtensorMap tmX0, const __grid_constant__ CUtensorMap tmF0,
                          const __grid_constant__ CUtensorMap tmX1, const __grid_constant__ CUtensorMap tmF1,
                          const ShrinkParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    __shared__ ShrinkSmem s;
    grid_dep_launch_dependents();  // the product that uses t may start with what it has

    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const int split = SPLITS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    int id = blockIdx.x / SPLITS;
    const int tile = id % p.tiles;
    id /= p.tiles;
    const int deal = id % p.deal, which = id / p.deal;
    const ShrinkSide side = p.side[which];
    const CUtensorMap* tmX = which ? &tmX1 : &tmX0;
    const CUtensorMap* tmF = which ? &tmF1 : &tmF0;
    const int b_bytes = p.b_bytes[which];
    const int row0 = tile * LT_ROWS;
    // each row's adapter, asked for before anything else
    const int g = threadIdx.x >= 128 ? row_adapter(p.adapter, row0 + static_cast<int>(threadIdx.x) - 128, p.rows,
                                                   p.adapters)
                                     : -1;
    const TcWatch watch{&s.abort_flag, p.status, p.wait_budget};
    const int per = (side.k_blocks + SPLITS - 1) / SPLITS;
    const int kb0 = min(split * per, side.k_blocks), kb1 = min(kb0 + per, side.k_blocks);

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(smem_u32(&s.full[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
        }
        mbar_init(smem_u32(&s.done), 1);
        mbar_init(smem_u32(&s.segment), 1);
        mbar_init(smem_u32(&s.taken), 4);
        s.abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(tmX);
        tma_prefetch_desc(tmF);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&s.tmem), p.tmem_cols);
        tmem_relinquish<1>();
    }
    // (128 threads make the plan, as the accumulator's warps are idle)
    if (threadIdx.x >= 128) {
        const float scale = p.scale && g >= 0 ? p.scale[g] : 1.0f;
        const int place = make_plan(s.plan, s.scratch, g, threadIdx.x - 128, [] { bar_sync(1, 128); });
        s.place[threadIdx.x - 128] = place;
        if (place >= 0)
            s.scale[place] = scale;  // (of every row with this adapter: the same)
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    if (which == 0 && deal == 0 && split == 0) {
        const int* from = reinterpret_cast<const int*>(&s.plan);
        int* to = reinterpret_cast<int*>(p.plan + tile);
        const int words = 4 + LT_ROWS + 4 * s.plan.count;  // the rows of absent adapters are not read
        for (int i = threadIdx.x; i < words; i += LS_THREADS)
            to[i] = from[i];
    }
    const int mine = s.plan.count > deal ? (s.plan.count - deal + p.deal - 1) / p.deal : 0;
    const int rounds = (mine + p.together - 1) / p.together;
    const int steps = rounds * (kb1 - kb0);
    // A round's K steps go in segments, after each of which but the last the accumulators of
    // its adapters' rows are added to the rows' sums.
    const int segment = LT_SEGMENT * p.chains;
    const int segments = (kb1 - kb0 + segment - 1) / segment;
    const uint32_t sums_at = tmem + p.chains * p.cols;
    // the i-th adapter of this CTA, by its place in the plan
    auto nth = [&](int i) { return deal + i * p.deal; };

    if (warp == 0) {
        int stage = 0, n = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i0 = 0; ok && i0 < mine; i0 += p.together) {
            const int some = min(p.together, mine - i0);
            for (int kb = kb0; kb < kb1; ++kb, ++n) {
                ok = warp_wait(smem_u32(&s.empty[stage]), phase ^ 1, watch);
                if (!ok)
                    break;
                const uint32_t bar = smem_u32(&s.full[stage]);
                const uint32_t base = smem_u32(ring) + stage * p.stage_bytes;
                const uint32_t dA = base + p.a_offset;
                if (kb != p.fault_skip_kblock && elect_one()) {  // (test hook, -1 in normal use)
                    mbar_arrive_expect_tx(bar, p.box_rows * 128 + some * b_bytes);
                    tma_load_2d(dA, tmX, bar, kb * TC_BK, row0);
                    for (int i = 0; i < some; ++i) {
                        const int z = side.one ? 0 : s.plan.ids[nth(i0 + i)];
                        const uint32_t dB = base + i * b_bytes;
                        if (side.across) {
                            for (int b = 0; b * 8192 < b_bytes; ++b)
                                tma_load_3d(dB + b * 8192, tmF, bar, b * 64, kb * TC_BK, z);
                        } else {
                            tma_load_3d(dB, tmF, bar, kb * TC_BK, 0, z);
                        }
                    }
                }
                __syncwarp();
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) {  // wait (bounded) for the copies in flight before shared memory goes away
            for (int i = 0; i < p.stages; ++i) {
                const int uses = n / p.stages + (i < n % p.stages);
                const long long t0 = clock64();
                while (uses > 0 && !mbar_try_wait(smem_u32(&s.full[i]), (uses - 1) & 1) &&
                       clock64() - t0 < p.wait_budget) {
                }
            }
        }
    } else if (warp == 1) {
        if (steps > 0) {
            int stage = 0;
            uint32_t phase = 0, added = 0;
            bool ok = true;
            for (int i0 = 0; ok && i0 < mine; i0 += p.together) {
                const int some = min(p.together, mine - i0);
                int n = 0;  // K step of the segment
                for (int kb = kb0; kb < kb1; ++kb, ++n) {
                    if (n == segment) {
                        if (elect_one())
                            tc_commit(smem_u32(&s.segment));
                        __syncwarp();
                        ok = warp_wait(smem_u32(&s.taken), added++ & 1, watch);
                        if (!ok)
                            break;
                        n = 0;
                    }
                    ok = warp_wait(smem_u32(&s.full[stage]), phase, watch);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t base = smem_u32(ring) + stage * p.stage_bytes;
                    const uint32_t a0 = base + p.a_offset;
                    const uint32_t d = tmem + n % p.chains * p.cols;
                    for (int i = 0; i < some; ++i) {
                        const uint32_t b0 = base + i * b_bytes;
                        const uint4 rows = *reinterpret_cast<const uint4*>(s.plan.rows[nth(i0 + i)]);
                        const uint32_t off[4] = {~rows.x, ~rows.y, ~rows.z, ~rows.w};
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < TC_BK / TC_UMMA_K; ++k)
                                tc_mma_f16_lanes(d, smem_desc_sw128(a0 + k * 32, 16, 1024),
                                                 side.across ? smem_desc_sw128(b0 + k * 2048, 8192, 1024)
                                                             : smem_desc_sw128(b0 + k * 32, 16, 1024),
                                                 side.idesc, n >= p.chains || k != 0, off);
                            if (i == some - 1)
                                tc_commit(smem_u32(&s.empty[stage]));
                        }
                        __syncwarp();
                    }
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (elect_one())
                tc_commit(smem_u32(&s.done));  // also after giving up: nothing may run on
            __syncwarp();
            const long long t0 = clock64();
            while (!mbar_try_wait(smem_u32(&s.done), 0) && clock64() - t0 < p.wait_budget) {
            }
        }
    }
    // The sums to shared memory; the ring holds nothing any more.
    __syncwarp();
    const int pitch = p.cols + 4;  // rows 16 bytes apart in the banks
    float* sums = reinterpret_cast<float*>(ring);
    if (warp >= 4) {
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int place = s.place[row];
        const int round = place >= 0 && place % p.deal == deal ? place / p.deal / p.together : -1;
        bool all = true;
        uint32_t added = 0;
        for (int r = 0; all && r < rounds; ++r)
            for (int n = 1; all && n < segments; ++n) {
                all = warp_wait(smem_u32(&s.segment), added++ & 1, watch);
                if (!all)
                    break;
                tc_fence_after();
                add_to_sums(tmem + lanes, p.chains, sums_at + lanes, p.cols, n == 1, r == round);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&s.taken));
            }
        if (steps > 0) {
            int ok = 1;
            if (lane == 0)
                ok = tc_wait(smem_u32(&s.done), 0, patient(watch, steps)) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (ok) {
                tc_fence_after();
                const int chains = min(p.chains, kb1 - kb0 - (segments - 1) * segment);
#pragma unroll 1
                for (int j = 0; j < p.cols; j += 16) {
                    const uint32_t from = tmem + lanes + j;
                    uint32_t v[16];
                    tmem_ld_32x32b_x16(from, v);
                    tmem_wait_ld(v);
                    // (the sums lie behind the last accumulator)
                    const int others = chains + (segments > 1);
#pragma unroll 1
                    for (int k = 1; k < others; ++k) {
                        const int c = k < chains ? k : p.chains;
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(from + c * p.cols, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(o[i]));
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        st_shared_v4(smem_u32(sums + row * pitch + j + i), v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
        } else {
            for (int j = 0; j < p.cols; ++j)
                sums[row * pitch + j] = 0.0f;
        }
        tc_fence_before();
    }
    if constexpr (SPLITS > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc<1>(tmem, p.tmem_cols);
    // Each CTA adds up and stores its share of the rows, eight values of a row a
    // thread.
    int gave_up = s.abort_flag;
    if constexpr (SPLITS > 1)
        for (int k = 0; k < SPLITS; ++k)
            gave_up |= __float_as_int(ld_cluster_f32(mapa_shared(smem_u32(&s.abort_flag), k)));
    constexpr int SHARE = LT_ROWS / SPLITS;
    const int eights = p.cols / 8;
    const int total = min(SHARE, p.rows - row0 - split * SHARE) * eights;  // none where negative
#pragma unroll 1
    for (int i = threadIdx.x; i < total && !gave_up; i += LS_THREADS) {
        const int row = split * SHARE + i / eights, j = i % eights * 8;
        const int place = s.place[row];
        if (place < 0 ? deal != 0 : place % p.deal != deal)
            continue;
        float sum[8] = {};
        if (place >= 0) {
            const uint32_t at = smem_u32(sums + row * pitch + j);
            float4 v[SPLITS][2];
#pragma unroll
            for (int k = 0; k < SPLITS; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    v[k][h] = ld_cluster_v4(SPLITS > 1 ? mapa_shared(at, k) + 16 * h : at + 16 * h);
            const float scale = s.scale[place];
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
                sum[4 * h] = scale * a.x;
                sum[4 * h + 1] = scale * a.y;
                sum[4 * h + 2] = scale * a.z;
                sum[4 * h + 3] = scale * a.w;
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
                sum[q] = j + q < p.rank ? sum[q] : 0.0f;
        }
        const int next = p.lay.chunk / 8;
        if (side.t_grad) {
            float left[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                left[q] = sum[q];
            uint4* to = parts_at(side.t_grad, row0 + row, p.lay, j);
            each_f16_part(left, [&](int part, const uint4& w) { to[part * next] = w; });
        }
        if (side.t) {
            uint4* to = parts_at(side.t, row0 + row, p.lay, j);
            each_part(sum, p.lay.parts, [&](int part, const uint4& w) { to[part * next] = w; });
        }
    }
    if constexpr (SPLITS > 1) {
        __syncwarp();
        cluster_sync();  // nobody leaves while others read its sums
    }
}

// Once for each device: the SM's memory is laid out for this kernel and the
// product's from the start, as it is not laid out anew while a block runs (a
// decoding batch took 28 us instead of 25).
template <int SPLITS>
cudaError_t share_sms()
{
    static std::atomic<uint64_t> done{0};
    static_assert(kMaxDevices <= 64, "a bit for each");
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err != cudaSuccess || device < 0 || device >= kMaxDevices || (done.load() >> device & 1))
        return err;
    err = cudaFuncSetAttribute(lora_shrink_tc_kernel<SPLITS>,
                               cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (err == cudaSuccess)
        done.fetch_or(1ull << device);
    return err;
}

// Sets the kernel up, once; how many of its clusters run at a time, with the
// smaller ring (shared) or the larger.
template <int SPLITS>
cudaError_t most_clusters(bool shared, int num_sms, int* cap)
{
    static ClusterCaps caps[2];
    cudaError_t err = share_sms<SPLITS>();
    int n[2] = {};
    for (int i = 0; i < 2 && err == cudaSuccess; ++i)  // (the larger last: it stays the kernel's limit)
        err = cluster_cap(lora_shrink_tc_kernel<SPLITS>, caps[i], SPLITS, LS_THREADS,
                          (i ? LS_RING : LS_RING_SHARED) + 1024, num_sms, &n[i]);
    *cap = n[shared ? 0 : 1];
    return err;
}

template <int SPLITS>
cudaError_t launch(const CUtensorMap (&m)[4], const ShrinkParams& p, unsigned clusters, int smem,
                   cudaStream_t stream)
{
    ClusterLaunch l(clusters * SPLITS, SPLITS, LS_THREADS, smem, stream);
    return l.run(lora_shrink_tc_kernel<SPLITS>, m[0], m[1], m[2], m[3], p);
}

// CTAs for every SM, in clusters that run all at once: first the contraction is
// split, then the adapters are dealt out.
cudaError_t launch(const CUtensorMap (&m)[4], ShrinkParams& p, int sides, int most_k, int most_adapters,
                   bool shared, int num_sms, cudaStream_t stream)
{
    static SplitCaps known[2];
    const int* most = nullptr;
    const cudaError_t err = split_caps(known[shared], [&](int i, int* n) {
        return i == 0   ? most_clusters<1>(shared, num_sms, n)
               : i == 1 ? most_clusters<2>(shared, num_sms, n)
               : i == 2 ? most_clusters<4>(shared, num_sms, n)
                        : most_clusters<8>(shared, num_sms, n);
    }, &most);
    if (err != cudaSuccess)
        return err;
    auto cap = [&](int i) { return std::min(most[i], num_sms >> i); };  // (one an SM)
    int i = 0;
    while (i < 3 && 2 << i <= most_k && p.tiles * sides <= cap(i + 1))
        ++i;
    p.deal = std::max(1, std::min(most_adapters, cap(i) / (p.tiles * sides)));
    const unsigned clusters = static_cast<unsigned>(p.tiles) * sides * p.deal;
    const int smem = (shared ? LS_RING_SHARED : LS_RING) + 1024;
    switch (i) {
    case 0:
        return launch<1>(m, p, clusters, smem, stream);
    case 1:
        return launch<2>(m, p, clusters, smem, stream);
    case 2:
        return launch<4>(m, p, clusters, smem, stream);
    default:
        return launch<8>(m, p, clusters, smem, stream);
    }
}

// A stage holds the factors of adapters that a tile has beside each other (two, or
// as many as 8 KiB hold), and after them X's rows, so that a K step of X is read
// once for them.
struct ShrinkRing {
    int factor, together, a_offset, box_rows, stage_bytes;
    bool shares;  // four stages leave room for the product's kernel on the SM
};
ShrinkRing shrink_ring(const LoraLaunch& l)
{
    ShrinkRing r;
    const int cols = (l.rank + 15) / 16 * 16;
    r.factor = (l.across ? (cols + 63) / 64 * 64 : cols) * 128;
    r.together = std::min(std::min(std::max(2, 8192 / r.factor), 32768 / r.factor),
                          std::min(std::min(l.adapters, LT_ROWS), l.rows));
    r.a_offset = r.together * r.factor;
    r.box_rows = std::min(LT_ROWS, (l.rows + 7) / 8 * 8);
    r.stage_bytes = r.a_offset + (r.box_rows * 128 + 1023) / 1024 * 1024;
    // The tensor core reads 128 rows of X whatever a copy brings: what follows
    // lies within the ring too (those lanes are not used).  At the end the
    // tile's sums lie in it.
    r.shares = 3 * r.stage_bytes + r.a_offset + 16384 <= LS_RING_SHARED &&
               LT_ROWS * (cols + 4) * 4 <= LS_RING_SHARED;
    return r;
}

}  // namespace

bool lora_shrink_shares(const LoraLaunch& l) { return l.adapters > 0 && shrink_ring(l).shares; }

cudaError_t lora_shrink_tc_launch(const LoraLaunch& first, const LoraLaunch* second, cudaStream_t stream)
{
    const LoraLaunch& l = first;
    ShrinkParams p{};
    p.adapter = l.adapter;
    p.scale = l.scale;
    p.plan = static_cast<LoraPlan*>(l.plan);
    p.rows = l.rows;
    p.adapters = l.adapters;
    p.rank = l.rank;
    p.cols = (l.rank + 15) / 16 * 16;
    p.lay = lora_parts(l.rank, l.parts);
    p.tiles = (l.rows + LT_ROWS - 1) / LT_ROWS;
    p.box_rows = std::min(LT_ROWS, (l.rows + 7) / 8 * 8);
    const uint32_t box_rows = static_cast<uint32_t>(p.box_rows);
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip_kblock = l.fault_skip_kblock;
    CUtensorMap m[4];
    const int sides = second ? 2 : 1;
    int most_k = 1;
    for (int i = 0; i < sides; ++i) {
        const LoraLaunch& s = i ? *second : first;
        const uint32_t cols = static_cast<uint32_t>(p.cols);
        p.side[i] = {(s.K + TC_BK - 1) / TC_BK, s.across, s.adapters == 1 || s.stride_f == 0,
                     tc_idesc(s.in_dtype == DT_BF16, LT_ROWS, p.cols, false, s.across), s.t, s.t_grad};
        p.b_bytes[i] = (s.across ? (p.cols + 63) / 64 * 64 : p.cols) * 128;
        most_k = std::max(most_k, p.side[i].k_blocks);
        const int64_t stride = p.side[i].one ? s.ldf : s.stride_f;
        const int64_t stacked = p.side[i].one ? 1 : s.adapters;
        if (!s.maps->get(&m[2 * i], s.in_dtype, s.X, 2, {s.K, s.rows, 1}, {s.ldx, 0}, {64, box_rows, 1}) ||
            !(s.across ? s.maps->get(&m[2 * i + 1], s.in_dtype, s.F, 3, {s.rank, s.K, stacked}, {s.ldf, stride},
                                    {64, TC_BK, 1})
                       : s.maps->get(&m[2 * i + 1], s.in_dtype, s.F, 3, {s.K, s.rank, stacked}, {s.ldf, stride},
                                    {64, cols, 1})))
            return cudaErrorNotSupported;
    }
    if (sides == 1) {
        m[2] = m[0];
        m[3] = m[1];
    }
    const ShrinkRing r = shrink_ring(first);
    if (second) {
        const ShrinkRing q = shrink_ring(*second);
        p.together = std::min(r.together, q.together);
        p.a_offset = std::max(r.a_offset, q.a_offset);
        p.stage_bytes = p.a_offset + (r.box_rows * 128 + 1023) / 1024 * 1024;
    } else {
        p.together = r.together;
        p.a_offset = r.a_offset;
        p.stage_bytes = r.stage_bytes;
    }
    const bool shared = !second && r.shares;
    // The tensor core drops what does not fit when it adds a step to an accumulator,
    // half a unit in the last place on average: 2000 deep sums were 3e-6 short.  The
    // steps take up to eight accumulators in turn, added with rounding every
    // LT_SEGMENT steps of each and at the end.  The product's kernel has 256 columns of a
    // shared SM's tensor memory.
    p.chains = std::max(1, std::min(8, (shared ? 256 : 512) / p.cols - 1));
    p.tmem_cols = 32;
    while (p.tmem_cols < static_cast<uint32_t>((p.chains + 1) * p.cols))
        p.tmem_cols *= 2;
    p.stages = std::min(LS_MAX_STAGES,
                        ((shared ? LS_RING_SHARED : LS_RING) - p.a_offset - 16384) / p.stage_bytes + 1);
    const int most_adapters = std::min(std::min(l.adapters, LT_ROWS), l.rows);
    return launch(m, p, sides, most_k, most_adapters, shared, l.num_sms, stream);
}

}  // namespace tmmo
