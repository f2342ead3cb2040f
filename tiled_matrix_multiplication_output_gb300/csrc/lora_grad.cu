// The adapters' gradients on the tensor cores: for each adapter, P^T t over its
// rows, P the layer's input or its output's gradient and t rank values.
//
// One tile is 128 columns of P (the lanes) by up to 256 columns of rank values in
// parts, whose sums are added at the end.  Both operands lie across the
// contraction, and an adapter's rows lie anywhere: the tile goes through the
// row tiles (128 rows) that hold any of them, found from the plans.  In one that
// holds other rows as well, two warps zero those in shared memory, in both
// operands, before it counts as loaded; 16-row slices without a row of the
// adapter are skipped.  Bound: reading P once for each adapter in a row tile
// (once in all where sequences are long), the rank values and the launch; where
// sequences are short, the zeroing, 0.8 us a step for two warps, so that four pairs of
// them work on the stages of the ring (3237 rows in runs of 59 by 1248 and 472 columns:
// a call 42 us with one pair, 34 with four).  4096 rows of 6 adapters, rank 16, both
// gradients of 4096 columns: 26 us, 10 of them HBM's.
//
// Launched as a programmatic dependent of the product that uses the same rank
// values, of which it needs nothing: it starts where that one's last tiles leave SMs
// idle.
#include <algorithm>
#include <cstring>

#include "grouped_maps.h"
#include "lora_tc.cuh"
#include "persistent.cuh"
#include "simt_types.h"

namespace tmmo {
namespace {

constexpr int LG_TEAMS = 4;      // pairs of warps that zero, each in its stages of the ring
// warps 0: copies, 1: MMA, 4-7: epilogue, the others: zeros
constexpr int LG_THREADS = 32 * (6 + 2 * LG_TEAMS);
constexpr int LG_MAX_STAGES = 8;
constexpr int LG_RING = 192 * 1024;  // beside 25 KiB of plans
constexpr int LG_CHUNKS = 4;     // chunks of 16 rank values in a tile
constexpr int LG_SEGMENT = 6;    // row tiles that one accumulator adds up
constexpr int LG_BOX = LT_ROWS * 128;  // bytes of 64 columns of a row tile

struct GradSide {
    int tiles_c;       // tiles of P's columns
    int cols;
    void* G;
    int64_t step_c, step_j, stride_g;
    bool words;        // rank values next to each other, rows on 16-byte boundaries
};

struct GradParams {
    GradSide side[2];
    int per[2], items;   // of an adapter on each side; of all
    int adapters, rank;
    int plans;
    const LoraPlan* plan;
    LoraParts lay;
    bool f16;            // parts of FP16
    int groups_j;        // tiles of rank values
    int stages, stage_bytes;
    int box_rows;        // rows that a copy brings (what lies behind is zeroed, as others' rows)
    uint32_t idesc;      // with N = 0
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

struct GradItem {
    int which, g, c0, chunk0, chunks;
    int n;  // columns of rank values that the tensor core reads
    int chains;  // accumulators that row tiles take in turn
    // row tiles after which they are added, with rounding, to FP32 sums in the epilogue
    // warps' registers (the tensor core drops what does not fit when it adds: over 8000 rows
    // of one sign 3e-5 in one accumulator)
    __device__ int segment() const { return LG_SEGMENT * chains; }
};

// The plans of all row tiles in shared memory, where they fit: every tile of the
// gradient searches them (about 2 us a tile from global memory, 0.2 from here).
constexpr int LG_PLANS = 512;     // row tiles
constexpr int LG_ENTRIES = 1024;  // adapters of all of them
constexpr int LG_SORTED = 256;    // adapters, at most, that are sorted
struct PlanTable {
    int first[LG_PLANS + 1];      // entries before each row tile
    int ids[LG_ENTRIES];
    alignas(16) uint4 rows[LG_ENTRIES];
    int whole;                    // whether they fit
    int sorted;                   // then: the adapters with the most row tiles first
    int tiles[LG_SORTED], order[LG_SORTED];
};

// (From L2: they are another grid's, and this one does not wait for its end.)
// Every thread of the block calls it; it ends in a block barrier.
__device__ __forceinline__ void load_plans(PlanTable& t, const GradParams& p)
{
    if (threadIdx.x == 0)
        t.whole = t.sorted = 0;
    if (threadIdx.x < LG_SORTED)
        t.tiles[threadIdx.x] = 0;
    if (p.plans <= LG_PLANS) {
        for (int i = threadIdx.x; i < p.plans; i += LG_THREADS)
            t.first[i + 1] = __ldcg(&p.plan[i].count);
        __syncthreads();
        if (threadIdx.x < 32) {
            int sum = 0;
            for (int base = 0; base < p.plans; base += 32) {
                const int i = base + threadIdx.x;
                int v = i < p.plans ? t.first[i + 1] : 0;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int o = __shfl_up_sync(0xffffffffu, v, d);
                    if (static_cast<int>(threadIdx.x) >= d)
                        v += o;
                }
                if (i < p.plans)
                    t.first[i + 1] = sum + v;
                sum += __shfl_sync(0xffffffffu, v, 31);
            }
            if (threadIdx.x == 0) {
                t.first[0] = 0;
                t.whole = sum <= LG_ENTRIES;
                t.sorted = t.whole && p.adapters <= LG_SORTED;
            }
        }
        __syncthreads();
        if (t.whole) {
            for (int e = threadIdx.x; e < t.first[p.plans]; e += LG_THREADS) {
                int lo = 0, hi = p.plans;  // the tile of entry e
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (t.first[mid] <= e)
                        lo = mid;
                    else
                        hi = mid;
                }
                const LoraPlan& plan = p.plan[lo];
                t.ids[e] = __ldcg(&plan.ids[e - t.first[lo]]);
                t.rows[e] = __ldcg(reinterpret_cast<const uint4*>(plan.rows[e - t.first[lo]]));
                if (t.sorted)
                    atomicAdd(&t.tiles[t.ids[e]], 1);
            }
            __syncthreads();
            if (t.sorted && static_cast<int>(threadIdx.x) < p.adapters) {
                const int mine = t.tiles[threadIdx.x];
                int place = 0;
                for (int g = 0; g < p.adapters; ++g)
                    place += t.tiles[g] > mine || (t.tiles[g] == mine && g < static_cast<int>(threadIdx.x));
                t.order[place] = threadIdx.x;
            }
        }
    }
    __syncthreads();
}

// Tile t of the gradients: adapters in the table's order, and of each both sides.
__device__ __forceinline__ GradItem grad_item(int t, const GradParams& p, const PlanTable& table)
{
    GradItem w;
    const int per = p.per[0] + p.per[1], place = t / per;
    t -= place * per;
    w.g = table.sorted ? table.order[place] : place;
    w.which = t >= p.per[0];
    t -= w.which ? p.per[0] : 0;
    w.c0 = t / p.groups_j * 128;
    w.chunk0 = t % p.groups_j * LG_CHUNKS;
    w.chunks = min(LG_CHUNKS, p.lay.chunks - w.chunk0);
    w.n = (w.chunks - 1) * 64 + p.lay.parts * p.lay.chunk;
    w.chains = LG_CHUNKS / w.chunks;
    return w;
}

// The row tiles that hold rows of adapter g, in order; a whole warp steps through
// them together.
class RowTiles {
public:
    __device__ RowTiles(const GradParams& p, const PlanTable& table, int g) : p_(p), table_(table), g_(g) {}
    // The next tile and its rows of g (a bit each); false at the end.
    __device__ bool next(int& tile, uint32_t (&rows)[4])
    {
        while (hits_ == 0) {
            base_ += 32;
            if (base_ >= p_.plans)
                return false;
            look();
        }
        const int src = __ffs(hits_) - 1;
        hits_ &= hits_ - 1;
        tile = base_ + src;
        rows[0] = __shfl_sync(0xffffffffu, mine_.x, src);
        rows[1] = __shfl_sync(0xffffffffu, mine_.y, src);
        rows[2] = __shfl_sync(0xffffffffu, mine_.z, src);
        rows[3] = __shfl_sync(0xffffffffu, mine_.w, src);
        return true;
    }

private:
    // Each lane looks for g in one of 32 plans.
    __device__ void look()
    {
        const int i = base_ + static_cast<int>(lane_id());
        bool found = false;
        if (i < p_.plans) {
            const bool near = table_.whole;
            const int first = near ? table_.first[i] : 0;
            const int count = near ? table_.first[i + 1] - first : __ldcg(&p_.plan[i].count);
            auto id = [&](int e) { return near ? table_.ids[first + e] : __ldcg(&p_.plan[i].ids[e]); };
            int lo = 0, hi = count;  // the first place whose id is not below g
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (id(mid) < g_)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            found = lo < count && id(lo) == g_;
            if (found)
                mine_ = near ? table_.rows[first + lo]
                             : __ldcg(reinterpret_cast<const uint4*>(p_.plan[i].rows[lo]));
        }
        hits_ = __ballot_sync(0xffffffffu, found);
    }

    const GradParams& p_;
    const PlanTable& table_;
    const int g_;
    int base_ = -32;
    uint32_t hits_ = 0;
    uint4 mine_ = {};
};

__device__ __forceinline__ bool all_rows(const uint32_t (&rows)[4])
{
    return (rows[0] & rows[1] & rows[2] & rows[3]) == ~0u;
}
// Whether slice k (16 rows) has any.
__device__ __forceinline__ bool has_slice(const uint32_t (&rows)[4], int k)
{
    return (rows[k >> 1] & (k & 1 ? 0xffff0000u : 0xffffu)) != 0;
}

// p[0 .. n) = v, of 16 values at most, on a 16-byte boundary.
template <typename OutT>
__device__ __forceinline__ void put_words(OutT* p, const float (&v)[16], int n)
{
    constexpr int EACH = 16 / sizeof(OutT);
    alignas(16) OutT h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        put(&h[i], v[i]);
#pragma unroll
    for (int i = 0; i < 16; i += EACH) {
        if (i + EACH <= n) {
            uint4 w;
            memcpy(&w, h + i, 16);
            *reinterpret_cast<uint4*>(p + i) = w;
        } else {
#pragma unroll
            for (int k = i; k < i + EACH; ++k)
                if (k < n)
                    p[k] = h[k];
        }
    }
}

struct GradSmem {
    uint64_t full[LG_MAX_STAGES], landed[LG_MAX_STAGES], empty[LG_MAX_STAGES], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int abort_flag;
    int progress;  // row tiles copied
    PlanTable plans;
};

template <typename OutT>
__global__ void __launch_bounds__(LG_THREADS, 1)
    lora_grad_tc_kernel(const __grid_constant__ CUtensorMap tmP0, const __grid_constant__ CUtensorMap tmT0,
                        const __grid_constant__ CUtensorMap tmP1, const __grid_constant__ CUtensorMap tmT1,
                        const __grid_constant__ GradParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = smem_u32(reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023)));
    __shared__ GradSmem s;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const TcWatch watch{&s.abort_flag, p.status, p.wait_budget};
    volatile int* const progress = &s.progress;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(smem_u32(&s.full[i]), 2);  // (either of the warps that zero)
            mbar_init(smem_u32(&s.landed[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&s.tfull[a]), 1);
            mbar_init(smem_u32(&s.tempty[a]), 4);
        }
        mbar_init(smem_u32(&s.drain), 1);
        s.abort_flag = 0;
        s.progress = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmP0);
        tma_prefetch_desc(&tmT0);
        tma_prefetch_desc(&tmP1);
        tma_prefetch_desc(&tmT1);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&s.tmem), 512);
        tmem_relinquish<1>();
    }
    load_plans(s.plans, p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int stage = 0, steps = 0;
        uint32_t phase = 0;
        uint32_t n_full[LG_MAX_STAGES] = {}, n_landed[LG_MAX_STAGES] = {};
        bool ok = true;
        for (int t = blockIdx.x; ok && t < p.items; t += gridDim.x) {
            const GradItem w = grad_item(t, p, s.plans);
            RowTiles tiles(p, s.plans, w.g);
            int tile, step = 0;
            uint32_t rows[4];
            while (ok && tiles.next(tile, rows)) {
                const bool whole = all_rows(rows);
                const bool skip = step++ == p.fault_skip_kblock;  // (test hook, -1 in normal use)
                ok = warp_wait(smem_u32(&s.empty[stage]), phase ^ 1, watch);
                if (ok && !skip && elect_one()) {
                    const uint32_t bar = smem_u32(whole ? &s.full[stage] : &s.landed[stage]);
                    const uint32_t a0 = ring + stage * p.stage_bytes, b0 = a0 + 2 * LG_BOX;
                    const CUtensorMap* tmP = w.which ? &tmP1 : &tmP0;
                    const CUtensorMap* tmT = w.which ? &tmT1 : &tmT0;
                    if (whole)
                        mbar_arrive(bar);
                    mbar_arrive_expect_tx(bar, (2 + w.chunks) * p.box_rows * 128);
                    tma_load_2d(a0, tmP, bar, w.c0, tile * LT_ROWS);
                    tma_load_2d(a0 + LG_BOX, tmP, bar, w.c0 + 64, tile * LT_ROWS);
                    for (int c = 0; c < w.chunks; ++c)
                        tma_load_2d(b0 + c * LG_BOX, tmT, bar, (w.chunk0 + c) * 64, tile * LT_ROWS);
                }
                __syncwarp();
                ++steps;
                if (lane == 0)
                    *progress = steps;
                if (ok) {
                    n_full[stage] += !skip;  // whichever barrier: full completes once a use
                    n_landed[stage] += !skip && !whole;
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        if (!ok && lane == 0) {  // wait (bounded) for the copies in flight before shared memory goes away
            auto drain = [&](uint64_t* bar, uint32_t uses) {
                const long long t0 = clock64();
                while (uses > 0 && !mbar_try_wait(smem_u32(bar), (uses - 1) & 1) &&
                       clock64() - t0 < p.wait_budget) {
                }
            };
            for (int i = 0; i < p.stages; ++i) {
                drain(&s.full[i], n_full[i]);
                drain(&s.landed[i], n_landed[i]);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        int stage = 0, local = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < p.items; t += gridDim.x) {
            const GradItem w = grad_item(t, p, s.plans);
            RowTiles tiles(p, s.plans, w.g);
            int tile;
            uint32_t rows[4];
            const uint32_t idesc = p.idesc | static_cast<uint32_t>(w.n >> 3) << 17;
            int n = 0;  // row tiles of the segment
            while (ok && tiles.next(tile, rows)) {
                const int acc = local & 1;
                if (n == 0)
                    ok = warp_wait(smem_u32(&s.tempty[acc]), ((local >> 1) & 1) ^ 1, watch);
                ok = ok && warp_wait(smem_u32(&s.full[stage]), phase, watch);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t a0 = ring + stage * p.stage_bytes, b0 = a0 + 2 * LG_BOX;
                const bool last = n == w.segment() - 1;
                if (elect_one()) {
                    bool first = n < w.chains;
                    const uint32_t to = tmem + acc * 256 + n % w.chains * w.chunks * 64;
#pragma unroll
                    for (int k = 0; k < LT_ROWS / TC_UMMA_K; ++k) {
                        if (!has_slice(rows, k))
                            continue;
                        tc_mma_f16<1>(to, smem_desc_sw128(a0 + k * 2048, LG_BOX, 1024),
                                      smem_desc_sw128(b0 + k * 2048, LG_BOX, 1024), idesc, !first);
                        first = false;
                    }
                    tc_commit(smem_u32(&s.empty[stage]));
                    if (last)
                        tc_commit(smem_u32(&s.tfull[acc]));
                }
                __syncwarp();
                n = last ? 0 : n + 1;
                local += last;
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (ok && n > 0) {
                if (elect_one())
                    tc_commit(smem_u32(&s.tfull[local & 1]));
                __syncwarp();
                ++local;
            }
        }
        // Wait (bounded) until every MMA issued so far has completed.
        if (elect_one())
            tc_commit(smem_u32(&s.drain));
        __syncwarp();
        const long long t0 = clock64();
        while (!mbar_try_wait(smem_u32(&s.drain), 0) && clock64() - t0 < p.wait_budget) {
        }
    } else if (warp < 4 || warp >= 8) {
        // ------------------------------------------------ rows of other adapters
        const int half = warp & 1;  // of the rows
        const int team = warp < 4 ? 0 : (warp - 6) / 2;
        int stage = 0;
        uint32_t parity = 0;  // a bit for each stage
        bool ok = true;
        for (int t = blockIdx.x; ok && t < p.items; t += gridDim.x) {
            const GradItem w = grad_item(t, p, s.plans);
            RowTiles tiles(p, s.plans, w.g);
            int tile;
            uint32_t rows[4];
            while (ok && tiles.next(tile, rows)) {
                // (a stage's steps are always the same team's: a barrier whose phases another
                // team waited for would tell this one nothing)
                if (stage % LG_TEAMS == team && !all_rows(rows)) {
                    // (whole row tiles before it, and other teams', are not waited for)
                    ok = warp_wait_behind(smem_u32(&s.landed[stage]), (parity >> stage) & 1, watch, progress);
                    if (!ok)
                        break;
                    parity ^= 1u << stage;
                    // a row is 128 contiguous bytes of each box (its swizzle stays
                    // within): a lane takes 16 of them, of one row in four
#pragma unroll 1
                    for (int r = 64 * half + (lane >> 3); r < 64 * half + 64; r += 4) {
                        if (((rows[r >> 5] >> (r & 31)) & 1) || !has_slice(rows, r >> 4))
                            continue;
                        uint32_t at = ring + stage * p.stage_bytes + r * 128 + (lane & 7) * 16;
                        for (int b = 0; b < 2 + w.chunks; ++b, at += LG_BOX)
                            st_shared_v4(at, 0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&s.full[stage]));
                }
                if (++stage == p.stages)
                    stage = 0;
            }
        }
    } else {
        // ------------------------------------------------ epilogue
        const int q = warp & 3;
        int local = 0;
        for (int t = blockIdx.x; t < p.items; t += gridDim.x) {
            const GradItem w = grad_item(t, p, s.plans);
            const GradSide& side = p.side[w.which];
            RowTiles tiles(p, s.plans, w.g);
            int tile;
            uint32_t rows[4];
            float sum[LG_CHUNKS][16] = {};
            bool ok = true;
            for (bool more = tiles.next(tile, rows); more;) {
                int n = 0;  // row tiles of the segment
                do {
                    ++n;
                    more = tiles.next(tile, rows);
                } while (more && n < w.segment());
                const int acc = local & 1;
                ok = warp_wait_behind(smem_u32(&s.tfull[acc]), (local >> 1) & 1, watch, progress);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
                const int chains = min(n, w.chains);
#pragma unroll
                for (int k = 0; k < LG_CHUNKS; ++k)
                    if (k < w.chunks)
#pragma unroll 1
                        for (int chain = 0; chain < chains; ++chain)
#pragma unroll 1
                            for (int part = 0; part < p.lay.parts; ++part) {
                                uint32_t v[16];
                                tmem_ld_32x32b_x16(from + (chain * w.chunks + k) * 64 + part * 16, v);
                                tmem_wait_ld(v);
                                const float scale = p.f16 ? f16_part_scale(part) : 1.0f;
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    sum[k][i] = fmaf(scale, __uint_as_float(v[i]), sum[k][i]);
                            }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&s.tempty[acc]));
                ++local;
            }
            if (!ok)
                break;
            const int c = w.c0 + q * 32 + static_cast<int>(lane);
            OutT* out = static_cast<OutT*>(side.G) + w.g * side.stride_g + c * side.step_c;
#pragma unroll
            for (int k = 0; k < LG_CHUNKS; ++k) {
                const int j = (w.chunk0 + k) * 16;
                if (k >= w.chunks || c >= side.cols)
                    continue;
                if (side.words) {
                    put_words(out + j, sum[k], p.rank - j);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (j + i < p.rank)
                            put(out + (j + i) * side.step_j, sum[k][i]);
                }
            }
        }
    }

    // ---------------------------------------------------- teardown
    __syncwarp();
    grid_dep_wait();  // this grid must not end before the one it follows
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc<1>(tmem, 512);
}

template <typename OutT>
cudaError_t launch(const CUtensorMap (&m)[4], const GradParams& p, int num_sms, bool dependent,
                   cudaStream_t stream)
{
    static ClusterCaps caps;
    int cap = 0;
    const cudaError_t err =
        cluster_cap(lora_grad_tc_kernel<OutT>, caps, 1, LG_THREADS, LG_RING + 1024, num_sms, &cap);
    if (err != cudaSuccess)
        return err;
    ClusterLaunch l(static_cast<unsigned>(std::min(p.items, num_sms)), 1, LG_THREADS, LG_RING + 1024, stream,
                    dependent);
    return l.run(lora_grad_tc_kernel<OutT>, m[0], m[1], m[2], m[3], p);
}

}  // namespace

cudaError_t lora_grad_tc_launch(const LoraGradLaunch* const (&sides)[2], bool dependent, cudaStream_t stream)
{
    const LoraGradLaunch& l = sides[0] ? *sides[0] : *sides[1];
    GradParams p{};
    p.adapters = l.adapters;
    p.rank = l.rank;
    p.plans = (l.rows + LT_ROWS - 1) / LT_ROWS;
    p.plan = static_cast<const LoraPlan*>(l.plan);
    p.f16 = l.in_dtype == DT_F16;
    p.lay = lora_parts(l.rank, p.f16 ? LT_F16_PARTS : l.parts);  // (of three or four parts: chunks of 16)
    p.groups_j = (p.lay.chunks + LG_CHUNKS - 1) / LG_CHUNKS;
    p.stage_bytes = LG_BOX * (2 + std::min(p.lay.chunks, LG_CHUNKS));
    p.stages = std::min(LG_MAX_STAGES, LG_RING / p.stage_bytes);
    p.idesc = tc_idesc(l.in_dtype == DT_BF16, 128, 0, true, true);
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip_kblock = l.fault_skip_kblock;
    p.box_rows = std::min(LT_ROWS, (l.rows + 7) / 8 * 8);
    const uint32_t box_rows = static_cast<uint32_t>(p.box_rows);
    CUtensorMap m[4];
    int64_t per[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
        if (!sides[i])
            continue;
        const LoraGradLaunch& s = *sides[i];
        const int64_t size = type_bytes(s.out_dtype);
        p.side[i] = {(s.cols + 127) / 128, s.cols, s.G, s.step_c, s.step_j, s.stride_g,
                     s.step_j == 1 && aligned16(s.G) && s.step_c * size % 16 == 0 && s.stride_g * size % 16 == 0};
        per[i] = static_cast<int64_t>(p.side[i].tiles_c) * p.groups_j;
        if (!s.maps->get(&m[2 * i], s.in_dtype, s.P, 2, {s.cols, s.rows, 1}, {s.ldp, 0}, {64, box_rows, 1}) ||
            !s.maps->get(&m[2 * i + 1], s.in_dtype, s.t, 2, {p.lay.columns(), s.rows, 1},
                        {p.lay.columns(), 0}, {64, box_rows, 1}))
            return cudaErrorNotSupported;
    }
    for (int i = 0; i < 2; ++i)
        if (!sides[i]) {
            m[2 * i] = m[2 - 2 * i];
            m[2 * i + 1] = m[3 - 2 * i];
        }
    const int64_t items = (per[0] + per[1]) * l.adapters;
    if (items > 0x7fffffff)
        return cudaErrorNotSupported;
    p.per[0] = static_cast<int>(per[0]);
    p.per[1] = static_cast<int>(per[1]);
    p.items = static_cast<int>(items);
    return with_type(l.out_dtype, [&](auto out) {
        return launch<decltype(out)>(m, p, l.num_sms, dependent, stream);
    });
}

}  // namespace tmmo
