// Newton-Schulz orthogonalisation of matrices with a short side of up to 128,
// in one launch: a cluster of blocks holds one matrix on chip from the first
// read of G to the write of the result.
//
// Such matrices are bound by latency: fifteen dependent products of a
// microsecond or two of tensor work each for five steps.  As separate
// launches a product costs 5 to 7 us whatever its size (set-up, copies from
// L2, stores back, the fences and barriers between grids).  Here
//
//   * X (m x n, m <= n; G transposed while it is read where it has more rows
//     than columns) is divided by columns over the blocks of the cluster.
//     Then the update X <- a X + B X is local to a block, and only
//     A = X X^T, a sum over the blocks, crosses between them;
//   * a thread keeps its values of X (96 or 128) in registers, in FP32, and
//     writes their operand form to shared memory, in the
//     128-byte-swizzled layout of a tensor-core operand.  One copy serves both
//     products: rows of 64 columns are a K-major operand of X X^T and an
//     MN-major one of B X;
//   * operands are two FP16 values an element, hi + lo, and a product is
//     hi hi + hi lo + lo hi in one accumulator, whatever the result's type:
//     with one value matrices as narrow as these would be 2e-3 off and the
//     narrowest up to 7e-3, more than a BF16 result's own rounding (1.66e-3).
//     It costs 15 us a call (128 x 128 36 us instead of 21);
//   * A and B share one buffer: each thread replaces its elements of A by
//     those of B once the product A A is complete, and every block computes
//     all of B for itself;
//   * the sum over blocks goes through distributed shared memory in FP32:
//     a block adds up 1 / SIZE of the rows, in rank order, and writes the
//     operand form to all of them;
//   * G is read once: the norm is taken from the registers.
//
// Five steps of a 128 x 128 matrix take 36 us with the launch; with several
// blocks the exchange adds about 3 us a step, most of it in two cluster
// barriers: 64 x 512 51 us, 128 x 2000 74, 128 x 4000 92.
// Matrices with a short side of up to 256 were tried in the same way and were
// slower than separate launches: the exchange of 256 x 256 FP32 sums took
// 12 us a step.
//
// Eight warps; one of them issues the MMAs, all of them wait for a product's
// completion (bounded) and read it from tensor memory.  A wait that runs out
// is reported as everywhere, the block then only takes part in barriers, and
// no block of its cluster stores what came of its unfinished sums.
#include <cuda_runtime.h>

#include <algorithm>

#include "newton_schulz.cuh"
#include "newton_schulz.h"
#include "persistent.cuh"

namespace tmmo {
namespace {

constexpr int NR_THREADS = 256;
constexpr int NR_MAX_SIZE = 16;  // blocks of a cluster

struct NsResident {
    const void* G;
    void* O;
    // element (i, j) of X at G[z * batch_g + i * row_g + j * col_g], and so in O
    long long batch_g, row_g, col_g, batch_o, row_o, col_o;
    int m, n;
    int num_sms;
    int share;                     // columns of X per block
    bool vec_o;                    // O's rows are on 16-byte boundaries
    int in_dtype, out_dtype;
    int steps;
    float eps;
    float coefficients[3 * NS_MAX_STEPS];
    int* status;
    long long wait_budget;
    int fault_skip;                // test hook: the product whose completion a cluster's first block
                                   // does not signal
};

constexpr int NR_CHUNK = 128 * 128;  // bytes of 64 columns (of 128 rows) of an operand
constexpr uint32_t NR_TMEM_COLS = 256;

// COLS: columns of X a block can hold.
template <int SIZE, int COLS>
struct NrLayout {
    static constexpr int A_LO = 2 * NR_CHUNK, X_LO = COLS / 64 * NR_CHUNK;  // from hi to lo
    static constexpr int OFF_A = 0;                               // 128 x 128, hi and lo
    static constexpr int OFF_X = OFF_A + 2 * A_LO;                // 128 x COLS, hi and lo
    static constexpr int OFF_STAGING = OFF_X + 2 * X_LO;
    // 128 FP32 rows from all blocks, to be added up here: whole, or in halves
    static constexpr int HALVES = COLS == 256 ? 2 : 1;
    static constexpr int STAGING_ROW = 512 / HALVES;
    static constexpr int OFF_BAR = OFF_STAGING + (SIZE > 1 ? 128 * STAGING_ROW : 0);
    static constexpr int SMEM_ALLOC = OFF_BAR + 64 + 1024;
    // (static shared memory: the sums of ns_block_sum)
    static_assert(SMEM_ALLOC + 512 <= 232448, "exceeds 227 KiB of shared memory");
};

// Shared-memory address of 8 columns (16 bytes) of an operand: 64-column
// chunks of 128 rows of 128 bytes, 128-byte swizzle.
__device__ __forceinline__ uint32_t nr_addr(uint32_t base, int row, int col)
{
    return base + (col >> 6) * NR_CHUNK + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4);
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr)
{
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster_b32(uint32_t addr, uint32_t w)
{
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(w) : "memory");
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const uint32_t (&w)[4])
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&w)[4])
{
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
}

// 32 consecutive columns of one row of X from G, `cnt` of them inside.
template <typename InT>
__device__ __forceinline__ void nr_load(const InT* g, long long step, int cnt, float (&v)[32])
{
    if (step == 1) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            float e[8];
            ns_load8(g + i, min(cnt - i, 8), e);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[i + k] = e[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] = i < cnt ? ns_value(g + i * step) : 0.0f;
    }
}

// A warp's 32 rows x 32 columns of the result; tall: the matrix lies
// transposed in O, so a column of X is contiguous over the lanes.
template <typename OutT>
__device__ __forceinline__ void nr_store(OutT* o, const NsResident& p, int row0, int cnt, uint32_t stg,
                                         uint32_t lane, const float (&v)[32])
{
    const int rows = min(p.m - row0, 32);
    if (p.col_o == 1) {
        ns_store_result(o, p.row_o, rows, cnt, p.vec_o, stg, lane, v);
    } else if (static_cast<int>(lane) < rows) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < cnt)
                o[lane * p.row_o + i * p.col_o] = ns_to_out<OutT>(v[i]);
    }
}

template <int SIZE, int COLS>
__global__ void __launch_bounds__(NR_THREADS, 1) ns_resident_kernel(const __grid_constant__ NsResident p)
{
    using L = NrLayout<SIZE, COLS>;
    constexpr int XCH = COLS / 64;  // 32-column chunks of X per thread
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t sA = sbase + L::OFF_A, sX = sbase + L::OFF_X;
    const uint32_t done_bar = sbase + L::OFF_BAR;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_BAR + 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + 12);
    float* sum_slot = reinterpret_cast<float*>(smem + L::OFF_BAR + 16);
    double* wide_slot = reinterpret_cast<double*>(smem + L::OFF_BAR + 32);

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const uint32_t lane = tid & 31;
    const int q = warp & 3, g = warp >> 2;  // TMEM lane quarter; which of two column chunks
    const int rank = SIZE > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const long long z = blockIdx.x / SIZE;
    const int col0 = rank * p.share;                             // this block's columns of X
    const int ncol = min(max(p.n - col0, 0), p.share);
    const TcWatch watch{abort_flag, p.status, p.wait_budget};

    if (tid == 0) {
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc<1>(smem_u32(tmem_slot), NR_TMEM_COLS);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot + (static_cast<uint32_t>(q * 32) << 16);

    // ---- X in registers: row q * 32 + lane, columns in chunks of 32 taken by
    // the two column groups in turn.  Zero outside the matrix; chunks wholly
    // outside are left out everywhere.
    const int row = q * 32 + static_cast<int>(lane);
    float x[XCH][32];
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < XCH; ++c) {
        const int col = (2 * c + g) * 32;
        const int cnt = row < p.m ? min(ncol - col, 32) : 0;
        const long long at = z * p.batch_g + row * p.row_g + (col0 + col) * p.col_g;
        if (p.in_dtype == DT_F32)
            nr_load(static_cast<const float*>(p.G) + at, p.col_g, cnt, x[c]);
        else if (p.in_dtype == DT_F16)
            nr_load(static_cast<const __half*>(p.G) + at, p.col_g, cnt, x[c]);
        else
            nr_load(static_cast<const __nv_bfloat16*>(p.G) + at, p.col_g, cnt, x[c]);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            s = fmaf(x[c][i], x[c][i], s);
    }
    s = ns_block_sum(s);
    if (!ns_squares_fit(s)) {  // (the same for the whole block)
        double wide = 0.0;
#pragma unroll
        for (int c = 0; c < XCH; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
                wide = fma(static_cast<double>(x[c][i]), static_cast<double>(x[c][i]), wide);
        wide = ns_block_sum(wide);
        if (tid == 0)
            *wide_slot = wide;
        if constexpr (SIZE == 1)
            __syncthreads();
    }
    float part[SIZE] = {s};
    if constexpr (SIZE > 1) {
        if (tid == 0)
            *sum_slot = s;
        __syncwarp();
        cluster_sync();
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < SIZE; ++k) {
            part[k] = ld_cluster_f32(mapa_shared(smem_u32(sum_slot), k));
            s += part[k];
        }
    }
    float2 factors;
    if (ns_squares_fit(s)) {
        factors = ns_factors(s, p.eps);
    } else {
        double sum = 0.0;
#pragma unroll
        for (int k = 0; k < SIZE; ++k) {
            if (ns_squares_fit(part[k]))
                sum += part[k];
            else
                sum += SIZE > 1 ? ld_cluster_f64(mapa_shared(smem_u32(wide_slot), k)) : *wide_slot;
        }
        factors = ns_factors_wide(sum, p.eps);
    }
#pragma unroll
    for (int c = 0; c < XCH; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[c][i] = x[c][i] * factors.x * factors.y;

    // Eight values as an operand: hi, and what it leaves.
    auto halves = [](const float* v, uint32_t (&h)[4], uint32_t (&l)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = ns_pack(v[2 * i], v[2 * i + 1]);
            const float2 r = ns_unpack(h[i]);
            l[i] = ns_pack(v[2 * i] - r.x, v[2 * i + 1] - r.y);
        }
    };
    auto put = [&](uint32_t at, uint32_t to_lo, const float* v) {
        uint32_t h[4], l[4];
        halves(v, h, l);
        st_shared_v4(at, h[0], h[1], h[2], h[3]);
        st_shared_v4(at + to_lo, l[0], l[1], l[2], l[3]);
    };
    auto put_x = [&]() {
#pragma unroll
        for (int c = 0; c < XCH; ++c) {
            if ((2 * c + g) * 32 < ncol) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    put(nr_addr(sX, row, (2 * c + g) * 32 + 8 * k), L::X_LO, x[c] + 8 * k);
            }
        }
    };
    put_x();

    // Descriptor constants.  K-major: 8-row groups 1024 bytes apart.
    // MN-major (X in the update): 64-column atoms a chunk apart.
    const uint64_t k_hi = (1ull << 46) | (2ull << 61) | (64ull << 32) | (1ull << 16);
    const uint64_t n_hi = (1ull << 46) | (2ull << 61) | (64ull << 32) |
                          (static_cast<uint64_t>(NR_CHUNK >> 4) << 16);
    const int m_steps = (p.m + 15) / 16;   // K steps over rows; all further rows are zero
    const int n_steps = (ncol + 15) / 16;  // over this block's columns
    const int width = (ncol + 31) / 32 * 32;
    int product = 0;
    bool ok = true;
    // Issues a product of 128 rows (K-major from `a`; `b` K-major as well, or
    // X MN-major; their lo halves a_lo and b_lo further) and waits for it.
    auto multiply = [&](uint32_t a, uint32_t a_lo, uint32_t b, uint32_t b_lo, bool b_mn, int steps, int n) {
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (ok && warp == 0) {
            tc_fence_after();
            const uint32_t idesc = tc_idesc(false, 128, n, false, b_mn);
            const uint32_t d = *tmem_slot;
            if (elect_one()) {
                for (int part = 0; part < 3; ++part) {  // hi hi, hi lo, lo hi
                    const uint32_t pa = a + (part == 2 ? a_lo : 0), pb = b + (part == 1 ? b_lo : 0);
                    for (int k = 0; k < steps; ++k) {
                        const uint32_t off = (k >> 2) * NR_CHUNK + (k & 3) * 32;
                        const uint32_t ka = (pa + off) >> 4, kb = (pb + (b_mn ? k * 2048 : off)) >> 4;
                        tc_mma_f16<1>(d, k_hi | (ka & 0x3FFF), (b_mn ? n_hi : k_hi) | (kb & 0x3FFF), idesc,
                                      part != 0 || k != 0);
                    }
                }
                if (p.fault_skip != product || rank != 0)  // test hook, -1 in normal use
                    tc_commit(done_bar);
            }
            __syncwarp();
        }
        if (ok && !tc_wait_warp(done_bar, static_cast<uint32_t>(product & 1), watch)) {
            ok = false;
            // What this block hands to the others from here on is no sum: with
            // its flag in all of them, none stores.  (They see it behind the
            // barriers of the exchange.)
            if constexpr (SIZE > 1) {
                if (lane < SIZE)
                    st_cluster_b32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), lane), 1);
            }
        }
        tc_fence_after();
        ++product;
    };

    // The loops over A's elements are kept rolled: unrolled, a step is long
    // straight-line code that is fetched anew every time.
#pragma unroll 1
    for (int step = 0; step < p.steps; ++step) {
        const float ca = p.coefficients[3 * step], cb = p.coefficients[3 * step + 1],
                    cc = p.coefficients[3 * step + 2];
        // ---- A = X X^T
        constexpr float alpha_a = NS_SA / (NS_SX * NS_SX);
        multiply(sX, L::X_LO, sX, L::X_LO, false, n_steps, 128);
        if constexpr (SIZE == 1) {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                const int col = (2 * g + c) * 32;
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + col, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        f[i] = alpha_a * __uint_as_float(v[8 * k + i]);
                    put(nr_addr(sA, row, col + 8 * k), L::A_LO, f);
                }
            }
        } else {
            // Every row goes to the block that adds it up, into its staging
            // buffer ([sender][row], 16-byte units swizzled against bank
            // conflicts), and that block adds the senders' rows in rank
            // order.  Rows are pushed, as remote stores do not wait.
            constexpr int HALVES = L::HALVES;            // 128 or 64 columns at a time
            constexpr int UNITS = 16 / HALVES;           // of 8 columns
            constexpr int SHARE = 128 / SIZE;            // rows that this block adds up
            constexpr int ITEMS = SHARE * UNITS;
            constexpr int MINE = (ITEMS + NR_THREADS - 1) / NR_THREADS;
            const uint32_t staging = sbase + L::OFF_STAGING;
            const int to = rank * SHARE + row % SHARE;
            const uint32_t dst =
                mapa_shared(staging + to * L::STAGING_ROW, static_cast<uint32_t>(row / SHARE));
#pragma unroll 1
            for (int h = 0; h < HALVES; ++h) {
                if (HALVES == 1 || g == h) {
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        const int col = (2 * g + c) * 32;
                        const int unit = HALVES == 1 ? col / 4 : c * 8;  // of 4 columns
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(tmem + col, v);
                        tmem_wait_ld(v);
                        if (n_steps == 0) {  // a block without columns adds nothing
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = 0;
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t w[4] = {v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]};
                            st_cluster_v4(dst + (((unit + k) ^ (to & 7)) << 4), w);
                        }
                    }
                }
                __syncwarp();
                cluster_sync();
#pragma unroll
                for (int j = 0; j < MINE; ++j) {
                    const int item = j * NR_THREADS + tid;
                    if (item < ITEMS) {
                        const int r = item / UNITS, u = 2 * (item % UNITS);
                        float a[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            a[i] = 0.0f;
#pragma unroll
                        for (int k = 0; k < SIZE; ++k) {
                            const int from = k * SHARE + r;
                            const uint32_t at = staging + from * L::STAGING_ROW;
                            uint32_t t[4], w[4];
                            ld_shared_v4(at + ((u ^ (from & 7)) << 4), t);
                            ld_shared_v4(at + (((u + 1) ^ (from & 7)) << 4), w);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                a[i] += __uint_as_float(t[i]);
                                a[4 + i] += __uint_as_float(w[i]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            a[i] *= alpha_a;
                        uint32_t hi[4], lo[4];
                        halves(a, hi, lo);
                        const uint32_t at = nr_addr(sA, rank * SHARE + r, 64 * h + 8 * (item % UNITS));
#pragma unroll
                        for (int k = 0; k < SIZE; ++k) {
                            const uint32_t peer = mapa_shared(at, k);
                            st_cluster_v4(peer, hi);
                            st_cluster_v4(peer + L::A_LO, lo);
                        }
                    }
                }
                // the sums are in every block, and the buffer is free for the
                // next half
                fence_proxy_async_cluster();
                __syncwarp();
                cluster_sync();
            }
        }
        // ---- B = b A + c A A, in A's place
        const float alpha_b = cc * (NS_SB / (NS_SA * NS_SA)), beta_b = cb * (NS_SB / NS_SA);
        multiply(sA, L::A_LO, sA, L::A_LO, false, m_steps, 128);
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
            const int col = (2 * g + c) * 32;
            uint32_t v[32];
            tmem_ld_32x32b_x32(tmem + col, v);
            uint32_t w[4][4], l[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                ld_shared_v4(nr_addr(sA, row, col + 8 * k), w[k]);
                ld_shared_v4(nr_addr(sA, row, col + 8 * k) + L::A_LO, l[k]);
            }
            tmem_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = ns_unpack(w[k][i]), r = ns_unpack(l[k][i]);
                    f[2 * i] = fmaf(beta_b, a.x + r.x, alpha_b * __uint_as_float(v[8 * k + 2 * i]));
                    f[2 * i + 1] = fmaf(beta_b, a.y + r.y, alpha_b * __uint_as_float(v[8 * k + 2 * i + 1]));
                }
                put(nr_addr(sA, row, col + 8 * k), L::A_LO, f);
            }
        }
        // ---- X = a X + B X
        multiply(sA, L::A_LO, sX, L::X_LO, true, width > 0 ? m_steps : 0, width > 0 ? width : 32);
#pragma unroll
        for (int c = 0; c < XCH; ++c) {
            if ((2 * c + g) * 32 < ncol) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + (2 * c + g) * 32, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    x[c][i] = fmaf(ca, x[c][i], (1.0f / NS_SB) * __uint_as_float(v[i]));
            }
        }
        if (step + 1 < p.steps)
            put_x();
    }

    // ---- the result
    if (!*abort_flag) {
#pragma unroll
        for (int c = 0; c < XCH; ++c) {
            const int col = (2 * c + g) * 32;
            const int cnt = min(ncol - col, 32), row0 = q * 32;
            if (cnt <= 0)
                continue;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                x[c][i] *= 1.0f / NS_SX;
            // (no MMA reads the operands any more: A's buffer, 4 KiB a warp,
            // serves as staging)
            const uint32_t stg = sA + warp * TC_STAGING_BYTES;
            const long long at = z * p.batch_o + row0 * p.row_o + (col0 + col) * p.col_o;
            if (p.out_dtype == DT_F32)
                nr_store(static_cast<float*>(p.O) + at, p, row0, cnt, stg, lane, x[c]);
            else if (p.out_dtype == DT_F16)
                nr_store(static_cast<__half*>(p.O) + at, p, row0, cnt, stg, lane, x[c]);
            else
                nr_store(static_cast<__nv_bfloat16*>(p.O) + at, p, row0, cnt, stg, lane, x[c]);
        }
    }

    // ---- teardown.  After a wait that ran out the MMAs issued may still be
    // running: one commit more, waited for (bounded), before TMEM is released.
    if (warp == 0 && !ok) {
        const uint32_t drain_bar = sbase + L::OFF_BAR + 24;
        if (elect_one()) {
            mbar_init(drain_bar, 1);
            fence_mbar_init();
            tc_commit(drain_bar);
        }
        __syncwarp();
        const long long t0 = clock64();
        while (!__all_sync(0xffffffffu, mbar_test_wait(drain_bar, 0))) {
            if (__any_sync(0xffffffffu, clock64() - t0 > p.wait_budget))
                break;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
        __syncwarp();
        tmem_dealloc<1>(*tmem_slot, NR_TMEM_COLS);
    }
    if constexpr (SIZE > 1) {  // no block leaves while its shared memory may be read
        __syncwarp();
        cluster_sync();
    }
}

// Launches a batch; with `clusters` only says how many of them run at a time.
template <int SIZE, int COLS>
cudaError_t launch_resident(const NsResident& p, int batch, cudaStream_t stream, int* clusters)
{
    using L = NrLayout<SIZE, COLS>;
    auto kern = ns_resident_kernel<SIZE, COLS>;
    static ClusterCaps caps;
    int cap = 0;
    const cudaError_t err = cluster_cap(kern, caps, SIZE, NR_THREADS, L::SMEM_ALLOC, p.num_sms, &cap);
    if (err != cudaSuccess)
        return err;
    if (cap < 0)
        return cudaErrorNotSupported;
    if (clusters) {
        *clusters = cap;
        return cudaSuccess;
    }
    ClusterLaunch launch(static_cast<unsigned>(batch) * SIZE, SIZE, NR_THREADS, L::SMEM_ALLOC, stream);
    return launch.run(kern, p);
}

// Columns of X for a block of a cluster: 192, what shared memory has room for
// beside A and the staging buffer, or 256 with an exchange in halves, which
// costs two cluster barriers a step more.
constexpr int NR_COLS = 192, NR_MAX_COLS = 256;

struct NrForm {
    int size = 0, cols = 0;  // blocks for one matrix (0: no cluster holds it), columns for a block
};

template <int COLS>
cudaError_t launch_cluster(const NsResident& p, int size, int batch, cudaStream_t stream, int* clusters)
{
    switch (size) {
    case 2:
        return launch_resident<2, COLS>(p, batch, stream, clusters);
    case 4:
        return launch_resident<4, COLS>(p, batch, stream, clusters);
    case 8:
        return launch_resident<8, COLS>(p, batch, stream, clusters);
    default:
        return launch_resident<16, COLS>(p, batch, stream, clusters);
    }
}

cudaError_t launch_form(const NsResident& p, NrForm f, int batch, cudaStream_t stream, int* clusters)
{
    if (f.size == 1)
        return launch_resident<1, NR_MAX_COLS>(p, batch, stream, clusters);
    return f.cols == NR_COLS ? launch_cluster<NR_COLS>(p, f.size, batch, stream, clusters)
                             : launch_cluster<NR_MAX_COLS>(p, f.size, batch, stream, clusters);
}

// The form for a batch.  One matrix alone takes 1.1 to 1.25 times as long with
// 256 columns a block as with twice the blocks (64 x 512 61 us / 51, 64 x 1000
// 70 / 57, 128 x 2000 82 / 74), but of those fewer run at a time: 16 x 128 x
// 1024 78 / 122, 64 x 16 x 2000 344 / 607.  So: 256 where it takes at most four
// fifths of the waves, or where 16 blocks of 192 do not hold the matrix
// (128 x 4000 92 us; as separate launches 267).
NrForm resident_form(const NsResident& p, int batch)
{
    if (p.m > 128 || p.n > NR_MAX_SIZE * NR_MAX_COLS)
        return {};
    if (p.n <= NR_MAX_COLS)
        return {1, NR_MAX_COLS};
    auto with = [&](int cols) {
        NrForm f{2, cols};
        while (f.size * cols < p.n)
            f.size *= 2;
        return f;
    };
    const NrForm narrow = with(NR_COLS), wide = with(NR_MAX_COLS);
    if (narrow.size > NR_MAX_SIZE)
        return wide;
    if (narrow.size == wide.size)
        return narrow;
    int few = 0, many = 0;
    if (launch_form(p, wide, batch, nullptr, &few) != cudaSuccess ||
        launch_form(p, narrow, batch, nullptr, &many) != cudaSuccess) {
        cudaGetLastError();  // whether the form chosen fits is asked once more
        return narrow;
    }
    const long long wide_waves = (batch + few - 1) / few, narrow_waves = (batch + many - 1) / many;
    return 5 * wide_waves <= 4 * narrow_waves ? wide : narrow;
}

NsResident resident_params(const NsLaunch& l)
{
    NsResident p{};
    p.m = std::min(l.rows, l.cols);
    p.n = std::max(l.rows, l.cols);
    p.num_sms = l.num_sms;
    return p;
}

}  // namespace

bool ns_resident_takes(const NsLaunch& l)
{
    const NsResident p = resident_params(l);
    const NrForm form = resident_form(p, l.batch);
    int clusters = 0;
    if (form.size > 0 && static_cast<long long>(l.batch) * form.size <= 0x7fffffffLL &&
        launch_form(p, form, l.batch, nullptr, &clusters) == cudaSuccess)
        return true;
    cudaGetLastError();  // a query that failed is not the separate launches' error
    return false;
}

cudaError_t ns_resident_launch(const NsLaunch& l, cudaStream_t stream)
{
    const bool tall = l.rows > l.cols;
    NsResident p = resident_params(l);
    const NrForm form = resident_form(p, l.batch);
    p.G = l.G;
    p.O = l.O;
    p.batch_g = l.batch_g;
    p.batch_o = l.batch_o;
    p.row_g = tall ? 1 : l.ldg;
    p.col_g = tall ? l.ldg : 1;
    p.row_o = tall ? 1 : l.ldo;
    p.col_o = tall ? l.ldo : 1;
    p.share = ((p.n + form.size - 1) / form.size + 15) / 16 * 16;
    p.vec_o = ns_vec_rows(l);
    p.in_dtype = l.in_dtype;
    p.out_dtype = l.out_dtype;
    p.steps = l.steps;
    p.eps = l.eps;
    std::copy(l.coefficients, l.coefficients + 3 * l.steps, p.coefficients);
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip = l.fault_skip_kblock;
    return launch_form(p, form, l.batch, stream, nullptr);
}

}  // namespace tmmo
