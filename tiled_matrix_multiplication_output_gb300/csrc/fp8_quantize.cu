// Quantisation of a matrix into 8-bit floating point with one FP32 scale for
// each block of 128.
//
// For a block b of X (1 x 128, 128 x 1 or 128 x 128 elements) and the 8-bit
// type's largest value F (448 for e4m3, 57344 for e5m2):
//
//     amax = max |x| over the finite x of b
//     s    = max(amax * (1 / F), 2^-126), or 1 where amax = 0
//     q    = rn8(x * (1 / s)), non-finite x -> the 8-bit NaN
//
// with 1 / F, both products and 1 / s rounded to FP32 (nearest even), so the
// codes are determined bit for bit.  2^-126 keeps 1 / s finite.
//
// Bound: HBM.  An element is read once (2 or 4 bytes) and written once for
// each form (1 byte).  A block of threads holds one 128 x 128 tile in
// registers: thread t owns 8 consecutive columns (t % 16) of 8 consecutive
// rows (t / 16), so a load instruction reads whole 256-byte row segments,
// all of a thread's loads are in flight together, and each block shape's
// largest magnitude is a reduction over registers -- over 16 lanes for
// 1 x 128, over the threads of a column for 128 x 1, over all for 128 x 128
// -- so the two vector forms that training needs (the forward product and
// the weight gradient contract over different axes) come from one read.
// Besides the bytes the arithmetic counts, as 13 elements pass an SM a cycle
// at the full rate: maxima are taken on packed 16-bit integers, values that
// are not finite are looked for in the maxima only, a row's scale is worked
// out by one lane.  Measured on GB300, 8192 x 8192 BF16: 128 x 128 32 us
// (6.3 TB/s, 0.93 of the measured copy bandwidth), 1 x 128 33, 128 x 1 35,
// both vectors 55 (4.8); FP32, 1 x 128, 55 (6.1).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fp8.h"
#include "launch.h"
#include "load8.cuh"

namespace tmmo {
namespace {

constexpr int QT = 128;        // tile side
constexpr int Q_THREADS = 256;
constexpr int Q_ROWS = 8;      // rows per thread
constexpr int Q_COLS = 8;      // columns per thread

enum { Q_ROW = 1, Q_COL = 2, Q_TILE = 4 };

// Magnitudes are compared as integers: with the sign bit cleared, IEEE values
// order like their bits, non-finite ones above all others.  A maximum at or
// above LIMIT (the bits of infinity) therefore says that a block holds a
// value that is not finite, and only then is it taken again over magnitudes
// that leave those out (`finite`).
template <typename T>
struct QIn;
template <>
struct QIn<float> {
    static constexpr int WORDS = 8;   // 32-bit words of 8 elements
    static constexpr uint32_t LIMIT = 0x7f800000u;
    static __device__ uint32_t mag(uint32_t w) { return w & 0x7fffffffu; }
    static __device__ uint32_t finite(uint32_t w)
    {
        const uint32_t m = mag(w);
        return m < LIMIT ? m : 0u;
    }
    static __device__ uint32_t vmax(uint32_t a, uint32_t b) { return max(a, b); }
    static __device__ uint32_t combine(uint32_t m) { return m; }
    static __device__ float value(uint32_t m) { return __uint_as_float(m); }
    static __device__ void unpack(const uint32_t (&w)[8], float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __uint_as_float(w[i]);
    }
};
// Two 16-bit values a word.
template <uint32_t INF>
struct QIn16 {
    static constexpr int WORDS = 4;
    static constexpr uint32_t LIMIT = INF;
    static __device__ uint32_t mag(uint32_t w) { return w & 0x7fff7fffu; }
    static __device__ uint32_t finite(uint32_t w)
    {
        const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
        return (lo < INF ? lo : 0u) | ((hi < INF ? hi : 0u) << 16);
    }
    static __device__ uint32_t vmax(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
    static __device__ uint32_t combine(uint32_t m) { return max(m & 0xffffu, m >> 16); }
};
template <>
struct QIn<__nv_bfloat16> : QIn16<0x7f80u> {
    static __device__ float value(uint32_t m) { return __uint_as_float(m << 16); }
    static __device__ void unpack(const uint32_t (&w)[4], float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct QIn<__half> : QIn16<0x7c00u> {
    static __device__ float value(uint32_t m)
    {
        return __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
    }
    static __device__ void unpack(const uint32_t (&w)[4], float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};

// 1 / F rounded to FP32.
__device__ __forceinline__ float q_inverse_max(int f8)
{
    return f8 == F8_E4M3 ? 9586981.0f * 0x1p-32f : 9586981.0f * 0x1p-39f;
}

__device__ __forceinline__ float q_scale(float amax, float inv_max)
{
    return amax > 0.0f ? fmaxf(__fmul_rn(amax, inv_max), 0x1p-126f) : 1.0f;
}

__device__ __forceinline__ uint32_t q_pair(float lo, float hi, __nv_fp8_interpretation_t kind)
{
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, kind);
}

struct QParams {
    const void* X;
    int64_t ldx;
    int rows, cols;
    int col_blocks;
    int f8;
    uint8_t *q_row, *q_col, *q_tile;
    float *s_row, *s_col, *s_tile;
    int64_t ld_row, ld_col, ld_tile;
    int64_t lds_row, lds_col, lds_tile;
};

// One thread's 8 codes x * r of one row; `n` of them lie inside the matrix.
// EXACT: some of them may be infinite.  Then x * r + x * 0 makes those NaN,
// where the saturating conversion alone would give +-F, and is x * r for the
// finite ones.  (A NaN stays one either way.)
template <bool EXACT>
__device__ __forceinline__ void q_store(uint8_t* dst, const float (&v)[8], const float (&r)[8],
                                        int n, int f8)
{
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        t[i] = EXACT ? fmaf(v[i], r[i], __fmul_rn(v[i], 0.0f)) : __fmul_rn(v[i], r[i]);
    uint32_t lo, hi;
    if (f8 == F8_E4M3) {
        lo = q_pair(t[0], t[1], __NV_E4M3) | (q_pair(t[2], t[3], __NV_E4M3) << 16);
        hi = q_pair(t[4], t[5], __NV_E4M3) | (q_pair(t[6], t[7], __NV_E4M3) << 16);
    } else {
        lo = q_pair(t[0], t[1], __NV_E5M2) | (q_pair(t[2], t[3], __NV_E5M2) << 16);
        hi = q_pair(t[4], t[5], __NV_E5M2) | (q_pair(t[6], t[7], __NV_E5M2) << 16);
    }
    if (n == 8) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    } else {
        for (int i = 0; i < n; ++i)
            dst[i] = static_cast<uint8_t>((i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) & 0xffu);
    }
}

// The largest magnitude of a thread's 8 elements of a row (a word, to be
// combined) and of its 8 columns over its rows.
template <typename In, bool EXACT>
__device__ __forceinline__ uint32_t q_mag(uint32_t w)
{
    return EXACT ? In::finite(w) : In::mag(w);
}

// The tile in registers: maxima, scales, codes.  EXACT as in q_store; without
// it, returns false as soon as a maximum shows a value that is not finite,
// for the whole block alike and before anything is written.
template <typename InT, int FORMS, bool EXACT>
__device__ __forceinline__ bool q_tile(const QParams& p, const uint32_t (&w)[Q_ROWS][QIn<InT>::WORDS],
                                       uint32_t (&s_max)[Q_THREADS / 32][16 * QIn<InT>::WORDS], int rb,
                                       int cb, int row0, int col0, int nrow, int ncol)
{
    using In = QIn<InT>;
    constexpr int W = In::WORDS;
    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    const int cg = tid & 15, rg = tid >> 4;
    const float inv_max = q_inverse_max(p.f8);

    // a maximum for each column of the thread over its rows, then over the
    // warp's two row groups and (through shared memory) the warps
    uint32_t m[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        m[j] = q_mag<In, EXACT>(w[0][j]);
#pragma unroll
        for (int i = 1; i < Q_ROWS; ++i)
            m[j] = In::vmax(m[j], q_mag<In, EXACT>(w[i][j]));
    }
    uint32_t all = m[0];
#pragma unroll
    for (int j = 1; j < W; ++j)
        all = In::vmax(all, m[j]);
    all = In::combine(all);
    if constexpr ((FORMS & Q_COL) != 0) {
        if (!EXACT && __syncthreads_or(all >= In::LIMIT))
            return false;
#pragma unroll
        for (int j = 0; j < W; ++j)
            m[j] = In::vmax(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        if (lane < 16) {
#pragma unroll
            for (int j = 0; j < W; ++j)
                s_max[warp][cg * W + j] = m[j];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < Q_THREADS / 32; ++k) {
#pragma unroll
            for (int j = 0; j < W; ++j)
                m[j] = In::vmax(m[j], s_max[k][cg * W + j]);
        }
    } else if constexpr ((FORMS & Q_TILE) != 0) {
        all = __reduce_max_sync(0xffffffffu, all);
        if (lane == 0)
            s_max[warp][0] = all;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < Q_THREADS / 32; ++k)
            all = max(all, s_max[k][0]);
        if (!EXACT && all >= In::LIMIT)
            return false;
    } else {
        if (!EXACT && __any_sync(0xffffffffu, all >= In::LIMIT))
            return false;  // (a warp's rows are its own)
    }

    float rc[8];  // the factors of the column or tile form
    if constexpr ((FORMS & Q_COL) != 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = W == 8 ? m[j % W] : (m[j >> 1] >> (16 * (j & 1))) & 0xffffu;
            const float s = q_scale(In::value(b), inv_max);
            rc[j] = __frcp_rn(s);
            if (rg == 0 && j < ncol)
                p.s_col[rb * p.lds_col + col0 + j] = s;
        }
    } else if constexpr ((FORMS & Q_TILE) != 0) {
        const float s = q_scale(In::value(all), inv_max);
        if (tid == 0)
            p.s_tile[rb * p.lds_tile + cb] = s;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            rc[j] = __frcp_rn(s);
    }
    // The factors of the thread's rows: maxima over the 16 lanes that share
    // them (two 16-bit ones a shuffle), then each lane takes one row's scale
    // and inverse, and the inverses go round.
    float rr[Q_ROWS];
    if constexpr ((FORMS & Q_ROW) != 0) {
        constexpr int PER = W == 8 ? 1 : 2;  // rows per word
        uint32_t t[Q_ROWS / PER];
#pragma unroll
        for (int i = 0; i < Q_ROWS; ++i) {
            uint32_t u = q_mag<In, EXACT>(w[i][0]);
#pragma unroll
            for (int j = 1; j < W; ++j)
                u = In::vmax(u, q_mag<In, EXACT>(w[i][j]));
            u = In::combine(u);
            t[i / PER] = i % PER ? t[i / PER] | (u << 16) : u;
        }
#pragma unroll
        for (int i = 0; i < Q_ROWS / PER; ++i) {
#pragma unroll
            for (int d = 8; d > 0; d >>= 1)
                t[i] = In::vmax(t[i], __shfl_xor_sync(0xffffffffu, t[i], d));
        }
        const int own = cg & 7;
        uint32_t u = t[0];
#pragma unroll
        for (int i = 1; i < Q_ROWS / PER; ++i)
            u = own / PER == i ? t[i] : u;
        if (PER == 2)
            u = (u >> (16 * (own & 1))) & 0xffffu;
        const float s = q_scale(In::value(u), inv_max);
        if (cg < nrow)
            p.s_row[cb * p.lds_row + row0 + cg] = s;
        const float r = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < Q_ROWS; ++i)
            rr[i] = __shfl_sync(0xffffffffu, r, i, 16);
    }
#pragma unroll
    for (int i = 0; i < Q_ROWS; ++i) {
        float v[8];
        In::unpack(w[i], v);
        if constexpr ((FORMS & Q_ROW) != 0) {
            float r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                r[j] = rr[i];
            if (i < nrow)
                q_store<EXACT>(p.q_row + static_cast<int64_t>(row0 + i) * p.ld_row + col0, v, r, ncol, p.f8);
        }
        if constexpr ((FORMS & Q_COL) != 0) {
            if (i < nrow)
                q_store<EXACT>(p.q_col + static_cast<int64_t>(row0 + i) * p.ld_col + col0, v, rc, ncol, p.f8);
        }
        if constexpr ((FORMS & Q_TILE) != 0) {
            if (i < nrow)
                q_store<EXACT>(p.q_tile + static_cast<int64_t>(row0 + i) * p.ld_tile + col0, v, rc, ncol,
                               p.f8);
        }
    }
    return true;
}

// Blocks on an SM: each holds 32 KiB (16-bit X) or 64 KiB in flight.
template <typename InT, int FORMS, bool VEC>
__global__ void __launch_bounds__(Q_THREADS, sizeof(InT) == 4 ? 2 : FORMS == (Q_ROW | Q_COL) ? 3 : 4)
    fp8_quantize_kernel(const QParams p)
{
    constexpr int W = QIn<InT>::WORDS;
    __shared__ uint32_t s_max[Q_THREADS / 32][16 * W];

    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int cb = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.col_blocks));
    const int rb = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.col_blocks));
    const int row0 = rb * QT + rg * Q_ROWS;
    const int col0 = cb * QT + cg * Q_COLS;
    const int ncol = min(max(p.cols - col0, 0), Q_COLS);   // columns of this thread inside X
    const int nrow = min(max(p.rows - row0, 0), Q_ROWS);

    // ---- load: zeros outside X, which change no maximum
    uint32_t w[Q_ROWS][W];
    const InT* src = static_cast<const InT*>(p.X) + static_cast<int64_t>(row0) * p.ldx + col0;
#pragma unroll
    for (int i = 0; i < Q_ROWS; ++i) {
        if (VEC && i < nrow && ncol == Q_COLS) {  // whole, on a 16-byte boundary
#pragma unroll
            for (int j = 0; j < W / 4; ++j) {
                const uint4 u = __ldcs(reinterpret_cast<const uint4*>(src + i * p.ldx) + j);
                w[i][4 * j] = u.x;
                w[i][4 * j + 1] = u.y;
                w[i][4 * j + 2] = u.z;
                w[i][4 * j + 3] = u.w;
            }
        } else {
            load8(src + i * p.ldx, i < nrow ? ncol : 0, w[i]);
        }
    }

    if (!q_tile<InT, FORMS, false>(p, w, s_max, rb, cb, row0, col0, nrow, ncol)) {
        if (FORMS != Q_ROW)
            __syncthreads();  // the maxima in shared memory have been read
        q_tile<InT, FORMS, true>(p, w, s_max, rb, cb, row0, col0, nrow, ncol);
    }
}

template <typename InT, int FORMS>
cudaError_t launch(const QParams& p, unsigned grid, bool vec, cudaStream_t s)
{
    note_launch();
    if (vec)
        fp8_quantize_kernel<InT, FORMS, true><<<grid, Q_THREADS, 0, s>>>(p);
    else
        fp8_quantize_kernel<InT, FORMS, false><<<grid, Q_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename InT>
cudaError_t launch_forms(const QParams& p, unsigned grid, bool vec, cudaStream_t s)
{
    if (p.q_tile)
        return launch<InT, Q_TILE>(p, grid, vec, s);
    if (p.q_row && p.q_col)
        return launch<InT, Q_ROW | Q_COL>(p, grid, vec, s);
    if (p.q_row)
        return launch<InT, Q_ROW>(p, grid, vec, s);
    return launch<InT, Q_COL>(p, grid, vec, s);
}

}  // namespace

cudaError_t fp8_quantize_launch(const Fp8Quantize& q, cudaStream_t stream)
{
    QParams p{};
    p.X = q.X;
    p.ldx = q.ldx;
    p.rows = q.rows;
    p.cols = q.cols;
    p.col_blocks = (q.cols + QT - 1) / QT;
    p.f8 = q.f8;
    p.q_row = static_cast<uint8_t*>(q.q_row);
    p.q_col = static_cast<uint8_t*>(q.q_col);
    p.q_tile = static_cast<uint8_t*>(q.q_tile);
    p.s_row = q.s_row;
    p.s_col = q.s_col;
    p.s_tile = q.s_tile;
    p.ld_row = q.ld_row;
    p.ld_col = q.ld_col;
    p.ld_tile = q.ld_tile;
    p.lds_row = q.lds_row;
    p.lds_col = q.lds_col;
    p.lds_tile = q.lds_tile;
    const long long blocks = static_cast<long long>((q.rows + QT - 1) / QT) * p.col_blocks;
    if (blocks > 0x7fffffffLL)
        return cudaErrorNotSupported;
    const int es = q.in_dtype == DT_F32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(q.X) & 15u) == 0 && (q.ldx * es) % 16 == 0;
    const unsigned grid = static_cast<unsigned>(blocks);
    switch (q.in_dtype) {
    case DT_F32:
        return launch_forms<float>(p, grid, vec, stream);
    case DT_F16:
        return launch_forms<__half>(p, grid, vec, stream);
    default:
        return launch_forms<__nv_bfloat16>(p, grid, vec, stream);
    }
}

}  // namespace tmmo
