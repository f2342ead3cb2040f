// C entry points of the block-scaled 8-bit operators: argument checks and
// the translation to the internal launchers.
#include <cuda_runtime.h>

#include <cstdint>

#include "device.h"
#include "fp8.h"
#include "launch.h"
#include "tiled_gemm.h"

namespace tmmo {
namespace {

bool valid_size(int64_t n) { return n >= 0 && n <= GEMM_MAX_DIM; }
bool valid_dtype(int t) { return t == GEMM_F32 || t == GEMM_F16 || t == GEMM_BF16; }
bool valid_f8(int t) { return t == GEMM_F8_E4M3 || t == GEMM_F8_E5M2; }
bool valid_block(int b) { return b == GEMM_FP8_ROW || b == GEMM_FP8_COL || b == GEMM_FP8_TILE; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }

// The least scale pitch of a stored rows x cols matrix.
int64_t least_lds(int block, int64_t rows, int64_t cols)
{
    return block == GEMM_FP8_ROW ? rows : block == GEMM_FP8_COL ? cols : blocks128(cols);
}

int check_output(const void* Q, int64_t ldq, const float* S, int64_t lds, int block, int64_t rows,
                 int64_t cols)
{
    if (!Q || !S || ldq < cols || lds < least_lds(block, rows, cols))
        return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(Q) || ldq % 16 != 0)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

int check_input(const void* X, int64_t ldx, int64_t rows, int64_t cols, int in_dtype, int f8)
{
    if (!valid_size(rows) || !valid_size(cols) || !valid_dtype(in_dtype) || !valid_f8(f8))
        return GEMM_ERR_INVALID_VALUE;
    if (rows > 0 && cols > 0 && (!X || ldx < cols))
        return GEMM_ERR_INVALID_VALUE;
    return GEMM_OK;
}

int status_of(cudaError_t err)
{
    if (err == cudaErrorNotSupported)
        return GEMM_ERR_UNSUPPORTED;
    return err == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

Fp8Quantize quantize_input(const void* X, int64_t ldx, int64_t rows, int64_t cols, int in_dtype,
                           int f8)
{
    Fp8Quantize q{};
    q.X = X;
    q.ldx = ldx;
    q.rows = static_cast<int>(rows);
    q.cols = static_cast<int>(cols);
    q.in_dtype = in_dtype;
    q.f8 = f8;
    return q;
}

// Checks one operand of a product, stored with K contiguous or (mn_major)
// across its rows, and fills the internal form.
int operand(const gemm_fp8_matrix_t& m, bool mn_major, int64_t outer, int64_t K, Fp8Operand* o)
{
    if (!valid_f8(m.type) || !valid_block(m.block))
        return GEMM_ERR_INVALID_VALUE;
    const int64_t rows = mn_major ? K : outer, cols = mn_major ? outer : K;
    if (!m.data || !m.scale || m.ld < cols || m.scale_ld < least_lds(m.block, rows, cols))
        return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(m.data) || m.ld % 16 != 0)
        return GEMM_ERR_UNSUPPORTED;
    if (m.block != GEMM_FP8_TILE && m.block != (mn_major ? GEMM_FP8_COL : GEMM_FP8_ROW))
        return GEMM_ERR_UNSUPPORTED;
    o->data = m.data;
    o->ld = m.ld;
    o->mn_major = mn_major;
    o->type = m.type;
    o->scale = m.scale;
    if (m.block == GEMM_FP8_TILE) {
        o->shift = 7;
        o->stride_k = mn_major ? m.scale_ld : 1;
        o->stride_o = mn_major ? 1 : m.scale_ld;
    } else {
        o->shift = 0;
        o->stride_k = m.scale_ld;
        o->stride_o = 1;
    }
    return GEMM_OK;
}

}  // namespace
}  // namespace tmmo

using namespace tmmo;

extern "C" int gemm_fp8_quantize(const void* X, int64_t ldx, int64_t rows, int64_t cols,
                                 gemm_dtype_t in_dtype, gemm_f8_t f8, gemm_fp8_block_t block,
                                 void* Q, int64_t ldq, float* S, int64_t lds, void* stream)
{
    int rc = check_input(X, ldx, rows, cols, in_dtype, f8);
    if (rc == GEMM_OK && !valid_block(block))
        rc = GEMM_ERR_INVALID_VALUE;
    if (rc != GEMM_OK || rows == 0 || cols == 0)
        return rc;
    rc = check_output(Q, ldq, S, lds, block, rows, cols);
    if (rc != GEMM_OK)
        return rc;
    Fp8Quantize q = quantize_input(X, ldx, rows, cols, in_dtype, f8);
    if (block == GEMM_FP8_ROW) {
        q.q_row = Q;
        q.ld_row = ldq;
        q.s_row = S;
        q.lds_row = lds;
    } else if (block == GEMM_FP8_COL) {
        q.q_col = Q;
        q.ld_col = ldq;
        q.s_col = S;
        q.lds_col = lds;
    } else {
        q.q_tile = Q;
        q.ld_tile = ldq;
        q.s_tile = S;
        q.lds_tile = lds;
    }
    return status_of(fp8_quantize_launch(q, static_cast<cudaStream_t>(stream)));
}

extern "C" int gemm_fp8_quantize_pair(const void* X, int64_t ldx, int64_t rows, int64_t cols,
                                      gemm_dtype_t in_dtype, gemm_f8_t f8, void* Q_row,
                                      int64_t ldq_row, float* S_row, int64_t lds_row, void* Q_col,
                                      int64_t ldq_col, float* S_col, int64_t lds_col, void* stream)
{
    int rc = check_input(X, ldx, rows, cols, in_dtype, f8);
    if (rc != GEMM_OK || rows == 0 || cols == 0)
        return rc;
    rc = check_output(Q_row, ldq_row, S_row, lds_row, GEMM_FP8_ROW, rows, cols);
    if (rc == GEMM_OK)
        rc = check_output(Q_col, ldq_col, S_col, lds_col, GEMM_FP8_COL, rows, cols);
    if (rc != GEMM_OK)
        return rc;
    Fp8Quantize q = quantize_input(X, ldx, rows, cols, in_dtype, f8);
    q.q_row = Q_row;
    q.ld_row = ldq_row;
    q.s_row = S_row;
    q.lds_row = lds_row;
    q.q_col = Q_col;
    q.ld_col = ldq_col;
    q.s_col = S_col;
    q.lds_col = lds_col;
    return status_of(fp8_quantize_launch(q, static_cast<cudaStream_t>(stream)));
}

extern "C" int gemm_fp8(const gemm_fp8_matrix_t* A, const gemm_fp8_matrix_t* B, void* C,
                        int64_t ldc, int64_t M, int64_t N, int64_t K, float alpha, float beta,
                        gemm_dtype_t out_dtype, void* stream)
{
    if (!A || !B || !valid_size(M) || !valid_size(N) || !valid_size(K) || !valid_dtype(out_dtype))
        return GEMM_ERR_INVALID_VALUE;
    if ((A->op != GEMM_OP_N && A->op != GEMM_OP_T) || (B->op != GEMM_OP_N && B->op != GEMM_OP_T))
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0)
        return GEMM_OK;
    if (!C || ldc < N)
        return GEMM_ERR_INVALID_VALUE;
    Fp8Launch l{};
    if (K > 0) {
        int rc = operand(*A, A->op == GEMM_OP_T, M, K, &l.a);
        if (rc == GEMM_OK)
            rc = operand(*B, B->op == GEMM_OP_N, N, K, &l.b);
        if (rc != GEMM_OK)
            return rc;
    }
    DeviceInfo d;
    if (device_info(&d) != cudaSuccess)
        return GEMM_ERR_CUDA;
    l.C = C;
    l.ldc = ldc;
    l.M = static_cast<int>(M);
    l.N = static_cast<int>(N);
    l.K = static_cast<int>(K);
    l.out_dtype = out_dtype;
    l.alpha = alpha;
    l.beta = beta;
    l.num_sms = d.num_sms;
    l.status = d.status;
    l.wait_budget = wait_budget_cycles();
    l.fault_skip_kblock = fault_skip_kblock();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return status_of(K > 0 ? fp8_gemm_launch(l, s) : fp8_empty_launch(l, s));
}
