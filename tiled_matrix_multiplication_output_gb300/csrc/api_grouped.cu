// C entry points of the products grouped by rows: argument checks and the
// translation to the internal launchers.
#include <cuda_runtime.h>

#include <cstdint>

#include "api_checks.h"
#include "device.h"
#include "grouped.h"
#include "launch.h"
#include "pack.h"
#include "tiled_gemm.h"

using namespace tmmo;

static_assert(kMaxGroups == GEMM_MAX_GROUPS, "the table's size");

namespace {

int check_grouping(int64_t rows, int64_t groups, int64_t N, int64_t K,
                   int in_dtype, int out_dtype)
{
    if (!valid_size(rows) || !valid_size(N) || !valid_size(K) || groups < 0 ||
        !valid_dtype(in_dtype) || !valid_dtype(out_dtype))
        return GEMM_ERR_INVALID_VALUE;
    if (groups > GEMM_MAX_GROUPS)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// The weights as a stack of stored matrices.
PackMatrix weights(const void* W, int64_t ldw, int64_t stride, int64_t groups, int64_t N, int64_t K,
                   int op)
{
    return {W, ldw, stride, groups, op == GEMM_OP_T ? N : K, op == GEMM_OP_T ? K : N};
}

}  // namespace

extern "C" size_t gemm_grouped_workspace_size(const void* X, int64_t ldx, const void* W, int64_t ldw,
                                              int64_t stride_w, int64_t rows, int64_t groups,
                                              int64_t N, int64_t K, gemm_op_t op_w,
                                              gemm_dtype_t in_dtype)
{
    if (in_dtype == GEMM_F32 || check_grouping(rows, groups, N, K, in_dtype, GEMM_F32) != GEMM_OK)
        return 0;
    PackMatrix x{X, ldx, 0, 1, rows, K}, w = weights(W, ldw, stride_w, groups, N, K, op_w);
    Packing packing;
    packing.add(&x);
    packing.add(&w, true);
    return packing.bytes();
}

extern "C" int gemm_grouped(const void* X, int64_t ldx, const void* W, int64_t ldw,
                            int64_t stride_w, gemm_op_t op_w, const int32_t* offsets, void* Y,
                            int64_t ldy, int64_t rows, int64_t groups, int64_t N, int64_t K,
                            float alpha, float beta, int zero_rest, gemm_dtype_t in_dtype,
                            gemm_dtype_t out_dtype, void* workspace, size_t workspace_bytes,
                            void* stream)
{
    int rc = check_grouping(rows, groups, N, K, in_dtype, out_dtype);
    if (rc == GEMM_OK && op_w != GEMM_OP_N && op_w != GEMM_OP_T)
        rc = GEMM_ERR_INVALID_VALUE;
    if (rc != GEMM_OK || rows == 0 || N == 0)
        return rc;
    if (!offsets || !Y || ldy < N)
        return GEMM_ERR_INVALID_VALUE;
    if (K > 0 && groups > 0 &&
        (!X || !W || ldx < K || ldw < (op_w == GEMM_OP_T ? K : N) || stride_w < 0))
        return GEMM_ERR_INVALID_VALUE;
    PackMatrix x{X, ldx, 0, 1, rows, K}, w = weights(W, ldw, stride_w, groups, N, K, op_w);
    Packing packing;
    if (in_dtype != GEMM_F32) {
        packing.add(&x);
        packing.add(&w, true);
    }
    if (bad_workspace(workspace, workspace_bytes, packing.bytes()))
        return GEMM_ERR_INVALID_VALUE;
    DeviceInfo d;
    if (device_info(&d) != cudaSuccess)
        return GEMM_ERR_CUDA;
    GroupedLaunch l{};
    l.by = {offsets, static_cast<int>(groups), static_cast<int>(rows)};
    l.X = X;
    l.ldx = ldx;
    l.W = W;
    l.ldw = ldw;
    l.stride_w = stride_w;
    l.w_t = op_w == GEMM_OP_T;
    l.Y = Y;
    l.ldy = ldy;
    l.N = static_cast<int>(N);
    l.K = static_cast<int>(K);
    l.alpha = alpha;
    l.beta = beta;
    l.zero_rest = zero_rest != 0;
    l.in_dtype = in_dtype;
    l.out_dtype = out_dtype;
    l.num_sms = d.num_sms;
    l.status = d.status;
    l.wait_budget = wait_budget_cycles();
    l.fault_skip_kblock = fault_skip_kblock();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (in_dtype == GEMM_F32 || K == 0 || groups == 0)
        return status_of(grouped_simt_launch(l, s));
    cudaError_t err = packing.run(workspace, d.num_sms, s);
    l.X = x.p;
    l.ldx = x.ld;
    l.W = w.p;
    l.ldw = w.ld;
    l.stride_w = w.stride;
    if (err == cudaSuccess)
        err = grouped_tc_launch(l, s);
    return status_of(err);
}

extern "C" size_t gemm_grouped_wgrad_workspace_size(const void* D, int64_t ldd, const void* X,
                                                    int64_t ldx, int64_t rows, int64_t N, int64_t K,
                                                    gemm_dtype_t in_dtype)
{
    if (in_dtype == GEMM_F32 || check_grouping(rows, 0, N, K, in_dtype, GEMM_F32) != GEMM_OK)
        return 0;
    PackMatrix m{D, ldd, 0, 1, rows, N}, x{X, ldx, 0, 1, rows, K};
    Packing packing;
    packing.add(&m);
    packing.add(&x);
    return packing.bytes();
}

extern "C" int gemm_grouped_wgrad(const void* D, int64_t ldd, const void* X, int64_t ldx,
                                  const int32_t* offsets, void* C, int64_t ldc, int64_t stride_c,
                                  int64_t rows, int64_t groups, int64_t N, int64_t K, float alpha,
                                  float beta, gemm_dtype_t in_dtype, gemm_dtype_t out_dtype,
                                  void* workspace, size_t workspace_bytes, void* stream)
{
    const int rc = check_grouping(rows, groups, N, K, in_dtype, out_dtype);
    if (rc != GEMM_OK || groups == 0 || N == 0 || K == 0)
        return rc;
    if (!offsets || !C || ldc < K || !apart(groups, stride_c, N, ldc, K))
        return GEMM_ERR_INVALID_VALUE;
    if (rows > 0 && (!D || !X || ldd < N || ldx < K))
        return GEMM_ERR_INVALID_VALUE;
    PackMatrix m{D, ldd, 0, 1, rows, N}, x{X, ldx, 0, 1, rows, K};
    Packing packing;
    if (in_dtype != GEMM_F32) {
        packing.add(&m);
        packing.add(&x);
    }
    if (bad_workspace(workspace, workspace_bytes, packing.bytes()))
        return GEMM_ERR_INVALID_VALUE;
    DeviceInfo d;
    if (device_info(&d) != cudaSuccess)
        return GEMM_ERR_CUDA;
    GroupedWgradLaunch l{};
    l.by = {offsets, static_cast<int>(groups), static_cast<int>(rows)};
    l.D = D;
    l.ldd = ldd;
    l.X = X;
    l.ldx = ldx;
    l.C = C;
    l.ldc = ldc;
    l.stride_c = stride_c;
    l.N = static_cast<int>(N);
    l.K = static_cast<int>(K);
    l.alpha = alpha;
    l.beta = beta;
    l.in_dtype = in_dtype;
    l.out_dtype = out_dtype;
    l.num_sms = d.num_sms;
    l.status = d.status;
    l.wait_budget = wait_budget_cycles();
    l.fault_skip_kblock = fault_skip_kblock();
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (in_dtype == GEMM_F32 || rows == 0)
        return status_of(grouped_wgrad_simt_launch(l, s));
    cudaError_t err = packing.run(workspace, d.num_sms, s);
    l.D = m.p;
    l.ldd = m.ld;
    l.X = x.p;
    l.ldx = x.ld;
    if (err == cudaSuccess)
        err = grouped_wgrad_tc_launch(l, s);
    return status_of(err);
}
