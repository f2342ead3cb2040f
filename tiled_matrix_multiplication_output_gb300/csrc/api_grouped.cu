// C entry points of the products grouped by rows: argument checks and the
// translation to the internal launchers.
#include <cuda_runtime.h>

#include <cstdint>

#include "api_checks.h"
#include "device.h"
#include "grouped.h"
#include "launch.h"
#include "tiled_gemm.h"

using namespace tmmo;

static_assert(kMaxGroups == GEMM_MAX_GROUPS, "the table's size");

namespace {

int check_grouping(const int32_t* offsets, int64_t rows, int64_t groups, int64_t N, int64_t K,
                   int in_dtype, int out_dtype)
{
    if (!valid_size(rows) || !valid_size(N) || !valid_size(K) || groups < 0 ||
        !valid_dtype(in_dtype) || !valid_dtype(out_dtype))
        return GEMM_ERR_INVALID_VALUE;
    if (groups > GEMM_MAX_GROUPS)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

}  // namespace

extern "C" size_t gemm_grouped_workspace_size(const void*, int64_t, const void*, int64_t, int64_t,
                                              int64_t, int64_t, int64_t, int64_t, gemm_op_t,
                                              gemm_dtype_t)
{
    return 0;
}

extern "C" int gemm_grouped(const void* X, int64_t ldx, const void* W, int64_t ldw,
                            int64_t stride_w, gemm_op_t op_w, const int32_t* offsets, void* Y,
                            int64_t ldy, int64_t rows, int64_t groups, int64_t N, int64_t K,
                            float alpha, float beta, int zero_rest, gemm_dtype_t in_dtype,
                            gemm_dtype_t out_dtype, void* workspace, size_t workspace_bytes,
                            void* stream)
{
    int rc = check_grouping(offsets, rows, groups, N, K, in_dtype, out_dtype);
    if (rc == GEMM_OK && op_w != GEMM_OP_N && op_w != GEMM_OP_T)
        rc = GEMM_ERR_INVALID_VALUE;
    if (rc != GEMM_OK || rows == 0 || N == 0)
        return rc;
    if (!offsets || !Y || ldy < N)
        return GEMM_ERR_INVALID_VALUE;
    if (K > 0 && groups > 0 &&
        (!X || !W || ldx < K || ldw < (op_w == GEMM_OP_T ? K : N) || stride_w < 0))
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
    return status_of(grouped_tc_takes(l) ? grouped_tc_launch(l, s) : grouped_simt_launch(l, s));
}

extern "C" size_t gemm_grouped_wgrad_workspace_size(const void*, int64_t, const void*, int64_t,
                                                    int64_t, int64_t, int64_t, gemm_dtype_t)
{
    return 0;
}

extern "C" int gemm_grouped_wgrad(const void* D, int64_t ldd, const void* X, int64_t ldx,
                                  const int32_t* offsets, void* C, int64_t ldc, int64_t stride_c,
                                  int64_t rows, int64_t groups, int64_t N, int64_t K, float alpha,
                                  float beta, gemm_dtype_t in_dtype, gemm_dtype_t out_dtype,
                                  void* workspace, size_t workspace_bytes, void* stream)
{
    const int rc = check_grouping(offsets, rows, groups, N, K, in_dtype, out_dtype);
    if (rc != GEMM_OK || groups == 0 || N == 0 || K == 0)
        return rc;
    if (!offsets || !C || ldc < K || (groups > 1 && !apart(stride_c, N, ldc, K)))
        return GEMM_ERR_INVALID_VALUE;
    if (rows > 0 && (!D || !X || ldd < N || ldx < K))
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
    return status_of(grouped_wgrad_tc_takes(l) ? grouped_wgrad_tc_launch(l, s)
                                               : grouped_wgrad_simt_launch(l, s));
}
