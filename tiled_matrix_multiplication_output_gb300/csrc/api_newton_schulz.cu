// C entry points of the Newton-Schulz orthogonalisation.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "device.h"
#include "newton_schulz.h"
#include "tiled_gemm.h"

using namespace tmmo;

namespace {

bool valid_dtype(int t) { return t == GEMM_F32 || t == GEMM_F16 || t == GEMM_BF16; }
bool valid_size(int64_t n) { return n >= 0 && n <= GEMM_MAX_DIM; }

constexpr int64_t kMaxBatch = 65535;

// Whether no two matrices of a batch share an element: each lies beyond the
// one before it, or each of its rows does (interleaved matrices).
bool apart(int64_t batch, int64_t rows, int64_t cols, int64_t ld, int64_t stride)
{
    return batch == 1 || (stride >= cols && (rows == 1 || (stride - cols) / (rows - 1) >= ld)) ||
           (stride >= cols && (ld - cols) / (batch - 1) >= stride);
}

}  // namespace

extern "C" size_t gemm_newton_schulz_workspace_size(int64_t batch, int64_t rows, int64_t cols)
{
    if (batch <= 0 || batch > kMaxBatch || rows <= 0 || cols <= 0 || !valid_size(rows) ||
        !valid_size(cols))
        return 0;
    return ns_workspace_bytes(batch, rows, cols);
}

extern "C" int gemm_newton_schulz(const void* G, int64_t ldg, int64_t batch_stride_g, void* O,
                                  int64_t ldo, int64_t batch_stride_o, int64_t batch, int64_t rows,
                                  int64_t cols, gemm_dtype_t in_dtype, gemm_dtype_t out_dtype,
                                  int steps, const float* coefficients, float eps, void* workspace,
                                  size_t workspace_bytes, void* stream)
{
    if (batch < 0 || batch > kMaxBatch || !valid_size(rows) || !valid_size(cols) ||
        !valid_dtype(in_dtype) || !valid_dtype(out_dtype))
        return GEMM_ERR_INVALID_VALUE;
    if (steps < 1 || steps > NS_MAX_STEPS || !coefficients || !(eps >= 0.0f) || !std::isfinite(eps))
        return GEMM_ERR_INVALID_VALUE;
    for (int i = 0; i < 3 * steps; ++i)
        if (!std::isfinite(coefficients[i]))
            return GEMM_ERR_INVALID_VALUE;
    if (batch == 0 || rows == 0 || cols == 0)
        return GEMM_OK;
    if (!G || !O || ldg < cols || ldo < cols)
        return GEMM_ERR_INVALID_VALUE;
    // G is only read, so that one matrix may serve the whole batch
    if (!apart(batch, rows, cols, ldo, batch_stride_o) ||
        (batch_stride_g != 0 && !apart(batch, rows, cols, ldg, batch_stride_g)))
        return GEMM_ERR_INVALID_VALUE;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < ns_workspace_bytes(batch, rows, cols))
        return GEMM_ERR_INVALID_VALUE;
    DeviceInfo d;
    if (device_info(&d) != cudaSuccess)
        return GEMM_ERR_CUDA;
    NsLaunch l{};
    l.G = G;
    l.ldg = ldg;
    l.batch_g = batch_stride_g;
    l.O = O;
    l.ldo = ldo;
    l.batch_o = batch_stride_o;
    l.batch = static_cast<int>(batch);
    l.rows = static_cast<int>(rows);
    l.cols = static_cast<int>(cols);
    l.in_dtype = in_dtype;
    l.out_dtype = out_dtype;
    l.steps = steps;
    l.coefficients = coefficients;
    l.eps = eps;
    l.workspace = workspace;
    l.num_sms = d.num_sms;
    l.status = d.status;
    l.wait_budget = wait_budget_cycles();
    l.fault_skip_kblock = fault_skip_kblock();
    const cudaError_t err = ns_launch(l, static_cast<cudaStream_t>(stream));
    if (err == cudaErrorNotSupported)
        return GEMM_ERR_UNSUPPORTED;
    return err == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}
