// Internal launcher of the Newton-Schulz orthogonalisation (host side).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "launch.h"

namespace tmmo {

constexpr int NS_MAX_STEPS = 32;

struct NsLaunch {
    const void* G;
    int64_t ldg, batch_g;   // elements from one row, one matrix, to the next
    void* O;
    int64_t ldo, batch_o;
    int batch, rows, cols;
    int in_dtype, out_dtype;
    int steps;
    const float* coefficients;  // host: steps x (a, b, c)
    float eps;
    void* workspace;        // 256-byte aligned, ns_workspace_bytes()
    int num_sms;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

// Whether the rows of the result are on 16-byte boundaries.
inline bool ns_vec_rows(const NsLaunch& l)
{
    const int64_t es = l.out_dtype == DT_F32 ? 4 : 2;
    return (reinterpret_cast<uintptr_t>(l.O) & 15u) == 0 && l.ldo * es % 16 == 0 &&
           (l.batch == 1 || l.batch_o * es % 16 == 0);
}

// Whether the products' operands are two FP16 values an element instead of one.
// With one the result is up to 2e-3 off exact arithmetic (relative, over all
// elements), about what rounding it to BF16 does (1.66e-3), for a third of the
// MMAs.  So: two where the result has more bits, and for a short side of up to
// 128, where one would be 2e-3 off and for the narrowest up to 7e-3 (and the
// one-launch form is bound by latency).
inline bool ns_split(const NsLaunch& l)
{
    return l.out_dtype != DT_BF16 || l.rows <= 128 || l.cols <= 128;
}

size_t ns_workspace_bytes(int64_t batch, int64_t rows, int64_t cols);

// The one-launch form for matrices that a cluster holds on chip
// (ns_resident.cu), and whether it takes a matrix.
bool ns_resident_takes(const NsLaunch& l);
cudaError_t ns_resident_launch(const NsLaunch& l, cudaStream_t stream);

cudaError_t ns_launch(const NsLaunch& l, cudaStream_t stream);

}  // namespace tmmo
