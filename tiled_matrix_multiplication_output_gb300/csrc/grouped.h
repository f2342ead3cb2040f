// Internal launchers of the products grouped by rows (host side).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace tmmo {

// Groups per call: the table of a block (grouped.cuh) lies in shared memory.
constexpr int kMaxGroups = 1024;

// Rows [offsets[g], offsets[g + 1]) belong to group g.
struct Grouping {
    const int32_t* offsets;  // groups + 1, device memory
    int groups;
    int rows;
};

// Y = alpha * X op(W[g]) + beta * Y, for the rows of each group g.
struct GroupedLaunch {
    Grouping by;
    const void* X;   // rows x K
    int64_t ldx;
    const void* W;   // groups of K x N (w_t: N x K)
    int64_t ldw, stride_w;
    bool w_t;
    void* Y;         // rows x N
    int64_t ldy;
    int N, K;
    float alpha, beta;
    bool zero_rest;  // write zeros to the rows of no group
    int in_dtype, out_dtype;  // DT_*
    int num_sms;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

// C[g] = alpha * D[rows of g]^T X[rows of g] + beta * C[g].
struct GroupedWgradLaunch {
    Grouping by;
    const void* D;   // rows x N
    int64_t ldd;
    const void* X;   // rows x K
    int64_t ldx;
    void* C;         // groups of N x K
    int64_t ldc, stride_c;
    int N, K;
    float alpha, beta;
    int in_dtype, out_dtype;
    int num_sms;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

// On the tensor cores: 16-bit operands with rows on 16-byte boundaries (pack.h),
// some groups, rows and K > 0.
cudaError_t grouped_tc_launch(const GroupedLaunch& l, cudaStream_t stream);
cudaError_t grouped_wgrad_tc_launch(const GroupedWgradLaunch& l, cudaStream_t stream);

// On the FP32 units: FP32 operands, and no operands at all (K == 0, no groups; no rows).
cudaError_t grouped_simt_launch(const GroupedLaunch& l, cudaStream_t stream);
cudaError_t grouped_wgrad_simt_launch(const GroupedWgradLaunch& l, cudaStream_t stream);

}  // namespace tmmo
