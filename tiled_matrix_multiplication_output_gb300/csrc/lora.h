// Internal launchers of low-rank adapters beside a shared projection (host
// side).
//
// One form serves both directions.  A row i of X with adapter g is multiplied
// by the shared weight and, through the adapter's two factors, by a low-rank
// one:
//     t_i = scale_g * X_i F_g^T          (rank values)
//     Y_i = X_i W^T + t_i E_g^T
// Forward: X is the input, F = A (rank x K), E = B (N x rank), W as stored
// (N x K).  Towards the input's gradient: X is the output's gradient, F = B^T,
// E = A^T and W^T; every matrix is then read across its stored rows.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace tmmo {

constexpr int kMaxRank = 256;

class TensorMaps;

struct LoraLaunch {
    const void* X;        // rows x K
    int64_t ldx;
    const void* W;        // N x K, or (across) K x N
    int64_t ldw;
    const void* F;        // adapters of rank x K, or (across) K x rank
    int64_t ldf, stride_f;
    const void* E;        // adapters of N x rank, or (across) rank x N
    int64_t lde, stride_e;
    bool across;
    const float* scale;   // one for each adapter, or null: 1
    const int32_t* adapter;  // one for each row; outside [0, adapters): none
    void* Y;              // rows x N
    int64_t ldy;
    int rows, N, K, adapters, rank;
    int in_dtype, out_dtype;  // DT_*
    void* t;              // the rank values: FP32, rows x rank, or in parts (lora_tc.cuh)
    int parts;
    void* t_grad;         // of FP16 operands: the same in FP16 parts, for the gradients (or null,
                          // as may then be t)
    void* plan;           // one for each 128 rows
    TensorMaps* maps;     // the call's
    int num_sms;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

// G_g(c, j) = sum over the rows i of adapter g of P[i, c] t[i, j].
struct LoraGradLaunch {
    const void* P;        // rows x cols
    int64_t ldp;
    const void* t;        // as LoraLaunch has them (of FP16 operands: t_grad)
    int parts;
    const void* plan;
    TensorMaps* maps;
    void* G;              // adapters; element (c, j) at c * step_c + j * step_j
    int64_t step_c, step_j, stride_g;
    const int32_t* adapter;
    int rows, cols, adapters, rank;
    int in_dtype, out_dtype;
    int num_sms;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;  // (of an adapter's row tiles)
};

// Bytes of a row tile's plan, and of rank values in parts for a row.
constexpr int LORA_PLAN_BYTES = 2576;
int lora_parts_bytes(int rank, int parts);

// On the tensor cores: 16-bit operands with rows on 16-byte boundaries (pack.h),
// no size of zero.  Shrink makes the plans and the rank values; of two products,
// whose rows have the same adapters, in one launch.  Expand may start while a
// shrink runs.
cudaError_t lora_shrink_tc_launch(const LoraLaunch& first, const LoraLaunch* second, cudaStream_t stream);
// Whether a shrink alone leaves room on its SMs for the product's kernel.
bool lora_shrink_shares(const LoraLaunch& l);
cudaError_t lora_expand_tc_launch(const LoraLaunch& l, cudaStream_t stream);
// The kernel for few output tiles, and whether it is the choice.
bool lora_small_takes(const LoraLaunch& l);
cudaError_t lora_small_tc_launch(const LoraLaunch& l, cudaStream_t stream);
// The same kernel that makes the rank values too (of the forward direction), and
// whether it is the choice: it needs no shrink, no plans and no rank values in memory.
bool lora_alone_takes(int64_t rows, int64_t N, int64_t K, int64_t adapters, int rank, int parts, int num_sms);
cudaError_t lora_alone_tc_launch(const LoraLaunch& l, cudaStream_t stream);
// Two gradients of the same rows in one launch (either may be null); dependent: the
// launch before is an expand of the same rank values.
cudaError_t lora_grad_tc_launch(const LoraGradLaunch* const (&sides)[2], bool dependent, cudaStream_t stream);

// On the FP32 units: FP32 operands, and sums of nothing.
cudaError_t lora_simt_shrink(const LoraLaunch& l, cudaStream_t stream);
cudaError_t lora_simt_expand(const LoraLaunch& l, cudaStream_t stream);
cudaError_t lora_simt_grad(const LoraGradLaunch& l, cudaStream_t stream);

}  // namespace tmmo
