// Internal launchers of the block-scaled 8-bit operators (host side).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace tmmo {

// Codes of the 8-bit types; they match gemm_f8_t.
enum { F8_E4M3 = 0, F8_E5M2 = 1 };

// One operand of a block-scaled product: outer x K (A: outer = M; B: outer =
// N), stored with K contiguous or, mn_major, with the outer axis contiguous.
struct Fp8Operand {
    const void* data;
    int64_t ld;           // elements from one stored row to the next
    bool mn_major;
    int type;             // F8_E4M3 or F8_E5M2
    // The scale of outer index o in K block kb (128 of K) is
    // scale[kb * stride_k + (o >> shift) * stride_o]
    const float* scale;
    int64_t stride_k, stride_o;
    int shift;            // 0: a scale for each outer index, 7: for 128 of them
};

struct Fp8Launch {
    Fp8Operand a, b;
    void* C;
    int64_t ldc;          // elements
    int M, N, K;
    int out_dtype;        // DT_*
    float alpha, beta;
    int num_sms;
    int* status;
    long long wait_budget;
    int fault_skip_kblock;
};

cudaError_t fp8_gemm_launch(const Fp8Launch& l, cudaStream_t stream);

// The kernel for few output tiles (fp8_small.cu), and whether it is the
// choice for a product.
bool fp8_small_takes(const Fp8Launch& l);
cudaError_t fp8_small_launch(const Fp8Launch& l, cudaStream_t stream);

// C = beta * C (zeros for beta = 0): the product over an empty K.
cudaError_t fp8_empty_launch(const Fp8Launch& l, cudaStream_t stream);

// Quantisation.  Any of the three outputs may be null; tile excludes the
// other two.
struct Fp8Quantize {
    const void* X;
    int64_t ldx;          // elements
    int rows, cols;
    int in_dtype;         // DT_*
    int f8;               // F8_*
    void* q_row;          // 1 x 128 blocks, scales [column block][row]
    float* s_row;
    int64_t ld_row, lds_row;
    void* q_col;          // 128 x 1 blocks, scales [row block][column]
    float* s_col;
    int64_t ld_col, lds_col;
    void* q_tile;         // 128 x 128 blocks, scales [row block][column block]
    float* s_tile;
    int64_t ld_tile, lds_tile;
};

cudaError_t fp8_quantize_launch(const Fp8Quantize& q, cudaStream_t stream);

}  // namespace tmmo
