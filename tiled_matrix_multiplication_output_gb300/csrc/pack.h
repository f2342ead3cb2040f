// Copies of 16-bit matrices to rows on 16-byte boundaries, for the kernels that
// read them by TMA (host side).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "device.h"

namespace tmmo {

// `count` matrices of rows x cols, `stride` elements after each other (count 1:
// any).
struct PackMatrix {
    const void* p;
    int64_t ld, stride;
    int64_t count, rows, cols;

    int64_t pitch() const { return (cols + 7) / 8 * 8; }  // of a copy
    // Whether TMA can read it as it lies (interleaved: matrices row by row).
    bool aligned(bool interleaved = false) const
    {
        return aligned16(p) && ld % 8 == 0 &&
               (count <= 1 || stride == 0 || (stride % 8 == 0 && (interleaved || stride >= ld)));
    }
    size_t bytes() const
    {
        const int64_t n = stride == 0 ? 1 : count;
        return static_cast<size_t>((n * rows * pitch() * 2 + 255) / 256 * 256);
    }
};

// The copies that a call needs, one after another in its workspace, made by one
// launch.
class Packing {
public:
    // Notes the matrix for a copy if it needs one.
    void add(PackMatrix* m, bool interleaved = false)
    {
        if (m->rows > 0 && m->cols > 0 && m->count > 0 && !m->aligned(interleaved))
            jobs_[n_++] = m;
    }
    size_t bytes() const
    {
        size_t sum = 0;
        for (int i = 0; i < n_; ++i)
            sum += jobs_[i]->bytes();
        return sum;
    }
    // Copies to `workspace` and makes the matrices refer to the copies.
    cudaError_t run(void* workspace, int num_sms, cudaStream_t stream);

private:
    PackMatrix* jobs_[5];
    int n_ = 0;
};

}  // namespace tmmo
