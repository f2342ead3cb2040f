// Rows of 16-bit elements at any address copied to rows on 16-byte boundaries:
// one read and one write of the matrix, in whole 16-byte words.
#include "pack.h"

#include <algorithm>

#include "launch.h"
#include "load8.cuh"

namespace tmmo {
namespace {

constexpr int PACK_THREADS = 256;

struct PackJob {
    const uint16_t* src;
    uint4* dst;
    int64_t ld, stride;
    int64_t rows, eights;  // rows of a matrix, groups of eight in a row
    int cols;
    int64_t begin;         // this job's first group of eight among all
};
struct PackJobs {
    PackJob job[5];
    int n;
    int64_t total;
};

__global__ void __launch_bounds__(PACK_THREADS) pack_kernel(const PackJobs q)
{
    const int64_t step = static_cast<int64_t>(gridDim.x) * PACK_THREADS;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * PACK_THREADS + threadIdx.x; i < q.total; i += step) {
        int k = 0;
        while (k + 1 < q.n && i >= q.job[k + 1].begin)
            ++k;
        const PackJob& j = q.job[k];
        const int64_t at = i - j.begin;
        const int64_t row = at / j.eights, c = at % j.eights * 8;
        uint32_t w[4];
        load8(j.src + row / j.rows * j.stride + row % j.rows * j.ld + c,
              min(8, static_cast<int>(j.cols - c)), w);
        j.dst[at] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace

cudaError_t Packing::run(void* workspace, int num_sms, cudaStream_t stream)
{
    if (n_ == 0)
        return cudaSuccess;
    PackJobs q{};
    char* to = static_cast<char*>(workspace);
    for (int i = 0; i < n_; ++i) {
        PackMatrix& m = *jobs_[i];
        if (m.stride == 0)
            m.count = 1;
        PackJob& j = q.job[q.n++];
        j.src = static_cast<const uint16_t*>(m.p);
        j.dst = reinterpret_cast<uint4*>(to);
        j.ld = m.ld;
        j.stride = m.stride;
        j.rows = m.rows;
        j.cols = static_cast<int>(m.cols);
        j.eights = m.pitch() / 8;
        j.begin = q.total;
        q.total += m.count * m.rows * j.eights;
        const size_t bytes = m.bytes();
        m.p = to;
        m.ld = m.pitch();
        m.stride = m.stride == 0 ? 0 : m.rows * m.ld;
        to += bytes;
    }
    const int64_t blocks = std::min<int64_t>((q.total + PACK_THREADS - 1) / PACK_THREADS, 16ll * num_sms);
    note_launch();
    pack_kernel<<<static_cast<unsigned>(blocks), PACK_THREADS, 0, stream>>>(q);
    return cudaGetLastError();
}

}  // namespace tmmo
