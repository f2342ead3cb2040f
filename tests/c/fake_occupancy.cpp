// The one-launch orthogonalisation's question whether a matrix fits, against a
// CUDA runtime in which the occupancy query fails: this file stands in for the
// runtime calls that ns_resident.cu makes, with the runtime's last error.
#include <cuda_runtime.h>

#include <cstdio>

#include "newton_schulz.h"

namespace {
cudaError_t g_last = cudaSuccess;
cudaError_t g_query = cudaSuccess;
int g_clusters = 1;
int g_failures = 1 << 30;  // the queries that fail before they work again

cudaError_t note(cudaError_t err)
{
    if (err != cudaSuccess)
        g_last = err;
    return err;
}
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* dev)
{
    *dev = 0;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*)
{
    *n = g_clusters;
    return g_failures-- > 0 ? note(g_query) : cudaSuccess;
}
cudaError_t cudaGetLastError()
{
    const cudaError_t err = g_last;
    g_last = cudaSuccess;
    return err;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return note(cudaErrorUnknown); }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t)
{
    return note(cudaErrorUnknown);
}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, CUstream_st*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaSuccess; }
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
}

namespace tmmo {
void note_launch() {}
}  // namespace tmmo

int main()
{
    tmmo::NsLaunch l{};
    l.batch = 1;
    l.rows = 64;
    l.cols = 700;
    g_query = cudaErrorInvalidValue;
    if (tmmo::ns_resident_takes(l) || g_last != cudaSuccess) {
        std::printf("a failed query: last error %d\n", static_cast<int>(g_last));
        return 1;
    }
    g_query = cudaSuccess;  // (a failure is not kept)
    if (!tmmo::ns_resident_takes(l) || g_last != cudaSuccess) {
        std::printf("a query that works again: last error %d\n", static_cast<int>(g_last));
        return 2;
    }
    l.cols = 350;           // another size, of which no cluster fits
    g_clusters = 0;
    if (tmmo::ns_resident_takes(l) || tmmo::ns_resident_takes(l) || g_last != cudaSuccess) {
        std::printf("no cluster fits: last error %d\n", static_cast<int>(g_last));
        return 3;
    }
    l.cols = 1000;          // two forms to choose from: the first query fails, then all work
    g_clusters = 1;
    g_query = cudaErrorInvalidValue;
    g_failures = 1;
    if (!tmmo::ns_resident_takes(l) || g_last != cudaSuccess) {
        std::printf("one of two queries failed: last error %d\n", static_cast<int>(g_last));
        return 4;
    }
    std::printf("ok\n");
    return 0;
}
