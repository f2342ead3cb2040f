// Host side of the block-scaled 8-bit product: tensor maps, the choice of
// kernel, and the product over an empty K.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "device.h"
#include "fp8_gemm.cuh"
#include "fp8_launch.cuh"
#include "persistent.cuh"

namespace tmmo {
namespace {

// C in boxes of 32 rows x 128 bytes, 128-byte swizzle.
bool encode_output(CUtensorMap* map, const Fp8Launch& l)
{
    auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (!fn)
        return false;
    const int es = out_bytes(l.out_dtype);
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(l.N), static_cast<cuuint64_t>(l.M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(l.ldc) * es};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / es), 32};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType type = l.out_dtype == DT_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : l.out_dtype == DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return fn(map, type, 2, l.C, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, int BN, int STAGES, bool COLV>
cudaError_t launch_tiles(const Fp8Launch& l, cudaStream_t stream)
{
    using L = Fp8Layout<CG, BN, STAGES>;
    auto kern = fp8_gemm_kernel<CG, BN, STAGES, COLV>;
    static ClusterCaps caps;
    int units_cap = 0;
    cudaError_t err = cluster_cap(kern, caps, CG, F8_THREADS, L::SMEM_ALLOC, l.num_sms, &units_cap);
    if (err != cudaSuccess)
        return err;
    units_cap = std::max(1, units_cap);
    CUtensorMap ta, tb;
    if (!encode_operand(&ta, l.a, l.M, l.K, 128) || !encode_operand(&tb, l.b, l.N, l.K, 128 / L::SUB))
        return cudaErrorNotSupported;
    Fp8Params p{};
    p.M = l.M;
    p.N = l.N;
    p.tiles_m = (l.M + TC_BM * CG - 1) / (TC_BM * CG);
    p.tiles_n = (l.N + BN - 1) / BN;
    const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
    if (tiles > 0x3fffffffLL)
        return cudaErrorNotSupported;
    p.k_blocks = (l.K + F8_BK - 1) / F8_BK;
    p.group_m = 8;
    p.idesc = fp8_idesc(l.a.type, l.b.type, TC_BM * CG, BN / L::SUB, l.a.mn_major, l.b.mn_major);
    p.a_mn = l.a.mn_major;
    p.b_mn = l.b.mn_major;
    p.sa = l.a.scale;
    p.sa_k = l.a.stride_k;
    p.sa_o = l.a.stride_o;
    p.sa_shift = l.a.shift;
    p.sb = l.b.scale;
    p.sb_k = l.b.stride_k;
    p.sb_o = l.b.stride_o;
    p.sb_shift = l.b.shift;
    p.C = l.C;
    p.ldc = l.ldc;
    p.out_dtype = l.out_dtype;
    p.alpha = l.alpha;
    p.beta = l.beta;
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip_kblock = l.fault_skip_kblock;
    CUtensorMap tc = ta;  // unused without tma_out
    p.tma_out = tma_output(l);
    if (p.tma_out && !encode_output(&tc, l))
        return cudaErrorNotSupported;
    // Waves of whole tiles; where the last one would fill at most half of the
    // CTA pairs, its tiles go to two pairs each.  Measured on GB300, us,
    // whole / in parts: 4096 x 4096 x 8192 (28 tiles of 76 in the last wave)
    // 112 / 106, with two scale vectors 155 / 141; 8192 x 8192 x 4096 (36)
    // 200 / 197.
    const int last = static_cast<int>(tiles % units_cap);
    const bool split = CG == 2 && last > 0 && 2 * last <= units_cap;
    p.whole = static_cast<int>(split ? tiles - last : tiles);
    p.items = static_cast<int>(split ? tiles + last : tiles);
    const int units = std::min(p.items, units_cap);
    ClusterLaunch launch(static_cast<unsigned>(units * CG), CG, F8_THREADS, L::SMEM_ALLOC, stream);
    return launch.run(kern, ta, tb, tc, p);
}

template <int CG, int BN, int STAGES>
cudaError_t launch_scales(const Fp8Launch& l, cudaStream_t stream)
{
    return l.b.shift == 0 ? launch_tiles<CG, BN, STAGES, true>(l, stream)
                          : launch_tiles<CG, BN, STAGES, false>(l, stream);
}

template <typename OutT>
__global__ void scale_rows_kernel(OutT* C, long long ldc, int M, int N, float beta)
{
    const long long total = static_cast<long long>(M) * N;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
        OutT* c = C + (i / N) * ldc + i % N;
        *c = fp8_to_out<OutT>(beta != 0.0f ? beta * out_to_f32(*c) : 0.0f);
    }
}

}  // namespace

cudaError_t fp8_empty_launch(const Fp8Launch& l, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(
        std::min<long long>((static_cast<long long>(l.M) * l.N + 255) / 256, 8LL * l.num_sms));
    note_launch();
    if (l.out_dtype == DT_F32)
        scale_rows_kernel<<<grid, 256, 0, stream>>>(static_cast<float*>(l.C), l.ldc, l.M, l.N, l.beta);
    else if (l.out_dtype == DT_F16)
        scale_rows_kernel<<<grid, 256, 0, stream>>>(static_cast<__half*>(l.C), l.ldc, l.M, l.N, l.beta);
    else
        scale_rows_kernel<<<grid, 256, 0, stream>>>(static_cast<__nv_bfloat16*>(l.C), l.ldc, l.M, l.N,
                                                    l.beta);
    return cudaGetLastError();
}

cudaError_t fp8_gemm_launch(const Fp8Launch& l, cudaStream_t stream)
{
    if (fp8_small_takes(l))
        return fp8_small_launch(l, stream);
    // Pair tiles of 256 x 256 take less from shared memory for a value, but a
    // tile's end costs more, and four times as many 128 x 128 tiles keep more
    // SMs busy.  So the smaller ones where they are one wave, or up to two (one
    // of pairs) of at most two K blocks.  Measured on GB300, us, pairs /
    // 128 x 128: 2400 x 900 (152 tiles) x 128 9.3 / 6.3, x 1024 12.2 / 8.4;
    // 1024 x 2432 x 4096 (152) 18.3 / 14.0, with two scale vectors 23.9 / 15.9;
    // 1300 x 2600 (231) x 256 6.9 / 6.3, x 512 7.8 / 7.7, x 1024 9.5 / 10.1.
    const long long tiles =
        static_cast<long long>((l.M + 127) / 128) * ((l.N + 127) / 128);
    const long long pair_tiles =
        static_cast<long long>((l.M + 255) / 256) * ((l.N + 255) / 256);
    if (tiles <= l.num_sms || (2 * pair_tiles <= l.num_sms && l.K <= 2 * F8_BK))
        return launch_scales<1, 128, 4>(l, stream);
    return launch_scales<2, 256, 4>(l, stream);
}

}  // namespace tmmo
