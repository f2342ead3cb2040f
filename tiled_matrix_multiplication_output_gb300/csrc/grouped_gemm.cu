// Launch of the row-grouped products on the tensor cores (grouped_tc.cuh).
#include "grouped_launch.cuh"

namespace tmmo {

cudaError_t grouped_tc_launch(const GroupedLaunch& l, cudaStream_t stream)
{
    GroupedTcParams p{};
    p.by = l.by;
    p.C = l.Y;
    p.ldc = l.ldy;
    p.N = l.N;
    p.K = l.K;
    // (in even shares, so that a segment's sums are taken while the next one is made)
    const int k_blocks = (l.K + TC_BK - 1) / TC_BK;
    p.segments = (k_blocks + GT_SEGMENT_PRODUCT - 1) / GT_SEGMENT_PRODUCT;
    p.segment = (k_blocks + p.segments - 1) / p.segments;
    p.segments = (k_blocks + p.segment - 1) / p.segment;
    p.tiles_f = (l.N + 255) / 256;
    p.alpha = l.alpha;
    p.beta = l.beta;
    p.zero_rest = l.zero_rest;
    p.unit = row_unit(l.Y, l.ldy * type_bytes(l.out_dtype), 0);
    p.one_weight = l.by.groups == 1 || l.stride_w == 0;
    p.swap = !p.one_weight && l.stride_w < l.ldw;  // matrices interleaved row by row
    p.idesc = tc_idesc(l.in_dtype == DT_BF16, 256, 0, !l.w_t, false);
    p.status = l.status;
    p.wait_budget = l.wait_budget;
    p.fault_skip_kblock = l.fault_skip_kblock;

    const int64_t inner = l.w_t ? l.K : l.N, outer = l.w_t ? l.N : l.K;
    const int64_t groups = p.one_weight ? 1 : l.by.groups;
    const int64_t stride = p.one_weight ? l.ldw : l.stride_w;
    const uint32_t deep = l.w_t ? TC_BM : TC_BK;
    GroupedMaps m;
    bool ok =
        (p.swap ? encode_map(&m.a, l.in_dtype, l.W, 3, {inner, groups, outer}, {stride, l.ldw}, {64, 1, deep})
                : encode_map(&m.a, l.in_dtype, l.W, 3, {inner, outer, groups}, {l.ldw, stride}, {64, deep, 1}));
    // The boxes that half of the largest possible tile is made of; a kernel asks
    // for no other.
    const int64_t half = (std::min<int64_t>(l.by.rows, GT_N) + 31) / 32 * 16;
    auto rows = [&](CUtensorMap* map, uint32_t n) {
        if (half < static_cast<int64_t>(n)) {
            *map = m.b16;
            return true;
        }
        return encode_map(map, l.in_dtype, l.X, 2, {l.K, l.by.rows, 1}, {l.ldx, 0}, {64, n, 1});
    };
    ok = ok && rows(&m.b16, 16) && rows(&m.b32, 32) && rows(&m.b64, 64) && rows(&m.b, TC_BM);
    if (!ok)
        return cudaErrorNotSupported;
    m.c = m.b;
    const int64_t most = (l.by.rows / GT_N + static_cast<int64_t>(std::min(l.by.groups, l.by.rows))) * p.tiles_f;
    return l.w_t ? launch_grouped_tc<GROUPED_T>(l.out_dtype, m, p, most, l.num_sms, stream)
                 : launch_grouped_tc<GROUPED_N>(l.out_dtype, m, p, most, l.num_sms, stream);
}

}  // namespace tmmo
