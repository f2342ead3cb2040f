// Device side of the row groups: the table every block builds from the
// offsets, and the tiles of the groups.
#pragma once

#include <cstdint>

#include "grouped.h"

namespace tmmo {

// first[g] .. first[g + 1]: the rows of group g; tile[g]: how many tiles the
// groups before g have.  Both have groups + 1 entries.
struct GroupTable {
    int* first;
    int* tile;

    static constexpr int BYTES = 2 * (kMaxGroups + 1) * static_cast<int>(sizeof(int));

    // The group of tile t < tile[groups].
    __device__ int group_of(int t, int groups) const
    {
        int lo = 0, hi = groups;  // tile[lo] <= t < tile[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tile[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    }
};

// Builds the table for tiles of `tile_rows` rows; every thread of the block
// calls it, and it ends in a block barrier.  Offsets are taken as the largest
// of those up to them, within [0, rows]: whatever they hold, groups neither
// overlap nor leave the matrix.
__device__ __forceinline__ GroupTable load_groups(int* smem, const Grouping& by, int tile_rows)
{
    GroupTable t{smem, smem + kMaxGroups + 1};
    const int n = by.groups + 1;
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        t.first[i] = min(max(by.offsets[i], 0), by.rows);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int largest = 0, tiles = 0;
        for (int base = 0; base < n; base += 32) {
            const int i = base + lane;
            int v = i < n ? t.first[i] : 0;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d)
                    v = max(v, o);
            }
            v = max(v, largest);
            int before = __shfl_up_sync(0xffffffffu, v, 1);
            if (lane == 0)
                before = base == 0 ? v : largest;
            // tiles of group i - 1, and their sum up to it
            int c = (v - before) / tile_rows + ((v - before) % tile_rows != 0);
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, c, d);
                if (lane >= d)
                    c += o;
            }
            c += tiles;
            if (i < n) {
                t.first[i] = v;
                t.tile[i] = c;
            }
            largest = __shfl_sync(0xffffffffu, v, 31);
            tiles = __shfl_sync(0xffffffffu, c, 31);
        }
    }
    __syncthreads();
    return t;
}

// Zeros in this thread's share of the rows that lie before the first group or
// behind the last.
template <typename OutT>
__device__ __forceinline__ void zero_rest_rows(const GroupTable& t, const Grouping& by, OutT* Y,
                                               int64_t ldy, int N, int64_t thread, int64_t threads)
{
    const int head = t.first[0], tail = t.first[by.groups];
    const int64_t total = static_cast<int64_t>(head + (by.rows - tail)) * N;
    for (int64_t i = thread; i < total; i += threads) {
        const int64_t r = i / N;
        Y[(r < head ? r : tail + (r - head)) * ldy + i % N] = OutT(0.0f);
    }
}

}  // namespace tmmo
