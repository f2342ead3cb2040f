// Eight consecutive elements of a row from any element-aligned address.
#pragma once

#include <cstdint>

namespace tmmo {

// The first n of eight consecutive 2- or 4-byte elements at p, as words (two
// 2-byte elements each), zeros for the others.  Loads are whole aligned
// 16-byte words, of which only those are touched that hold at least one of
// the n elements; where p is not on a 16-byte boundary the words are shifted
// into place.  Threads that take consecutive eights of a row then read it in
// full lines whatever its alignment; element by element, unaligned rows took
// 3 to 4 times as long.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, uint32_t (&w)[2 * sizeof(T)])
{
    constexpr int W = 2 * sizeof(T);
    constexpr int QUADS = W / 4;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint32_t off = static_cast<uint32_t>(a) & 15u;
    const uint4* q = reinterpret_cast<const uint4*>(a - off);
    const int end = n > 0 ? static_cast<int>(off) + n * static_cast<int>(sizeof(T)) : 0;
    uint32_t t[W + 4];
#pragma unroll
    for (int k = 0; k <= QUADS; ++k) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (16 * k < end)
            u = __ldcs(q + k);
        t[4 * k] = u.x;
        t[4 * k + 1] = u.y;
        t[4 * k + 2] = u.z;
        t[4 * k + 3] = u.w;
    }
    if (off & 4) {
#pragma unroll
        for (int j = 0; j < W + 3; ++j)
            t[j] = t[j + 1];
    }
    if (off & 8) {
#pragma unroll
        for (int j = 0; j < W + 1; ++j)
            t[j] = t[j + 2];
    }
    if (sizeof(T) == 2 && (off & 2)) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            t[j] = __funnelshift_r(t[j], t[j + 1], 16);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
        if (sizeof(T) == 4)
            w[j] = j < n ? t[j] : 0u;
        else
            w[j] = 2 * j + 1 < n ? t[j] : 2 * j < n ? t[j] & 0xffffu : 0u;
    }
}

}  // namespace tmmo
