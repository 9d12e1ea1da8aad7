// rows.h -- reading a matrix's rows eight elements a thread, and the launches that do.
#pragma once

#include <type_traits>

#include "gemm.h"

namespace ar {
namespace lm {
using namespace detail;

namespace {

// Eight elements by loads of A bytes (the rows' alignment), as far as they go.
template <class Raw, int A>
__device__ __forceinline__ void get8(const void* in, uint64_t at, uint64_t left, Raw (&x)[8])
{
    if constexpr (A > static_cast<int>(sizeof(Raw))) {
        if (left >= 8) {
            using Unit = typename std::conditional<A == 16, u32x4, u32x2>::type;
            constexpr int N = sizeof(x) / A;
            Unit v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = gptr<Unit>(static_cast<const char*>(in) + at * sizeof(Raw))[i];
            __builtin_memcpy(x, v, sizeof(x));
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<uint64_t>(i) < left ? gptr<Raw>(in)[at + i] : Raw(0);
}

inline uint64_t round_up(uint64_t x, uint64_t m) { return (x + m - 1) / m * m; }

// Threads a row of `units` and the grid that takes `rows` of them.
inline int lanes_for(uint64_t units)
{
    int lanes = 1;
    while (lanes < kBlock && static_cast<uint64_t>(lanes) < units) lanes *= 2;
    return lanes;
}
inline dim3 grid_for(uint64_t rows, int lanes)
{
    const uint64_t per = kBlock / lanes;
    return dim3(static_cast<uint32_t>((rows + per - 1) / per));
}

}  // namespace
}  // namespace lm
}  // namespace ar
