// orthogonalize.h -- what orthogonalize.hip and its kernel for small matrices share:
// the matrix that is orthogonalised, and how results are written.
#pragma once

#include "gemm_halves.h"
#include "rows.h"

namespace ar {
namespace lm {
namespace {

template <class F>
using RawOf = typename std::conditional<F::kEpv == 8, uint16_t, float>::type;

// Four elements as floats.
template <class F>
__device__ __forceinline__ void widen4(const RawOf<F>* raw, float* x)
{
    if constexpr (F::kEpv == 8) {
        u32x2 v;
        __builtin_memcpy(&v, raw, 8);
        F::unpack4(v, x);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = raw[i];
    }
}

// ---------------------------------------------------------------------------
// the matrix that is orthogonalised
// ---------------------------------------------------------------------------
struct SourceShape {
    uint64_t rows, cols, ld_in, ld_momentum;
    float decay, rest;  // rest = 1 - decay
    int nesterov;
};
inline SourceShape source_shape(const OrthogonalizeArgs& a)
{
    return SourceShape{a.rows, a.cols, a.ld_in, a.ld_momentum, static_cast<float>(a.decay), static_cast<float>(1.0 - a.decay),
                       a.nesterov};
}
struct SourcePointers {
    const void* in;  // the matrix, or the gradient
    const float* momentum_in;
    float* momentum_out;
};

// Eight elements of a row of U, from column c on: the matrix itself, or the
// momentum's update, FIRST: which is also stored.
template <class F, bool MUON, bool VEC>
struct Source {
    using Raw = RawOf<F>;
    static constexpr int A = VEC ? 16 : sizeof(Raw), AM = VEC ? 16 : 4;

    template <bool FIRST>
    static __device__ __forceinline__ void get(const SourceShape& p, const SourcePointers& x, uint64_t row, uint64_t c,
                                               float (&u)[8])
    {
        const uint64_t left = p.cols - c;
        Raw raw[8];
        get8<Raw, A>(x.in, row * p.ld_in + c, left, raw);
        widen4<F>(raw, u);
        widen4<F>(raw + 4, u + 4);
        if constexpr (MUON) {
            float m[8];
            const uint64_t at = row * p.ld_momentum + c;
            get8<float, AM>(FIRST ? x.momentum_in : x.momentum_out, at, left, m);
            if constexpr (FIRST) {
#pragma unroll
                for (int i = 0; i < 8; ++i) m[i] = p.decay * m[i] + p.rest * u[i];
                float* to = x.momentum_out + at;
                if (VEC && left >= 8) {
                    f32x4 v[2];
                    __builtin_memcpy(v, m, sizeof(m));
                    reinterpret_cast<f32x4*>(to)[0] = v[0];
                    reinterpret_cast<f32x4*>(to)[1] = v[1];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (static_cast<uint64_t>(i) < left) to[i] = m[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = p.nesterov ? p.decay * m[i] + p.rest * u[i] : m[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = static_cast<uint64_t>(i) < left ? u[i] : 0.0f;
    }
};

template <int THREADS>
__device__ __forceinline__ double block_sum(double x, double* waves)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0;
    for (int w = 0; w < THREADS / 64; ++w) x += waves[w];
    return x;
}

__device__ __forceinline__ void put_halves(char* row, uint32_t k, const float (&x)[8])
{
    u32x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h, l;
        split_halves(x[2 * i], x[2 * i + 1], &h, &l);
        hi[i] = h;
        lo[i] = l;
    }
    *reinterpret_cast<u32x4*>(row + halves_at(k, 0)) = hi;
    *reinterpret_cast<u32x4*>(row + halves_at(k, 1)) = lo;
}

}  // namespace
}  // namespace lm
}  // namespace ar
