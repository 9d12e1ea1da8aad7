// gemm.h -- the matrix-core product that the cross entropy is made of.
//
//   C[m][n] = sum_k A[m][k] * B[n][k]
//
// for 16-bit A and B whose rows are contiguous along K, 16-byte aligned and a
// multiple of kTileK long; C stays in fp32 registers and goes to an epilogue.
// A workgroup takes kTileM rows of A and BN of B; 64-deep tiles of both go
// from memory straight into LDS, two stages deep, so that the loads of one
// stage run under the matrix instructions of the other.
//
// LDS holds 128-byte rows as eight 16-byte columns; column c of row r lies at
// c ^ (r & 7), so that the 16 rows of a fragment read spread over all banks.
// The direct load writes lane after lane, so the permutation is made on the
// side of the global address.
#pragma once

#include "../kernels_impl.h"
#include "lm_kernels.h"

namespace ar {
namespace lm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct MmaBF16 {
    using Frag = bf16x8;
    using Format = detail::BF16;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
struct MmaF16 {
    using Frag = f16x8;
    using Format = detail::F16;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// Rows of A and B beyond M and N are read as the last ones (their results are
// dropped by the epilogue), so no access leaves the operands.
struct GemmArgs {
    const uint16_t* a;
    const uint16_t* b;
    uint64_t lda, ldb;  // elements
    uint32_t m, n;
    uint32_t k;         // of one split; a multiple of kTileK
    uint32_t k_all;     // splits * k may pass it
    uint32_t tiles_m, tiles_n, splits;
};

// Where a lane's results lie: acc[i][j][r] is C[m][n] with
//   m = m0 + 16 i + 4 (lane / 16) + r,  n = n0 + 16 j + lane % 16.
template <int MT, int NT>
struct Tile {
    f32x4 v[MT][NT];
};

template <class T, int BN, int WM, int WN, class Epilogue>
__global__ __launch_bounds__(64 * WM * WN) void gemm(const GemmArgs g, const Epilogue epi)
{
    constexpr int BM = kTileM, BK = kTileK;
    constexpr int THREADS = 64 * WM * WN;
    constexpr int MT = BM / (16 * WM), NT = BN / (16 * WN);
    constexpr int A_LOADS = BM * 8 / THREADS;                        // 16-byte loads of a thread for one stage of A
    constexpr int B_LOADS = (BN * 8 + THREADS - 1) / THREADS;
    __shared__ __attribute__((aligned(1024))) uint16_t lds_a[2][BM * BK];
    __shared__ __attribute__((aligned(1024))) uint16_t lds_b[2][BN * BK];

    // Workgroups go round the eight XCDs one by one; each XCD gets a
    // contiguous part of the tile order, in which tiles of eight row blocks
    // follow each other, so that what an XCD works on at a time shares rows of
    // both operands in its L2.
    const uint32_t total = gridDim.x;
    uint32_t id = blockIdx.x;
    {
        const uint32_t xcd = id & 7, part = total >> 3, rest = total & 7;
        id = xcd * part + (xcd < rest ? xcd : rest) + (id >> 3);
    }
    const uint32_t per_split = g.tiles_m * g.tiles_n;
    const uint32_t split = id / per_split;
    id -= split * per_split;
    constexpr uint32_t GROUP = 8;
    const uint32_t group = id / (GROUP * g.tiles_n), first = group * GROUP;
    const uint32_t high = min(GROUP, g.tiles_m - first);
    const uint32_t in = id - group * GROUP * g.tiles_n;
    const uint32_t tm = first + in % high, tn = in / high;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const uint32_t m_base = tm * BM, n_base = tn * BN;
    const uint32_t k0 = split * g.k;
    const uint32_t k1 = min(k0 + g.k, g.k_all);

    const uint16_t* pa[A_LOADS];
    const uint16_t* pb[B_LOADS];
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) {
        const int at = i * THREADS + tid, row = at >> 3, col = (at & 7) ^ (row & 7);
        const uint32_t r = min(m_base + row, g.m - 1);
        pa[i] = g.a + static_cast<uint64_t>(r) * g.lda + k0 + col * 8;
    }
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i) {
        const int at = i * THREADS + tid, row = at >> 3, col = (at & 7) ^ (row & 7);
        const uint32_t r = min(n_base + row, g.n - 1);
        pb[i] = g.b + static_cast<uint64_t>(r) * g.ldb + k0 + col * 8;
    }
    auto load = [&](int stage) {
#pragma unroll
        for (int i = 0; i < A_LOADS; ++i) {
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)pa[i],
                                             (__attribute__((address_space(3))) void*)(&lds_a[stage][(i * THREADS + wave * 64) * 8]),
                                             16, 0, 0);
            pa[i] += BK;
        }
#pragma unroll
        for (int i = 0; i < B_LOADS; ++i) {
            if ((BN * 8) % THREADS == 0 || i * THREADS + wave * 64 < BN * 8) {  // the same for a whole wave
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)pb[i],
                                                 (__attribute__((address_space(3))) void*)(&lds_b[stage][(i * THREADS + wave * 64) * 8]),
                                                 16, 0, 0);
                pb[i] += BK;
            }
        }
    };

    Tile<MT, NT> acc;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc.v[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int frow = lane & 15, fcol = lane >> 4;
    if (k0 < k1) load(0);  // a split past the end has nothing to add
    int stage = 0;
    for (uint32_t k = k0; k < k1; k += BK, stage ^= 1) {
        __syncthreads();  // this stage has arrived, and nobody reads the other one any more
        if (k + BK < k1) load(stage ^ 1);
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk) {
            const int col = ((kk * 4 + fcol) ^ (frow & 7)) * 8;
            typename T::Frag fa[MT], fb[NT];
#pragma unroll
            for (int i = 0; i < MT; ++i)
                fa[i] = *reinterpret_cast<const typename T::Frag*>(
                    &lds_a[stage][((wm * MT + i) * 16 + frow) * BK + col]);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                fb[j] = *reinterpret_cast<const typename T::Frag*>(
                    &lds_b[stage][((wn * NT + j) * 16 + frow) * BK + col]);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc.v[i][j] = T::mma(fa[i], fb[j], acc.v[i][j]);
        }
    }
    epi(acc, m_base + wm * MT * 16, n_base + wn * NT * 16, g, tm * WM + wm, split);
}

template <class T, int BN, int WM, int WN, class Epilogue>
hipError_t launch_gemm(GemmArgs g, const Epilogue& epi, hipStream_t stream)
{
    g.tiles_m = (g.m + kTileM - 1) / kTileM;
    g.tiles_n = (g.n + BN - 1) / BN;
    hipLaunchKernelGGL((gemm<T, BN, WM, WN, Epilogue>), dim3(g.tiles_m * g.tiles_n * g.splits), dim3(64 * WM * WN), 0,
                       stream, g, epi);
    return hipGetLastError();
}

}  // namespace lm
}  // namespace ar
