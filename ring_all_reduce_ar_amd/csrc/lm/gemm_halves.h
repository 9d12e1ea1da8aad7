// gemm_halves.h -- products of fp32 values held as two fp16 numbers each.
//
//   x 2^11 = hi + lo,  hi = fp16(x 2^11),  lo = fp16(x 2^11 - hi)
//
// hi + lo holds 22 bits of x (and all of a x below 2^-24 to steps of 2^-36);
// of the four products of a pair, lo lo is left out, at 2^-22 of the whole, and
// hi lo, lo hi and hi hi are summed in fp32: three matrix instructions where
// one fp32 product of the library's takes as long as eight. |x| is below 32.
//
// A row holds, for each 32 of its depth, 32 hi and 32 lo: 128 bytes, the row of
// a stage in LDS, its 16-byte columns permuted as gemm.h's.
#pragma once

#include "gemm.h"

namespace ar {
namespace lm {
namespace {

constexpr int kHalvesDepth = 32;
constexpr float kHalvesScale = 2048.0f, kHalvesUnit = 1.0f / (2048.0f * 2048.0f);  // of a product

// Bytes of a row of `depth` (a multiple of 32).
__host__ __device__ constexpr uint64_t halves_bytes(uint64_t depth) { return depth * 4; }
__host__ __device__ constexpr uint32_t halves_at(uint32_t k, uint32_t piece)
{
    return (k >> 5) * 128 + piece * 64 + (k & 31) * 2;
}

// The pieces of two values that are held times 2^11 already, the first in the low halves.
__device__ __forceinline__ void split_halves(float x, float y, uint32_t* hi, uint32_t* lo)
{
    *hi = MmaF16::pack2(x, y);
    const f16x2 h = __builtin_bit_cast(f16x2, *hi);
    *lo = MmaF16::pack2(x - static_cast<float>(h[0]), y - static_cast<float>(h[1]));
}

// A batch of products C = A B^T of one size: C[m][n] = sum_k A[m][k] B[n][k].
struct HalvesArgs {
    const char* a;
    const char* b;
    uint64_t batch_a, batch_b;  // bytes from one matrix to the next
    uint32_t lda, ldb;          // bytes
    uint32_t m, n, steps;       // steps of 32 of the depth
    uint32_t tiles_m, tiles_n;
    uint32_t per_matrix;        // tiles; of a symmetric product those with tm >= tn
    int symmetric;
    // the first `whole` tiles of all matrices are one workgroup's each, the others'
    // sums are split along the depth and joined by a launch of its own
    uint32_t whole, splits;
    float* partial;  // [tile - whole][split][16-byte vector of a thread][thread]
};

template <int B>
struct HalvesShape {
    static_assert(B == 128 || B == 64, "tiles");
    static constexpr int kStages = B == 128 ? 2 : 4;
    static constexpr uint32_t kB = B * 128, kStage = 2 * kB;
    static constexpr int kLoads = B / 32;  // of one operand, a stage and a thread
    static constexpr int kWave = B / 2, kTiles = kWave / 16;
};

// A tile leaves through LDS in rows of pieces.
template <int B>
struct HalvesStaging {
    static constexpr int N = HalvesShape<B>::kTiles;
    char* lds;
    uint32_t wm, wn;          // the wave's first row and column within the tile
    uint32_t m_base, n_base;  // the tile's

    // Rows of B * 4 bytes, the 16-byte columns permuted within groups of eight.
    static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t byte, uint32_t key)
    {
        return row * (B * 4) + (byte ^ ((key & 7) * 16));
    }

    // out[n][m], rows `ld` bytes apart, for the first `rows` n and `depth` m (a multiple of 32).
    __device__ __forceinline__ void store_by_column(const Tile<N, N>& x, char* out, uint64_t ld, uint32_t rows,
                                                    uint32_t depth) const
    {
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t row = wn + j * 16 + (lane & 15), k = wm + i * 16 + quad * 4;
                const f32x4 v = x.v[i][j];
                u32x2 hi, lo;
                uint32_t h0, h1, l0, l1;
                split_halves(v[0], v[1], &h0, &l0);
                split_halves(v[2], v[3], &h1, &l1);
                hi = u32x2{h0, h1};
                lo = u32x2{l0, l1};
                *reinterpret_cast<u32x2*>(lds + at(row, halves_at(k, 0), row)) = hi;
                *reinterpret_cast<u32x2*>(lds + at(row, halves_at(k, 1), row)) = lo;
            }
        __syncthreads();
        copy_rows(out, ld, n_base, rows, m_base, depth, 0);
    }

    // out[m][n]: neighbouring columns lie in neighbouring lanes, which exchange
    // halves, so that each has two columns of two rows.
    __device__ __forceinline__ void store_by_row(const Tile<N, N>& x, char* out, uint64_t ld, uint32_t rows,
                                                 uint32_t depth) const
    {
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4, odd = lane & 1;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const f32x4 v = x.v[i][j];
                uint32_t p01[2], p23[2];
                split_halves(v[0], v[1], &p01[0], &p01[1]);
                split_halves(v[2], v[3], &p23[0], &p23[1]);
                const uint32_t row = wm + i * 16 + quad * 4 + odd * 2, k = wn + j * 16 + (lane & 14);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t give = odd ? p01[q] : p23[q], keep = odd ? p23[q] : p01[q];
                    const uint32_t got = __builtin_amdgcn_mov_dpp(give, 0xB1, 0xF, 0xF, true);  // lane ^ 1
                    const uint32_t lo = odd ? got : keep, hi = odd ? keep : got;
                    const uint32_t byte = halves_at(k, q);
                    *reinterpret_cast<uint32_t*>(lds + at(row, byte, row >> 1)) = __builtin_amdgcn_perm(hi, lo, 0x05040100);
                    *reinterpret_cast<uint32_t*>(lds + at(row + 1, byte, row >> 1)) =
                        __builtin_amdgcn_perm(hi, lo, 0x07060302);
                }
            }
        __syncthreads();
        copy_rows(out, ld, m_base, rows, n_base, depth, 1);
    }

private:
    __device__ __forceinline__ void copy_rows(char* out, uint64_t ld, uint32_t row0, uint32_t rows, uint32_t k0,
                                              uint32_t depth, int key_shift) const
    {
        constexpr uint32_t kChunks = B / 4;  // 16 bytes
        const uint32_t c = threadIdx.x % kChunks;
        if (k0 + c / 8 * 32 >= depth) return;
#pragma unroll 4
        for (uint32_t r = threadIdx.x / kChunks; r < B; r += 256 / kChunks) {
            if (row0 + r >= rows) break;
            *reinterpret_cast<u32x4*>(out + static_cast<uint64_t>(row0 + r) * ld + halves_bytes(k0) + c * 16) =
                *reinterpret_cast<const u32x4*>(lds + at(r, c * 16, r >> key_shift));
        }
    }
};

// The tile of a workgroup. Whole ones: XCD after XCD a contiguous part of the
// order, as tile_of_workgroup; then the parts of split ones.
__device__ __forceinline__ uint32_t halves_tile_id(const HalvesArgs& g, uint32_t* split)
{
    *split = 0;
    if (blockIdx.x >= g.whole) {
        const uint32_t id = blockIdx.x - g.whole;
        *split = id % g.splits;
        return g.whole + id / g.splits;
    }
    const uint32_t xcd = blockIdx.x & 7, part = g.whole >> 3, rest = g.whole & 7;
    return xcd * part + min(xcd, rest) + (blockIdx.x >> 3);
}
__device__ __forceinline__ void halves_place(const HalvesArgs& g, uint32_t id, uint32_t* matrix, uint32_t* tm,
                                             uint32_t* tn)
{
    *matrix = id / g.per_matrix;
    id -= *matrix * g.per_matrix;
    if (g.symmetric) {
        uint32_t r = static_cast<uint32_t>((sqrtf(8.0f * id + 1.0f) - 1.0f) * 0.5f);
        while (r * (r + 1) / 2 > id) --r;
        while ((r + 1) * (r + 2) / 2 <= id) ++r;
        *tm = r;
        *tn = id - r * (r + 1) / 2;
        return;
    }
    constexpr uint32_t GROUP = 8;
    const uint32_t group = id / (GROUP * g.tiles_n), first = group * GROUP;
    const uint32_t high = min(GROUP, g.tiles_m - first);
    const uint32_t in = id - group * GROUP * g.tiles_n;
    *tm = first + in % high;
    *tn = in / high;
}

// B x B tiles, four waves of B/2 x B/2, two workgroups a CU: one waits or stores
// while the other multiplies. JOIN: the split tiles' sums.
template <int B, bool JOIN, class Epilogue>
__global__ __launch_bounds__(256, 2) void gemm_halves(const HalvesArgs g, const Epilogue epi)
{
    using S = HalvesShape<B>;
    using T = MmaF16;
    constexpr int N = S::kTiles;
    __shared__ __attribute__((aligned(1024))) char lds[S::kStages * S::kStage];
    uint32_t matrix, tm, tn, split = 0;
    const uint32_t id = JOIN ? g.whole + blockIdx.x : halves_tile_id(g, &split);
    halves_place(g, id, &matrix, &tm, &tn);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = (wave >> 1) * S::kWave, wn = (wave & 1) * S::kWave;
    const uint32_t m_base = tm * B, n_base = tn * B;

    f32x4* partial = nullptr;
    if (JOIN || id >= g.whole)
        partial = reinterpret_cast<f32x4*>(g.partial) + (static_cast<uint64_t>(id - g.whole) * g.splits + split) * (N * N * 256) + tid;
    Tile<N, N> acc;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) acc.v[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if constexpr (JOIN) {
        for (uint32_t k = 0; k < g.splits; ++k, partial += N * N * 256)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) acc.v[i][j] += partial[(i * N + j) * 256];
    } else {
        uint32_t from = 0, to = g.steps;
        if (partial) {
            const uint32_t part = (g.steps + g.splits - 1) / g.splits;
            from = min(split * part, g.steps);
            to = min(from + part, g.steps);
        }
        auto rows_of = [&](const char* p, uint64_t batch, uint32_t ld, uint32_t r0, uint32_t rows) {
            const uint32_t left = rows > r0 ? min(rows - r0, static_cast<uint32_t>(B)) : 0;
            return __builtin_amdgcn_make_buffer_rsrc(
                const_cast<char*>(p + matrix * batch + static_cast<uint64_t>(r0) * ld), 0, static_cast<int>(left * ld), 0x00020000);
        };
        const __amdgpu_buffer_rsrc_t ra = rows_of(g.a, g.batch_a, g.lda, m_base, g.m);
        const __amdgpu_buffer_rsrc_t rb = rows_of(g.b, g.batch_b, g.ldb, n_base, g.n);
        const uint32_t col = static_cast<uint32_t>((tid & 7) ^ ((tid >> 3) & 7)) * 16;
        uint32_t off_a[S::kLoads], off_b[S::kLoads];
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            off_a[i] = (i * 32 + (tid >> 3)) * g.lda + col;
            off_b[i] = (i * 32 + (tid >> 3)) * g.ldb + col;
        }
        auto fetch = [&](uint32_t where, uint32_t step) {
            const uint32_t at = step * 128;
            const bool in = step < to;
            char* p = lds + where + wave * 1024;
#pragma unroll
            for (int i = 0; i < S::kLoads; ++i) load_to_lds(ra, p + i * 4096, in ? off_a[i] : kPastEnd, at);
#pragma unroll
            for (int i = 0; i < S::kLoads; ++i) load_to_lds(rb, p + S::kB + i * 4096, in ? off_b[i] : kPastEnd, at);
        };

        const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
        const int frow = lane & 15, fcol = lane >> 4;
        const uint32_t swizzled = static_cast<uint32_t>((fcol ^ (frow & 7)) * 16);
        const uint32_t pa = base + (wm + frow) * 128 + swizzled, pb = base + S::kB + (wn + frow) * 128 + swizzled;
        constexpr int kAhead = S::kStages - 1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i * S::kStage, from + i);
        uint32_t stage = 0, ahead = kAhead * S::kStage;
        i32x4 fa[N][2], fb[N][2];
        for (uint32_t k = from; k < to; ++k) {
            // this stage has arrived in every wave, and nobody reads the one before any more
            arrive<(kAhead - 1) * 2 * S::kLoads>();
            fetch(ahead, k + kAhead);
            const uint32_t xa = pa + stage, xb = pb + stage;
            if constexpr (B == 128) {
                read_fragments<0, 0>(fa, fb[0], fb[1], xa, xa ^ 64, xb, xb ^ 64);
                read_fragments4(fb[2], fb[3], (xb ^ 0) + 4096, (xb ^ 64) + 4096);
            } else {
                read_few<2, 2>(fa, fb, xa, xa ^ 64, xb, xb ^ 64);
            }
            constexpr int kOfA[3] = {0, 1, 0}, kOfB[3] = {1, 0, 0};  // the smaller products first
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        acc.v[i][j] = T::mma(__builtin_bit_cast(T::Frag, fa[i][kOfA[p]]),
                                             __builtin_bit_cast(T::Frag, fb[j][kOfB[p]]), acc.v[i][j]);
            ahead = stage;
            stage = stage == kAhead * S::kStage ? 0 : stage + S::kStage;
        }
        // the loads past the end have arrived too: LDS is the epilogue's
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (partial) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) partial[(i * N + j) * 256] = acc.v[i][j];
            return;
        }
    }
    epi(acc, m_base + wm, n_base + wn, g, matrix, HalvesStaging<B>{lds, wm, wn, m_base, n_base}, tm, tn);
}

}  // namespace
}  // namespace lm
}  // namespace ar
