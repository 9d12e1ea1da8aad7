// gemm_halves.h -- products of fp32 values held as two fp16 numbers each.
//
//   x 2^11 = hi + lo,  hi = fp16(x 2^11),  lo = fp16(x 2^11 - hi)
//
// hi + lo holds 22 bits of x; below |x| = 2^-13, where lo is subnormal, it holds x in
// steps of 2^-35. The elements of a matrix of norm 1 are about 1 / sqrt(rows cols),
// 2^-12.5 of 4096 x 8192, 2^-17 of the largest taken: five steps on such, simulated,
// are off by 1.2-1.5 times what 22 bits of every element would leave. Of the four products of a pair, lo lo is left out,
// at 2^-22 of the whole, and hi lo, lo hi and hi hi are summed in fp32: three matrix
// instructions where one fp32 product of the library's takes as long as eight. |x| is
// below 32.
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

// B x B tiles. 256: multiply_large's, one workgroup of eight waves of 128 x 64 a
// CU. 128, 64: four waves of B/2 x B/2, two workgroups a CU: one waits or stores
// while the other multiplies.
template <int B>
struct HalvesShape {
    static_assert(B == 256 || B == 128 || B == 64, "tiles");
    static constexpr int kThreads = B == 256 ? 512 : 256;
    static constexpr int kStages = B == 64 ? 4 : 2;
    static constexpr uint32_t kB = B * 128, kStage = 2 * kB;
    static constexpr int kLoads = B / 32;  // of one operand, a stage and a thread
    static constexpr uint32_t kWaveM = B / 2, kWaveN = B == 256 ? 64 : B / 2;
    static constexpr int MT = kWaveM / 16, NT = kWaveN / 16;
    static constexpr uint32_t kWavesN = B / kWaveN;
};

// A tile leaves through LDS in rows of pieces: at once, or, of 256, a half of
// each wave's columns (or rows) after the other.
template <int B>
struct HalvesStaging {
    using S = HalvesShape<B>;
    static constexpr int MT = S::MT, NT = S::NT, kParts = B == 256 ? 2 : 1;
    char* lds;
    uint32_t wm, wn;          // the wave's row and column among the waves
    uint32_t m_base, n_base;  // the tile's

    // Rows of B * 4 bytes, the 16-byte columns permuted within groups of eight.
    static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t byte, uint32_t key)
    {
        return row * (B * 4) + (byte ^ ((key & 7) * 16));
    }

    // out[n][m], rows `ld` bytes apart, for the first `rows` n and `depth` m (a multiple of 32).
    __device__ __forceinline__ void store_by_column(const Tile<MT, NT>& x, char* out, uint64_t ld, uint32_t rows,
                                                    uint32_t depth) const
    {
        constexpr int J = NT / kParts;
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if constexpr (B == 256) __builtin_amdgcn_sched_barrier(0);  // bounds the registers in use
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint32_t row = (wn * J + j) * 16 + (lane & 15), k = wm * S::kWaveM + i * 16 + quad * 4;
                    const f32x4 v = x.v[i][part * J + j];
                    uint32_t h0, h1, l0, l1;
                    split_halves(v[0], v[1], &h0, &l0);
                    split_halves(v[2], v[3], &h1, &l1);
                    *reinterpret_cast<u32x2*>(lds + at(row, halves_at(k, 0), row)) = u32x2{h0, h1};
                    *reinterpret_cast<u32x2*>(lds + at(row, halves_at(k, 1), row)) = u32x2{l0, l1};
                }
            }
            __syncthreads();
            copy_rows<J * 16, S::kWaveN>(out, ld, n_base + part * J * 16, rows, m_base, depth, 0);
        }
    }

    // out[m][n]: neighbouring columns lie in neighbouring lanes, which exchange
    // halves, so that each has two columns of two rows.
    __device__ __forceinline__ void store_by_row(const Tile<MT, NT>& x, char* out, uint64_t ld, uint32_t rows,
                                                 uint32_t depth) const
    {
        constexpr int I = MT / kParts;
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4, odd = lane & 1;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if constexpr (B == 256) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    const f32x4 v = x.v[part * I + i][j];
                    uint32_t p01[2], p23[2];
                    split_halves(v[0], v[1], &p01[0], &p01[1]);
                    split_halves(v[2], v[3], &p23[0], &p23[1]);
                    const uint32_t row = (wm * I + i) * 16 + quad * 4 + odd * 2, k = wn * S::kWaveN + j * 16 + (lane & 14);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t give = odd ? p01[q] : p23[q], keep = odd ? p23[q] : p01[q];
                        const uint32_t got = __builtin_amdgcn_mov_dpp(give, 0xB1, 0xF, 0xF, true);  // lane ^ 1
                        const uint32_t lo = odd ? got : keep, hi = odd ? keep : got;
                        const uint32_t byte = halves_at(k, q);
                        *reinterpret_cast<uint32_t*>(lds + at(row, byte, row >> 1)) =
                            __builtin_amdgcn_perm(hi, lo, 0x05040100);
                        *reinterpret_cast<uint32_t*>(lds + at(row + 1, byte, row >> 1)) =
                            __builtin_amdgcn_perm(hi, lo, 0x07060302);
                    }
                }
            }
            __syncthreads();
            copy_rows<I * 16, S::kWaveM>(out, ld, m_base + part * I * 16, rows, n_base, depth, 1);
        }
    }

private:
    // Row r of LDS is row r % PART of the part of wave r / PART, of WAVE rows each.
    template <uint32_t PART, uint32_t WAVE>
    __device__ __forceinline__ void copy_rows(char* out, uint64_t ld, uint32_t row0, uint32_t rows, uint32_t k0,
                                              uint32_t depth, int key_shift) const
    {
        constexpr uint32_t kChunks = B / 4;  // 16 bytes
        const uint32_t c = threadIdx.x % kChunks;
        if (k0 + c / 8 * 32 >= depth) return;
#pragma unroll 4
        for (uint32_t r = threadIdx.x / kChunks; r < B / kParts; r += S::kThreads / kChunks) {
            const uint32_t to = row0 + r / PART * WAVE + r % PART;
            if (to >= rows) continue;
            *reinterpret_cast<u32x4*>(out + to * ld + halves_bytes(k0) + c * 16) =
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

// The product of one tile, into `acc`.
template <int B>
__device__ __forceinline__ void multiply_halves(char* lds, const char* a, const char* b, const HalvesArgs& g,
                                                uint32_t m_base, uint32_t n_base, uint32_t steps,
                                                Tile<HalvesShape<B>::MT, HalvesShape<B>::NT>& acc)
{
    using S = HalvesShape<B>;
    using T = MmaF16;
    constexpr int N = S::NT;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = (wave >> 1) * S::kWaveM, wn = (wave & 1) * S::kWaveN;
    auto rows_of = [&](const char* p, uint32_t ld, uint32_t r0, uint32_t rows) {
        const uint32_t left = rows > r0 ? min(rows - r0, static_cast<uint32_t>(B)) : 0;
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p + static_cast<uint64_t>(r0) * ld), 0,
                                                 static_cast<int>(left * ld), 0x00020000);
    };
    const __amdgpu_buffer_rsrc_t ra = rows_of(a, g.lda, m_base, g.m);
    const __amdgpu_buffer_rsrc_t rb = rows_of(b, g.ldb, n_base, g.n);
    const uint32_t col = static_cast<uint32_t>((tid & 7) ^ ((tid >> 3) & 7)) * 16;
    uint32_t off_a[S::kLoads], off_b[S::kLoads];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
        off_a[i] = (i * 32 + (tid >> 3)) * g.lda + col;
        off_b[i] = (i * 32 + (tid >> 3)) * g.ldb + col;
    }
    auto fetch = [&](uint32_t where, uint32_t step) {
        const uint32_t at = step * 128;
        const bool in = step < steps;
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
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) acc.v[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int kAhead = S::kStages - 1;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i * S::kStage, i);
    uint32_t stage = 0, ahead = kAhead * S::kStage;
    i32x4 fa[N][2], fb[N][2];
    for (uint32_t k = 0; k < steps; ++k) {
        // this stage has arrived in every wave, and nobody reads the one before any more
        arrive<(kAhead - 1) * 2 * S::kLoads>();
        fetch(ahead, k + kAhead);
        const uint32_t xa = pa + stage, xb = pb + stage;
        if constexpr (B == 128) {
            read_fragments<0, 0>(fa, fb[0], fb[1], xa, xa ^ 64, xb, xb ^ 64);
            read_fragments4(fb[2], fb[3], xb + 4096, (xb ^ 64) + 4096);
        } else {
            read_few<2, 2>(fa, fb, xa, xa ^ 64, xb, xb ^ 64);
        }
        constexpr int kOfA[3] = {0, 1, 0}, kOfB[3] = {1, 0, 0};  // the smaller products first
        // (of 48 products, ahead of the other workgroup's reads: 4096 x 8192 4.64 -> 4.54 ms;
        // of 12 it costs: 3 x 1027 x 770 271 -> 274 us)
        if constexpr (B == 128) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    acc.v[i][j] = T::mma(__builtin_bit_cast(T::Frag, fa[i][kOfA[p]]),
                                         __builtin_bit_cast(T::Frag, fb[j][kOfB[p]]), acc.v[i][j]);
        if constexpr (B == 128) __builtin_amdgcn_s_setprio(0);
        ahead = stage;
        stage = stage == kAhead * S::kStage ? 0 : stage + S::kStage;
    }
    // the loads past the end have arrived too: LDS is the epilogue's
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// JOIN: the split tiles' sums.
template <int B, bool JOIN, class Epilogue>
__global__ __launch_bounds__(HalvesShape<B>::kThreads, 2) void gemm_halves(const HalvesArgs g, const Epilogue epi)
{
    using S = HalvesShape<B>;
    constexpr int MT = S::MT, NT = S::NT;
    __shared__ __attribute__((aligned(1024))) char lds[S::kStages * S::kStage];
    uint32_t matrix, tm, tn, split = 0;
    const uint32_t id = JOIN ? g.whole + blockIdx.x : halves_tile_id(g, &split);
    halves_place(g, id, &matrix, &tm, &tn);
    const int tid = threadIdx.x;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = wave / S::kWavesN, wn = wave % S::kWavesN;
    const uint32_t m_base = tm * B, n_base = tn * B;

    // (decided by `id`, the same in all lanes, and not by the pointer: descriptors
    // that may differ from lane to lane are loaded through in loops)
    const bool cut = JOIN || id >= g.whole;
    f32x4* partial = reinterpret_cast<f32x4*>(g.partial) + tid;
    if (cut) partial += (static_cast<uint64_t>(id - g.whole) * g.splits + split) * (MT * NT * S::kThreads);
    Tile<MT, NT> acc;
    if constexpr (JOIN) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc.v[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        // two parts' loads at a time: sixteen of 16 tiles of 128 in 15 us rather than 29
        constexpr uint32_t kPart = MT * NT * S::kThreads;
        uint32_t k = 0;
        for (; k + 2 <= g.splits; k += 2, partial += 2 * kPart) {
            f32x4 x[MT * NT], y[MT * NT];
#pragma unroll
            for (int i = 0; i < MT * NT; ++i) x[i] = partial[i * S::kThreads];
#pragma unroll
            for (int i = 0; i < MT * NT; ++i) y[i] = partial[i * S::kThreads + kPart];
#pragma unroll
            for (int i = 0; i < MT * NT; ++i) acc.v[i / NT][i % NT] += x[i];
#pragma unroll
            for (int i = 0; i < MT * NT; ++i) acc.v[i / NT][i % NT] += y[i];
        }
        for (; k < g.splits; ++k, partial += kPart)
#pragma unroll
            for (int i = 0; i < MT * NT; ++i) acc.v[i / NT][i % NT] += partial[i * S::kThreads];
    } else {
        uint32_t from = 0, to = g.steps;
        if (cut) {
            const uint32_t part = (g.steps + g.splits - 1) / g.splits;
            from = min(split * part, g.steps);
            to = min(from + part, g.steps);
        }
        const char *a = g.a + matrix * g.batch_a + from * 128ull, *b = g.b + matrix * g.batch_b + from * 128ull;
        if constexpr (B == 256)
            multiply_large<MmaF16, true>(lds, LargeOperand{a, g.lda, m_base, g.m}, LargeOperand{b, g.ldb, n_base, g.n},
                                         (to - from) * kTileK, acc);
        else
            multiply_halves<B>(lds, a, b, g, m_base, n_base, to - from, acc);
        if (cut) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) partial[(i * NT + j) * S::kThreads] = acc.v[i][j];
            return;
        }
    }
    epi(acc, m_base + wm * S::kWaveM, n_base + wn * S::kWaveN, g, matrix, HalvesStaging<B>{lds, wm, wn, m_base, n_base}, tm,
        tn);
}

}  // namespace
}  // namespace lm
}  // namespace ar
