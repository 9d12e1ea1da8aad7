// gemm.h -- the matrix-core products that the cross entropy is made of.
//
//   C[m][n] = sum_k A[m][k] * B[n][k]
//
// for A and B whose rows are contiguous along K and 16-byte aligned; C
// stays in fp32 registers and goes to an epilogue. Tiles of both go from
// memory straight into LDS. Three kernels: gemm_large for 256 x 256 tiles,
// gemm_pieces for fp32 operands in three bf16 pieces, and gemm_few for few
// rows of B, which is bound by reading A.
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
using detail::u32x2;
using detail::u32x4;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A matrix instruction: the operands' storage, and a fragment, 16 bytes of a
// row's depth for each lane.
struct MmaBF16 {
    using Elem = uint16_t;
    using Frag = bf16x8;
    using Format = detail::BF16;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // Two floats, rounded to nearest even, the first in the low half.
    static __device__ __forceinline__ uint32_t pack2(float x, float y)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
    }
};
struct MmaF16 {
    using Elem = uint16_t;
    using Frag = f16x8;
    using Format = detail::F16;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack2(float x, float y)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, f16x2));
    }
};

// Its depth is four; the order in which a row's depth is summed is free as long
// as both operands keep to it, so a lane's four values are four of them.
struct MmaF32 {
    using Elem = float;
    using Frag = f32x4;
    using Format = detail::F32;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
};

// Rows of A and B beyond M and N, and depths beyond k_all, are read as zeros.
struct GemmArgs {
    const char* a;
    const char* b;
    uint64_t lda, ldb;  // bytes
    uint32_t m, n;
    uint32_t k;         // elements of one split; a multiple of kTileK if there are several
    uint32_t k_all;     // whole 16-byte columns (32 elements of pieces); splits * k may pass it
    uint32_t tiles_m, tiles_n, splits;
};

// Where a lane's results lie: acc[i][j][r] is C[m][n] with
//   m = m0 + 16 i + 4 (lane / 16) + r,  n = n0 + 16 j + lane % 16.
template <int MT, int NT>
struct Tile {
    f32x4 v[MT][NT];
};

// A byte offset that lies past every buffer: the load gives zeros.
constexpr uint32_t kPastEnd = 0x80000000u;

// Up to 64 rows from row `r0` of a matrix of `rows` rows, `ld` (below 2^25)
// bytes apart; rows past the end lie outside the buffer.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const char* p, uint64_t ld, uint32_t r0, uint32_t rows)
{
    const uint32_t left = rows > r0 ? min(rows - r0, 64u) : 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p + static_cast<uint64_t>(r0) * ld), 0,
                                             static_cast<int>(left * static_cast<uint32_t>(ld)), 0x00020000);
}

// Sixteen bytes a lane, straight into LDS from `to` (of the wave) on; the
// instruction's own offset would move both ends, so `at` is the scalar one.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, char* to, uint32_t off, uint32_t at)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, off, at, 0, 0);
}

// Workgroups go round the eight XCDs one by one; each XCD gets a contiguous
// part of the tile order, in which tiles of eight row blocks follow each
// other, so that what an XCD works on at a time shares rows of both operands
// in its L2.
__device__ __forceinline__ void tile_of_workgroup(const GemmArgs& g, uint32_t* tm, uint32_t* tn, uint32_t* split)
{
    const uint32_t total = gridDim.x, xcd = blockIdx.x & 7, part = total >> 3, rest = total & 7;
    uint32_t id = xcd * part + min(xcd, rest) + (blockIdx.x >> 3);
    const uint32_t per_split = g.tiles_m * g.tiles_n;
    *split = id / per_split;
    id -= *split * per_split;
    constexpr uint32_t GROUP = 8;
    const uint32_t group = id / (GROUP * g.tiles_n), first = group * GROUP;
    const uint32_t high = min(GROUP, g.tiles_m - first);
    const uint32_t in = id - group * GROUP * g.tiles_n;
    *tm = first + in % high;
    *tn = in / high;
}

// ---------------------------------------------------------------------------
// storing a tile of 16-bit results in rows, through LDS
// ---------------------------------------------------------------------------
// A lane's results are four rows of one column; stored as they lie they make
// pieces of 32 bytes. A 256 x 256 tile of 16-bit values fills the 128 KiB that
// the product's stages held, and leaves in whole rows of 512 bytes; `nt`:
// non-temporal stores.
struct NoStaging {
    static constexpr bool kOn = false;
};
struct Staging {
    static constexpr bool kOn = true;
    char* lds;
    uint32_t m, n;            // the wave's first row and column within the tile
    uint32_t m_base, n_base;  // the tile's

    // Rows of 32 16-byte columns, permuted by the row within groups of eight
    // so that the lanes of one write spread over the banks.
    static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t byte, uint32_t key)
    {
        return row * 512 + (byte ^ ((key & 7) * 16));
    }

    // out[n][m], `ld` apart, for the first `rows` n and `cols` m (a multiple of 8).
    template <class T, int MT, int NT>
    __device__ __forceinline__ void store_by_column(const Tile<MT, NT>& x, uint16_t* out, uint64_t ld, uint32_t rows,
                                                    uint32_t cols, bool nt) const
    {
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            __builtin_amdgcn_sched_barrier(0);  // bounds the registers in use
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t row = n + j * 16 + (lane & 15), col = m + i * 16 + quad * 4;
                const f32x4 v = x.v[i][j];
                *reinterpret_cast<u32x2*>(lds + at(row, col * 2, row)) = u32x2{T::pack2(v[0], v[1]), T::pack2(v[2], v[3])};
            }
        }
        __syncthreads();
        copy_rows(out, ld, n_base, rows, m_base, cols, 0, nt);
    }

    // out[m][n]: neighbouring columns lie in neighbouring lanes, which
    // exchange halves, so that each has two columns of two rows.
    template <class T, int MT, int NT>
    __device__ __forceinline__ void store_by_row(const Tile<MT, NT>& x, const float (&factor)[NT], uint16_t* out,
                                                 uint64_t ld, uint32_t rows, uint32_t cols, bool nt) const
    {
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4, odd = lane & 1;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const f32x4 v = x.v[i][j] * factor[j];
                const uint32_t p01 = T::pack2(v[0], v[1]), p23 = T::pack2(v[2], v[3]);
                const uint32_t give = odd ? p01 : p23, keep = odd ? p23 : p01;
                const uint32_t got = __builtin_amdgcn_mov_dpp(give, 0xB1, 0xF, 0xF, true);  // lane ^ 1
                const uint32_t lo = odd ? got : keep, hi = odd ? keep : got;
                const uint32_t row = m + i * 16 + quad * 4 + odd * 2, byte = (n + j * 16 + (lane & 14)) * 2;
                *reinterpret_cast<uint32_t*>(lds + at(row, byte, row >> 1)) = __builtin_amdgcn_perm(hi, lo, 0x05040100);
                *reinterpret_cast<uint32_t*>(lds + at(row + 1, byte, row >> 1)) = __builtin_amdgcn_perm(hi, lo, 0x07060302);
            }
        }
        __syncthreads();
        copy_rows(out, ld, m_base, rows, n_base, cols, 1, nt);
    }

private:
    __device__ __forceinline__ void copy_rows(uint16_t* out, uint64_t ld, uint32_t row0, uint32_t rows, uint32_t col0,
                                              uint32_t cols, int key_shift, bool nt) const
    {
        const uint32_t c = threadIdx.x & 31;
#pragma unroll 4
        for (uint32_t r = threadIdx.x >> 5; r < 256; r += 16) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(lds + at(r, c * 16, r >> key_shift));
            if (row0 + r >= rows || col0 + c * 8 >= cols) continue;
            u32x4* to = reinterpret_cast<u32x4*>(out + static_cast<uint64_t>(row0 + r) * ld + col0 + c * 8);
            if (nt) __builtin_nontemporal_store(v, to);
            else *to = v;
        }
    }
};

// ---------------------------------------------------------------------------
// the large tile
// ---------------------------------------------------------------------------
typedef int i32x4 __attribute__((ext_vector_type(4)));

// Twelve 16-byte fragments from LDS and the wait for them: four groups of 16
// rows at a0 (the first 32 of the depth) and a1 (the other 32), A_OFF bytes
// on, and two groups at b0 and b1, B_OFF bytes on. One block of instructions:
// the compiler would wait for the direct loads in flight before any LDS read
// of its own.
template <int A_OFF, int B_OFF>
__device__ __forceinline__ void read_fragments(i32x4 (&a)[4][2], i32x4 (&b0)[2], i32x4 (&b1)[2], uint32_t pa0,
                                               uint32_t pa1, uint32_t pb0, uint32_t pb1)
{
    asm volatile(
        "ds_read_b128 %0, %12 offset:%16\n"
        "ds_read_b128 %1, %13 offset:%16\n"
        "ds_read_b128 %2, %12 offset:%17\n"
        "ds_read_b128 %3, %13 offset:%17\n"
        "ds_read_b128 %4, %12 offset:%18\n"
        "ds_read_b128 %5, %13 offset:%18\n"
        "ds_read_b128 %6, %12 offset:%19\n"
        "ds_read_b128 %7, %13 offset:%19\n"
        "ds_read_b128 %8, %14 offset:%20\n"
        "ds_read_b128 %9, %15 offset:%20\n"
        "ds_read_b128 %10, %14 offset:%21\n"
        "ds_read_b128 %11, %15 offset:%21\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[1][0]), "=&v"(a[1][1]), "=&v"(a[2][0]), "=&v"(a[2][1]),
          "=&v"(a[3][0]), "=&v"(a[3][1]), "=&v"(b0[0]), "=&v"(b0[1]), "=&v"(b1[0]), "=&v"(b1[1])
        : "v"(pa0), "v"(pa1), "v"(pb0), "v"(pb1), "n"(A_OFF), "n"(A_OFF + 2048), "n"(A_OFF + 4096), "n"(A_OFF + 6144),
          "n"(B_OFF), "n"(B_OFF + 2048)
        : "memory");
}

__device__ __forceinline__ void read_fragments4(i32x4 (&b0)[2], i32x4 (&b1)[2], uint32_t pb0, uint32_t pb1)
{
    asm volatile(
        "ds_read_b128 %0, %4\n"
        "ds_read_b128 %1, %5\n"
        "ds_read_b128 %2, %4 offset:2048\n"
        "ds_read_b128 %3, %5 offset:2048\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(b0[0]), "=&v"(b0[1]), "=&v"(b1[0]), "=&v"(b1[1])
        : "v"(pb0), "v"(pb1)
        : "memory");
}

// MT groups of 16 rows at a0 and a1, NT at b0 and b1.
template <int MT, int NT>
__device__ __forceinline__ void read_few(i32x4 (&a)[MT][2], i32x4 (&b)[NT][2], uint32_t a0, uint32_t a1, uint32_t b0,
                                         uint32_t b1)
{
    if constexpr (MT == 2 && NT == 2) {
        asm volatile(
            "ds_read_b128 %0, %8\n"
            "ds_read_b128 %1, %9\n"
            "ds_read_b128 %2, %8 offset:2048\n"
            "ds_read_b128 %3, %9 offset:2048\n"
            "ds_read_b128 %4, %10\n"
            "ds_read_b128 %5, %11\n"
            "ds_read_b128 %6, %10 offset:2048\n"
            "ds_read_b128 %7, %11 offset:2048\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[1][0]), "=&v"(a[1][1]), "=&v"(b[0][0]), "=&v"(b[0][1]),
              "=&v"(b[1][0]), "=&v"(b[1][1])
            : "v"(a0), "v"(a1), "v"(b0), "v"(b1)
            : "memory");
    } else {
        static_assert(MT == 1 && NT == 1, "");
        asm volatile(
            "ds_read_b128 %0, %4\n"
            "ds_read_b128 %1, %5\n"
            "ds_read_b128 %2, %6\n"
            "ds_read_b128 %3, %7\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(b[0][0]), "=&v"(b[0][1])
            : "v"(a0), "v"(a1), "v"(b0), "v"(b1)
            : "memory");
    }
}

// All but the newest N direct loads have arrived, in every wave.
template <int N>
__device__ __forceinline__ void arrive()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)\n s_barrier" : : "n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// One operand's part: rows row0 .. of `rows`, from depth 0 on.
struct LargeOperand {
    const char* p;
    uint64_t ld;  // bytes
    uint32_t row0, rows;
};

// 256 x 256 x 64 tiles, 8 waves of 128 x 64. The two waves of a SIMD (w and
// w + 4) take turns: while one issues a half step's 32 matrix instructions,
// the other reads its fragments for the next half step and issues direct
// loads. Half step 0 of step k multiplies the first 64 of the wave's rows of
// A, half step 1 the other 64. Direct loads run up to two steps ahead: a
// quarter of a stage is loaded again as soon as its last reader's barrier is
// passed, and only the oldest loads are waited for. 8192 x 4096 x 13312 bf16 in
// 600 us, 1.49 PFLOP/s, as much as a large library product reaches (1.3-1.48);
// with one barrier a step and all loads waited for it took 929.
//
// HALVES: the 64 of a step are 32 hi and 32 lo of pairs (gemm_halves.h), of whose
// products lo lo is left out and the smaller ones come first.
template <class T, bool HALVES>
__device__ __forceinline__ void multiply_large(char* lds, const LargeOperand& oa, const LargeOperand& ob, uint32_t depth,
                                               Tile<8, 4>& acc)
{
    constexpr uint32_t kStage = 65536, kA1 = 16384, kB = 32768, kB1 = 49152;
    const uint32_t steps = (depth + kTileK - 1) / kTileK;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;

    const uint32_t col = static_cast<uint32_t>((tid & 7) ^ ((tid >> 3) & 7)) * 8;
    const uint32_t off_a = (tid >> 3) * static_cast<uint32_t>(oa.ld) + col * 2;
    const uint32_t off_b = (tid >> 3) * static_cast<uint32_t>(ob.ld) + col * 2;
    auto part = [](const LargeOperand& o, uint32_t at) { return row_buffer(o.p, o.ld, o.row0 + at, o.rows); };
    const __amdgpu_buffer_rsrc_t ra0 = part(oa, 0), ra1 = part(oa, 64), ra2 = part(oa, 128), ra3 = part(oa, 192);
    const __amdgpu_buffer_rsrc_t rb0 = part(ob, 0), rb1 = part(ob, 64), rb2 = part(ob, 128), rb3 = part(ob, 192);
    auto fetch = [&](__amdgpu_buffer_rsrc_t x, __amdgpu_buffer_rsrc_t y, uint32_t to, uint32_t off, uint32_t step) {
        const uint32_t at = step * kTileK;
        const uint32_t v = at + col < depth ? off : kPastEnd;
        char* p = lds + to + wave * 1024;
        load_to_lds(x, p, v, at * 2);
        load_to_lds(y, p + 8192, v, at * 2);
    };

#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc.v[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    i32x4 fa0[4][2], fa1[4][2], fb[4][2];
    auto multiply = [&](i32x4 (&f)[4][2], int i0) {
        __builtin_amdgcn_s_setprio(1);
        constexpr int kOfA[3] = {0, 1, 0}, kOfB[3] = {HALVES ? 1 : 0, HALVES ? 0 : 1, 0};
#pragma unroll
        for (int p = 0; p < (HALVES ? 3 : 2); ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc.v[i0 + i][j] = T::mma(__builtin_bit_cast(typename T::Frag, f[i][kOfA[p]]),
                                              __builtin_bit_cast(typename T::Frag, fb[j][kOfB[p]]), acc.v[i0 + i][j]);
        __builtin_amdgcn_s_setprio(0);
    };

    if (steps) {
        const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
        const int frow = lane & 15, fcol = lane >> 4;
        const uint32_t swizzled = static_cast<uint32_t>((fcol ^ (frow & 7)) * 16);
        uint32_t pa = base + (wm * 64 + frow) * 128 + swizzled;
        uint32_t pb = base + kB + (wn * 64 + frow) * 128 + swizzled;
        fetch(ra0, ra2, 0, off_a, 0);
        fetch(rb0, rb1, kB, off_b, 0);
        fetch(rb2, rb3, kB1, off_b, 0);
        fetch(ra1, ra3, kA1, off_a, 0);
        fetch(ra0, ra2, kStage, off_a, 1);
        fetch(rb0, rb1, kStage + kB, off_b, 1);
        arrive<6>();
        read_fragments4(fa0[0], fa0[1], pa, pa ^ 64);
        if (wave >= 4) meet();
        uint32_t stage = 0;
        for (uint32_t k = 0; k < steps; ++k) {
            fetch(rb2, rb3, (stage ^ kStage) + kB1, off_b, k + 1);
            fetch(ra1, ra3, (stage ^ kStage) + kA1, off_a, k + 1);
            read_fragments<0, 4096>(fb, fa0[2], fa0[3], pb, pb ^ 64, pa, pa ^ 64);
            arrive<6>();
            multiply(fa0, 0);
            meet();
            fetch(ra0, ra2, stage, off_a, k + 2);
            fetch(rb0, rb1, stage + kB, off_b, k + 2);
            read_fragments<kA1, 0>(fa1, fa0[0], fa0[1], pa, pa ^ 64, pa ^ kStage, pa ^ kStage ^ 64);
            arrive<6>();
            multiply(fa1, 4);
            meet();
            pa ^= kStage;
            pb ^= kStage;
            stage ^= kStage;
        }
        if (wave < 4) meet();
        // the loads past the end have arrived too: LDS is the epilogue's
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }
}

template <class T, class Epilogue>
__global__ __launch_bounds__(512, 2) void gemm_large(const GemmArgs g, const Epilogue epi)
{
    __shared__ __attribute__((aligned(1024))) char lds[2 * 65536];
    uint32_t tm, tn, split;
    tile_of_workgroup(g, &tm, &tn, &split);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const uint32_t m_base = tm * 256, n_base = tn * 256;
    const uint32_t k0 = split * g.k;
    const uint32_t depth = k0 < g.k_all ? min(g.k, g.k_all - k0) : 0;
    Tile<8, 4> acc;
    multiply_large<T, false>(lds, LargeOperand{g.a + static_cast<uint64_t>(k0) * 2, g.lda, m_base, g.m},
                             LargeOperand{g.b + static_cast<uint64_t>(k0) * 2, g.ldb, n_base, g.n}, depth, acc);
    epi(acc, m_base + wm * 128, n_base + wn * 64, g, tm * 2 + wm, split, Staging{lds, wm * 128u, wn * 64u, m_base, n_base});
}

// ---------------------------------------------------------------------------
// few rows of B
// ---------------------------------------------------------------------------
// The time is that of reading A once: 64 rows of A and 16 or 64 of B, stages of
// 128 bytes a row, all but one of them in flight, each waited for when it is
// due; two workgroups a CU, so that one starts or ends while the other reads.
// fp32 rows are read as they are: their matrix instructions' 157 TFLOP/s keep
// up with the memory here. From HBM, microseconds a loss, against tiles of 256
// rows (and four stages, one workgroup a CU): 3 tokens x 65536 x 2048 fp16 57
// against 67, 1 x 128256 x 2048 bf16 101 against 123, 40 x 65536 x 2048 fp16 65
// against 70; 16 x 131072 x 4096 bf16 185 against 179.
constexpr int kFewM = 64;

template <int BN>
struct FewShape {
    static_assert(BN == 16 || BN == 64, "tiles");
    static constexpr int kThreads = 256;
    static constexpr int kRows = kThreads / 8;              // of one load
    static constexpr int kRowsB = BN > kRows ? BN : kRows;  // every wave has as many loads in flight
    static constexpr int kLoadsA = kFewM / kRows, kLoadsB = kRowsB / kRows;
    static constexpr int kStages = BN == 16 ? 6 : 4;
    static constexpr uint32_t kB = kFewM * 128, kStage = kB + kRowsB * 128;
    static constexpr int WN = BN == 16 ? 1 : 2, WM = 4 / WN;  // waves
    static constexpr int MT = kFewM / (16 * WM), NT = BN / (16 * WN);
};

template <class T, int BN, class Epilogue>
__global__ __launch_bounds__(256, 2) void gemm_few(const GemmArgs g, const Epilogue epi)
{
    using S = FewShape<BN>;
    constexpr int MT = S::MT, NT = S::NT;
    __shared__ __attribute__((aligned(1024))) char lds[S::kStages * S::kStage];
    uint32_t tm, tn, split;
    tile_of_workgroup(g, &tm, &tn, &split);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = wave / S::WN, wn = wave % S::WN;
    const uint32_t m_base = tm * kFewM, n_base = tn * BN;
    const uint32_t k0 = split * g.k;
    const uint32_t depth = k0 < g.k_all ? min(g.k, g.k_all - k0) : 0;
    constexpr uint32_t EB = sizeof(typename T::Elem), kDepth = 128 / EB;
    const uint32_t steps = (depth + kDepth - 1) / kDepth;

    const uint32_t col = static_cast<uint32_t>((tid & 7) ^ ((tid >> 3) & 7)) * 16;  // bytes
    const uint32_t off_a = (tid >> 3) * static_cast<uint32_t>(g.lda) + col;
    const uint32_t off_b = (tid >> 3) * static_cast<uint32_t>(g.ldb) + col;
    const char *a = g.a + static_cast<uint64_t>(k0) * EB, *b = g.b + static_cast<uint64_t>(k0) * EB;
    const uint32_t n_rows = min(g.n, n_base + BN);
    auto fetch = [&](uint32_t to, uint32_t step) {
        const uint32_t at = step * 128;
        const bool in = at + col < depth * EB;
        char* p = lds + to + wave * 1024;
#pragma unroll
        for (int i = 0; i < S::kLoadsA; ++i)
            load_to_lds(row_buffer(a, g.lda, m_base + i * S::kRows, g.m), p + i * S::kRows * 128, in ? off_a : kPastEnd, at);
#pragma unroll
        for (int i = 0; i < S::kLoadsB; ++i)
            load_to_lds(row_buffer(b, g.ldb, n_base + i * S::kRows, n_rows), p + S::kB + i * S::kRows * 128,
                        in ? off_b : kPastEnd, at);
    };

    Tile<MT, NT> acc;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc.v[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (steps) {
        const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
        const int frow = lane & 15, fcol = lane >> 4;
        const uint32_t swizzled = static_cast<uint32_t>((fcol ^ (frow & 7)) * 16);
        const uint32_t pa = base + (wm * MT * 16 + frow) * 128 + swizzled;
        const uint32_t pb = base + S::kB + (wn * NT * 16 + frow) * 128 + swizzled;
        constexpr int kAhead = S::kStages - 1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i * S::kStage, i);
        uint32_t stage = 0, ahead = kAhead * S::kStage;
        i32x4 fa[MT][2], fb[NT][2];
        for (uint32_t k = 0; k < steps; ++k) {
            // this stage has arrived in every wave, and nobody reads the one before any more
            arrive<(kAhead - 1) * (S::kLoadsA + S::kLoadsB)>();
            fetch(ahead, k + kAhead);
            const uint32_t xa = pa + stage, xb = pb + stage;
            read_few<MT, NT>(fa, fb, xa, xa ^ 64, xb, xb ^ 64);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc.v[i][j] = T::mma(__builtin_bit_cast(typename T::Frag, fa[i][kk]),
                                             __builtin_bit_cast(typename T::Frag, fb[j][kk]), acc.v[i][j]);
            ahead = stage;
            stage = stage == kAhead * S::kStage ? 0 : stage + S::kStage;
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    epi(acc, m_base + wm * MT * 16, n_base + wn * NT * 16, g, tm * S::WM + wm, split, NoStaging{});
}

// ---------------------------------------------------------------------------
// fp32 operands in three bf16 pieces
// ---------------------------------------------------------------------------
// x = x1 + x2 + x3 with 8 significant bits each. A row holds, for each 32 of
// its depth, 32 first pieces, 32 second and 32 third ones (192 bytes). Six of
// the nine products of pieces are summed, smallest first: 3 1, 2 2, 1 3, 2 1, 1 2,
// 1 1. The other three are below 2^-24 of the whole.
constexpr int kPieces = 3;
constexpr int kPieceDepth = 32;
constexpr int kPiecesN = 128;  // columns of a tile

// The first or the second of two 16-bit pieces, as floats.
__device__ __forceinline__ float low_piece(uint32_t w) { return detail::as_f(w << 16); }
__device__ __forceinline__ float high_piece(uint32_t w) { return detail::as_f(w & 0xFFFF0000u); }

// The pieces of two floats below kCutFrom (or of d, whose other factors these
// are), the first in the low halves.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&p)[3])
{
    p[0] = MmaBF16::pack2(x, y);
    const float rx = x - low_piece(p[0]), ry = y - high_piece(p[0]);
    p[1] = MmaBF16::pack2(rx, ry);
    p[2] = MmaBF16::pack2(rx - low_piece(p[1]), ry - high_piece(p[1]));
}

// The pieces of any two floats. From kCutFrom on a number is cut rather than
// rounded to its pieces: the largest ones would round to an infinity, and pieces
// of one sign leave no product beyond fp32's range with infinities of both (x1
// y2 of a y below kCutFrom stays within the range). The products left out are
// then below 2^-21 where both factors are cut. An infinity is the third piece,
// which meets the other factor's first alone, beside a first piece of +-1: its
// products are the infinity of their sign, and no number with a zero.
constexpr float kCutFrom = 256.0f;
__device__ __forceinline__ void split_pair_any(float x, float y, uint32_t (&p)[3])
{
    auto cut = [](float v) { return detail::as_f(detail::as_u(v) & 0xFFFF0000u); };
    auto first = [&](float v) {
        return __builtin_isinf(v) ? __builtin_copysignf(1.0f, v) : __builtin_fabsf(v) >= kCutFrom ? cut(v) : v;
    };
    auto second = [&](float v, float rest) {
        return __builtin_isinf(rest) ? 0.0f : __builtin_fabsf(v) >= kCutFrom ? cut(rest) : rest;
    };
    p[0] = MmaBF16::pack2(first(x), first(y));
    const float rx = x - low_piece(p[0]), ry = y - high_piece(p[0]);
    p[1] = MmaBF16::pack2(second(x, rx), second(y, ry));
    p[2] = MmaBF16::pack2(rx - low_piece(p[1]), ry - high_piece(p[1]));
}

// Twelve fragments: two groups of 16 rows at x and two at y, three pieces each.
template <int X_OFF, int Y_OFF>
__device__ __forceinline__ void read_pieces(i32x4 (&x0)[3], i32x4 (&x1)[3], i32x4 (&y0)[3], i32x4 (&y1)[3], uint32_t x,
                                            uint32_t y)
{
    asm volatile(
        "ds_read_b128 %0, %12 offset:%14\n"
        "ds_read_b128 %1, %12 offset:%15\n"
        "ds_read_b128 %2, %12 offset:%16\n"
        "ds_read_b128 %3, %12 offset:%17\n"
        "ds_read_b128 %4, %12 offset:%18\n"
        "ds_read_b128 %5, %12 offset:%19\n"
        "ds_read_b128 %6, %13 offset:%20\n"
        "ds_read_b128 %7, %13 offset:%21\n"
        "ds_read_b128 %8, %13 offset:%22\n"
        "ds_read_b128 %9, %13 offset:%23\n"
        "ds_read_b128 %10, %13 offset:%24\n"
        "ds_read_b128 %11, %13 offset:%25\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x0[0]), "=&v"(x0[1]), "=&v"(x0[2]), "=&v"(x1[0]), "=&v"(x1[1]), "=&v"(x1[2]), "=&v"(y0[0]),
          "=&v"(y0[1]), "=&v"(y0[2]), "=&v"(y1[0]), "=&v"(y1[1]), "=&v"(y1[2])
        : "v"(x), "v"(y), "n"(X_OFF), "n"(X_OFF + 8192), "n"(X_OFF + 16384), "n"(X_OFF + 1024), "n"(X_OFF + 9216),
          "n"(X_OFF + 17408), "n"(Y_OFF), "n"(Y_OFF + 8192), "n"(Y_OFF + 16384), "n"(Y_OFF + 1024), "n"(Y_OFF + 9216),
          "n"(Y_OFF + 17408)
        : "memory");
}

// A 256 x 128 tile of 16-bit values in the layout of pieces leaves in two
// halves, each in whole rows: the first and the last 32 of each wave's 64 rows
// (or columns), so that all waves work on both.
struct PieceStaging {
    static constexpr bool kOn = true;
    char* lds;
    uint32_t wm, wn;          // the wave's 64 rows and 64 columns within the tile
    uint32_t m_base, n_base;  // the tile's

    static __device__ __forceinline__ uint32_t byte_of(uint32_t k, uint32_t piece)
    {
        return (k >> 5) * 192 + piece * 64 + (k & 31) * 2;
    }

    // out[n][m in pieces] for the first `rows` n and `cols` m (a multiple of 32).
    __device__ __forceinline__ void store_by_column(const Tile<4, 4>& x, uint16_t* out, uint64_t ld, uint32_t rows,
                                                    uint32_t cols) const
    {
        constexpr uint32_t kRow = 256 * 6 + 16;  // the 16 keep the rows of a write off each other's banks
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            __syncthreads();
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int j = half * 2 + jj;
                __builtin_amdgcn_sched_barrier(0);  // bounds the registers in use
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    char* row = lds + (wn * 32 + jj * 16 + (lane & 15)) * kRow;
                    const f32x4 v = x.v[i][j];
                    uint32_t p01[3], p23[3];
                    split_pair(v[0], v[1], p01);
                    split_pair(v[2], v[3], p23);
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        *reinterpret_cast<u32x2*>(row + byte_of(wm * 64 + i * 16 + quad * 4, k)) = u32x2{p01[k], p23[k]};
                }
            }
            __syncthreads();
            copy_rows<96, kRow>(out, ld, n_base + half * 32, 64, rows, m_base * 3, cols * 3);
        }
    }

    // out[m][n in pieces]; neighbouring columns are exchanged as in Staging.
    __device__ __forceinline__ void store_by_row(const Tile<4, 4>& x, const float (&factor)[4], uint16_t* out,
                                                 uint64_t ld, uint32_t rows, uint32_t cols) const
    {
        constexpr uint32_t kRow = 128 * 6 + 16;
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4, odd = lane & 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int ii = 0; ii < 2; ++ii) {
                    const int i = half * 2 + ii;
                    char* row = lds + (wm * 32 + ii * 16 + quad * 4 + odd * 2) * kRow;
                    const f32x4 v = x.v[i][j] * factor[j];
                    uint32_t p01[3], p23[3];
                    split_pair(v[0], v[1], p01);
                    split_pair(v[2], v[3], p23);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const uint32_t give = odd ? p01[k] : p23[k], keep = odd ? p23[k] : p01[k];
                        const uint32_t got = __builtin_amdgcn_mov_dpp(give, 0xB1, 0xF, 0xF, true);  // lane ^ 1
                        const uint32_t lo = odd ? got : keep, hi = odd ? keep : got;
                        const uint32_t at = byte_of(wn * 64 + j * 16 + (lane & 14), k);
                        *reinterpret_cast<uint32_t*>(row + at) = __builtin_amdgcn_perm(hi, lo, 0x05040100);
                        *reinterpret_cast<uint32_t*>(row + kRow + at) = __builtin_amdgcn_perm(hi, lo, 0x07060302);
                    }
                }
            }
            __syncthreads();
            copy_rows<48, kRow>(out, ld, m_base + half * 32, 128, rows, n_base * 3, cols * 3);
        }
    }

private:
    template <uint32_t CHUNKS, uint32_t ROW>
    __device__ __forceinline__ void copy_rows(uint16_t* out, uint64_t ld, uint32_t row0, uint32_t high, uint32_t rows,
                                              uint32_t col0, uint32_t cols) const
    {
#pragma unroll 4
        for (uint32_t i = threadIdx.x; i < high * CHUNKS; i += 512) {
            const uint32_t r = i / CHUNKS, c = i % CHUNKS;
            const u32x4 v = *reinterpret_cast<const u32x4*>(lds + r * ROW + c * 16);
            const uint32_t to = row0 + r / 32 * 64 + r % 32;
            if (to < rows && col0 + c * 8 < cols)
                *reinterpret_cast<u32x4*>(out + static_cast<uint64_t>(to) * ld + col0 + c * 8) = v;
        }
    }
};

// gemm_large's scheme on 256 x 128 x 32 tiles of three pieces, 8 waves of 64 x
// 64: 48 matrix instructions a half step. 1021 x 32003 x 770 fp32 in 214 us: 1.48
// PFLOP/s of bf16 products with the padding, where a library fp32 product of
// the size takes 379. g.k, g.k_all: depths; lda,
// ldb: six bytes for each of the padded depth.
template <class Epilogue>
__global__ __launch_bounds__(512, 2) void gemm_pieces(const GemmArgs g, const Epilogue epi)
{
    using T = MmaBF16;
    constexpr uint32_t kStage = 73728, kA1 = 24576, kB = 49152;
    __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
    uint32_t tm, tn, split;
    tile_of_workgroup(g, &tm, &tn, &split);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = wave >> 1, wn = wave & 1;
    const uint32_t m_base = tm * 256, n_base = tn * kPiecesN;
    const uint32_t k0 = split * g.k;
    const uint32_t depth = k0 < g.k_all ? min(g.k, g.k_all - k0) : 0;
    const uint32_t steps = depth / kPieceDepth;

    // A load takes 128 rows of one piece: the first or the last 32 of each
    // wave's 64 rows of A, or the rows of B. 64-byte rows of four 16-byte
    // columns; column c of row r lies at c ^ (r / 2 & 3).
    const uint32_t row = tid >> 2, col = (tid & 3) ^ ((row >> 1) & 3);
    const uint32_t off_a = ((row >> 5) * 64 + (row & 31)) * static_cast<uint32_t>(g.lda) + col * 16;
    const uint32_t off_b = row * static_cast<uint32_t>(g.ldb) + col * 16;
    auto rows_from = [&](const char* p, uint64_t ld, uint32_t r0, uint32_t rows) {
        const uint32_t left = rows > r0 ? min(rows - r0, 256u) : 0;
        return __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(p + static_cast<uint64_t>(k0) * (kPieces * 2) + static_cast<uint64_t>(r0) * ld), 0,
            static_cast<int>(left * static_cast<uint32_t>(ld)), 0x00020000);
    };
    const __amdgpu_buffer_rsrc_t ra0 = rows_from(g.a, g.lda, m_base, g.m), ra1 = rows_from(g.a, g.lda, m_base + 32, g.m);
    const __amdgpu_buffer_rsrc_t rb = rows_from(g.b, g.ldb, n_base, g.n);
    auto fetch = [&](__amdgpu_buffer_rsrc_t x, uint32_t to, uint32_t off, uint32_t step) {
        const uint32_t v = step < steps ? off : kPastEnd, at = step * (kPieceDepth * kPieces * 2);
        char* p = lds + to + wave * 1024;
        load_to_lds(x, p, v, at);
        load_to_lds(x, p + 8192, v, at + 64);
        load_to_lds(x, p + 16384, v, at + 128);
    };

    Tile<4, 4> acc;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc.v[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    i32x4 fa0[2][3], fa1[2][3], fb[4][3];
    auto multiply = [&](i32x4 (&f)[2][3], int i0) {
        constexpr int kOfA[6] = {2, 1, 0, 1, 0, 0}, kOfB[6] = {0, 1, 2, 0, 1, 0};
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int k = 0; k < 6; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc.v[i0 + i][j] = T::mma(__builtin_bit_cast(T::Frag, f[i][kOfA[k]]),
                                              __builtin_bit_cast(T::Frag, fb[j][kOfB[k]]), acc.v[i0 + i][j]);
        __builtin_amdgcn_s_setprio(0);
    };

    if (steps) {
        const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
        const uint32_t frow = lane & 15, fcol = lane >> 4;
        const uint32_t swizzled = (fcol ^ ((frow >> 1) & 3)) * 16;
        uint32_t pa = base + (wm * 32 + frow) * 64 + swizzled, pa_next = pa + kStage;
        uint32_t pb = base + kB + (wn * 64 + frow) * 64 + swizzled, pb_next = pb + kStage;
        fetch(ra0, 0, off_a, 0);
        fetch(rb, kB, off_b, 0);
        fetch(ra1, kA1, off_a, 0);
        fetch(ra0, kStage, off_a, 1);
        fetch(rb, kStage + kB, off_b, 1);
        arrive<9>();
        read_pieces<0, 0>(fa0[0], fa0[1], fa1[0], fa1[1], pa, pa);
        meet();  // the first quarter is read: step 0 loads it again
        if (wave >= 4) meet();
        uint32_t stage = 0, other = kStage;
        for (uint32_t k = 0; k < steps; ++k) {
            fetch(ra1, other + kA1, off_a, k + 1);
            fetch(ra0, stage, off_a, k + 2);
            read_pieces<0, 2048>(fb[0], fb[1], fb[2], fb[3], pb, pb);
            arrive<9>();
            multiply(fa0, 0);
            meet();
            fetch(rb, stage + kB, off_b, k + 2);
            read_pieces<kA1, 0>(fa1[0], fa1[1], fa0[0], fa0[1], pa, pa_next);
            arrive<9>();
            multiply(fa1, 2);
            meet();
            uint32_t t = pa; pa = pa_next; pa_next = t;
            t = pb; pb = pb_next; pb_next = t;
            t = stage; stage = other; other = t;
        }
        if (wave < 4) meet();
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }
    epi(acc, m_base + wm * 64, n_base + wn * 64, g, tm * 4 + wm, split, PieceStaging{lds, wm, wn, m_base, n_base});
}

template <class Epilogue>
hipError_t launch_gemm_pieces(GemmArgs g, const Epilogue& epi, hipStream_t stream)
{
    g.tiles_m = (g.m + kTileM - 1) / kTileM;
    g.tiles_n = (g.n + kPiecesN - 1) / kPiecesN;
    hipLaunchKernelGGL((gemm_pieces<Epilogue>), dim3(g.tiles_m * g.tiles_n * g.splits), dim3(512), 0, stream, g, epi);
    return hipGetLastError();
}

template <class T, int BN, class Epilogue>
hipError_t launch_gemm_few(GemmArgs g, const Epilogue& epi, hipStream_t stream)
{
    g.tiles_m = (g.m + kFewM - 1) / kFewM;
    g.tiles_n = (g.n + BN - 1) / BN;
    hipLaunchKernelGGL((gemm_few<T, BN, Epilogue>), dim3(g.tiles_m * g.tiles_n * g.splits), dim3(FewShape<BN>::kThreads),
                       0, stream, g, epi);
    return hipGetLastError();
}

template <class T, class Epilogue>
hipError_t launch_gemm_large(GemmArgs g, const Epilogue& epi, hipStream_t stream)
{
    g.tiles_m = (g.m + kTileM - 1) / kTileM;
    g.tiles_n = (g.n + 255) / 256;
    hipLaunchKernelGGL((gemm_large<T, Epilogue>), dim3(g.tiles_m * g.tiles_n * g.splits), dim3(512), 0, stream, g, epi);
    return hipGetLastError();
}

}  // namespace lm
}  // namespace ar
