// orthogonalize_small.hip -- matrices that fit one workgroup's LDS, in one launch.
//
// A launch for each of the 15 products of five steps takes 4 us whatever its
// size. Here a workgroup has a matrix for itself: X by rows and by columns, D and
// the bracket lie in LDS as pairs of fp16 numbers, the sum of squares is its own,
// and barriers part the products. Whatever fits is faster so than by launches: 4 x 64 x
// 192 fp32 in 38 us rather than 72, 16 x 16 in 13 rather than 66, 96 x 96 in 42 rather
// than 83, 1024 x 64 x 192 in 0.5 ms rather than 2.8.
#include <cmath>

#include "orthogonalize.h"

namespace ar {
namespace lm {

namespace {

constexpr int kThreads = 512, kWaves = 8;
constexpr uint32_t kLds = 160 * 1024 - 1024;
constexpr int kMostUnits = 5;   // of a wave's part of X
constexpr int kMostEights = 5;  // of a thread's part of U

// Rows of pairs, 16 bytes more than whole 128s, so that 16 rows spread over all
// banks.
__host__ __device__ constexpr uint32_t pitch_of(uint32_t depth) { return depth * 4 + 16; }

struct SmallShape {
    uint32_t m, n;      // m <= n, up to whole 32s
    uint32_t x, xt, d, q, bytes;  // offsets
};
__host__ __device__ inline SmallShape small_shape(uint64_t rows, uint64_t cols)
{
    SmallShape s{};
    const uint64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    s.m = static_cast<uint32_t>((m + 31) / 32 * 32);
    s.n = static_cast<uint32_t>((n + 31) / 32 * 32);
    s.xt = s.m * pitch_of(s.n);
    s.d = s.xt + s.n * pitch_of(s.m);
    s.q = s.d + s.m * pitch_of(s.m);
    s.bytes = s.q + s.m * pitch_of(s.m);
    return s;
}

// What a workgroup of the launch has: pointers of matrix i from i * stride on: in,
// momentum_in, momentum_out, weights_in, out[ranks], or in and out alone.
constexpr int kMostPointers = 400;
struct SmallArgs {
    void* pointers[kMostPointers];
    SourceShape shape;
    uint64_t ld_out;
    int stride, nranks, steps;
    float keep, gain;  // of the update
    double eps;
    // of each step: D = A + shift_d I (if there is one), the bracket = c D D + shift_q I or c A + shift_q I
    struct Step {
        float c, shift_d, shift_q;
        int square;
    } step[16];
};

__device__ __forceinline__ uint32_t this_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// A unit: 16 rows of A by 32 of B, `steps` of the depth.
__device__ __forceinline__ void multiply_unit(const char* a, uint32_t pitch_a, const char* b, uint32_t pitch_b,
                                              uint32_t steps, f32x4 (&acc)[2])
{
    const uint32_t lane = threadIdx.x & 63, row = lane & 15, col = (lane >> 4) * 16;
    a += row * pitch_a + col;
    b += row * pitch_b + col;
    acc[0] = acc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    // (the next step's fragments are read before this one's are multiplied)
    struct Fragments {
        f16x8 x[2], y[2][2];
    };
    auto read = [&](Fragments& f, uint32_t k) {
        const uint32_t at = min(k, steps - 1) * 128;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            f.x[p] = *reinterpret_cast<const f16x8*>(a + at + p * 64);
#pragma unroll
            for (int j = 0; j < 2; ++j) f.y[j][p] = *reinterpret_cast<const f16x8*>(b + at + j * 16 * pitch_b + p * 64);
        }
    };
    auto multiply = [&](const Fragments& f) {
        constexpr int kOfA[3] = {0, 1, 0}, kOfB[3] = {1, 0, 0};  // the smaller products first
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[j] = MmaF16::mma(f.x[kOfA[p]], f.y[j][kOfB[p]], acc[j]);
    };
    Fragments f, g;
    read(f, 0);
    uint32_t k = 0;
#pragma unroll 1
    for (; k + 2 <= steps; k += 2) {
        read(g, k + 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(f);
        read(f, k + 2);
        __builtin_amdgcn_sched_barrier(0);
        multiply(g);
    }
    if (k < steps) multiply(f);
}

// out = factor A B^T + shift I for symmetric results of s.m rows, whose [n][m]
// is as good as their [m][n].
__device__ __forceinline__ void symmetric(const char* a, uint32_t pitch, uint32_t depth, char* out, const SmallShape& s,
                                          uint32_t m_true, float factor, float shift)
{
    const uint32_t lane = threadIdx.x & 63, quad = lane >> 4, wave = this_wave();
    const uint32_t across = s.m / 32, units = s.m / 16 * across, pitch_out = pitch_of(s.m);
    for (uint32_t u = wave; u < units; u += kWaves) {
        const uint32_t m0 = u / across * 16, n0 = u % across * 32;
        f32x4 acc[2];
        multiply_unit(a + m0 * pitch, pitch, a + n0 * pitch, pitch, depth / 32, acc);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t row = n0 + j * 16 + (lane & 15), k = m0 + quad * 4;
            float v[4];
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r) v[r] = factor * acc[j][r] + (k + r == row && row < m_true ? shift : 0.0f);
            uint32_t h0, h1, l0, l1;
            split_halves(v[0], v[1], &h0, &l0);
            split_halves(v[2], v[3], &h1, &l1);
            char* at = out + row * pitch_out;
            *reinterpret_cast<u32x2*>(at + halves_at(k, 0)) = u32x2{h0, h1};
            *reinterpret_cast<u32x2*>(at + halves_at(k, 1)) = u32x2{l0, l1};
        }
    }
}

// The results of a wave's units, or the weights by them, whose loads all come
// first: behind a store each would be waited for by itself.
template <class W, bool MUON>
__device__ __forceinline__ void finish(const SmallArgs& p, void* const* mine, const f32x4 (&acc)[kMostUnits][2],
                                       const SmallShape& s, uint32_t m_true, uint32_t n_true, bool tall)
{
    const uint32_t lane = threadIdx.x & 63, quad = lane >> 4, wave = this_wave(), across = s.n / 32;
    auto each = [&](auto fn) {
#pragma unroll
        for (int i = 0; i < kMostUnits; ++i) {
            const uint32_t unit = wave + i * kWaves;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) {
                    const uint32_t m = unit / across * 16 + quad * 4 + r, n = unit % across * 32 + j * 16 + (lane & 15);
                    if (m < m_true && n < n_true) fn(i, j, r, tall ? n * p.ld_out + m : m * p.ld_out + n);
                }
        }
    };
    float w[kMostUnits][2][4];
    if constexpr (MUON) each([&](int i, int j, uint32_t r, uint64_t at) { w[i][j][r] = W::ld(mine[3], at); });
    each([&](int i, int j, uint32_t r, uint64_t at) {
        const float o = acc[i][j][r] * kHalvesUnit;
        if constexpr (MUON) {
            const float x = __builtin_fmaf(-p.gain, o, w[i][j][r] * p.keep);
            for (int rank = 0; rank < p.nranks; ++rank) W::st(mine[4 + rank], at, x);
        } else {
            W::st(mine[1], at, o);
        }
    });
}

template <class F, class W, bool MUON>
__global__ __launch_bounds__(kThreads) void orthogonalize_small(const SmallArgs p)
{
    __shared__ __attribute__((aligned(16))) char lds[kLds];
    __shared__ double waves[kWaves];
    const SmallShape s = small_shape(p.shape.rows, p.shape.cols);
    const bool tall = p.shape.rows > p.shape.cols;
    const uint32_t rows = static_cast<uint32_t>(p.shape.rows), cols = static_cast<uint32_t>(p.shape.cols);
    const uint32_t m_true = min(rows, cols), n_true = max(rows, cols);
    const int tid = threadIdx.x;
    const uint32_t lane = tid & 63, quad = lane >> 4, wave = this_wave();
    void* const* mine = p.pointers + blockIdx.x * p.stride;
    SourcePointers src{mine[0], nullptr, nullptr};
    if constexpr (MUON) {
        src.momentum_in = static_cast<const float*>(mine[1]);
        src.momentum_out = static_cast<float*>(mine[2]);
    }

    // U in registers, its squares, then X in both orders with zeros around it.
    // Neighbouring lanes have neighbouring rows: with neighbouring columns their
    // transposed stores met in two banks, 50 us rather than 38 at 32 x 544.
    const uint32_t eights = (cols + 7) / 8, count = rows * eights;
    float u[kMostEights][8];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kMostEights; ++i) {
        const uint32_t at = tid + i * kThreads;
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] = 0.0f;
        if (at < count) Source<F, MUON, false>::template get<true>(p.shape, src, at % rows, at / rows * 8, u[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += static_cast<double>(u[i][e]) * u[i][e];
    }
    for (uint32_t i = tid; i < s.d / 16; i += kThreads) reinterpret_cast<u32x4*>(lds)[i] = u32x4{0, 0, 0, 0};
    const double norm = sqrt(block_sum<kThreads>(sum, waves));  // (its barrier is the zeros')
    const float scale = static_cast<float>(kHalvesScale / (norm < p.eps ? p.eps : norm));
    char *x = lds, *xt = lds + s.xt, *d = lds + s.d, *q = lds + s.q;
    const uint32_t pitch_x = pitch_of(s.n), pitch_m = pitch_of(s.m);
#pragma unroll
    for (int i = 0; i < kMostEights; ++i) {
        const uint32_t item = tid + i * kThreads;
        if (item >= count) continue;
        const uint32_t r = item % rows, c = item / rows * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] *= scale;
        put_halves(tall ? xt + r * pitch_m : x + r * pitch_x, c, u[i]);  // (up to 7 zeros behind the row, within its pad)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (c + e >= cols) continue;
            uint32_t hi, lo;
            split_halves(u[i][e], 0.0f, &hi, &lo);
            char* at = tall ? x + (c + e) * pitch_x : xt + (c + e) * pitch_m;
            *reinterpret_cast<uint16_t*>(at + halves_at(r, 0)) = static_cast<uint16_t>(hi);
            *reinterpret_cast<uint16_t*>(at + halves_at(r, 1)) = static_cast<uint16_t>(lo);
        }
    }
    __syncthreads();

    for (int step = 0; step < p.steps; ++step) {
        // (hidden from the compiler, which would keep every unit's addresses over all steps)
        uint32_t across = s.n / 32;
        asm volatile("" : "+s"(across));
        const uint32_t units = s.m / 16 * across;
        const SmallArgs::Step st = p.step[step];
        if (st.square) {
            symmetric(x, pitch_x, s.n, d, s, m_true, 1.0f / kHalvesScale, st.shift_d);
            __syncthreads();
            symmetric(d, pitch_m, s.m, q, s, m_true, st.c, st.shift_q);
        } else {
            symmetric(x, pitch_x, s.n, q, s, m_true, st.c, st.shift_q);
        }
        __syncthreads();
        f32x4 acc[kMostUnits][2];
#pragma unroll
        for (int i = 0; i < kMostUnits; ++i) {
            const uint32_t unit = wave + i * kWaves;
            if (unit < units)
                multiply_unit(q + unit / across * 16 * pitch_m, pitch_m, xt + unit % across * 32 * pitch_m, pitch_m,
                              s.m / 32, acc[i]);
        }
        if (step + 1 == p.steps) {
            finish<W, MUON>(p, mine, acc, s, m_true, n_true, tall);
            return;
        }
        __syncthreads();  // X is read
#pragma unroll
        for (int i = 0; i < kMostUnits; ++i) {
            const uint32_t unit = wave + i * kWaves;
            if (unit >= units) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t k = unit / across * 16 + quad * 4, n = unit % across * 32 + j * 16 + (lane & 15);
                const f32x4 v = acc[i][j] * (1.0f / kHalvesScale);
                uint32_t p01[2], p23[2];
                split_halves(v[0], v[1], &p01[0], &p01[1]);
                split_halves(v[2], v[3], &p23[0], &p23[1]);
                // by rows a lane takes two columns of two rows from its neighbour and itself
                const uint32_t odd = lane & 1;
                char *by_column = xt + n * pitch_m, *by_row = x + (k + odd * 2) * pitch_x;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    *reinterpret_cast<u32x2*>(by_column + halves_at(k, e)) = u32x2{p01[e], p23[e]};
                    const uint32_t give = odd ? p01[e] : p23[e], keep = odd ? p23[e] : p01[e];
                    const uint32_t got = __builtin_amdgcn_mov_dpp(give, 0xB1, 0xF, 0xF, true);  // lane ^ 1
                    const uint32_t left = odd ? got : keep, right = odd ? keep : got;
                    const uint32_t at = halves_at(n & ~1u, e);
                    *reinterpret_cast<uint32_t*>(by_row + at) = __builtin_amdgcn_perm(right, left, 0x05040100);
                    *reinterpret_cast<uint32_t*>(by_row + pitch_x + at) = __builtin_amdgcn_perm(right, left, 0x07060302);
                }
            }
        }
        __syncthreads();
    }
}

template <class F, class W, bool MUON>
hipError_t launch(const SmallArgs& p, uint32_t matrices, hipStream_t s)
{
    hipLaunchKernelGGL((orthogonalize_small<F, W, MUON>), dim3(matrices), dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

template <class F>
hipError_t by_result(const OrthogonalizeArgs& a, const SmallArgs& p, uint32_t matrices, hipStream_t s)
{
    if (!a.weights_in) return launch<F, F, false>(p, matrices, s);
    return a.out_dtype == a.dtype ? launch<F, F, true>(p, matrices, s) : launch<F, F32, true>(p, matrices, s);
}

}  // namespace

bool is_small(uint64_t rows, uint64_t cols, int steps)
{
    if (rows > 4096 || cols > 4096 || steps > 16) return false;
    const SmallShape s = small_shape(rows, cols);
    return s.bytes <= kLds && s.m / 16 * (s.n / 32) <= kMostUnits * kWaves &&
           rows * ((cols + 7) / 8) <= static_cast<uint64_t>(kMostEights) * kThreads;
}

hipError_t launch_orthogonalize_small(const OrthogonalizeArgs& a, hipStream_t stream)
{
    SmallArgs p{};
    p.shape = source_shape(a);
    p.ld_out = a.ld_out;
    p.nranks = a.nranks;
    p.steps = a.steps;
    p.keep = static_cast<float>(1.0 - a.lr * a.weight_decay);
    p.gain = static_cast<float>(a.lr * a.update_scale);
    p.eps = a.eps;
    for (int i = 0; i < a.steps; ++i) {
        const double ca = a.coefficients[3 * i], cb = a.coefficients[3 * i + 1], cc = a.coefficients[3 * i + 2];
        const bool square = cc != 0.0;
        p.step[i] = {static_cast<float>((square ? cc : cb) / kHalvesScale),
                     static_cast<float>(square ? cb / (2.0 * cc) * kHalvesScale : 0.0),
                     static_cast<float>((square ? ca - cb * cb / (4.0 * cc) : ca) * kHalvesScale), square};
    }
    p.stride = a.weights_in ? 4 + a.nranks : 2;
    const uint64_t most = static_cast<uint64_t>(kMostPointers / p.stride);
    for (uint64_t first = 0; first < a.count; first += most) {
        const uint64_t count = a.count - first < most ? a.count - first : most;
        for (uint64_t i = 0; i < count; ++i) {
            void** to = p.pointers + i * p.stride;
            *to++ = const_cast<void*>(a.in[first + i]);
            if (a.weights_in) {
                *to++ = const_cast<float*>(a.momentum_in[first + i]);
                *to++ = a.momentum_out[first + i];
                *to++ = const_cast<void*>(a.weights_in[first + i]);
            }
            for (int r = 0; r < a.nranks; ++r) *to++ = a.out[(first + i) * a.nranks + r];
        }
        hipError_t e;
        switch (a.dtype) {
        case AR_FLOAT32: e = by_result<F32>(a, p, static_cast<uint32_t>(count), stream); break;
        case AR_FLOAT16: e = by_result<F16>(a, p, static_cast<uint32_t>(count), stream); break;
        case AR_BFLOAT16: e = by_result<BF16>(a, p, static_cast<uint32_t>(count), stream); break;
        default: return hipErrorInvalidValue;
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lm
}  // namespace ar
