// orthogonalize.hip -- matrices made nearly orthogonal by Newton-Schulz products,
// alone and as the update of a step with momentum.
//
//   X = U / max(|U|, eps),  then `steps` times  X <- (a I + b A + c A A) X,  A = X X^T
//
// on the smaller side (m rows of n, m <= n), which leaves each singular value s
// as p(p(..p(s))), p(s) = a s + b s^3 + c s^5. The bracket is built without a sum
// of matrices: with D = A + (b / 2c) I it is c D D + (a - b^2 / 4c) I, so both
// products change a diagonal only.
//
// Small singular values grow by a factor of a in each step (485 in five of them),
// and what a rounding adds to X grows alike: in bf16, results are off by 4-30%, in
// fp16 by up to 6% of their norm's largest element. X, D and the bracket are held as two
// fp16 numbers each (gemm_halves.h), 22 bits, whose results are those of fp32
// products.
//
// Products want both operands contiguous along the sum: A = X X^T takes X by
// rows, the last one X by columns, so X is written in both orders. The smaller
// side's products are symmetric: their tiles below the diagonal are written
// twice.
#include <algorithm>

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
// Pointers of a group of matrices.
struct GroupIn {
    const void* in[kMostGroup];             // or gradients
    const float* momentum_in[kMostGroup];
    float* momentum_out[kMostGroup];
    uint64_t rows, cols, ld_in, ld_momentum;
    float decay, rest;  // rest = 1 - decay
    int nesterov;
};

// Eight elements of a row of U, from column c on: the matrix itself, or the
// momentum's update, FIRST: which is also stored.
template <class F, bool MUON, bool VEC>
struct Source {
    using Raw = RawOf<F>;
    static constexpr int A = VEC ? 16 : sizeof(Raw), AM = VEC ? 16 : 4;

    template <bool FIRST>
    static __device__ __forceinline__ void get(const GroupIn& p, uint32_t matrix, uint64_t row, uint64_t c, float (&u)[8])
    {
        const uint64_t left = p.cols - c;
        Raw raw[8];
        get8<Raw, A>(p.in[matrix], row * p.ld_in + c, left, raw);
        widen4<F>(raw, u);
        widen4<F>(raw + 4, u + 4);
        if constexpr (MUON) {
            float m[8];
            const uint64_t at = row * p.ld_momentum + c;
            get8<float, AM>(FIRST ? p.momentum_in[matrix] : p.momentum_out[matrix], at, left, m);
            if constexpr (FIRST) {
#pragma unroll
                for (int i = 0; i < 8; ++i) m[i] = p.decay * m[i] + p.rest * u[i];
                float* to = p.momentum_out[matrix] + at;
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

// partial[matrix][block] = its part of the sum of squares, in fp64: neither
// squares beyond fp32's range nor small elements are lost.
template <class F, bool MUON, bool VEC>
__global__ __launch_bounds__(kBlock) void measure_matrices(const GroupIn p, int lanes, double* partial)
{
    __shared__ double waves[kBlock / 64];
    const uint32_t per = kBlock / lanes;
    double sum = 0.0;
    for (uint64_t r = static_cast<uint64_t>(blockIdx.x) * per + threadIdx.x / lanes; r < p.rows;
         r += static_cast<uint64_t>(gridDim.x) * per)
        for (uint64_t c = (threadIdx.x & (lanes - 1)) * 8ull; c < p.cols; c += lanes * 8ull) {
            float u[8];
            Source<F, MUON, VEC>::template get<true>(p, blockIdx.y, r, c, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += static_cast<double>(u[i]) * u[i];
        }
    sum = block_sum<kBlock>(sum, waves);
    if (threadIdx.x == 0) partial[static_cast<uint64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = sum;
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

// X in pieces, in the given order and transposed, zeros up to whole steps of
// the depth. 64 x 64 tiles through LDS, as pack_transposed.
template <class F, bool MUON, bool VEC>
__global__ __launch_bounds__(kBlock) void lay_out_matrices(const GroupIn p, const double* partial, int parts, double eps,
                                                           char* straight, uint64_t batch_s, char* turned,
                                                           uint64_t batch_t)
{
    __shared__ float tile[64][65];
    __shared__ double waves[kBlock / 64];
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += kBlock) sum += partial[static_cast<uint64_t>(blockIdx.y) * parts + i];
    const double norm = sqrt(block_sum<kBlock>(sum, waves));
    const float factor = static_cast<float>(kHalvesScale / (norm < eps ? eps : norm));
    straight += blockIdx.y * batch_s;
    turned += blockIdx.y * batch_t;
    const uint64_t pad_r = (p.rows + 31) / 32 * 32, pad_c = (p.cols + 31) / 32 * 32;
    const uint32_t high = static_cast<uint32_t>((p.rows + 63) / 64);
    const uint64_t r0 = static_cast<uint64_t>(blockIdx.x % high) * 64, c0 = static_cast<uint64_t>(blockIdx.x / high) * 64;
    const int slot = threadIdx.x & 7;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = i * 32 + (threadIdx.x >> 3);
        const uint64_t r = r0 + row, c = c0 + slot * 8;
        float x[8] = {};
        if (r < p.rows && c < p.cols) Source<F, MUON, VEC>::template get<false>(p, blockIdx.y, r, c, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] *= factor;
            tile[row][slot * 8 + k] = x[k];
        }
        if (r < p.rows && c < pad_c) put_halves(straight + r * halves_bytes(pad_c), static_cast<uint32_t>(c), x);
    }
    __syncthreads();
    if (r0 + slot * 8 >= pad_r) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = i * 32 + (threadIdx.x >> 3);
        if (c0 + c >= p.cols) continue;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = tile[slot * 8 + k][c];
        put_halves(turned + (c0 + c) * halves_bytes(pad_r), static_cast<uint32_t>(r0 + slot * 8), x);
    }
}

// ---------------------------------------------------------------------------
// epilogues
// ---------------------------------------------------------------------------
// out = factor C + shift I for the symmetric product C.
struct SymmetricEpilogue {
    char* out;
    uint64_t batch;
    uint32_t ld, pad;  // bytes, elements
    float factor, shift;

    template <int N, class S>
    __device__ __forceinline__ void operator()(Tile<N, N>& acc, uint32_t m0, uint32_t n0, const HalvesArgs& g,
                                               uint32_t matrix, const S& stage, uint32_t tm, uint32_t tn) const
    {
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t row = m0 + i * 16 + quad * 4 + r, col = n0 + j * 16 + (lane & 15);
                    acc.v[i][j][r] = factor * acc.v[i][j][r] + (row == col && row < g.m ? shift : 0.0f);
                }
        char* to = out + matrix * batch;
        stage.store_by_column(acc, to, ld, g.n, pad);
        if (tm != tn) stage.store_by_row(acc, to, ld, g.m, pad);
    }
};

// X of the next step, by rows and by columns.
struct NextEpilogue {
    char* rows;     // [m][n]
    char* columns;  // [n][m]
    uint64_t batch_r, batch_c;
    uint32_t pad_n, pad_m;

    template <int N, class S>
    __device__ __forceinline__ void operator()(Tile<N, N>& acc, uint32_t, uint32_t, const HalvesArgs& g, uint32_t matrix,
                                               const S& stage, uint32_t, uint32_t) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) acc.v[i][j] *= 1.0f / kHalvesScale;
        stage.store_by_column(acc, columns + matrix * batch_c, halves_bytes(pad_m), g.n, pad_m);
        stage.store_by_row(acc, rows + matrix * batch_r, halves_bytes(pad_n), g.m, pad_n);
    }
};

// The result: C[m][n] is out[n][m], four neighbours of a row in a lane.
template <class F>
struct ResultEpilogue {
    void* out[kMostGroup];
    uint64_t ld;
    int vec;

    template <int N, class S>
    __device__ __forceinline__ void operator()(Tile<N, N>& acc, uint32_t m0, uint32_t n0, const HalvesArgs& g,
                                               uint32_t matrix, const S&, uint32_t, uint32_t) const
    {
        each_four(acc, m0, n0, g, [&](uint32_t row, uint32_t col, float (&x)[4], uint32_t left) {
            put(out[matrix], row * ld + col, x, left, vec);
        });
    }

    // fn(row, column, four results, how many of them there are)
    template <int N, class Fn>
    static __device__ __forceinline__ void each_four(const Tile<N, N>& acc, uint32_t m0, uint32_t n0, const HalvesArgs& g,
                                                     Fn fn)
    {
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t row = n0 + j * 16 + (lane & 15);
            if (row >= g.n) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t col = m0 + i * 16 + quad * 4;
                if (col >= g.m) continue;
                float x[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = acc.v[i][j][r] * kHalvesUnit;
                fn(row, col, x, g.m - col);
            }
        }
    }
    static __device__ __forceinline__ void put(void* out, uint64_t at, const float (&x)[4], uint32_t left, int vec)
    {
        if (vec && left >= 4) {
            if constexpr (F::kEpv == 8) *reinterpret_cast<u32x2*>(static_cast<char*>(out) + at * 2) = F::pack4(x);
            else *reinterpret_cast<u32x4*>(static_cast<char*>(out) + at * 4) = F::pack(x);
        } else {
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r)
                if (r < left) F::st(out, at + r, x[r]);
        }
    }
};

// weights_out = keep weights_in - gain O, to every rank.
template <class F>
struct UpdateEpilogue {
    const void* in[kMostGroup];
    void* out[kMostGroupOut];  // [matrix][rank]
    uint64_t ld;
    int nranks, vec;
    float keep, gain;

    template <int N, class S>
    __device__ __forceinline__ void operator()(Tile<N, N>& acc, uint32_t m0, uint32_t n0, const HalvesArgs& g,
                                               uint32_t matrix, const S&, uint32_t, uint32_t) const
    {
        using R = ResultEpilogue<F>;
        using Raw = RawOf<F>;
        const void* from = in[matrix];
        R::each_four(acc, m0, n0, g, [&](uint32_t row, uint32_t col, float (&x)[4], uint32_t left) {
            const uint64_t at = row * ld + col;
            Raw w[4] = {};
            if (vec && left >= 4) {
                using Unit = typename std::conditional<sizeof(Raw) == 2, u32x2, u32x4>::type;
                const Unit v = *reinterpret_cast<const Unit*>(static_cast<const char*>(from) + at * sizeof(Raw));
                __builtin_memcpy(w, &v, sizeof(w));
            } else {
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r)
                    if (r < left) w[r] = static_cast<const Raw*>(from)[at + r];
            }
            float old[4];
            widen4<F>(w, old);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = __builtin_fmaf(-gain, x[r], old[r] * keep);
            for (int k = 0; k < nranks; ++k) R::put(out[matrix * nranks + k], at, x, left, vec);
        });
    }
};

// ---------------------------------------------------------------------------
// one call
// ---------------------------------------------------------------------------
constexpr uint64_t kCUs = 256;

struct Layout {
    uint64_t m, n, pad_m, pad_n;
    uint64_t rows, columns, square;  // bytes of X by rows, by columns, of D
    int parts;                       // of a matrix's sum of squares
    uint64_t per_matrix;             // bytes of all
};
Layout layout_of(uint64_t rows, uint64_t cols)
{
    Layout l;
    l.m = std::min(rows, cols);
    l.n = std::max(rows, cols);
    l.pad_m = round_up(l.m, kHalvesDepth);
    l.pad_n = round_up(l.n, kHalvesDepth);
    l.rows = round_up(l.m * halves_bytes(l.pad_n), 256);
    l.columns = round_up(l.n * halves_bytes(l.pad_m), 256);
    l.square = round_up(l.m * halves_bytes(l.pad_m), 256);
    l.parts = static_cast<int>(std::min<uint64_t>((rows * cols + kBlock * 32 - 1) / (kBlock * 32), 256));
    l.per_matrix = l.rows + 2 * l.columns + 2 * l.square + round_up(l.parts * sizeof(double), 256);
    return l;
}

// Matrices of a group: as many as their pointers fit kernel arguments, and about
// kGroupBytes of workspace; a matrix beyond that fills the chip alone.
constexpr uint64_t kGroupBytes = uint64_t(4) << 30;
uint64_t group_of(uint64_t count, const Layout& l, int nranks)
{
    const uint64_t most = std::min<uint64_t>(kMostGroup, kMostGroupOut / std::max(nranks, 1));
    return std::max<uint64_t>(1, std::min({count, most, kGroupBytes / l.per_matrix}));
}

template <class Epilogue>
hipError_t launch_halves(HalvesArgs g, uint64_t matrices, int tile, const Epilogue& epi, hipStream_t s)
{
    const uint32_t b = static_cast<uint32_t>(tile);
    g.tiles_m = (g.m + b - 1) / b;
    g.tiles_n = (g.n + b - 1) / b;
    g.per_matrix = g.symmetric ? g.tiles_m * (g.tiles_m + 1) / 2 : g.tiles_m * g.tiles_n;
    const dim3 grid(static_cast<uint32_t>(g.per_matrix * matrices));
    if (tile == 128) hipLaunchKernelGGL((gemm_halves<128, Epilogue>), grid, dim3(256), 0, s, g, epi);
    else hipLaunchKernelGGL((gemm_halves<64, Epilogue>), grid, dim3(256), 0, s, g, epi);
    return hipGetLastError();
}

// Tiles of 64 where those of 128 leave CUs idle.
int tile_of(uint64_t m, uint64_t n, uint64_t matrices, bool symmetric)
{
    const uint64_t tm = (m + 127) / 128, tn = (n + 127) / 128;
    return matrices * (symmetric ? tm * (tm + 1) / 2 : tm * tn) >= kCUs ? 128 : 64;
}

struct Group {
    const OrthogonalizeArgs& a;
    const Layout& l;
    uint64_t first, count;
    char* ws;
    hipStream_t s;

    HalvesArgs product(const char* x, uint64_t batch_x, uint64_t rows_x, const char* y, uint64_t batch_y, uint64_t rows_y,
                       uint64_t depth, bool symmetric) const
    {
        HalvesArgs g{};
        g.a = x;
        g.b = y;
        g.batch_a = batch_x;
        g.batch_b = batch_y;
        g.lda = g.ldb = static_cast<uint32_t>(halves_bytes(depth));
        g.m = static_cast<uint32_t>(rows_x);
        g.n = static_cast<uint32_t>(rows_y);
        g.steps = static_cast<uint32_t>(depth / kHalvesDepth);
        g.symmetric = symmetric;
        return g;
    }

    template <class F>
    hipError_t prepare(double* partial, char* straight, uint64_t batch_s, char* turned, uint64_t batch_t) const
    {
        GroupIn p{};
        uintptr_t mis = a.ld_in * sizeof(RawOf<F>);
        if (a.momentum_in) mis |= a.ld_momentum * 4;
        for (uint64_t i = 0; i < count; ++i) {
            p.in[i] = a.in[first + i];
            mis |= reinterpret_cast<uintptr_t>(p.in[i]);
            if (!a.momentum_in) continue;
            p.momentum_in[i] = a.momentum_in[first + i];
            p.momentum_out[i] = a.momentum_out[first + i];
            mis |= reinterpret_cast<uintptr_t>(p.momentum_in[i]) | reinterpret_cast<uintptr_t>(p.momentum_out[i]);
        }
        p.rows = a.rows;
        p.cols = a.cols;
        p.ld_in = a.ld_in;
        p.ld_momentum = a.ld_momentum;
        p.decay = static_cast<float>(a.decay);
        p.rest = static_cast<float>(1.0 - a.decay);
        p.nesterov = a.nesterov;
        const int lanes = lanes_for((a.cols + 7) / 8);
        const uint64_t tiles = ((a.rows + 63) / 64) * ((a.cols + 63) / 64);
        auto launch = [&](auto measure, auto lay_out) {
            const uint32_t y = static_cast<uint32_t>(count);
            hipLaunchKernelGGL(measure, dim3(l.parts, y), dim3(kBlock), 0, s, p, lanes, partial);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL(lay_out, dim3(static_cast<uint32_t>(tiles), y), dim3(kBlock), 0, s, p, partial, l.parts, a.eps,
                               straight, batch_s, turned, batch_t);
            return hipGetLastError();
        };
        const bool vec = mis % 16 == 0;
        if (a.momentum_in)
            return vec ? launch(measure_matrices<F, true, true>, lay_out_matrices<F, true, true>)
                       : launch(measure_matrices<F, true, false>, lay_out_matrices<F, true, false>);
        return vec ? launch(measure_matrices<F, false, true>, lay_out_matrices<F, false, true>)
                   : launch(measure_matrices<F, false, false>, lay_out_matrices<F, false, false>);
    }

    template <class F>
    hipError_t finish(const HalvesArgs& g, int tile) const
    {
        constexpr uint64_t e = sizeof(RawOf<F>);
        uintptr_t mis = a.ld_out * e;
        if (!a.weights_in) {
            ResultEpilogue<F> epi{};
            for (uint64_t i = 0; i < count; ++i) {
                epi.out[i] = a.out[first + i];
                mis |= reinterpret_cast<uintptr_t>(epi.out[i]);
            }
            epi.ld = a.ld_out;
            epi.vec = mis % (4 * e) == 0;
            return launch_halves(g, count, tile, epi, s);
        }
        UpdateEpilogue<F> epi{};
        for (uint64_t i = 0; i < count; ++i) {
            epi.in[i] = a.weights_in[first + i];
            mis |= reinterpret_cast<uintptr_t>(epi.in[i]);
            for (int r = 0; r < a.nranks; ++r) {
                void* out = a.out[(first + i) * a.nranks + r];
                epi.out[i * a.nranks + r] = out;
                mis |= reinterpret_cast<uintptr_t>(out);
            }
        }
        epi.ld = a.ld_out;
        epi.nranks = a.nranks;
        epi.vec = mis % (4 * e) == 0;
        epi.keep = static_cast<float>(1.0 - a.lr * a.weight_decay);
        epi.gain = static_cast<float>(a.lr * a.update_scale);
        return launch_halves(g, count, tile, epi, s);
    }

    hipError_t run() const
    {
        char* at = ws;
        auto take = [&](uint64_t bytes) {
            char* here = at;
            at += bytes * count;
            return here;
        };
        char* x = take(l.rows);
        char* xt[2] = {take(l.columns), take(l.columns)};
        char *d = take(l.square), *q = take(l.square);
        double* partial = reinterpret_cast<double*>(take(round_up(l.parts * sizeof(double), 256)));
        const bool tall = a.rows > a.cols;
        char *straight = tall ? xt[0] : x, *turned = tall ? x : xt[0];
        const uint64_t batch_s = tall ? l.columns : l.rows, batch_t = tall ? l.rows : l.columns;
        hipError_t e;
        switch (a.dtype) {
        case AR_FLOAT32: e = prepare<F32>(partial, straight, batch_s, turned, batch_t); break;
        case AR_FLOAT16: e = prepare<F16>(partial, straight, batch_s, turned, batch_t); break;
        case AR_BFLOAT16: e = prepare<BF16>(partial, straight, batch_s, turned, batch_t); break;
        default: return hipErrorInvalidValue;
        }
        if (e != hipSuccess) return e;
        const int square_tile = tile_of(l.m, l.m, count, true), wide_tile = tile_of(l.m, l.n, count, false);
        const uint32_t ld_square = static_cast<uint32_t>(halves_bytes(l.pad_m)), pad_m = static_cast<uint32_t>(l.pad_m);
        for (int step = 0; step < a.steps; ++step) {
            const double ca = a.coefficients[3 * step], cb = a.coefficients[3 * step + 1], cc = a.coefficients[3 * step + 2];
            // operands are held times 2^11, products times 2^22
            auto symmetric = [&](char* out, double factor, double shift) {
                return SymmetricEpilogue{out, l.square, ld_square, pad_m, static_cast<float>(factor / kHalvesScale),
                                         static_cast<float>(shift * kHalvesScale)};
            };
            const HalvesArgs xx = product(x, l.rows, l.m, x, l.rows, l.m, l.pad_n, true);
            if (cc != 0.0) {
                if ((e = launch_halves(xx, count, square_tile, symmetric(d, 1.0, cb / (2.0 * cc)), s)) != hipSuccess) return e;
                e = launch_halves(product(d, l.square, l.m, d, l.square, l.m, l.pad_m, true), count, square_tile,
                                  symmetric(q, cc, ca - cb * cb / (4.0 * cc)), s);
            } else {
                e = launch_halves(xx, count, square_tile, symmetric(q, cb, ca), s);
            }
            if (e != hipSuccess) return e;
            if (step + 1 < a.steps) {
                const NextEpilogue next{x, xt[(step + 1) & 1], l.rows, l.columns, static_cast<uint32_t>(l.pad_n), pad_m};
                e = launch_halves(product(q, l.square, l.m, xt[step & 1], l.columns, l.n, l.pad_m, false), count, wide_tile,
                                  next, s);
                if (e != hipSuccess) return e;
            }
        }
        // four neighbours of a row of the result lie in a lane
        char* last = xt[(a.steps - 1) & 1];
        const HalvesArgs g = tall ? product(q, l.square, l.m, last, l.columns, l.n, l.pad_m, false)
                                  : product(last, l.columns, l.n, q, l.square, l.m, l.pad_m, false);
        switch (a.out_dtype) {
        case AR_FLOAT32: return finish<F32>(g, wide_tile);
        case AR_FLOAT16: return finish<F16>(g, wide_tile);
        case AR_BFLOAT16: return finish<BF16>(g, wide_tile);
        default: return hipErrorInvalidValue;
        }
    }
};

}  // namespace

uint64_t orthogonalize_bytes(uint64_t count, uint64_t rows, uint64_t cols)
{
    if (count == 0 || rows == 0 || cols == 0) return 0;
    const Layout l = layout_of(rows, cols);
    return group_of(count, l, 1) * l.per_matrix;
}

hipError_t launch_orthogonalize(const OrthogonalizeArgs& a, char* ws, hipStream_t stream)
{
    const Layout l = layout_of(a.rows, a.cols);
    const uint64_t most = group_of(a.count, l, a.nranks);
    for (uint64_t first = 0; first < a.count; first += most) {
        const hipError_t e = Group{a, l, first, std::min(most, a.count - first), ws, stream}.run();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lm
}  // namespace ar
