// orthogonalize.hip -- matrices made nearly orthogonal by Newton-Schulz products,
// alone and as the update of a step with momentum.
//
//   X = U / max(|U|, eps),  then `steps` times  X <- (a I + b A + c A A) X,  A = X X^T
//
// on the smaller side (m rows of n, m <= n), which leaves each singular value s
// as p(p(..p(s))), p(s) = a s + b s^3 + c s^5. The bracket Q is built without a sum
// of matrices: with D = A + (b / 2c) I it is c D D + (a - b^2 / 4c) I, so both
// products change a diagonal only.
//
// Where the matrix is clearly wider than high, X is left alone for up to three
// steps: the next A is Q A Q, since all of these are polynomials of A, and the
// steps' brackets are multiplied into P, by which X is multiplied at the end.
// These products are of the smaller side alone and symmetric: a segment of k
// steps costs m^2 (n + (4k - 3) m + 2n) products (of half of a symmetric result)
// where steps by themselves take k m^2 (3n + m). Errors of A for small singular
// values grow with a^2 a step there, in X with a, which bounds a segment's length
// (segment_size): the default's five steps mostly go as three and two.
//
// Small singular values grow by a factor of a in each step (485 in five of them),
// and what a rounding adds to X grows alike: in bf16, results are off by 4-30%, in
// fp16 by up to 6% of their norm's largest element. X, D and the bracket are held as two
// fp16 numbers each (gemm_halves.h), 22 bits, whose results are off by as much as those
// of fp32 products, up to four times that, or by about 1e-6 of the result.
//
// Products want both operands contiguous along the sum: A = X X^T takes X by
// rows, the last one X by columns, so X is written in both orders. The smaller
// side's products are symmetric: their tiles below the diagonal are written
// twice.
#include <algorithm>
#include <cmath>
#include <vector>

#include "orthogonalize.h"

namespace ar {
namespace lm {

namespace {

// Pointers of a group of matrices.
struct GroupIn {
    const void* in[kMostGroup];             // or gradients
    const float* momentum_in[kMostGroup];
    float* momentum_out[kMostGroup];
    SourceShape shape;

    __device__ __forceinline__ SourcePointers of(uint32_t matrix) const
    {
        return SourcePointers{in[matrix], momentum_in[matrix], momentum_out[matrix]};
    }
};

// partial[matrix][block] = its part of the sum of squares, in fp64: neither
// squares beyond fp32's range nor small elements are lost.
template <class F, bool MUON, bool VEC>
__global__ __launch_bounds__(kBlock) void measure_matrices(const GroupIn p, int lanes, double* partial)
{
    __shared__ double waves[kBlock / 64];
    const uint32_t per = kBlock / lanes;
    double sum = 0.0;
    for (uint64_t r = static_cast<uint64_t>(blockIdx.x) * per + threadIdx.x / lanes; r < p.shape.rows;
         r += static_cast<uint64_t>(gridDim.x) * per)
        for (uint64_t c = (threadIdx.x & (lanes - 1)) * 8ull; c < p.shape.cols; c += lanes * 8ull) {
            float u[8];
            Source<F, MUON, VEC>::template get<true>(p.shape, p.of(blockIdx.y), r, c, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += static_cast<double>(u[i]) * u[i];
        }
    sum = block_sum<kBlock>(sum, waves);
    if (threadIdx.x == 0) partial[static_cast<uint64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = sum;
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
    const uint64_t pad_r = (p.shape.rows + 31) / 32 * 32, pad_c = (p.shape.cols + 31) / 32 * 32;
    const uint32_t high = static_cast<uint32_t>((p.shape.rows + 63) / 64);
    const uint64_t r0 = static_cast<uint64_t>(blockIdx.x % high) * 64, c0 = static_cast<uint64_t>(blockIdx.x / high) * 64;
    const int slot = threadIdx.x & 7;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = i * 32 + (threadIdx.x >> 3);
        const uint64_t r = r0 + row, c = c0 + slot * 8;
        float x[8] = {};
        if (r < p.shape.rows && c < p.shape.cols) Source<F, MUON, VEC>::template get<false>(p.shape, p.of(blockIdx.y), r, c, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] *= factor;
            tile[row][slot * 8 + k] = x[k];
        }
        if (r < p.shape.rows && c < pad_c) put_halves(straight + r * halves_bytes(pad_c), static_cast<uint32_t>(c), x);
    }
    __syncthreads();
    if (r0 + slot * 8 >= pad_r) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = i * 32 + (threadIdx.x >> 3);
        if (c0 + c >= p.shape.cols) continue;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = tile[slot * 8 + k][c];
        put_halves(turned + (c0 + c) * halves_bytes(pad_r), static_cast<uint32_t>(r0 + slot * 8), x);
    }
}

// ---------------------------------------------------------------------------
// epilogues
// ---------------------------------------------------------------------------
// factor C + shift I of the symmetric product C, and of that again, if there
// are two to be written.
struct SymmetricEpilogue {
    char* out[2];  // the first may be null
    uint64_t batch;
    uint32_t ld, pad;  // bytes, elements
    float factor[2], shift[2];

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const HalvesArgs& g,
                                               uint32_t matrix, const S& stage, uint32_t tm, uint32_t tn) const
    {
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!out[k]) continue;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc.v[i][j][r] *= factor[k];
            if (tm == tn && shift[k] != 0.0f) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t row = m0 + i * 16 + quad * 4 + r, col = n0 + j * 16 + (lane & 15);
                            acc.v[i][j][r] += row == col && row < g.m ? shift[k] : 0.0f;
                        }
            }
            char* to = out[k] + matrix * batch;
            stage.store_by_column(acc, to, ld, g.n, pad);
            if (tm != tn) stage.store_by_row(acc, to, ld, g.m, pad);
        }
    }
};

// X of the next step, by rows and by columns.
struct NextEpilogue {
    char* rows;     // [m][n]
    char* columns;  // [n][m]
    uint64_t batch_r, batch_c;
    uint32_t pad_n, pad_m;
    float factor;

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& acc, uint32_t, uint32_t, const HalvesArgs& g, uint32_t matrix,
                                               const S& stage, uint32_t, uint32_t) const
    {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc.v[i][j] *= factor;
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
    float unit;

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const HalvesArgs& g,
                                               uint32_t matrix, const S&, uint32_t, uint32_t) const
    {
        each_four(acc, m0, n0, g, unit, [&](uint32_t row, uint32_t col, float (&x)[4], uint32_t left) {
            put(out[matrix], row * ld + col, x, left, vec);
        });
    }

    // fn(row, column, four results, how many of them there are)
    template <int MT, int NT, class Fn>
    static __device__ __forceinline__ void each_four(const Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const HalvesArgs& g,
                                                     float unit, Fn fn)
    {
        const uint32_t lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t row = n0 + j * 16 + (lane & 15);
            if (row >= g.n) continue;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t col = m0 + i * 16 + quad * 4;
                if (col >= g.m) continue;
                float x[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = acc.v[i][j][r] * unit;
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
    float keep, gain, unit;

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const HalvesArgs& g,
                                               uint32_t matrix, const S&, uint32_t, uint32_t) const
    {
        using R = ResultEpilogue<F>;
        using Raw = RawOf<F>;
        const void* from = in[matrix];
        R::each_four(acc, m0, n0, g, unit, [&](uint32_t row, uint32_t col, float (&x)[4], uint32_t left) {
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
constexpr uint32_t kCUs = 256;
constexpr int kSegment = 3;  // steps
constexpr double kMostTop = 4.0;
constexpr double kLateGrowth = 16.0, kAnyGrowth = 4.0;  // of errors of A in one

// How a product goes through its tiles: of which size, and in how many parts
// those behind the last full round of workgroups are split.
struct Tiling {
    int tile;
    uint32_t splits;  // 1: none
    double cost;      // microseconds
};
constexpr uint32_t kLeastSteps = 16;  // of a split sum
constexpr uint64_t kPartialBytes = uint64_t(2 * kCUs) * 128 * 128 * 4;

// Microseconds that fit the products measured, to within a fifth: a step of 32 with
// all slots taken (two workgroups a CU; one of 256), with half of them, and what a
// full round and a last one cost beside their steps. The same product 400 times on
// end, 4096 x 8192 x 4096: 530 us in tiles of 256, 615 of 128, 893 of 64; 8 symmetric
// 1024 x 1024 x 1024: 58, 37 and 39. The parts of split tiles are joined by a launch of
// its own: symmetric 4096 x 4096 x 4096, 16 tiles of 128 behind a round of 512, 230 us
// whole, 177 in four parts, 175 in twelve, 193 in 32. Boxes differ by a tenth and more
// (271, 204, 208 and 263 on another), and between a call's other products, at the
// power limit, the first takes 635 and the last 192 + 16 for the join; the forms' order
// is the same.
struct TileCost {
    int tile;
    uint32_t slots;
    double full, half, round, last, join;
};
constexpr TileCost kTileCosts[] = {{64, 2 * kCUs, 0.45, 0.27, 2.0, 3.0, 0.25},
                                   {128, 2 * kCUs, 1.2, 0.75, 11.0, 4.5, 0.9},
                                   {256, kCUs, 1.9, 1.55, 17.0, 7.0, 0.0}};

uint64_t tiles_of(uint64_t m, uint64_t n, uint64_t matrices, bool symmetric, int tile)
{
    const uint64_t tm = (m + tile - 1) / tile, tn = (n + tile - 1) / tile;
    return matrices * (symmetric ? tm * (tm + 1) / 2 : tm * tn);
}

Tiling tiling_of(uint64_t m, uint64_t n, uint64_t depth, uint64_t matrices, bool symmetric)
{
    Tiling best{64, 1, 0.0};
    const double steps = static_cast<double>(depth / kHalvesDepth);
    for (const TileCost& c : kTileCosts) {
        if (symmetric && c.tile == 256) continue;
        const uint64_t tiles = tiles_of(m, n, matrices, symmetric, c.tile), rounds = tiles / c.slots, rest = tiles % c.slots;
        for (uint32_t splits : {1u, 2u, 3u, 4u, 6u, 8u, 12u, 16u}) {
            if (splits > 1 && (rest == 0 || rest * splits > c.slots || depth < kLeastSteps * kHalvesDepth || c.tile == 256))
                break;
            double t = rounds * (steps * c.full + c.round);
            if (rest) {
                // workgroups end one by one: the last ones start early
                const double each = std::ceil(steps / splits) * (2 * rest * splits > c.slots ? c.full : c.half);
                t += c.last + each * (rounds ? 0.65 : 1.0) + (splits > 1 ? 5.0 + splits * c.join : 0.0);
            }
            if (best.cost == 0.0 || t < best.cost) best = Tiling{c.tile, splits, t};
        }
    }
    return best;
}

struct Layout {
    uint64_t m, n, pad_m, pad_n;
    uint64_t rows, columns, square;  // bytes of X by rows, by columns, of D
    int parts;                       // of a matrix's sum of squares
    bool segments;                   // the way the steps go
    int squares;                     // matrices of the smaller side
    uint64_t per_matrix;             // bytes of all
};

// Whether steps go in segments: products of the smaller side alone, 14 in five
// steps beside two of each with the larger one, or five of each kind; what a
// launch costs beside its product decides for small ones. By steps / in segments,
// us: 3 x 1027 x 770 281 / 291, 4 x 64 x 192 72 / 82, 2 x 2100 x 1030 464 / 410, 5 x 770
// x 3000 603 / 454, 4096 x 8192 5470 / 4490, 8 x 2048 x 4096 6060 / 5080.
bool in_segments(uint64_t m, uint64_t n, uint64_t count)
{
    constexpr double kLaunch = 2.0;
    const double gram = tiling_of(m, m, round_up(n, kHalvesDepth), count, true).cost + kLaunch,
                 square = tiling_of(m, m, round_up(m, kHalvesDepth), count, true).cost + kLaunch,
                 wide = tiling_of(m, n, round_up(m, kHalvesDepth), count, false).cost + kLaunch;
    return 2 * gram + 14 * square + 2 * wide < 5 * (gram + square + wide);
}
Layout layout_of(uint64_t rows, uint64_t cols, uint64_t count)
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
    l.segments = in_segments(l.m, l.n, std::min<uint64_t>(count, kMostGroup));
    l.squares = l.segments ? 7 : 2;
    l.per_matrix = l.rows + 2 * l.columns + l.squares * l.square + round_up(l.parts * sizeof(double), 256);
    return l;
}

// Whether a product may be deep enough for parts.
bool may_split(const Layout& l) { return l.pad_n >= kLeastSteps * kHalvesDepth; }

// Matrices of a group: as many as their pointers fit kernel arguments, and about
// kGroupBytes of workspace; a matrix beyond that fills the chip alone.
constexpr uint64_t kGroupBytes = uint64_t(4) << 30;
uint64_t group_of(uint64_t count, const Layout& l, int nranks)
{
    const uint64_t most = std::min<uint64_t>(kMostGroup, kMostGroupOut / std::max(nranks, 1));
    return std::max<uint64_t>(1, std::min({count, most, kGroupBytes / l.per_matrix}));
}

template <int B, class Epilogue>
hipError_t launch_tiles(HalvesArgs g, uint64_t matrices, uint32_t splits, const Epilogue& epi, hipStream_t s)
{
    g.tiles_m = (g.m + B - 1) / B;
    g.tiles_n = (g.n + B - 1) / B;
    g.per_matrix = g.symmetric ? g.tiles_m * (g.tiles_m + 1) / 2 : g.tiles_m * g.tiles_n;
    const uint32_t tiles = static_cast<uint32_t>(g.per_matrix * matrices);
    g.splits = splits;
    g.whole = splits > 1 ? tiles - tiles % (2 * kCUs) : tiles;
    hipLaunchKernelGGL((gemm_halves<B, false, Epilogue>), dim3(g.whole + (tiles - g.whole) * splits),
                       dim3(HalvesShape<B>::kThreads), 0, s, g, epi);
    hipError_t e = hipGetLastError();
    if constexpr (B < 256) {
        if (e == hipSuccess && g.whole < tiles) {
            hipLaunchKernelGGL((gemm_halves<B, true, Epilogue>), dim3(tiles - g.whole), dim3(HalvesShape<B>::kThreads), 0, s,
                               g, epi);
            e = hipGetLastError();
        }
    }
    return e;
}

template <class Epilogue>
hipError_t launch_halves(const HalvesArgs& g, uint64_t matrices, const Epilogue& epi, hipStream_t s)
{
    const Tiling t = tiling_of(g.m, g.n, static_cast<uint64_t>(g.steps) * kHalvesDepth, matrices, g.symmetric);
    if constexpr (!std::is_same<Epilogue, SymmetricEpilogue>::value) {
        if (t.tile == 256) return launch_tiles<256>(g, matrices, 1, epi, s);
    }
    return t.tile == 128 ? launch_tiles<128>(g, matrices, t.splits, epi, s)
                         : launch_tiles<64>(g, matrices, t.splits, epi, s);
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
        g.partial = sums();
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
        p.shape = source_shape(a);
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
    hipError_t finish(const HalvesArgs& g, float unit) const
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
            epi.unit = unit;
            epi.vec = mis % (4 * e) == 0;
            return launch_halves(g, count, epi, s);
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
        epi.unit = unit;
        return launch_halves(g, count, epi, s);
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
        char* square[7] = {};
        for (int i = 0; i < l.squares; ++i) square[i] = take(l.square);
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
        const std::vector<StepBounds> bounds = l.segments ? bounds_of_steps() : std::vector<StepBounds>();
        int turn = 0;  // which of xt holds X
        for (int k = 0; k < a.steps;) {
            const int size = l.segments ? segment_size(k, bounds) : 1;
            const char* p;
            double p_scale;
            if ((e = segment(x, square, k, size, bounds, &p, &p_scale)) != hipSuccess) return e;
            k += size;
            const float unit = static_cast<float>(1.0 / p_scale);  // X keeps its 2^11
            if (k == a.steps) {
                // four neighbours of a row of the result lie in a lane
                const HalvesArgs g = tall ? product(p, l.square, l.m, xt[turn], l.columns, l.n, l.pad_m, false)
                                          : product(xt[turn], l.columns, l.n, p, l.square, l.m, l.pad_m, false);
                const float out_unit = unit / kHalvesScale;
                switch (a.out_dtype) {
                case AR_FLOAT32: return finish<F32>(g, out_unit);
                case AR_FLOAT16: return finish<F16>(g, out_unit);
                case AR_BFLOAT16: return finish<BF16>(g, out_unit);
                default: return hipErrorInvalidValue;
                }
            }
            const NextEpilogue next{x, xt[turn ^ 1], l.rows, l.columns, static_cast<uint32_t>(l.pad_n),
                                    static_cast<uint32_t>(l.pad_m), unit};
            e = launch_halves(product(p, l.square, l.m, xt[turn], l.columns, l.n, l.pad_m, false), count, next, s);
            if (e != hipSuccess) return e;
            turn ^= 1;
        }
        return hipSuccess;  // not reached: there is at least one step
    }

    // What a step makes of singular values of up to 1 before the first.
    struct StepBounds {
        double bracket;  // of the bracket's eigenvalues
        double top;      // of the singular values after it; infinite from where they pass kMostTop
    };
    std::vector<StepBounds> bounds_of_steps() const
    {
        std::vector<StepBounds> all;
        double top = 1.0;
        for (int k = 0; k < a.steps; ++k) {
            const double ca = a.coefficients[3 * k], cb = a.coefficients[3 * k + 1], cc = a.coefficients[3 * k + 2];
            double bracket = 0.0, next = 0.0;
            for (int j = 0; j <= 1000 && top <= kMostTop; ++j) {
                const double v = top * j / 1000.0, u = std::fabs(ca + cb * v * v + cc * v * v * v * v);
                bracket = std::max(bracket, u);
                next = std::max(next, u * v);
            }
            top = top <= kMostTop && next * 1.001 <= kMostTop ? next * 1.001 : INFINITY;
            all.push_back({std::max(bracket * 1.001, 1e-3), top});
        }
        return all;
    }

    // The steps of the segment that starts with step k, up to three. In a segment an
    // error of A grows with a^2 a step but for the last, whose bracket takes it over.
    // The rounding of X at the segment's start, which steps by themselves have too,
    // grows with a in every step to come: the former may grow no more than that. In the
    // first segment A is known to little more than its largest singular values' part,
    // whose rounding weighs the more the fewer rows there are: growth up to half of that
    // and m / 2. In later ones A has the size 1 whatever the matrix was: up to
    // kLateGrowth, and half of what singular values have grown so far. (Up to kAnyGrowth
    // is no matter.)
    // Largest errors of 30 kinds of singular values as multiples of those of fp32
    // products (where either is above 1e-6 of the result), 5 of 770 x 3000, in segments
    // of three whatever the growth / so / by steps: 3 steps of the default 9.8 / 2.8 / 2.6, 4
    // steps 8.0 / 1.4 / 1.7, 5 steps 2.1 / 2.1 / 1.6, 8 steps 24 / 1.6 / 1.6, 5 steps of (8.3,
    // -24, 17), (4.1, -2.9, 0.5) .. 17 / 2.4 / 1.6, the first 3 of them 53 / 2.7 / 2.7; 5
    // steps of the default of 40 x 883, simulated, 21 / 1.5 / 2.0.
    // The brackets' product is held at a scale for the largest singular values that
    // there may be; where these would pass kMostTop, which those of the matrix need not,
    // steps go by themselves.
    int segment_size(int k, const std::vector<StepBounds>& bounds) const
    {
        auto growth = [&](int from, int to) {
            double g = 1.0;
            for (int i = from; i < to; ++i) g *= std::max(1.0, std::fabs(a.coefficients[3 * i]));
            return g;
        };
        const double all = growth(k, a.steps) * 1.001;  // (equal products, in whatever order, are not more)
        const double most = std::max(kAnyGrowth, k ? std::min({all, growth(0, k) / 2, kLateGrowth})
                                                   : std::min(all, static_cast<double>(l.m)) / 2);
        int size = std::min(a.steps - k, kSegment);
        while (size > 1 && (std::pow(growth(k, k + size - 1), 2) > most || bounds[k + size - 1].top > kMostTop)) --size;
        return size;
    }

    // Steps k .. k + size - 1 of X's rows `x`: *p is the product of their brackets,
    // held times *p_scale.
    hipError_t segment(const char* x, char* const square[7], int k, int size, const std::vector<StepBounds>& bounds,
                       const char** p, double* p_scale) const
    {
        char *d = square[0], *q[2] = {square[1], square[4]}, *gram = square[2], *t = square[3], *prod[2] = {square[5], square[6]};
        hipError_t e;
        double largest = 1.0;  // of P's eigenvalues
        for (int i = 0; i < size; ++i) {
            const double ca = a.coefficients[3 * (k + i)], cb = a.coefficients[3 * (k + i) + 1],
                         cc = a.coefficients[3 * (k + i) + 2];
            char* bracket = q[i & 1];
            // A, if a later step needs it, and D (or the bracket itself of a cubic)
            SymmetricEpilogue epi = symmetric(cc != 0.0 ? d : bracket, cc != 0.0 ? 1.0 : cb, cc != 0.0 ? cb / (2.0 * cc) : ca);
            if (i + 1 < size) {
                epi.out[0] = gram;
                epi.factor[0] = 1.0f / kHalvesScale;
                epi.factor[1] *= kHalvesScale;
            }
            const HalvesArgs g = i == 0 ? product(x, l.rows, l.m, x, l.rows, l.m, l.pad_n, true)
                                        : square_product(t, q[(i - 1) & 1]);
            if ((e = launch_halves(g, count, epi, s)) != hipSuccess) return e;
            if (cc != 0.0) {
                e = launch_halves(square_product(d, d), count, symmetric(bracket, cc, ca - cb * cb / (4.0 * cc)), s);
                if (e != hipSuccess) return e;
            }
            if (size > 1) largest *= bounds[k + i].bracket;
            auto scale_of = [](double bound) { return kHalvesScale * std::exp2(-std::max(0.0, std::ceil(std::log2(bound / 8.0)))); };
            if (i == 0) {
                *p = bracket;
                *p_scale = kHalvesScale;
            } else {
                const double scale = scale_of(largest);
                char* to = prod[i & 1];
                SymmetricEpilogue join = symmetric(to, 1.0, 0.0);
                join.factor[1] = static_cast<float>(scale / (kHalvesScale * *p_scale));
                if ((e = launch_halves(square_product(bracket, *p), count, join, s)) != hipSuccess) return e;
                *p = to;
                *p_scale = scale;
            }
            if (i + 1 < size) {  // A Q, then (A Q) Q at the head of the loop
                if ((e = launch_halves(square_product(gram, bracket), count, symmetric(t, 1.0, 0.0), s)) != hipSuccess)
                    return e;
            }
        }
        return hipSuccess;
    }

    // (behind the group's matrices)
    float* sums() const { return reinterpret_cast<float*>(ws + count * l.per_matrix); }

    HalvesArgs square_product(const char* u, const char* v) const
    {
        return product(u, l.square, l.m, v, l.square, l.m, l.pad_m, true);
    }
    // Operands are held times 2^11, products times 2^22.
    SymmetricEpilogue symmetric(char* out, double factor, double shift) const
    {
        SymmetricEpilogue epi{};
        epi.out[1] = out;
        epi.batch = l.square;
        epi.ld = static_cast<uint32_t>(halves_bytes(l.pad_m));
        epi.pad = static_cast<uint32_t>(l.pad_m);
        epi.factor[1] = static_cast<float>(factor / kHalvesScale);
        epi.shift[1] = static_cast<float>(shift * kHalvesScale);
        return epi;
    }
};

}  // namespace

uint64_t orthogonalize_bytes(uint64_t count, uint64_t rows, uint64_t cols)
{
    if (count == 0 || rows == 0 || cols == 0) return 0;
    const Layout l = layout_of(rows, cols, count);
    return group_of(count, l, 1) * l.per_matrix + (may_split(l) ? kPartialBytes : 0);
}

hipError_t launch_orthogonalize(const OrthogonalizeArgs& a, char* ws, hipStream_t stream)
{
    if (is_small(a.rows, a.cols, a.steps)) return launch_orthogonalize_small(a, stream);
    const Layout l = layout_of(a.rows, a.cols, a.count);
    const uint64_t most = group_of(a.count, l, a.nranks);
    for (uint64_t first = 0; first < a.count; first += most) {
        const hipError_t e = Group{a, l, first, std::min(most, a.count - first), ws, stream}.run();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lm
}  // namespace ar
