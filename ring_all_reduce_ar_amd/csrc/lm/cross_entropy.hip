// cross_entropy.hip -- softmax cross entropy of a linear head, in pieces of
// the vocabulary, without keeping the logits; log probabilities with their
// entropy and alternatives take the same way with the epilogues of log_probs.h.
//
//   z[t][v] = x[t] . w[v],  lse[t] = log sum_v exp z[t][v],  loss[t] = lse[t] - z[t][y[t]]
//   d[t][v] = g[t] (exp(z[t][v] - lse[t]) - [v = y[t]]),  dX = d W,  dW = d^T X
//
// Forward: each tile of z leaves the maximum and the sum of exponentials of
// its part of a row; a second kernel joins them. Backward, for each piece of
// the vocabulary: z again, d from it into the workspace (rounded to the
// operands' 16 bits, for the matrix cores), and the two products. All products
// are gemm.h's, with both operands contiguous along the summed axis, so W and
// X are also laid out transposed, and d is written in both orders.
//
// fp32 operands are laid out as three bf16 pieces each: six bf16 products give
// the fp32 product to 2^-24 at 2.5 PFLOP/s / 6, where the fp32 matrix instructions
// end at 0.16. Up to 64 tokens the time is that of reading the weight, which then
// stays as it is, and so it does where there are few tiles (small_tiles).
#include <algorithm>
#include <type_traits>
#include <utility>

#include "few_gradients.h"

namespace ar {
namespace lm {

namespace {

// ---------------------------------------------------------------------------
// laying out operands
// ---------------------------------------------------------------------------
// Stores eight depths k..k+7 (k a multiple of 8) of a row: as they are, or in pieces.
template <int PARTS, class Raw>
__device__ __forceinline__ void put8(char* row, uint64_t k, const Raw (&x)[8])
{
    if constexpr (PARTS == 1) {
        u32x4 v[sizeof(x) / 16];
        __builtin_memcpy(v, x, sizeof(x));
#pragma unroll
        for (uint32_t i = 0; i < sizeof(x) / 16; ++i) *reinterpret_cast<u32x4*>(row + k * sizeof(Raw) + i * 16) = v[i];
    } else {
        uint32_t p[4][3], top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, as_u(x[i]) & 0x7FFFFFFFu);
        if (top < as_u(kCutFrom)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) split_pair(x[2 * i], x[2 * i + 1], p[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) split_pair_any(x[2 * i], x[2 * i + 1], p[i]);
        }
        char* at = row + (k / kPieceDepth) * (kPieceDepth * kPieces * 2) + k % kPieceDepth * 2;
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
            *reinterpret_cast<u32x4*>(at + q * (kPieceDepth * 2)) = u32x4{p[0][q], p[1][q], p[2][q], p[3][q]};
    }
}

// Bytes of one element of an operand.
template <int PARTS, class Raw>
constexpr uint64_t operand_bytes() { return PARTS == 1 ? sizeof(Raw) : kPieces * 2; }

// out[r] = in[r] in pieces (or as it is, on a 16-byte boundary), zeros from
// `width` up to `pad`. `lanes` (a power of two) threads a row. Bound by HBM:
// 32003 x 770 fp32 in pieces in 38 us, 6.6 TB/s.
template <int PARTS, class Raw, int A>
__global__ __launch_bounds__(kBlock) void pack_rows(const void* in, uint64_t ld, uint64_t rows, uint64_t width,
                                                    uint64_t pad, char* out, int lanes)
{
    const uint64_t r = static_cast<uint64_t>(blockIdx.x) * (kBlock / lanes) + threadIdx.x / lanes;
    if (r >= rows) return;
    for (uint64_t c = (threadIdx.x & (lanes - 1)) * 8ull; c < pad; c += lanes * 8ull) {
        Raw x[8];
        get8<Raw, A>(in, r * ld + c, c < width ? width - c : 0, x);
        put8<PARTS>(out + r * pad * operand_bytes<PARTS, Raw>(), c, x);
    }
}

// out[c] = the column c of `in` for rows below `rows`, zeros up to `pad` (a
// multiple of 8) and in rows whose target is ignored (whatever they hold).
// 64 x 64 tiles through LDS; a lane takes eight rows of one column, eight lanes
// 128 bytes of 16-bit elements. 20480 x 4096 bf16 in 55 us, 6.1 TB/s; 32003 x 770
// fp32 in pieces in 53 us, 4.7 TB/s.
template <int PARTS, class Raw, int A>
__global__ __launch_bounds__(kBlock) void pack_transposed(const void* in, uint64_t ld, uint64_t rows, uint64_t width,
                                                          uint64_t pad, char* out, Indices targets, int masked,
                                                          int64_t ignore, uint64_t vocab)
{
    __shared__ Raw tile[64][sizeof(Raw) == 2 ? 66 : 65];
    const uint32_t high = static_cast<uint32_t>((pad + 63) / 64);
    const uint64_t r0 = static_cast<uint64_t>(blockIdx.x % high) * 64, c0 = static_cast<uint64_t>(blockIdx.x / high) * 64;
    const int slot = threadIdx.x & 7;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = i * 32 + (threadIdx.x >> 3);
        const uint64_t r = r0 + row, c = c0 + slot * 8;
        Raw x[8] = {};
        if (r < rows && c < width && (!masked || load_target(targets, r, ignore, vocab) >= 0))
            get8<Raw, A>(in, r * ld + c, width - c, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) tile[row][slot * 8 + k] = x[k];
    }
    __syncthreads();
    if (r0 + slot * 8 >= pad) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = i * 32 + (threadIdx.x >> 3);
        if (c0 + c >= width) continue;
        Raw x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = tile[slot * 8 + k][c];
        put8<PARTS>(out + (c0 + c) * pad * operand_bytes<PARTS, Raw>(), r0 + slot * 8, x);
    }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
struct Stats {
    float top, sum;
};

// A wave's part of each token's row: its maximum, the sum of exponentials
// below it, and the target's logit where it falls in here.
struct StatsEpilogue {
    Stats* stats;         // [stat row][token]
    float* target_logit;  // [token]
    Indices targets;
    int64_t ignore;
    uint64_t vocab;
    uint64_t v0;          // the piece's first vocabulary row
    uint64_t row0;        // the piece's first row of `stats`

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const GemmArgs& g,
                                               uint32_t mrow, uint32_t, const S&) const
    {
        if (m0 + MT * 16 <= g.m) parts<true>(acc, m0, n0, g, mrow);
        else parts<false>(acc, m0, n0, g, mrow);
    }

private:
    // FULL: all of the wave's rows are rows of the vocabulary.
    template <bool FULL, int MT, int NT>
    __device__ __forceinline__ void parts(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const GemmArgs& g,
                                          uint32_t mrow) const
    {
        const int lane = threadIdx.x & 63, quad = lane >> 4;
        const uint32_t mine = m0 + quad * 4;  // vocabulary rows of the piece: mine + 16 i + r
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t t = n0 + j * 16 + (lane & 15);
            const bool ok = t < g.n;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (FULL || mine + 16 * i + r < g.m) top = fmaxf(top, acc.v[i][j][r]);
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float base = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (FULL || mine + 16 * i + r < g.m)
                        sum += __builtin_amdgcn_exp2f((acc.v[i][j][r] - base) * kLog2e);
            sum += __shfl_xor(sum, 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            if (ok && quad == 0) stats[(row0 + mrow) * g.n + t] = Stats{top, sum};
            const uint32_t at = ok ? target_at<MT>(load_target(targets, t, ignore, vocab), v0 + mine) : kNoTarget;
            if (!__any(at != kNoTarget)) continue;  // few tiles hold a target
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (at == static_cast<uint32_t>(16 * i + r)) target_logit[t] = acc.v[i][j][r];
        }
    }
};

// Two parts of one row's sum. A part of nothing has the top -infinity; a NaN
// stays in the sum.
__device__ __forceinline__ Stats join_parts(Stats a, Stats b)
{
    const float m = fmaxf(a.top, b.top);
    const float sum = m == -INFINITY ? a.sum + b.sum
                                     : a.sum * __builtin_amdgcn_exp2f((a.top - m) * kLog2e) +
                                           b.sum * __builtin_amdgcn_exp2f((b.top - m) * kLog2e);
    return Stats{m, sum};
}

// Joins the parts of each token's row: X tokens a workgroup, kJoinBlock / X
// threads for each. Neighbouring tokens lie side by side, so many tokens take
// 16 (128 bytes) and few tokens as few as there are, for more threads to a
// row: the loss of 3 x 65536 x 2048 fp16 takes 71 us rather than 110 with 16.
template <int X>
__global__ __launch_bounds__(kJoinBlock) void join_stats(const Stats* stats, uint64_t stat_rows,
                                                         const float* target_logit, Indices targets, int64_t ignore,
                                                         uint64_t vocab, uint64_t ntokens, float* losses, float* lse)
{
    constexpr int Y = kJoinBlock / X;
    __shared__ Stats part[Y][X];
    const int x = threadIdx.x % X, y = threadIdx.x / X;
    const uint64_t t = static_cast<uint64_t>(blockIdx.x) * X + x;
    Stats s{-INFINITY, 0.0f};
    if (t < ntokens) {
#pragma unroll 4
        for (uint64_t r = y; r < stat_rows; r += Y) s = join_parts(s, stats[r * ntokens + t]);
    }
    part[y][x] = s;
#pragma unroll
    for (int h = Y / 2; h >= 1; h /= 2) {
        __syncthreads();
        if (y < h) part[y][x] = join_parts(part[y][x], part[y + h][x]);
    }
    if (y == 0 && t < ntokens) {
        s = part[0][x];
        const float l = s.top + logf(s.sum);
        lse[t] = l;
        losses[t] = load_target(targets, t, ignore, vocab) >= 0 ? l - target_logit[t] : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(1024) void row_scale(const float* g, Indices targets, int64_t ignore, uint64_t vocab,
                                                  uint64_t ntokens, RowScale* out)
{
    __shared__ float waves[16];
    float top = 0.0f;
    for (uint64_t t = threadIdx.x; t < ntokens; t += 1024)
        if (load_target(targets, t, ignore, vocab) >= 0) top = fmaxf(top, fabsf(g[t]));
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) top = fmaxf(top, waves[w]);
        out->top = fmaxf(top, 0x1p-126f);  // whose reciprocal is finite
    }
}

// d of one piece of the vocabulary, in both orders: d[t][v] by the rule (LossD
// or LogProbD) for the hidden gradient, whose rows take g[t] at the end, and
// dt[v][t] the same times g[t] / max |g| for the weight's.
template <class T, class Rule>
struct DEpilogue {
    typename T::Elem* d;
    typename T::Elem* dt;
    Rule rule;
    const RowScale* scale;
    Indices targets;
    int64_t ignore;
    uint64_t vocab, v0, piece_pad, t_pad;
    int nt;  // d is more than the last-level cache holds

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const GemmArgs& g, uint32_t,
                                               uint32_t, const S& stage) const
    {
        const int lane = threadIdx.x & 63;
        float factor[NT];  // of a token's column of dt
        const float inv = 1.0f / scale->top;
        const uint32_t mine = m0 + (lane >> 4) * 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t t = n0 + j * 16 + (lane & 15);
            const int64_t y = t < g.n ? load_target(targets, t, ignore, vocab) : -1;
            const uint32_t at = target_at<MT>(y, v0 + mine);
            const uint32_t keep = y >= 0 ? ~0u : 0u;  // zeros for an ignored token, even from a NaN
            const typename Rule::Row row = rule.row(t, y >= 0);
            factor[j] = y >= 0 ? row.g * inv : 0.0f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc.v[i][j][r] = as_f(as_u(rule(row, acc.v[i][j][r])) & keep);
            __builtin_amdgcn_sched_barrier(0);  // bounds the registers in use
            if (__any(at != kNoTarget)) {       // few tiles hold a target
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc.v[i][j][r] += at == static_cast<uint32_t>(16 * i + r) ? rule.at_target(row) : 0.0f;
            }
            if (m0 + MT * 16 > g.m) {  // zeros below the vocabulary
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc.v[i][j][r] = mine + 16 * i + r < g.m ? acc.v[i][j][r] : 0.0f;
            }
        }
        const uint32_t cols = static_cast<uint32_t>(piece_pad), tcols = static_cast<uint32_t>(t_pad);
        if constexpr (std::is_same<S, PieceStaging>::value) {
            if (d) stage.store_by_column(acc, d, piece_pad * kPieces, g.n, cols);
            if (dt) stage.store_by_row(acc, factor, dt, t_pad * kPieces, g.m, tcols);
        } else if constexpr (S::kOn) {
            if (d) stage.template store_by_column<T>(acc, d, piece_pad, g.n, cols, nt);
            if (dt) stage.template store_by_row<T>(acc, factor, dt, t_pad, g.m, tcols, nt);
        } else {
            store(acc, factor, m0, n0, g);
        }
    }

private:
    template <int MT, int NT>
    __device__ __forceinline__ void store(const Tile<MT, NT>& acc, const float (&factor)[NT], uint32_t m0, uint32_t n0,
                                          const GemmArgs& g) const
    {
        const int lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t t = n0 + j * 16 + (lane & 15);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t v = m0 + quad * 4 + 16 * i;
                const f32x4 x = acc.v[i][j];
                if (d && t < g.n && v < piece_pad) {
                    auto* at = d + static_cast<uint64_t>(t) * piece_pad + v;
                    if constexpr (sizeof(*at) == 4) *reinterpret_cast<f32x4*>(at) = x;
                    else *reinterpret_cast<u32x2*>(at) = u32x2{T::pack2(x[0], x[1]), T::pack2(x[2], x[3])};
                }
                if (dt && t < t_pad) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (v + r < g.m) T::Format::st(dt, static_cast<uint64_t>(v + r) * t_pad + t, x[r] * factor[j]);
                }
            }
        }
    }
};

// Calls put(row, column, value) for a tile's results in C[row][column].
template <int MT, int NT, class Put>
__device__ __forceinline__ void each_result(const Tile<MT, NT>& c, uint32_t m0, uint32_t n0, const GemmArgs& g, Put put)
{
    const int lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t row = m0 + quad * 4 + 16 * i + r;
            if (row >= g.m) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t col = n0 + j * 16 + (lane & 15);
                if (col < g.n) put(row, col, c.v[i][j][r]);
            }
        }
}

// One split's sums of a gradient: acc[split][row][h]; the hidden gradient's go
// over all pieces of the vocabulary. The product's rows are the columns h, or
// (BY_ROW) the gradient's rows.
template <bool BY_ROW>
struct SumEpilogue {
    float* acc;
    uint64_t rows, width;
    int add;

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& c, uint32_t m0, uint32_t n0, const GemmArgs& g, uint32_t,
                                               uint32_t split, const S&) const
    {
        float* part = acc + split * rows * width;
        if constexpr (BY_ROW) {
            each_result(c, m0, n0, g, [&](uint32_t t, uint32_t h, float x) {
                float* at = part + t * width + h;
                *at = add ? *at + x : x;
            });
            return;
        }
        const int lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t t = n0 + j * 16 + (lane & 15);
            if (t >= g.n) continue;
            float* row = part + t * width;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t h = m0 + quad * 4 + 16 * i;
                if (width % 4 == 0) {
                    if (h < g.m) {
                        f32x4* at = reinterpret_cast<f32x4*>(row + h);
                        *at = add ? *at + c.v[i][j] : c.v[i][j];
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (h + r < g.m) row[h + r] = add ? row[h + r] + c.v[i][j][r] : c.v[i][j][r];
                }
            }
        }
    }
};

// out[row][h] = round(scale unit * the splits' sum), U elements a thread, `lanes`
// threads a row. The hidden gradient's scale is g[t], and 0 for ignored tokens;
// the weight's is max |g|. 8192 x 4096 into bf16 in 37 us, 5.4 TB/s.
template <class F, int U, bool WEIGHT>
__global__ __launch_bounds__(kBlock) void finish_sum(const float* acc, int splits, const float* g, Indices targets,
                                                     int64_t ignore, uint64_t vocab, const RowScale* top, float unit,
                                                     uint64_t rows, uint64_t width, void* out, uint64_t ld, int lanes)
{
    const uint64_t row = static_cast<uint64_t>(blockIdx.x) * (kBlock / lanes) + threadIdx.x / lanes;
    if (row >= rows) return;
    const bool on = WEIGHT || load_target(targets, row, ignore, vocab) >= 0;
    const float scale = (WEIGHT ? top->top : on ? g[row] : 0.0f) * unit;
    for (uint64_t c = (threadIdx.x & (lanes - 1)) * static_cast<uint64_t>(U); c < width;
         c += lanes * static_cast<uint64_t>(U)) {
        float s[U] = {};
#pragma unroll 8
        for (int k = 0; k < splits; ++k) {
            const float* from = acc + (static_cast<uint64_t>(k) * rows + row) * width + c;
            if constexpr (U == 1) {
                s[0] += from[0];
            } else {
#pragma unroll
                for (int u = 0; u < U; u += 4) {
                    const f32x4 v = *reinterpret_cast<const f32x4*>(from + u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u + e] += v[e];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = on ? s[u] * scale : 0.0f;
        if constexpr (U == 1) F::st(out, row * ld + c, s[0]);
        else stv_at<false>(out, (row * ld + c) * (16 / F::kEpv), F::pack(s));
    }
}

// grad_weight[v][h] = round(max |g| unit * sum). The product's rows are the
// columns h, or (BY_VOCAB) the vocabulary's.
template <class F, class T, bool BY_VOCAB>
struct WeightEpilogue {
    void* out;
    uint64_t ld;
    const RowScale* scale;
    float unit;  // the inverse of what d is held times
    int vec;  // the elements that can be stored together: 1, 4, or 8 of 16 bits
    int nt;   // the gradient is more than the last-level cache holds

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& c, uint32_t m0, uint32_t n0, const GemmArgs& g, uint32_t,
                                               uint32_t, const S& stage) const
    {
        const int lane = threadIdx.x & 63, quad = lane >> 4;
        const float s = scale->top * unit;
        if constexpr (BY_VOCAB) {
            each_result(c, m0, n0, g, [&](uint32_t v, uint32_t h, float x) { F::st(out, v * ld + h, x * s); });
            return;
        }
        if constexpr (std::is_same<S, Staging>::value) {
            if (vec == 8 && g.m % 8 == 0) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < MT; ++i) c.v[i][j] *= s;
                stage.template store_by_column<T>(c, static_cast<uint16_t*>(out), ld, g.n, g.m, nt);
                return;
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t v = n0 + j * 16 + (lane & 15);
            if (v >= g.n) continue;
            const uint64_t row = static_cast<uint64_t>(v) * ld;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t h = m0 + quad * 4 + 16 * i;
                float x[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = c.v[i][j][r] * s;
                if (vec >= 4 && h + 3 < g.m) {
                    if constexpr (F::kEpv == 8)
                        *reinterpret_cast<u32x2*>(static_cast<char*>(out) + (row + h) * 2) = F::pack4(x);
                    else
                        *reinterpret_cast<u32x4*>(static_cast<char*>(out) + (row + h) * 4) = F::pack(x);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (h + r < g.m) F::st(out, row + h + r, x[r]);
                }
            }
        }
    }
};

// ---------------------------------------------------------------------------
// one call
// ---------------------------------------------------------------------------
template <int PARTS, class Raw>
hipError_t pack(const void* in, uint64_t ld, uint64_t rows, uint64_t width, uint64_t pad, char* out, hipStream_t s)
{
    const uintptr_t mis = reinterpret_cast<uintptr_t>(in) | ld * sizeof(Raw);
    const int lanes = lanes_for(pad / 8);
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid_for(rows, lanes), dim3(kBlock), 0, s, in, ld, rows, width, pad, out, lanes);
        return hipGetLastError();
    };
    return mis % 16 == 0  ? launch(pack_rows<PARTS, Raw, 16>)
           : mis % 8 == 0 ? launch(pack_rows<PARTS, Raw, 8>)
                          : launch(pack_rows<PARTS, Raw, sizeof(Raw)>);
}

template <int PARTS, class Raw>
hipError_t transpose(const void* in, uint64_t ld, uint64_t rows, uint64_t width, uint64_t pad, char* out,
                     const CrossEntropyArgs& a, int masked, hipStream_t s)
{
    const uintptr_t mis = reinterpret_cast<uintptr_t>(in) | ld * sizeof(Raw);
    const dim3 grid(static_cast<uint32_t>((pad + 63) / 64 * ((width + 63) / 64)));
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, s, in, ld, rows, width, pad, out, a.targets, masked,
                           a.ignore_index, a.vocab);
        return hipGetLastError();
    };
    return mis % 16 == 0  ? launch(pack_transposed<PARTS, Raw, 16>)
           : mis % 8 == 0 ? launch(pack_transposed<PARTS, Raw, 8>)
                          : launch(pack_transposed<PARTS, Raw, sizeof(Raw)>);
}

template <class T, int PARTS, class Epilogue>
hipError_t product(const GemmArgs& g, int tile_n, const Epilogue& epi, hipStream_t s)
{
    if constexpr (PARTS == kPieces) {
        return launch_gemm_pieces(g, epi, s);
    } else {
        if (tile_n == 16) return launch_gemm_few<T, 16>(g, epi, s);
        if constexpr (sizeof(typename T::Elem) == 2) {
            if (tile_n == 256) return launch_gemm_large<T>(g, epi, s);
        }
        return launch_gemm_few<T, 64>(g, epi, s);
    }
}

GemmArgs swapped(GemmArgs g)
{
    std::swap(g.a, g.b);
    std::swap(g.lda, g.ldb);
    std::swap(g.m, g.n);
    return g;
}

// Whether the gradients' products have the model's columns as rows of B rather
// than of A: tiles of pieces are 256 x 128, so that a width of 770 is padded to
// 1024 as rows of A and to 896 as rows of B (1021 x 32003: 354 -> 293 and 280 ->
// 243 us).
bool columns_in_b(uint64_t width, uint64_t other)
{
    return round_up(width, kPiecesN) * round_up(other, kTileM) < round_up(width, kTileM) * round_up(other, kPiecesN);
}

// Rows of statistics that the logits of `rows` vocabulary rows leave: one for
// each wave along a tile.
uint64_t stat_rows_of(uint64_t rows, int tile_n)
{
    if (tile_n > 64) return (rows + kTileM - 1) / kTileM * (tile_n == 256 ? 2 : 4);
    return (rows + kFewM - 1) / kFewM * (tile_n == 16 ? 4 : 2);
}

// Tiles along the vocabulary that one launch takes: work-items are counted in 32 bits.
uint64_t most_tiles(uint64_t ntokens, uint64_t tile_n)
{
    const uint64_t across = (ntokens + tile_n - 1) / tile_n;
    return (uint64_t(1) << 21) / (across ? across : 1);
}

// Up to so many tokens, one for each CU, eight waves find the alternatives of one.
// Logits and alternatives by eight waves / by one, us, of 256 and of 384 tokens: 5 of
// 32000 (x 64 bf16) 27 / 25 and 34 / 27, 20 of 65536 35 / 42 and 57 / 50, 50 of 131072
// 122 / 178 and 218 / 197.
constexpr uint64_t kSelectFew = 256;

// What is larger than the last-level cache is stored around it: 8192 x 131072 x
// 4096 bf16, loss and gradients, 25.3 -> 25.0 ms.
constexpr uint64_t kStreamBytes = uint64_t(256) << 20;

// F: the storage type; T: the matrix instruction's.
template <class F, class T, int PARTS>
struct Call {
    using Raw = typename std::conditional<PARTS == 1, typename T::Elem, float>::type;  // as the caller's tensors hold it
    using Elem = typename T::Elem;
    static constexpr uint64_t EB = sizeof(Raw), OB = operand_bytes<PARTS, Raw>();
    const CrossEntropyArgs& a;
    const CrossEntropyPlan& p;
    char* ws;
    hipStream_t s;

    // Whether the logits are made from the weight's rows as they lie, though not on
    // 16 bytes. (The cross entropy lays them out: its results are as they were.)
    bool by_rows() const
    {
        return PARTS == 1 && a.log_probs && (a.losses || p.few) && p.tile_n == 16 && p.pack_weight &&
               rows_fit(a.width * EB);
    }
    template <class Epilogue>
    hipError_t few_logits(GemmArgs g, const Epilogue& epi) const
    {
        if constexpr (PARTS == 1) {
            if (!by_rows()) return launch_gemm_few<T, 16>(g, epi, s);
            g.k_all = static_cast<uint32_t>(a.width);
            return launch_gemm_rows<T>(g, epi, s);
        }
        return hipErrorInvalidValue;  // few tokens are never in pieces
    }

    // The logits' operands, packed where the plan says so, and their pitch in bytes.
    hipError_t hidden(const char** out, uint64_t* ld) const
    {
        if (!p.pack_hidden && !by_rows()) {
            *out = static_cast<const char*>(a.hidden);
            *ld = a.ld_hidden * EB;
            return hipSuccess;
        }
        *out = ws + p.hidden;
        *ld = p.k_pad * OB;
        return pack<PARTS, Raw>(a.hidden, a.ld_hidden, a.ntokens, a.width, p.k_pad, ws + p.hidden, s);
    }
    hipError_t weight(uint64_t v0, uint64_t rows, const char** out, uint64_t* ld) const
    {
        const char* from = static_cast<const char*>(a.weight) + v0 * a.ld_weight * EB;
        if (!p.pack_weight || by_rows()) {
            *out = from;
            *ld = a.ld_weight * EB;
            return hipSuccess;
        }
        *out = ws + p.weight;
        *ld = p.k_pad * OB;
        return pack<PARTS, Raw>(from, a.ld_weight, rows, a.width, p.k_pad, ws + p.weight, s);
    }
    GemmArgs logits_args(const char* w, uint64_t ldw, const char* x, uint64_t ldx, uint64_t rows, uint64_t tokens) const
    {
        GemmArgs g{};
        g.a = w;
        g.b = x;
        g.lda = ldw;
        g.ldb = ldx;
        g.m = static_cast<uint32_t>(rows);
        g.n = static_cast<uint32_t>(tokens);
        // an operand that lies as given ends at the width, then whole 16-byte columns
        g.k = g.k_all = static_cast<uint32_t>(p.pack_hidden && p.pack_weight ? p.k_pad : a.width);
        g.splits = 1;
        return g;
    }

    // A gradient's product, whose rows of A are the model's columns and which has
    // `other` rows of B, or the other way round.
    template <class ByColumn, class ByRow>
    hipError_t in_order(const GemmArgs& g, uint64_t other, int tile_n, const ByColumn& by_column,
                        const ByRow& by_row) const
    {
        if constexpr (PARTS == kPieces) {
            if (columns_in_b(a.width, other)) return product<T, PARTS>(swapped(g), tile_n, by_row, s);
        }
        return product<T, PARTS>(g, tile_n, by_column, s);
    }

    template <bool WEIGHT>
    hipError_t finish(const float* sums, int splits, const RowScale* scale, float unit, const float* row_g, uint64_t rows,
                      void* out, uint64_t ld) const
    {
        // (few results take a thread each: 6 x 256 of 64 parts in 5 us, by vectors and of 128 parts in 37)
        const bool vec = a.width % F::kEpv == 0 && ld % F::kEpv == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
                         rows * a.width >= (1u << 18);
        const int lanes = lanes_for(vec ? a.width / F::kEpv : a.width);
        auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid_for(rows, lanes), dim3(kBlock), 0, s, sums, splits, row_g, a.targets,
                               a.ignore_index, a.vocab, scale, unit, rows, a.width, out, ld, lanes);
            return hipGetLastError();
        };
        return vec ? launch(finish_sum<F, F::kEpv, WEIGHT>) : launch(finish_sum<F, 1, WEIGHT>);
    }

    hipError_t forward() const
    {
        const char *x, *w;
        uint64_t ldx, ldw, row0 = 0;
        hipError_t e = hidden(&x, &ldx);
        if (e != hipSuccess) return e;
        Stats* stats = reinterpret_cast<Stats*>(ws + p.stats);
        float* target_logit = reinterpret_cast<float*>(ws + p.target_logit);
        const uint64_t piece = p.pack_weight ? p.piece : most_tiles(a.ntokens, p.tile_n) * kTileM;  // pieces bound what is packed
        for (uint64_t v0 = 0; v0 < a.vocab; v0 += piece) {
            const uint64_t rows = a.vocab - v0 < piece ? a.vocab - v0 : piece;
            if ((e = weight(v0, rows, &w, &ldw)) != hipSuccess) return e;
            const StatsEpilogue epi{stats, target_logit, a.targets, a.ignore_index, a.vocab, v0, row0};
            if ((e = product<T, PARTS>(logits_args(w, ldw, x, ldx, rows, a.ntokens), p.tile_n, epi, s)) != hipSuccess) return e;
            row0 += stat_rows_of(rows, p.tile_n);
        }
        auto join = [&](auto kernel, uint32_t tokens) {
            hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>((a.ntokens + tokens - 1) / tokens)), dim3(kJoinBlock), 0,
                               s, stats, row0, target_logit, a.targets, a.ignore_index, a.vocab, a.ntokens, a.losses,
                               a.lse);
            return hipGetLastError();
        };
        if (a.ntokens <= 32) return join(join_stats<1>, 1);
        if (a.ntokens <= 512) return join(join_stats<4>, 4);
        return join(join_stats<16>, 16);
    }

    // The same for log probabilities, a chunk of tokens after the other where
    // their logits are kept for alternatives.
    hipError_t forward_log_probs() const
    {
        const char *x, *w;
        uint64_t ldx, ldw;
        hipError_t e = hidden(&x, &ldx);
        if (e != hipSuccess) return e;
        LogParts* parts = reinterpret_cast<LogParts*>(ws + p.stats);
        float* target_logit = reinterpret_cast<float*>(ws + p.target_logit);
        float* logits = a.top ? reinterpret_cast<float*>(ws + p.logits) : nullptr;
        const uint64_t piece = p.pack_weight && !by_rows() ? p.piece : most_tiles(p.chunk, p.tile_n) * kTileM;
        for (uint64_t t0 = 0; t0 < a.ntokens; t0 += p.chunk) {
            const uint64_t tokens = std::min(a.ntokens - t0, p.chunk);
            uint64_t row0 = 0;
            for (uint64_t v0 = 0; v0 < a.vocab; v0 += piece) {
                const uint64_t rows = std::min(a.vocab - v0, piece);
                if ((e = weight(v0, rows, &w, &ldw)) != hipSuccess) return e;
                const LogPartsEpilogue epi{parts, target_logit, logits, a.targets, a.ignore_index, a.vocab, v0, row0,
                                           t0, a.scale};
                const GemmArgs g = logits_args(w, ldw, x + t0 * ldx, ldx, rows, tokens);
                e = p.tile_n == 16 ? few_logits(g, epi) : product<T, PARTS>(g, p.tile_n, epi, s);
                if (e != hipSuccess) return e;
                row0 += stat_rows_of(rows, p.tile_n);
            }
            const LogProbOut out{a.targets, a.ignore_index, a.vocab, t0, tokens, target_logit, a.losses, a.entropy, a.lse};
            auto grid = [&](uint64_t per) { return dim3(static_cast<uint32_t>((tokens + per - 1) / per)); };
            if (a.top) {
                const uint32_t group = p.tile_n == 256 ? 128 : p.tile_n > 64 ? 64 : p.tile_n == 16 ? 16 : 32;
                auto select = [&](auto kernel, uint64_t per, uint32_t threads) {
                    hipLaunchKernelGGL(kernel, grid(per), dim3(threads), 0, s, parts, row0, logits, group, a.top, out,
                                       a.top_log_probs, a.top_ids);
                };
                if (tokens <= kSelectFew) select(select_top<8>, 1, 512);
                else select(select_top<1>, 4, 256);
            } else {
                auto join = [&](auto kernel, uint64_t per) {
                    hipLaunchKernelGGL(kernel, grid(per), dim3(kJoinBlock), 0, s, parts, row0, out);
                };
                if (tokens <= 32) join(join_log_probs<1>, 1);
                else if (tokens <= 512) join(join_log_probs<4>, 4);
                else join(join_log_probs<16>, 16);
            }
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        return hipSuccess;
    }

    hipError_t backward() const
    {
        RowScale* scale = reinterpret_cast<RowScale*>(ws + p.row_scale);
        if (a.log_probs) {
            float* rows = reinterpret_cast<float*>(ws + p.row_gradients);
            const RowGradients r{rows, rows + a.ntokens, rows + 2 * a.ntokens};
            hipLaunchKernelGGL(row_gradients, dim3(1), dim3(1024), 0, s, a.grad_losses, a.grad_entropy, a.scale, a.targets,
                               a.ignore_index, a.vocab, a.ntokens, r, scale);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            const LogProbD rule{a.lse, a.grad_entropy ? a.entropy : nullptr, r, a.scale};
            return p.few ? backward_few(rule) : backward_by(rule, 1.0f / kLogProbScale, r.g);
        }
        hipLaunchKernelGGL(row_scale, dim3(1), dim3(1024), 0, s, a.grad_losses, a.targets, a.ignore_index, a.vocab,
                           a.ntokens, scale);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        return backward_by(LossD{a.lse, a.grad_losses}, 1.0f / kDScale, a.grad_losses);
    }

    hipError_t backward_few(const LogProbD& rule) const
    {
        float* d = reinterpret_cast<float*>(ws + p.d);
        const char *x, *w;
        uint64_t ldx, ldw;
        hipError_t e = hidden(&x, &ldx);
        if (e != hipSuccess) return e;
        const uint64_t piece = p.pack_weight && !by_rows() ? p.piece : most_tiles(a.ntokens, p.tile_n) * kTileM;
        for (uint64_t v0 = 0; v0 < a.vocab; v0 += piece) {
            const uint64_t rows = std::min(a.vocab - v0, piece);
            if ((e = weight(v0, rows, &w, &ldw)) != hipSuccess) return e;
            const FewDEpilogue epi{d, rule, a.targets, a.ignore_index, a.vocab, v0};
            if ((e = few_logits(logits_args(w, ldw, x, ldx, rows, a.ntokens), epi)) != hipSuccess) return e;
        }
        FewArgs f{};
        f.weight = a.weight;
        f.hidden = a.hidden;
        f.grad_weight = a.grad_weight;
        f.partial = a.grad_hidden ? reinterpret_cast<float*>(ws + p.grad_hidden_acc) : nullptr;
        f.d = d;
        f.targets = a.targets;
        f.ignore = a.ignore_index;
        f.vocab = a.vocab;
        f.ntokens = a.ntokens;
        f.width = a.width;
        f.ld_weight = a.ld_weight;
        f.ld_hidden = a.ld_hidden;
        f.ld_grad_weight = a.ld_grad_weight;
        return launch_few_gradients<F>(f, p.splits, a.grad_hidden, a.ld_grad_hidden, s);
    }

    template <class Rule>
    hipError_t backward_by(const Rule& rule, float unit, const float* row_g) const
    {
        const char *x = nullptr, *w = nullptr;
        uint64_t ldx = 0, ldw = 0;
        hipError_t e = a.ntokens ? hidden(&x, &ldx) : hipSuccess;
        if (e != hipSuccess) return e;
        Elem* d = a.grad_hidden && a.ntokens ? reinterpret_cast<Elem*>(ws + p.d) : nullptr;
        Elem* dt = a.grad_weight ? reinterpret_cast<Elem*>(ws + p.dt) : nullptr;
        char *wt = ws + p.weight_t, *xt = ws + p.hidden_t;
        float* acc = reinterpret_cast<float*>(ws + p.grad_hidden_acc);
        const RowScale* scale = reinterpret_cast<const RowScale*>(ws + p.row_scale);
        if (dt && a.ntokens &&
            (e = transpose<PARTS, Raw>(a.hidden, a.ld_hidden, a.ntokens, a.width, p.t_pad, xt, a, 1, s)) != hipSuccess)
            return e;
        for (uint64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
            const uint64_t rows = a.vocab - v0 < p.piece ? a.vocab - v0 : p.piece;
            const uint64_t pad = round_up(rows, kTileK);
            if (a.ntokens) {  // no token: the weight's gradient is the empty sum
                if ((e = weight(v0, rows, &w, &ldw)) != hipSuccess) return e;
                const DEpilogue<T, Rule> epi{d, dt, rule, scale, a.targets, a.ignore_index, a.vocab, v0, pad, p.t_pad,
                                             a.ntokens * pad * OB > kStreamBytes};
                if ((e = product<T, PARTS>(logits_args(w, ldw, x, ldx, rows, a.ntokens), p.tile_n, epi, s)) != hipSuccess) return e;
            }
            if (d) {
                const char* from = static_cast<const char*>(a.weight) + v0 * a.ld_weight * EB;
                if ((e = transpose<PARTS, Raw>(from, a.ld_weight, rows, a.width, pad, wt, a, 0, s)) != hipSuccess) return e;
                GemmArgs g{};
                g.a = wt;
                g.b = reinterpret_cast<const char*>(d);
                g.lda = g.ldb = pad * OB;
                g.m = static_cast<uint32_t>(a.width);
                g.n = static_cast<uint32_t>(a.ntokens);
                g.k_all = static_cast<uint32_t>(pad);
                g.splits = static_cast<uint32_t>(p.splits);
                g.k = static_cast<uint32_t>(round_up((pad + p.splits - 1) / p.splits, kTileK));
                const SumEpilogue<false> by_column{acc, a.ntokens, a.width, v0 > 0};
                const SumEpilogue<true> by_token{acc, a.ntokens, a.width, v0 > 0};
                if ((e = in_order(g, a.ntokens, p.tile_n, by_column, by_token)) != hipSuccess) return e;
            }
            if (dt) {
                GemmArgs g{};
                g.a = xt;
                g.b = reinterpret_cast<const char*>(dt);
                g.lda = g.ldb = p.t_pad * OB;
                g.m = static_cast<uint32_t>(a.width);
                g.n = static_cast<uint32_t>(rows);
                g.k_all = static_cast<uint32_t>(p.t_pad);
                g.splits = static_cast<uint32_t>(p.weight_splits);
                g.k = static_cast<uint32_t>(round_up((p.t_pad + p.weight_splits - 1) / p.weight_splits, kTileK));
                char* out = static_cast<char*>(a.grad_weight) + v0 * a.ld_grad_weight * EB;
                if (p.weight_splits > 1) {
                    float* sums = reinterpret_cast<float*>(ws + p.grad_weight_acc);
                    const SumEpilogue<false> by_column{sums, rows, a.width, 0};
                    const SumEpilogue<true> by_vocab{sums, rows, a.width, 0};
                    if ((e = in_order(g, rows, 256, by_column, by_vocab)) != hipSuccess) return e;
                    if ((e = finish<true>(sums, p.weight_splits, scale, unit, row_g, rows, out, a.ld_grad_weight)) != hipSuccess) return e;
                } else {
                    const uintptr_t mis = reinterpret_cast<uintptr_t>(out) | a.ld_grad_weight * EB;
                    const int vec = EB == 2 && mis % 16 == 0 ? 8 : mis % (4 * EB) == 0 ? 4 : 1;
                    const int nt = a.vocab * a.width * EB > kStreamBytes;
                    const WeightEpilogue<F, T, false> by_column{out, a.ld_grad_weight, scale, unit, vec, nt};
                    const WeightEpilogue<F, T, true> by_vocab{out, a.ld_grad_weight, scale, unit, vec, nt};
                    if ((e = in_order(g, rows, 256, by_column, by_vocab)) != hipSuccess) return e;
                }
            }
        }
        if (d) e = finish<false>(acc, p.splits, scale, unit, row_g, a.ntokens, a.grad_hidden, a.ld_grad_hidden);
        return e;
    }
};

// What a call's products cost with pieces of `rows` rows, in depth steps of the
// busiest CU: a product takes whole rounds of one tile a CU.
constexpr uint64_t kCUs = 256;
constexpr uint64_t kMostSplits = 64;
struct Shape {
    uint64_t ntokens, width;
    uint64_t tile_m, tile_n;          // tiles of the logits' and the hidden gradient's product
    uint64_t weight_m, weight_n;      // and of the weight gradient's
    uint64_t step;
    bool pieces;
    bool log_probs;
};

uint64_t up(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// Tiles of a gradient's product with `other` rows.
uint64_t gradient_tiles(const Shape& x, uint64_t other, uint64_t tile_m, uint64_t tile_n)
{
    return x.pieces && columns_in_b(x.width, other) ? up(x.width, kPiecesN) * up(other, kTileM)
                                                    : up(x.width, tile_m) * up(other, tile_n);
}

// The best number of parts for a sum over `depth` with so many tiles, and its
// cost. A round costs about eight steps to start and to end in; parts are
// written and read again, about two steps each; `join` is the cost of a launch
// that only a split sum needs. One round of tiles of 64 rows is best too, though
// two workgroups of them fit a CU: both gradients of 16 tokens x 32000 x 2048 bf16
// take 163 us in 8 parts (256 workgroups), 181 in 4, 168 in 16, 174 in 32 and 230
// unsplit, of 64 x 32000 x 4096 333 in 4 parts, 351 in 16, 432 unsplit.
double split_cost(uint64_t tiles, uint64_t depth, uint64_t step, double join, int* splits)
{
    double best = 0;
    for (uint64_t rounds = 0; rounds <= 2; ++rounds) {  // unsplit, or parts that fill one round or two
        uint64_t k = 1;
        if (rounds) {
            k = std::min({rounds * kCUs / std::max<uint64_t>(tiles, 1), kMostSplits, depth / 128});
            if (k < 2) continue;
        }
        const double c = static_cast<double>(up(tiles * k, kCUs) * (up(up(depth, step), k) + 8)) +
                         (k > 1 ? 2.0 * k + join : 0.0);
        if (best == 0 || c < best) {
            best = c;
            *splits = static_cast<int>(k);
        }
    }
    return best;
}

// The same for the gradients of log probabilities, with any number of parts, and
// parts that cost what their `bytes` take to be written and read (and a load's
// latency, of which several are under way). Few tiles of few results take parts
// that fill no round: forward and gradients, us, by split_cost / so, of 3971 tokens x
// 1551 x 64 bf16, whose weight gradient has 7 tiles, 154 / 82, of 2877 x 624 x 326 129 / 95, of
// 600 x 8000 x 256 202 / 91, of 1021 x 32000 x 1024 fp16 341 / 341.
double parts_cost(uint64_t tiles, uint64_t depth, uint64_t step, double join, uint64_t bytes, int* splits)
{
    constexpr double kBytesAStep = 2.5e6;  // 0.85 us at 3 TB/s
    double best = 0;
    for (const uint64_t k : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
        if (k > 1 && (k > kMostSplits || tiles * k > 2 * kCUs || depth < k * 128)) break;
        const double c = static_cast<double>(up(tiles * k, kCUs) * (up(up(depth, step), k) + 8)) +
                         (k > 1 ? k * (0.25 + 2 * static_cast<double>(bytes) / kBytesAStep) + join : 0.0);
        if (best == 0 || c < best) {
            best = c;
            *splits = static_cast<int>(k);
        }
    }
    return best;
}

double piece_cost(const Shape& x, uint64_t rows, int* splits, int* weight_splits)
{
    const double logits =
        static_cast<double>(up(up(rows, x.tile_m) * up(x.ntokens, x.tile_n), kCUs) * (up(x.width, x.step) + 8));
    if (x.log_probs)
        return logits +
               parts_cost(gradient_tiles(x, x.ntokens, x.tile_m, x.tile_n), rows, x.step, 0, x.ntokens * x.width * 4, splits) +
               parts_cost(gradient_tiles(x, rows, x.weight_m, x.weight_n), x.ntokens, x.step, 8, rows * x.width * 4,
                          weight_splits) +
               24;
    return logits +
           split_cost(gradient_tiles(x, x.ntokens, x.tile_m, x.tile_n), rows, x.step, 0, splits) +
           split_cost(gradient_tiles(x, rows, x.weight_m, x.weight_n), x.ntokens, x.step, 8, weight_splits) +
           24;  // four launches
}

// Whether tiles of 64 x 64 (a few hundred of them) end sooner than the few
// large ones of the logits: a step of a 64 x 64 tile takes about 0.35 us, of
// fp32 0.45, where a step of a 256 x 256 tile takes 0.85 us and of 256 x 128
// in pieces 1.28.
bool small_tiles(uint64_t ntokens, uint64_t vocab, uint64_t width, bool f32, bool backward)
{
    if (ntokens <= 64) return true;
    auto tiles = [](uint64_t m, uint64_t n) { return up(m, 64) * up(n, 64); };
    if (tiles(vocab, ntokens) > 2 * kCUs) return false;
    return !f32 || !backward || (tiles(width, ntokens) <= 2 * kCUs && tiles(width, vocab) <= 2 * kCUs);
}

}  // namespace

namespace {
constexpr uint64_t kPieceBytes = uint64_t(1) << 30;

// Tokens whose logits are kept at a time: 1 GiB of them, or one tile's.
constexpr uint64_t kLogitBytes = uint64_t(1) << 30;
uint64_t logit_chunk(uint64_t vocab)
{
    return std::max<uint64_t>(kLogitBytes / (round_up(vocab, kTileM) * 4) / 256, 1) * 256;
}
uint64_t logit_bytes(uint64_t tokens, uint64_t v_pad) { return round_up(tokens, 16) * v_pad * 4; }
uint64_t stats_bytes(HeadKind kind) { return kind.log_probs ? sizeof(LogParts) : sizeof(Stats); }
}  // namespace

// Each buffer's largest size over the plans of up to `ntokens` tokens: they
// differ in tiles, in the fp32 operands' form and in the parts of split sums,
// which are at most two rounds of tiles or kMostSplits times a whole sum.
uint64_t cross_entropy_bytes(uint64_t ntokens, uint64_t vocab, uint64_t width, ar_dtype_t dtype, HeadKind kind)
{
    const bool backward = kind.backward;
    const bool f32 = dtype == AR_FLOAT32;
    const uint64_t ob = f32 ? kPieces * 2 : 2, k_pad = round_up(width, f32 ? 32 : kTileK), t_pad = round_up(ntokens, kTileK);
    const uint64_t v_pad = round_up(vocab, kTileM), few = std::min<uint64_t>(ntokens, 64);
    const uint64_t row_bytes = ob * (k_pad + (backward ? 2 * t_pad + width : 0));
    const uint64_t piece = std::min(v_pad * row_bytes, std::max(kPieceBytes, kTileM * row_bytes));
    uint64_t bytes = ntokens * k_pad * ob + piece + 16 * 256;
    if (!backward)
        // 2 or 4 rows of statistics for 256 of the vocabulary, up to 16 for few
        // tokens; small tiles of more tokens come to less than 2^17 of them
        return bytes + (v_pad / kTileM + 1) * (ntokens * (f32 ? 4 : 2) + few * 16) * stats_bytes(kind) + ntokens * 4 +
               (1u << 17) * stats_bytes(kind) + (kind.top ? logit_bytes(std::min(ntokens, logit_chunk(vocab)), v_pad) : 0);
    constexpr uint64_t kRounds = 2 * kCUs * kTileM * 256 * 4;
    const uint64_t hidden_sum = ntokens * width * 4, weight_sum = v_pad * width * 4;
    return bytes + width * t_pad * ob + std::max(hidden_sum, std::min(hidden_sum * kMostSplits, kRounds)) +
           std::min(weight_sum * kMostSplits, kRounds) + sizeof(RowScale) +
           (kind.log_probs ? ntokens * 12 + 4 * 256 + v_pad * kFewTokens * 4 + few_partial_bytes(vocab, width) : 0);
}

CrossEntropyPlan plan_cross_entropy(uint64_t ntokens, uint64_t vocab, uint64_t width, ar_dtype_t dtype, HeadKind kind)
{
    const bool backward = kind.backward;
    CrossEntropyPlan p{};
    p.chunk = kind.top ? std::min(ntokens, logit_chunk(vocab)) : ntokens;
    const bool f32 = dtype == AR_FLOAT32;
    const bool small = small_tiles(ntokens, vocab, width, f32, backward);
    p.pieces = f32 && !small;
    p.tile_n = ntokens <= 16 ? 16 : small ? 64 : f32 ? kPiecesN : 256;
    const uint64_t ob = p.pieces ? kPieces * 2 : f32 ? 4 : 2, step = f32 ? 32 : kTileK;
    p.k_pad = round_up(width, step);
    p.t_pad = round_up(ntokens, p.tile_n == 16 ? 16 : kTileK);  // the tiles cover it: they write its zeros
    p.pack_hidden = p.pack_weight = true;  // the caller clears these where the operands can be read as they lie
    // A piece's buffers come to at most kPieceBytes, or one tile's; pieces are whole tiles.
    const uint64_t row_bytes = ob * (p.k_pad + (backward ? 2 * p.t_pad + width : 0));
    const uint64_t whole = round_up(vocab, kTileM) / kTileM;
    uint64_t most = kPieceBytes / (row_bytes * kTileM);
    if (most > 4096) most = 4096;  // the transposed piece's rows stay within a buffer's 2^31 bytes
    most = std::min(most, most_tiles(ntokens, p.tile_n));
    most = most < 1 ? 1 : most > whole ? whole : most;
    p.splits = p.weight_splits = 1;
    p.few = backward && kind.log_probs && ntokens && ntokens <= kFewTokens && width >= kFewWidth &&
            width < (1u << 20);  // (column chunks are counted in 16 bits)
    if (!backward || p.few) {
        const uint64_t pieces = (whole + most - 1) / most;
        p.piece = (whole + pieces - 1) / pieces * kTileM;
    } else {
        // From half the largest size on, the one whose tiles fill the CUs best.
        // 8192 x 131072 x 4096: the tiles of pieces of 20224 rows take ten, two and
        // five rounds for 9.9, 2 and 4.9; of 13312 rows the weight gradient's 832
        // take four for 3.25.
        const uint64_t tile_m = small ? kFewM : kTileM, tile_n = static_cast<uint64_t>(p.tile_n);
        const Shape shape = f32 ? Shape{ntokens, width, tile_m, tile_n, tile_m, small ? 64u : tile_n, step, p.pieces, kind.log_probs}
                                : Shape{ntokens, width, tile_m, tile_n, kTileM, 256, step, false, kind.log_probs};
        double best = 0;
        const uint64_t stride = most / 64 + 1;
        for (uint64_t m = most; m >= (most + 1) / 2 && m >= 1; m = m > stride ? m - stride : 0) {
            const uint64_t rows = m * kTileM, full = vocab / rows, rest = vocab - full * rows;
            int splits = 1, weight_splits = 1, unused;
            double c = piece_cost(shape, full ? rows : rest, &splits, &weight_splits) * (full ? full : 1);
            if (full && rest) c += piece_cost(shape, rest, &unused, &unused);
            if (best == 0 || c < best) {
                best = c;
                p.piece = rows;
                p.splits = splits;
                p.weight_splits = weight_splits;
            }
        }
    }
    // in pieces, or, where the weight is read as it lies, in as few launches as there can be
    for (const uint64_t rows : {p.piece, most_tiles(ntokens, p.tile_n) * kTileM}) {
        const uint64_t full = vocab / rows, rest = vocab % rows;
        p.stat_rows = std::max(p.stat_rows, full * stat_rows_of(rows, p.tile_n) +
                                                (rest ? stat_rows_of(rest, p.tile_n) : 0));
    }
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    p.hidden = take(ntokens * p.k_pad * ob);
    p.weight = take(p.piece * p.k_pad * ob);
    if (!backward) {
        p.stats = take(p.stat_rows * p.chunk * stats_bytes(kind));
        p.target_logit = take(p.chunk * 4);
        if (kind.top) p.logits = take(logit_bytes(p.chunk, round_up(vocab, kTileM)));
    } else if (p.few) {
        p.splits = static_cast<int>(few_parts(ntokens, vocab, width, f32));
        p.d = take(vocab * kFewTokens * 4);
        p.grad_hidden_acc = take(static_cast<uint64_t>(p.splits) * ntokens * width * 4);
        p.row_scale = take(sizeof(RowScale));
        p.row_gradients = take(ntokens * 12);
    } else {
        p.d = take(ntokens * p.piece * ob);
        p.dt = take(p.piece * p.t_pad * ob);
        p.weight_t = take(width * p.piece * ob);
        p.hidden_t = take(width * p.t_pad * ob);
        p.grad_hidden_acc = take(static_cast<uint64_t>(p.splits) * ntokens * width * 4);
        if (p.weight_splits > 1) p.grad_weight_acc = take(static_cast<uint64_t>(p.weight_splits) * p.piece * width * 4);
        p.row_scale = take(sizeof(RowScale));
        if (kind.log_probs) p.row_gradients = take(ntokens * 12);
    }
    p.bytes = at;
    return p;
}

namespace {
// fn(call) by the operands' type and form.
template <class Fn>
hipError_t by_type(const CrossEntropyArgs& a, const CrossEntropyPlan& p, ar_dtype_t dtype, char* ws, hipStream_t stream,
                   const Fn& fn)
{
    switch (dtype) {
    case AR_FLOAT32:
        return p.pieces ? fn(Call<F32, MmaBF16, kPieces>{a, p, ws, stream}) : fn(Call<F32, MmaF32, 1>{a, p, ws, stream});
    case AR_FLOAT16: return fn(Call<F16, MmaF16, 1>{a, p, ws, stream});
    case AR_BFLOAT16: return fn(Call<BF16, MmaBF16, 1>{a, p, ws, stream});
    default: return hipErrorInvalidValue;
    }
}
}  // namespace

hipError_t launch_cross_entropy(const CrossEntropyArgs& a, const CrossEntropyPlan& p, ar_dtype_t dtype, char* ws,
                                hipStream_t stream)
{
    return by_type(a, p, dtype, ws, stream,
                   [&](const auto& call) { return a.log_probs ? call.forward_log_probs() : call.forward(); });
}

hipError_t launch_cross_entropy_backward(const CrossEntropyArgs& a, const CrossEntropyPlan& p, ar_dtype_t dtype,
                                         char* ws, hipStream_t stream)
{
    return by_type(a, p, dtype, ws, stream, [](const auto& call) { return call.backward(); });
}

}  // namespace lm
}  // namespace ar
