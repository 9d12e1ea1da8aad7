// cross_entropy.hip -- softmax cross entropy of a linear head, in pieces of
// the vocabulary, without keeping the logits.
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
// fp32 operands are laid out as three bf16 pieces each (kF32Parts): six bf16
// products give the fp32 product to 2^-24 at 2.5 PFLOP/s / 6, where the fp32
// matrix instructions end at 0.16.
#include <type_traits>

#include "gemm.h"

namespace ar {
namespace lm {
using namespace detail;

namespace {

// d is held times 2^14: a probability of 1e-8 is still a normal fp16, and
// |p - 1| 2^14 is far below its largest.
constexpr float kDBits = 14.0f, kDScale = 16384.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPartA[kF32Parts] = {0, 0, 1, 0, 1, 2};
constexpr int kPartB[kF32Parts] = {0, 1, 0, 2, 1, 0};

__device__ __forceinline__ int64_t load_target(const Indices& x, uint64_t t, int64_t ignore, uint64_t vocab)
{
    const int64_t y = x.is64 ? gptr<int64_t>(x.p)[t] : static_cast<int64_t>(gptr<int32_t>(x.p)[t]);
    return y == ignore || static_cast<uint64_t>(y) >= vocab ? -1 : y;
}

// Where target y lies among a lane's rows v, v + 1 .. of MT groups of 16.
constexpr uint32_t kNoTarget = UINT32_MAX;
template <int MT>
__device__ __forceinline__ uint32_t target_at(int64_t y, uint64_t v)
{
    const uint64_t at = static_cast<uint64_t>(y) - v;
    return y >= 0 && at < MT * 16 ? static_cast<uint32_t>(at) : kNoTarget;
}

// The three bf16 pieces of a float; a value that is no number stays in the first.
__device__ __forceinline__ void split3(float x, uint32_t (&p)[3])
{
    p[0] = f32_to_bf16(x);
    const float r1 = x - bf16_to_f32(p[0]);
    const bool finite = __builtin_isfinite(bf16_to_f32(p[0]));
    p[1] = finite ? f32_to_bf16(r1) : 0;
    const float r2 = r1 - bf16_to_f32(p[1]);
    p[2] = finite ? f32_to_bf16(r2) : 0;
}

// ---------------------------------------------------------------------------
// laying out operands
// ---------------------------------------------------------------------------
// out[r][part * pad + c] = in[r][c], zeros up to `pad`.
template <class F, int PARTS, bool IS_A>
__global__ __launch_bounds__(kBlock) void pack_rows(const void* in, uint64_t ld, uint64_t rows, uint64_t width,
                                                    uint64_t pad, uint16_t* out)
{
    const uint64_t n = rows * pad;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n;
         i += static_cast<uint64_t>(gridDim.x) * kBlock) {
        const uint64_t r = i / pad, c = i - r * pad;
        if constexpr (PARTS == 1) {
            out[i] = c < width ? gptr<uint16_t>(in)[r * ld + c] : 0;
        } else {
            uint32_t p[3];
            split3(c < width ? F::ld(in, r * ld + c) : 0.0f, p);
#pragma unroll
            for (int k = 0; k < PARTS; ++k)
                out[(r * PARTS + k) * pad + c] = static_cast<uint16_t>(p[IS_A ? kPartA[k] : kPartB[k]]);
        }
    }
}

// out[c][part * pad + r] = in[r][c] for r < rows, zeros up to `pad` and in
// rows whose target is ignored (whatever they hold). 64x64 tiles through LDS.
template <class F, int PARTS>
__global__ __launch_bounds__(kBlock) void pack_transposed(const void* in, uint64_t ld, uint64_t rows, uint64_t width,
                                                          uint64_t pad, uint16_t* out, Indices targets, int masked,
                                                          int64_t ignore, uint64_t vocab)
{
    using Raw = typename std::conditional<PARTS == 1, uint16_t, float>::type;
    __shared__ Raw tile[64][65];
    const uint64_t r0 = static_cast<uint64_t>(blockIdx.x) * 64, c0 = static_cast<uint64_t>(blockIdx.y) * 64;
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    for (int i = y; i < 64; i += 4) {
        const uint64_t r = r0 + i, c = c0 + x;
        Raw v = 0;
        if (r < rows && c < width && (!masked || load_target(targets, r, ignore, vocab) >= 0))
            v = gptr<Raw>(in)[r * ld + c];
        tile[i][x] = v;
    }
    __syncthreads();
    for (int i = y; i < 64; i += 4) {
        const uint64_t r = r0 + x, c = c0 + i;
        if (r >= pad || c >= width) continue;
        if constexpr (PARTS == 1) {
            out[c * pad + r] = tile[x][i];
        } else {
            uint32_t p[3];
            split3(tile[x][i], p);
#pragma unroll
            for (int k = 0; k < PARTS; ++k) out[(c * PARTS + k) * pad + r] = static_cast<uint16_t>(p[kPartA[k]]);
        }
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
                    if (at == 16 * i + r) target_logit[t] = acc.v[i][j][r];
        }
    }
};

// Joins the parts of each token's row: 16 tokens a workgroup, 16 parts at a time.
__global__ __launch_bounds__(kBlock) void join_stats(const Stats* stats, uint64_t stat_rows, const float* target_logit,
                                                     Indices targets, int64_t ignore, uint64_t vocab, uint64_t ntokens,
                                                     float* losses, float* lse)
{
    __shared__ Stats part[16][17];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    const uint64_t t = static_cast<uint64_t>(blockIdx.x) * 16 + x;
    float top = -INFINITY, sum = 0.0f;
    if (t < ntokens) {
        for (uint64_t r = y; r < stat_rows; r += 16) {
            const Stats s = stats[r * ntokens + t];
            const float m = fmaxf(top, s.top);
            if (m == -INFINITY) {
                sum += s.sum;  // nothing yet, or a NaN
            } else {
                sum = sum * __builtin_amdgcn_exp2f((top - m) * kLog2e) + s.sum * __builtin_amdgcn_exp2f((s.top - m) * kLog2e);
            }
            top = m;
        }
    }
    part[y][x] = Stats{top, sum};
    __syncthreads();
    if (y == 0 && t < ntokens) {
        for (int k = 1; k < 16; ++k) {
            const Stats s = part[k][x];
            const float m = fmaxf(top, s.top);
            if (m == -INFINITY) {
                sum += s.sum;
            } else {
                sum = sum * __builtin_amdgcn_exp2f((top - m) * kLog2e) + s.sum * __builtin_amdgcn_exp2f((s.top - m) * kLog2e);
            }
            top = m;
        }
        const float l = top + logf(sum);
        lse[t] = l;
        losses[t] = load_target(targets, t, ignore, vocab) >= 0 ? l - target_logit[t] : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct RowScale {
    float top;  // the largest |g| of the rows that count, 1 if there is none
};

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
        out->top = top > 0.0f ? top : 1.0f;
    }
}

// d of one piece, in both orders: d[t][part * piece_pad + v] = 2^14 (p - [v =
// y]) for the hidden gradient (whose rows take g[t] at the end) and
// dt[v][part * t_pad + t] the same times g[t] / max |g| for the weight's.
template <class T, int PARTS>
struct DEpilogue {
    uint16_t* d;
    uint16_t* dt;
    const float* lse;
    const float* g_losses;
    const RowScale* scale;
    Indices targets;
    int64_t ignore;
    uint64_t vocab, v0, piece_pad, t_pad;

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const GemmArgs& g, uint32_t,
                                               uint32_t, const S& stage) const
    {
        const int lane = threadIdx.x & 63;
        float factor[NT];  // of a token's column of dt
        bool all = m0 + MT * 16 <= g.m;
        const float inv = 1.0f / scale->top;
        uint32_t at[NT];
        bool on[NT];
        float l[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t t = n0 + j * 16 + (lane & 15);
            const int64_t y = t < g.n ? load_target(targets, t, ignore, vocab) : -1;
            at[j] = target_at<MT>(y, v0 + m0 + (lane >> 4) * 4);
            on[j] = y >= 0;
            l[j] = on[j] ? lse[t] : 0.0f;
            factor[j] = on[j] ? g_losses[t] * inv : 0.0f;
            all = all && on[j];
        }
        if (__all(all)) differences<true>(acc, at, on, l, m0, g);
        else differences<false>(acc, at, on, l, m0, g);
        if constexpr (S::kOn && PARTS == 1) {
            if (d) stage.template store_by_column<T>(acc, d, piece_pad, g.n, static_cast<uint32_t>(piece_pad));
            if (dt) stage.template store_by_row<T>(acc, factor, dt, t_pad, g.m, static_cast<uint32_t>(t_pad));
        } else {
            store(acc, factor, m0, n0, g);
        }
    }

private:
    // acc = 2^14 (exp(acc - lse) - [v = y]). FULL: every row is one of the
    // vocabulary and every token counts; else zeros where not.
    template <bool FULL, int MT, int NT>
    __device__ __forceinline__ void differences(Tile<MT, NT>& acc, const uint32_t (&at)[NT], const bool (&on)[NT],
                                                const float (&l)[NT], uint32_t m0, const GemmArgs& g) const
    {
        const uint32_t mine = m0 + ((threadIdx.x & 63) >> 4) * 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(acc.v[i][j][r] - l[j], kLog2e, kDBits));
                    acc.v[i][j][r] = FULL || (on[j] && mine + 16 * i + r < g.m) ? p : 0.0f;
                }
            __builtin_amdgcn_sched_barrier(0);
            if (!__any(at[j] != kNoTarget)) continue;  // few tiles hold a target
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc.v[i][j][r] -= at[j] == 16 * i + r ? kDScale : 0.0f;
        }
    }

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
                    if constexpr (PARTS == 1) {
                        *reinterpret_cast<u32x2*>(d + static_cast<uint64_t>(t) * piece_pad + v) =
                            u32x2{T::pack2(x[0], x[1]), T::pack2(x[2], x[3])};
                    } else {
                        uint32_t p[4][3];
#pragma unroll
                        for (int r = 0; r < 4; ++r) split3(x[r], p[r]);
#pragma unroll
                        for (int k = 0; k < PARTS; ++k) {
                            const int q = kPartB[k];
                            *reinterpret_cast<u32x2*>(d + (static_cast<uint64_t>(t) * PARTS + k) * piece_pad + v) =
                                u32x2{p[0][q] | (p[1][q] << 16), p[2][q] | (p[3][q] << 16)};
                        }
                    }
                }
                if (dt && t < t_pad) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (v + r >= g.m) continue;
                        const float s = x[r] * factor[j];
                        if constexpr (PARTS == 1) {
                            T::Format::st(dt, static_cast<uint64_t>(v + r) * t_pad + t, s);
                        } else {
                            uint32_t p[3];
                            split3(s, p);
#pragma unroll
                            for (int k = 0; k < PARTS; ++k)
                                dt[(static_cast<uint64_t>(v + r) * PARTS + k) * t_pad + t] =
                                    static_cast<uint16_t>(p[kPartB[k]]);
                        }
                    }
                }
            }
        }
    }
};

// One split's sums of the hidden gradient: acc[split][t][h], over all pieces.
struct HiddenEpilogue {
    float* acc;
    uint64_t width;
    int add;

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& c, uint32_t m0, uint32_t n0, const GemmArgs& g, uint32_t,
                                               uint32_t split, const S&) const
    {
        const int lane = threadIdx.x & 63, quad = lane >> 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t t = n0 + j * 16 + (lane & 15);
            if (t >= g.n) continue;
            float* row = acc + (static_cast<uint64_t>(split) * g.n + t) * width;
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

// grad_hidden[t][h] = round(g[t] 2^-14 * the splits' sum), 0 for ignored tokens.
template <class F>
__global__ __launch_bounds__(kBlock) void finish_hidden(const float* acc, int splits, const float* g, Indices targets,
                                                        int64_t ignore, uint64_t vocab, uint64_t ntokens,
                                                        uint64_t width, void* out, uint64_t ld)
{
    const uint64_t n = ntokens * width;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n;
         i += static_cast<uint64_t>(gridDim.x) * kBlock) {
        const uint64_t t = i / width;
        float s = acc[i];
        for (int k = 1; k < splits; ++k) s += acc[static_cast<uint64_t>(k) * n + i];
        const bool on = load_target(targets, t, ignore, vocab) >= 0;
        F::st(out, t * ld + (i - t * width), on ? s * (g[t] * (1.0f / kDScale)) : 0.0f);
    }
}

// grad_weight[v][h] = round(max |g| 2^-14 * sum).
template <class F>
struct WeightEpilogue {
    void* out;
    uint64_t ld;
    const RowScale* scale;
    int vec;  // 4 elements at a time: the pitch and the address allow it

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& c, uint32_t m0, uint32_t n0, const GemmArgs& g, uint32_t,
                                               uint32_t, const S&) const
    {
        const int lane = threadIdx.x & 63, quad = lane >> 4;
        const float s = scale->top * (1.0f / kDScale);
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
                if (vec && h + 3 < g.m) {
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
int blocks_for(uint64_t units)
{
    const uint64_t want = (units + kBlock - 1) / kBlock;
    return static_cast<int>(want < 1 ? 1 : want > 16384 ? 16384 : want);
}

template <class F, int PARTS, bool IS_A>
hipError_t pack(const void* in, uint64_t ld, uint64_t rows, uint64_t width, uint64_t pad, uint16_t* out, hipStream_t s)
{
    hipLaunchKernelGGL((pack_rows<F, PARTS, IS_A>), dim3(blocks_for(rows * pad)), dim3(kBlock), 0, s, in, ld, rows,
                       width, pad, out);
    return hipGetLastError();
}

template <class T, class Epilogue>
hipError_t logits(const GemmArgs& g, int tile_n, const Epilogue& epi, hipStream_t s)
{
    if (tile_n == 16) return launch_gemm<T, 16, 8, 1>(g, epi, s);
    if (tile_n == 64) return launch_gemm<T, 64, 4, 2>(g, epi, s);
    return launch_gemm<T, 256, 2, 4>(g, epi, s);
}

// F: the storage type; T: the matrix instruction's.
template <class F, class T, int PARTS>
struct Call {
    const CrossEntropyArgs& a;
    const CrossEntropyPlan& p;
    char* ws;
    hipStream_t s;

    uint64_t part_k() const { return p.k_pad / PARTS; }

    // The logits' operands, packed where the plan says so.
    hipError_t hidden(const uint16_t** out, uint64_t* ld) const
    {
        if (!p.pack_hidden) {
            *out = static_cast<const uint16_t*>(a.hidden);
            *ld = a.ld_hidden;
            return hipSuccess;
        }
        uint16_t* to = reinterpret_cast<uint16_t*>(ws + p.hidden);
        *out = to;
        *ld = p.k_pad;
        return pack<F, PARTS, false>(a.hidden, a.ld_hidden, a.ntokens, a.width, part_k(), to, s);
    }
    hipError_t weight(uint64_t v0, uint64_t rows, const uint16_t** out, uint64_t* ld) const
    {
        const char* from = static_cast<const char*>(a.weight) + v0 * a.ld_weight * (16 / F::kEpv);
        if (!p.pack_weight) {
            *out = reinterpret_cast<const uint16_t*>(from);
            *ld = a.ld_weight;
            return hipSuccess;
        }
        uint16_t* to = reinterpret_cast<uint16_t*>(ws + p.weight);
        *out = to;
        *ld = p.k_pad;
        return pack<F, PARTS, true>(from, a.ld_weight, rows, a.width, part_k(), to, s);
    }
    GemmArgs logits_args(const uint16_t* w, uint64_t ldw, const uint16_t* x, uint64_t ldx, uint64_t rows) const
    {
        GemmArgs g{};
        g.a = w;
        g.b = x;
        g.lda = ldw;
        g.ldb = ldx;
        g.m = static_cast<uint32_t>(rows);
        g.n = static_cast<uint32_t>(a.ntokens);
        g.k = g.k_all = static_cast<uint32_t>(p.k_pad);
        g.splits = 1;
        return g;
    }

    hipError_t forward() const
    {
        const uint16_t *x, *w;
        uint64_t ldx, ldw, row0 = 0;
        hipError_t e = hidden(&x, &ldx);
        if (e != hipSuccess) return e;
        Stats* stats = reinterpret_cast<Stats*>(ws + p.stats);
        float* target_logit = reinterpret_cast<float*>(ws + p.target_logit);
        const uint64_t waves_m = p.tile_n == 16 ? 8 : p.tile_n == 64 ? 4 : 2;
        for (uint64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
            const uint64_t rows = a.vocab - v0 < p.piece ? a.vocab - v0 : p.piece;
            if ((e = weight(v0, rows, &w, &ldw)) != hipSuccess) return e;
            const StatsEpilogue epi{stats, target_logit, a.targets, a.ignore_index, a.vocab, v0, row0};
            if ((e = logits<T>(logits_args(w, ldw, x, ldx, rows), p.tile_n, epi, s)) != hipSuccess) return e;
            row0 += (rows + kTileM - 1) / kTileM * waves_m;
        }
        hipLaunchKernelGGL(join_stats, dim3(static_cast<uint32_t>((a.ntokens + 15) / 16)), dim3(kBlock), 0, s, stats,
                           row0, target_logit, a.targets, a.ignore_index, a.vocab, a.ntokens, a.losses, a.lse);
        return hipGetLastError();
    }

    hipError_t backward() const
    {
        const uint16_t *x = nullptr, *w = nullptr;
        uint64_t ldx = 0, ldw = 0;
        hipError_t e = a.ntokens ? hidden(&x, &ldx) : hipSuccess;
        if (e != hipSuccess) return e;
        uint16_t* d = a.grad_hidden && a.ntokens ? reinterpret_cast<uint16_t*>(ws + p.d) : nullptr;
        uint16_t* dt = a.grad_weight ? reinterpret_cast<uint16_t*>(ws + p.dt) : nullptr;
        uint16_t* wt = reinterpret_cast<uint16_t*>(ws + p.weight_t);
        uint16_t* xt = reinterpret_cast<uint16_t*>(ws + p.hidden_t);
        float* acc = reinterpret_cast<float*>(ws + p.grad_hidden_acc);
        RowScale* scale = reinterpret_cast<RowScale*>(ws + p.row_scale);
        const uint32_t cols = static_cast<uint32_t>((a.width + 63) / 64);
        hipLaunchKernelGGL(row_scale, dim3(1), dim3(1024), 0, s, a.grad_losses, a.targets, a.ignore_index, a.vocab,
                           a.ntokens, scale);
        if (dt && a.ntokens)
            hipLaunchKernelGGL((pack_transposed<F, PARTS>), dim3(static_cast<uint32_t>(p.t_pad / 64), cols),
                               dim3(kBlock), 0, s, a.hidden, a.ld_hidden, a.ntokens, a.width, p.t_pad, xt, a.targets, 1,
                               a.ignore_index, a.vocab);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        for (uint64_t v0 = 0; v0 < a.vocab; v0 += p.piece) {
            const uint64_t rows = a.vocab - v0 < p.piece ? a.vocab - v0 : p.piece;
            const uint64_t pad = (rows + kTileK - 1) / kTileK * kTileK;
            if (a.ntokens) {  // no token: the weight's gradient is the empty sum
                if ((e = weight(v0, rows, &w, &ldw)) != hipSuccess) return e;
                const DEpilogue<T, PARTS> epi{d, dt, a.lse, a.grad_losses, scale, a.targets,
                                                               a.ignore_index, a.vocab, v0, pad, p.t_pad};
                if ((e = logits<T>(logits_args(w, ldw, x, ldx, rows), p.tile_n, epi, s)) != hipSuccess) return e;
            }
            if (d) {
                const char* from = static_cast<const char*>(a.weight) + v0 * a.ld_weight * (16 / F::kEpv);
                hipLaunchKernelGGL((pack_transposed<F, PARTS>), dim3(static_cast<uint32_t>(pad / 64), cols),
                                   dim3(kBlock), 0, s, from, a.ld_weight, rows, a.width, pad, wt, a.targets, 0,
                                   a.ignore_index, a.vocab);
                if ((e = hipGetLastError()) != hipSuccess) return e;
                GemmArgs g{};
                g.a = wt;
                g.b = d;
                g.lda = g.ldb = pad * PARTS;
                g.m = static_cast<uint32_t>(a.width);
                g.n = static_cast<uint32_t>(a.ntokens);
                g.k_all = static_cast<uint32_t>(pad * PARTS);
                g.splits = static_cast<uint32_t>(p.splits);
                g.k = (g.k_all / kTileK + g.splits - 1) / g.splits * kTileK;
                const HiddenEpilogue he{acc, a.width, v0 > 0};
                if ((e = logits<T>(g, p.tile_n, he, s)) != hipSuccess) return e;
            }
            if (dt) {
                GemmArgs g{};
                g.a = xt;
                g.b = dt;
                g.lda = g.ldb = p.t_pad * PARTS;
                g.m = static_cast<uint32_t>(a.width);
                g.n = static_cast<uint32_t>(rows);
                g.k = g.k_all = static_cast<uint32_t>(p.t_pad * PARTS);
                g.splits = 1;
                constexpr int EB = 16 / F::kEpv;
                char* out = static_cast<char*>(a.grad_weight) + v0 * a.ld_grad_weight * EB;
                const WeightEpilogue<F> we{out, a.ld_grad_weight, scale,
                                           reinterpret_cast<uintptr_t>(out) % (4 * EB) == 0 && a.ld_grad_weight % 4 == 0};
                if ((e = launch_gemm<T, 256, 2, 4>(g, we, s)) != hipSuccess) return e;
            }
        }
        if (d) {
            hipLaunchKernelGGL((finish_hidden<F>), dim3(blocks_for(a.ntokens * a.width)), dim3(kBlock), 0, s, acc,
                               p.splits, a.grad_losses, a.targets, a.ignore_index, a.vocab, a.ntokens, a.width,
                               a.grad_hidden, a.ld_grad_hidden);
            e = hipGetLastError();
        }
        return e;
    }
};

uint64_t round_up(uint64_t x, uint64_t m) { return (x + m - 1) / m * m; }

}  // namespace

CrossEntropyPlan plan_cross_entropy(uint64_t ntokens, uint64_t vocab, uint64_t width, ar_dtype_t dtype, bool backward)
{
    CrossEntropyPlan p{};
    const bool f32 = dtype == AR_FLOAT32;
    p.parts = f32 ? kF32Parts : 1;
    // six parts of a multiple of 32 are a multiple of kTileK
    p.k_pad = f32 ? round_up(width, 32) * p.parts : round_up(width, kTileK);
    p.t_pad = round_up(ntokens, kTileK);
    // (backward, the tiles cover all of t_pad: they write its zeros)
    p.tile_n = ntokens <= 16 && !backward ? 16 : ntokens <= 64 ? 64 : 256;
    p.pack_hidden = p.pack_weight = true;  // the caller clears these where the operands can be read as they lie
    // A piece's buffers come to about kPieceBytes; pieces are whole tiles.
    constexpr uint64_t kPieceBytes = uint64_t(640) << 20;
    uint64_t a_row = 2 * p.k_pad;
    if (backward) a_row += 2 * p.parts * (2 * p.t_pad + width);
    uint64_t piece = kPieceBytes / a_row / kTileM * kTileM;
    if (piece < kTileM) piece = kTileM;
    const uint64_t whole = round_up(vocab, kTileM);
    const uint64_t pieces = (whole + piece - 1) / piece;
    p.piece = round_up((vocab + pieces - 1) / (pieces ? pieces : 1), kTileM);
    if (p.piece == 0) p.piece = kTileM;
    p.piece_pad = p.piece;
    // The hidden gradient sums over a piece: its product is split along that
    // axis until there are a few workgroups for each CU.
    const uint64_t tiles = (round_up(width, kTileM) / kTileM) * ((ntokens + p.tile_n - 1) / p.tile_n);
    p.splits = 1;
    while (p.splits < 16 && tiles * p.splits < 256 && p.piece / (2 * p.splits) >= 512) p.splits *= 2;
    const uint64_t waves_m = p.tile_n == 16 ? 8 : p.tile_n == 64 ? 4 : 2;
    const uint64_t tiles_v = (p.piece / kTileM) * ((vocab + p.piece - 1) / p.piece);
    p.stat_rows = tiles_v * waves_m;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    p.hidden = take(ntokens * p.k_pad * 2);
    p.weight = take(p.piece * p.k_pad * 2);
    if (!backward) {
        p.stats = take(p.stat_rows * ntokens * sizeof(Stats));
        p.target_logit = take(ntokens * 4);
    } else {
        p.d = take(ntokens * p.piece_pad * p.parts * 2);
        p.dt = take(p.piece * p.t_pad * p.parts * 2);
        p.weight_t = take(width * p.piece_pad * p.parts * 2);
        p.hidden_t = take(width * p.t_pad * p.parts * 2);
        p.grad_hidden_acc = take(static_cast<uint64_t>(p.splits) * ntokens * width * 4);
        p.row_scale = take(sizeof(RowScale));
    }
    p.bytes = at;
    return p;
}

hipError_t launch_cross_entropy(const CrossEntropyArgs& a, const CrossEntropyPlan& p, ar_dtype_t dtype, char* ws,
                                hipStream_t stream)
{
    switch (dtype) {
    case AR_FLOAT32: return Call<F32, MmaBF16, kF32Parts>{a, p, ws, stream}.forward();
    case AR_FLOAT16: return Call<F16, MmaF16, 1>{a, p, ws, stream}.forward();
    case AR_BFLOAT16: return Call<BF16, MmaBF16, 1>{a, p, ws, stream}.forward();
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_cross_entropy_backward(const CrossEntropyArgs& a, const CrossEntropyPlan& p, ar_dtype_t dtype,
                                         char* ws, hipStream_t stream)
{
    switch (dtype) {
    case AR_FLOAT32: return Call<F32, MmaBF16, kF32Parts>{a, p, ws, stream}.backward();
    case AR_FLOAT16: return Call<F16, MmaF16, 1>{a, p, ws, stream}.backward();
    case AR_BFLOAT16: return Call<BF16, MmaBF16, 1>{a, p, ws, stream}.backward();
    default: return hipErrorInvalidValue;
    }
}

}  // namespace lm
}  // namespace ar
