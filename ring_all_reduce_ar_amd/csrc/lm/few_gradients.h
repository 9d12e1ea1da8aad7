// few_gradients.h -- both gradients of a linear head for up to 16 tokens.
//
//   dX[t] = sum_v d[t][v] W[v],   dW[v] = sum_t d[t][v] X[t]
//
// With so few tokens each element of W takes part in a few sums only: the time is
// that of reading W and writing dW once, which one pass over the rows v does, with
// the tokens' rows of X and of dX's sums in registers and d[.][v] in scalar ones.
// The matrix cores would want W transposed (read, written and read again) and d
// in 16 bits; here d is fp32. Forward and gradients by the products and so, us: 1
// token x 32000 x 4096 bf16 376 / 214, 8 of them 385 / 237, 16 383 / 312. From 8 tokens on
// the pass is bound by its sums (16: 128 of them for 8 bytes of W), up to 4 by HBM,
// 6.0 TB/s.
#pragma once

#include "log_probs.h"
#include "rows.h"

namespace ar {
namespace lm {
namespace {

constexpr int kFewTokens = 16;
constexpr uint64_t kFewWidth = 8;  // a vector at least

// d of a piece of the vocabulary, [vocabulary row][16 tokens], with the tokens'
// gradients; zeros for ignored ones and none.
struct FewDEpilogue {
    float* d;
    LogProbD rule;
    Indices targets;
    int64_t ignore;
    uint64_t vocab, v0;

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const GemmArgs& g, uint32_t,
                                               uint32_t, const S&) const
    {
        const uint32_t lane = threadIdx.x & 63, mine = m0 + (lane >> 4) * 4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t t = n0 + j * 16 + (lane & 15);
            const int64_t y = t < g.n ? load_target(targets, t, ignore, vocab) : -1;
            const uint32_t at = target_at<MT>(y, v0 + mine);
            const LogProbD::Row row = rule.row(t, y >= 0);
            const float scale = row.g * (1.0f / kLogProbScale);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) {
                    const uint32_t v = mine + 16 * i + r;
                    float x = rule(row, acc.v[i][j][r]);
                    if (at == 16 * i + r) x += rule.at_target(row);
                    if (v < g.m) d[(v0 + v) * kFewTokens + t] = y >= 0 ? x * scale : 0.0f;
                }
        }
    }
};

struct FewArgs {
    const void* weight;
    const void* hidden;
    void* grad_weight;  // or null
    float* partial;     // or null: [part][token][width] of grad_hidden
    const float* d;
    Indices targets;
    int64_t ignore;
    uint64_t vocab, ntokens, width, ld_weight, ld_hidden, ld_grad_weight, rows_each;
};

__device__ __forceinline__ void store_any(void* p, uint64_t byte, u32x4 v) { __builtin_memcpy(gptr<char>(p) + byte, &v, 16); }
__device__ __forceinline__ void store_any(void* p, uint64_t byte, u32x2 v) { __builtin_memcpy(gptr<char>(p) + byte, &v, 8); }
__device__ __forceinline__ void load_any(const void* p, uint64_t byte, u32x4* v) { __builtin_memcpy(v, gptr<char>(p) + byte, 16); }
__device__ __forceinline__ void load_any(const void* p, uint64_t byte, u32x2* v) { __builtin_memcpy(v, gptr<char>(p) + byte, 8); }

// U neighbours of a row at any address.
template <class F, int U>
__device__ __forceinline__ void get_row(const void* p, uint64_t at, float (&x)[U])
{
    constexpr int E = 16 / F::kEpv;  // bytes
    if constexpr (U * E == 16) {
        u32x4 v;
        load_any(p, at * E, &v);
        F::unpack(v, x);
    } else {
        u32x2 v;
        load_any(p, at * E, &v);
        F::unpack4(v, x);
    }
}
template <class F, int U>
__device__ __forceinline__ void put_row(void* p, uint64_t at, const float (&x)[U])
{
    constexpr int E = 16 / F::kEpv;
    if constexpr (F::kEpv == 4) {
        store_any(p, at * E, F::pack(x));
    } else {
        using T = typename std::conditional<std::is_same<F, F16>::value, MmaF16, MmaBF16>::type;
        if constexpr (U == 8)
            store_any(p, at * E, u32x4{T::pack2(x[0], x[1]), T::pack2(x[2], x[3]), T::pack2(x[4], x[5]), T::pack2(x[6], x[7])});
        else
            store_any(p, at * E, u32x2{T::pack2(x[0], x[1]), T::pack2(x[2], x[3])});
    }
}

// Column chunks of 64 U (blockIdx.y), rows of the vocabulary in parts
// (blockIdx.x), of which each wave takes every fourth row; NT: 4, 8 or 16 tokens.
// A lane at a row's end takes the last U columns, those of its neighbour among
// them, with the same results: no load or store is less than a vector.
template <class F, int NT, int U>
__global__ __launch_bounds__(256) void few_gradients(const FewArgs p)
{
    __shared__ float sums[4][64 * U];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t first = (static_cast<uint64_t>(blockIdx.y) * 64 + lane) * U;
    const uint64_t c = min(first, p.width - U);
    const bool mine = first < p.width;
    float x[NT][U], acc[NT][U];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int u = 0; u < U; ++u) x[t][u] = acc[t][u] = 0.0f;
        // (an ignored token's row may hold anything)
        if (static_cast<uint32_t>(t) < p.ntokens && load_target(p.targets, t, p.ignore, p.vocab) >= 0)
            get_row<F, U>(p.hidden, t * p.ld_hidden + c, x[t]);
    }
    const uint64_t lo = blockIdx.x * p.rows_each, hi = min(lo + p.rows_each, p.vocab);
    // (constant: nothing here writes it, so it is read into scalar registers)
    const auto* ds = (const __attribute__((address_space(4))) float*)p.d;
    constexpr int ROWS = 4;  // of a wave, whose loads are under way together
    for (uint64_t v0 = lo + wave; v0 < hi; v0 += 4 * ROWS) {
        float w[ROWS][U], dt[ROWS][NT];
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
#pragma unroll
            for (int t = 0; t < NT; ++t) dt[k][t] = ds[min(v0 + 4 * k, hi - 1) * kFewTokens + t];
        if (p.partial) {
#pragma unroll
            for (int k = 0; k < ROWS; ++k) get_row<F, U>(p.weight, min(v0 + 4 * k, hi - 1) * p.ld_weight + c, w[k]);
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            const uint64_t v = v0 + 4 * k;
            if (v >= hi) continue;
            float out[U] = {};
            if (p.partial) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < U; ++u) acc[t][u] = __builtin_fmaf(dt[k][t], w[k][u], acc[t][u]);
            }
            if (!p.grad_weight) continue;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < U; ++u) out[u] = __builtin_fmaf(dt[k][t], x[t][u], out[u]);
            if (mine) put_row<F, U>(p.grad_weight, v * p.ld_grad_weight + c, out);
        }
    }
    if (!p.partial) return;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (static_cast<uint32_t>(t) >= p.ntokens) continue;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) sums[wave][u * 64 + lane] = acc[t][u];
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < 64 * U; i += 256) {
            const uint64_t from = (static_cast<uint64_t>(blockIdx.y) * 64 + i % 64) * U;
            if (from < p.width)
                p.partial[(blockIdx.x * p.ntokens + t) * p.width + min(from, p.width - U) + i / 64] =
                    (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
        }
    }
}

// grad_hidden from the parts: a workgroup has 64 columns of a token, its waves
// every fourth part. An ignored token's is 0, whatever its parts hold: its d is 0,
// but 0 times an infinity or a NaN of the weight is NaN.
template <class F>
__global__ __launch_bounds__(256) void join_few(const float* partial, uint64_t parts, Indices targets, int64_t ignore,
                                                uint64_t vocab, uint64_t ntokens, uint64_t width, void* out, uint64_t ld)
{
    __shared__ float sums[4][64];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t c = static_cast<uint64_t>(blockIdx.x) * 64 + lane, t = blockIdx.y;
    const bool on = load_target(targets, t, ignore, vocab) >= 0;
    float s = 0.0f;
    if (c < width) {
#pragma unroll 8
        for (uint64_t k = wave; k < parts; k += 4) s += partial[(k * ntokens + t) * width + c];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < width)
        F::st(out, t * ld + c, on ? (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]) : 0.0f);
}

// Columns of a thread: as many as its registers take beside the tokens' rows, with
// waves enough (8 tokens of fp16: 150 us with 8 columns, 118 with 4).
constexpr int few_columns(uint64_t ntokens, bool f32) { return !f32 && ntokens <= 4 ? 8 : 4; }

// Parts of the vocabulary: about eight workgroups a CU with all column chunks, of
// 32 rows at least.
inline uint64_t few_parts(uint64_t ntokens, uint64_t vocab, uint64_t width, bool f32)
{
    const uint64_t chunk = 64 * few_columns(ntokens, f32), chunks = (width + chunk - 1) / chunk;
    const uint64_t parts = chunks < 2048 ? 2048 / chunks : 1, most = (vocab + 31) / 32;
    return parts < most ? parts : most;
}
// Of any number of tokens up to 16: parts * width is at most 2048 chunks.
inline uint64_t few_partial_bytes(uint64_t vocab, uint64_t width)
{
    const uint64_t most = 2048ull * 64 * 8 * 8 * 4, rows = ((vocab + 31) / 32) * width * kFewTokens * 4;
    return most + width * kFewTokens * 4 < rows ? most + width * kFewTokens * 4 : rows;
}

template <class F>
hipError_t launch_few_gradients(FewArgs p, uint64_t parts, void* grad_hidden, uint64_t ld_grad_hidden, hipStream_t s)
{
    constexpr bool f32 = F::kEpv == 4;
    const uint64_t chunk = 64 * few_columns(p.ntokens, f32);
    p.rows_each = (p.vocab + parts - 1) / parts;
    const dim3 grid(static_cast<uint32_t>(parts), static_cast<uint32_t>((p.width + chunk - 1) / chunk));
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, p); };
    constexpr int kWide = f32 ? 4 : 8;
    if (p.ntokens <= 4) launch(few_gradients<F, 4, kWide>);
    else if (p.ntokens <= 8) launch(few_gradients<F, 8, 4>);
    else launch(few_gradients<F, 16, 4>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.partial) return e;
    hipLaunchKernelGGL((join_few<F>), dim3(static_cast<uint32_t>((p.width + 63) / 64), static_cast<uint32_t>(p.ntokens)),
                       dim3(256), 0, s, p.partial, parts, p.targets, p.ignore, p.vocab, p.ntokens, p.width, grad_hidden,
                       ld_grad_hidden);
    return hipGetLastError();
}

}  // namespace
}  // namespace lm
}  // namespace ar
