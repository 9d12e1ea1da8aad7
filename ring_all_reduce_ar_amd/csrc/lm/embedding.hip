// embedding.hip -- the embedding lookup, and its gradient by sorted tokens.
//
//   out[t] = round(scale * W[token[t] - first_row]), zero where that row is not here
//   dW[v]  = round(scale * sum over {t : token[t] - first_row = v}, t ascending, of dout[t])
//
// The gradient sorts the tokens (stable radix sort), so that a row's
// contributions lie side by side in token order: each row is summed in fp32 in
// one fixed order and written once, with no float atomics, and the rows that no
// token meets are written as zeros in the same launch.
#include "../kernels_impl.h"
#include "lm_kernels.h"

namespace ar {
namespace lm {
using namespace detail;

namespace {

__device__ __forceinline__ int64_t load_index(const Indices& x, uint64_t i)
{
    return x.is64 ? gptr<int64_t>(x.p)[i] : static_cast<int64_t>(gptr<int32_t>(x.p)[i]);
}

// The row of token t, or `rows` where it is not one of [0, rows).
__device__ __forceinline__ uint64_t row_of(const Indices& x, uint64_t t, int64_t first_row, uint64_t rows)
{
    const uint64_t r = static_cast<uint64_t>(load_index(x, t)) - static_cast<uint64_t>(first_row);
    return r < rows ? r : rows;
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
// `lanes` (a power of two up to kBlock) threads a row, kBlock / lanes rows a
// workgroup; VEC: 16-byte vectors, else elements.
template <class F, bool VEC>
__global__ __launch_bounds__(kBlock) void lookup(const LookupArgs a, int lanes)
{
    constexpr int E = F::kEpv;
    const int per = kBlock / lanes;
    const uint64_t units = VEC ? a.width / E : a.width;
    const int lane = threadIdx.x & (lanes - 1);
    for (uint64_t t = static_cast<uint64_t>(blockIdx.x) * per + threadIdx.x / lanes; t < a.ntokens;
         t += static_cast<uint64_t>(gridDim.x) * per) {
        const uint64_t row = row_of(a.tokens, t, a.first_row, a.rows);
        const bool here = row < a.rows;
        const uint64_t src = (here ? row : 0) * a.ld_weight, dst = t * a.ld_out;
        for (uint64_t c = lane; c < units; c += lanes) {
            if constexpr (VEC) {
                float x[E];
                u32x4 v = {0, 0, 0, 0};
                if (here) v = ldv_at<false>(a.weight, src * (16 / E) + c * 16);
                F::unpack(v, x);
#pragma unroll
                for (int j = 0; j < E; ++j) x[j] *= a.scale;
                if (!here) {
#pragma unroll
                    for (int j = 0; j < E; ++j) x[j] = 0.0f;
                }
                stv_at<false>(a.out, dst * (16 / E) + c * 16, F::pack(x));
            } else {
                F::st(a.out, dst + c, here ? F::ld(a.weight, src + c) * a.scale : 0.0f);
            }
        }
    }
}

template <class F>
hipError_t lookup_launch(const LookupArgs& a, bool vec, hipStream_t s)
{
    const uint64_t units = vec ? a.width / F::kEpv : a.width;
    int lanes = 1;
    while (lanes < kBlock && static_cast<uint64_t>(lanes) < units) lanes *= 2;
    const uint64_t per = kBlock / lanes;
    const uint64_t want = (a.ntokens + per - 1) / per;
    const int grid = static_cast<int>(want < (1u << 20) ? want : (1u << 20));
    if (vec) hipLaunchKernelGGL((lookup<F, true>), dim3(grid), dim3(kBlock), 0, s, a, lanes);
    else hipLaunchKernelGGL((lookup<F, false>), dim3(grid), dim3(kBlock), 0, s, a, lanes);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// stable radix sort of the tokens' rows, least significant digit first
// ---------------------------------------------------------------------------
// Digits of one workgroup's keys, bin-major: hist[bin * blocks + block]. The
// first pass reads the tokens and clears the presence bits; the last one sets
// them.
__global__ __launch_bounds__(kBlock) void sort_count(const LookupGradArgs a, int src, int shift, int bits, int first,
                                                     int last)
{
    __shared__ uint32_t bins[kSortBins];
    const int nb = 1 << bits;
    for (int i = threadIdx.x; i < nb; i += kBlock) bins[i] = 0;
    if (first) {
        const uint64_t words = (a.rows + 31) / 32;
        for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x; i < words;
             i += static_cast<uint64_t>(gridDim.x) * kBlock)
            a.present[i] = 0;
    }
    __syncthreads();
    const uint64_t lo = static_cast<uint64_t>(blockIdx.x) * kSortBlockKeys;
    for (int k = threadIdx.x; k < kSortBlockKeys; k += kBlock) {
        const uint64_t t = lo + k;
        if (t >= a.ntokens) break;
        const uint32_t key =
            first ? static_cast<uint32_t>(row_of(a.tokens, t, a.first_row, a.rows)) : a.key[src][t];
        atomicAdd(&bins[(key >> shift) & (nb - 1)], 1u);
        (void)last;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nb; i += kBlock) a.hist[static_cast<uint64_t>(i) * gridDim.x + blockIdx.x] = bins[i];
}

// Exclusive sums over `n` counts, by one workgroup.
__global__ __launch_bounds__(1024) void sort_scan(uint32_t* hist, uint64_t n)
{
    __shared__ uint32_t waves[16];
    __shared__ uint32_t carry;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0) carry = 0;
    __syncthreads();
    for (uint64_t lo = 0; lo < n; lo += 1024) {
        const uint64_t i = lo + threadIdx.x;
        const uint32_t v = i < n ? hist[i] : 0;
        uint32_t s = v;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t o = __shfl_up(s, d, 64);
            if (lane >= d) s += o;
        }
        if (lane == 63) waves[wave] = s;
        __syncthreads();
        uint32_t before = carry, all = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            if (w < wave) before += waves[w];
            all += waves[w];
        }
        if (i < n) hist[i] = before + s - v;
        __syncthreads();
        if (threadIdx.x == 0) carry += all;
        __syncthreads();
    }
}

// Moves a workgroup's keys to their places, in rounds of kBlock keys so that
// equal digits keep their order: a key's place is its bin's next free one,
// plus the equal digits of earlier waves in the round, plus those of earlier
// lanes in its wave.
__global__ __launch_bounds__(kBlock) void sort_move(const LookupGradArgs a, int src, int shift, int bits, int first,
                                                    int last)
{
    constexpr int W = kBlock / 64;
    __shared__ uint32_t next[kSortBins];
    __shared__ uint32_t mine[W][kSortBins];
    const int nb = 1 << bits, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < nb; i += kBlock) {
        next[i] = a.hist[static_cast<uint64_t>(i) * gridDim.x + blockIdx.x];
#pragma unroll
        for (int w = 0; w < W; ++w) mine[w][i] = 0;
    }
    const uint64_t lo = static_cast<uint64_t>(blockIdx.x) * kSortBlockKeys;
    for (int k = 0; k < kSortBlockKeys && lo + k < a.ntokens; k += kBlock) {
        __syncthreads();
        const uint64_t t = lo + k + threadIdx.x;
        const bool ok = t < a.ntokens;
        uint32_t key = 0, pos = 0;
        if (ok) {
            key = first ? static_cast<uint32_t>(row_of(a.tokens, t, a.first_row, a.rows)) : a.key[src][t];
            pos = first ? static_cast<uint32_t>(t) : a.pos[src][t];
        }
        const uint32_t digit = (key >> shift) & (nb - 1);
        uint64_t same = __ballot(ok);
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot((digit >> b) & 1);
            same &= ((digit >> b) & 1) ? m : ~m;
        }
        const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
        if (ok && rank == 0) mine[wave][digit] = __popcll(same);
        __syncthreads();
        if (ok) {
            uint32_t to = next[digit] + rank;
            for (int w = 0; w < wave; ++w) to += mine[w][digit];
            a.key[src ^ 1][to] = key;
            a.pos[src ^ 1][to] = pos;
            if (last && key < a.rows) atomicOr(&a.present[key >> 5], 1u << (key & 31));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nb; i += kBlock) {
            uint32_t add = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                add += mine[w][i];
                mine[w][i] = 0;
            }
            next[i] += add;
        }
    }
}

// ---------------------------------------------------------------------------
// sums over runs of equal rows
// ---------------------------------------------------------------------------
// U consecutive elements of a row: a 16-byte vector of the narrower of the
// two types, or one element.
template <class G, int U>
__device__ __forceinline__ void put_row(const LookupGradArgs& a, uint64_t row, uint64_t c, const float* acc)
{
    const uint64_t at = row * a.ld_grad_weight + c;
    float x[U];
#pragma unroll
    for (int j = 0; j < U; ++j) x[j] = acc[j] * a.scale;
    if constexpr (U == 1) {
        if (a.accumulate) x[0] += G::ld(a.grad_weight, at);
        G::st(a.grad_weight, at, x[0]);
    } else {
        constexpr int E = G::kEpv;
#pragma unroll
        for (int k = 0; k < U; k += E) {
            const uint64_t b = (at + k) * (16 / E);
            if (a.accumulate) {
                float y[E];
                G::unpack(ldv_at<false>(a.grad_weight, b), y);
#pragma unroll
                for (int j = 0; j < E; ++j) x[k + j] += y[j];
            }
            stv_at<false>(a.grad_weight, b, G::pack(x + k));
        }
    }
}

template <class F, int U>
__device__ __forceinline__ void add_row(const LookupGradArgs& a, uint64_t t, uint64_t c, float* acc)
{
    const uint64_t at = t * a.ld_grad_out + c;
    if constexpr (U == 1) {
        acc[0] += F::ld(a.grad_out, at);
    } else {
        constexpr int E = F::kEpv;
#pragma unroll
        for (int k = 0; k < U; k += E) {
            float y[E];
            F::unpack(ldv_at<false>(a.grad_out, (at + k) * (16 / E)), y);
#pragma unroll
            for (int j = 0; j < E; ++j) acc[k + j] += y[j];
        }
    }
}

// Workgroups below `chunks` sum kGradChunk positions of the sorted order each:
// a run inside the chunk is written to its row, a run that began before it or
// goes on after it leaves a partial sum (slot 0: from the chunk's start; slot
// 1: to its end). The others write zeros to the rows without tokens.
template <class F, class G, int U>
__global__ __launch_bounds__(kBlock) void grad_sum(const LookupGradArgs a, uint32_t chunks, int sorted)
{
    const uint32_t* key = a.key[sorted];
    const uint32_t* pos = a.pos[sorted];
    const uint32_t rows = static_cast<uint32_t>(a.rows);
    if (blockIdx.x < chunks) {
        const uint64_t p0 = static_cast<uint64_t>(blockIdx.x) * kGradChunk;
        const uint64_t p1 = min(p0 + kGradChunk, a.ntokens);
        const uint32_t before = p0 > 0 ? key[p0 - 1] : UINT32_MAX;
        const uint32_t after = p1 < a.ntokens ? key[p1] : UINT32_MAX;
        for (uint64_t c = static_cast<uint64_t>(threadIdx.x) * U; c < a.width; c += kBlock * U) {
            float acc[U] = {};
            uint32_t cur = key[p0];
            bool from_start = true;  // the run began at the chunk's first position
            for (uint64_t p = p0; p < p1; ++p) {
                if (cur >= rows) break;  // tokens of no row come last
                add_row<F, U>(a, pos[p], c, acc);
                const uint32_t nxt = p + 1 < p1 ? key[p + 1] : after;
                const bool ends = p + 1 == p1;
                if (nxt != cur || ends) {
                    const bool open_front = from_start && before == cur;
                    const bool open_back = ends && after == cur;
                    if (!open_front && !open_back) {
                        put_row<G, U>(a, cur, c, acc);
                    } else {
                        float* to = a.partial + (2ull * blockIdx.x + (open_front ? 0 : 1)) * a.width + c;
#pragma unroll
                        for (int j = 0; j < U; ++j) to[j] = acc[j];
                    }
#pragma unroll
                    for (int j = 0; j < U; ++j) acc[j] = 0.0f;
                    from_start = false;
                    cur = nxt;
                }
            }
        }
        return;
    }
    const float zero[U] = {};
    for (uint64_t r = blockIdx.x - chunks; r < a.rows; r += gridDim.x - chunks) {
        if ((a.present[r >> 5] >> (r & 31)) & 1) continue;
        for (uint64_t c = static_cast<uint64_t>(threadIdx.x) * U; c < a.width; c += kBlock * U)
            put_row<G, U>(a, r, c, zero);
    }
}

// Joins the partial sums of a run that goes over chunk borders, in order: one
// workgroup for each chunk in which such a run begins.
template <class G, int U>
__global__ __launch_bounds__(kBlock) void grad_join(const LookupGradArgs a, uint32_t chunks, int sorted)
{
    const uint32_t* key = a.key[sorted];
    const uint64_t p0 = static_cast<uint64_t>(blockIdx.x) * kGradChunk, p1 = p0 + kGradChunk;
    if (p1 >= a.ntokens) return;
    const uint32_t row = key[p1 - 1];
    if (row >= a.rows || key[p1] != row) return;            // no run goes on
    if (key[p0] == row && p0 > 0 && key[p0 - 1] == row) return;  // it began in an earlier chunk
    for (uint64_t c = static_cast<uint64_t>(threadIdx.x) * U; c < a.width; c += kBlock * U) {
        float acc[U];
        const float* from = a.partial + (2ull * blockIdx.x + 1) * a.width + c;
#pragma unroll
        for (int j = 0; j < U; ++j) acc[j] = from[j];
        for (uint32_t b = blockIdx.x + 1; b < chunks; ++b) {
            const uint64_t q0 = static_cast<uint64_t>(b) * kGradChunk;
            if (key[q0] != row) break;
            from = a.partial + 2ull * b * a.width + c;
#pragma unroll
            for (int j = 0; j < U; ++j) acc[j] += from[j];
        }
        put_row<G, U>(a, row, c, acc);
    }
}

template <class F, class G, int U>
hipError_t grad_launch(const LookupGradArgs& a, uint32_t chunks, int sorted, int num_cus, hipStream_t s)
{
    const uint64_t rows_wanted = a.accumulate ? 0 : a.rows;
    const uint64_t cap = static_cast<uint64_t>(num_cus) * 32;
    const uint32_t zero = static_cast<uint32_t>(rows_wanted < cap ? rows_wanted : cap);
    if (chunks + zero) hipLaunchKernelGGL((grad_sum<F, G, U>), dim3(chunks + zero), dim3(kBlock), 0, s, a, chunks, sorted);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || chunks < 2) return e;
    hipLaunchKernelGGL((grad_join<G, U>), dim3(chunks), dim3(kBlock), 0, s, a, chunks, sorted);
    return hipGetLastError();
}

template <class F, class G>
hipError_t grad_vec(const LookupGradArgs& a, bool vec, uint32_t chunks, int sorted, int num_cus, hipStream_t s)
{
    constexpr int U = F::kEpv > G::kEpv ? F::kEpv : G::kEpv;
    return vec ? grad_launch<F, G, U>(a, chunks, sorted, num_cus, s) : grad_launch<F, G, 1>(a, chunks, sorted, num_cus, s);
}

// No token: the presence bits alone.
__global__ __launch_bounds__(kBlock) void clear_present(uint32_t* present, uint64_t words)
{
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x; i < words;
         i += static_cast<uint64_t>(gridDim.x) * kBlock)
        present[i] = 0;
}

}  // namespace

hipError_t launch_lookup(const LookupArgs& a, ar_dtype_t dtype, bool vec, int num_cus, hipStream_t stream)
{
    (void)num_cus;
    switch (dtype) {
    case AR_FLOAT32: return lookup_launch<F32>(a, vec, stream);
    case AR_FLOAT16: return lookup_launch<F16>(a, vec, stream);
    case AR_BFLOAT16: return lookup_launch<BF16>(a, vec, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_lookup_grad(const LookupGradArgs& a, ar_dtype_t dtype, ar_dtype_t grad_dtype, bool vec, int num_cus,
                              hipStream_t stream)
{
    int sorted = 0;
    const uint32_t chunks = static_cast<uint32_t>((a.ntokens + kGradChunk - 1) / kGradChunk);
    if (a.ntokens) {
        const uint32_t blocks = static_cast<uint32_t>((a.ntokens + kSortBlockKeys - 1) / kSortBlockKeys);
        int bits = 1;
        while ((a.rows >> bits) != 0) ++bits;  // keys are 0..rows
        const int passes = (bits + 8) / 9, digit = (bits + passes - 1) / passes;
        for (int p = 0; p < passes; ++p) {
            const int first = p == 0, last = p == passes - 1, shift = p * digit, src = sorted;
            hipLaunchKernelGGL(sort_count, dim3(blocks), dim3(kBlock), 0, stream, a, src, shift, digit, first, last);
            hipLaunchKernelGGL(sort_scan, dim3(1), dim3(1024), 0, stream, a.hist,
                               static_cast<uint64_t>(blocks) << digit);
            hipLaunchKernelGGL(sort_move, dim3(blocks), dim3(kBlock), 0, stream, a, src, shift, digit, first, last);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            sorted ^= 1;
        }
    } else {
        hipLaunchKernelGGL(clear_present, dim3(64), dim3(kBlock), 0, stream, a.present, (a.rows + 31) / 32);
    }
    if (dtype == AR_FLOAT32) return grad_vec<F32, F32>(a, vec, chunks, sorted, num_cus, stream);
    if (dtype == AR_FLOAT16)
        return grad_dtype == AR_FLOAT32 ? grad_vec<F16, F32>(a, vec, chunks, sorted, num_cus, stream)
                                        : grad_vec<F16, F16>(a, vec, chunks, sorted, num_cus, stream);
    return grad_dtype == AR_FLOAT32 ? grad_vec<BF16, F32>(a, vec, chunks, sorted, num_cus, stream)
                                    : grad_vec<BF16, BF16>(a, vec, chunks, sorted, num_cus, stream);
}

}  // namespace lm
}  // namespace ar
