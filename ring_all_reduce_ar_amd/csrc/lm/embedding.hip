// embedding.hip -- the embedding lookup, and its gradient by sorted tokens.
//
//   out[t] = round(scale * W[token[t] - first_row]), zero where that row is not here
//   dW[v]  = round(scale * sum over {t : token[t] - first_row = v}, t ascending, of dout[t])
//
// The gradient sorts the tokens (stable radix sort), so that a row's
// contributions lie side by side in token order: each row is summed in fp32 in
// one fixed order and written once, with no float atomics, and the rows that no
// token meets are written as zeros in the same launch.
#include <algorithm>

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

// Sixteen bytes at any address (a row of odd width starts anywhere): the
// hardware takes a vector access at an element's alignment.
__device__ __forceinline__ u32x4 load16(const void* base, uint64_t byte)
{
    u32x4 v;
    __builtin_memcpy(&v, gptr<char>(base) + byte, 16);
    return v;
}
__device__ __forceinline__ void store16(void* base, uint64_t byte, u32x4 v)
{
    __builtin_memcpy(gptr<char>(base) + byte, &v, 16);
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
// `lanes` (a power of two up to kBlock) threads a row, kBlock / lanes rows a
// workgroup, 16 bytes a thread and what is left of a row by elements. Stores are
// cached: with non-temporal ones 16384 x 4096 fp16 returns in 26 us rather than
// 43, but what reads the rows next takes the time instead, 79 against 81 us for
// both. Rows that do not lie on 16 bytes: 16384 x 4093 fp16 in 58 us, where
// elements take 101.
template <class F>
__global__ __launch_bounds__(kBlock) void lookup(const LookupArgs a, int lanes)
{
    constexpr int E = F::kEpv, EB = 16 / E;
    const int per = kBlock / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    for (uint64_t t = static_cast<uint64_t>(blockIdx.x) * per + threadIdx.x / lanes; t < a.ntokens;
         t += static_cast<uint64_t>(gridDim.x) * per) {
        const uint64_t row = row_of(a.tokens, t, a.first_row, a.rows);
        const bool here = row < a.rows;
        const uint64_t src = (here ? row : 0) * a.ld_weight, dst = t * a.ld_out;
        for (uint64_t c = static_cast<uint64_t>(lane) * E; c < a.width; c += static_cast<uint64_t>(lanes) * E) {
            if (c + E <= a.width) {
                float x[E];
                u32x4 v = {0, 0, 0, 0};
                if (here) v = load16(a.weight, (src + c) * EB);
                F::unpack(v, x);
#pragma unroll
                for (int j = 0; j < E; ++j) x[j] = here ? x[j] * a.scale : 0.0f;
                store16(a.out, (dst + c) * EB, F::pack(x));
            } else {
                for (uint64_t k = c; k < a.width; ++k) F::st(a.out, dst + k, here ? F::ld(a.weight, src + k) * a.scale : 0.0f);
            }
        }
    }
}

template <class F>
hipError_t lookup_launch(const LookupArgs& a, hipStream_t s)
{
    const uint64_t units = (a.width + F::kEpv - 1) / F::kEpv;
    int lanes = 1;
    while (lanes < kBlock && static_cast<uint64_t>(lanes) < units) lanes *= 2;
    const uint64_t per = kBlock / lanes;
    const uint64_t want = (a.ntokens + per - 1) / per;
    const int grid = static_cast<int>(want < (1u << 20) ? want : (1u << 20));
    hipLaunchKernelGGL((lookup<F>), dim3(grid), dim3(kBlock), 0, s, a, lanes);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// zeros for the rows that no token meets
// ---------------------------------------------------------------------------
// Rows [r0, r1) for which `met` is false, by `blocks` workgroups of THREADS
// threads, of which this is the `block`-th; `lanes` (a power of two) threads a
// row, kFillRows neighbouring rows one after the other. Any alignment: 16-byte
// stores from the row's first boundary on. Beyond the last-level cache (NT)
// non-temporal stores leave it to the gradient's rows: 131072 x 4096 bf16 with
// 32768 tokens 289 us, with cached stores 305.
constexpr int kFillRows = 4;
template <class G, bool NT, int THREADS, class Met>
__device__ __forceinline__ void fill_rows(const LookupGradArgs& a, uint64_t r0, uint64_t r1, uint32_t block,
                                          uint32_t blocks, uint32_t lanes, Met met)
{
    constexpr uint32_t EB = 16 / G::kEpv;
    const uint32_t lane = threadIdx.x & (lanes - 1), per = THREADS / lanes;
    constexpr int B = kFillRows;
    for (uint64_t r = r0 + static_cast<uint64_t>(block) * per * B + threadIdx.x / lanes; r < r1;
         r += static_cast<uint64_t>(blocks) * per * B) {
        bool skip[B];
#pragma unroll
        for (int k = 0; k < B; ++k) skip[k] = r + k * per >= r1 || met(r + k * per);
#pragma unroll
        for (int k = 0; k < B; ++k) {
            if (skip[k]) continue;
            char* row = static_cast<char*>(a.grad_weight) + (r + k * per) * a.ld_grad_weight * EB;
            const uint64_t bytes = a.width * EB, to_line = -reinterpret_cast<uintptr_t>(row) & 15;
            const uint64_t head = to_line < bytes ? to_line : bytes, body = (bytes - head) / 16, tail = head + body * 16;
            for (uint64_t v = lane; v < body; v += lanes) stv_at<NT>(row + head, v * 16, u32x4{0, 0, 0, 0});
            for (uint64_t b = lane * EB; b < head + (bytes - tail); b += lanes * EB)
                G::st(row + (b < head ? b : tail + (b - head)), 0, 0.0f);
        }
    }
}

// ---------------------------------------------------------------------------
// stable radix sort of the tokens' rows, least significant digit first
// ---------------------------------------------------------------------------
// At most kSortBlocks workgroups take `rounds` rounds of kSortThreads keys
// each. hist[pass][block][digit] counts the keys of a workgroup; those of the
// first pass come from the tokens, those of a later one are counted (whole
// numbers, in any order) by the pass before as it moves keys to that
// workgroup's range. So a pass is one launch: each workgroup sums the counts
// that lie before its own by itself, 512 columns of at most 128.
__global__ __launch_bounds__(kSortThreads) void sort_count(const LookupGradArgs a, uint32_t rounds, int bits)
{
    __shared__ uint32_t bins[kSortBins];
    const int nb = 1 << bits;
    for (int i = threadIdx.x; i < nb; i += kSortThreads) bins[i] = 0;
    __syncthreads();
    const uint64_t lo = static_cast<uint64_t>(blockIdx.x) * rounds * kSortThreads;
    for (uint32_t k = 0; k < rounds; ++k) {
        const uint64_t t = lo + k * kSortThreads + threadIdx.x;
        if (t >= a.ntokens) break;
        const uint32_t key = static_cast<uint32_t>(row_of(a.tokens, t, a.first_row, a.rows));
        atomicAdd(&bins[key & (nb - 1)], 1u);
        if (key < a.rows) a.present[key] = 1;  // by any number of threads
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nb; i += kSortThreads) a.hist[blockIdx.x * kSortBins + i] = bins[i];
}

// Moves a workgroup's keys to their places, in rounds so that equal digits keep
// their order: a key's place is its digit's next free one, plus the equal
// digits of earlier waves in the round, plus those of earlier lanes in its
// wave. Workgroups from `blocks` on write zeros to a part of the rows without
// tokens: the few that sort leave most of the chip idle.
template <class G, bool NT>
__global__ __launch_bounds__(kSortThreads) void sort_move(const LookupGradArgs a, uint32_t blocks, uint32_t rounds,
                                                          int pass, int shift, int bits, int last, uint64_t r0,
                                                          uint64_t r1, uint32_t lanes)
{
    constexpr int W = kSortThreads / 64;
    __shared__ uint32_t next[kSortBins];
    __shared__ uint32_t mine[W][kSortBins];
    __shared__ uint32_t sums[kSortBins / 64];
    if (blockIdx.x >= blocks) {
        fill_rows<G, NT, kSortThreads>(a, r0, r1, blockIdx.x - blocks, gridDim.x - blocks, lanes,
                                       [&](uint64_t r) { return a.present[r] != 0; });
        return;
    }
    const int nb = 1 << bits, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, src = pass & 1;
    const uint32_t* hist = a.hist + static_cast<uint64_t>(pass) * kSortBlocks * kSortBins;
    uint32_t* hist_next = a.hist + static_cast<uint64_t>(pass + 1) * kSortBlocks * kSortBins;
    {
        // the keys of smaller digits, and those of this digit in earlier workgroups
        const int d = threadIdx.x;
        uint32_t before = 0, all = 0, upto = 0;
        if (d < kSortBins) {
            if (d < nb) {
#pragma unroll 8
                for (uint32_t b = 0; b < blocks; ++b) {
                    const uint32_t c = hist[b * kSortBins + d];
                    all += c;
                    if (b < blockIdx.x) before += c;
                }
            }
            upto = all;
#pragma unroll
            for (int k = 1; k < 64; k *= 2) {
                const uint32_t o = __shfl_up(upto, k, 64);
                if (lane >= k) upto += o;
            }
            if (lane == 63) sums[wave] = upto;
        }
        for (int i = threadIdx.x; i < W * kSortBins; i += kSortThreads) (&mine[0][0])[i] = 0;
        __syncthreads();
        if (d < kSortBins) {
            uint32_t base = upto - all + before;
            for (int w = 0; w < wave; ++w) base += sums[w];
            next[d] = base;
        }
    }
    const uint64_t lo = static_cast<uint64_t>(blockIdx.x) * rounds * kSortThreads;
    for (uint32_t k = 0; k < rounds && lo + k * kSortThreads < a.ntokens; ++k) {
        const uint64_t t = lo + k * kSortThreads + threadIdx.x;
        const bool ok = t < a.ntokens;
        uint32_t key = 0, pos = 0;
        if (ok) {
            key = pass == 0 ? static_cast<uint32_t>(row_of(a.tokens, t, a.first_row, a.rows)) : a.key[src][t];
            pos = pass == 0 ? static_cast<uint32_t>(t) : a.pos[src][t];
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
        uint32_t to = 0;
        if (ok) {
            to = next[digit] + rank;
            for (int w = 0; w < wave; ++w) to += mine[w][digit];
            a.key[src ^ 1][to] = key;
            a.pos[src ^ 1][to] = pos;
        }
        if (!last) {
            // Counts for the next pass, one addition for a wave's keys of equal
            // digits that go to one workgroup's range: a frequent token's keys
            // would meet at one address one by one.
            const uint32_t digit_next = (key >> (shift + bits)) & (nb - 1), block = to / (rounds * kSortThreads);
            for (int b = 0; b < bits; ++b) {
                const uint64_t m = __ballot((digit_next >> b) & 1);
                same &= ((digit_next >> b) & 1) ? m : ~m;
            }
            const int leader = same ? __builtin_ctzll(same) : lane;
            const bool with = __shfl(block, leader, 64) == block;
            const uint64_t group = __ballot(with) & same;
            uint32_t* at = &hist_next[block * kSortBins + digit_next];
            if (ok && lane == leader) atomicAdd(at, static_cast<uint32_t>(__popcll(group)));
            else if (ok && !with) atomicAdd(at, 1u);
        }
        if (k + 1 == rounds) break;
        __syncthreads();
        for (int i = threadIdx.x; i < nb; i += kSortThreads) {
            uint32_t add = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                add += mine[w][i];
                mine[w][i] = 0;
            }
            next[i] += add;
        }
        __syncthreads();
    }
}

// The same for at most kSortThreads tokens, one a thread: all passes in one
// workgroup's LDS. 7 tokens into 2996 x 32: 22 us a call with the launches of the
// general sort, 12 with this one and grad_small; 836 into 30274 x 32: 37 and 30.
__global__ __launch_bounds__(kSortThreads) void sort_small(const LookupGradArgs a, int passes, int bits)
{
    constexpr int W = kSortThreads / 64;
    __shared__ uint32_t mine[W][kSortBins];
    __shared__ uint32_t base[kSortBins];
    __shared__ uint32_t sums[kSortBins / 64];
    __shared__ uint32_t keys[kSortThreads], places[kSortThreads];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, nb = 1 << bits;
    const bool ok = static_cast<uint64_t>(t) < a.ntokens;
    uint32_t key = ok ? static_cast<uint32_t>(row_of(a.tokens, t, a.first_row, a.rows)) : 0, pos = t;
    for (int pass = 0; pass < passes; ++pass) {
        for (int i = t; i < W * kSortBins; i += kSortThreads) (&mine[0][0])[i] = 0;
        __syncthreads();
        const uint32_t digit = (key >> (pass * bits)) & (nb - 1);
        uint64_t same = __ballot(ok);
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot((digit >> b) & 1);
            same &= ((digit >> b) & 1) ? m : ~m;
        }
        const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
        if (ok && rank == 0) mine[wave][digit] = __popcll(same);
        __syncthreads();
        uint32_t all = 0, upto = 0;
        if (t < kSortBins) {
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const uint32_t c = mine[w][t];
                mine[w][t] = all;
                all += c;
            }
            upto = all;
#pragma unroll
            for (int k = 1; k < 64; k *= 2) {
                const uint32_t o = __shfl_up(upto, k, 64);
                if (lane >= k) upto += o;
            }
            if (lane == 63) sums[wave] = upto;
        }
        __syncthreads();
        if (t < kSortBins) {
            uint32_t before = upto - all;
            for (int w = 0; w < wave; ++w) before += sums[w];
            base[t] = before;
        }
        __syncthreads();
        if (ok) {
            const uint32_t to = base[digit] + mine[wave][digit] + rank;
            keys[to] = key;
            places[to] = pos;
        }
        __syncthreads();
        if (ok) {
            key = keys[t];
            pos = places[t];
        }
        __syncthreads();
    }
    if (ok) {
        a.key[0][t] = key;
        a.pos[0][t] = pos;
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
__device__ __forceinline__ void get_row(const LookupGradArgs& a, uint64_t t, uint64_t c, float* x)
{
    const uint64_t at = t * a.ld_grad_out + c;
    if constexpr (U == 1) {
        x[0] = F::ld(a.grad_out, at);
    } else {
        constexpr int E = F::kEpv;
#pragma unroll
        for (int k = 0; k < U; k += E) F::unpack(ldv_at<false>(a.grad_out, (at + k) * (16 / E)), x + k);
    }
}

// `lanes` threads (a power of two, at least kGradLanes) sum a chunk of K
// positions of the sorted order over U columns: a run inside the chunk is
// written to its row, a run that began before it or goes on after it leaves a
// partial sum (slot 0: from the chunk's start; slot 1: to its end). Eight rows
// are loaded together and added in order.
template <class F, class G, int U, int K>
__device__ __forceinline__ void sum_chunks(const LookupGradArgs& a, uint32_t chunks, int sorted, uint32_t lanes,
                                           uint32_t block, uint32_t slice)
{
    constexpr int B = 8;
    __shared__ uint32_t keys[kBlock / kGradLanes][K + 2];  // the one before the chunk, its own, the one after
    __shared__ uint32_t places[kBlock / kGradLanes][K];
    const uint32_t rows = static_cast<uint32_t>(a.rows), per = kBlock / lanes;
    const uint64_t first = static_cast<uint64_t>(block) * per * K;  // the workgroup's first position
    for (uint32_t i = threadIdx.x; i < per * (K + 2); i += kBlock) {
        const uint32_t g = i / (K + 2), k = i % (K + 2);
        const uint64_t p = first + static_cast<uint64_t>(g) * K + k;  // one past the place
        const bool in = p >= 1 && p <= a.ntokens;
        keys[g][k] = in ? a.key[sorted][p - 1] : UINT32_MAX;
        if (k >= 1 && k <= K) places[g][k - 1] = in ? a.pos[sorted][p - 1] : 0;
    }
    __syncthreads();
    const uint32_t group = threadIdx.x / lanes, chunk = block * per + group;
    const uint64_t c = (static_cast<uint64_t>(slice) * lanes + (threadIdx.x & (lanes - 1))) * U;
    if (chunk >= chunks || c >= a.width) return;
    const uint32_t* key = &keys[group][1];
    const uint32_t* pos = places[group];
    float acc[U] = {};
    bool from_start = true;  // the run began at the chunk's first position
    for (int p = 0; p < K && key[p] < rows; p += B) {  // tokens of no row come last
        float x[B][U];  // loaded whether they count or not: under a branch each load would be waited for by itself
#pragma unroll
        for (int k = 0; k < B; ++k) get_row<F, U>(a, pos[p + k], c, x[k]);
        uint32_t at[B + 1];
#pragma unroll
        for (int k = 0; k <= B; ++k) at[k] = key[p + k];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const uint32_t cur = at[k], nxt = at[k + 1];
            if (cur >= rows) break;
#pragma unroll
            for (int j = 0; j < U; ++j) acc[j] += x[k][j];
            if (nxt == cur && p + k + 1 < K) continue;
            const bool open_front = from_start && key[-1] == cur, open_back = nxt == cur;
            if (!open_front && !open_back) {
                put_row<G, U>(a, cur, c, acc);
            } else {
                float* to = a.partial + (2ull * chunk + (open_front ? 0 : 1)) * a.width + c;
#pragma unroll
                for (int j = 0; j < U; ++j) to[j] = acc[j];
            }
#pragma unroll
            for (int j = 0; j < U; ++j) acc[j] = 0.0f;
            from_start = false;
        }
    }
}

// `base`: the workgroups of earlier launches, here and below (see in_launches).
template <class F, class G, int U, int K>
__global__ __launch_bounds__(kBlock) void grad_sum(const LookupGradArgs a, uint32_t base, uint32_t chunks, int sorted,
                                                   uint32_t lanes, uint32_t bx)
{
    const uint32_t id = base + blockIdx.x;
    sum_chunks<F, G, U, K>(a, chunks, sorted, lanes, id % bx, id / bx);
}

// The sums and the zeros of at most kSortThreads tokens: the first bx * by
// workgroups sum, the others fill the rows that are not among the sorted keys.
template <class F, class G, int U, bool NT>
__global__ __launch_bounds__(kBlock) void grad_small(const LookupGradArgs a, uint32_t base, uint32_t chunks,
                                                     uint32_t lanes, uint32_t bx, uint32_t by, uint32_t fillers,
                                                     uint32_t fill_lanes)
{
    const uint32_t id = base + blockIdx.x;
    if (id < bx * by) {
        sum_chunks<F, G, U, kGradChunkFew>(a, chunks, 0, lanes, id % bx, id / bx);
        return;
    }
    __shared__ uint32_t keys[kSortThreads];
    const uint32_t n = static_cast<uint32_t>(a.ntokens);
    for (uint32_t i = threadIdx.x; i < n; i += kBlock) keys[i] = a.key[0][i];
    __syncthreads();
    fill_rows<G, NT, kBlock>(a, 0, a.rows, id - bx * by, fillers, fill_lanes, [&](uint64_t r) {
        uint32_t lo = 0, hi = n;  // the first key that is not below r
        while (lo < hi) {
            const uint32_t mid = (lo + hi) / 2;
            if (keys[mid] < r) lo = mid + 1;
            else hi = mid;
        }
        return lo < n && keys[lo] == r;
    });
}

// Joins the partial sums of a run that goes over chunk borders, in order:
// `lanes` threads for each chunk of `len` positions in which such a run begins.
// Sixteen chunks' keys and sums are loaded together, whether the run goes on
// over all of them or not (the most frequent token of a text has a tenth of all
// positions).
template <class G, int U>
__global__ __launch_bounds__(kBlock) void grad_join(const LookupGradArgs a, uint32_t base, uint32_t chunks, uint32_t len,
                                                    int sorted, uint32_t lanes, uint32_t bx)
{
    constexpr int B = 16;
    const uint32_t* key = a.key[sorted];
    const uint32_t id = base + blockIdx.x, chunk = id % bx * (kBlock / lanes) + threadIdx.x / lanes;
    const uint64_t c = (static_cast<uint64_t>(id / bx) * lanes + (threadIdx.x & (lanes - 1))) * U;
    const uint64_t p0 = static_cast<uint64_t>(chunk) * len, p1 = p0 + len;
    if (p1 >= a.ntokens || c >= a.width) return;
    const uint32_t row = key[p1 - 1];
    if (row >= a.rows || key[p1] != row) return;                 // no run goes on
    if (key[p0] == row && p0 > 0 && key[p0 - 1] == row) return;  // it began in an earlier chunk
    float acc[U];
    const float* from = a.partial + (2ull * chunk + 1) * a.width + c;
#pragma unroll
    for (int j = 0; j < U; ++j) acc[j] = from[j];
    for (uint32_t b = chunk + 1, on = 1; on; b += B) {
        uint32_t at[B];
        float x[B][U];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const uint32_t q = min(b + k, chunks - 1);
            at[k] = key[static_cast<uint64_t>(q) * len];
            from = a.partial + 2ull * q * a.width + c;
#pragma unroll
            for (int j = 0; j < U; ++j) x[k][j] = from[j];
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            on = on && b + k < chunks && at[k] == row;
            if (!on) continue;
#pragma unroll
            for (int j = 0; j < U; ++j) acc[j] += x[k][j];
        }
    }
    put_row<G, U>(a, row, c, acc);
}

// The presence flags and the counts that the sort adds to.
__global__ __launch_bounds__(kBlock) void clear_words(uint32_t* words, uint64_t n)
{
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n;
         i += static_cast<uint64_t>(gridDim.x) * kBlock)
        words[i] = 0;
}

template <class G, bool NT>
__global__ __launch_bounds__(kSortThreads) void fill_all(const LookupGradArgs a, uint32_t lanes)
{
    fill_rows<G, NT, kSortThreads>(a, 0, a.rows, blockIdx.x, gridDim.x, lanes, [](uint64_t) { return false; });
}

uint32_t lanes_for(uint64_t units, uint32_t least, uint32_t most)
{
    uint32_t lanes = least;
    while (lanes < most && lanes < units) lanes *= 2;
    return lanes;
}

// Workgroups that fill the rows of the matrix, THREADS threads each, and the
// threads of one row.
template <class G>
void fill_shape(const LookupGradArgs& a, uint32_t threads, int num_cus, uint32_t* blocks, uint32_t* lanes)
{
    *lanes = lanes_for((a.width * (16 / G::kEpv) + 15) / 16, 1, 256);
    const uint64_t each = threads / *lanes * kFillRows, wanted = (a.rows + each - 1) / each;
    *blocks = static_cast<uint32_t>(std::min<uint64_t>(wanted, static_cast<uint64_t>(num_cus) * 8 * (kSortThreads / threads)));
}

// Sorts the tokens and fills; *sorted tells in which of the buffers they end.
template <class G, bool NT>
hipError_t sort_and_fill(const LookupGradArgs& a, int* sorted, int num_cus, hipStream_t s)
{
    uint32_t fillers, lanes;
    fill_shape<G>(a, kSortThreads, num_cus, &fillers, &lanes);
    const uint64_t clearers = (a.clear_words + kBlock - 1) / kBlock;
    hipLaunchKernelGGL(clear_words, dim3(static_cast<uint32_t>(std::min<uint64_t>(clearers, 1024))), dim3(kBlock), 0, s,
                       reinterpret_cast<uint32_t*>(a.present), a.clear_words);
    const uint64_t all = (a.ntokens + kSortThreads - 1) / kSortThreads;
    const uint32_t rounds = static_cast<uint32_t>((all + kSortBlocks - 1) / kSortBlocks);
    const uint32_t blocks = static_cast<uint32_t>((all + rounds - 1) / rounds);
    const int passes = sort_passes(a.rows), bits = (sort_bits(a.rows) + passes - 1) / passes;
    hipLaunchKernelGGL(sort_count, dim3(blocks), dim3(kSortThreads), 0, s, a, rounds, bits);
    for (int p = 0; p < passes; ++p) {
        const uint64_t r0 = a.rows * p / passes, r1 = a.rows * (p + 1) / passes;
        hipLaunchKernelGGL((sort_move<G, NT>), dim3(blocks + (a.accumulate ? 0 : fillers)), dim3(kSortThreads), 0, s, a,
                           blocks, rounds, p, p * bits, bits, p == passes - 1, r0, r1, lanes);
    }
    *sorted = passes & 1;
    return hipGetLastError();
}

// Launches `blocks` workgroups in parts whose work-items are counted in 32 bits:
// launch(base, part).
template <class Launch>
hipError_t in_launches(uint64_t blocks, const Launch& launch)
{
    constexpr uint64_t most = (uint64_t(1) << 32) / kBlock - 1;
    if (blocks > UINT32_MAX) return hipErrorInvalidValue;  // more bytes of partial sums than a device has
    for (uint64_t base = 0; base < blocks; base += most)
        launch(static_cast<uint32_t>(base), dim3(static_cast<uint32_t>(std::min(blocks - base, most))));
    return hipGetLastError();
}

template <class F, class G, int U, bool NT>
hipError_t grad_launch(const LookupGradArgs& a, int num_cus, hipStream_t s)
{
    if (a.ntokens == 0) {
        uint32_t fillers, fill_lanes;
        fill_shape<G>(a, kSortThreads, num_cus, &fillers, &fill_lanes);
        hipLaunchKernelGGL((fill_all<G, NT>), dim3(fillers), dim3(kSortThreads), 0, s, a, fill_lanes);
        return hipGetLastError();
    }
    const uint32_t len = grad_chunk(a.ntokens), chunks = static_cast<uint32_t>((a.ntokens + len - 1) / len);
    const uint64_t units = (a.width + U - 1) / U;
    const uint32_t lanes = lanes_for(units, kGradLanes, kBlock), per = kBlock / lanes;
    // bx workgroups along the chunks, times the slices of a row
    const uint32_t bx = (chunks + per - 1) / per, by = static_cast<uint32_t>((units + lanes - 1) / lanes);
    const uint64_t blocks = static_cast<uint64_t>(bx) * by;
    int sorted = 0;
    hipError_t e;
    if (a.ntokens <= kSortThreads) {
        const int passes = sort_passes(a.rows), bits = (sort_bits(a.rows) + passes - 1) / passes;
        hipLaunchKernelGGL(sort_small, dim3(1), dim3(kSortThreads), 0, s, a, passes, bits);
        uint32_t fillers, fill_lanes;
        fill_shape<G>(a, kBlock, num_cus, &fillers, &fill_lanes);
        if (a.accumulate) fillers = 0;
        e = in_launches(blocks + fillers, [&](uint32_t base, dim3 part) {
            hipLaunchKernelGGL((grad_small<F, G, U, NT>), part, dim3(kBlock), 0, s, a, base, chunks, lanes, bx, by, fillers,
                               fill_lanes);
        });
    } else {
        if ((e = sort_and_fill<G, NT>(a, &sorted, num_cus, s)) != hipSuccess) return e;
        e = in_launches(blocks, [&](uint32_t base, dim3 part) {
            if (len == kGradChunkFew)
                hipLaunchKernelGGL((grad_sum<F, G, U, kGradChunkFew>), part, dim3(kBlock), 0, s, a, base, chunks, sorted,
                                   lanes, bx);
            else
                hipLaunchKernelGGL((grad_sum<F, G, U, kGradChunk>), part, dim3(kBlock), 0, s, a, base, chunks, sorted,
                                   lanes, bx);
        });
    }
    if (e != hipSuccess || chunks == 1) return e;
    return in_launches(blocks, [&](uint32_t base, dim3 part) {
        hipLaunchKernelGGL((grad_join<G, U>), part, dim3(kBlock), 0, s, a, base, chunks, len, sorted, lanes, bx);
    });
}

// Rows that do not lie on 16 bytes are summed by elements: by vectors at any
// address 23784 x 3549 bf16 takes 108 us rather than 99, 8191 x 1027 74 rather
// than 69.
template <class F, class G>
hipError_t grad_call(const LookupGradArgs& a, bool vec, bool nt, int num_cus, hipStream_t s)
{
    constexpr int U = F::kEpv > G::kEpv ? F::kEpv : G::kEpv;
    if (nt) return vec ? grad_launch<F, G, U, true>(a, num_cus, s) : grad_launch<F, G, 1, true>(a, num_cus, s);
    return vec ? grad_launch<F, G, U, false>(a, num_cus, s) : grad_launch<F, G, 1, false>(a, num_cus, s);
}

}  // namespace

hipError_t launch_lookup(const LookupArgs& a, ar_dtype_t dtype, hipStream_t stream)
{
    switch (dtype) {
    case AR_FLOAT32: return lookup_launch<F32>(a, stream);
    case AR_FLOAT16: return lookup_launch<F16>(a, stream);
    case AR_BFLOAT16: return lookup_launch<BF16>(a, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_lookup_grad(const LookupGradArgs& a, ar_dtype_t dtype, ar_dtype_t grad_dtype, bool vec, bool nt,
                              int num_cus, hipStream_t stream)
{
    if (dtype == AR_FLOAT32) return grad_call<F32, F32>(a, vec, nt, num_cus, stream);
    if (dtype == AR_FLOAT16)
        return grad_dtype == AR_FLOAT32 ? grad_call<F16, F32>(a, vec, nt, num_cus, stream)
                                        : grad_call<F16, F16>(a, vec, nt, num_cus, stream);
    return grad_dtype == AR_FLOAT32 ? grad_call<BF16, F32>(a, vec, nt, num_cus, stream)
                                    : grad_call<BF16, BF16>(a, vec, nt, num_cus, stream);
}

}  // namespace lm
}  // namespace ar
