// log_probs.h -- log probabilities under a linear head: what cross_entropy.hip's
// products need beyond the loss.
//
//   z[t][v] = s x[t] . w[v],  lse[t] = log sum_v exp z[t][v],  lp[t] = z[t][y[t]] - lse[t]
//   H[t] = -sum_v p log p = log S - (sum_v e^u u) / S,  u = z - max z <= 0, S = sum_v e^u
//   dz[t][v] = s (a[t] ([v = y[t]] - p) - b[t] p (log p + H[t])),  a, b the gradients of lp and H
//
// Both terms of H are at least 0, so nothing cancels. A wave's part of a row is
// a group of neighbouring vocabulary rows, whose maximum the softmax needs
// anyway: the `top` largest logits lie in the `top` groups of largest maxima
// (the first of equal ones first), so alternatives cost one store of the logits
// and a read of those groups alone.
#pragma once

#include <type_traits>

#include "head.h"

namespace ar {
namespace lm {
namespace {

// ---------------------------------------------------------------------------
// logits of few tokens from rows at any address
// ---------------------------------------------------------------------------
// Direct loads to LDS want rows on 16 bytes. For up to 16 tokens a row of A is one
// wave's alone and need not go through LDS: each lane loads its fragments, 16 bytes
// at an element's alignment, kRowsAhead of them under way, and only the tokens'
// rows, laid out as gemm_few has them, lie in LDS, all of their depth (which bounds
// it). Laying the weight out first moves it three times: forward, us, by that and so,
// 3 tokens x 88513 x 1157 bf16 149 / 75 (this kernel 66, 3.1 TB/s), 16 x 50000 x 3001
// fp16 with 5 alternatives 239 / 152, 1 x 131072 x 999 fp32 437 / 102. With 4 / 8 / 16
// loads under way the first takes 76 / 76 / 88 and the last 107 / 103 / 102.
constexpr int kRowsThreads = 512, kRowsAhead = 8;
constexpr uint32_t kRowsLds = 144 * 1024;

// The tokens' rows in LDS, 16 bytes apart from whole 128s.
__host__ __device__ constexpr uint64_t rows_pitch(uint64_t depth_bytes) { return (depth_bytes + 127) / 128 * 128 + 16; }
constexpr bool rows_fit(uint64_t depth_bytes) { return 16 * rows_pitch(depth_bytes) <= kRowsLds; }

// g.k_all: the width; g.b: rows of whole 128-byte steps, zeros behind the width.
template <class T, class Epilogue>
__global__ __launch_bounds__(kRowsThreads) void gemm_rows(const GemmArgs g, const Epilogue epi)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr uint32_t EB = sizeof(typename T::Elem), kEach = 16 / EB;
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t bytes = g.k_all * EB, steps = bytes / 64, pitch = static_cast<uint32_t>(rows_pitch(bytes));
    const uint32_t chunks = (bytes + 127) / 128 * 8;
    for (uint32_t i = threadIdx.x; i < 16 * chunks; i += kRowsThreads) {
        const uint32_t row = i / chunks, at = i % chunks * 16;
        const u32x4 none = {0, 0, 0, 0};
        *reinterpret_cast<u32x4*>(lds + row * pitch + at) =
            row < g.n ? *reinterpret_cast<const u32x4*>(g.b + row * g.ldb + at) : none;
    }
    __syncthreads();

    // two tiles of 64 rows a workgroup, as gemm_few numbers them
    const uint32_t tm = blockIdx.x * 2 + (wave >> 2), m0 = tm * kFewM + (wave & 3) * 16;
    const uint32_t row = min(m0 + (lane & 15), g.m - 1), col = (lane >> 4) * 16;
    const char *a = g.a + row * g.lda, *b = lds + (lane & 15) * pitch + col;
    auto load = [&](uint32_t step) {
        i32x4 v;
        __builtin_memcpy(&v, a + min(step, steps - 1) * 64 + col, 16);
        return v;
    };
    Tile<1, 1> acc;
    acc.v[0][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](i32x4 x, uint32_t step) {
        const i32x4 y = *reinterpret_cast<const i32x4*>(b + step * 64);
        acc.v[0][0] = T::mma(__builtin_bit_cast(typename T::Frag, x), __builtin_bit_cast(typename T::Frag, y), acc.v[0][0]);
    };
    if (steps) {
        i32x4 f[kRowsAhead];
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) f[i] = load(i);
        uint32_t k = 0;
        for (; k + kRowsAhead <= steps; k += kRowsAhead)
#pragma unroll
            for (int i = 0; i < kRowsAhead; ++i) {
                const i32x4 x = f[i];
                f[i] = load(k + i + kRowsAhead);
                multiply(x, k + i);
            }
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i)
            if (k + i < steps) multiply(f[i], k + i);
    }
    if (steps * 64 < bytes) {  // what is left of the rows
        typename T::Elem x[kEach] = {};
        const uint32_t at = steps * 64 + col;
#pragma unroll
        for (uint32_t e = 0; e < kEach; ++e)
            if (at + e * EB < bytes) __builtin_memcpy(&x[e], a + at + e * EB, EB);
        i32x4 v;
        __builtin_memcpy(&v, x, 16);
        multiply(v, steps);
    }
    if (tm < g.tiles_m) epi(acc, m0, 0, g, tm * 4 + (wave & 3), 0, NoStaging{});
}

template <class T, class Epilogue>
hipError_t launch_gemm_rows(GemmArgs g, const Epilogue& epi, hipStream_t stream)
{
    g.tiles_m = (g.m + kFewM - 1) / kFewM;
    const uint32_t lds = static_cast<uint32_t>(16 * rows_pitch(g.k_all * sizeof(typename T::Elem)));
    hipLaunchKernelGGL((gemm_rows<T, Epilogue>), dim3((g.tiles_m + 1) / 2), dim3(kRowsThreads), lds, stream, g, epi);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
struct LogParts {
    float top, sum, dot;  // of u = z - top: the sums of e^u and of e^u u
};

// The logits of a chunk of tokens, kept for their alternatives: group after
// group of 16 MT vocabulary rows, in it blocks of 16 tokens, in those MT blocks
// of 16 x 16, so that one store of a wave is 1024 bytes on end.
__host__ __device__ constexpr uint64_t logit_at(uint64_t group, uint64_t token_blocks, uint64_t token, uint32_t groups_of_16,
                                                uint32_t row)
{
    return ((group * token_blocks + token / 16) * groups_of_16 + row / 16) * 256 + token % 16 * 16 + row % 16;
}

// A wave's part of each token's row, as StatsEpilogue, and its logits.
struct LogPartsEpilogue {
    LogParts* parts;      // [group][token of the chunk]
    float* target_logit;  // [token of the chunk]
    float* logits;        // or null
    Indices targets;
    int64_t ignore;
    uint64_t vocab, v0, row0;
    uint64_t first_token;
    float scale;

    template <int MT, int NT, class S>
    __device__ __forceinline__ void operator()(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const GemmArgs& g,
                                               uint32_t mrow, uint32_t, const S&) const
    {
        if (m0 + MT * 16 <= g.m) write<true>(acc, m0, n0, g, mrow);
        else write<false>(acc, m0, n0, g, mrow);
    }

private:
    template <bool FULL, int MT, int NT>
    __device__ __forceinline__ void write(Tile<MT, NT>& acc, uint32_t m0, uint32_t n0, const GemmArgs& g,
                                          uint32_t mrow) const
    {
        const int lane = threadIdx.x & 63, quad = lane >> 4;
        const uint32_t mine = m0 + quad * 4;
        const uint64_t blocks = (g.n + 15) / 16;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (n0 + j * 16 >= g.n) break;
            const uint32_t t = n0 + j * 16 + (lane & 15);
            const bool ok = t < g.n;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                acc.v[i][j] *= scale;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (FULL || mine + 16 * i + r < g.m) top = fmaxf(top, acc.v[i][j][r]);
            }
            if (logits) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    __builtin_nontemporal_store(acc.v[i][j], reinterpret_cast<f32x4*>(
                                                                 logits + logit_at(row0 + mrow, blocks, t, MT, 16 * i + quad * 4)));
            }
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float base = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (FULL || mine + 16 * i + r < g.m) {
                        const float u = acc.v[i][j][r] - base, e = __builtin_amdgcn_exp2f(u * kLog2e);
                        sum += e;
                        dot += e > 0.0f ? e * u : 0.0f;  // a logit of -infinity adds nothing
                    }
            sum += __shfl_xor(sum, 16, 64);
            dot += __shfl_xor(dot, 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            dot += __shfl_xor(dot, 32, 64);
            if (ok && quad == 0) parts[(row0 + mrow) * g.n + t] = LogParts{top, sum, dot};
            const uint32_t at =
                ok ? target_at<MT>(load_target(targets, first_token + t, ignore, vocab), v0 + mine) : kNoTarget;
            if (!__any(at != kNoTarget)) continue;  // few tiles hold a target
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (at == static_cast<uint32_t>(16 * i + r)) target_logit[t] = acc.v[i][j][r];
        }
    }
};

__device__ __forceinline__ LogParts join_parts(LogParts a, LogParts b)
{
    // (the part of nothing has the top -infinity and sums of 0)
    const float m = fmaxf(a.top, b.top), base = m == -INFINITY ? 0.0f : m;
    const float da = fmaxf(a.top - base, -1e4f), db = fmaxf(b.top - base, -1e4f);
    const float fa = __builtin_amdgcn_exp2f(da * kLog2e), fb = __builtin_amdgcn_exp2f(db * kLog2e);
    return LogParts{m, a.sum * fa + b.sum * fb, (a.dot + da * a.sum) * fa + (b.dot + db * b.sum) * fb};
}

struct LogProbOut {
    Indices targets;
    int64_t ignore;
    uint64_t vocab, first_token, ntokens;  // the chunk's tokens
    const float* target_logit;             // of the chunk
    float *log_probs, *entropy, *lse;      // of the call; entropy may be null

    // The target's logit, if it is not ignored: a kernel asks for it before
    // the rest of its work, whose loads then hide these two.
    struct Aim {
        bool on;
        float logit;
    };
    __device__ __forceinline__ Aim aim(uint64_t t) const
    {
        const bool on = load_target(targets, first_token + t, ignore, vocab) >= 0;
        return Aim{on, on ? target_logit[t] : 0.0f};
    }
    __device__ __forceinline__ void put(uint64_t t, const LogParts& s, const Aim& aim) const
    {
        const uint64_t at = first_token + t;
        const float log_sum = logf(s.sum), l = s.top + log_sum;
        lse[at] = l;
        log_probs[at] = aim.on ? aim.logit - l : 0.0f;
        if (entropy) entropy[at] = log_sum - s.dot / s.sum;
    }
};

// Joins the parts of each token's row, as join_stats.
template <int X>
__global__ __launch_bounds__(kJoinBlock) void join_log_probs(const LogParts* parts, uint64_t groups, LogProbOut out)
{
    constexpr int Y = kJoinBlock / X;
    __shared__ LogParts part[Y][X];
    const int x = threadIdx.x % X, y = threadIdx.x / X;
    const uint64_t t = static_cast<uint64_t>(blockIdx.x) * X + x;
    LogParts s{-INFINITY, 0.0f, 0.0f};
    LogProbOut::Aim aim{};
    if (t < out.ntokens) {
        if (y == 0) aim = out.aim(t);
#pragma unroll 4
        for (uint64_t r = y; r < groups; r += Y) s = join_parts(s, parts[r * out.ntokens + t]);
    }
    part[y][x] = s;
#pragma unroll
    for (int h = Y / 2; h >= 1; h /= 2) {
        __syncthreads();
        if (y < h) part[y][x] = join_parts(part[y][x], part[y + h][x]);
    }
    if (y == 0 && t < out.ntokens) out.put(t, part[0][x], aim);
}

// ---------------------------------------------------------------------------
// alternatives
// ---------------------------------------------------------------------------
// The order of alternatives as one number: the larger value first, of equal ones
// the smaller id. NaN counts as -infinity, -0 as 0; 0 is below every key.
__device__ __forceinline__ uint64_t order_key(float z, uint32_t id)
{
    const uint32_t bits = as_u(z != z ? -INFINITY : z + 0.0f);
    const uint32_t high = bits & 0x80000000u ? ~bits : bits | 0x80000000u;
    return static_cast<uint64_t>(high) << 32 | ~id;
}
__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t high = static_cast<uint32_t>(key >> 32);
    return as_f(high & 0x80000000u ? high ^ 0x80000000u : ~high);
}
__device__ __forceinline__ uint32_t key_id(uint64_t key) { return ~static_cast<uint32_t>(key); }

// The largest value of a wave, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    auto step = [&](auto dpp, auto rows) {
        const uint32_t y = __builtin_amdgcn_update_dpp(0, x, decltype(dpp)::value, decltype(rows)::value, 0xF, false);
        x = x > y ? x : y;
    };
    step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});  // the lane below in a row of 16
    step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row 0 to 1, 2 to 3
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});  // row 1 to 2 and 3
    return __builtin_amdgcn_readlane(x, 63);
}

// How many of the first `count` lanes' keys are above this lane's; the others' are 0.
__device__ __forceinline__ uint32_t rank_of(uint64_t key, uint32_t count)
{
    uint32_t rank = 0;
    auto above = [&](uint32_t i) {
        const uint64_t other = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(key >> 32, i))) << 32 |
                               static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(key), i));
        rank += other > key ? 1 : 0;
    };
    for (uint32_t i = 0; i < count; i += 8) {
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) above(i + k);
    }
    return rank;
}

// A value that at least `top` keys reach, from each lane's largest. Up to 8: the
// least of the maxima of eight sets of lanes (of their upper halves), which about
// 22 of 512 keys reach; more: the top-th largest.
__device__ __forceinline__ uint64_t bound_of(uint64_t best, int top)
{
    if (top <= 8) {
        uint32_t x = static_cast<uint32_t>(best >> 32);
        auto step = [&](auto dpp) {
            const uint32_t y = __builtin_amdgcn_mov_dpp(x, decltype(dpp)::value, 0xF, 0xF, true);
            x = x > y ? x : y;
        };
        step(std::integral_constant<int, 0xB1>{});   // lane ^ 1
        step(std::integral_constant<int, 0x4E>{});   // lane ^ 2
        step(std::integral_constant<int, 0x141>{});  // the other four of eight
        const uint32_t least = ~wave_max(~x);
        return least ? static_cast<uint64_t>(least) << 32 : 1;
    }
    const uint64_t at_place = __ballot(best != 0 && rank_of(best, 64) == static_cast<uint32_t>(top - 1));
    return at_place ? __shfl(best, __builtin_ctzll(at_place), 64) : 1;
}

// A wave's list of the `top` (at most 64) largest keys that it has met, lane l
// holding the l-th.
constexpr int kTopBatch = 8;
struct TopList {
    uint64_t mine = 0;   // this lane's place
    uint64_t last = 0;   // the list's last key: what is not above it has no place

    // Keys of one batch (0: none), each met once. `room`: 64 keys in LDS of the
    // wave's own. A bound from the lanes' largest keys mostly leaves at most 64, one
    // for each lane, which find their places by counting the larger ones. If not,
    // places are filled one by one; 20 of 640 keys took 8 us so.
    __device__ __forceinline__ void add(uint64_t (&key)[kTopBatch], int top, uint64_t* room)
    {
        const uint32_t lane = threadIdx.x & 63;
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < kTopBatch; ++i) best = key[i] > best ? key[i] : best;
        if (!__any(best > last)) return;
        best = mine > best ? mine : best;
        uint32_t all = static_cast<uint32_t>(__builtin_popcountll(__ballot(mine != 0)));
#pragma unroll
        for (int i = 0; i < kTopBatch; ++i) all += static_cast<uint32_t>(__builtin_popcountll(__ballot(key[i] != 0)));
        uint64_t least = 1;
        if (all > 64) least = bound_of(best, top);
        uint32_t count = 0;
        auto give = [&](uint64_t k) {
            const uint64_t in = __ballot(k >= least);
            const uint32_t to = count + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(in >> 32),
                                                                  __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(in), 0));
            if (k >= least && to < 64) room[to] = k;
            count += static_cast<uint32_t>(__builtin_popcountll(in));
        };
        give(mine);
#pragma unroll
        for (int i = 0; i < kTopBatch; ++i) give(key[i]);
        uint64_t list = 0;
        if (count <= 64) {
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const uint64_t one = lane < count ? room[lane] : 0;
            const uint32_t place = rank_of(one, count);
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (lane < count && place < static_cast<uint32_t>(top)) room[place] = one;
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            list = lane < min(count, static_cast<uint32_t>(top)) ? room[lane] : 0;
            __builtin_amdgcn_wave_barrier();
        } else {
            uint64_t held = mine;
            for (int k = 0; k < top; ++k) {
                const uint32_t high = wave_max(static_cast<uint32_t>(best >> 32));
                if (high == 0) break;  // no more keys
                const bool first = static_cast<uint32_t>(best >> 32) == high;
                const uint32_t low = wave_max(first ? static_cast<uint32_t>(best) : 0u);
                const uint64_t won = static_cast<uint64_t>(high) << 32 | low;
                if (lane == static_cast<uint32_t>(k)) list = won;
                if (best == won) {  // one lane: it goes on with its next one
                    held = held == won ? 0 : held;
                    best = held;
#pragma unroll
                    for (int i = 0; i < kTopBatch; ++i) {
                        key[i] = key[i] == won ? 0 : key[i];
                        best = key[i] > best ? key[i] : best;
                    }
                }
            }
        }
        mine = list;
        last = __shfl(mine, top - 1, 64);
    }
};

// The alternatives of a chunk's tokens, and with them the join of their parts.
// W waves work on a token and join their lists through LDS: 8 for few tokens,
// where the time is latency, 1 (4 tokens a workgroup) for many.
template <int W>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void select_top(const LogParts* parts, uint64_t groups,
                                                                    const float* logits, uint32_t group_rows, int top,
                                                                    LogProbOut out, float* top_log_probs,
                                                                    int32_t* top_ids)
{
    constexpr int TOKENS = W == 1 ? 4 : 1;
    __shared__ uint64_t lists[W == 1 ? 1 : W][64], rooms[TOKENS * W][64];
    __shared__ LogParts sums[W];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int slot = W == 1 ? wave : 0, w = W == 1 ? 0 : wave;
    const uint64_t t = static_cast<uint64_t>(blockIdx.x) * TOKENS + slot, n = out.ntokens;
    const bool on = t < n;  // (the same for a wave; all meet at the barriers)

    // the waves' lists become one, in every wave
    auto join_lists = [&](TopList& list) {
        if constexpr (W > 1) {
            __syncthreads();
            lists[w][lane] = list.mine;
            __syncthreads();
            list = TopList{};
            uint64_t key[kTopBatch] = {};
            static_assert(W <= kTopBatch, "one batch takes all lists");
            // (the keys of a list in neighbouring lanes, so that every lane has large ones)
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int e = i * 64 + lane;
                if (e < W * top) key[i] = lists[e / top][e % top];
            }
            list.add(key, top, rooms[wave]);
        }
    };

    TopList best;
    LogParts s{-INFINITY, 0.0f, 0.0f};
    LogProbOut::Aim aim{};
    if (on) {
        if (w == 0) aim = out.aim(t);
        for (uint64_t g0 = static_cast<uint64_t>(w) * 64 * kTopBatch; g0 < groups; g0 += W * 64 * kTopBatch) {
            // all loads first: within a branch each would be waited for by itself
            LogParts p[kTopBatch];
            uint64_t key[kTopBatch];
#pragma unroll
            for (int i = 0; i < kTopBatch; ++i) p[i] = parts[min(g0 + i * 64 + lane, groups - 1) * n + t];
#pragma unroll
            for (int i = 0; i < kTopBatch; ++i) {
                const uint64_t g = g0 + i * 64 + lane;
                const bool in = g < groups;
                key[i] = in ? order_key(p[i].top, static_cast<uint32_t>(g)) : 0;
                s = join_parts(s, in ? p[i] : LogParts{-INFINITY, 0.0f, 0.0f});
            }
            best.add(key, top, rooms[wave]);
        }
#pragma unroll
        for (int m = 1; m <= 32; m *= 2)
            s = join_parts(s, LogParts{__shfl_xor(s.top, m, 64), __shfl_xor(s.sum, m, 64), __shfl_xor(s.dot, m, 64)});
    }
    join_lists(best);
    if constexpr (W > 1) {
        if (lane == 0) sums[w] = s;
        __syncthreads();
        s = sums[0];
#pragma unroll
        for (int i = 1; i < W; ++i) s = join_parts(s, sums[i]);
    }

    TopList found;
    // up to two batches take one wave no longer than a join of several waves' lists
    const uint32_t per_batch = 64 * kTopBatch / group_rows;  // groups
    const bool alone = W == 1 || static_cast<uint32_t>(top) <= 2 * per_batch;
    if (on && (w == 0 || !alone)) {
        const uint64_t blocks = (n + 15) / 16;
        struct Batch {
            float z[kTopBatch];
            uint32_t ids[kTopBatch];
        };
        auto load = [&](uint32_t k0, Batch& x) {
#pragma unroll
            for (int i = 0; i < kTopBatch; ++i) {
                const uint32_t e = i * 64 + lane, k = k0 + e / group_rows, row = e % group_rows;
                const uint64_t group = __shfl(best.mine, k & 63, 64);
                const bool in = k < static_cast<uint32_t>(top) && group != 0;
                x.ids[i] = in ? key_id(group) * group_rows + row : UINT32_MAX;
                x.z[i] = logits[in ? logit_at(key_id(group), blocks, t, group_rows / 16, row) : 0];
            }
        };
        const uint32_t stride = (alone ? 1 : W) * per_batch;
        Batch x;
        load(w * per_batch, x);
        for (uint32_t k0 = w * per_batch; k0 < static_cast<uint32_t>(top); k0 += stride) {
            uint64_t key[kTopBatch];
#pragma unroll
            for (int i = 0; i < kTopBatch; ++i) key[i] = x.ids[i] < out.vocab ? order_key(x.z[i], x.ids[i]) : 0;
            if (k0 + stride < static_cast<uint32_t>(top)) load(k0 + stride, x);  // under way meanwhile
            found.add(key, top, rooms[wave]);
        }
    }
    if (!alone) join_lists(found);
    if (!on || w != 0) return;
    const float l = s.top + logf(s.sum);
    if (lane == 0) out.put(t, s, aim);
    if (lane < top) {
        const uint64_t at = (out.first_token + t) * top + lane;
        top_log_probs[at] = key_value(found.mine) - l;
        top_ids[at] = static_cast<int32_t>(key_id(found.mine));
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// d of a row is held over the row's larger gradient g = s max(|a|, |b|): |p
// (log p + H)| is below 6 for a vocabulary of 2^28, so that 2^12 d stays within
// fp16, where its steps are then 2^-36. Rounding d to the operands' 16 bits, which the
// matrix cores want, shows in bf16: gradients of 6000 x 131072 x 4096 are off by 0.0024
// of their size, where a d of fp32 and one rounding at the end are off by 0.0017; in
// fp16 (2048 x 32000 x 1024) by 0.00074 either way.
constexpr float kLogProbBits = 12.0f, kLogProbScale = 4096.0f;

struct RowGradients {
    float* g;  // [token]
    float* a;  // over g / s
    float* b;
};

__global__ __launch_bounds__(1024) void row_gradients(const float* grad_log_probs, const float* grad_entropy,
                                                      float scale, Indices targets, int64_t ignore, uint64_t vocab,
                                                      uint64_t ntokens, RowGradients out, RowScale* top_out)
{
    __shared__ float waves[16];
    float top = 0.0f;
    for (uint64_t t = threadIdx.x; t < ntokens; t += 1024) {
        float g = 0.0f, a = 0.0f, b = 0.0f;
        if (load_target(targets, t, ignore, vocab) >= 0) {
            const float x = grad_log_probs[t], y = grad_entropy ? grad_entropy[t] : 0.0f;
            const float most = fmaxf(fabsf(x), fabsf(y));
            g = scale * most;
            // (subnormal gradients take a factor of their own: their reciprocal may be infinite)
            const float up = most < 0x1p-100f ? 0x1p40f : 1.0f;
            a = most == 0.0f ? 0.0f : x * up / (most * up);
            b = most == 0.0f ? 0.0f : y * up / (most * up);
            if (x != x || y != y) g = NAN;
            top = fmaxf(top, g);
        }
        out.g[t] = g;
        out.a[t] = a;
        out.b[t] = b;
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) top = fmaxf(top, waves[w]);
        top_out->top = fmaxf(top, 0x1p-126f);  // whose reciprocal is finite
    }
}

// The part of d that a tile's epilogue computes before it is stored: 2^12 (a
// [v = y] - p (a + b (log p + H))).
struct LogProbD {
    const float* lse;
    const float* entropy;  // null where no gradient comes through it
    RowGradients rows;
    float scale;

    struct Row {
        float lse, entropy, a, b, g;
    };
    __device__ __forceinline__ Row row(uint64_t t, bool on) const
    {
        return on ? Row{lse[t], entropy ? entropy[t] : 0.0f, rows.a[t], rows.b[t], rows.g[t]} : Row{};
    }
    __device__ __forceinline__ float operator()(const Row& x, float product) const
    {
        float log_p = __builtin_fmaf(product, scale, -x.lse);
        log_p = log_p < -200.0f ? -200.0f : log_p;  // finite, of probability 0
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(log_p, kLog2e, kLogProbBits));
        return -p * __builtin_fmaf(x.b, log_p + x.entropy, x.a);
    }
    __device__ __forceinline__ float at_target(const Row& x) const { return x.a * kLogProbScale; }
};

// The same for the loss: 2^14 (p - [v = y]).
struct LossD {
    const float* lse;
    const float* g;

    struct Row {
        float lse, g;
    };
    __device__ __forceinline__ Row row(uint64_t t, bool on) const { return on ? Row{lse[t], g[t]} : Row{}; }
    __device__ __forceinline__ float operator()(const Row& x, float product) const
    {
        return __builtin_amdgcn_exp2f(__builtin_fmaf(product - x.lse, kLog2e, kDBits));
    }
    __device__ __forceinline__ float at_target(const Row&) const { return -kDScale; }
};

}  // namespace
}  // namespace lm
}  // namespace ar
