// head.h -- what the operators of a linear head share: targets, and the constants
// of their epilogues.
#pragma once

#include "gemm.h"

namespace ar {
namespace lm {
using namespace detail;

namespace {

// d is held times 2^14: a probability of 1e-8 is still a normal fp16, and
// |p - 1| 2^14 is far below its largest.
constexpr float kDBits = 14.0f, kDScale = 16384.0f;
constexpr float kLog2e = 1.4426950408889634f;

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

struct RowScale {
    float top;  // the largest |g| of the rows that count, at least the least normal number
};

constexpr int kJoinBlock = 512;

}  // namespace
}  // namespace lm
}  // namespace ar
