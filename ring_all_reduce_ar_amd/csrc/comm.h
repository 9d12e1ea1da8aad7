// comm.h -- host-side state and helpers shared by the ABI's sources (api.cpp
// and lm/lm_api.cpp): the communicator, error reporting and argument checks.
// Not installed; the public ABI is include/allreduce.h.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <vector>

#include "allreduce.h"
#include "kernels.h"

#define AR_EXPORT extern "C" __attribute__((visibility("default")))

struct ar_comm {
    int nranks = 0;
    int device = 0;
    int num_cus = 256;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    bool debug = false;
    bool step_timing = false;
    ar_access_t access = AR_ACCESS_AUTO;  // access flavour of the one-launch calls (ar_comm_set_access)
    std::vector<hipEvent_t> events;  // step boundaries of the last timed call
    int last_steps = -1;
    // AR_MODE_RING_GRAPH: instantiated graphs keyed by call signature.
    struct GraphEntry {
        std::vector<uintptr_t> key;
        hipGraphExec_t exec;
        uint64_t last_use;
    };
    static constexpr size_t kMaxGraphs = 16;
    std::vector<GraphEntry> graphs;
    uint64_t use_clock = 0;
    hipStream_t capture_stream = nullptr;
    // ar_all_reduce_noalloc: this device's AR_NOALLOC_SCRATCH_BYTES array,
    // looked up at creation (or why the lookup failed).
    void* scratch = nullptr;
    std::string scratch_err;
};

namespace ar {

// Sets this thread's error text and returns `code` (api.cpp).
ar_result_t fail(ar_result_t code, const char* fmt, ...);
ar_result_t hip_fail(hipError_t e, const char* what);

namespace host {

inline size_t elem_size(ar_dtype_t d)
{
    switch (d) {
    case AR_FLOAT32: return 4;
    case AR_FLOAT16: return 2;
    case AR_BFLOAT16: return 2;
    case AR_INT32: return 4;
    }
    return 0;
}

inline bool valid_dtype(int d) { return d >= AR_FLOAT32 && d <= AR_INT32; }
inline bool valid_op(int o) { return o >= AR_SUM && o <= AR_PROD; }
inline bool valid_mode(int m) { return m >= AR_MODE_FUSED && m <= AR_MODE_TREE_STEPWISE; }
inline bool tree_mode(int m) { return m == AR_MODE_TREE || m == AR_MODE_TREE_STEPWISE; }

inline const char* dtype_name(ar_dtype_t d)
{
    static const char* names[] = {"fp32", "fp16", "bf16", "int32"};
    return valid_dtype(d) ? names[d] : "?";
}

// a * b without overflow, else false.
inline bool mul_ok(size_t a, size_t b, size_t* out)
{
    if (a != 0 && b > SIZE_MAX / a) return false;
    *out = a * b;
    return true;
}

inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Restores the caller's current device on scope exit.
struct DeviceGuard {
    int prev = -1;
    hipError_t err = hipSuccess;
    explicit DeviceGuard(int dev)
    {
        err = hipGetDevice(&prev);
        if (err == hipSuccess && prev != dev) err = hipSetDevice(dev);
        else if (err == hipSuccess) prev = -1;
    }
    ~DeviceGuard()
    {
        if (prev >= 0) (void)hipSetDevice(prev);
    }
};

struct Interval {
    uintptr_t lo, hi;
    const char* what;
    int rank;
};

// Sorts `iv` by start. An interval overlaps an earlier one exactly when it
// starts before the largest end seen so far (empty intervals overlap
// nothing); on the first such pair returns true with *a the later interval
// and *b the earlier one.
inline bool find_overlap(std::vector<Interval>& iv, size_t* a, size_t* b)
{
    std::sort(iv.begin(), iv.end(), [](const Interval& x, const Interval& y) { return x.lo < y.lo; });
    size_t last = SIZE_MAX;  // the interval with the largest end so far
    for (size_t i = 0; i < iv.size(); ++i) {
        if (iv[i].hi == iv[i].lo) continue;
        if (last != SIZE_MAX && iv[i].lo < iv[last].hi) {
            *a = i;
            *b = last;
            return true;
        }
        if (last == SIZE_MAX || iv[i].hi > iv[last].hi) last = i;
    }
    return false;
}

// The last-level cache of MI355X (Infinity Cache): a fused call whose
// distinct bytes fit in it uses cached loads/stores, else non-temporal ones.
constexpr uint64_t kLastLevelCacheBytes = uint64_t(256) << 20;

// Above this footprint the fused all-reduce streams by default. A footprint
// of more than half the cache is unlikely to be resident in full, and cold
// calls gain more from non-temporal access than warm ones lose: 8 ranks,
// fp32, cold (every call from HBM) / warm (repeated on one buffer set), in
// microseconds, cached two-tile against non-temporal rank-major kernels:
// 16 MiB per rank 59.4 / 41.0 against 48.7 / 48.1 (at the threshold, stays
// cached); 20 MiB 71.6 / 50.0 against 61.1 / 60.0; 25 MiB 87.0 / 62.1
// against 75.2 / 73.6. Streaming wins there unless the data is warm more
// than about half the time; at 16 ranks x 8 MiB it loses cold too (56.7
// against 60.6), which the threshold keeps cached.
constexpr uint64_t kAllReduceStreamBytes = kLastLevelCacheBytes / 2;

// The access flavour of a one-launch call (ar_comm_set_access): AUTO streams
// (non-temporal loads and stores) above `auto_bytes` of footprint
// (kAllReduceStreamBytes for the all-reduce, the whole cache for the other
// collectives), STREAMING always, CACHED above the whole cache only. The
// launch shapes follow the flavour chosen.
inline bool call_nt(const ar_comm* comm, uint64_t footprint_bytes, uint64_t auto_bytes)
{
    switch (comm->access) {
    case AR_ACCESS_STREAMING: return true;
    case AR_ACCESS_CACHED: return footprint_bytes > kLastLevelCacheBytes;
    default: return footprint_bytes > auto_bytes;
    }
}

// Work-items per grid dimension fit 32 bits.
constexpr uint64_t kMaxGridX = (uint64_t(1) << 32) / ar::kBlock - 1;

}  // namespace host
}  // namespace ar
