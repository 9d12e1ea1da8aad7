// lm_kernels.h -- internal interface between lm_api.cpp and the kernels of the
// language-model operators (clip.hip, embedding.hip, cross_entropy.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "kernels.h"

namespace ar {
namespace lm {

// ---- gradient norm and clip -------------------------------------------------
// Norm passes leave one double per workgroup in the workspace, at most
// kClipSlots, which one workgroup then joins.
constexpr int kClipSlots = 8192;

struct ClipWorkspace {
    double total;   // the norm
    float scale;    // min(1, max_norm / (total + eps))
    float pad[13];
    double partial[kClipSlots];
};

enum ClipKind {
    kClipMeasure = 0,  // one source a piece: its part of the norm
    kClipReduce = 1,   // n sources, one destination: the ring's fold, and its part of the norm
    kClipApply = 2     // one source, any number of destinations: source * scale
};

// Vectors a thread takes together.
__host__ __device__ constexpr int clip_tiles(ClipKind kind, int nsources, int elem_bytes)
{
    return kind == kClipReduce ? rank_major_any_tiles(nsources, elem_bytes) : 4;
}

// One batch: `a.h.n` sources and then `ndst` destinations for each tensor of
// the table. `first`: the batch's partials are stored rather than joined to
// those of earlier batches.
hipError_t launch_clip_pass(ClipKind kind, const MultiArgs& a, int ndst, ar_dtype_t dtype, ar_op_t op, ar_norm_t norm,
                            bool nt, bool first, int grid, ClipWorkspace* ws, hipStream_t stream);
// Joins `slots` partials into the norm and the scale; `norm_out` may be null.
hipError_t launch_clip_join(int slots, ar_norm_t norm, double max_norm, ClipWorkspace* ws, float* norm_out,
                            hipStream_t stream);

// ---- embedding ----------------------------------------------------------------
struct Indices {
    const void* p;
    int is64;
};

struct LookupArgs {
    const void* weight;
    void* out;
    Indices tokens;
    uint64_t ntokens, rows, width, ld_weight, ld_out;
    int64_t first_row;
    float scale;
};
hipError_t launch_lookup(const LookupArgs& a, ar_dtype_t dtype, bool vec, int num_cus, hipStream_t stream);

// Keys of one radix pass for a workgroup, and positions of the sorted order
// for a workgroup of the sum.
constexpr int kSortBlockKeys = 2048;
constexpr int kSortBins = 512;
constexpr int kGradChunk = 32;

struct LookupGradArgs {
    const void* grad_out;
    void* grad_weight;
    Indices tokens;
    uint64_t ntokens, rows, width, ld_grad_out, ld_grad_weight;
    int64_t first_row;
    float scale;
    int accumulate;
    // workspace
    uint32_t* key[2];
    uint32_t* pos[2];
    uint32_t* hist;     // kSortBins * sort blocks
    uint32_t* present;  // one bit for each row
    float* partial;     // 2 * width floats for each chunk
};
hipError_t launch_lookup_grad(const LookupGradArgs& a, ar_dtype_t dtype, ar_dtype_t grad_dtype, bool vec, int num_cus,
                              hipStream_t stream);

// ---- cross entropy --------------------------------------------------------------
// The matrix core's tile: kTileM rows of the first operand by 256, 128, 64 or
// 16 of the second, kTileK deep.
constexpr int kTileM = 256;
constexpr int kTileK = 64;

struct CrossEntropyArgs {
    const void* hidden;
    const void* weight;
    Indices targets;
    float* losses;             // forward
    float* lse;                // written forward, read backward
    const float* grad_losses;  // backward
    void* grad_hidden;
    void* grad_weight;
    uint64_t ntokens, vocab, width;
    uint64_t ld_hidden, ld_weight, ld_grad_hidden, ld_grad_weight;
    int64_t ignore_index;
};

// How one call goes through the vocabulary, and where its buffers lie in the
// workspace (bytes from its start; unused ones are 0 long).
struct CrossEntropyPlan {
    uint64_t piece;        // vocabulary rows a piece
    uint64_t k_pad;        // the width, up to whole steps
    uint64_t t_pad;        // tokens, up to a multiple of kTileK
    bool pack_hidden, pack_weight;
    int tile_n;            // token tile of the logits' product
    int splits;            // parts of the vocabulary axis in the hidden gradient's product
    uint64_t stat_rows;    // rows of partial softmax statistics
    // offsets
    uint64_t hidden, weight, stats, target_logit, d, dt, weight_t, hidden_t, grad_hidden_acc, row_scale, bytes;
};
CrossEntropyPlan plan_cross_entropy(uint64_t ntokens, uint64_t vocab, uint64_t width, ar_dtype_t dtype, bool backward);

hipError_t launch_cross_entropy(const CrossEntropyArgs& a, const CrossEntropyPlan& p, ar_dtype_t dtype, char* ws,
                                hipStream_t stream);
hipError_t launch_cross_entropy_backward(const CrossEntropyArgs& a, const CrossEntropyPlan& p, ar_dtype_t dtype,
                                         char* ws, hipStream_t stream);

}  // namespace lm
}  // namespace ar
