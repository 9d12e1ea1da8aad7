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
// kClipSlots. Up to kClipJoinEach of them are joined by each workgroup that
// scales, behind its first loads: 150000 bf16 elements in 15 us a call rather
// than 20 with a launch in between. 1600 of them (8 ranks x 25 MiB) cost as much
// in every workgroup as the launch does, 90 against 87 us.
constexpr int kClipSlots = 8192;
constexpr int kClipJoinEach = 256;

struct ClipWorkspace {
    float scale;  // min(1, max_norm / (norm + eps)), where a launch of its own joins
    float pad[15];
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

// One batch: `a.h.n` sources and then the destinations for each tensor of the
// table. kClipMeasure and kClipReduce; `first`: the batch's partials are stored
// rather than joined to those of earlier batches.
hipError_t launch_clip_norm(ClipKind kind, const MultiArgs& a, ar_dtype_t dtype, ar_op_t op, ar_norm_t norm, bool nt,
                            bool first, int grid, ClipWorkspace* ws, hipStream_t stream);
// Joins `slots` partials into the norm and the scale; `norm_out` may be null.
hipError_t launch_clip_join(int slots, ar_norm_t norm, double max_norm, ClipWorkspace* ws, float* norm_out,
                            hipStream_t stream);
// kClipApply with `ndst` destinations a tensor: by the scale of `slots`
// partials, or, where that is 0, by the joined one.
hipError_t launch_clip_apply(const MultiArgs& a, int ndst, ar_dtype_t dtype, ar_norm_t norm, bool nt, int slots,
                             double max_norm, int grid, ClipWorkspace* ws, float* norm_out, hipStream_t stream);

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
hipError_t launch_lookup(const LookupArgs& a, ar_dtype_t dtype, hipStream_t stream);

// The sort: at most kSortBlocks workgroups of kSortThreads threads, digits of
// at most 9 bits. The sum: a chunk of positions of the sorted order for at least
// kGradLanes threads. Up to kGradFew tokens the chunks are short, since there are
// CUs to spare: the sums of 1143 x 576 bf16 take 7 us rather than 16. Where short
// chunks end to pay depends on the width; gradients with short against long
// ones, us: 50000 x 64 fp16 of 8192 tokens 33 / 41, of 16384 42 / 45, of 24000 49 / 47;
// 50000 x 1024 bf16 of 4096 tokens 40 / 47, of 8192 46 / 48, of 12000 54 / 51; 131072 x
// 4096 bf16 of 2048 tokens 213 / 219, of 4096 219 / 219, of 8192 230 / 222.
constexpr int kSortThreads = 1024;
constexpr int kSortBlocks = 128;
constexpr int kSortBins = 512;
constexpr int kGradChunk = 32, kGradChunkFew = 8;
constexpr uint64_t kGradFew = 8192;
inline uint32_t grad_chunk(uint64_t ntokens) { return ntokens <= kGradFew ? kGradChunkFew : kGradChunk; }
constexpr int kGradLanes = 4;

// Bits of a key (keys are 0..rows), and the passes over 9 of them at a time.
inline int sort_bits(uint64_t rows)
{
    int bits = 1;
    while ((rows >> bits) != 0) ++bits;
    return bits;
}
inline int sort_passes(uint64_t rows) { return (sort_bits(rows) + 8) / 9; }

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
    uint8_t* present;      // a flag for each row, and right behind them
    uint32_t* hist;        // [sort_passes][kSortBlocks][kSortBins]
    uint64_t clear_words;  // of both
    float* partial;        // 2 * width floats for each chunk
};
// `vec`: rows of both matrices in 16-byte vectors; `nt`: non-temporal zeros.
hipError_t launch_lookup_grad(const LookupGradArgs& a, ar_dtype_t dtype, ar_dtype_t grad_dtype, bool vec, bool nt,
                              int num_cus, hipStream_t stream);

// ---- cross entropy --------------------------------------------------------------
// The matrix core's tile: kTileM rows of the first operand by 256 or 128 of the
// second, or, for few tokens, 64 by 64 or 16; kTileK deep.
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
    uint64_t t_pad;        // tokens, up to a multiple of kTileK (of 16 if there are no more)
    bool pieces;           // fp32 operands in bf16 pieces
    bool pack_hidden, pack_weight;
    int tile_n;            // token tile of the logits' product
    int splits;            // parts of the vocabulary axis in the hidden gradient's product
    int weight_splits;     // parts of the token axis in the weight gradient's
    uint64_t stat_rows;    // rows of partial softmax statistics
    // offsets
    uint64_t hidden, weight, stats, target_logit, d, dt, weight_t, hidden_t, grad_hidden_acc, grad_weight_acc, row_scale, bytes;
};
// At least the bytes of the plans of `ntokens` and of fewer tokens.
uint64_t cross_entropy_bytes(uint64_t ntokens, uint64_t vocab, uint64_t width, ar_dtype_t dtype, bool backward);
CrossEntropyPlan plan_cross_entropy(uint64_t ntokens, uint64_t vocab, uint64_t width, ar_dtype_t dtype, bool backward);

hipError_t launch_cross_entropy(const CrossEntropyArgs& a, const CrossEntropyPlan& p, ar_dtype_t dtype, char* ws,
                                hipStream_t stream);
hipError_t launch_cross_entropy_backward(const CrossEntropyArgs& a, const CrossEntropyPlan& p, ar_dtype_t dtype,
                                         char* ws, hipStream_t stream);

}  // namespace lm
}  // namespace ar
