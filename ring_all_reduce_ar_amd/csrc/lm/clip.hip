// clip.hip -- the global norm over many gradient tensors, and the clip.
//
//   total = sqrt(sum x^2) or max |x|,   scale = min(1, max_norm / (total + eps)),   out = round(x * scale)
//
// Squares and their sums are doubles: they neither overflow nor lose small
// gradients beside large ones, and fp64 adds at the rate of HBM cost nothing
// here. Each workgroup leaves one partial, and they are joined in a fixed order,
// so the same call gives the same bits: by every workgroup of the scaling pass
// for itself where there are few (kClipJoinEach), else by a launch of one.
#include "../kernels_impl.h"
#include "lm_kernels.h"

namespace ar {
namespace lm {
using namespace detail;

namespace {

constexpr double kClipEps = 1e-6;
constexpr int kJoinBlock = 1024;

// Joins two partial norms; the maximum keeps a NaN.
__device__ __forceinline__ double join_norm(double a, double b, int inf)
{
    return inf ? __builtin_elementwise_maximum(a, b) : a + b;
}

__device__ __forceinline__ double wave_join(double v, int inf)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = join_norm(v, __shfl_xor(v, m, 64), inf);
    return v;
}

template <int THREADS>
__device__ __forceinline__ double block_join(double v, int inf)
{
    __shared__ double part[THREADS / 64];
    v = wave_join(v, inf);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v = join_norm(v, part[w], inf);
    return v;
}

template <int E>
__device__ __forceinline__ void take(const float* x, int inf, double& sum, float& top)
{
    if (inf) {
#pragma unroll
        for (int j = 0; j < E; ++j) top = fp_max(top, __builtin_fabsf(x[j]));
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) sum = __builtin_fma(static_cast<double>(x[j]), static_cast<double>(x[j]), sum);
    }
}

// All partials, by every thread of a workgroup.
template <int THREADS>
__device__ __forceinline__ double join_partials(const ClipWorkspace* ws, int slots, int inf)
{
    double v = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < slots; i += THREADS) v = join_norm(v, ws->partial[i], inf);
    return block_join<THREADS>(v, inf);
}

__device__ __forceinline__ double norm_of(double joined, int inf) { return inf ? joined : __builtin_sqrt(joined); }

__device__ __forceinline__ float scale_of(double total, double max_norm)
{
    if (__builtin_isinf(max_norm) && !__builtin_isnan(total)) return 1.0f;  // no limit, also of an infinite norm
    const double s = max_norm / (total + kClipEps);
    return static_cast<float>(s > 1.0 ? 1.0 : s);  // a NaN stays one
}

// One pass over a batch of tensors (see ClipKind), bound by HBM: for 8 x 134M
// fp16 the reduction takes 415 us and the scaling into 8 copies 420, 5.8 TB/s
// each; 8 x 33.5M fp32 are measured at 6.5 TB/s and scaled at 6.0. A tile is M kBlock-vector
// quarters of a piece, or kBlock elements where the pointers of a tensor
// differ in their offset from a 16-byte boundary.
template <class F, int KIND, int OP, bool NT, int M>
__global__ __launch_bounds__(kBlock) void clip_pass(const MultiArgs a, int ndst, int inf, int first, int slots,
                                                    double max_norm, ClipWorkspace* ws, float* norm_out)
{
    constexpr int E = F::kEpv;
    const MultiHeader& h = a.h;
    const int n = h.n;
    cbyte* ctable = (cbyte*)(a.blob);
    cpiece* pieces = (cpiece*)(ctable + h.pieces_offset);
    double sum = 0.0;
    float top = 0.0f;
    float scale = 1.0f;
    bool scaled = KIND != kClipApply;
    // Called by the whole workgroup, after its first loads were issued.
    auto need_scale = [&] {
        if (scaled) return;
        scaled = true;
        if (slots) {
            const double total = norm_of(join_partials<kBlock>(ws, slots, inf), inf);
            scale = scale_of(total, max_norm);
            if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(total);
        } else {
            scale = ws->scale;
        }
    };
    for (uint32_t tile = blockIdx.x; tile < h.ntiles; tile += gridDim.x) {
        const MultiPiece pc = load_piece(pieces + multi_find_piece(pieces, h.npieces, tile));
        cuptr* block = (cuptr*)(ctable) + pc.ptrs;
        const void* const* src = (const void* const*)(block);
        void* const* dst = (void* const*)(block + n);
        const uint32_t ti = tile - pc.tile0;
        const uint64_t j_end = pc.j0 + pc.len;
        // one element of the piece
        auto element = [&](uint64_t i) {
            float x[1];
            if constexpr (KIND == kClipReduce) {
                const float v = finalize<OP>(fold_elem<F, OP>(src, pc.chunk, n, i), n);
                F::st(dst[0], i, v);
                x[0] = F::ld(dst[0], i);  // as rounded
            } else {
                x[0] = F::ld(src[0], i);
            }
            if constexpr (KIND == kClipApply) {
                for (int r = 0; r < ndst; ++r) F::st(dst[r], i, x[0] * scale);
            } else {
                take<1>(x, inf, sum, top);
            }
        };
        if (pc.flags & kPieceVec) {
            const uint64_t a0 = (pc.flags >> kPieceShiftBit) & kPieceShiftMask;
            const uint64_t boff = a0 * (16 / E);
            uint64_t vb, ve;
            piece_vectors(pc.j0, j_end, a0, E, &vb, &ve);
            const uint64_t v = vb + static_cast<uint64_t>(ti) * (M * kBlock) + threadIdx.x;
            if (ve > vb) {
                // lanes past the piece read its first vector and drop it
                uint64_t off[M];
                bool ok[M];
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    ok[m] = v + m * kBlock < ve;
                    off[m] = (ok[m] ? v + m * kBlock : vb) * 16 + boff;
                }
                float acc[M][E];
                if constexpr (KIND == kClipReduce) {
                    fold_rank_major_any<F, OP, NT, M>(src, pc.chunk, n, off, acc);
#pragma unroll
                    for (int m = 0; m < M; ++m) {
#pragma unroll
                        for (int j = 0; j < E; ++j) acc[m][j] = finalize<OP>(acc[m][j], n);
                        const u32x4 out = F::pack(acc[m]);
                        if (ok[m]) stv_at<false>(dst[0], off[m], out);
                        F::unpack(out, acc[m]);
                    }
                } else {
                    u32x4 x[M];
                    load_stage<M, NT>(x, src[0], off);
                    need_scale();
#pragma unroll
                    for (int m = 0; m < M; ++m) F::unpack(x[m], acc[m]);
                }
                if constexpr (KIND == kClipApply) {
                    u32x4 out[M];
#pragma unroll
                    for (int m = 0; m < M; ++m) {
#pragma unroll
                        for (int j = 0; j < E; ++j) acc[m][j] *= scale;
                        out[m] = F::pack(acc[m]);
                    }
                    for (int r = 0; r < ndst; ++r)
#pragma unroll
                        for (int m = 0; m < M; ++m)
                            if (ok[m]) stv_at<NT>(dst[r], off[m], out[m]);
                } else {
#pragma unroll
                    for (int m = 0; m < M; ++m)
                        if (ok[m]) take<E>(acc[m], inf, sum, top);
                }
            }
            need_scale();
            if (ti == 0) {
                // elements before the first whole vector and after the last
                const uint64_t vstart = a0 + vb * E, vend = a0 + ve * E;
                const uint64_t head_end = vstart < j_end ? (vstart > pc.j0 ? vstart : pc.j0) : j_end;
                const uint64_t nhead = head_end - pc.j0;
                const uint64_t tail_lo = vend > head_end ? vend : head_end;
                const uint64_t tail_start = tail_lo < j_end ? tail_lo : j_end;
                const uint64_t ntail = j_end - tail_start;
                for (uint64_t k = threadIdx.x; k < nhead + ntail; k += kBlock)
                    element(k < nhead ? pc.j0 + k : tail_start + (k - nhead));
            }
        } else {
            need_scale();
            const uint64_t i = pc.j0 + static_cast<uint64_t>(ti) * kBlock + threadIdx.x;
            if (i < j_end) element(i);
        }
    }
    if constexpr (KIND != kClipApply) {
        const double v = block_join<kBlock>(inf ? static_cast<double>(top) : sum, inf);
        if (threadIdx.x == 0) {
            double* slot = ws->partial + blockIdx.x;
            *slot = first ? v : join_norm(*slot, v, inf);
        }
    }
}

__global__ __launch_bounds__(kJoinBlock) void clip_join(int slots, int inf, double max_norm, ClipWorkspace* ws,
                                                        float* norm_out)
{
    const double total = norm_of(join_partials<kJoinBlock>(ws, slots, inf), inf);
    if (threadIdx.x == 0) {
        ws->scale = scale_of(total, max_norm);
        if (norm_out) *norm_out = static_cast<float>(total);
    }
}

struct PassArgs {
    int ndst, inf, first, slots;
    double max_norm;
    ClipWorkspace* ws;
    float* norm_out;
};

template <class F, int KIND, int OP, bool NT, int M>
hipError_t pass_tiles(const MultiArgs& a, const PassArgs& p, int grid, hipStream_t s)
{
    hipLaunchKernelGGL((clip_pass<F, KIND, OP, NT, M>), dim3(grid), dim3(kBlock), 0, s, a, p.ndst, p.inf, p.first,
                       p.slots, p.max_norm, p.ws, p.norm_out);
    return hipGetLastError();
}

template <class F, int KIND, int OP, bool NT>
hipError_t pass_m(const MultiArgs& a, const PassArgs& p, int grid, hipStream_t s)
{
    constexpr int EB = 16 / F::kEpv;
    if constexpr (KIND == kClipReduce) {
        constexpr int MA = clip_tiles(kClipReduce, kRankMajorAnyMany, EB), MF = clip_tiles(kClipReduce, 1, EB);
        return a.h.n >= kRankMajorAnyMany ? pass_tiles<F, KIND, OP, NT, MA>(a, p, grid, s)
                                          : pass_tiles<F, KIND, OP, NT, MF>(a, p, grid, s);
    } else {
        return pass_tiles<F, KIND, OP, NT, clip_tiles(static_cast<ClipKind>(KIND), 1, EB)>(a, p, grid, s);
    }
}

template <class F, bool NT>
hipError_t pass_kind(ClipKind kind, const MultiArgs& a, ar_op_t op, const PassArgs& p, int grid, hipStream_t s)
{
    switch (kind) {
    case kClipMeasure: return pass_m<F, kClipMeasure, AR_SUM, NT>(a, p, grid, s);
    case kClipApply: return pass_m<F, kClipApply, AR_SUM, NT>(a, p, grid, s);
    case kClipReduce:
        if (op == AR_SUM) return pass_m<F, kClipReduce, AR_SUM, NT>(a, p, grid, s);
        if (op == AR_AVG) return pass_m<F, kClipReduce, AR_AVG, NT>(a, p, grid, s);
    }
    return hipErrorInvalidValue;
}

template <class F>
hipError_t pass_nt(ClipKind kind, const MultiArgs& a, ar_op_t op, bool nt, const PassArgs& p, int grid, hipStream_t s)
{
    return nt ? pass_kind<F, true>(kind, a, op, p, grid, s) : pass_kind<F, false>(kind, a, op, p, grid, s);
}

hipError_t pass(ClipKind kind, const MultiArgs& a, ar_dtype_t dtype, ar_op_t op, bool nt, const PassArgs& p, int grid,
                hipStream_t s)
{
    switch (dtype) {
    case AR_FLOAT32: return pass_nt<F32>(kind, a, op, nt, p, grid, s);
    case AR_FLOAT16: return pass_nt<F16>(kind, a, op, nt, p, grid, s);
    case AR_BFLOAT16: return pass_nt<BF16>(kind, a, op, nt, p, grid, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_clip_norm(ClipKind kind, const MultiArgs& a, ar_dtype_t dtype, ar_op_t op, ar_norm_t norm, bool nt,
                            bool first, int grid, ClipWorkspace* ws, hipStream_t stream)
{
    return pass(kind, a, dtype, op, nt, PassArgs{1, norm == AR_NORM_INF, first, 0, 0.0, ws, nullptr}, grid, stream);
}

hipError_t launch_clip_apply(const MultiArgs& a, int ndst, ar_dtype_t dtype, ar_norm_t norm, bool nt, int slots,
                             double max_norm, int grid, ClipWorkspace* ws, float* norm_out, hipStream_t stream)
{
    return pass(kClipApply, a, dtype, AR_SUM, nt, PassArgs{ndst, norm == AR_NORM_INF, 0, slots, max_norm, ws, norm_out},
                grid, stream);
}

hipError_t launch_clip_join(int slots, ar_norm_t norm, double max_norm, ClipWorkspace* ws, float* norm_out,
                            hipStream_t stream)
{
    hipLaunchKernelGGL(clip_join, dim3(1), dim3(kJoinBlock), 0, stream, slots, norm == AR_NORM_INF ? 1 : 0, max_norm,
                       ws, norm_out);
    return hipGetLastError();
}

}  // namespace lm
}  // namespace ar
