// lm_api.cpp -- the C ABI of the language-model operators: argument checks,
// tables and workspace layout, and the launches. As in api.cpp every check
// runs before the first HIP call. No exception leaves an entry point.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "../comm.h"
#include "lm_kernels.h"

using namespace ar::host;
using ar::fail;
using ar::hip_fail;

namespace {

constexpr uint64_t kMaxIndex = uint64_t(1) << 31;  // tokens, rows: positions and keys are 32 bits

// Runs `fn`, turning what it throws (host allocations) into a result code.
template <class Fn>
ar_result_t guarded(Fn&& fn)
{
    try {
        return fn();
    } catch (const std::bad_alloc&) {
        return fail(AR_ERR_OUT_OF_MEMORY, "host allocation failed");
    } catch (...) {
        return fail(AR_ERR_INTERNAL, "unexpected exception");
    }
}

ar_result_t check_float(ar_dtype_t dtype)
{
    if (!valid_dtype(dtype)) return fail(AR_ERR_INVALID_ARGUMENT, "invalid dtype %d", static_cast<int>(dtype));
    if (dtype == AR_INT32) return fail(AR_ERR_UNSUPPORTED, "int32 is not a type of this operator");
    return AR_SUCCESS;
}

ar_result_t check_workspace(const ar_comm* comm, size_t need)
{
    if (comm->ws_bytes < need)
        return fail(AR_ERR_INVALID_ARGUMENT, "this call needs a workspace of %zu bytes, the comm has %zu", need,
                    comm->ws_bytes);
    return AR_SUCCESS;
}

// ---------------------------------------------------------------------------
// gradient norm and clip
// ---------------------------------------------------------------------------
// The tables of one pass: batches of tensors whose pointers and pieces fit
// the kernel arguments.
class Batches {
public:
    Batches(ar::lm::ClipKind kind, int nsrc, int ndst, size_t elem)
        : nsrc_(nsrc), ndst_(ndst), elem_(elem),
          tile_vecs_(static_cast<uint64_t>(ar::lm::clip_tiles(kind, nsrc, static_cast<int>(elem))) * ar::kBlock)
    {
    }

    // `ptrs`: nsrc sources, then ndst destinations, of `count` elements; the
    // tensor starts at element `off` of the bucket that is cut into ring
    // chunks of q elements (q = 0: no chunks).
    void add(const void* const* ptrs, uint64_t count, uint64_t off, uint64_t q)
    {
        const int np = nsrc_ + ndst_;
        const uintptr_t mis = reinterpret_cast<uintptr_t>(ptrs[0]) % 128;
        bool vec = true, line = true;
        for (int i = 0; i < np; ++i) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(ptrs[i]);
            vec = vec && p % 16 == mis % 16;
            line = line && p % 128 == mis;
        }
        const uint64_t a0 = (line ? (128 - mis) % 128 : (16 - mis % 16) % 16) / elem_;
        const uint64_t c0 = q ? off / q : 0, c1 = q ? (off + count - 1) / q : 0;
        const size_t need = np * sizeof(void*) + (c1 - c0 + 1) * sizeof(ar::MultiPiece);
        if (ptrs_.size() * sizeof(void*) + pieces_.size() * sizeof(ar::MultiPiece) + need > ar::kMultiBlobBytes) flush();
        for (uint64_t c = c0; c <= c1; ++c) {
            const uint64_t lo = q ? std::max(off, c * q) : off, hi = q ? std::min(off + count, (c + 1) * q) : off + count;
            ar::MultiPiece pc{};
            pc.j0 = lo - off;
            pc.len = hi - lo;
            pc.tile0 = static_cast<uint32_t>(tiles_);
            pc.ptrs = static_cast<uint16_t>(ptrs_.size());
            pc.chunk = static_cast<uint8_t>(c);
            pc.flags = static_cast<uint8_t>(vec ? ar::kPieceVec | (a0 << ar::kPieceShiftBit) : 0);
            uint64_t t;
            if (vec) {
                uint64_t vb, ve;
                ar::piece_vectors(pc.j0, pc.j0 + pc.len, a0, 16 / elem_, &vb, &ve);
                t = std::max<uint64_t>(1, ceil_div(ve - vb, tile_vecs_));
            } else {
                t = ceil_div(pc.len, ar::kBlock);
            }
            tiles_ += t;
            if (tiles_ > UINT32_MAX) overflow_ = true;
            pieces_.push_back(pc);
        }
        ptrs_.insert(ptrs_.end(), ptrs, ptrs + np);
    }

    ar_result_t finish()
    {
        flush();
        return overflow_ ? fail(AR_ERR_INVALID_ARGUMENT, "a batch of tensors needs more than 2^32 tiles") : AR_SUCCESS;
    }

    const std::vector<ar::MultiArgs>& list() const { return list_; }

private:
    void flush()
    {
        if (pieces_.empty()) return;
        ar::MultiArgs a{};
        a.h.n = nsrc_;
        a.h.npieces = static_cast<int>(pieces_.size());
        a.h.ntiles = static_cast<uint32_t>(tiles_);
        a.h.pieces_offset = static_cast<uint32_t>(ptrs_.size() * sizeof(void*));
        std::memcpy(a.blob, ptrs_.data(), ptrs_.size() * sizeof(void*));
        std::memcpy(a.blob + a.h.pieces_offset, pieces_.data(), pieces_.size() * sizeof(ar::MultiPiece));
        list_.push_back(a);
        ptrs_.clear();
        pieces_.clear();
        tiles_ = 0;
    }

    int nsrc_, ndst_;
    size_t elem_;
    uint64_t tile_vecs_;
    uint64_t tiles_ = 0;
    bool overflow_ = false;
    std::vector<const void*> ptrs_;
    std::vector<ar::MultiPiece> pieces_;
    std::vector<ar::MultiArgs> list_;
};

// What is written may overlap neither what else is written nor what is read;
// inputs may overlap each other.
ar_result_t check_disjoint(const std::vector<Interval>& reads, const std::vector<Interval>& writes)
{
    for (size_t i = 0; i < writes.size(); ++i) {
        auto hits = [&](const Interval& x) {
            return x.hi > x.lo && writes[i].hi > writes[i].lo && x.lo < writes[i].hi && writes[i].lo < x.hi;
        };
        for (const Interval& x : reads)
            if (hits(x)) return fail(AR_ERR_INVALID_ARGUMENT, "%s overlaps %s", writes[i].what, x.what);
        for (size_t k = i + 1; k < writes.size(); ++k)
            if (hits(writes[k])) return fail(AR_ERR_INVALID_ARGUMENT, "%s overlaps %s", writes[i].what, writes[k].what);
    }
    return AR_SUCCESS;
}

// Tensor t of rank r, checked: pointers, alignment, sizes, overlaps (with
// norm_out and the workspace too). `recv` may be null (a norm alone);
// `rank0_only`: only rank 0's send pointers are read.
ar_result_t check_tensors(const ar_comm* comm, int ntensors, const void* const send[], void* const recv[],
                          const size_t counts[], ar_dtype_t dtype, bool rank0_only, const float* norm_out,
                          uint64_t* total, uint64_t* touched)
{
    if (ntensors < 0 || ntensors > AR_MAX_TENSORS)
        return fail(AR_ERR_INVALID_ARGUMENT, "ntensors %d is outside 0..%d", ntensors, AR_MAX_TENSORS);
    const int n = comm->nranks;
    const size_t e = elem_size(dtype);
    std::vector<Interval> iv;
    *total = *touched = 0;
    for (int t = 0; t < ntensors; ++t) {
        size_t bytes = 0;
        if (!mul_ok(counts[t], e, &bytes) || *total + counts[t] < *total)
            return fail(AR_ERR_INVALID_ARGUMENT, "counts[%d] = %zu overflows", t, counts[t]);
        *total += counts[t];
        if (counts[t] == 0) continue;
        for (int r = 0; r < n; ++r) {
            const void* sp = send[static_cast<size_t>(t) * n + r];
            const void* dp = recv ? recv[static_cast<size_t>(t) * n + r] : nullptr;
            if (!sp || (recv && !dp)) return fail(AR_ERR_INVALID_ARGUMENT, "tensor %d rank %d buffer is NULL", t, r);
            const uintptr_t s = reinterpret_cast<uintptr_t>(sp), d = reinterpret_cast<uintptr_t>(dp);
            if (s % e || d % e)
                return fail(AR_ERR_INVALID_ARGUMENT, "tensor %d rank %d buffer is not aligned to %zu bytes", t, r, e);
            if (s > UINTPTR_MAX - bytes || d > UINTPTR_MAX - bytes)
                return fail(AR_ERR_INVALID_ARGUMENT, "tensor %d rank %d buffer wraps the address space", t, r);
            // What is only read may be read twice; what is written may
            // overlap nothing but its own send tensor.
            if (!recv) {
                if (!rank0_only || r == 0) iv.push_back({s, s + bytes, "gradient", t});
                continue;
            }
            if (s == d) {
                iv.push_back({s, s + bytes, "in-place tensor", t});
            } else {
                if (!rank0_only || r == 0) iv.push_back({s, s + bytes, "send tensor", t});
                iv.push_back({d, d + bytes, "recv tensor", t});
            }
        }
    }
    const uintptr_t w = reinterpret_cast<uintptr_t>(comm->ws), norm = reinterpret_cast<uintptr_t>(norm_out);
    std::vector<Interval> own = {{w, w + sizeof(ar::lm::ClipWorkspace), "workspace", -1}};
    if (norm_out) own.push_back({norm, norm + sizeof(float), "norm_out", -1});
    for (const Interval& x : iv) *touched += x.hi - x.lo;
    if (!recv) return check_disjoint(iv, own);
    iv.insert(iv.end(), own.begin(), own.end());
    size_t oa, ob;
    if (find_overlap(iv, &oa, &ob))
        return fail(AR_ERR_INVALID_ARGUMENT, "%s %d overlaps %s %d (only send == recv may alias)", iv[oa].what,
                    iv[oa].rank, iv[ob].what, iv[ob].rank);
    return AR_SUCCESS;
}

ar_result_t check_clip(const ar_comm* comm, int ntensors, const void* const send[], void* const recv[], bool writes,
                       const size_t counts[], ar_dtype_t dtype, ar_norm_t norm, double max_norm, const float* norm_out)
{
    if (!comm) return fail(AR_ERR_INVALID_ARGUMENT, "comm is NULL");
    if (ntensors > 0 && (!send || !counts || (writes && !recv)))
        return fail(AR_ERR_INVALID_ARGUMENT, "NULL buffer or counts array");
    ar_result_t rc = check_float(dtype);
    if (rc != AR_SUCCESS) return rc;
    if (norm != AR_NORM_L2 && norm != AR_NORM_INF)
        return fail(AR_ERR_INVALID_ARGUMENT, "invalid norm %d", static_cast<int>(norm));
    if (writes && !(max_norm >= 0.0))
        return fail(AR_ERR_INVALID_ARGUMENT, "max_norm %g is not a number of at least 0", max_norm);
    if (reinterpret_cast<uintptr_t>(norm_out) % sizeof(float))
        return fail(AR_ERR_INVALID_ARGUMENT, "norm_out is not aligned to 4 bytes");
    return check_workspace(comm, sizeof(ar::lm::ClipWorkspace));
}

// The passes that end in the norm, the join, and the passes that scale.
ar_result_t run_clip(const ar_comm* comm, ar::lm::ClipKind first_kind, const Batches& first, const Batches* apply,
                     int ndst, ar_dtype_t dtype, ar_op_t op, ar_norm_t norm, double max_norm, uint64_t touched,
                     float* norm_out, hipStream_t stream)
{
    DeviceGuard g(comm->device);
    if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
    auto* ws = static_cast<ar::lm::ClipWorkspace*>(comm->ws);
    // A norm alone streams at any size: 40 MiB fp32 in 10.2 us rather than 11.6 with
    // cached loads where they are in the last-level cache, 12.9 rather than 13.1 from
    // HBM, 250 MiB in 42.7 and 44.8 rather than 43.3 and 47.7.
    const bool nt = call_nt(comm, touched, apply ? kLastLevelCacheBytes : 0);
    uint32_t most = 0;
    for (const auto& a : first.list()) most = std::max(most, a.h.ntiles);
    const int grid = static_cast<int>(std::min<uint32_t>(most, ar::lm::kClipSlots));
    bool head = true;
    for (const auto& a : first.list()) {
        const hipError_t e = ar::lm::launch_clip_norm(first_kind, a, dtype, op, norm, nt, head, grid, ws, stream);
        if (e != hipSuccess) return hip_fail(e, "kernel launch");
        head = false;
    }
    const bool each = apply && !apply->list().empty() && grid <= ar::lm::kClipJoinEach;
    if (!each) {
        const hipError_t e = ar::lm::launch_clip_join(grid, norm, max_norm, ws, norm_out, stream);
        if (e != hipSuccess) return hip_fail(e, "kernel launch");
    }
    if (!apply) return AR_SUCCESS;
    for (const auto& a : apply->list()) {
        const int gx = static_cast<int>(std::min<uint64_t>(a.h.ntiles, kMaxGridX));
        const hipError_t e = ar::lm::launch_clip_apply(a, ndst, dtype, norm, nt, each ? grid : 0, max_norm, gx, ws,
                                                       norm_out, stream);
        if (e != hipSuccess) return hip_fail(e, "kernel launch");
    }
    return AR_SUCCESS;
}

ar_result_t clip_impl(ar_comm* comm, int ntensors, const void* const send[], void* const recv[], bool writes,
                      const size_t counts[], ar_dtype_t dtype, ar_grads_t layout, ar_norm_t norm, double max_norm,
                      float* norm_out, hipStream_t stream)
{
    ar_result_t rc = check_clip(comm, ntensors, send, recv, writes, counts, dtype, norm, max_norm, norm_out);
    if (rc != AR_SUCCESS) return rc;
    if (layout != AR_GRADS_REPLICATED && layout != AR_GRADS_SHARDED)
        return fail(AR_ERR_INVALID_ARGUMENT, "invalid layout %d", static_cast<int>(layout));
    if (!writes && !norm_out) return fail(AR_ERR_INVALID_ARGUMENT, "norm_out is NULL");
    uint64_t total, touched;
    const bool replicated = layout == AR_GRADS_REPLICATED;
    rc = check_tensors(comm, ntensors, send, writes ? recv : nullptr, counts, dtype, replicated, norm_out, &total,
                       &touched);
    if (rc != AR_SUCCESS) return rc;
    const int n = comm->nranks;
    const size_t e = elem_size(dtype);
    const int ndst = replicated ? n : 1;
    Batches measure(ar::lm::kClipMeasure, 1, 0, e), apply(ar::lm::kClipApply, 1, ndst, e);
    std::vector<const void*> ptrs(1 + static_cast<size_t>(ndst));
    for (int t = 0; t < ntensors; ++t) {
        if (counts[t] == 0) continue;
        const size_t at = static_cast<size_t>(t) * n;
        for (int r = 0; r < (replicated ? 1 : n); ++r) {
            measure.add(&send[at + r], counts[t], 0, 0);
            if (!writes) continue;
            ptrs[0] = send[at + r];
            for (int k = 0; k < ndst; ++k) ptrs[1 + k] = recv[at + r + k];
            apply.add(ptrs.data(), counts[t], 0, 0);
        }
    }
    if ((rc = measure.finish()) != AR_SUCCESS || (rc = apply.finish()) != AR_SUCCESS) return rc;
    return run_clip(comm, ar::lm::kClipMeasure, measure, writes ? &apply : nullptr, ndst, dtype, AR_SUM, norm, max_norm,
                    touched, norm_out, stream);
}

// ---------------------------------------------------------------------------
// rows of a matrix
// ---------------------------------------------------------------------------
// Checks `rows` rows of `width` elements, `ld` apart (0: width); *ld is made
// explicit and the bytes that the matrix spans are returned as an interval.
ar_result_t check_matrix(const char* what, const void* p, uint64_t rows, uint64_t width, size_t* ld, size_t elem,
                         std::vector<Interval>* iv)
{
    if (*ld == 0) *ld = width;
    if (*ld < width) return fail(AR_ERR_INVALID_ARGUMENT, "%s: row pitch %zu is below the width", what, *ld);
    if (rows == 0) return AR_SUCCESS;
    if (!p) return fail(AR_ERR_INVALID_ARGUMENT, "%s is NULL", what);
    size_t bytes = 0, elems = 0;
    if (!mul_ok(rows, *ld, &elems) || !mul_ok(elems, elem, &bytes))
        return fail(AR_ERR_INVALID_ARGUMENT, "%s: its size overflows", what);
    bytes -= (*ld - width) * elem;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a % elem) return fail(AR_ERR_INVALID_ARGUMENT, "%s is not aligned to %zu bytes", what, elem);
    if (a > UINTPTR_MAX - bytes) return fail(AR_ERR_INVALID_ARGUMENT, "%s wraps the address space", what);
    if (iv) iv->push_back({a, a + bytes, what, 0});
    return AR_SUCCESS;
}

ar_result_t check_index(ar_index_t index)
{
    return index == AR_INDEX_INT32 || index == AR_INDEX_INT64
               ? AR_SUCCESS
               : fail(AR_ERR_INVALID_ARGUMENT, "invalid index type %d", static_cast<int>(index));
}

size_t index_bytes(ar_index_t index) { return index == AR_INDEX_INT64 ? 8 : 4; }

// A vector of `n` elements.
ar_result_t check_vector(const char* what, const void* p, uint64_t n, size_t elem, std::vector<Interval>* iv)
{
    size_t ld = 1;
    return check_matrix(what, p, n, 1, &ld, elem, iv);
}

bool rows16(const void* p, size_t ld, size_t elem) { return aligned16(p) && ld * elem % 16 == 0; }

// ---------------------------------------------------------------------------
// embedding
// ---------------------------------------------------------------------------
struct GradLayout {
    size_t key[2], pos[2], hist, present, partial, bytes;
};

bool grad_layout(uint64_t ntokens, uint64_t rows, uint64_t width, GradLayout* l)
{
    if (ntokens >= kMaxIndex || rows >= kMaxIndex || width >= kMaxIndex) return false;
    size_t at = 0;
    bool ok = true;
    auto take = [&](size_t a, size_t b) {
        const size_t here = at;
        size_t bytes = 0;
        ok = ok && mul_ok(a, b, &bytes) && at <= SIZE_MAX / 2 && bytes <= SIZE_MAX / 4;
        if (ok) at += (bytes + 255) / 256 * 256;
        return here;
    };
    for (int k = 0; k < 2; ++k) l->key[k] = take(ntokens, 4);
    for (int k = 0; k < 2; ++k) l->pos[k] = take(ntokens, 4);
    l->present = take(rows, 1);
    l->hist = take(ar::lm::sort_passes(rows), ntokens ? ar::lm::kSortBlocks * ar::lm::kSortBins * 4 : 0);
    // (chunks of few tokens are short: what serves a number of tokens serves fewer)
    const uint64_t few = std::min(ntokens, ar::lm::kGradFew);
    l->partial = take(2 * std::max(ceil_div(ntokens, ar::lm::grad_chunk(ntokens)), ceil_div(few, ar::lm::grad_chunk(few))),
                      width * 4);
    l->bytes = std::max<size_t>(at, 16);
    return ok;
}

ar_result_t check_sizes(uint64_t ntokens, uint64_t rows, uint64_t width, const char* rows_name)
{
    if (ntokens >= kMaxIndex || rows >= kMaxIndex || width >= kMaxIndex)
        return fail(AR_ERR_INVALID_ARGUMENT, "ntokens, %s and width must be below 2^31", rows_name);
    if (width == 0) return fail(AR_ERR_INVALID_ARGUMENT, "width is 0");
    return AR_SUCCESS;
}

// ---------------------------------------------------------------------------
// cross entropy
// ---------------------------------------------------------------------------
constexpr uint64_t kMaxGrid = uint64_t(1) << 31;

// Depths (the width, and the tokens of a weight gradient) are below 2^24, of
// fp32 below 2^20: 64 or 256 rows of an operand lie within 2^31 bytes.
bool plan_fits(uint64_t ntokens, uint64_t vocab, uint64_t width, ar_dtype_t dtype)
{
    const uint64_t most = uint64_t(1) << (dtype == AR_FLOAT32 ? 20 : 24);
    return ntokens < most && width < most && vocab < kMaxIndex / 8 &&
           ceil_div(ntokens, 128) * ceil_div(vocab, 256) < kMaxGrid / 16;
}

// The operand can be read as it lies.
bool direct(const void* p, size_t ld, uint64_t width, size_t elem, bool pieces)
{
    return !pieces && width * elem % 16 == 0 && rows16(p, ld, elem) && ld < (size_t(1) << 25) / elem;
}

}  // namespace

AR_EXPORT size_t ar_clip_workspace_bytes(void) { return sizeof(ar::lm::ClipWorkspace); }

AR_EXPORT ar_result_t ar_grad_norm(ar_comm_t comm, int ntensors, const void* const grads[], const size_t counts[],
                                   ar_dtype_t dtype, ar_grads_t layout, ar_norm_t norm, float* norm_out,
                                   hipStream_t stream)
{
    return guarded([&] {
        return clip_impl(comm, ntensors, grads, nullptr, false, counts, dtype, layout, norm, 0.0, norm_out, stream);
    });
}

AR_EXPORT ar_result_t ar_clip_grads(ar_comm_t comm, int ntensors, const void* const sendbufs[], void* const recvbufs[],
                                    const size_t counts[], ar_dtype_t dtype, ar_grads_t layout, ar_norm_t norm,
                                    double max_norm, float* norm_out, hipStream_t stream)
{
    return guarded([&] {
        return clip_impl(comm, ntensors, sendbufs, recvbufs, true, counts, dtype, layout, norm, max_norm, norm_out,
                         stream);
    });
}

AR_EXPORT ar_result_t ar_all_reduce_clip(ar_comm_t comm, int ntensors, const void* const sendbufs[],
                                         void* const recvbufs[], const size_t counts[], ar_dtype_t dtype, ar_op_t op,
                                         ar_norm_t norm, double max_norm, float* norm_out, hipStream_t stream)
{
    return guarded([&] {
        ar_result_t rc = check_clip(comm, ntensors, sendbufs, recvbufs, true, counts, dtype, norm, max_norm,
                                    norm_out);
        if (rc != AR_SUCCESS) return rc;
        if (!valid_op(op)) return fail(AR_ERR_INVALID_ARGUMENT, "invalid op %d", static_cast<int>(op));
        if (op != AR_SUM && op != AR_AVG) return fail(AR_ERR_UNSUPPORTED, "gradients are clipped after AR_SUM or AR_AVG");
        uint64_t total, touched;
        rc = check_tensors(comm, ntensors, sendbufs, recvbufs, counts, dtype, false, norm_out, &total, &touched);
        if (rc != AR_SUCCESS) return rc;
        const int n = comm->nranks;
        const size_t e = elem_size(dtype);
        const uint64_t q = ceil_div(total, static_cast<uint64_t>(n));
        Batches reduce(ar::lm::kClipReduce, n, 1, e), apply(ar::lm::kClipApply, 1, n, e);
        std::vector<const void*> ptrs(1 + static_cast<size_t>(n));
        uint64_t off = 0;
        for (int t = 0; t < ntensors; ++t) {
            if (counts[t] == 0) continue;
            const size_t at = static_cast<size_t>(t) * n;
            std::copy(sendbufs + at, sendbufs + at + n, ptrs.begin());
            ptrs[n] = recvbufs[at];
            reduce.add(ptrs.data(), counts[t], off, q);
            ptrs[0] = recvbufs[at];
            std::copy(recvbufs + at, recvbufs + at + n, ptrs.begin() + 1);
            apply.add(ptrs.data(), counts[t], 0, 0);
            off += counts[t];
        }
        if ((rc = reduce.finish()) != AR_SUCCESS || (rc = apply.finish()) != AR_SUCCESS) return rc;
        return run_clip(comm, ar::lm::kClipReduce, reduce, &apply, n, dtype, op, norm, max_norm, touched, norm_out,
                        stream);
    });
}

AR_EXPORT ar_result_t ar_embedding(ar_comm_t comm, const void* weight, const void* tokens, ar_index_t index, void* out,
                                   size_t ntokens, size_t rows, size_t width, size_t ld_weight, size_t ld_out,
                                   long long first_row, float scale, ar_dtype_t dtype, hipStream_t stream)
{
    return guarded([&] {
        if (!comm) return fail(AR_ERR_INVALID_ARGUMENT, "comm is NULL");
        ar_result_t rc = check_float(dtype);
        if (rc == AR_SUCCESS) rc = check_index(index);
        if (rc == AR_SUCCESS) rc = check_sizes(ntokens, rows, width, "rows");
        std::vector<Interval> reads, writes;
        const size_t e = elem_size(dtype);
        if (rc == AR_SUCCESS) rc = check_matrix("weight", weight, rows, width, &ld_weight, e, &reads);
        if (rc == AR_SUCCESS) rc = check_matrix("out", out, ntokens, width, &ld_out, e, &writes);
        if (rc == AR_SUCCESS) rc = check_vector("tokens", tokens, ntokens, index_bytes(index), &reads);
        if (rc == AR_SUCCESS) rc = check_disjoint(reads, writes);
        if (rc != AR_SUCCESS || ntokens == 0) return rc;
        DeviceGuard g(comm->device);
        if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
        const ar::lm::LookupArgs a{weight, out,       {tokens, index == AR_INDEX_INT64}, ntokens, rows, width,
                                   ld_weight, ld_out, first_row,                         scale};
        const hipError_t err = ar::lm::launch_lookup(a, dtype, stream);
        return err == hipSuccess ? AR_SUCCESS : hip_fail(err, "kernel launch");
    });
}

AR_EXPORT size_t ar_embedding_workspace_bytes(size_t ntokens, size_t rows, size_t width)
{
    GradLayout l;
    return grad_layout(ntokens, rows, width, &l) ? l.bytes : static_cast<size_t>(-1);
}

AR_EXPORT ar_result_t ar_embedding_backward(ar_comm_t comm, const void* grad_out, const void* tokens, ar_index_t index,
                                            void* grad_weight, size_t ntokens, size_t rows, size_t width,
                                            size_t ld_grad_out, size_t ld_grad_weight, long long first_row,
                                            float scale, ar_dtype_t dtype, ar_dtype_t grad_dtype, int accumulate,
                                            hipStream_t stream)
{
    return guarded([&] {
        if (!comm) return fail(AR_ERR_INVALID_ARGUMENT, "comm is NULL");
        ar_result_t rc = check_float(dtype);
        if (rc == AR_SUCCESS) rc = check_float(grad_dtype);
        if (rc != AR_SUCCESS) return rc;
        if (grad_dtype != dtype && grad_dtype != AR_FLOAT32)
            return fail(AR_ERR_UNSUPPORTED, "grad_dtype is dtype or fp32");
        rc = check_index(index);
        if (rc == AR_SUCCESS) rc = check_sizes(ntokens, rows, width, "rows");
        std::vector<Interval> reads, writes;
        const size_t e = elem_size(dtype), ge = elem_size(grad_dtype);
        if (rc == AR_SUCCESS) rc = check_matrix("grad_out", grad_out, ntokens, width, &ld_grad_out, e, &reads);
        if (rc == AR_SUCCESS) rc = check_matrix("grad_weight", grad_weight, rows, width, &ld_grad_weight, ge, &writes);
        if (rc == AR_SUCCESS) rc = check_vector("tokens", tokens, ntokens, index_bytes(index), &reads);
        if (rc != AR_SUCCESS || rows == 0) return rc;
        GradLayout l;
        if (!grad_layout(ntokens, rows, width, &l)) return fail(AR_ERR_INVALID_ARGUMENT, "the workspace size overflows");
        if ((rc = check_workspace(comm, l.bytes)) != AR_SUCCESS) return rc;
        const uintptr_t w = reinterpret_cast<uintptr_t>(comm->ws);
        writes.push_back({w, w + l.bytes, "workspace", 0});
        if ((rc = check_disjoint(reads, writes)) != AR_SUCCESS) return rc;
        if (ntokens == 0 && accumulate) return AR_SUCCESS;
        DeviceGuard g(comm->device);
        if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
        char* ws = static_cast<char*>(comm->ws);
        ar::lm::LookupGradArgs a{};
        a.grad_out = grad_out;
        a.grad_weight = grad_weight;
        a.tokens = {tokens, index == AR_INDEX_INT64};
        a.ntokens = ntokens;
        a.rows = rows;
        a.width = width;
        a.ld_grad_out = ld_grad_out;
        a.ld_grad_weight = ld_grad_weight;
        a.first_row = first_row;
        a.scale = scale;
        a.accumulate = accumulate ? 1 : 0;
        for (int k = 0; k < 2; ++k) {
            a.key[k] = reinterpret_cast<uint32_t*>(ws + l.key[k]);
            a.pos[k] = reinterpret_cast<uint32_t*>(ws + l.pos[k]);
        }
        a.present = reinterpret_cast<uint8_t*>(ws + l.present);
        a.hist = reinterpret_cast<uint32_t*>(ws + l.hist);
        a.clear_words = (l.partial - l.present) / 4;
        a.partial = reinterpret_cast<float*>(ws + l.partial);
        const size_t unit = 16 / std::min(e, ge);  // elements a thread takes together
        const bool vec = width % unit == 0 && rows16(grad_weight, ld_grad_weight, ge) &&
                         (ntokens == 0 || rows16(grad_out, ld_grad_out, e));
        const uint64_t touched = ntokens * width * e + (accumulate ? 0 : rows * width * ge);
        const bool nt = call_nt(comm, touched, kLastLevelCacheBytes);
        const hipError_t err = ar::lm::launch_lookup_grad(a, dtype, grad_dtype, vec, nt, comm->num_cus, stream);
        return err == hipSuccess ? AR_SUCCESS : hip_fail(err, "kernel launch");
    });
}

AR_EXPORT size_t ar_linear_cross_entropy_workspace_bytes(size_t ntokens, size_t vocab, size_t width, ar_dtype_t dtype,
                                                         int backward)
{
    if (!valid_dtype(dtype) || dtype == AR_INT32 || width == 0 || !plan_fits(ntokens, vocab, width, dtype))
        return static_cast<size_t>(-1);
    return ar::lm::cross_entropy_bytes(ntokens, vocab, width, dtype, backward != 0);
}

namespace {

ar_result_t cross_entropy_common(ar_comm* comm, const void* hidden, const void* weight, const void* targets,
                                 ar_index_t index, size_t ntokens, size_t vocab, size_t width, size_t* ld_hidden,
                                 size_t* ld_weight, ar_dtype_t dtype, bool backward, std::vector<Interval>* reads,
                                 ar::lm::CrossEntropyPlan* plan)
{
    if (!comm) return fail(AR_ERR_INVALID_ARGUMENT, "comm is NULL");
    ar_result_t rc = check_float(dtype);
    if (rc == AR_SUCCESS) rc = check_index(index);
    if (rc == AR_SUCCESS) rc = check_sizes(ntokens, vocab, width, "vocab");
    if (rc != AR_SUCCESS) return rc;
    if (vocab == 0) return fail(AR_ERR_INVALID_ARGUMENT, "vocab is 0");
    if (!plan_fits(ntokens, vocab, width, dtype))
        return fail(AR_ERR_INVALID_ARGUMENT, "ntokens %zu, vocab %zu, width %zu: too large for one call", ntokens,
                    vocab, width);
    const size_t e = elem_size(dtype);
    rc = check_matrix("hidden", hidden, ntokens, width, ld_hidden, e, reads);
    if (rc == AR_SUCCESS) rc = check_matrix("weight", weight, vocab, width, ld_weight, e, reads);
    if (rc == AR_SUCCESS) rc = check_vector("targets", targets, ntokens, index_bytes(index), reads);
    if (rc != AR_SUCCESS) return rc;
    *plan = ar::lm::plan_cross_entropy(ntokens, vocab, width, dtype, backward);
    plan->pack_hidden = !direct(hidden, *ld_hidden, width, e, plan->pieces);
    plan->pack_weight = !direct(weight, *ld_weight, width, e, plan->pieces);
    return check_workspace(comm, ar::lm::cross_entropy_bytes(ntokens, vocab, width, dtype, backward));
}

}  // namespace

AR_EXPORT ar_result_t ar_linear_cross_entropy(ar_comm_t comm, const void* hidden, const void* weight,
                                              const void* targets, ar_index_t index, float* losses, float* lse,
                                              size_t ntokens, size_t vocab, size_t width, size_t ld_hidden,
                                              size_t ld_weight, long long ignore_index, ar_dtype_t dtype,
                                              hipStream_t stream)
{
    return guarded([&] {
        std::vector<Interval> reads, writes;
        ar::lm::CrossEntropyPlan p;
        ar_result_t rc = cross_entropy_common(comm, hidden, weight, targets, index, ntokens, vocab, width, &ld_hidden,
                                              &ld_weight, dtype, false, &reads, &p);
        if (rc == AR_SUCCESS) rc = check_vector("losses", losses, ntokens, 4, &writes);
        if (rc == AR_SUCCESS) rc = check_vector("lse", lse, ntokens, 4, &writes);
        if (rc != AR_SUCCESS) return rc;
        const uintptr_t w = reinterpret_cast<uintptr_t>(comm->ws);
        writes.push_back({w, w + p.bytes, "workspace", 0});
        if ((rc = check_disjoint(reads, writes)) != AR_SUCCESS || ntokens == 0) return rc;
        DeviceGuard g(comm->device);
        if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
        ar::lm::CrossEntropyArgs a{};
        a.hidden = hidden;
        a.weight = weight;
        a.targets = {targets, index == AR_INDEX_INT64};
        a.losses = losses;
        a.lse = lse;
        a.ntokens = ntokens;
        a.vocab = vocab;
        a.width = width;
        a.ld_hidden = ld_hidden;
        a.ld_weight = ld_weight;
        a.ignore_index = ignore_index;
        const hipError_t err = ar::lm::launch_cross_entropy(a, p, dtype, static_cast<char*>(comm->ws), stream);
        return err == hipSuccess ? AR_SUCCESS : hip_fail(err, "kernel launch");
    });
}

AR_EXPORT ar_result_t ar_linear_cross_entropy_backward(ar_comm_t comm, const void* hidden, const void* weight,
                                                       const void* targets, ar_index_t index, const float* lse,
                                                       const float* grad_losses, void* grad_hidden, void* grad_weight,
                                                       size_t ntokens, size_t vocab, size_t width, size_t ld_hidden,
                                                       size_t ld_weight, size_t ld_grad_hidden, size_t ld_grad_weight,
                                                       long long ignore_index, ar_dtype_t dtype, hipStream_t stream)
{
    return guarded([&] {
        std::vector<Interval> reads, writes;
        ar::lm::CrossEntropyPlan p;
        ar_result_t rc = cross_entropy_common(comm, hidden, weight, targets, index, ntokens, vocab, width, &ld_hidden,
                                              &ld_weight, dtype, true, &reads, &p);
        if (rc != AR_SUCCESS) return rc;
        const size_t e = elem_size(dtype);
        rc = check_vector("lse", lse, ntokens, 4, &reads);
        if (rc == AR_SUCCESS) rc = check_vector("grad_losses", grad_losses, ntokens, 4, &reads);
        if (rc == AR_SUCCESS && grad_hidden)
            rc = check_matrix("grad_hidden", grad_hidden, ntokens, width, &ld_grad_hidden, e, &writes);
        if (rc == AR_SUCCESS && grad_weight)
            rc = check_matrix("grad_weight", grad_weight, vocab, width, &ld_grad_weight, e, &writes);
        if (rc != AR_SUCCESS) return rc;
        if (!grad_hidden && !grad_weight)
            return fail(AR_ERR_INVALID_ARGUMENT, "grad_hidden and grad_weight are both NULL");
        const uintptr_t w = reinterpret_cast<uintptr_t>(comm->ws);
        writes.push_back({w, w + p.bytes, "workspace", 0});
        if ((rc = check_disjoint(reads, writes)) != AR_SUCCESS) return rc;
        if (ntokens == 0 && !grad_weight) return AR_SUCCESS;
        DeviceGuard g(comm->device);
        if (g.err != hipSuccess) return hip_fail(g.err, "hipSetDevice");
        ar::lm::CrossEntropyArgs a{};
        a.hidden = hidden;
        a.weight = weight;
        a.targets = {targets, index == AR_INDEX_INT64};
        a.lse = const_cast<float*>(lse);
        a.grad_losses = grad_losses;
        a.grad_hidden = grad_hidden;
        a.grad_weight = grad_weight;
        a.ntokens = ntokens;
        a.vocab = vocab;
        a.width = width;
        a.ld_hidden = ld_hidden;
        a.ld_weight = ld_weight;
        a.ld_grad_hidden = ld_grad_hidden;
        a.ld_grad_weight = ld_grad_weight;
        a.ignore_index = ignore_index;
        const hipError_t err = ar::lm::launch_cross_entropy_backward(a, p, dtype, static_cast<char*>(comm->ws), stream);
        return err == hipSuccess ? AR_SUCCESS : hip_fail(err, "kernel launch");
    });
}
