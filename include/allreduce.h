/*
 * allreduce.h -- C ABI of liballreduce, a ring all-reduce engine for one
 * AMD Instinct MI355X (gfx950) on which N "virtual ranks" are N separate
 * device buffers.
 *
 * Sources (web pages, cited by title and section):
 *  [P1] mhpq.cn news/451051, article on how all-reduce keeps every card's
 *       model identical: s2.1 (all-reduce semantics; SUM, AVG = sum then
 *       divide by N, MAX, MIN, PROD), s2.2 (every rank takes part with
 *       matching shapes; deterministic result), s3.2 (ring = reduce-scatter
 *       then all-gather), s5.3 (reduce fp16/bf16 gradients in fp32).
 *  [P2] xxqk.cn news/376101, article on AllReduce bottlenecks: s4.3 (do not
 *       mix dtypes inside one reduction).
 *  [P3] geek-doc.cn, "训练梯度同步与集合通信:从参数服务器到 Ring AllReduce":
 *       section 三 (the two ring phases of N-1 steps each), section 四
 *       (2(N-1)/N * M bytes per rank; alpha-beta model), section 六
 *       (reduce-scatter and all-gather used on their own, as in ZeRO/FSDP).
 *  [P4] anrans.github.io handbook, "集合通信原语": section 五个原语
 *       (all_reduce, reduce_scatter_tensor gives rank r block r,
 *       all_gather_into_tensor concatenates in rank order), section
 *       环形 all-reduce 与通信量 (the ring's index schedule), section α-β 模型
 *       (one-shot direct-read all-reduce for small messages).
 *
 * The pages' interface is one call per process and rank. Here one call
 * carries every rank's buffer: sendbufs[r] / recvbufs[r] are rank r's
 * device buffers, r = 0..nranks-1, so no rank can miss the call.
 *
 * Conventions for every entry point:
 *  - Pointers in sendbufs[] / recvbufs[] are device pointers on the comm's
 *    device; the arrays themselves are host memory, read only during the
 *    call. The caller owns all device memory, the workspace and the stream,
 *    and keeps them alive until the enqueued work has completed.
 *  - Calls are stream-ordered and asynchronous: they return once the work is
 *    enqueued on `stream` (NULL = the device's null stream).
 *  - Errors are returned, never raised: no call aborts or exits. A failing
 *    call enqueues nothing, except AR_ERR_HIP, which reports a launch error
 *    after earlier steps may have been enqueued. ar_last_error() gives a
 *    thread-local message for the last failure.
 *  - count == 0 (or recvcount/sendcount == 0) is a successful no-op.
 *  - Results are deterministic: the same inputs give the same bits on every
 *    call, and the ring modes (fused, stepwise, graph) give the same bits.
 *  - A comm holds mutable state (workspace, timing events, graph cache): calls
 *    on one comm must not run concurrently from several host threads. Calls
 *    on different comms may.
 */
#ifndef LIBALLREDUCE_ALLREDUCE_H
#define LIBALLREDUCE_ALLREDUCE_H

#include <stddef.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define AR_MAX_RANKS 64
#define AR_MAX_TENSORS 65536
/* Bytes of the library-owned device scratch array that ar_all_reduce_noalloc
 * uses on each GPU (64 MiB). */
#define AR_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

typedef struct ar_comm* ar_comm_t;

typedef enum {
    AR_SUCCESS = 0,
    AR_ERR_INVALID_ARGUMENT = 1, /* bad pointer, enum, size, alias or workspace */
    AR_ERR_UNSUPPORTED = 2,      /* a valid request the library does not serve */
    AR_ERR_HIP = 3,              /* a HIP runtime call or kernel launch failed */
    AR_ERR_OUT_OF_MEMORY = 4,    /* host allocation for the comm failed */
    AR_ERR_INTERNAL = 5
} ar_result_t;

/* Storage types. fp16 and bf16 are reduced in fp32 and rounded once, to
 * nearest even, at the end [P1 s5.3]; int32 wraps modulo 2^32. One dtype
 * per call [P2 s4.3]. */
typedef enum { AR_FLOAT32 = 0, AR_FLOAT16 = 1, AR_BFLOAT16 = 2, AR_INT32 = 3 } ar_dtype_t;

/* Reduce ops [P1 s2.1]. AVG is the sum divided once by nranks (fp: one
 * correctly rounded fp32 divide; int32: truncation toward zero). MAX/MIN
 * return NaN when either operand is NaN and order +0 above -0. */
typedef enum { AR_SUM = 0, AR_AVG = 1, AR_MAX = 2, AR_MIN = 3, AR_PROD = 4 } ar_op_t;

/* AR_MODE_FUSED: one launch that reads every rank's element once and writes
 * the result to every output -- the direct-read ("one-shot") pattern [P4
 * section α-β 模型] -- folding the ranks in ring order, so its bits equal the
 * ring's.
 * AR_MODE_RING_STEPWISE: the ring itself, one launch per ring step:
 * N-1 reduce-scatter steps then N-1 all-gather steps [P3 section 三;
 * P4 section 环形 all-reduce 与通信量].
 * AR_MODE_RING_GRAPH: the same ring steps, captured once into a HIP graph
 * per call signature (collective, buffer pointers, count, dtype, op,
 * workspace) and replayed as one graph launch afterwards, which removes the
 * per-step launch cost that the alpha term of the alpha-beta model charges
 * [P3 section 四; P4 section α-β 模型: graph-captured custom all-reduce].
 * A comm keeps up to 16 graphs (least recently used evicted). The pointers
 * in a cached graph are fixed: a later call with the same pointers and sizes
 * replays it whatever the buffers now hold. Must not be used while `stream`
 * is itself being captured (INVALID_ARGUMENT): capture AR_MODE_RING_STEPWISE
 * or AR_MODE_FUSED instead -- both are capture-safe (no synchronous calls,
 * no memsets, no allocation). Same bits as the other modes. */
/* AR_MODE_TREE and AR_MODE_TREE_STEPWISE (all-reduce only; other
 * collectives return UNSUPPORTED): the tree variant [P3 section 六]. Ranks
 * combine in pairs, the pair results combine in pairs again, and after
 * ceil(log2 N) levels rank 0 holds the reduction, which is broadcast back
 * down: level l pairs rank r (a multiple of 2^(l+1)) with r + 2^l. Every
 * element is folded in that order (no chunks), so for fp SUM/AVG/PROD the
 * bits differ from the ring's; the difference is bounded by
 * 4*N*eps*sum|x_i| (eps = 2^-23, plus one output ulp for fp16/bf16).
 * AR_MODE_TREE: one launch, each element's tree evaluated in registers.
 * AR_MODE_TREE_STEPWISE: 2*ceil(log2 N) launches (the pages' step count);
 * fp16/bf16 partials need ar_workspace_bytes(...) of fp32 workspace. */
typedef enum {
    AR_MODE_FUSED = 0,
    AR_MODE_RING_STEPWISE = 1,
    AR_MODE_RING_GRAPH = 2,
    AR_MODE_TREE = 3,
    AR_MODE_TREE_STEPWISE = 4
} ar_mode_t;

/* Access flavour of the one-launch calls; see ar_comm_set_access. */
typedef enum {
    AR_ACCESS_AUTO = 0,
    AR_ACCESS_STREAMING = 1,
    AR_ACCESS_CACHED = 2
} ar_access_t;

typedef enum {
    AR_COLL_ALL_REDUCE = 0,
    AR_COLL_REDUCE_SCATTER = 1,
    AR_COLL_ALL_GATHER = 2,
    AR_COLL_ALL_TO_ALL = 3
} ar_collective_t;

/* Create a communicator for `nranks` (1..AR_MAX_RANKS) virtual ranks on HIP
 * device `hip_device`. On success *comm owns host state and a few HIP
 * events; release it with ar_comm_destroy. Errors: INVALID_ARGUMENT for a
 * NULL comm pointer or nranks out of range, HIP if the device cannot be
 * queried, OUT_OF_MEMORY. */
ar_result_t ar_comm_create(ar_comm_t* comm, int nranks, int hip_device);

/* Destroy a communicator (NULL is a no-op). Work already enqueued that uses
 * it must have completed. */
ar_result_t ar_comm_destroy(ar_comm_t comm);

/* Number of ranks the communicator was created with, or -1 for NULL. */
int ar_comm_nranks(ar_comm_t comm);

/* Device workspace (bytes) a call needs; 0 when none. `count` is the
 * collective's own count argument (count, recvcount or sendcount).
 * The ring modes (stepwise and graph) need it: all-reduce of fp16/bf16
 * keeps fp32 partial sums, 4*count bytes; reduce-scatter keeps the partials
 * of all nranks blocks, 4*nranks*recvcount bytes. AR_MODE_TREE_STEPWISE
 * with fp16/bf16 keeps floor(N/2) fp32 partial buffers:
 * 4*floor(N/2)*roundup(count, 4) bytes. Everything else: 0. Returns (size_t)-1 for
 * invalid arguments or if the size overflows. */
size_t ar_workspace_bytes(ar_collective_t coll, int nranks, size_t count, ar_dtype_t dtype, ar_mode_t mode);

/* Attach a caller-owned device workspace (16-byte aligned, `bytes` long) to
 * the communicator; NULL/0 detaches it. The library never allocates device
 * memory itself. Calls that share a workspace must be ordered on one
 * stream. Errors: INVALID_ARGUMENT for a NULL comm, a misaligned pointer,
 * or bytes > 0 with a NULL pointer. */
ar_result_t ar_comm_set_workspace(ar_comm_t comm, void* dev_ptr, size_t bytes);

/* All-reduce [P1 s2.1; P3 section 三; P4 section 五个原语]: after the call
 * recvbufs[r][i] = op over ranks of sendbufs[r][i], i < count, identical for
 * every r. Chunk c of the ring is elements [c*q, min((c+1)*q, count)) with
 * q = ceil(count/nranks), and chunk c is folded in rank order
 * c, c+1, ..., c+nranks-1 (mod nranks): acc = x_c; acc = x_{c+k} (+) acc.
 * sendbufs[r] and recvbufs[r] each hold `count` elements of `dtype`.
 * In place is allowed (sendbufs[r] == recvbufs[r]); any other overlap
 * between any two of the 2*nranks buffers (or the workspace) is
 * INVALID_ARGUMENT. Ring-mode fp16/bf16 needs a workspace of
 * ar_workspace_bytes(...) bytes, else INVALID_ARGUMENT. Pointers must be
 * aligned to the element size (else INVALID_ARGUMENT). With every pointer
 * 16-byte aligned the fused kernel moves 16-byte vectors (chunk ends that
 * fall inside a vector are done element by element); the stepwise steps
 * also need q to be a multiple of 16/sizeof(dtype). Other layouts take
 * element-wise kernels. The results are the same bits either way. */
ar_result_t ar_all_reduce(ar_comm_t comm, const void* const sendbufs[], void* const recvbufs[], size_t count,
                          ar_dtype_t dtype, ar_op_t op, ar_mode_t mode, hipStream_t stream);

/* Allocation-free all-reduce, for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc. Same arguments, results (bit for bit) and errors as
 * ar_all_reduce, with these differences:
 *  - the fp32 partial sums of the ring-stepwise and tree-stepwise fp16/bf16
 *    paths live in a library-owned device array of AR_NOALLOC_SCRATCH_BYTES
 *    on each GPU (set up by ar_comm_create, held until the process ends);
 *    the comm's workspace is not used. A call that would need more, i.e.
 *    ar_workspace_bytes(AR_COLL_ALL_REDUCE, ...) > AR_NOALLOC_SCRATCH_BYTES
 *    (ring-stepwise fp16/bf16 beyond 16,777,216 elements per rank), is
 *    INVALID_ARGUMENT;
 *  - AR_MODE_RING_GRAPH is UNSUPPORTED (instantiating a graph allocates);
 *  - step timing (ar_comm_set_step_timing) records nothing for this call.
 * The call allocates nothing: no hipMalloc, hipFree, event or graph. The
 * caller still owns the send and recv buffers and the stream.
 * Every call on one GPU shares that GPU's array, which keeps the last call's
 * contents (nothing in it needs to start at zero: each step writes a slot
 * before any later step reads it). Calls on one GPU that may overlap in time
 * (unordered streams, several host threads) race on the array: the caller
 * must order them. INVALID_ARGUMENT also if ar_comm_create could not look
 * up the array's address on the comm's device (ar_last_error says why). */
ar_result_t ar_all_reduce_noalloc(ar_comm_t comm, const void* const sendbufs[], void* const recvbufs[], size_t count,
                                  ar_dtype_t dtype, ar_op_t op, ar_mode_t mode, hipStream_t stream);

/* Reduce-scatter [P3 section 六; P4 section 五个原语]: sendbufs[r] holds
 * nranks*recvcount elements; recvbufs[c] (recvcount elements) receives
 * block c of the reduction, block c being folded in the same ring order as
 * in ar_all_reduce, so reduce-scatter followed by all-gather equals
 * all-reduce bit for bit. In place: recvbufs[r] == sendbufs[r] +
 * r*recvcount elements. The ring modes need a workspace of
 * ar_workspace_bytes(...) bytes. Errors as ar_all_reduce. */
ar_result_t ar_reduce_scatter(ar_comm_t comm, const void* const sendbufs[], void* const recvbufs[],
                              size_t recvcount, ar_dtype_t dtype, ar_op_t op, ar_mode_t mode, hipStream_t stream);

/* All-gather [P3 section 六; P4 section 五个原语]: sendbufs[r] holds
 * sendcount elements; every recvbufs[r] (nranks*sendcount elements)
 * receives the nranks send blocks in rank order. In place:
 * sendbufs[r] == recvbufs[r] + r*sendcount elements. Errors as
 * ar_all_reduce (no workspace is needed). */
ar_result_t ar_all_gather(ar_comm_t comm, const void* const sendbufs[], void* const recvbufs[], size_t sendcount,
                          ar_dtype_t dtype, ar_mode_t mode, hipStream_t stream);

/* All-to-all, the "transpose" primitive [P4 section 五个原语 (all_to_all_single:
 * rank r's p-th block goes to rank p); P3 section 六]: sendbufs[r] holds
 * nranks blocks of blockcount elements; block r of recvbufs[p] receives
 * block p of sendbufs[r], for every r and p. Each rank sends (n-1)/n of its
 * data. AR_MODE_FUSED moves every block in one launch; the ring modes take n
 * steps, step s moving block (r + s) mod n of every rank r (step 0 is each
 * rank's own block). No workspace. Send and recv buffers must not overlap at
 * all (there is no in-place form); errors otherwise as ar_all_reduce. */
ar_result_t ar_all_to_all(ar_comm_t comm, const void* const sendbufs[], void* const recvbufs[], size_t blockcount,
                          ar_dtype_t dtype, ar_mode_t mode, hipStream_t stream);

/* Coalesced multi-tensor all-reduce: many gradient tensors reduced in one
 * call without packing them into a bucket first -- the pages' gradient
 * bucketing and small-tensor fusion [P1 s5.1-s5.2 (DDP buckets, default
 * 25 MB); P2 s5.3 (merge same-shape gradients into one call); P3 section 四
 * (fuse small tensors so the per-step latency is paid once)].
 * Tensor t of rank r is sendbufs[t*nranks + r] / recvbufs[t*nranks + r]
 * with counts[t] elements (t < ntensors <= AR_MAX_TENSORS; empty tensors
 * allowed). The tensors of a rank form one virtual flat bucket, in tensor
 * order; the ring's chunks are taken over that bucket, so every element gets
 * exactly the bits ar_all_reduce gives on the packed bucket. Each tensor may
 * be in place (send == recv); any other overlap is INVALID_ARGUMENT.
 * AR_MODE_FUSED only (other modes: UNSUPPORTED). Launches: one per batch of
 * tensors whose rank pointers fit the kernel arguments (about 3.8 KB; a
 * tensor in place on every rank takes n pointers, otherwise 2n: e.g. about
 * 40 in-place tensors per launch at 8 ranks, 6 at 64). Tensors whose rank
 * pointers all sit at the same offset from a 16-byte boundary are read and
 * written in 16-byte vectors; others element by element. When the pointers
 * also share their offset from a 128-byte line (views at one offset into
 * per-rank buckets), the vectors start on the tensor's first whole line,
 * which keeps every wave's access to whole lines. No workspace. */
ar_result_t ar_all_reduce_multi(ar_comm_t comm, int ntensors, const void* const sendbufs[], void* const recvbufs[],
                                const size_t counts[], ar_dtype_t dtype, ar_op_t op, ar_mode_t mode,
                                hipStream_t stream);

/* Per-step timing of stepwise calls (the alpha-beta model's per-step cost,
 * [P3 section 四; P4 section α-β 模型]). When enabled, each stepwise call
 * records a HIP event before its first step and after every step; fused
 * and graph-mode calls record one interval. Recording adds a little
 * per-step overhead and is not meant for the caller's own graph capture. */
ar_result_t ar_comm_set_step_timing(ar_comm_t comm, int enable);

/* Access flavour of the one-launch calls (fused and tree all-reduce, fused
 * reduce-scatter, all-gather and all-to-all, multi-tensor all-reduce): with
 * non-temporal ("streaming") loads and stores, which pass data through the
 * caches without keeping it, or with ordinary cached ones, which let a call
 * on buffers still in the 256 MB last-level cache run from it.
 *  AR_ACCESS_AUTO (the default): non-temporal when the call's distinct bytes
 *    exceed half the last-level cache for the all-reduce (a footprint that
 *    large is unlikely to be resident in full, and cold calls gain more than
 *    warm ones lose: 8 ranks x 25 MiB fp32, 73 against 86 us cold, 71
 *    against 62 us warm) and the whole cache for the other collectives;
 *  AR_ACCESS_STREAMING: non-temporal at every size, for buffers known to
 *    come from HBM;
 *  AR_ACCESS_CACHED: cached whenever the footprint fits in the cache, for
 *    buffers a kernel has just written (e.g. a gradient bucket right after
 *    the backward pass).
 * Launch shapes follow the flavour chosen; results are the same bits either
 * way. The ring-stepwise and graph modes always use cached access except the
 * all-to-all steps beyond the cache. The setting is per comm and takes
 * effect from the next call. NULL comm or an unknown value:
 * INVALID_ARGUMENT. */
ar_result_t ar_comm_set_access(ar_comm_t comm, ar_access_t access);

/* ar_comm_set_access(comm, enable ? AR_ACCESS_STREAMING : AR_ACCESS_AUTO). */
ar_result_t ar_comm_set_streaming(ar_comm_t comm, int enable);

/* Step durations (ms) of the last timed call on this comm: waits for that
 * call's last event, writes min(cap, steps) values to out and the step
 * count to *nsteps. INVALID_ARGUMENT if timing was off or nothing was
 * timed yet. */
ar_result_t ar_last_step_times_ms(ar_comm_t comm, float* out, int cap, int* nsteps);

/* ---- language-model operators around the gradient all-reduce -------------
 *
 * What a training step does next to the all-reduce: the global norm of the
 * gradients and their clip, the embedding at one end of the model and the
 * softmax cross entropy of the linear head at the other, whose gradients are
 * the largest tensors of a data-parallel bucket.
 *
 * The clip calls carry every rank's buffers, as ar_all_reduce_multi; the
 * embedding and cross-entropy calls work on one rank's data (a rank's forward
 * or backward pass) and take the comm for its device and workspace. Types are
 * fp32, fp16 and bf16 (int32: UNSUPPORTED). All calls are stream-ordered,
 * deterministic and capture-safe, and allocate no device memory. Calls that
 * need a workspace take the comm's (ar_comm_set_workspace), of at least the
 * size that the operator's ..._workspace_bytes gives, else INVALID_ARGUMENT;
 * what they leave in it is of no further use. Row pitches (ld_...) are in
 * elements, 0 meaning the row length. Buffers that a call writes may overlap
 * none that it reads or writes (and not the workspace) except where a call
 * says so; anything else is INVALID_ARGUMENT. */

/* Type of token and target numbers. */
typedef enum { AR_INDEX_INT32 = 0, AR_INDEX_INT64 = 1 } ar_index_t;

/* Norm over all elements: sqrt(sum x^2), or max |x|. */
typedef enum { AR_NORM_L2 = 0, AR_NORM_INF = 1 } ar_norm_t;

/* How the ranks hold the gradients. REPLICATED: every rank the same values,
 * as after an all-reduce; the norm is rank 0's, only rank 0's send buffers are
 * read, and every rank's recv buffers get its clipped values. SHARDED: every
 * rank its own part, as after a reduce-scatter; the norm goes over all ranks'
 * elements. */
typedef enum { AR_GRADS_REPLICATED = 0, AR_GRADS_SHARDED = 1 } ar_grads_t;

/* Workspace of the three calls below; the same for every size. */
size_t ar_clip_workspace_bytes(void);

/* *norm_out (device) = the norm of all gradients, rounded from fp64 sums of
 * fp64 squares, so that neither squares beyond fp32's range nor small
 * gradients beside large ones are lost. Tensor t of rank r is
 * grads[t*nranks + r] with counts[t] elements. NaN where an element is NaN; 0
 * over no elements. */
ar_result_t ar_grad_norm(ar_comm_t comm, int ntensors, const void* const grads[], const size_t counts[],
                         ar_dtype_t dtype, ar_grads_t layout, ar_norm_t norm, float* norm_out, hipStream_t stream);

/* Clips gradients to a global norm: recv = send * min(1, max_norm / (norm +
 * 1e-6)), the factor rounded once to fp32 and the product once to dtype. An
 * infinite norm gives the factor 0 (finite elements become 0, infinite ones
 * NaN), a NaN norm makes every element NaN; norm_out (device, may be NULL)
 * tells. max_norm: at least 0; an infinite one clips nothing (the factor is 1,
 * of an infinite norm too). In place per tensor and rank (send == recv) is
 * allowed. */
ar_result_t ar_clip_grads(ar_comm_t comm, int ntensors, const void* const sendbufs[], void* const recvbufs[],
                          const size_t counts[], ar_dtype_t dtype, ar_grads_t layout, ar_norm_t norm, double max_norm,
                          float* norm_out, hipStream_t stream);

/* ar_all_reduce_multi (SUM or AVG; other ops UNSUPPORTED) and ar_clip_grads of
 * its replicated result as one call (the same but for the order in which the
 * norm's fp64 squares are summed), in fewer passes: the reduction writes one copy and its norm, the clip reads that copy and writes
 * every rank's: 2(N+1)S bytes where the two calls move (3N+2)S. In place per
 * tensor and rank is allowed. */
ar_result_t ar_all_reduce_clip(ar_comm_t comm, int ntensors, const void* const sendbufs[], void* const recvbufs[],
                               const size_t counts[], ar_dtype_t dtype, ar_op_t op, ar_norm_t norm, double max_norm,
                               float* norm_out, hipStream_t stream);

/* Embedding lookup: out[t] = weight[tokens[t] - first_row] * scale, the product
 * in fp32 and rounded once; a row of zeros where tokens[t] - first_row is not
 * in [0, rows). weight holds rows first_row .. first_row + rows - 1 of the
 * vocabulary: where ranks share one, an all-reduce (SUM) of their outputs is
 * the whole lookup. No workspace. */
ar_result_t ar_embedding(ar_comm_t comm, const void* weight, const void* tokens, ar_index_t index, void* out,
                         size_t ntokens, size_t rows, size_t width, size_t ld_weight, size_t ld_out,
                         long long first_row, float scale, ar_dtype_t dtype, hipStream_t stream);

/* Workspace of ar_embedding_backward, also for fewer tokens; (size_t)-1 for
 * sizes it does not take. */
size_t ar_embedding_workspace_bytes(size_t ntokens, size_t rows, size_t width);

/* Its gradient: grad_weight[v] = scale * sum of grad_out[t] over the tokens t
 * with tokens[t] - first_row = v, summed in fp32 in a fixed order and rounded
 * once to grad_dtype (dtype or fp32). Every row is written, zeros where no
 * token falls; with accumulate != 0 the sum is added to what the row holds
 * (e.g. the head's gradient of a shared weight), and other rows are left
 * alone. Tokens outside [first_row, first_row + rows) add nothing. */
ar_result_t ar_embedding_backward(ar_comm_t comm, const void* grad_out, const void* tokens, ar_index_t index,
                                  void* grad_weight, size_t ntokens, size_t rows, size_t width, size_t ld_grad_out,
                                  size_t ld_grad_weight, long long first_row, float scale, ar_dtype_t dtype,
                                  ar_dtype_t grad_dtype, int accumulate, hipStream_t stream);

/* Workspace of ar_linear_cross_entropy (backward = 0) or its gradient
 * (backward != 0), also for fewer tokens; (size_t)-1 for sizes they do not
 * take. */
size_t ar_linear_cross_entropy_workspace_bytes(size_t ntokens, size_t vocab, size_t width, ar_dtype_t dtype,
                                               int backward);

/* Softmax cross entropy of the linear head weight [vocab][width] on hidden
 * [ntokens][width], in pieces of the vocabulary, without keeping the logits:
 *   z[t][v] = hidden[t] . weight[v],  lse[t] = log sum_v exp(z[t][v]),
 *   losses[t] = lse[t] - z[t][targets[t]].
 * A token whose target is ignore_index or outside [0, vocab) is ignored: its
 * loss is 0 (its lse is still given). Products of fp16 and bf16 are summed in
 * fp32; fp32 products are exact to 2^-24 (fp32 matrix instructions up to 64
 * tokens and for small problems, else bf16 pieces that hold all 24 bits; 2^-21
 * where both factors are of 256 or more). Products with an infinity, and beyond fp32's range, are the
 * infinity of their sign: a logit of -infinity adds nothing to lse, one of
 * +infinity, or a NaN, makes the token's lse and loss NaN. losses and lse are
 * fp32. ntokens and width are below 2^24, of fp32 below 2^20, vocab below 2^28.
 * Operands whose rows are on 16-byte boundaries and whole multiples of 16 bytes
 * long are read as they lie (fp32 ones by fp32 matrix instructions only); others
 * are first laid out in the workspace, at most 1 GiB of the weight at a time. */
ar_result_t ar_linear_cross_entropy(ar_comm_t comm, const void* hidden, const void* weight, const void* targets,
                                    ar_index_t index, float* losses, float* lse, size_t ntokens, size_t vocab,
                                    size_t width, size_t ld_hidden, size_t ld_weight, long long ignore_index,
                                    ar_dtype_t dtype, hipStream_t stream);

/* Its gradients, given lse of the forward call and the gradient of each loss
 * (e.g. 1 / number of tokens that count, for their mean):
 *   d[t][v] = grad_losses[t] * (exp(z[t][v] - lse[t]) - [v = targets[t]]),
 *   grad_hidden = d weight,  grad_weight = d^T hidden,
 * both of dtype and either may be NULL. Ignored tokens have zero grad_hidden
 * and add nothing to grad_weight, whatever their hidden row holds. For fp16
 * and bf16, d is rounded to that type once (scaled by 2^14 and, for grad_weight,
 * by the largest |grad_losses|, so that small probabilities do not underflow: in
 * fp16 steps of 2^-38, of the largest |grad_losses| for grad_weight, are left);
 * sums are fp32 and hold the 2^14. An infinite grad_losses of a token that
 * counts makes grad_weight NaN. */
ar_result_t ar_linear_cross_entropy_backward(ar_comm_t comm, const void* hidden, const void* weight,
                                             const void* targets, ar_index_t index, const float* lse,
                                             const float* grad_losses, void* grad_hidden, void* grad_weight,
                                             size_t ntokens, size_t vocab, size_t width, size_t ld_hidden,
                                             size_t ld_weight, size_t ld_grad_hidden, size_t ld_grad_weight,
                                             long long ignore_index, ar_dtype_t dtype, hipStream_t stream);

/* Workspace of ar_linear_log_probs with `top` alternatives (backward = 0) or of
 * its gradient (backward != 0; top is not looked at), also for fewer tokens and
 * fewer alternatives (but for at least one, if those are to be found);
 * (size_t)-1 for sizes they do not take. */
size_t ar_linear_log_probs_workspace_bytes(size_t ntokens, size_t vocab, size_t width, ar_dtype_t dtype, int top,
                                           int backward);

/* Log probabilities of given tokens under the linear head of
 * ar_linear_cross_entropy, at the inverse temperature `scale` (finite, above 0):
 *   z[t][v] = scale * (hidden[t] . weight[v]),  lse[t] = log sum_v exp z[t][v],
 *   log_probs[t] = z[t][targets[t]] - lse[t],
 *   entropy[t] = -sum_v p log p with p = exp(z[t][v] - lse[t])   (may be NULL).
 * The `top` (0 to 64, at most vocab) largest z of every token go to
 * top_log_probs[t][k] = z - lse[t] and top_ids[t][k], the largest first and of
 * equal ones the smaller id first; a NaN counts as -infinity among them.
 * Both may be NULL if top is 0. A token whose target is ignore_index or outside
 * [0, vocab) has the log probability 0; its other results are given. Products,
 * infinities, NaN and limits are as in ar_linear_cross_entropy (a logit of
 * -infinity adds nothing to the entropy; one of +infinity, or a NaN, makes all
 * results of its token but top_ids NaN); with alternatives vocab is below 2^24, and the
 * workspace holds the logits of up to 1 GiB worth of tokens (of 256 tokens at
 * the least). */
ar_result_t ar_linear_log_probs(ar_comm_t comm, const void* hidden, const void* weight, const void* targets,
                                ar_index_t index, float* log_probs, float* entropy, float* lse, int top,
                                float* top_log_probs, int* top_ids, size_t ntokens, size_t vocab, size_t width,
                                size_t ld_hidden, size_t ld_weight, float scale, long long ignore_index,
                                ar_dtype_t dtype, hipStream_t stream);

/* Its gradients, given lse and entropy of the forward call and the gradients of
 * each log probability and entropy (grad_entropy may be NULL: none comes
 * through it, and entropy is not read):
 *   dz[t][v] = grad_log_probs[t] ([v = targets[t]] - p) - grad_entropy[t] p (log p + entropy[t]),
 *   grad_hidden = scale dz weight,  grad_weight = scale dz^T hidden,
 * both of dtype and either may be NULL. A token whose target is ignore_index or
 * outside [0, vocab) has zero grad_hidden and adds nothing to grad_weight,
 * whatever its hidden row and gradients hold. For fp16 and bf16, dz over the
 * larger of the token's two gradients is rounded to that type once (times 2^12:
 * in fp16 steps of 2^-36 are left); sums are fp32. */
ar_result_t ar_linear_log_probs_backward(ar_comm_t comm, const void* hidden, const void* weight, const void* targets,
                                         ar_index_t index, const float* lse, const float* entropy,
                                         const float* grad_log_probs, const float* grad_entropy, void* grad_hidden,
                                         void* grad_weight, size_t ntokens, size_t vocab, size_t width,
                                         size_t ld_hidden, size_t ld_weight, size_t ld_grad_hidden,
                                         size_t ld_grad_weight, float scale, long long ignore_index, ar_dtype_t dtype,
                                         hipStream_t stream);

/* Workspace of the two calls below for so many matrices, on any number of
 * ranks; (size_t)-1 for sizes they do not take. */
size_t ar_orthogonalize_workspace_bytes(int nmatrices, size_t rows, size_t cols);

/* Makes matrices of one size nearly orthogonal by Newton-Schulz products, the
 * update of the Muon optimiser:
 *   X = in / max(|in|, eps)                        (|.| the root of the sum of squares)
 *   X <- a X + (b A + c A A) X,  A = X X^T         (`steps` times, 1 to 32)
 *   out = X,
 * on the transposed matrix where it has more rows than columns, which gives the
 * same. coefficients (host): a, b and c of every step, or NULL for 3.4445,
 * -4.7750, 2.0315 in each; |a| is at most 16, |b| and |c| at most 32, and c is 0 or
 * so large that |b| <= 16 |c| and b^2 <= 64 |c|. Sums are fp32 or fp64; X and what
 * is made of it is held to 22 bits, below 2^-13 in steps of 2^-35, within |x| < 32
 * (beyond, results are NaN).
 * A matrix that holds a NaN or an infinity, or whose iteration diverges, gives
 * NaN; one of zeros gives zeros. in and out are of dtype. In place (in[t] ==
 * out[t] of one pitch) is allowed; what a matrix spans with its pitch overlaps no
 * other that is written. Sides are below 2^20, the smaller up to 2^16, a matrix up to
 * 2^34 elements. eps: at least 1e-30. nmatrices <= AR_MAX_TENSORS. */
ar_result_t ar_orthogonalize(ar_comm_t comm, int nmatrices, const void* const in[], void* const out[], size_t rows,
                             size_t cols, size_t ld_in, size_t ld_out, int steps, const double coefficients[],
                             double eps, ar_dtype_t dtype, hipStream_t stream);

/* The whole update of weight matrices of one size, given gradients that are the
 * same on every rank, as after an all-reduce:
 *   momentum_out = decay * momentum_in + (1 - decay) * grads,
 *   U = nesterov ? decay * momentum_out + (1 - decay) * grads : momentum_out,
 *   weights_out = (1 - lr * weight_decay) * weights_in - lr * update_scale * X,
 * with X the orthogonalised U as above, in fp32. grads (dtype), momentum (fp32)
 * and weights_in are one buffer a matrix; weights_out[t*nranks + r] is rank r's
 * replica, all of which get the same. weights_in and weights_out are of
 * weight_dtype: dtype or fp32. decay: in [0, 1); lr, weight_decay, update_scale
 * and their products with lr are finite in fp32. In place is allowed for the
 * momentum (momentum_in[t] == momentum_out[t]) and for the weights (one of a
 * matrix's replicas == weights_in[t]). */
ar_result_t ar_muon_update(ar_comm_t comm, int nmatrices, const void* const grads[], const float* const momentum_in[],
                           float* const momentum_out[], const void* const weights_in[], void* const weights_out[],
                           size_t rows, size_t cols, size_t ld_grads, size_t ld_momentum, size_t ld_weights,
                           double decay, int nesterov, double lr, double weight_decay, double update_scale, int steps,
                           const double coefficients[], double eps, ar_dtype_t dtype, ar_dtype_t weight_dtype,
                           hipStream_t stream);

/* Static description of a result code. */
const char* ar_result_string(ar_result_t result);

/* Thread-local detail of the last failed call on this thread ("" if none). */
const char* ar_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBALLREDUCE_ALLREDUCE_H */
