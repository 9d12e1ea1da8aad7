"""Python binding of liballreduce (the C ABI in include/allreduce.h).

Argument marshalling only: every step of the all-reduce runs in the HIP
kernels of ``liballreduce.so``. The functions carry the C names and raise
``ArError`` where the C call returns a non-success code. Buffers may be
passed as torch tensors (their ``data_ptr()`` is taken) or as integer device
addresses; streams as ``torch.cuda.Stream``, an integer ``hipStream_t`` or
``None`` (torch's current stream on the comm's device).

The library is built in-tree by ``python ring_all_reduce_ar_amd/build.py``;
importing this package without it raises ImportError: there is no fallback.
"""
from __future__ import annotations

import array
import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liballreduce.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python ring_all_reduce_ar_amd/build.py` first")

# One process must hold one HIP runtime. torch ships its own libamdhip64 /
# libhsa-runtime64; importing torch first loads them, and liballreduce.so's
# dependency on libamdhip64.so.7 then binds to that same runtime instead of
# loading a second one from /opt/rocm (two HSA runtimes in one process leave
# the second without a device).
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIB_PATH)

MAX_RANKS = 64  # AR_MAX_RANKS
MAX_TENSORS = 65536  # AR_MAX_TENSORS
NOALLOC_SCRATCH_BYTES = 64 << 20  # AR_NOALLOC_SCRATCH_BYTES

# ar_result_t
AR_SUCCESS, AR_ERR_INVALID_ARGUMENT, AR_ERR_UNSUPPORTED, AR_ERR_HIP, AR_ERR_OUT_OF_MEMORY, AR_ERR_INTERNAL = range(6)
# ar_dtype_t
AR_FLOAT32, AR_FLOAT16, AR_BFLOAT16, AR_INT32 = range(4)
# ar_op_t
AR_SUM, AR_AVG, AR_MAX, AR_MIN, AR_PROD = range(5)
# ar_mode_t
AR_MODE_FUSED, AR_MODE_RING_STEPWISE, AR_MODE_RING_GRAPH, AR_MODE_TREE, AR_MODE_TREE_STEPWISE = range(5)
# ar_access_t
AR_ACCESS_AUTO, AR_ACCESS_STREAMING, AR_ACCESS_CACHED = range(3)
ACCESS_NAMES = {"auto": AR_ACCESS_AUTO, "streaming": AR_ACCESS_STREAMING, "cached": AR_ACCESS_CACHED}
# ar_index_t, ar_norm_t, ar_grads_t
AR_INDEX_INT32, AR_INDEX_INT64 = range(2)
AR_NORM_L2, AR_NORM_INF = range(2)
AR_GRADS_REPLICATED, AR_GRADS_SHARDED = range(2)
INDEX_NAMES = {"i32": AR_INDEX_INT32, "i64": AR_INDEX_INT64}
NORM_NAMES = {"l2": AR_NORM_L2, "inf": AR_NORM_INF}
GRADS_NAMES = {"replicated": AR_GRADS_REPLICATED, "sharded": AR_GRADS_SHARDED}
# ar_collective_t
AR_COLL_ALL_REDUCE, AR_COLL_REDUCE_SCATTER, AR_COLL_ALL_GATHER, AR_COLL_ALL_TO_ALL = range(4)

DTYPE_NAMES = {"f32": AR_FLOAT32, "f16": AR_FLOAT16, "bf16": AR_BFLOAT16, "i32": AR_INT32}
OP_NAMES = {"sum": AR_SUM, "avg": AR_AVG, "max": AR_MAX, "min": AR_MIN, "prod": AR_PROD}
MODE_NAMES = {"fused": AR_MODE_FUSED, "stepwise": AR_MODE_RING_STEPWISE, "graph": AR_MODE_RING_GRAPH,
              "tree": AR_MODE_TREE, "tree_stepwise": AR_MODE_TREE_STEPWISE}

EXPORTED_SYMBOLS = (
    "ar_comm_create", "ar_comm_destroy", "ar_comm_nranks", "ar_workspace_bytes", "ar_comm_set_workspace",
    "ar_all_reduce", "ar_all_reduce_noalloc", "ar_reduce_scatter", "ar_all_gather", "ar_all_to_all", "ar_all_reduce_multi",
    "ar_comm_set_step_timing", "ar_comm_set_access", "ar_comm_set_streaming", "ar_last_step_times_ms",
    "ar_clip_workspace_bytes", "ar_grad_norm", "ar_clip_grads", "ar_all_reduce_clip",
    "ar_embedding", "ar_embedding_workspace_bytes", "ar_embedding_backward",
    "ar_linear_cross_entropy_workspace_bytes", "ar_linear_cross_entropy", "ar_linear_cross_entropy_backward",
    "ar_linear_log_probs_workspace_bytes", "ar_linear_log_probs", "ar_linear_log_probs_backward",
    "ar_orthogonalize_workspace_bytes", "ar_orthogonalize", "ar_muon_update",
    "ar_result_string", "ar_last_error",
)

_c_int, _c_size, _vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
_ptr_array = ctypes.POINTER(ctypes.c_void_p)

_lib.ar_comm_create.argtypes = [ctypes.POINTER(_vp), _c_int, _c_int]
_lib.ar_comm_destroy.argtypes = [_vp]
_lib.ar_comm_nranks.argtypes = [_vp]
_lib.ar_comm_nranks.restype = _c_int
_lib.ar_workspace_bytes.argtypes = [_c_int, _c_int, _c_size, _c_int, _c_int]
_lib.ar_workspace_bytes.restype = _c_size
_lib.ar_comm_set_workspace.argtypes = [_vp, _vp, _c_size]
_lib.ar_all_reduce.argtypes = [_vp, _ptr_array, _ptr_array, _c_size, _c_int, _c_int, _c_int, _vp]
_lib.ar_all_reduce_noalloc.argtypes = [_vp, _ptr_array, _ptr_array, _c_size, _c_int, _c_int, _c_int, _vp]
_lib.ar_reduce_scatter.argtypes = [_vp, _ptr_array, _ptr_array, _c_size, _c_int, _c_int, _c_int, _vp]
_lib.ar_all_gather.argtypes = [_vp, _ptr_array, _ptr_array, _c_size, _c_int, _c_int, _vp]
_lib.ar_all_to_all.argtypes = [_vp, _ptr_array, _ptr_array, _c_size, _c_int, _c_int, _vp]
_lib.ar_all_reduce_multi.argtypes = [_vp, _c_int, _ptr_array, _ptr_array, ctypes.POINTER(_c_size), _c_int, _c_int,
                                     _c_int, _vp]
_lib.ar_comm_set_step_timing.argtypes = [_vp, _c_int]
_lib.ar_comm_set_streaming.argtypes = [_vp, _c_int]
_lib.ar_comm_set_access.argtypes = [_vp, _c_int]
_lib.ar_last_step_times_ms.argtypes = [_vp, ctypes.POINTER(ctypes.c_float), _c_int, ctypes.POINTER(_c_int)]
_size_array, _c_i64 = ctypes.POINTER(_c_size), ctypes.c_longlong
_lib.ar_clip_workspace_bytes.argtypes = []
_lib.ar_clip_workspace_bytes.restype = _c_size
_lib.ar_grad_norm.argtypes = [_vp, _c_int, _ptr_array, _size_array, _c_int, _c_int, _c_int, _vp, _vp]
_lib.ar_clip_grads.argtypes = [_vp, _c_int, _ptr_array, _ptr_array, _size_array, _c_int, _c_int, _c_int,
                               ctypes.c_double, _vp, _vp]
_lib.ar_all_reduce_clip.argtypes = _lib.ar_clip_grads.argtypes
_lib.ar_embedding.argtypes = [_vp, _vp, _vp, _c_int, _vp] + [_c_size] * 5 + [_c_i64, ctypes.c_float, _c_int, _vp]
_lib.ar_embedding_workspace_bytes.argtypes = [_c_size] * 3
_lib.ar_embedding_workspace_bytes.restype = _c_size
_lib.ar_embedding_backward.argtypes = [_vp, _vp, _vp, _c_int, _vp] + [_c_size] * 5 + [_c_i64, ctypes.c_float, _c_int,
                                                                                   _c_int, _c_int, _vp]
_lib.ar_linear_cross_entropy_workspace_bytes.argtypes = [_c_size] * 3 + [_c_int, _c_int]
_lib.ar_linear_cross_entropy_workspace_bytes.restype = _c_size
_lib.ar_linear_cross_entropy.argtypes = [_vp, _vp, _vp, _vp, _c_int, _vp, _vp] + [_c_size] * 5 + [_c_i64, _c_int, _vp]
_lib.ar_linear_cross_entropy_backward.argtypes = ([_vp, _vp, _vp, _vp, _c_int, _vp, _vp, _vp, _vp] + [_c_size] * 7 +
                                                  [_c_i64, _c_int, _vp])
_lib.ar_linear_log_probs_workspace_bytes.argtypes = [_c_size] * 3 + [_c_int] * 3
_lib.ar_linear_log_probs_workspace_bytes.restype = _c_size
_lib.ar_linear_log_probs.argtypes = ([_vp, _vp, _vp, _vp, _c_int, _vp, _vp, _vp, _c_int, _vp, _vp] + [_c_size] * 5 +
                                     [ctypes.c_float, _c_i64, _c_int, _vp])
_lib.ar_linear_log_probs_backward.argtypes = ([_vp, _vp, _vp, _vp, _c_int] + [_vp] * 6 + [_c_size] * 7 +
                                              [ctypes.c_float, _c_i64, _c_int, _vp])
_double_array = ctypes.POINTER(ctypes.c_double)
_lib.ar_orthogonalize_workspace_bytes.argtypes = [_c_int] + [_c_size] * 2
_lib.ar_orthogonalize_workspace_bytes.restype = _c_size
_lib.ar_orthogonalize.argtypes = ([_vp, _c_int, _ptr_array, _ptr_array] + [_c_size] * 4 +
                                  [_c_int, _double_array, ctypes.c_double, _c_int, _vp])
_lib.ar_muon_update.argtypes = ([_vp, _c_int] + [_ptr_array] * 5 + [_c_size] * 5 + [ctypes.c_double, _c_int] +
                                [ctypes.c_double] * 3 + [_c_int, _double_array, ctypes.c_double, _c_int, _c_int, _vp])
_lib.ar_result_string.argtypes = [_c_int]
_lib.ar_result_string.restype = ctypes.c_char_p
_lib.ar_last_error.argtypes = []
_lib.ar_last_error.restype = ctypes.c_char_p
for _name in ("ar_comm_create", "ar_comm_destroy", "ar_comm_set_workspace", "ar_all_reduce", "ar_all_reduce_noalloc",
              "ar_reduce_scatter",
              "ar_all_gather", "ar_all_to_all", "ar_all_reduce_multi", "ar_comm_set_step_timing",
              "ar_comm_set_streaming", "ar_comm_set_access", "ar_last_step_times_ms",
              "ar_grad_norm", "ar_clip_grads", "ar_all_reduce_clip", "ar_embedding", "ar_embedding_backward",
              "ar_linear_cross_entropy", "ar_linear_cross_entropy_backward", "ar_linear_log_probs",
              "ar_linear_log_probs_backward", "ar_orthogonalize", "ar_muon_update"):
    getattr(_lib, _name).restype = _c_int


class ArError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        detail = (_lib.ar_last_error() or b"").decode(errors="replace")
        super().__init__(f"{where}: {ar_result_string(code)} ({code}): {detail}")


def _check(code: int, where: str):
    if code != AR_SUCCESS:
        raise ArError(code, where)


def ar_result_string(code: int) -> str:
    return _lib.ar_result_string(code).decode()


def ar_last_error() -> str:
    return (_lib.ar_last_error() or b"").decode(errors="replace")


def _enum(value, names, what):
    if isinstance(value, str):
        if value not in names:
            raise ValueError(f"unknown {what} {value!r}; expected one of {sorted(names)}")
        return names[value]
    return int(value)


def torch_dtype_code(dtype) -> int:
    import torch
    table = {torch.float32: AR_FLOAT32, torch.float16: AR_FLOAT16, torch.bfloat16: AR_BFLOAT16, torch.int32: AR_INT32}
    if dtype not in table:
        raise TypeError(f"unsupported dtype {dtype}")
    return table[dtype]


def _addr(buf) -> int:
    if isinstance(buf, int):
        return buf
    if hasattr(buf, "data_ptr"):
        if not buf.is_contiguous():
            raise ValueError("rank buffers must be contiguous")
        return buf.data_ptr()
    raise TypeError(f"expected a tensor or an int address, got {type(buf).__name__}")


_PTR_ARRAY_TYPES = {}  # length -> ctypes array type (building the type costs more than the array)


def _ptrs(bufs):
    n = len(bufs)
    t = _PTR_ARRAY_TYPES.get(n)
    if t is None:
        t = _PTR_ARRAY_TYPES[n] = ctypes.c_void_p * n
    # Addresses alone: many times faster than one ctypes object each. Every element
    # is looked at: an array takes an integer tensor of one element by its value.
    if n and type(bufs[0]) is int and set(map(type, bufs)) == {int}:
        try:
            return t.from_buffer(array.array("Q", bufs))
        except OverflowError:
            pass
    return t(*[b if type(b) is int else _addr(b) for b in bufs])


def _ptr_pair(sendbufs, recvbufs):
    """The send and recv pointer arrays; one array serves both when the same
    list is passed for both (in place)."""
    s = _ptrs(sendbufs)
    return s, (s if recvbufs is sendbufs else _ptrs(recvbufs))


# torch.cuda.current_stream(device).cuda_stream without the Stream object around it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device: int):
    if stream is None:
        return _current_stream(device) if _current_stream else torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Comm:
    """Owns an ``ar_comm_t``; ``handle`` is the raw pointer."""

    def __init__(self, nranks: int, device: int = 0):
        h = ctypes.c_void_p()
        _check(_lib.ar_comm_create(ctypes.byref(h), nranks, device), "ar_comm_create")
        self.handle = h
        self.nranks = nranks
        self.device = device

    def close(self):
        if self.handle:
            _lib.ar_comm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def _h(comm):
    return comm.handle if isinstance(comm, Comm) else comm


def ar_comm_create(nranks: int, device: int = 0) -> Comm:
    return Comm(nranks, device)


def ar_comm_destroy(comm: Comm):
    comm.close()


def ar_comm_nranks(comm) -> int:
    return _lib.ar_comm_nranks(_h(comm))


def ar_workspace_bytes(coll, nranks: int, count: int, dtype, mode) -> int:
    v = _lib.ar_workspace_bytes(int(coll), nranks, count, _enum(dtype, DTYPE_NAMES, "dtype"),
                                _enum(mode, MODE_NAMES, "mode"))
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("ar_workspace_bytes: invalid arguments or overflow")
    return v


def ar_comm_set_workspace(comm, buf, nbytes: int | None = None):
    """Attach a device workspace (tensor or address); ``None`` detaches."""
    if buf is None:
        _check(_lib.ar_comm_set_workspace(_h(comm), None, 0), "ar_comm_set_workspace")
        return
    if nbytes is None:
        nbytes = buf.numel() * buf.element_size()
    _check(_lib.ar_comm_set_workspace(_h(comm), _addr(buf), nbytes), "ar_comm_set_workspace")


def ar_all_reduce(comm, sendbufs, recvbufs, count: int, dtype, op, mode="fused", stream=None):
    _check(_lib.ar_all_reduce(_h(comm), *_ptr_pair(sendbufs, recvbufs), count, _enum(dtype, DTYPE_NAMES, "dtype"),
                              _enum(op, OP_NAMES, "op"), _enum(mode, MODE_NAMES, "mode"),
                              _stream(stream, comm.device if isinstance(comm, Comm) else 0)), "ar_all_reduce")


def ar_all_reduce_noalloc(comm, sendbufs, recvbufs, count: int, dtype, op, mode="fused", stream=None):
    """ar_all_reduce with its partial sums in the library's device scratch
    array instead of the comm's workspace; allocates nothing."""
    _check(_lib.ar_all_reduce_noalloc(_h(comm), *_ptr_pair(sendbufs, recvbufs), count,
                                      _enum(dtype, DTYPE_NAMES, "dtype"), _enum(op, OP_NAMES, "op"),
                                      _enum(mode, MODE_NAMES, "mode"),
                                      _stream(stream, comm.device if isinstance(comm, Comm) else 0)),
           "ar_all_reduce_noalloc")


def ar_reduce_scatter(comm, sendbufs, recvbufs, recvcount: int, dtype, op, mode="fused", stream=None):
    _check(_lib.ar_reduce_scatter(_h(comm), *_ptr_pair(sendbufs, recvbufs), recvcount,
                                  _enum(dtype, DTYPE_NAMES, "dtype"), _enum(op, OP_NAMES, "op"),
                                  _enum(mode, MODE_NAMES, "mode"),
                                  _stream(stream, comm.device if isinstance(comm, Comm) else 0)), "ar_reduce_scatter")


def ar_all_gather(comm, sendbufs, recvbufs, sendcount: int, dtype, mode="fused", stream=None):
    _check(_lib.ar_all_gather(_h(comm), *_ptr_pair(sendbufs, recvbufs), sendcount,
                              _enum(dtype, DTYPE_NAMES, "dtype"), _enum(mode, MODE_NAMES, "mode"),
                              _stream(stream, comm.device if isinstance(comm, Comm) else 0)), "ar_all_gather")


def ar_all_to_all(comm, sendbufs, recvbufs, blockcount: int, dtype, mode="fused", stream=None):
    _check(_lib.ar_all_to_all(_h(comm), *_ptr_pair(sendbufs, recvbufs), blockcount,
                              _enum(dtype, DTYPE_NAMES, "dtype"), _enum(mode, MODE_NAMES, "mode"),
                              _stream(stream, comm.device if isinstance(comm, Comm) else 0)), "ar_all_to_all")


def ar_all_reduce_multi(comm, sendbufs, recvbufs, counts, dtype, op, mode="fused", stream=None):
    """sendbufs / recvbufs: one list of per-rank buffers per tensor
    (``sendbufs[t][r]``), or a flat tensor-major list; counts[t] elements."""
    nt = len(counts)
    flat_s = [b for row in sendbufs for b in row] if nt and isinstance(sendbufs[0], (list, tuple)) else list(sendbufs)
    flat_r = [b for row in recvbufs for b in row] if nt and isinstance(recvbufs[0], (list, tuple)) else list(recvbufs)
    arr = (ctypes.c_size_t * max(nt, 1))(*counts)
    _check(_lib.ar_all_reduce_multi(_h(comm), nt, *_ptr_pair(flat_s, flat_r), arr, _enum(dtype, DTYPE_NAMES, "dtype"),
                                    _enum(op, OP_NAMES, "op"), _enum(mode, MODE_NAMES, "mode"),
                                    _stream(stream, comm.device if isinstance(comm, Comm) else 0)),
           "ar_all_reduce_multi")


def ar_comm_set_step_timing(comm, enable: bool):
    _check(_lib.ar_comm_set_step_timing(_h(comm), 1 if enable else 0), "ar_comm_set_step_timing")


def ar_comm_set_streaming(comm, enable: bool):
    _check(_lib.ar_comm_set_streaming(_h(comm), 1 if enable else 0), "ar_comm_set_streaming")


def ar_comm_set_access(comm, access):
    """access: "auto", "streaming", "cached" or an AR_ACCESS_* value."""
    _check(_lib.ar_comm_set_access(_h(comm), _enum(access, ACCESS_NAMES, "access")), "ar_comm_set_access")


def ar_last_step_times_ms(comm, cap: int = 2 * MAX_RANKS + 1):
    out = (ctypes.c_float * cap)()
    n = ctypes.c_int()
    _check(_lib.ar_last_step_times_ms(_h(comm), out, cap, ctypes.byref(n)), "ar_last_step_times_ms")
    return [out[i] for i in range(min(n.value, cap))]


# Language-model operators ----------------------------------------------------
def _flat(bufs):
    """A tensor-major list of buffers from one list of per-rank buffers per
    tensor, or as it is."""
    return [b for row in bufs for b in row] if len(bufs) and isinstance(bufs[0], (list, tuple)) else bufs


def _counts(counts):
    return (ctypes.c_size_t * max(len(counts), 1))(*counts)


def _device(comm) -> int:
    return comm.device if isinstance(comm, Comm) else 0


def _check_size(value: int, where: str) -> int:
    if value == ctypes.c_size_t(-1).value:
        raise ValueError(f"{where}: invalid arguments or overflow")
    return value


def ar_clip_workspace_bytes() -> int:
    return _lib.ar_clip_workspace_bytes()


def ar_grad_norm(comm, grads, counts, norm_out, dtype, layout="replicated", norm="l2", stream=None):
    """The global norm of many gradient tensors into the device float
    ``norm_out``. ``grads``: one list of per-rank buffers per tensor
    (``grads[t][r]``), or a flat tensor-major list; counts[t] elements."""
    _check(_lib.ar_grad_norm(_h(comm), len(counts), _ptrs(_flat(grads)), _counts(counts),
                             _enum(dtype, DTYPE_NAMES, "dtype"), _enum(layout, GRADS_NAMES, "layout"),
                             _enum(norm, NORM_NAMES, "norm"), _addr(norm_out), _stream(stream, _device(comm))),
           "ar_grad_norm")


def ar_clip_grads(comm, sendbufs, recvbufs, counts, max_norm: float, norm_out, dtype, layout="replicated", norm="l2",
                  stream=None):
    """recv = send * min(1, max_norm / (norm + 1e-6)) over all tensors.
    Buffers as in ar_all_reduce_multi; norm_out: a device float or None."""
    s = _flat(sendbufs)
    r = s if recvbufs is sendbufs else _flat(recvbufs)
    _check(_lib.ar_clip_grads(_h(comm), len(counts), *_ptr_pair(s, r), _counts(counts),
                              _enum(dtype, DTYPE_NAMES, "dtype"), _enum(layout, GRADS_NAMES, "layout"),
                              _enum(norm, NORM_NAMES, "norm"), max_norm,
                              None if norm_out is None else _addr(norm_out), _stream(stream, _device(comm))),
           "ar_clip_grads")


def ar_all_reduce_clip(comm, sendbufs, recvbufs, counts, max_norm: float, norm_out, dtype, op="avg", norm="l2",
                       stream=None):
    """ar_all_reduce_multi (sum or avg) and ar_clip_grads of its result in one call."""
    s = _flat(sendbufs)
    r = s if recvbufs is sendbufs else _flat(recvbufs)
    _check(_lib.ar_all_reduce_clip(_h(comm), len(counts), *_ptr_pair(s, r), _counts(counts),
                                   _enum(dtype, DTYPE_NAMES, "dtype"), _enum(op, OP_NAMES, "op"),
                                   _enum(norm, NORM_NAMES, "norm"), max_norm,
                                   None if norm_out is None else _addr(norm_out), _stream(stream, _device(comm))),
           "ar_all_reduce_clip")


def _index(index, buf) -> int:
    """The index type: as named, or the tensor's own."""
    if index is not None:
        return _enum(index, INDEX_NAMES, "index")
    if isinstance(buf, int):
        raise TypeError("index numbers passed as an address need their type: index='i32' or 'i64'")
    if buf.dtype == torch.int64:
        return AR_INDEX_INT64
    if buf.dtype == torch.int32:
        return AR_INDEX_INT32
    raise TypeError(f"unsupported index dtype {buf.dtype}")


def _rows(buf, ld: int):
    """(address, row pitch) of a matrix: a tensor's own pitch where none is
    given, its rows being contiguous."""
    if isinstance(buf, int):
        return buf, ld
    if buf is None:
        return None, ld
    if ld:
        return buf.data_ptr(), ld
    pitch, shape = buf.stride(), buf.shape
    if len(shape) != 2:
        return _addr(buf), 0
    if pitch[1] != 1 and shape[1] > 1:
        raise ValueError("the rows of a matrix must be contiguous")
    if shape[0] <= 1:
        return buf.data_ptr(), 0
    if pitch[0] < shape[1]:  # as an expanded tensor's
        raise ValueError("the rows of a matrix must not overlap")
    return buf.data_ptr(), pitch[0]


def ar_embedding(comm, weight, tokens, out, ntokens: int, rows: int, width: int, dtype, scale: float = 1.0,
                 first_row: int = 0, ld_weight: int = 0, ld_out: int = 0, index=None, stream=None):
    """out[t] = weight[tokens[t] - first_row] * scale, zeros where that row is
    not in [0, rows)."""
    w, ld_weight = _rows(weight, ld_weight)
    o, ld_out = _rows(out, ld_out)
    _check(_lib.ar_embedding(_h(comm), w, _addr(tokens), _index(index, tokens), o, ntokens, rows, width, ld_weight,
                             ld_out, first_row, scale, _enum(dtype, DTYPE_NAMES, "dtype"),
                             _stream(stream, _device(comm))), "ar_embedding")


def ar_embedding_workspace_bytes(ntokens: int, rows: int, width: int) -> int:
    return _check_size(_lib.ar_embedding_workspace_bytes(ntokens, rows, width), "ar_embedding_workspace_bytes")


def ar_embedding_backward(comm, grad_out, tokens, grad_weight, ntokens: int, rows: int, width: int, dtype,
                          grad_dtype=None, scale: float = 1.0, first_row: int = 0, ld_grad_out: int = 0,
                          ld_grad_weight: int = 0, accumulate: bool = False, index=None, stream=None):
    """grad_weight[v] (+)= scale * the sum of grad_out[t] over the tokens of row v."""
    d = _enum(dtype, DTYPE_NAMES, "dtype")
    g, ld_grad_out = _rows(grad_out, ld_grad_out)
    w, ld_grad_weight = _rows(grad_weight, ld_grad_weight)
    _check(_lib.ar_embedding_backward(_h(comm), g, _addr(tokens), _index(index, tokens), w, ntokens, rows, width,
                                      ld_grad_out, ld_grad_weight, first_row, scale, d,
                                      d if grad_dtype is None else _enum(grad_dtype, DTYPE_NAMES, "grad_dtype"),
                                      1 if accumulate else 0, _stream(stream, _device(comm))), "ar_embedding_backward")


def ar_linear_cross_entropy_workspace_bytes(ntokens: int, vocab: int, width: int, dtype, backward: bool = False) -> int:
    return _check_size(_lib.ar_linear_cross_entropy_workspace_bytes(ntokens, vocab, width,
                                                                    _enum(dtype, DTYPE_NAMES, "dtype"),
                                                                    1 if backward else 0),
                       "ar_linear_cross_entropy_workspace_bytes")


def ar_linear_cross_entropy(comm, hidden, weight, targets, losses, lse, ntokens: int, vocab: int, width: int, dtype,
                            ignore_index: int = -100, ld_hidden: int = 0, ld_weight: int = 0, index=None, stream=None):
    """losses[t] = lse[t] - z[t][targets[t]] with z = hidden weight^T and lse its
    logsumexp, without keeping z."""
    x, ld_hidden = _rows(hidden, ld_hidden)
    w, ld_weight = _rows(weight, ld_weight)
    _check(_lib.ar_linear_cross_entropy(_h(comm), x, w, _addr(targets), _index(index, targets), _addr(losses),
                                        _addr(lse), ntokens, vocab, width, ld_hidden, ld_weight, ignore_index,
                                        _enum(dtype, DTYPE_NAMES, "dtype"), _stream(stream, _device(comm))),
           "ar_linear_cross_entropy")


def ar_linear_cross_entropy_backward(comm, hidden, weight, targets, lse, grad_losses, grad_hidden, grad_weight,
                                     ntokens: int, vocab: int, width: int, dtype, ignore_index: int = -100,
                                     ld_hidden: int = 0, ld_weight: int = 0, ld_grad_hidden: int = 0,
                                     ld_grad_weight: int = 0, index=None, stream=None):
    """grad_hidden and grad_weight (either may be None) from lse and the gradient of each loss."""
    x, ld_hidden = _rows(hidden, ld_hidden)
    w, ld_weight = _rows(weight, ld_weight)
    gx, ld_grad_hidden = _rows(grad_hidden, ld_grad_hidden)
    gw, ld_grad_weight = _rows(grad_weight, ld_grad_weight)
    _check(_lib.ar_linear_cross_entropy_backward(_h(comm), x, w, _addr(targets), _index(index, targets), _addr(lse),
                                                 _addr(grad_losses), gx, gw, ntokens, vocab, width, ld_hidden,
                                                 ld_weight, ld_grad_hidden, ld_grad_weight, ignore_index,
                                                 _enum(dtype, DTYPE_NAMES, "dtype"), _stream(stream, _device(comm))),
           "ar_linear_cross_entropy_backward")


_TENSOR_TYPES = {AR_FLOAT32: torch.float32, AR_FLOAT16: torch.float16, AR_BFLOAT16: torch.bfloat16}


def _typed(code: int, **bufs):
    """Tensors (alone or in lists) hold what the call takes them for: memory of
    another type would be read and written past its end."""
    want = _TENSOR_TYPES.get(code)
    if want is None:  # refused with the call
        return
    for what, some in bufs.items():
        for b in some if isinstance(some, (list, tuple)) else (some,):
            if getattr(b, "dtype", want) is not want:
                raise TypeError(f"{what}: the call takes {want}, not {b.dtype}")


def ar_linear_log_probs_workspace_bytes(ntokens: int, vocab: int, width: int, dtype, top: int = 0,
                                        backward: bool = False) -> int:
    return _check_size(_lib.ar_linear_log_probs_workspace_bytes(ntokens, vocab, width,
                                                                _enum(dtype, DTYPE_NAMES, "dtype"), top,
                                                                1 if backward else 0),
                       "ar_linear_log_probs_workspace_bytes")


def ar_linear_log_probs(comm, hidden, weight, targets, log_probs, entropy, lse, ntokens: int, vocab: int, width: int,
                        dtype, top: int = 0, top_log_probs=None, top_ids=None, scale: float = 1.0,
                        ignore_index: int = -100, ld_hidden: int = 0, ld_weight: int = 0, index=None, stream=None):
    """log_probs[t] = z[t][targets[t]] - lse[t] with z = scale * hidden weight^T,
    its entropy (or None), and the ``top`` likeliest tokens' log probabilities
    and ids (int32)."""
    d = _enum(dtype, DTYPE_NAMES, "dtype")
    _typed(d, hidden=hidden, weight=weight)
    _typed(AR_FLOAT32, log_probs=log_probs, entropy=entropy, lse=lse, top_log_probs=top_log_probs)
    x, ld_hidden = _rows(hidden, ld_hidden)
    w, ld_weight = _rows(weight, ld_weight)
    if not isinstance(top_ids, (int, type(None))) and top_ids.dtype != torch.int32:
        raise TypeError(f"top_ids are int32, not {top_ids.dtype}")
    _check(_lib.ar_linear_log_probs(_h(comm), x, w, _addr(targets), _index(index, targets), _addr(log_probs),
                                    None if entropy is None else _addr(entropy), _addr(lse), top,
                                    None if top_log_probs is None else _addr(top_log_probs),
                                    None if top_ids is None else _addr(top_ids), ntokens, vocab, width, ld_hidden,
                                    ld_weight, scale, ignore_index, d, _stream(stream, _device(comm))),
           "ar_linear_log_probs")


def ar_linear_log_probs_backward(comm, hidden, weight, targets, lse, entropy, grad_log_probs, grad_entropy,
                                 grad_hidden, grad_weight, ntokens: int, vocab: int, width: int, dtype,
                                 scale: float = 1.0, ignore_index: int = -100, ld_hidden: int = 0, ld_weight: int = 0,
                                 ld_grad_hidden: int = 0, ld_grad_weight: int = 0, index=None, stream=None):
    """grad_hidden and grad_weight (either may be None) from lse, entropy and the
    gradients of each log probability and entropy (grad_entropy may be None, and
    entropy then too)."""
    d = _enum(dtype, DTYPE_NAMES, "dtype")
    _typed(d, hidden=hidden, weight=weight, grad_hidden=grad_hidden, grad_weight=grad_weight)
    _typed(AR_FLOAT32, lse=lse, entropy=entropy, grad_log_probs=grad_log_probs, grad_entropy=grad_entropy)
    x, ld_hidden = _rows(hidden, ld_hidden)
    w, ld_weight = _rows(weight, ld_weight)
    gx, ld_grad_hidden = _rows(grad_hidden, ld_grad_hidden)
    gw, ld_grad_weight = _rows(grad_weight, ld_grad_weight)
    _check(_lib.ar_linear_log_probs_backward(_h(comm), x, w, _addr(targets), _index(index, targets), _addr(lse),
                                             None if entropy is None else _addr(entropy), _addr(grad_log_probs),
                                             None if grad_entropy is None else _addr(grad_entropy), gx, gw, ntokens,
                                             vocab, width, ld_hidden, ld_weight, ld_grad_hidden, ld_grad_weight, scale,
                                             ignore_index, d, _stream(stream, _device(comm))),
           "ar_linear_log_probs_backward")


def ar_orthogonalize_workspace_bytes(nmatrices: int, rows: int, cols: int) -> int:
    return _check_size(_lib.ar_orthogonalize_workspace_bytes(nmatrices, rows, cols), "ar_orthogonalize_workspace_bytes")


def _matrices(bufs, ld: int):
    """(addresses, row pitch) of a list of matrices of one size: the tensors' own
    pitch, the same for all, where none is given."""
    bufs = _flat(bufs)
    if not len(bufs) or isinstance(bufs[0], int):
        return _ptrs(bufs), ld
    # rows alike, as in most lists: one look serves for all (a pitch below the width is refused with the
    # call, but for an expanded tensor's 0, which would stand for dense rows there)
    if not ld:
        strides = {b.stride() for b in bufs}
        first = bufs[0].stride()
        if len(strides) == 1 and len(first) == 2 and first[0] and first[1] == 1 and bufs[0].shape[0] > 1:
            return _ptrs([b.data_ptr() for b in bufs]), first[0]
    rows = [_rows(b, ld) for b in bufs]
    if any(pitch != rows[0][1] for _, pitch in rows):
        raise ValueError("the matrices of a list have one row pitch")
    return _ptrs([p for p, _ in rows]), rows[0][1]


def _coefficients(coefficients, steps: int):
    if coefficients is None:
        return None
    flat = [float(x) for step in coefficients for x in (step if isinstance(step, (list, tuple)) else [step])]
    if len(flat) == 3:
        flat *= steps
    if len(flat) != 3 * steps:
        raise ValueError(f"{steps} steps take 3 or {3 * steps} coefficients, not {len(flat)}")
    return (ctypes.c_double * len(flat))(*flat)


def _same_length(what: str, got: int, want: int):
    if got != want:
        raise ValueError(f"{what}: {got} matrices where there are {want}")


def ar_orthogonalize(comm, ins, outs, rows: int, cols: int, dtype, steps: int = 5, coefficients=None, eps: float = 1e-7,
                     ld_in: int = 0, ld_out: int = 0, stream=None):
    """outs[t] = ins[t] / max(norm, eps) after ``steps`` Newton-Schulz steps, for
    lists of matrices [rows][cols]. coefficients: (a, b, c), or three for each
    step."""
    _same_length("outs", len(outs), len(ins))
    d = _enum(dtype, DTYPE_NAMES, "dtype")
    _typed(d, ins=ins, outs=() if outs is ins else outs)
    p, ld_in = _matrices(ins, ld_in)
    q, ld_out = (p, ld_in) if outs is ins and not ld_out else _matrices(outs, ld_out)
    _check(_lib.ar_orthogonalize(_h(comm), len(ins), p, q, rows, cols, ld_in, ld_out, steps,
                                 _coefficients(coefficients, steps), eps, d, _stream(stream, _device(comm))),
           "ar_orthogonalize")


def ar_muon_update(comm, grads, momentum_in, momentum_out, weights_in, weights_out, rows: int, cols: int, dtype,
                   weight_dtype=None, decay: float = 0.95, nesterov: bool = True, lr: float = 0.02,
                   weight_decay: float = 0.0, update_scale: float = 1.0, steps: int = 5, coefficients=None,
                   eps: float = 1e-7, ld_grads: int = 0, ld_momentum: int = 0, ld_weights: int = 0, stream=None):
    """The update of weight matrices [rows][cols] by orthogonalised momentum.
    weights_out: one list of per-rank replicas per matrix (``weights_out[t][r]``),
    or a flat matrix-major list; the others one buffer per matrix."""
    n = len(grads)
    flat = _flat(weights_out)
    nranks = max(comm.nranks if isinstance(comm, Comm) else ar_comm_nranks(comm), 1)
    for what, got, want in (("momentum_in", len(momentum_in), n), ("momentum_out", len(momentum_out), n),
                            ("weights_in", len(weights_in), n),
                            ("weights_out", len(flat), n * nranks)):
        _same_length(what, got, want)
    d = _enum(dtype, DTYPE_NAMES, "dtype")
    dw = d if weight_dtype is None else _enum(weight_dtype, DTYPE_NAMES, "weight_dtype")
    _typed(d, grads=grads)
    _typed(AR_FLOAT32, momentum_in=momentum_in, momentum_out=() if momentum_out is momentum_in else momentum_out)
    _typed(dw, weights_in=weights_in, weights_out=flat)
    g, ld_grads = _matrices(grads, ld_grads)
    mi, ld_in = _matrices(momentum_in, ld_momentum)
    mo, ld_momentum = (mi, ld_in) if momentum_out is momentum_in else _matrices(momentum_out, ld_momentum)
    wi, ld_read = _matrices(weights_in, ld_weights)
    wo, ld_weights = _matrices(flat, ld_weights)
    if n and ((ld_in or cols) != (ld_momentum or cols) or (ld_read or cols) != (ld_weights or cols)):
        raise ValueError("momentum_in and momentum_out, and weights_in and weights_out, have one row pitch each")
    _check(_lib.ar_muon_update(_h(comm), n, g, mi, mo, wi, wo, rows, cols, ld_grads, ld_momentum, ld_weights, decay,
                               1 if nesterov else 0, lr, weight_decay, update_scale, steps,
                               _coefficients(coefficients, steps), eps, d, dw, _stream(stream, _device(comm))),
           "ar_muon_update")
