"""The language-model operators without a GPU: workspace sizes, and refusals,
which come before the first HIP call (a communicator with no device behind it
serves: a refused call reads its first fields only)."""
import ctypes
import random

import pytest
import torch

import ring_all_reduce_ar_amd as ar

BASE = 1 << 20  # made-up device addresses, never touched
GAP = 1 << 24


class _Fields(ctypes.Structure):
    _fields_ = [("nranks", ctypes.c_int), ("device", ctypes.c_int), ("num_cus", ctypes.c_int),
                ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t), ("rest", ctypes.c_ubyte * 1024)]


def host_comm(nranks=1, ws_bytes=1 << 40):
    f = _Fields(nranks=nranks, device=0, num_cus=256, ws=1 << 44, ws_bytes=ws_bytes)
    f_ptr = ctypes.c_void_p(ctypes.addressof(f))
    f_ptr.keep = f
    return f_ptr


def at(k):
    return BASE + k * GAP


def refused(code, fn, *args, **kw):
    with pytest.raises(ar.ArError) as e:
        fn(*args, **kw, stream=0)
    assert e.value.code == code, str(e.value)
    assert ar.ar_last_error()


BAD, NOT_SERVED = ar.AR_ERR_INVALID_ARGUMENT, ar.AR_ERR_UNSUPPORTED


def test_workspace_sizes():
    assert ar.ar_clip_workspace_bytes() < 1 << 20
    assert ar.ar_embedding_workspace_bytes(0, 10, 4) >= 0
    small, large = (ar.ar_embedding_workspace_bytes(t, 1000, 64) for t in (100, 100_000))
    assert 0 < small < large
    for bad in ((1 << 31, 10, 4), (10, 1 << 31, 4), (10, 10, 1 << 31)):
        with pytest.raises(ValueError):
            ar.ar_embedding_workspace_bytes(*bad)
    for dtype in ("f32", "f16", "bf16"):
        f, b = (ar.ar_linear_cross_entropy_workspace_bytes(1000, 50_000, 512, dtype, backward=x) for x in (False, True))
        assert 0 < f < b < 4 << 30
    # the logits are not kept: far less than one byte for each of them
    assert ar.ar_linear_cross_entropy_workspace_bytes(65_536, 262_144, 1024, "bf16") < 65_536 * 262_144 // 4
    for bad in ((10, 10, 0, "f32"), (1 << 31, 10, 8, "f32"), (10, 1 << 31, 8, "bf16"), (10, 10, 8, "i32")):
        with pytest.raises(ValueError):
            ar.ar_linear_cross_entropy_workspace_bytes(*bad)


def test_null_comm():
    p = ctypes.c_void_p()
    refused(BAD, ar.ar_grad_norm, p, [at(0)], [4], at(1), "f32")
    refused(BAD, ar.ar_clip_grads, p, [at(0)], [at(1)], [4], 1.0, at(2), "f32")
    refused(BAD, ar.ar_all_reduce_clip, p, [at(0)], [at(1)], [4], 1.0, at(2), "f32")
    refused(BAD, ar.ar_embedding, p, at(0), at(1), at(2), 4, 4, 4, "f32", index="i32")
    refused(BAD, ar.ar_embedding_backward, p, at(0), at(1), at(2), 4, 4, 4, "f32", index="i32")
    refused(BAD, ar.ar_linear_cross_entropy, p, at(0), at(1), at(2), at(3), at(4), 4, 4, 4, "f32", index="i32")
    refused(BAD, ar.ar_linear_cross_entropy_backward, p, at(0), at(1), at(2), at(3), at(4), at(5), at(6), 4, 4, 4,
            "f32", index="i32")


@pytest.mark.parametrize("fn", ["clip", "reduce"])
def test_clip_refusals(fn):
    def call(code, send, recv, counts, max_norm=1.0, comm=None, dtype="f32", **kw):
        f = ar.ar_clip_grads if fn == "clip" else ar.ar_all_reduce_clip
        refused(code, f, host_comm(2) if comm is None else comm, send, recv, counts, max_norm, at(40), dtype, **kw)

    s, d = [at(0), at(1)], [at(2), at(3)]
    call(NOT_SERVED, s, d, [8], dtype="i32")
    call(BAD, s, d, [8], dtype=17)
    call(BAD, s, d, [8], norm=5)
    call(BAD, s, d, [8], max_norm=-1.0)
    call(BAD, s, d, [8], max_norm=float("nan"))
    call(BAD, s, d, [8], comm=host_comm(2, ar.ar_clip_workspace_bytes() - 1))
    call(BAD, [at(0), 0], d, [8])
    call(BAD, s, [0, at(3)], [8])
    call(BAD, [at(0) + 2, at(1)], d, [8])
    call(BAD, s, [at(0) + 16, at(3)], [8])         # recv overlaps rank 0's send
    call(BAD, s, [at(2), at(2) + 4], [8])          # two recv tensors overlap
    call(BAD, s, [at(2), 1 << 44], [8])            # recv overlaps the workspace
    call(BAD, s, d, [1 << 62])
    if fn == "clip":
        call(BAD, s, d, [8], layout=7)
        call(BAD, [at(0), at(1)], [at(0), at(0) + 8], [8], layout="sharded")
        refused(BAD, ar.ar_grad_norm, host_comm(2), s, [8], at(4), "f32", layout=9)
        refused(BAD, ar.ar_grad_norm, host_comm(2), s, [8], 0, "f32")
        refused(BAD, ar.ar_grad_norm, host_comm(2), s, [8], at(4) + 2, "f32")
        refused(NOT_SERVED, ar.ar_grad_norm, host_comm(2), s, [8], at(4), "i32")
    else:
        call(NOT_SERVED, s, d, [8], op="max")
        call(BAD, s, d, [8], op=9)
        call(BAD, [at(0), at(0)], d, [8])          # two ranks share a send buffer


def test_embedding_refusals():
    def look(code, w=at(0), t=at(1), o=at(2), n=4, rows=8, width=16, dtype="f32", **kw):
        refused(code, ar.ar_embedding, host_comm(), w, t, o, n, rows, width, dtype, **{"index": "i32", **kw})

    look(NOT_SERVED, dtype="i32")
    look(BAD, index=4)
    look(BAD, width=0)
    look(BAD, n=1 << 31)
    look(BAD, w=0)
    look(BAD, t=0)
    look(BAD, o=0)
    look(BAD, ld_weight=15)
    look(BAD, ld_out=15)
    look(BAD, w=at(0) + 2)
    look(BAD, t=at(1) + 2)
    look(BAD, t=at(1) + 4, index="i64")
    look(BAD, o=at(0) + 64)
    look(BAD, rows=(1 << 31) - 1, width=(1 << 31) - 1, ld_weight=1 << 62)

    def grad(code, g=at(0), t=at(1), w=at(2), n=4, rows=8, width=16, dtype="bf16", grad_dtype="bf16", comm=None, **kw):
        refused(code, ar.ar_embedding_backward, comm or host_comm(), g, t, w, n, rows, width, dtype, grad_dtype,
                **{"index": "i32", **kw})

    grad(NOT_SERVED, dtype="i32")
    grad(NOT_SERVED, grad_dtype="f16")
    grad(NOT_SERVED, dtype="f32", grad_dtype="bf16")
    grad(BAD, comm=host_comm(1, ar.ar_embedding_workspace_bytes(4, 8, 16) - 1))
    grad(BAD, g=at(2) + 2)
    grad(BAD, w=1 << 44)
    grad(BAD, g=(1 << 44) + 2)
    grad(BAD, ld_grad_out=8)
    grad(BAD, w=0)


def test_cross_entropy_refusals():
    def loss(code, x=at(0), w=at(1), y=at(2), out=at(3), lse=at(4), n=4, vocab=8, width=16, dtype="bf16", comm=None, **kw):
        refused(code, ar.ar_linear_cross_entropy, comm or host_comm(), x, w, y, out, lse, n, vocab, width, dtype,
                **{"index": "i64", **kw})

    loss(NOT_SERVED, dtype="i32")
    loss(BAD, index=3)
    loss(BAD, vocab=0)
    loss(BAD, width=0)
    loss(BAD, n=1 << 31)
    loss(BAD, x=0)
    loss(BAD, w=at(1) + 1)
    loss(BAD, y=at(2) + 4)
    loss(BAD, out=at(3) + 2)
    loss(BAD, lse=0)
    loss(BAD, lse=at(3) + 8)
    loss(BAD, out=at(0) + 4)
    loss(BAD, ld_hidden=8)
    loss(BAD, ld_weight=8)
    loss(BAD, comm=host_comm(1, ar.ar_linear_cross_entropy_workspace_bytes(4, 8, 16, "bf16") - 1))

    def grad(code, gx=at(5), gw=at(6), lse=at(3), g=at(4), comm=None, n=4, **kw):
        refused(code, ar.ar_linear_cross_entropy_backward, comm or host_comm(), at(0), at(1), at(2), lse, g, gx, gw, n, 8,
                16, "bf16", **{"index": "i64", **kw})

    grad(BAD, gx=None, gw=None)
    grad(BAD, gx=at(6))
    grad(BAD, gx=at(0))
    grad(BAD, gw=at(1) + 2)
    grad(BAD, gw=1 << 44)
    grad(BAD, lse=0)
    grad(BAD, g=0)
    grad(BAD, ld_grad_hidden=3)
    grad(BAD, ld_grad_weight=3)
    grad(BAD, comm=host_comm(1, ar.ar_linear_cross_entropy_workspace_bytes(4, 8, 16, "bf16", backward=True) - 1))


def test_binding_takes_row_pitches_from_tensors():
    x = torch.zeros(6, 10)
    assert ar._rows(x[:, :4], 0) == (x.data_ptr(), 10)
    assert ar._rows(x, 12) == (x.data_ptr(), 12)
    assert ar._rows(x[:1, :4], 0) == (x.data_ptr(), 0)
    assert ar._rows(None, 0) == (None, 0)
    with pytest.raises(ValueError):
        ar._rows(x.t(), 0)
    with pytest.raises(TypeError):
        ar._index(None, 1234)
    with pytest.raises(TypeError):
        ar._index(None, x)
    with pytest.raises(ValueError):
        ar.ar_grad_norm(host_comm(), [at(0)], [4], at(1), "f32", layout="mirrored", stream=0)


def test_depths_that_no_buffer_spans():
    """fp32 widths and tokens below 2^20, 16-bit ones below 2^24."""
    size = ar.ar_linear_cross_entropy_workspace_bytes
    for dtype, most in (("f32", 1 << 20), ("bf16", 1 << 24)):
        assert size(64, 300, most - 1, dtype) > 0 and size(most - 1, 300, 8, dtype) > 0
        for bad in ((64, 300, most), (most, 300, 8)):
            with pytest.raises(ValueError):
                size(*bad, dtype)


def test_lists_of_addresses():
    """Addresses alone, tensors among them, and what is neither."""
    x = torch.zeros(4)
    assert list(ar._ptrs([1, 2, (1 << 64) - 8])) == [1, 2, (1 << 64) - 8]
    assert list(ar._ptrs([16, x])) == [16, x.data_ptr()] and list(ar._ptrs((x, 16))) == [x.data_ptr(), 16]
    assert list(ar._ptrs([])) == []
    for bad in ([1, "2"], [1, 2.0], [1, None], ["1"]):
        with pytest.raises(TypeError):
            ar._ptrs(bad)


def test_rows_of_matrices():
    """A tensor's own pitch; rows that overlap or have gaps inside are refused."""
    x = torch.zeros(6, 8)
    assert ar._rows(x, 0) == (x.data_ptr(), 8) and ar._rows(x[:, 2:5], 0) == (x.data_ptr() + 8, 8)
    assert ar._rows(x[1:2], 0) == (x.data_ptr() + 32, 0) and ar._rows(x[::2], 0) == (x.data_ptr(), 16)
    assert ar._rows(x, 12) == (x.data_ptr(), 12) and ar._rows(64, 3) == (64, 3) and ar._rows(None, 0) == (None, 0)
    for bad in (x[:, ::2], x.t(), torch.zeros(1, 8).expand(6, 8), x.as_strided((4, 8), (4, 1))):
        with pytest.raises(ValueError):
            ar._rows(bad, 0)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses are not for a GPU")
def test_a_workspace_serves_fewer_tokens():
    """What the size function gives for n tokens passes the check of every call
    with fewer: such a call gets as far as HIP."""
    rng = random.Random(1)

    def passes(fn, *args, **kw):
        with pytest.raises(ar.ArError) as e:
            fn(*args, **kw, stream=0)
        assert e.value.code == ar.AR_ERR_HIP, str(e.value)

    for _ in range(150):
        n, vocab, width = (int(2 ** rng.uniform(0, k)) for k in (14, 18, 13))
        dtype = rng.choice(["f32", "f16", "bf16"])
        ws = [ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, dtype, backward=b) for b in (False, True)]
        emb = ar.ar_embedding_workspace_bytes(n, vocab, width)
        for m in {n, max(1, n - 1), (n + 1) // 2, min(n, 64), min(n, 65), min(n, 16), min(n, 17), 1, rng.randint(1, n)}:
            far = [(1 << 45) * k for k in range(1, 8)]
            passes(ar.ar_linear_cross_entropy, host_comm(ws_bytes=ws[0]), far[0], far[1], far[2], far[3], far[4], m, vocab,
                   width, dtype, index="i64")
            passes(ar.ar_linear_cross_entropy_backward, host_comm(ws_bytes=ws[1]), far[0], far[1], far[2], far[3],
                   far[4], far[5], far[6], m, vocab, width, dtype, index="i64")
            passes(ar.ar_embedding_backward, host_comm(ws_bytes=emb), far[0], far[1], far[2], m, vocab, width, dtype,
                   index="i32")
