"""Orthogonalised updates without a GPU: workspace sizes, refusals and lists of
matrices, which come before the first HIP call."""
import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_lm_host import BAD, NOT_SERVED, at, host_comm, refused

SIZE = ar.ar_orthogonalize_workspace_bytes


def test_workspace_sizes():
    assert SIZE(0, 10, 10) == 0 and SIZE(3, 0, 10) == 0
    one, four, many = SIZE(1, 300, 500), SIZE(4, 300, 500), SIZE(1000, 300, 500)
    assert 300 * 500 * 12 < one and one < four <= 4 * one < many <= 32 * one
    assert SIZE(1, 300, 500) == SIZE(1, 500, 300)
    # a list of large matrices goes through the workspace in groups
    assert SIZE(32, 4096, 8192) <= (4 << 30) + SIZE(1, 4096, 8192)
    for bad in ((-1, 4, 4), (1, 1 << 20, 4), (1, 4, 1 << 20), (1, 1 << 17, 1 << 17), (1, 1 << 16, 1 << 19),
                (ar.MAX_TENSORS + 1, 4, 4)):
        with pytest.raises(ValueError):
            SIZE(*bad)


BAD_COEFFICIENTS = [(float("nan"), 0, 0), (1, float("inf"), 1), (17, -1, 1), (1, -33, 20), (1, 1, 33), (1, 1, 0.05), (1, -20, 2)]


def test_orthogonalize_refusals():
    def call(code, x=None, y=None, rows=8, cols=16, comm=None, dtype="bf16", **kw):
        refused(code, ar.ar_orthogonalize, comm or host_comm(), [at(0), at(1)] if x is None else x,
                [at(2), at(3)] if y is None else y, rows, cols, dtype, **kw)

    call(NOT_SERVED, dtype="i32")
    call(BAD, dtype=9)
    for steps in (0, -1, 33):
        call(BAD, steps=steps)
    for co in BAD_COEFFICIENTS:
        call(BAD, coefficients=co)
        call(BAD, coefficients=[(1, 1, 1), co], steps=2)
    for eps in (0.0, -1.0, 1e-40, float("inf"), float("nan")):
        call(BAD, eps=eps)
    call(BAD, rows=1 << 20)
    call(BAD, rows=1 << 17, cols=1 << 17)
    call(BAD, x=[at(0), 0])
    call(BAD, y=[at(2), 0])
    call(BAD, x=[at(0), at(1) + 1])
    call(BAD, y=[at(2), at(2)])
    call(BAD, y=[at(2), at(2) + 8 * 16 * 2 - 2])
    call(BAD, y=[at(0) + 2, at(3)])      # over its own matrix, but not in place
    call(BAD, y=[at(1), at(3)])          # over another one's
    call(BAD, x=[at(0), at(0) + 64], y=[at(0), at(3)])
    call(BAD, y=[at(2), 1 << 44])
    call(BAD, x=[at(0), 1 << 44])
    call(BAD, ld_in=15)
    call(BAD, ld_out=15)
    call(BAD, y=[at(0), at(1)], ld_in=16, ld_out=20)  # in place of another pitch
    call(BAD, comm=host_comm(1, SIZE(2, 8, 16) - 1))
    with pytest.raises(ValueError):
        call(BAD, y=[at(2)])
    with pytest.raises(ValueError):
        call(BAD, coefficients=[(1, 1, 1), (1, 1, 1)], steps=3)


def test_update_refusals():
    def call(code, g=None, mi=None, mo=None, wi=None, wo=None, comm=None, dtype="bf16", weight_dtype="f32", **kw):
        lists = [x if x is not None else [at(2 * k), at(2 * k + 1)] for k, x in enumerate((g, mi, mo, wi))]
        wo = [[at(8), at(9)], [at(10), at(11)]] if wo is None else wo
        refused(code, ar.ar_muon_update, comm or host_comm(2), *lists, [b for row in wo for b in row], 8, 16, dtype,
                weight_dtype, **kw)

    call(NOT_SERVED, dtype="i32")
    call(NOT_SERVED, weight_dtype="i32")
    call(NOT_SERVED, weight_dtype="f16")
    call(NOT_SERVED, dtype="f32", weight_dtype="bf16")
    for decay in (-0.1, 1.0, float("nan")):
        call(BAD, decay=decay)
    for k in ("lr", "weight_decay", "update_scale"):
        call(BAD, **{k: float("inf")})
        call(BAD, **{k: float("nan")})
        call(BAD, **{k: 1e39})
    call(BAD, lr=1e20, update_scale=1e20)
    call(BAD, lr=-1e20, weight_decay=1e20)
    call(BAD, steps=0)
    call(BAD, eps=0.0)
    for k in ("g", "mi", "mo", "wi"):
        call(BAD, **{k: [at(20), 0]})
        call(BAD, **{k: [at(20), at(21) + 1]})
    call(BAD, wo=[[at(8), at(9)], [at(10), 0]])
    call(BAD, mo=[at(4), at(4)])
    call(BAD, mo=[at(3), at(2)])                          # in place, but of the other matrix
    call(BAD, mo=[at(0), at(5)])                          # over a gradient
    call(BAD, wo=[[at(7), at(9)], [at(10), at(11)]])      # over the other matrix
    call(BAD, wo=[[at(8), at(8)], [at(10), at(11)]])
    call(BAD, wo=[[at(4) + 4, at(9)], [at(10), at(11)]])  # over the momentum
    call(BAD, wo=[[at(6) + 4, at(9)], [at(10), at(11)]])
    call(BAD, wo=[[1 << 44, at(9)], [at(10), at(11)]])
    call(BAD, ld_grads=15)
    call(BAD, ld_momentum=15)
    call(BAD, ld_weights=15)
    call(BAD, comm=host_comm(2, SIZE(2, 8, 16) - 1))


def test_null_comm_and_arrays():
    rc = ar._lib.ar_orthogonalize(None, 0, None, None, 4, 4, 0, 0, 5, None, 1e-7, ar.AR_FLOAT32, None)
    assert rc == BAD
    rc = ar._lib.ar_orthogonalize(host_comm(), 1, None, None, 4, 4, 0, 0, 5, None, 1e-7, ar.AR_FLOAT32, None)
    assert rc == BAD
    rc = ar._lib.ar_muon_update(host_comm(), 1, None, None, None, None, None, 4, 4, 0, 0, 0, 0.9, 1, 0.1, 0.0, 1.0, 5, None,
                                1e-7, ar.AR_FLOAT32, ar.AR_FLOAT32, None)
    assert rc == BAD
    assert ar._lib.ar_orthogonalize(host_comm(), 0, None, None, 4, 4, 0, 0, 5, None, 1e-7, ar.AR_FLOAT32, None) == ar.AR_SUCCESS


def test_lists_of_matrices():
    """Tensors give their own pitch, the same for all."""
    x = torch.zeros(6, 10)
    p, ld = ar._matrices([x[:, :4], x[:3, 5:9]], 0)
    assert list(p) == [x.data_ptr(), x.data_ptr() + 20] and ld == 10
    assert list(ar._matrices([64, 128], 12)[0]) == [64, 128] and ar._matrices([64], 12)[1] == 12
    assert ar._matrices([x[:, :4]], 12)[1] == 12 and ar._matrices([], 0)[1] == 0
    assert list(ar._matrices([x, x[:, :4]], 12)[0]) == [x.data_ptr()] * 2
    with pytest.raises(ValueError):
        ar._matrices([x[:, :4], torch.zeros(6, 4)], 0)
    with pytest.raises(ValueError):
        ar._matrices([x.t()], 0)
    assert list(ar._coefficients((1, 2, 3), 2)) == [1, 2, 3, 1, 2, 3] and ar._coefficients(None, 4) is None
