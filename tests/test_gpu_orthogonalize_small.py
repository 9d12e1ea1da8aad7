"""Orthogonalised matrices of the sizes that one workgroup takes, and of those
just beyond, against the same iteration in fp32.

A step's own error, of the bracket's size: D is stored to 2^-23 and enters c D D
twice, whose small halves' product is left out at 2^-22 of it, and the bracket is
stored to 2^-23; with the default's coefficients that is 4.3 * 2^-23 of it, at
most 2^-21 with X's own 2^-23. fp32 rounds X to 2^-24 in every step, though its
error may come out smaller: at most eight times its error, or steps * 2^-21.
"""
import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_gpu_lm import T, U, comms, nan_like  # noqa: F401
from test_gpu_orthogonalize import iterate, matrices, workspace
from test_gpu_orthogonalize_large import spread

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (1, 7), (9, 1), (2, 300), (16, 16), (31, 33), (32, 64), (63, 65), (64, 192), (192, 64), (65, 64), (96, 97),
         (100, 60), (8, 2500), (32, 600), (600, 32), (40, 450), (128, 128), (129, 127), (100, 257), (257, 100), (260, 511)]


def check(x, y, dtype, steps=5):
    ref = iterate(x.double(), steps)
    plain, size = float((iterate(x.float(), steps).double() - ref).norm()), float(ref.norm())
    most = max(8 * plain, steps * 2.0 ** -21 * size)
    assert most <= 1e-3 * size
    off = float((y.double() - ref).norm())
    assert off <= most + (U[dtype] * size if dtype != "f32" else 0.0), (off, plain, size)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(comms, dtype, rows, cols):  # noqa: F811
    comm = workspace(comms, 3, rows, cols)
    ins = matrices(50, 3, rows, cols, dtype)
    for steps in (5, 1, 3):
        outs = [nan_like(rows, cols, dtype=dtype) for _ in ins]
        ar.ar_orthogonalize(comm, ins, outs, rows, cols, dtype, steps=steps)
        for x, y in zip(ins, outs):
            check(x, y, dtype, steps)


@pytest.mark.parametrize("decades", [2, 4])
@pytest.mark.parametrize("rows,cols", [(16, 16), (64, 192), (192, 64), (32, 600), (60, 61), (129, 127), (260, 511)])
def test_singular_values_far_apart(comms, rows, cols, decades):  # noqa: F811
    comm = workspace(comms, 1, rows, cols)
    x, y = spread(rows, cols, decades), nan_like(rows, cols, dtype="f32")
    ar.ar_orthogonalize(comm, [x], [y], rows, cols, "f32")
    check(x, y, "f32")
