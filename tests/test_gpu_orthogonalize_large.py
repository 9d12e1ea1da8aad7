"""Orthogonalised matrices of the sizes that take tiles of 128 and 256, sums in
parts and steps in segments, against the same iteration in fp32.

Stored pairs of fp16 numbers are off by at most 2^-22 where fp32 rounds to
2^-24, and a product's small halves, left out, are another 2^-22 of it: an error
is at most eight times that of the same iteration in fp32, which in turn is a
small part of the result, so that a wrong tile shows.
"""
import math

import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_gpu_lm import T, U, U32, comms, gen, margins_untouched, nan_like, normal, placed  # noqa: F401
from test_gpu_orthogonalize import iterate, matrices, update_ref, workspace

pytestmark = pytest.mark.gpu

POLAR = [(8.28721, -23.59588, 17.30038), (4.10706, -2.94785, 0.54484), (3.94869, -2.90890, 0.55181),
         (3.31842, -2.48848, 0.51004), (2.300652, -1.66890, 0.418807)]


def cosines(rows, n):
    """The first rows of an orthogonal matrix."""
    k = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None]
    j = torch.arange(n, dtype=torch.float64, device="cuda")[None]
    q = torch.cos(math.pi / n * (j + 0.5) * k) * math.sqrt(2.0 / n)
    q[0] *= math.sqrt(0.5)
    return q


def spread(rows, cols, decades):
    """A matrix whose singular values span so many decades."""
    m = min(rows, cols)
    s = torch.logspace(0, -decades, m, dtype=torch.float64, device="cuda")
    return ((cosines(m, rows).t() * s) @ cosines(m, cols)).float()


def check_as_fp32(x, y, dtype, steps=5, co=None):
    ref = iterate(x.double(), steps, co)
    plain, size = float((iterate(x.float(), steps, co).double() - ref).norm()), float(ref.norm())
    most = 8 * plain + (U[dtype] * size if dtype != "f32" else 0.0)
    assert 8 * plain <= 1e-3 * size  # a bound that means something
    off = float((y.double() - ref).norm())
    assert off <= most, (off, plain, size)


def check(comms, count, rows, cols, dtype, steps=5, co=None, seed=40, pitch=0):  # noqa: F811
    comm = workspace(comms, count, rows, cols)
    ins = matrices(seed, count, rows, cols, dtype, pitch=pitch)
    outs = [placed(nan_like(rows, cols, dtype=dtype), 0, pitch and cols + pitch) for _ in range(count)]
    ar.ar_orthogonalize(comm, ins, outs, rows, cols, dtype, steps=steps, coefficients=co)
    for x, y in zip(ins, outs):
        check_as_fp32(x, y, dtype, steps, co)
        assert margins_untouched(y)
    again = [torch.full((rows, cols), float("nan"), dtype=T[dtype], device="cuda") for _ in range(count)]
    ar.ar_orthogonalize(comm, ins, again, rows, cols, dtype, steps=steps, coefficients=co)
    assert all(torch.equal(x, y) for x, y in zip(outs, again))


@pytest.mark.parametrize("count,rows,cols,dtype", [
    (1, 1500, 1700, "f32"),                          # symmetric tiles of 64, the others of 128 in parts
    (8, 1500, 1700, "f32"), (6, 1700, 1500, "f32"),  # of 128, and of 256 with rows and columns left over
    (2, 1500, 6000, "f32"), (2, 6000, 1500, "f32"),  # segments; all of 128 in parts
    (1, 2049, 8200, "f32"), (1, 8200, 2049, "bf16"),
    (3, 5000, 1500, "f32"), (4, 1500, 3100, "f16"),  # segments with tiles of 256
    (1, 1600, 9000, "f32"), (2, 2100, 2300, "f32"), (1, 4000, 4100, "f32"), (1, 4096, 8192, "f32"),
    (2, 2100, 1030, "bf16"), (40, 600, 700, "f32")])  # two groups of different tiles
def test_sizes(comms, count, rows, cols, dtype):  # noqa: F811
    check(comms, count, rows, cols, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_on_no_vector(comms, dtype):  # noqa: F811
    check(comms, 5, 771, 3001, dtype, pitch=3)
    check(comms, 5, 3001, 771, dtype, pitch=3)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("rows,cols,count", [(770, 3000, 5), (3000, 770, 5), (1500, 1700, 6)])
def test_steps(comms, steps, rows, cols, count):  # noqa: F811
    """Segments of one to three steps, and steps by themselves."""
    check(comms, count, rows, cols, "f32", steps=steps)


@pytest.mark.parametrize("rows,cols,count", [(770, 3000, 5), (6000, 1500, 2), (1100, 1300, 1), (96, 160, 2)])
def test_coefficients_of_every_step(comms, rows, cols, count):  # noqa: F811
    check(comms, count, rows, cols, "f32", steps=5, co=POLAR)
    check(comms, count, rows, cols, "f32", steps=6, co=(1.5, -0.5, 0.0))


@pytest.mark.parametrize("decades", [2, 4, 6])
@pytest.mark.parametrize("rows,cols", [(900, 3300), (3300, 900), (2049, 8200), (1500, 1700)])
def test_singular_values_far_apart(comms, rows, cols, decades):  # noqa: F811
    comm = workspace(comms, 1, rows, cols)
    x, y = spread(rows, cols, decades), nan_like(rows, cols, dtype="f32")
    ar.ar_orthogonalize(comm, [x], [y], rows, cols, "f32")
    check_as_fp32(x, y, "f32")


@pytest.mark.parametrize("steps", [4, 6, 8, 10])
@pytest.mark.parametrize("rows,cols", [(770, 3000), (3000, 770)])
def test_many_steps(comms, rows, cols, steps):  # noqa: F811
    """Several segments; of a list, whose first matrix is compared."""
    comm = workspace(comms, 5, rows, cols)
    x = spread(rows, cols, 2)
    outs = [nan_like(rows, cols, dtype="f32") for _ in range(5)]
    ar.ar_orthogonalize(comm, [x] * 5, outs, rows, cols, "f32", steps=steps)
    check_as_fp32(x, outs[0], "f32", steps)
    assert all(torch.equal(y, outs[0]) for y in outs)


@pytest.mark.parametrize("count,rows,cols,dtype,ranks", [(3, 5000, 1500, "f32", 1), (8, 1500, 1700, "bf16", 2),
                                                         (6, 1100, 1300, "bf16", 3), (1, 2049, 8200, "f16", 1)])
def test_update(comms, count, rows, cols, dtype, ranks):  # noqa: F811
    comm = workspace(comms, count, rows, cols, ranks)
    g = gen(41)
    h = {"decay": 0.9, "nesterov": True, "lr": 0.5, "weight_decay": 0.2, "update_scale": 2.0}
    grads, mom = matrices(42, count, rows, cols, dtype), matrices(43, count, rows, cols, "f32", 3e-4)
    w = [normal(g, rows, cols, std=0.02) for _ in range(count)]
    out = [[nan_like(rows, cols, dtype="f32") for _ in range(ranks)] for _ in range(count)]
    old = [m.clone() for m in mom]
    ar.ar_muon_update(comm, grads, mom, mom, w, out, rows, cols, dtype, "f32", **h)
    for a, b, m, c, replicas in zip(grads, old, mom, w, out):
        new, x, ref = update_ref(a.double(), b.double(), c.double(), h)
        plain = float((update_ref(a.float(), b, c, h)[1].double() - x).norm())
        size = float(x.norm())
        assert 8 * plain <= 1e-3 * size
        terms = h["decay"] * b.double().abs() + (1 - h["decay"]) * a.double().abs()
        assert ((m.double() - new).abs() <= 4 * U32 * terms).all()
        off = float((replicas[0].double() - ref).norm())
        # (X's error times lr update_scale = 1, and the roundings of two products and their sum)
        assert off <= 8 * plain + 4 * U32 * (float(ref.norm()) + size), (off, plain, size)
        assert all(torch.equal(y, replicas[0]) for y in replicas)


@pytest.mark.parametrize("rows,cols,count", [(770, 3000, 5), (3000, 770, 5), (520, 640, 2), (1100, 1300, 1)])
def test_coefficients_that_singular_values_of_one_would_not_bear(comms, rows, cols, count):  # noqa: F811
    """(0.5, 32, 32) takes small singular values to 0 and large ones beyond all bounds;
    the matrices here have small ones. c D D of D = A + I / 2 is 16 times the bracket: each
    step is off by up to 2^-17 of it, by the roundings of D and what a product leaves out."""
    comm = workspace(comms, count, rows, cols)
    g = gen(44)
    ins = [normal(g, rows, cols) for _ in range(count)]
    outs = [nan_like(rows, cols, dtype="f32") for _ in ins]
    co, steps = (0.5, 32.0, 32.0), 5
    ar.ar_orthogonalize(comm, ins, outs, rows, cols, "f32", steps=steps, coefficients=co)
    for x, y in zip(ins, outs):
        ref = iterate(x.double(), steps, co)
        assert float((y.double() - ref).norm()) <= steps * 2.0 ** -17 * float(ref.norm())
    for co in ((0.5, 32.0, 32.0), (4.0, 32.0, 32.0)):
        zeros = [torch.zeros(rows, cols, device="cuda") for _ in range(count)]
        ar.ar_orthogonalize(comm, zeros, outs, rows, cols, "f32", steps=32, coefficients=co)
        assert all((y == 0).all() for y in outs)


@pytest.mark.parametrize("steps", [4, 5, 6, 8])
@pytest.mark.parametrize("rows,cols", [(40, 883), (72, 1100), (1222, 106), (1409, 49), (128, 2500), (256, 1024), (300, 2000)])
def test_thin_matrices_with_one_large_singular_value(comms, rows, cols, steps):  # noqa: F811
    """Few rows: a rounding of A weighs the more beside the others' part of it."""
    comm = workspace(comms, 9, rows, cols)
    g = gen(45)
    ins = [normal(g, rows, rank) @ normal(g, rank, cols) + noise * normal(g, rows, cols)
           for rank in (1, 4, 16) for noise in (1.0, 0.5, 0.3)]
    outs = [nan_like(rows, cols, dtype="f32") for _ in ins]
    ar.ar_orthogonalize(comm, ins, outs, rows, cols, "f32", steps=steps)
    for x, y in zip(ins, outs):
        check_as_fp32(x, y, "f32", steps)
