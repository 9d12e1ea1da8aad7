"""Orthogonalised matrices and the weights' update with them on a GPU, against
the same iteration in 64 bits.

Bounds are of Frobenius norms. A rounding error E of X grows in one step by at
most L = max |p'(s)| over the singular values that occur, p(s) = a s + b s^3 + c
s^5; each step adds what its own roundings make. A sum of k fp32 products is
taken to be off by 6 sqrt(k) 2^-24 of the sum of magnitudes (the probabilistic
bound of rounding analysis at six deviations), stored pairs of fp16 numbers by
2^-22, and the product of their small halves, which is left out, by 2^-22.
"""
import math

import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_gpu_lm import T, TINY, U, U32, close, comms, gen, margins_untouched, nan_like, normal, placed  # noqa: F401

pytestmark = pytest.mark.gpu

QUINTIC = (3.4445, -4.7750, 2.0315)
U22 = 2.0 ** -22
EPS = 1e-7


def coefficients(co, steps):
    co = co or QUINTIC
    return [co] * steps if not isinstance(co[0], (tuple, list)) else list(co)


def iterate(u, steps=5, co=None, eps=EPS):
    """The definition, in the type of u."""
    tall = u.shape[0] > u.shape[1]
    x = u.t().contiguous() if tall else u
    x = x / x.double().square().sum().sqrt().clamp(min=eps).to(x.dtype)
    for a, b, c in coefficients(co, steps):
        gram = x @ x.t().contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t().contiguous() if tall else x


def error_bound(rows, cols, steps=5, co=None):
    m, n = min(rows, cols), max(rows, cols)
    top, e, rank = 1.0, U22 * 2, min(m, 1e9)
    grid = torch.linspace(0, 1, 2001, dtype=torch.float64)
    for a, b, c in coefficients(co, steps):
        s = grid * top
        slope = float((a + 3 * b * s ** 2 + 5 * c * s ** 4).abs().max())
        x_f = top * math.sqrt(rank) if top < 1.0 or e > U22 * 2 else 1.0  # the first X has the norm 1
        shift = b / (2 * c) if c else 0.0
        d_2 = max(abs(shift), abs(top ** 2 + shift), top ** 2)
        d_f = d_2 * math.sqrt(rank)
        a_err = (6 * math.sqrt(n) * U32 + 2 * U22) * x_f ** 2
        if c:
            d_err = a_err + U22 * d_f
            q_err = abs(c) * (2 * d_2 * d_err + (6 * math.sqrt(m) * U32 + 2 * U22) * d_f ** 2)
            q_f = (abs(a) + abs(b) * top ** 2 + abs(c) * top ** 4) * math.sqrt(rank)
        else:
            q_err, q_f = abs(b) * a_err, (abs(a) + abs(b) * top ** 2) * math.sqrt(rank)
        q_err += U22 * q_f
        own = q_err * top + (6 * math.sqrt(m) * U32 + 3 * U22) * q_f * x_f
        e = slope * e + own
        top = float((a * s + b * s ** 3 + c * s ** 5).abs().max())
    return e


def check_result(got, ref, dtype, bound):
    assert torch.isfinite(got.float()).all()
    off = float((got.double() - ref).norm())
    most = bound + U[dtype] * float(ref.norm()) + TINY[dtype] * math.sqrt(ref.numel())
    assert off <= most, (off, most)


def workspace(comms, count, rows, cols, ranks=1):  # noqa: F811
    return comms(ranks, max(ar.ar_orthogonalize_workspace_bytes(count, rows, cols), 256))


def matrices(seed, count, rows, cols, dtype, std=1e-3, offset=0, pitch=0):
    g = gen(seed)
    out = []
    for _ in range(count):
        r = min(4, rows, cols)
        x = normal(g, rows, r) @ normal(g, r, cols) + normal(g, rows, cols)
        out.append(placed((x * std).to(T[dtype]), offset, pitch and cols + pitch))
    return out


def check(comms, count, rows, cols, dtype, seed=1, steps=5, co=None, offset=0, pitch=0, std=1e-3):  # noqa: F811
    comm = workspace(comms, count, rows, cols)
    ins = matrices(seed, count, rows, cols, dtype, std, offset, pitch)
    outs = [placed(nan_like(rows, cols, dtype=dtype), offset, pitch and cols + 2 * pitch) for _ in range(count)]
    ar.ar_orthogonalize(comm, ins, outs, rows, cols, dtype, steps=steps, coefficients=co)
    bound = error_bound(rows, cols, steps, co)
    for x, y in zip(ins, outs):
        check_result(y, iterate(x.double(), steps, co), dtype, bound)
        assert margins_untouched(y)
    again = [torch.full((rows, cols), float("nan"), dtype=T[dtype], device="cuda") for _ in range(count)]
    ar.ar_orthogonalize(comm, ins, again, rows, cols, dtype, steps=steps, coefficients=co)
    assert all(torch.equal(x, y) for x, y in zip(outs, again))


SIZES = [(1, 1), (1, 7), (9, 1), (2, 300), (16, 16), (31, 33), (32, 64), (63, 65), (64, 192), (65, 64), (100, 257), (128, 128),
         (129, 127), (200, 1000), (257, 511), (770, 130)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_matrices(comms, dtype, rows, cols):  # noqa: F811
    check(comms, 3, rows, cols, dtype)


@pytest.mark.parametrize("rows,cols,dtype", [(1, 1_000_003, "f32"), (3, 600_001, "bf16"), (700_001, 2, "f16"),
                                             ((1 << 20) - 1, 1, "f32")])
def test_long_and_thin(comms, rows, cols, dtype):  # noqa: F811
    check(comms, 2, rows, cols, dtype, seed=3)


@pytest.mark.parametrize("count,rows,cols,dtype", [(1, 1500, 1700, "f32"), (2, 2100, 1030, "bf16"), (20, 520, 640, "f32"),
                                                   (70, 130, 90, "bf16"), (40, 64, 64, "f16")])
def test_large_tiles_and_groups(comms, count, rows, cols, dtype):  # noqa: F811
    """Tiles of 128, and lists of several groups."""
    check(comms, count, rows, cols, dtype, seed=2)


@pytest.mark.parametrize("dtype,offset,pitch", [("f32", 1, 0), ("f32", 0, 4), ("bf16", 0, 8), ("bf16", 3, 0), ("f16", 0, 3),
                                                ("f16", 8, 64)])
def test_strided_rows(comms, dtype, offset, pitch):  # noqa: F811
    check(comms, 2, 72, 136, dtype, offset=offset, pitch=pitch)
    check(comms, 2, 136, 72, dtype, offset=offset, pitch=pitch)


@pytest.mark.parametrize("steps,co", [(1, None), (2, None), (8, (1.5, -0.5, 0.0)), (3, (1.875, -1.25, 0.375)),
                                      (4, [(8.28721, -23.59588, 17.30038), (4.10706, -2.94785, 0.54484), (3.94869, -2.90890, 0.55181),
                                           (3.31842, -2.48848, 0.51004)])])
@pytest.mark.parametrize("rows,cols", [(96, 160), (300, 128)])
def test_steps_and_coefficients(comms, steps, co, rows, cols):  # noqa: F811
    check(comms, 2, rows, cols, "f32", steps=steps, co=co)


@pytest.mark.parametrize("std", [1e-30, 1e-12, 1.0, 1e15, 1e30])
def test_any_size_of_numbers(comms, std):  # noqa: F811
    """Squares below and beyond fp32's range; below eps the result is in / eps after the steps."""
    check(comms, 2, 64, 96, "f32", std=std)


def test_orthogonal_in_orthogonal_out(comms):  # noqa: F811
    """s Q of an orthogonal Q: every singular value takes the same way."""
    m, n = 96, 256
    q = torch.linalg.qr(torch.randn(n, m, generator=gen(3), device="cuda", dtype=torch.float64)).Q.t().contiguous()
    s = 1 / math.sqrt(m)
    for a, b, c in [QUINTIC] * 5:
        s = a * s + b * s ** 3 + c * s ** 5
    comm = workspace(comms, 1, m, n)
    x, y = (7.0 * q).float(), nan_like(m, n, dtype="f32")
    ar.ar_orthogonalize(comm, [x], [y], m, n, "f32")
    check_result(y, s * q, "f32", error_bound(m, n))


@pytest.mark.parametrize("rows,cols", [(512, 1024), (700, 700)])
def test_as_exact_as_fp32_products(comms, rows, cols):  # noqa: F811
    """Pairs of fp16 numbers round to 2^-22 and leave 2^-22 out where fp32 rounds
    to 2^-24: at most eight times the error of the same iteration in fp32; where
    singular values span six decades too."""
    g = gen(4)
    comm = workspace(comms, 2, rows, cols)
    m = min(rows, cols)
    u = torch.linalg.qr(torch.randn(rows, m, generator=g, device="cuda", dtype=torch.float64)).Q
    v = torch.linalg.qr(torch.randn(cols, m, generator=g, device="cuda", dtype=torch.float64)).Q
    spread = (u * torch.logspace(0, -6, m, dtype=torch.float64, device="cuda")) @ v.t().contiguous()
    ins = [normal(g, rows, cols), spread.float()]
    outs = [nan_like(rows, cols, dtype="f32") for _ in ins]
    ar.ar_orthogonalize(comm, ins, outs, rows, cols, "f32")
    for x, y in zip(ins, outs):
        ref = iterate(x.double())
        plain = float((iterate(x).double() - ref).norm())
        assert float((y.double() - ref).norm()) <= 8 * plain


def test_zeros_and_numbers_that_are_none(comms):  # noqa: F811
    """Zeros stay zeros; a NaN or an infinity spoils its own matrix alone."""
    for rows, cols in ((64, 100), (300, 260)):
        comm = workspace(comms, 4, rows, cols)
        ins = matrices(5, 4, rows, cols, "bf16")
        clean = [nan_like(rows, cols, dtype="bf16") for _ in ins]
        ar.ar_orthogonalize(comm, ins, clean, rows, cols, "bf16")
        ins[0].zero_()
        ins[1][3, 5] = float("nan")
        ins[2][7, 2] = float("inf")
        outs = [nan_like(rows, cols, dtype="bf16") for _ in ins]
        ar.ar_orthogonalize(comm, ins, outs, rows, cols, "bf16")
        assert (outs[0] == 0).all()
        assert torch.isnan(outs[1]).all() and torch.isnan(outs[2]).all()
        assert torch.equal(outs[3], clean[3])


def test_in_place_and_nothing(comms):  # noqa: F811
    for rows, cols in ((100, 60), (60, 100)):
        comm = workspace(comms, 3, rows, cols)
        ins = matrices(6, 3, rows, cols, "f32")
        outs = [nan_like(rows, cols, dtype="f32") for _ in ins]
        ar.ar_orthogonalize(comm, ins, outs, rows, cols, "f32")
        ar.ar_orthogonalize(comm, ins, ins, rows, cols, "f32")
        assert all(torch.equal(x, y) for x, y in zip(ins, outs))
    ar.ar_orthogonalize(comm, [], [], 4, 4, "f32")
    ar.ar_orthogonalize(comm, [0], [0], 0, 4, "f32")


def test_rows_past_32_bits(comms):  # noqa: F811
    """Rows whose offsets pass 2^32 bytes give what the same rows on end give."""
    for rows, cols, pitch in ((70, 30, 1 << 24), (300, 130, 1 << 22)):
        comm = workspace(comms, 1, rows, cols)
        near = matrices(8, 1, rows, cols, "f32")[0]
        big = torch.empty(2 * rows * pitch, device="cuda")
        far, out = (big.as_strided((rows, cols), (pitch, 1), k * rows * pitch + 1) for k in range(2))
        far.copy_(near)
        want = torch.empty_like(near)
        ar.ar_orthogonalize(comm, [near], [want], rows, cols, "f32")
        ar.ar_orthogonalize(comm, [far], [out], rows, cols, "f32")
        assert torch.equal(out, want)


# ---------------------------------------------------------------------------
# the update of weights
# ---------------------------------------------------------------------------
def update_ref(g, m, w, h, steps=5):
    new = h["decay"] * m + (1 - h["decay"]) * g
    u = h["decay"] * new + (1 - h["decay"]) * g if h["nesterov"] else new
    x = iterate(u, steps)
    return new, x, (1 - h["lr"] * h["weight_decay"]) * w - h["lr"] * h["update_scale"] * x


def check_update(comms, count, rows, cols, dtype, weight_dtype, ranks=1, nesterov=True, seed=7, in_place=False,  # noqa: F811
                 pitch=0, offset=0, steps=5):
    comm = workspace(comms, count, rows, cols, ranks)
    g = gen(seed)
    h = {"decay": 0.9, "nesterov": nesterov, "lr": 0.03, "weight_decay": 0.2, "update_scale": 1.7}
    grads = matrices(seed, count, rows, cols, dtype, offset=offset, pitch=pitch)
    mom = matrices(seed + 1, count, rows, cols, "f32", 3e-4, offset=offset, pitch=pitch)
    w = [placed(normal(g, rows, cols, dtype=weight_dtype, std=0.2), offset, pitch and cols + pitch) for _ in range(count)]
    terms = [h["decay"] * b.double().abs() + (1 - h["decay"]) * a.double().abs() for a, b in zip(grads, mom)]
    refs = [update_ref(a.double(), b.double(), c.double(), h, steps) for a, b, c in zip(grads, mom, w)]
    if in_place:
        mom_out = mom
        out = [[x] + [placed(nan_like(rows, cols, dtype=weight_dtype), offset, pitch and cols + pitch)
                      for _ in range(ranks - 1)] for x in w]
    else:
        mom_out = [placed(nan_like(rows, cols, dtype="f32"), offset, pitch and cols + pitch) for _ in range(count)]
        out = [[placed(nan_like(rows, cols, dtype=weight_dtype), offset, pitch and cols + pitch) for _ in range(ranks)]
               for _ in range(count)]
    ar.ar_muon_update(comm, grads, mom, mom_out, w, out, rows, cols, dtype, weight_dtype, steps=steps, **h)
    # U is off by two or three roundings of its terms, whose sizes its own may be below
    bound = error_bound(rows, cols, steps)
    for (new, x, ref), m, replicas, size in zip(refs, mom_out, out, terms):
        assert ((m.double() - new).abs() <= 4 * U32 * size + TINY["f32"]).all()
        # and grows with every step as the first X does
        grown = 4 ** steps * 8 * U32
        for y in replicas:
            assert torch.equal(y, replicas[0])
        off = float((replicas[0].double() - ref).norm())
        gain = h["lr"] * h["update_scale"]
        most = gain * (bound + grown) + (U[weight_dtype] + 4 * U32) * float(ref.norm()) + 4 * U32 * gain * float(x.norm())
        assert off <= most, (off, most)
        assert all(margins_untouched(y) for y in replicas) and margins_untouched(m)


@pytest.mark.parametrize("dtype,weight_dtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("rows,cols", [(1, 5), (64, 64), (65, 130), (300, 200), (128, 384)])
def test_update(comms, dtype, weight_dtype, rows, cols):  # noqa: F811
    check_update(comms, 3, rows, cols, dtype, weight_dtype)
    check_update(comms, 2, rows, cols, dtype, weight_dtype, nesterov=False, steps=3)


@pytest.mark.parametrize("ranks,count", [(2, 5), (5, 3), (64, 8)])
def test_update_of_every_rank(comms, ranks, count):  # noqa: F811
    """Replicas of all ranks; 64 ranks take groups of six matrices."""
    check_update(comms, count, 70, 96, "bf16", "bf16", ranks=ranks)


@pytest.mark.parametrize("ranks", [1, 3])
def test_update_in_place(comms, ranks):  # noqa: F811
    check_update(comms, 3, 96, 200, "bf16", "f32", ranks=ranks, in_place=True)


@pytest.mark.parametrize("dtype,offset,pitch", [("bf16", 1, 0), ("bf16", 0, 8), ("f32", 0, 1), ("f16", 3, 5)])
def test_update_of_strided_rows(comms, dtype, offset, pitch):  # noqa: F811
    check_update(comms, 2, 72, 100, dtype, dtype, offset=offset, pitch=pitch, ranks=2)
    check_update(comms, 2, 100, 72, dtype, "f32", offset=offset, pitch=pitch)


def test_update_of_large_tiles(comms):  # noqa: F811
    check_update(comms, 6, 1100, 1300, "bf16", "bf16", ranks=2)


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols,count", [(96, 160, 3), (64, 100, 3), (600, 1100, 2)])
def test_on_another_stream_and_in_a_graph(comms, rows, cols, count):  # noqa: F811
    """Averaged, clipped and applied in place: three steps of a captured graph
    between eager work, each against the eager steps."""
    ranks = 2
    comm = comms(ranks, max(ar.ar_orthogonalize_workspace_bytes(count, rows, cols), ar.ar_clip_workspace_bytes()))
    grads = [matrices(20 + r, count, rows, cols, "bf16") for r in range(ranks)]
    grads = [[grads[r][t].contiguous() for r in range(ranks)] for t in range(count)]
    reduced = [[torch.empty_like(x) for x in row] for row in grads]
    mom = [torch.zeros(rows, cols, device="cuda") for _ in range(count)]
    first = [normal(gen(30 + t), rows, cols, std=0.1) for t in range(count)]
    weights = [[w.clone() for _ in range(ranks)] for w in first]
    norm = torch.zeros(1, device="cuda")

    def step(stream):
        ar.ar_all_reduce_clip(comm, grads, reduced, [rows * cols] * count, 0.01, norm, "bf16", "avg", stream=stream)
        ar.ar_muon_update(comm, [row[0] for row in reduced], mom, mom, [row[0] for row in weights], weights, rows, cols,
                          "bf16", "f32", weight_decay=0.1, stream=stream)

    def reset():
        for t in range(count):
            mom[t].zero_()
            for w in weights[t]:
                w.copy_(first[t])

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    reset()
    eager = []
    for _ in range(3):
        step(None)
        torch.cuda.synchronize()
        eager.append([w.clone() for row in weights for w in row] + [m.clone() for m in mom])
    reset()
    for want in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([w for row in weights for w in row] + mom, want))
        matrices(99, 1, 50, 60, "f32")  # the program's own work in between
    assert not torch.equal(weights[0][0], first[0])
