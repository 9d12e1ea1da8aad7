"""The language-model operators at sizes that take another way through the
kernels: tiles for few tokens, depths that end inside a step, several sort
passes and rounds, long runs of one token, matrices beyond 2^32 bytes."""
import math

import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_gpu_lm import (TINY, U, U32, check_loss, close, clip_bound, comms, embedding_grad_ref,  # noqa: F401
                         gen, loss_inputs, loss_ref, nan_like, normal, placed, margins_untouched)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# cross entropy
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,vocab,width", [
    (3, 66_000, 64),    # 16-token tiles of 256 vocabulary rows: as many as CUs
    (40, 66_000, 40),   # 64-token tiles, a depth below one step
    (1, 4097, 8), (16, 4096, 264), (17, 300, 1032), (64, 5000, 136),  # tiles of 64 rows, ends inside a step
    (130, 515, 8), (257, 1025, 1016),  # large tiles with one row or column over
    (1, 1, 4), (2, 2, 1),
])
def test_loss_of_other_shapes(comms, dtype, n, vocab, width):  # noqa: F811
    check_loss(comms, n, vocab, width, dtype, 50)


@pytest.mark.parametrize("dtype,n,vocab,width", [("bf16", 300, 600, 200), ("f16", 10, 600, 200), ("f32", 10, 600, 200)])
def test_depth_ends_before_what_lies_behind(comms, dtype, n, vocab, width):  # noqa: F811
    """Rows that are read as they lie, with NaN between them (see `placed`)."""
    check_loss(comms, n, vocab, width, dtype, 51, pitch=16, offset=8)


@pytest.mark.parametrize("n", [20, 100])
def test_losses_do_not_depend_on_other_tokens(comms, n):  # noqa: F811
    """The same bits for a token whatever the others are."""
    vocab, width = 2000, 128
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "bf16"))
    x, w, y, _ = loss_inputs(n, vocab, width, "bf16", 52, ignored=0.0)
    a, b, lse = (nan_like(n, dtype="f32") for _ in range(3))
    ar.ar_linear_cross_entropy(comm, x, w, y, a, lse, n, vocab, width, "bf16")
    x[::2] = float("nan")
    ar.ar_linear_cross_entropy(comm, x, w, y, b, lse, n, vocab, width, "bf16")
    assert torch.equal(a[1::2], b[1::2]) and torch.isnan(b[::2]).all()


@pytest.mark.parametrize("n", [20, 100])
@pytest.mark.parametrize("least", [0.0, 2.0 ** -130])
def test_loss_gradients_below_the_normal_numbers(comms, n, least):  # noqa: F811
    """Gradients of the losses that are subnormal, or all zero: their reciprocal
    has no part in the result. A subnormal is off by half of the least, 2^-150."""
    vocab, width = 500, 64
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "f32", backward=True))
    x, w, y, gl = loss_inputs(n, vocab, width, "f32", 57)
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    ar.ar_linear_cross_entropy(comm, x, w, y, losses, lse, n, vocab, width, "f32")
    one, small = ([nan_like(n, width, dtype="f32"), nan_like(vocab, width, dtype="f32")] for _ in range(2))
    gl = torch.full_like(gl, 1.0)
    ar.ar_linear_cross_entropy_backward(comm, x, w, y, lse, gl, *one, n, vocab, width, "f32")
    ar.ar_linear_cross_entropy_backward(comm, x, w, y, lse, gl * least, *small, n, vocab, width, "f32")
    for a, b in zip(one, small):
        # the scale of the smaller ones, g 2^-14, is itself rounded to a subnormal
        close(b, a.double() * least, a.double().abs() * 2.0 ** -149 + 2.0 ** -148)


@pytest.mark.parametrize("n,dtype", [(4, "bf16"), (70, "f16")])
def test_loss_of_a_weight_beyond_4_gib(comms, n, dtype):  # noqa: F811
    vocab, width = 300_000, 8192
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, dtype))
    g = gen(53)
    x = normal(g, n, width, dtype=dtype)
    w = torch.empty(vocab, width, dtype=x.dtype, device="cuda")
    z, mag = [], []
    xd = x.double()
    for lo in range(0, vocab, 50_000):
        part = w[lo:lo + 50_000]
        part.copy_(normal(g, part.shape[0], width, std=2.0 / math.sqrt(width)))
        z.append(xd @ part.double().t())
        mag.append(xd.abs() @ part.double().abs().t())
    z, mag = torch.cat(z, 1), torch.cat(mag, 1)
    y = torch.randint(vocab - 1000, vocab, (n,), generator=g, device="cuda")
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    ar.ar_linear_cross_entropy(comm, x, w, y, losses, lse, n, vocab, width, dtype)
    # as loss_ref: sums of `width` products, then of the vocabulary's exponentials
    ez = mag * ((width + 2) * U32)
    ref = torch.logsumexp(z, 1)
    span = z.max(1).values - z.min(1).values
    el = ez.max(1).values + (span * 4 + vocab + 32) * U32 + ref.abs() * 2 * U32
    close(lse, ref, el)
    at = y[:, None]
    loss = ref - z.gather(1, at)[:, 0]
    close(losses, loss, el + ez.gather(1, at)[:, 0] + loss.abs() * U32)


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,rows,width,dtype,grad_dtype", [
    (200_000, 70_000, 8, "bf16", "f32"),    # two rounds a workgroup, two passes
    (30_000, 300_000, 12, "f16", "f16"),    # three passes
    (3000, 511, 40, "f32", "f32"), (3000, 512, 40, "f32", "f32"),  # one pass, and the first size with two
    (70_000, 3, 64, "bf16", "bf16"),        # runs over hundreds of chunks
    (5000, 90_000, 1001, "bf16", "f32"),    # more than the last-level cache of zeros, at odd addresses
])
def test_embedding_grad_of_other_shapes(comms, n, rows, width, dtype, grad_dtype):  # noqa: F811
    comm = comms(1, ar.ar_embedding_workspace_bytes(n, rows, width))
    g = gen(54)
    t = (torch.rand(n, generator=g, device="cuda") ** 3 * rows).long().clamp_(max=rows - 1)
    dout = normal(g, n, width, dtype=dtype)
    ref, mags, most = embedding_grad_ref(t, dout, rows, 0, 0.5)
    dw = placed(nan_like(rows, width, dtype=grad_dtype), 1, 0)
    ar.ar_embedding_backward(comm, dout, t, dw, n, rows, width, dtype, grad_dtype, scale=0.5)
    close(dw, ref, mags * ((most + 2) * U32) + ref.abs() * U[grad_dtype] + TINY[grad_dtype])
    assert margins_untouched(dw)
    again = placed(nan_like(rows, width, dtype=grad_dtype), 1, 0)
    ar.ar_embedding_backward(comm, dout, t, again, n, rows, width, dtype, grad_dtype, scale=0.5)
    assert torch.equal(again, dw)


def test_embedding_beyond_4_gib(comms):  # noqa: F811
    rows, width, n = 600_000, 4096, 300
    comm = comms(1, ar.ar_embedding_workspace_bytes(n, rows, width))
    g = gen(55)
    w = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    t = torch.randint(rows - 1000, rows, (n,), generator=g, device="cuda")
    t[::3] = torch.randint(0, 1000, (len(t[::3]),), generator=g, device="cuda")
    w[t] = normal(g, n, width, dtype="bf16")
    out = nan_like(n, width, dtype="bf16")
    ar.ar_embedding(comm, w, t, out, n, rows, width, "bf16")
    assert torch.equal(out, w[t])
    w.fill_(float("nan"))
    ar.ar_embedding_backward(comm, out, t, w, n, rows, width, "bf16")
    met = torch.zeros(rows, dtype=torch.bool, device="cuda")
    met[t] = True
    assert all(not part[~m].any() for part, m in zip(w.split(50_000), met.split(50_000)))
    at, where = torch.unique(t, return_inverse=True)
    ref, mags = (torch.zeros(len(at), width, dtype=torch.float64, device="cuda") for _ in range(2))
    ref.index_add_(0, where, out.double())
    mags.index_add_(0, where, out.double().abs())
    close(w[at], ref, mags * (n * U32) + ref.abs() * U["bf16"])


# ---------------------------------------------------------------------------
# clip
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("total", [255 * 4096, 256 * 4096, 257 * 4096, 9000 * 4096 + 5])
def test_clip_around_the_number_of_partials(comms, total):  # noqa: F811
    """Partial norms that each workgroup joins, that one launch joins, and more
    tiles than partials."""
    comm = comms(1)
    x = normal(gen(56), total)
    y, out = nan_like(total, dtype="f32"), nan_like(1, dtype="f32")
    ref = float(torch.linalg.vector_norm(x.double()))
    for call in ("clip", "reduce"):
        y.fill_(float("nan"))
        if call == "clip":
            ar.ar_clip_grads(comm, [[x]], [[y]], [total], 1.0, out, "f32")
        else:
            ar.ar_all_reduce_clip(comm, [[x]], [[y]], [total], 1.0, out, "f32")
        assert abs(float(out) - ref) <= ref * (U32 + 1e-12)
        close(y, x.double() / (ref + 1e-6), clip_bound(x.double() / (ref + 1e-6), "f32"))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,vocab,width", [(4200, 300, 72), (2500, 700, 130), (6, 70_000, 40), (700, 6000, 136)])
def test_loss_with_split_sums(comms, dtype, n, vocab, width):  # noqa: F811
    """Gradients whose few tiles are summed in parts, along the tokens or the
    vocabulary, in either order of the operands."""
    check_loss(comms, n, vocab, width, dtype, 58)


def test_loss_of_more_tiles_than_a_launch_counts(comms):  # noqa: F811
    """2^20 tokens over 600 000 rows: 9.6 million tiles of 512 threads. A
    sample of the tokens against 64 bits, all of them against each other: tokens
    with equal rows have equal results."""
    n, vocab, width, kinds = 1 << 20, 600_000, 8, 64
    try:
        comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "bf16"))
    except torch.cuda.OutOfMemoryError:
        pytest.skip("needs about 40 GB of workspace")
    g = gen(59)
    x = normal(g, kinds, width, dtype="bf16").repeat(n // kinds, 1)
    w = normal(g, vocab, width, dtype="bf16")
    y = torch.randint(0, vocab, (kinds,), generator=g, device="cuda").repeat(n // kinds)
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    ar.ar_linear_cross_entropy(comm, x, w, y, losses, lse, n, vocab, width, "bf16")
    z, ez, rl, el, rloss, eloss, kept, at = loss_ref(x[:kinds], w, y[:kinds], -100)
    close(lse[:kinds], rl, el)
    close(losses[:kinds], rloss, eloss)
    assert torch.equal(losses, losses[:kinds].repeat(n // kinds)) and torch.equal(lse, lse[:kinds].repeat(n // kinds))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wide_rows(comms, dtype):  # noqa: F811
    """Widths beyond 65535 blocks of a launch's second dimension."""
    width = 4_200_072
    check_loss(comms, 3, 20, 262_144 + 8, dtype, 60)
    comm = comms(1, ar.ar_embedding_workspace_bytes(40, 6, width))
    t = torch.randint(0, 6, (40,), generator=gen(61), device="cuda")
    dout = normal(gen(62), 40, width, dtype=dtype)
    ref, mags, most = embedding_grad_ref(t, dout, 6, 0, 1.0)
    dw = nan_like(6, width, dtype=dtype)
    ar.ar_embedding_backward(comm, dout, t, dw, 40, 6, width, dtype)
    close(dw, ref, mags * ((most + 2) * U32) + ref.abs() * U[dtype] + TINY[dtype])
