"""The language-model operators where numbers reach their type's limits, against
64 bits: what a mask holds, infinities, the largest finite numbers."""
import math

import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_gpu_lm import (T, TINY, U, U32, close, comms, gen, loss_inputs, loss_ref, nan_like, normal)  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# cross entropy
# ---------------------------------------------------------------------------
SIZES = [("f32", 700, 6000, 136),  # fp32 in bf16 pieces
         ("f32", 70, 500, 72), ("f32", 9, 6000, 40),  # fp32 matrix instructions
         ("bf16", 300, 3000, 136), ("f16", 300, 3000, 136), ("bf16", 9, 6000, 40)]


@pytest.mark.parametrize("dtype,n,vocab,width", SIZES)
@pytest.mark.parametrize("mask,bias", [("min", 1.0), ("min", 0.7), ("min", 300.7), ("min", 0.0), ("inf", 1.0), ("inf", 0.7),
                                       ("inf", 300.7), ("far", 1.1)])
def test_rows_masked_through_a_column(comms, dtype, n, vocab, width, mask, bias):  # noqa: F811
    """Every seventh row of the vocabulary has the type's lowest number, -infinity
    or a very low number in its last column, other rows zero; the hidden rows'
    last column is `bias`. Masked rows have the probability 0, and all results are
    those of the other rows alone (where the bias is 0, of all rows without the
    last column). Bounds as in check_loss."""
    x, w, y, gl = loss_inputs(n, vocab, width - 1, dtype, 70, ignored=0.1)
    lowest = {"min": torch.finfo(T[dtype]).min, "inf": -math.inf, "far": -1.3e30 if dtype != "f16" else -6e4}[mask]
    masked = torch.arange(vocab, device="cuda") % 7 == 3
    on = bias != 0.0
    if on:  # a target is no masked row
        y = torch.where((y >= 0) & (y % 7 == 3), y - 1, y)
    bias *= 1e30 if mask == "far" and dtype != "f16" else 1.0
    xm = torch.cat([x, torch.full((n, 1), bias, device="cuda").to(x.dtype)], 1)
    wm = torch.cat([w, torch.where(masked, lowest, 0.0)[:, None].to(w.dtype)], 1)
    need = max(ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, dtype, backward=b) for b in (False, True))
    comm = comms(1, need)
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    ar.ar_linear_cross_entropy(comm, xm, wm, y, losses, lse, n, vocab, width, dtype)
    rows = torch.nonzero(~masked)[:, 0] if on else torch.arange(vocab, device="cuda")
    where = torch.full((vocab,), -1, device="cuda")
    where[rows] = torch.arange(len(rows), device="cuda")
    kept = (y != -100) & (y >= 0) & (y < vocab)
    yr = torch.where(kept, where[y.clamp(0, vocab - 1)], -100)
    z, ez, rl, el, rloss, eloss, kept, at = loss_ref(x, w[rows], yr, -100)
    close(lse, rl, el, "lse")
    close(losses, rloss, eloss + 1e-300, "losses")
    gx, gw = nan_like(n, width, dtype=dtype), nan_like(vocab, width, dtype=dtype)
    ar.ar_linear_cross_entropy_backward(comm, xm, wm, y, lse, gl, gx, gw, n, vocab, width, dtype)
    d = torch.exp(z - rl[:, None])
    p = d.clone()
    d.scatter_add_(1, at, torch.full_like(d[:, :1], -1.0))
    d *= kept[:, None]
    ud = U[dtype] if dtype != "f32" else 4 * U32
    ed = (p * (ez + el[:, None] + 8 * U32) * 1.01 + d.abs() * (ud + 4 * U32) + TINY[dtype] / 16384) * kept[:, None]
    wd, gd = w[rows].double(), gl.double()[:, None]
    terms = (vocab if dtype != "f32" else 6 * vocab + 16) + 64
    ref = gd * (d @ wd)
    bound = gd * (ed @ wd.abs() + terms * U32 * (d.abs() @ wd.abs())) + ref.abs() * (U[dtype] + 4 * U32) + TINY[dtype]
    close(gx[:, :-1], ref, bound, "grad_hidden")
    if on and mask != "inf":  # 0 times the lowest number, and d times 0
        assert (gx[:, -1] == 0).all()
    terms = (n if dtype != "f32" else 6 * n + 16) + 64
    xd = xm[:, :-1].double()
    top = float((gd[:, 0] * kept).max())
    ew = gd * ed + (gd * d.abs()) * (ud + 4 * U32) + top * TINY[dtype] / 16384
    ref = (gd * d).t().contiguous() @ xd
    bound = ew.t().contiguous() @ xd.abs() + terms * U32 * ((gd * d.abs()).t().contiguous() @ xd.abs())
    close(gw[rows][:, :-1], ref, bound + ref.abs() * (U[dtype] + 4 * U32) + TINY[dtype], "grad_weight")
    if on:
        assert (gw[masked] == 0).all()


@pytest.mark.parametrize("dtype,n,vocab,width", SIZES)
def test_rows_of_minus_infinity(comms, dtype, n, vocab, width):  # noqa: F811
    """Logits that are all -infinity have the logsumexp -infinity, and infinite
    products of both signs or with a zero are no number; other tokens keep
    their bits."""
    x, w, y, _ = loss_inputs(n, vocab, width, dtype, 71, ignored=0.0)
    w[:, 3] = w[:, 3].abs() + 0.01
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, dtype))
    a, b, lse, lse_b = (nan_like(n, dtype="f32") for _ in range(4))
    ar.ar_linear_cross_entropy(comm, x, w, y, a, lse, n, vocab, width, dtype)
    x[2, 3] = -math.inf
    x[5, 4] = math.inf
    x[7, 3] = math.nan
    ar.ar_linear_cross_entropy(comm, x, w, y, b, lse_b, n, vocab, width, dtype)
    assert float(lse_b[2]) == -math.inf and not torch.isfinite(b[[2, 5, 7]]).any()
    same = torch.ones(n, dtype=torch.bool, device="cuda")
    same[[2, 5, 7]] = False
    assert torch.equal(a[same], b[same]) and torch.equal(lse[same], lse_b[same])


@pytest.mark.parametrize("n,vocab", [(700, 6000), (40, 300)])
def test_products_of_large_fp32_numbers(comms, n, vocab):  # noqa: F811
    """Each logit is one product, of numbers around 2^e and 2^-e for e from -60 to
    60: one of them is cut to its pieces rather than rounded, and the terms left out
    are within loss_ref's 2^-21 of each product."""
    width = 40
    g = gen(72)
    e = torch.randint(-60, 61, (width,), generator=g, device="cuda").double()
    column = torch.arange(n, device="cuda") % width
    x = torch.zeros(n, width, device="cuda")
    x[torch.arange(n, device="cuda"), column] = ((1 + torch.rand(n, generator=g, device="cuda")) * 2.0 ** e[column]).float()
    size = torch.randint(-3, 3, (vocab, width), generator=g, device="cuda").double() - e
    w = ((1 + torch.rand(vocab, width, generator=g, device="cuda")) * 2.0 ** size).float()
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "f32"))
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    ar.ar_linear_cross_entropy(comm, x, w, y, losses, lse, n, vocab, width, "f32")
    z, ez, rl, el, rloss, eloss, kept, at = loss_ref(x, w, y, -100)
    close(lse, rl, el, "lse")
    close(losses, rloss, eloss, "losses")


# ---------------------------------------------------------------------------
# clip
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("norm", ["l2", "inf"])
@pytest.mark.parametrize("size", [1000, 2_000_001])  # partial norms joined by every workgroup, and by a launch
def test_no_limit_clips_nothing(comms, dtype, norm, size):  # noqa: F811
    """An infinite max_norm leaves every element as it is, whatever the norm; of a
    NaN norm it is NaN as by any limit."""
    comm = comms(2)
    out = torch.zeros(1, device="cuda")
    for value in (1.0, math.inf, -math.inf, math.nan):
        x = [[normal(gen(73), size, dtype=dtype) for _ in range(2)]]
        x[0][1][77] = value
        for call in ("sharded", "replicated", "reduce"):
            y = [[nan_like(size, dtype=dtype) for _ in range(2)]]
            if call == "reduce":
                want = [[nan_like(size, dtype=dtype) for _ in range(2)]]
                ar.ar_all_reduce_multi(comm, x, want, [size], dtype, "sum")
                ar.ar_all_reduce_clip(comm, x, y, [size], math.inf, out, dtype, "sum", norm)
            else:
                want = x if call == "sharded" else [[x[0][0], x[0][0]]]
                ar.ar_clip_grads(comm, x, y, [size], math.inf, out, dtype, call, norm)
            for a, b in zip(y[0], want[0]):
                if math.isnan(value) and call != "replicated":
                    assert torch.isnan(a).all() and torch.isnan(out).all()
                else:
                    assert torch.equal(a, b)
                    assert math.isinf(float(out)) == (math.isinf(value) and call != "replicated")


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,rows,width", [(9, 1, (1 << 31) - 1),     # sorted by one workgroup
                                          (1025, 5, 33_500_001)])
def test_embedding_grad_of_more_blocks_than_a_launch_counts(comms, n, rows, width):  # noqa: F811
    """2^24 workgroups of 256 threads and more, which are 2^32 work-items. Whole
    numbers, so that every sum is exact."""
    try:
        comm = comms(1, ar.ar_embedding_workspace_bytes(n, rows, width))
        dout = torch.empty(n, width, dtype=torch.bfloat16, device="cuda")
        dw = torch.full((rows, width), math.nan, device="cuda")
        column = (torch.arange(width, dtype=torch.int32, device="cuda") % 97).to(torch.bfloat16)
    except torch.cuda.OutOfMemoryError:
        pytest.skip("needs about 110 GB")
    for t in range(n):
        torch.add(column, float(t % 7), out=dout[t])
    tokens = torch.arange(n, device="cuda") % rows
    ar.ar_embedding_backward(comm, dout, tokens, dw, n, rows, width, "bf16", "f32")
    for r in range(rows):
        mine = range(r, n, rows)
        want = float(sum(t % 7 for t in mine))
        for lo in range(0, width, 1 << 27):
            part = column[lo:lo + (1 << 27)].float() * len(mine) + want
            assert torch.equal(dw[r, lo:lo + (1 << 27)], part), (r, lo)
