"""Log probabilities under a linear head, their entropy, alternatives and
gradients on a GPU against their definitions in 64 bits. Bounds count roundings,
as in test_gpu_lm.py, from which the inputs and helpers come."""
import math

import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_gpu_lm import (T, TINY, U, U32, close, comms, gen, loss_inputs, margins_untouched, nan_like,  # noqa: F401
                         normal, placed)

pytestmark = pytest.mark.gpu


def workspace(n, vocab, width, dtype, top=0):
    return max(ar.ar_linear_log_probs_workspace_bytes(n, vocab, width, dtype, top=top, backward=b) for b in (False, True))


def head_ref(x, w, y, ignore, scale):
    """Everything in 64 bits, and bounds of the fp32 results' errors."""
    n, width, vocab = x.shape[0], x.shape[1], w.shape[0]
    xd, wd = x.double(), w.double()
    r = {"z": scale * (xd @ wd.t())}
    # sums of products as in a cross entropy, and the rounding of the scale's product
    terms = width + 2 if x.dtype != torch.float32 else 6 * width + 16
    r["ez"] = scale * (xd.abs() @ wd.abs().t()) * terms * U32 + r["z"].abs() * U32
    yl = y.long()
    r["kept"] = (yl != ignore) & (yl >= 0) & (yl < vocab)
    r["at"] = yl.clamp(0, vocab - 1)[:, None]
    r["lse"] = torch.logsumexp(r["z"], 1)
    logp = r["z"] - r["lse"][:, None]
    p = torch.exp(logp)
    r["log_p"], r["p"] = logp, p
    r["lp"] = torch.where(r["kept"], logp.gather(1, r["at"])[:, 0], 0.0)
    r["entropy"] = -torch.where(p > 0, p * logp, 0.0).sum(1)
    top = r["z"].max(1).values
    span = top - r["z"].min(1).values
    ez = r["ez"].max(1).values
    own = (span * 4 + vocab + 32) * U32  # of a sum of exponentials, relative
    r["el"] = ez + own + r["lse"].abs() * 2 * U32
    r["elp"] = torch.where(r["kept"], r["el"] + r["ez"].gather(1, r["at"])[:, 0] + r["lp"].abs() * U32, 0.0)
    # H = log S + D, D = sum p (top - z): a change of z moves H by p |log p + H|
    # for each of them, at most 2 H in all; S and D are sums of one sign
    spread = (p * (top[:, None] - r["z"])).sum(1)
    r["eh"] = 2 * r["entropy"] * ez + own * (1 + 2 * spread) + (r["entropy"].abs() + spread) * 4 * U32 + 1e-300
    return r


def forward(comm, x, w, y, n, vocab, width, dtype, top=0, scale=1.0, ignore=5, entropy=True, **kw):
    out = {k: nan_like(n, dtype="f32") for k in ("log_probs", "entropy", "lse")}
    if not entropy:
        out["entropy"] = None
    out["top"] = nan_like(n, top, dtype="f32") if top else None
    out["ids"] = torch.full((n, top), -7, dtype=torch.int32, device="cuda") if top else None
    ar.ar_linear_log_probs(comm, x, w, y, out["log_probs"], out["entropy"], out["lse"], n, vocab, width, dtype, top=top,
                           top_log_probs=out["top"], top_ids=out["ids"], scale=scale, ignore_index=ignore, **kw)
    return out


def check_forward(got, r, rows=slice(None)):
    close(got["lse"][rows], r["lse"][rows], r["el"][rows], "lse")
    close(got["log_probs"], r["lp"], r["elp"] + 1e-300, "log_probs")
    close(got["entropy"][rows], r["entropy"][rows], r["eh"][rows], "entropy")


def check(comms, n, vocab, width, dtype, seed, scale=1.25, ignore=5, top=0, entropy=True, **kw):
    x, w, y, a = loss_inputs(n, vocab, width, dtype, seed, **kw)
    b = (torch.rand(n, generator=gen(seed + 100), device="cuda") - 0.7) * (3.0 / n) if entropy else None
    a = a - 0.4 / n
    comm = comms(1, workspace(n, vocab, width, dtype, top))
    r = head_ref(x, w, y, ignore, scale)
    kept, at = r["kept"], r["at"]
    x[~kept] = float("nan")  # an ignored row may hold anything
    got = forward(comm, x, w, y, n, vocab, width, dtype, top, scale, ignore)
    check_forward(got, r, kept)
    pitch, offset = kw.get("pitch", 0), kw.get("offset", 0)
    gx = placed(nan_like(n, width, dtype=dtype), offset, pitch and width + pitch)
    gw = placed(nan_like(vocab, width, dtype=dtype), offset, pitch and width + pitch)

    def backward(gx, gw):
        ar.ar_linear_log_probs_backward(comm, x, w, y, got["lse"], got["entropy"] if entropy else None, a, b, gx, gw, n,
                                        vocab, width, dtype, scale=scale, ignore_index=ignore)

    backward(gx, gw)
    ad, bd = a.double()[:, None] * kept[:, None], (b.double()[:, None] if entropy else 0.0) * kept[:, None]
    size = torch.maximum(ad.abs(), torch.as_tensor(bd, device="cuda").abs())  # d is held over this
    inner = r["log_p"] + r["entropy"][:, None]
    d = -r["p"] * (ad + bd * inner)
    d.scatter_add_(1, at, ad)
    ud = U[dtype] if dtype != "f32" else 4 * U32
    e = r["ez"] + r["el"][:, None]
    ed = (r["p"] * (abs(ad) * (e + 12 * U32) + abs(bd) * ((e + 12 * U32) * (1 + inner.abs()) + r["eh"][:, None])) * 1.01 +
          d.abs() * (ud + 8 * U32) + size * TINY[dtype] / 4096)
    # the target's d is a difference: its rounding counts from the sum's size
    ed.scatter_add_(1, at, ad.abs() * 4 * U32)
    d, ed = scale * d, scale * ed
    sums = (vocab if dtype != "f32" else 6 * vocab + 16) + 64
    wd = w.double().abs()
    ref = d @ w.double()
    close(gx, ref, ed @ wd + sums * U32 * (d.abs() @ wd) + ref.abs() * (U[dtype] + 4 * U32) + TINY[dtype], "grad_hidden")
    xz = torch.where(kept[:, None], x.double(), 0.0)
    sums = (n if dtype != "f32" else 6 * n + 16) + 64
    # the weight's copy of d is over the largest of all rows instead
    ew = ed + d.abs() * (ud + 8 * U32) + scale * float(size.max()) * TINY[dtype] / 4096
    ref = d.t().contiguous() @ xz
    bound = ew.t().contiguous() @ xz.abs() + sums * U32 * (d.abs().t().contiguous() @ xz.abs())
    close(gw, ref, bound + ref.abs() * (U[dtype] + 4 * U32) + TINY[dtype], "grad_weight")
    assert margins_untouched(gx) and margins_untouched(gw)
    for both in ((gx, None), (None, gw)):  # the same bits again, and each alone
        out = [None if t is None else torch.full_like(t, float("nan")) for t in both]
        backward(*out)
        assert all(s is None or torch.equal(s, t) for s, t in zip(out, both))


SHAPES = [(1, 1, 1), (1, 300, 64), (3, 257, 128), (16, 1000, 72), (17, 255, 64), (64, 2000, 320), (65, 513, 33),
          (255, 256, 64), (300, 3001, 192), (513, 777, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,vocab,width", SHAPES)
def test_values_and_gradients(comms, dtype, n, vocab, width):  # noqa: F811
    check(comms, n, vocab, width, dtype, 50)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,vocab,width", [(2, 300, 64), (70, 513, 33), (400, 20_000, 64)])
def test_without_entropy(comms, dtype, n, vocab, width):  # noqa: F811
    check(comms, n, vocab, width, dtype, 51, scale=0.5, entropy=False)


@pytest.mark.parametrize("dtype,pitch,offset", [("bf16", 8, 0), ("bf16", 3, 0), ("f16", 0, 1), ("f32", 5, 1), ("f16", 64, 8)])
def test_strided_rows(comms, dtype, pitch, offset):  # noqa: F811
    check(comms, 130, 700, 128, dtype, 52, pitch=pitch, offset=offset, index="i32", top=3)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,vocab,width,pitch,offset", [(1, 5, 8, 0, 0), (1, 3000, 513, 0, 1), (2, 700, 9, 3, 0), (4, 40_000, 64, 0, 0),
                                                        (5, 333, 1100, 0, 0), (8, 1999, 260, 5, 3), (9, 64, 2056, 0, 0),
                                                        (16, 9001, 77, 1, 0), (12, 31, 8, 8, 8)])
def test_few_tokens(comms, dtype, n, vocab, width, pitch, offset):  # noqa: F811
    """Both gradients in one pass over the weight, rows at any address."""
    check(comms, n, vocab, width, dtype, 55, pitch=pitch, offset=offset, ignored=0.3)


# widths whose tokens' rows just fit a workgroup's shared memory and do not, and no 16 bytes
@pytest.mark.parametrize("n,vocab,width,dtype,pitch", [(16, 130, 4543, "bf16", 0), (15, 67, 4609, "f16", 0),
                                                       (3, 64, 2271, "f32", 2), (2, 65, 2305, "f32", 0), (7, 200, 37, "f32", 1),
                                                       (1, 193, 31, "f16", 0), (13, 1, 517, "bf16", 0)])
def test_few_tokens_odd_rows(comms, n, vocab, width, dtype, pitch):  # noqa: F811
    check(comms, n, vocab, width, dtype, 56, pitch=pitch, top=min(vocab, 4), ignored=0.2)


@pytest.mark.parametrize("ignored", [0.0, 0.5, 1.0])
def test_ignored_tokens(comms, ignored):  # noqa: F811
    check(comms, 70, 400, 64, "bf16", 53, ignored=ignored, top=2)


@pytest.mark.parametrize("n,vocab,width,dtype", [(4096, 60_001, 64, "bf16"), (2000, 30_000, 96, "f32")])
def test_in_pieces(comms, n, vocab, width, dtype):  # noqa: F811
    """Sizes whose buffers take several pieces of the vocabulary."""
    check(comms, n, vocab, width, dtype, 54)


def test_no_tokens(comms):  # noqa: F811
    comm = comms(1, workspace(0, 300, 64, "bf16", 4))
    w = normal(gen(1), 300, 64, dtype="bf16")
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    ar.ar_linear_log_probs(comm, 0, w, t, 0, 0, 0, 0, 300, 64, "bf16", top=4, top_log_probs=0, top_ids=0)
    gw = nan_like(300, 64, dtype="bf16")
    ar.ar_linear_log_probs_backward(comm, 0, w, t, 0, 0, 0, 0, None, gw, 0, 300, 64, "bf16")
    assert (gw == 0).all()


# ---------------------------------------------------------------------------
# alternatives
# ---------------------------------------------------------------------------
def on_grid(n, vocab, width, dtype, seed, span=16):
    """Operands whose logits are whole numbers below 2^24: exact in fp32 in any
    order, with many equal ones."""
    g = gen(seed)
    x = torch.randint(-span, span + 1, (n, width), generator=g, device="cuda").to(T[dtype])
    w = torch.randint(-span, span + 1, (vocab, width), generator=g, device="cuda").to(T[dtype])
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    return x, w, y


def check_top(comms, n, vocab, width, dtype, top, scale=2.0 ** -7, seed=60, span=16):
    x, w, y = on_grid(n, vocab, width, dtype, seed, span)
    comm = comms(1, workspace(n, vocab, width, dtype, top))
    got = forward(comm, x, w, y, n, vocab, width, dtype, top, scale, -100)
    z = torch.cat([part.double() @ w.double().t() for part in x.split(512)]) * scale
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(got["ids"].long(), ids)
    lse = torch.logsumexp(z, 1)
    bound = ((z.max(1).values - z.min(1).values) * 4 + vocab + 32) * U32 + (lse.abs() + z.abs().max(1).values) * 2 * U32
    close(got["lse"], lse, bound, "lse")
    close(got["top"], z.gather(1, ids) - lse[:, None], bound[:, None] + 1e-300, "alternatives")
    close(got["log_probs"], z.gather(1, y[:, None])[:, 0] - lse, bound, "log_probs")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,vocab,width,top", [(1, 1, 8, 1), (1, 7, 8, 7), (2, 64, 40, 64), (5, 1000, 64, 20), (16, 4099, 72, 5),
                                               (17, 300, 64, 64), (64, 5000, 136, 8), (65, 513, 33, 3), (600, 3001, 72, 1),
                                               (600, 20_011, 64, 64), (515, 777, 264, 33)])
def test_alternatives(comms, dtype, n, vocab, width, top):  # noqa: F811
    check_top(comms, n, vocab, width, dtype, top)


@pytest.mark.parametrize("n", [3, 40, 700])
def test_equal_alternatives(comms, n):  # noqa: F811
    """Few distinct logits: the smallest ids of the equal ones."""
    check_top(comms, n, 6000, 8, "bf16", 64, scale=1.0, span=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alternatives_of_chunks(comms, dtype):  # noqa: F811
    """More tokens than their logits are kept of at a time (1 GiB: 3584 of 69,900)."""
    check_top(comms, 4000, 69_900, 64, dtype, 5)


def test_alternatives_of_many_groups(comms):  # noqa: F811
    """More groups than one pass of eight waves looks at, and of one wave."""
    check_top(comms, 3, 150_001, 16, "bf16", 20)
    check_top(comms, 520, 150_001, 16, "bf16", 20)


def test_alternatives_of_the_largest_vocabulary(comms):  # noqa: F811
    check_top(comms, 2, (1 << 24) - 1, 8, "bf16", 64)


def test_many_tokens_of_a_small_vocabulary(comms):  # noqa: F811
    check(comms, 70_001, 37, 16, "f16", 57, top=3)


@pytest.mark.parametrize("dtype,n", [("f32", 3), ("f32", 300), ("bf16", 3), ("f16", 700)])
def test_masked_rows(comms, dtype, n):  # noqa: F811
    """Rows of the vocabulary masked by -infinity: probability 0, no part in the
    entropy, and they come last, in the order of their ids, where they are
    needed to fill the alternatives."""
    vocab, width, top = 1000, 64, 12
    x, w, y = on_grid(n, vocab, width, dtype, 61)
    x[:, 0] = 1.0
    rest = torch.tensor([3, 500, 501, 999], device="cuda")
    open_rows = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    open_rows[rest] = True
    w[~open_rows, 0] = -math.inf
    y = rest[torch.arange(n, device="cuda") % 4]
    y[0] = 17  # a masked target
    comm = comms(1, workspace(n, vocab, width, dtype, top))
    scale = 2.0 ** -7
    got = forward(comm, x, w, y, n, vocab, width, dtype, top, scale, -100)
    z = x.double() @ w[rest].double().t() * scale
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    bound = 1000 * U32 * (1 + z.abs().max())
    assert float((got["lse"].double() - lse).abs().max()) <= bound
    assert float((got["entropy"].double() + (p * (z - lse[:, None])).sum(1)).abs().max()) <= 4 * bound
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    masked = torch.nonzero(~open_rows)[:top - 4, 0]
    assert torch.equal(got["ids"].long(), torch.cat([rest[order], masked.expand(n, -1)], 1))
    assert (got["top"][:, 4:] == -math.inf).all() and torch.isfinite(got["top"][:, :4]).all()
    assert float(got["log_probs"][0]) == -math.inf and torch.isfinite(got["log_probs"][1:]).all()
    a, b = torch.full((n,), 0.5, device="cuda"), torch.full((n,), 0.25, device="cuda")
    gx, gw = nan_like(n, width, dtype=dtype), nan_like(vocab, width, dtype=dtype)
    ar.ar_linear_log_probs_backward(comm, x, w, y, got["lse"], got["entropy"], a, b, None, gw, n, vocab, width, dtype,
                                    scale=scale)
    finite = open_rows.clone()
    finite[17] = True
    assert torch.isfinite(gw.float()).all() and (gw[~finite] == 0).all()


@pytest.mark.parametrize("n", [33, 700])
def test_numbers_that_are_none(comms, n):  # noqa: F811
    """A NaN or a +infinity makes its own token's results NaN and no other's."""
    vocab, width, top = 500, 64, 4
    x, w, y, _ = loss_inputs(n, vocab, width, "f16", 62, ignored=0.0)
    comm = comms(1, workspace(n, vocab, width, "f16", top))
    clean = forward(comm, x, w, y, n, vocab, width, "f16", top, ignore=-100)
    x[7, 3] = float("nan")
    x[9, 5] = float("inf")
    got = forward(comm, x, w, y, n, vocab, width, "f16", top, ignore=-100)
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[[7, 9]] = False
    for k in ("log_probs", "entropy", "lse", "top"):
        assert torch.isnan(got[k][~others]).all(), k
        assert torch.equal(got[k][others], clean[k][others]), k
    assert torch.equal(got["ids"][others], clean["ids"][others])
    assert ((got["ids"] >= 0) & (got["ids"] < vocab)).all()


@pytest.mark.parametrize("factor", [300.0, -300.0, 0.0])
def test_large_and_equal_logits(comms, factor):  # noqa: F811
    n, vocab, width = 40, 900, 64
    comm = comms(1, workspace(n, vocab, width, "bf16", 3))
    x, w, y, _ = loss_inputs(n, vocab, width, "bf16", 63, ignored=0.0)
    x = x * factor
    got = forward(comm, x, w, y, n, vocab, width, "bf16", 3, ignore=-100)
    check_forward(got, head_ref(x, w, y, -100, 1.0))
    if factor == 0.0:
        assert (got["ids"] == torch.arange(3, device="cuda")).all()


def test_it_is_the_cross_entropy(comms):  # noqa: F811
    """At scale 1 the log probability is the loss with its sign turned, without
    its entropy too, and so are the gradients but for the steps of d."""
    n, vocab, width = 300, 3001, 192
    x, w, y, gl = loss_inputs(n, vocab, width, "bf16", 64)
    comm = comms(1, max(workspace(n, vocab, width, "bf16"),
                        ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "bf16", backward=True)))
    got = forward(comm, x, w, y, n, vocab, width, "bf16", entropy=False)
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    ar.ar_linear_cross_entropy(comm, x, w, y, losses, lse, n, vocab, width, "bf16", ignore_index=5)
    r = head_ref(x, w, y, 5, 1.0)
    assert float(((got["log_probs"] + losses).abs().double() / (2 * r["elp"] + 1e-300))[r["kept"]].max()) <= 1
    assert (got["log_probs"][~r["kept"]] == 0).all()


def test_gradients_by_differences(comms):  # noqa: F811
    """Central differences of sum a lp + b H along random directions, as for the loss."""
    n, vocab, width, scale = 12, 150, 20, 1.5
    comm = comms(1, workspace(n, vocab, width, "f32"))
    x, w, y, a = loss_inputs(n, vocab, width, "f32", 65, ignored=0.2)
    g = gen(66)
    b = torch.rand(n, generator=g, device="cuda") / n
    kept = (y != 5) & (y >= 0) & (y < vocab)

    def total(xx, ww):
        got = forward(comm, xx, ww, y, n, vocab, width, "f32", scale=scale)
        return float((got["log_probs"].double() * a + got["entropy"].double() * b * kept).sum()), got

    h = 2.0 ** -6
    _, base = total(x, w)
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    ar.ar_linear_log_probs_backward(comm, x, w, y, base["lse"], base["entropy"], a, b, gx, gw, n, vocab, width, "f32",
                                    scale=scale, ignore_index=5)
    size = float(base["log_probs"].abs().sum() + base["lse"].abs().sum() + base["entropy"].sum())
    for _ in range(3):
        ex, ew = normal(g, n, width) / math.sqrt(width), normal(g, vocab, width) / width
        up, down = total(x + h * ex, w + h * ew)[0], total(x - h * ex, w - h * ew)[0]
        left = float((gx.double() * ex.double()).sum() + (gw.double() * ew.double()).sum())
        dz = scale * float(((ex.double() @ w.double().t()).abs() + (x.double() @ ew.double().t()).abs()).max()) + 1
        # third derivatives: of lp at most dz^3, of H at most (3 + |log p| + H) dz^3 < 20 dz^3
        truncation = float((a.abs() + 20 * b).sum()) * h * h * dz ** 3
        rounding = float((a.abs() + b).max()) * size * 1200 * U32 / h
        assert abs((up - down) / (2 * h) - left) <= truncation + rounding


@pytest.mark.parametrize("tiny", [0.0, 2.0 ** -130, 2.0 ** -140])
def test_gradients_of_nothing_and_almost_nothing(comms, tiny):  # noqa: F811
    """Zero gradients give zeros; subnormal ones beside ordinary ones no NaN."""
    n, vocab, width = 40, 300, 64
    x, w, y, a = loss_inputs(n, vocab, width, "bf16", 67, ignored=0.0)
    comm = comms(1, workspace(n, vocab, width, "bf16"))
    got = forward(comm, x, w, y, n, vocab, width, "bf16", ignore=-100)
    b = a.clone()
    a[::2], b[::2] = tiny, -tiny
    gx, gw = nan_like(n, width, dtype="bf16"), nan_like(vocab, width, dtype="bf16")
    ar.ar_linear_log_probs_backward(comm, x, w, y, got["lse"], got["entropy"], a, b, gx, gw, n, vocab, width, "bf16")
    assert torch.isfinite(gx.float()).all() and torch.isfinite(gw.float()).all()
    if tiny == 0.0:
        assert (gx[::2] == 0).all() and (gx[1::2] != 0).any()


@pytest.mark.parametrize("n", [6, 40])
def test_gradients_of_ignored_tokens_may_be_anything(comms, n):  # noqa: F811
    vocab, width = 300, 72
    x, w, y, a = loss_inputs(n, vocab, width, "bf16", 69, ignored=0.5)
    y[0] = 5
    kept = (y != 5) & (y >= 0) & (y < vocab)
    comm = comms(1, workspace(n, vocab, width, "bf16"))
    got = forward(comm, x, w, y, n, vocab, width, "bf16")
    b = 0.5 * a

    def backward():
        gx, gw = nan_like(n, width, dtype="bf16"), nan_like(vocab, width, dtype="bf16")
        ar.ar_linear_log_probs_backward(comm, x, w, y, got["lse"], got["entropy"], a, b, gx, gw, n, vocab, width, "bf16",
                                        ignore_index=5)
        return gx, gw

    want = backward()
    assert (want[0][~kept] == 0).all() and torch.isfinite(want[1].float()).all()
    a[~kept], b[~kept] = float("nan"), float("inf")
    got["lse"][~kept], got["entropy"][~kept] = float("nan"), float("inf")
    assert all(torch.equal(s, t) for s, t in zip(backward(), want))


def test_rows_past_32_bits(comms):  # noqa: F811
    """Rows of the weight and of its gradient whose offsets pass 2^32 bytes, on 16
    bytes and not, of few tokens and of many."""
    vocab, width, step = 2305, 40, 1 << 20
    base, grad = (torch.empty(vocab * step, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for n, offset, pitch in ((3, 0, step), (2, 1, step - 1), (40, 0, step), (40, 1, step - 1)):
        w = base.as_strided((vocab, width), (pitch, 1), offset)
        gw = grad.as_strided((vocab, width), (pitch, 1), offset)
        x, w0, y, a = loss_inputs(n, vocab, width, "bf16", 74, ignored=0.0)
        w.copy_(w0)
        comm = comms(1, workspace(n, vocab, width, "bf16", 4))
        near, far = (forward(comm, x, m, y, n, vocab, width, "bf16", 4, ignore=-100) for m in (w0, w))
        check_forward(far, head_ref(x, w0, y, -100, 1.0))
        assert torch.equal(near["ids"], far["ids"])
        gx, want = nan_like(n, width, dtype="bf16"), nan_like(vocab, width, dtype="bf16")
        for m, out in ((w0, want), (w, gw)):
            ar.ar_linear_log_probs_backward(comm, x, m, y, near["lse"], near["entropy"], a, a, gx, out, n, vocab, width, "bf16")
        # sums of other orders: one rounding of the logits apart, twice
        scale = want.double().abs().max()
        assert float((gw.double() - want.double()).abs().max()) <= float(scale) * 2 * U["bf16"]


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,vocab,width,top", [(600, 900, 64, 5), (4, 5000, 100, 20), (9, 700, 77, 0)])
def test_on_another_stream_and_in_a_graph(comms, n, vocab, width, top):  # noqa: F811
    """A policy-gradient step captured and replayed between eager work, each
    replay against the eager result on the same inputs."""
    comm = comms(1, workspace(n, vocab, width, "bf16", top))
    x, w, y, a = loss_inputs(n, vocab, width, "bf16", 68)
    b = torch.full((n,), -0.01 / n, device="cuda")
    out = {k: nan_like(n, dtype="f32") for k in ("log_probs", "entropy", "lse")}
    out |= {"top": nan_like(n, max(top, 1), dtype="f32"), "ids": torch.zeros(n, max(top, 1), dtype=torch.int32, device="cuda"),
            "gx": torch.empty_like(x), "gw": torch.empty_like(w)}

    def step(stream):
        ar.ar_linear_log_probs(comm, x, w, y, out["log_probs"], out["entropy"], out["lse"], n, vocab, width, "bf16",
                               top=top, top_log_probs=out["top"], top_ids=out["ids"], stream=stream)
        ar.ar_linear_log_probs_backward(comm, x, w, y, out["lse"], out["entropy"], a, b, out["gx"], out["gw"], n, vocab,
                                        width, "bf16", stream=stream)

    def fill(seed):
        x.copy_(normal(gen(seed), n, width, dtype="bf16"))
        for t in out.values():
            t.fill_(-3)

    side = torch.cuda.Stream()
    fill(70)
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    for seed in (71, 72, 73):
        fill(seed)
        step(None)
        torch.cuda.synchronize()
        eager = {k: t.clone() for k, t in out.items()}
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        for k, t in out.items():
            assert torch.equal(t, eager[k]), k
