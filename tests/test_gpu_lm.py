"""The language-model operators on a GPU against their definitions in 64 bits.

Tolerances count roundings: u(t) = eps/2 of a type is the largest relative
error of one rounding, and a sum of k fp32 products in any order is off by at
most k * 2^-24 times the sum of their magnitudes. Outputs start as NaN bits, so
an element that is never written shows.
"""
import math

import pytest
import torch

import ring_all_reduce_ar_amd as ar

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {k: torch.finfo(t).eps / 2 for k, t in T.items()}
TINY = {k: torch.finfo(t).smallest_normal * torch.finfo(t).eps for k, t in T.items()}  # the least subnormal
U32 = 2.0 ** -24
ITYPE = {"i32": torch.int32, "i64": torch.int64}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(T[dtype])


def nan_like(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=T[dtype], device="cuda")


def placed(x, offset=0, pitch=0):
    """A copy of `x` whose storage starts `offset` elements past an aligned
    address and whose rows are `pitch` apart (0: dense); what lies between is NaN."""
    rows, cols = (1, x.numel()) if x.dim() == 1 else x.shape
    pitch = pitch or cols
    raw = torch.full((offset + rows * pitch + 64,), float("nan"), dtype=x.dtype, device="cuda")
    view = raw[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
    view.copy_(x.view(rows, cols))
    view = view.view(-1) if x.dim() == 1 else view
    view.raw = raw
    return view


def margins_untouched(view):
    """Nothing outside the view's elements was written (they were NaN)."""
    raw = view.raw.clone()
    flat = raw.as_strided(view.shape, view.stride(), view.storage_offset())
    flat.fill_(float("nan"))
    return bool(torch.isnan(raw.float()).all())


def close(got, ref, bound, what=""):
    got = got.double()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - ref).abs() / bound.clamp_min(1e-300)).max()):.3g} times the bound")


@pytest.fixture(scope="module")
def comms():
    made = {}

    def get(nranks, need=1 << 20):
        if nranks not in made:
            made[nranks] = [ar.Comm(nranks, 0), None]
        c = made[nranks]
        if c[1] is None or c[1].numel() < need:
            c[1] = torch.empty(need, dtype=torch.uint8, device="cuda")
            ar.ar_comm_set_workspace(c[0], c[1])
        c[1].fill_(0xFF)  # nothing may rely on what the workspace holds
        return c[0]

    yield get
    torch.cuda.synchronize()
    for c, _ in made.values():
        c.close()


# ---------------------------------------------------------------------------
# gradient norm and clip
# ---------------------------------------------------------------------------
SIZES = {
    "one": [1],
    "small": [1, 2, 7, 8, 9, 63, 64, 65, 255, 256, 257, 1000],
    "gaps": [0, 5, 0, 4096, 3, 0],
    "tiles": [4095, 4096, 4097, 16_384, 100_003, 40_000],
    "many": [1 + (37 * i) % 211 for i in range(700)],
}


def gradients(g, sizes, ranks, dtype, offset, std=1e-2):
    return [[placed(normal(g, s, dtype=dtype, std=std), (offset + 3 * r if offset else 0)) for r in range(ranks)]
            for s in sizes]


def norm_of(tensors, kind):
    x = torch.cat([t.double().reshape(-1) for t in tensors])
    if x.numel() == 0:
        return 0.0
    return float(x.square().sum().sqrt() if kind == "l2" else x.abs().max())


def clip_bound(ref, dtype):
    # the factor's rounding to fp32, the product's, and the result's
    return ref.abs() * (2 * U32 + U[dtype] + 1e-10) + TINY[dtype] / 2


@pytest.mark.parametrize("layout", ["replicated", "sharded"])
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("dtype,offset,norm", [("f32", 0, "l2"), ("bf16", 0, "l2"), ("f16", 1, "l2"), ("f32", 3, "inf"),
                                              ("bf16", 0, "inf")])
def test_clip(comms, layout, sizes, dtype, offset, norm):
    ranks = 3
    counts = SIZES[sizes]
    comm = comms(ranks)
    send = gradients(gen(1), counts, ranks, dtype, offset)
    if layout == "replicated":
        for row in send:
            for t in row[1:]:
                t.copy_(row[0])
    total = norm_of([row[r] for row in send for r in range(1 if layout == "replicated" else ranks)], norm)
    out = torch.full((1,), float("nan"), device="cuda")
    ar.ar_grad_norm(comm, send, counts, out, dtype, layout, norm)
    assert abs(float(out) - total) <= total * (U32 + 1e-12)
    for max_norm in (total / 3, 2 * total, 0.0):
        scale = min(1.0, max_norm / (total + 1e-6))
        recv = [[placed(nan_like(s, dtype=dtype), 0 if not offset else offset + 1) for _ in range(ranks)] for s in counts]
        out.fill_(float("nan"))
        ar.ar_clip_grads(comm, send, recv, counts, max_norm, out, dtype, layout, norm)
        assert abs(float(out) - total) <= total * (U32 + 1e-12)
        for s, d in zip(send, recv):
            for r in range(ranks):
                ref = s[0 if layout == "replicated" else r].double() * scale
                close(d[r], ref, clip_bound(ref, dtype))
                assert margins_untouched(d[r])
    # in place, the same bits
    ar.ar_clip_grads(comm, send, recv, counts, total / 3, None, dtype, layout, norm)
    ar.ar_clip_grads(comm, send, send, counts, total / 3, out, dtype, layout, norm)
    for s, d in zip(send, recv):
        assert all(torch.equal(a, b) for a, b in zip(s, d))


@pytest.mark.parametrize("ranks", [1, 2, 3, 5, 8, 9, 16, 64])
@pytest.mark.parametrize("dtype,op,sizes,offset", [("f32", "avg", "tiles", 0), ("bf16", "sum", "small", 1),
                                                   ("f16", "avg", "gaps", 0), ("bf16", "avg", "many", 0),
                                                   ("f16", "sum", "tiles", 3)])
def test_reduce_clip_is_the_two_calls(comms, ranks, dtype, op, sizes, offset):
    counts = SIZES[sizes][:150]
    comm = comms(ranks)
    send = gradients(gen(2), counts, ranks, dtype, offset)
    reduced = [[torch.empty_like(t) for t in row] for row in send]
    ar.ar_all_reduce_multi(comm, send, reduced, counts, dtype, op)
    want_norm, got_norm = (torch.zeros(1, device="cuda") for _ in range(2))
    total = norm_of([row[0] for row in reduced], "l2")
    for max_norm, norm in ((total / 2, "l2"), (10 * total, "l2"), (total / 100, "inf")):
        want = [[torch.empty_like(t) for t in row] for row in send]
        ar.ar_clip_grads(comm, reduced, want, counts, max_norm, want_norm, dtype, "replicated", norm)
        got = [[placed(nan_like(s, dtype=dtype), offset) for _ in range(ranks)] for s in counts]
        ar.ar_all_reduce_clip(comm, send, got, counts, max_norm, got_norm, dtype, op, norm)
        # the sums' order may differ between the calls: fp64 sums, one fp32 ulp at most
        assert abs(float(got_norm) - float(want_norm)) <= 2 * U32 * float(want_norm)
        for w, d in zip(want, got):
            for r in range(ranks):
                close(d[r], w[r].double(), w[r].double().abs() * (4 * U32 + 2 * U[dtype]) + TINY[dtype])
                assert torch.equal(d[r], d[0]) and margins_untouched(d[r])
    inplace = [[t.clone() for t in row] for row in send]
    ar.ar_all_reduce_clip(comm, inplace, inplace, counts, total / 100, None, dtype, op, "inf")
    assert all(torch.equal(a, b) for x, y in zip(inplace, got) for a, b in zip(x, y))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_clip_of_numbers_that_are_none(comms, dtype):
    comm = comms(2)
    out = torch.zeros(1, device="cuda")
    for norm in ("l2", "inf"):
        for value in (float("nan"), float("inf"), -float("inf")):
            send = gradients(gen(3), [100, 5000], 2, dtype, 0)
            send[1][0][4321] = value
            recv = [[torch.empty_like(t) for t in row] for row in send]
            for call in ("sharded", "reduce"):
                if call == "reduce":
                    ar.ar_all_reduce_clip(comm, send, recv, [100, 5000], 1.0, out, dtype, "avg", norm)
                else:
                    ar.ar_clip_grads(comm, send, recv, [100, 5000], 1.0, out, dtype, call, norm)
                hit = recv[1][0]
                if math.isnan(value):
                    assert torch.isnan(out).all() and all(torch.isnan(t).all() for row in recv for t in row)
                else:
                    assert math.isinf(float(out)) and torch.isnan(hit[4321])
                    assert (hit[:4321] == 0).all() and (recv[0][1] == 0).all()
            # what the norm is not taken of does not count
            send[1][0][4321] = 0.0
            send[1][1][7] = value
            ar.ar_clip_grads(comm, send, recv, [100, 5000], 1e-3, out, dtype, "replicated", norm)
            assert math.isfinite(float(out)) and all(torch.isfinite(t).all() for row in recv for t in row)


def test_clip_over_the_range_of_fp32(comms):
    """Squares that fp32 cannot hold, and none at all."""
    comm = comms(1)
    out = torch.zeros(1, device="cuda")
    for size in (1e30, 1e-30):
        x = normal(gen(4), 10_000, std=1.0) * size
        ar.ar_grad_norm(comm, [[x]], [10_000], out, "f32")
        ref = norm_of([x], "l2")
        assert abs(float(out) - ref) <= ref * (U32 + 1e-12)
    out.fill_(float("nan"))
    ar.ar_grad_norm(comm, [], [], out, "f32")
    assert float(out) == 0.0
    x = torch.zeros(1000, device="cuda")
    ar.ar_clip_grads(comm, [[x]], [[x]], [1000], 1.0, out, "f32")
    assert float(out) == 0.0 and not x.any()
    x = torch.ones(10, device="cuda")
    ar.ar_clip_grads(comm, [[x]], [[x]], [10], float("inf"), out, "f32")
    assert (x == 1).all()


def test_clip_large(comms):
    """More tiles than partial sums, streaming access, and two tensors of
    which one is beyond 2^31 bytes."""
    comm = comms(1)
    counts = [600_000_011, 100_000_000]
    g = gen(5)
    x = [[torch.empty(c, dtype=torch.float32, device="cuda").normal_(generator=g)] for c in counts]
    total = math.sqrt(sum(float((p.double() ** 2).sum()) for row in x for t in row for p in t.split(1 << 26)))
    out = torch.zeros(1, device="cuda")
    y = [[torch.empty_like(t) for t in row] for row in x]
    ar.ar_clip_grads(comm, x, y, counts, 1.0, out, "f32")
    assert abs(float(out) - total) <= total * (U32 + 1e-11)
    scale = 1.0 / (total + 1e-6)
    for a, b in zip(x, y):
        for p, q in zip(a[0].split(1 << 26), b[0].split(1 << 26)):
            ref = p.double() * scale
            close(q, ref, clip_bound(ref, "f32"))


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
WIDTHS = [(1, 0, 0), (8, 0, 0), (33, 40, 1), (64, 72, 0), (256, 0, 3), (1000, 1003, 0), (2056, 0, 0)]  # width, pitch, offset


def tokens_of(kind, n, rows, first, seed=0):
    g = gen(seed + 10)
    if kind == "same":
        t = torch.full((n,), rows // 2, device="cuda")
    elif kind == "skewed":
        t = (torch.rand(n, generator=g, device="cuda") ** 4 * rows).long().clamp_(max=rows - 1)
    else:
        t = torch.randint(0, rows, (n,), generator=g, device="cuda")
    t = t + first
    if kind == "outside":  # below, above and far away
        t[::3] = first - 1 - torch.arange(len(t[::3]), device="cuda") % 5
        t[1::4] = first + rows + torch.arange(len(t[1::4]), device="cuda")
    return t


@pytest.mark.parametrize("width,pitch,offset", WIDTHS)
@pytest.mark.parametrize("n,rows,kind", [(1, 1, "any"), (5, 7, "outside"), (300, 1000, "any"), (4099, 513, "skewed")])
@pytest.mark.parametrize("dtype,index,first", [("f32", "i64", 0), ("bf16", "i32", 100), ("f16", "i64", -3)])
def test_lookup(comms, width, pitch, offset, n, rows, kind, dtype, index, first):
    comm = comms(1)
    w = placed(normal(gen(6), rows, width, dtype=dtype), offset, pitch)
    t = tokens_of(kind, n, rows, first).to(ITYPE[index])
    at = t.long() - first
    here = (at >= 0) & (at < rows)
    for scale in (1.0, 22.6274):
        out = placed(nan_like(n, width, dtype=dtype), offset, pitch)
        ar.ar_embedding(comm, w, t, out, n, rows, width, dtype, scale=scale, first_row=first)
        ref = torch.where(here[:, None], w[at.clamp(0, rows - 1)].double() * float(torch.tensor(scale)), 0.0)
        close(out, ref, ref.abs() * (U32 + U[dtype]) + TINY[dtype] / 2)
        assert margins_untouched(out)


GRAD_TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


def embedding_grad_ref(t, dout, rows, first, scale):
    at = t.long() - first
    here = (at >= 0) & (at < rows)
    x = torch.where(here[:, None], dout.double(), 0.0)
    at = at.clamp(0, rows - 1)
    total, mags = (torch.zeros(rows, dout.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    total.index_add_(0, at, x)
    mags.index_add_(0, at, x.abs())
    most = int(torch.bincount(at[here], minlength=1).max()) if bool(here.any()) else 0
    return total * scale, mags * abs(scale), most


@pytest.mark.parametrize("width,pitch,offset", WIDTHS)
@pytest.mark.parametrize("n,rows,kind", [(1, 1, "any"), (31, 7, "outside"), (33, 100, "same"), (64, 1, "any"),
                                         (2049, 513, "skewed"), (3000, 70_000, "outside"), (5000, 5, "any")])
@pytest.mark.parametrize("dtype,grad_dtype", GRAD_TYPES)
def test_embedding_grad(comms, width, pitch, offset, n, rows, kind, dtype, grad_dtype):
    if width > 300 and rows > 10_000:
        pytest.skip("covered by the smaller of the two")
    first, scale = 11, 1.5
    comm = comms(1, ar.ar_embedding_workspace_bytes(n, rows, width))
    t = tokens_of(kind, n, rows, first)
    dout = placed(normal(gen(7), n, width, dtype=dtype), offset, pitch)
    ref, mags, most = embedding_grad_ref(t, dout, rows, first, scale)
    bound = mags * ((most + 2) * U32) + ref.abs() * U[grad_dtype] + TINY[grad_dtype]
    dw = placed(nan_like(rows, width, dtype=grad_dtype), offset, pitch)
    ar.ar_embedding_backward(comm, dout, t, dw, n, rows, width, dtype, grad_dtype, scale=scale, first_row=first)
    close(dw, ref, bound)
    assert margins_untouched(dw)
    again = placed(nan_like(rows, width, dtype=grad_dtype), offset, pitch)
    ar.ar_embedding_backward(comm, dout, t.int(), again, n, rows, width, dtype, grad_dtype, scale=scale, first_row=first)
    assert torch.equal(again, dw)  # and with the other index type
    # added to what is there; rows without tokens keep theirs, whatever it is
    old = placed(normal(gen(8), rows, width, dtype=grad_dtype), offset, pitch)
    met = torch.zeros(rows, dtype=torch.bool, device="cuda")
    at = t - first
    met[at[(at >= 0) & (at < rows)]] = True
    old[~met] = float("nan")
    was = old.clone()
    ar.ar_embedding_backward(comm, dout, t, old, n, rows, width, dtype, grad_dtype, scale=scale, first_row=first,
                             accumulate=True)
    assert torch.isnan(old[~met].float()).all()
    sum_ref = was[met].double() + ref[met]
    close(old[met], sum_ref, (mags * ((most + 3) * U32))[met] + was[met].double().abs() * U32 +
          sum_ref.abs() * (U32 + U[grad_dtype]) + TINY[grad_dtype])


def test_embedding_of_no_tokens(comms):
    comm = comms(1, ar.ar_embedding_workspace_bytes(0, 100, 24))
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    x = torch.zeros(0, 24, device="cuda")
    w = torch.full((100, 24), float("nan"), device="cuda")
    ar.ar_embedding(comm, w, t, x, 0, 100, 24, "f32")
    ar.ar_embedding_backward(comm, 0, t, w, 0, 100, 24, "f32", accumulate=True)
    assert torch.isnan(w).all()
    ar.ar_embedding_backward(comm, 0, t, w, 0, 100, 24, "f32")
    assert (w == 0).all()


def test_embedding_gradient_by_differences(comms):
    """<dW, E> = d/de sum(G * lookup(W + e E)): the lookup is linear, so the
    difference of two lookups is exact up to their roundings."""
    n, rows, width, scale = 500, 60, 40, 2.0
    comm = comms(1, ar.ar_embedding_workspace_bytes(n, rows, width))
    g = gen(9)
    t = tokens_of("outside", n, rows, 0)
    w, e = normal(g, rows, width), normal(g, rows, width)
    go = normal(g, n, width)
    dw = torch.empty_like(w)
    ar.ar_embedding_backward(comm, go, t, dw, n, rows, width, "f32", scale=scale)
    a, b = torch.empty(n, width, device="cuda"), torch.empty(n, width, device="cuda")
    ar.ar_embedding(comm, w + e, t, a, n, rows, width, "f32", scale=scale)
    ar.ar_embedding(comm, w - e, t, b, n, rows, width, "f32", scale=scale)
    left = float((dw.double() * e.double()).sum())
    right = float((go.double() * (a.double() - b.double())).sum()) / 2
    size = float((go.double().abs() * (a.double().abs() + b.double().abs())).sum())
    assert abs(left - right) <= size * (n + 8) * U32


# ---------------------------------------------------------------------------
# cross entropy
# ---------------------------------------------------------------------------
def loss_inputs(n, vocab, width, dtype, seed, ignored=0.2, index="i64", pitch=0, offset=0):
    g = gen(seed)
    x = placed(normal(g, n, width, dtype=dtype), offset, pitch and width + pitch)
    w = placed(normal(g, vocab, width, dtype=dtype, std=2.0 / math.sqrt(width)), offset, pitch and width + 2 * pitch)
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    drop = torch.rand(n, generator=g, device="cuda") < ignored
    y[drop] = torch.tensor([-100, vocab, 5], device="cuda")[torch.randint(0, 3, (int(drop.sum()),), generator=g,
                                                                        device="cuda")]
    gl = torch.rand(n, generator=g, device="cuda") / n
    return x, w, y.to(ITYPE[index]), gl


def loss_ref(x, w, y, ignore):
    """z, lse, losses in 64 bits, and bounds of their errors."""
    n, width, vocab = x.shape[0], x.shape[1], w.shape[0]
    xd, wd = x.double(), w.double()
    z = xd @ wd.t()
    mag = xd.abs() @ wd.abs().t()
    # fp32 sums of `width` products (six times as many of pieces of fp32
    # operands, which leave out less than 8 * 2^-24 of each product)
    terms = width + 2 if x.dtype != torch.float32 else 6 * width + 16
    ez = mag * terms * U32
    yl = y.long()
    kept = (yl != ignore) & (yl >= 0) & (yl < vocab)
    lse = torch.logsumexp(z, 1)
    at = yl.clamp(0, vocab - 1)[:, None]
    loss = torch.where(kept, lse - z.gather(1, at)[:, 0], 0.0)
    # exp2 of a rounded argument (|z - top| * 2^-23 and a few ulp), a sum of
    # at most vocab terms, each part rescaled, and the logarithm
    span = (z.max(1).values - z.min(1).values)
    el = ez.max(1).values + (span * 4 + vocab + 32) * U32 + lse.abs() * 2 * U32
    eloss = torch.where(kept, el + ez.gather(1, at)[:, 0] + loss.abs() * U32, 0.0)
    return z, ez, lse, el, loss, eloss, kept, at


def check_loss(comms, n, vocab, width, dtype, seed, grads=True, ignore=5, **kw):
    x, w, y, gl = loss_inputs(n, vocab, width, dtype, seed, **kw)
    need = ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, dtype, backward=True)
    comm = comms(1, max(need, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, dtype)))
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    z, ez, rl, el, rloss, eloss, kept, at = loss_ref(x, w, y, ignore)
    x[~kept] = x[~kept] if not grads else float("nan")  # an ignored row may hold anything
    ar.ar_linear_cross_entropy(comm, x, w, y, losses, lse, n, vocab, width, dtype, ignore_index=ignore)
    close(lse[kept], rl[kept], el[kept], "lse")
    close(losses, rloss, eloss + 1e-300, "losses")
    if not grads:
        return
    pitch, offset = kw.get("pitch", 0), kw.get("offset", 0)
    gx = placed(nan_like(n, width, dtype=dtype), offset, pitch and width + pitch)
    gw = placed(nan_like(vocab, width, dtype=dtype), offset, pitch and width + pitch)
    ar.ar_linear_cross_entropy_backward(comm, x, w, y, lse, gl, gx, gw, n, vocab, width, dtype, ignore_index=ignore)
    p = torch.exp(z - rl[:, None])
    d = p.clone()
    d.scatter_add_(1, at, torch.full_like(d[:, :1], -1.0))
    d *= kept[:, None]
    # p's error from z's and lse's, and d's rounding to the operands' type
    ud = U[dtype] if dtype != "f32" else 4 * U32
    ed = (p * (ez + el[:, None] + 8 * U32) * 1.01 + d.abs() * (ud + 4 * U32) + TINY[dtype] / 16384) * kept[:, None]
    sums = (vocab if dtype != "f32" else 6 * vocab + 16) + 64
    wd, gd = w.double().abs(), gl.double()[:, None]
    ref = gd * (d @ w.double())
    bound = gd * (ed @ wd + sums * U32 * (d.abs() @ wd)) + ref.abs() * (U[dtype] + 4 * U32) + TINY[dtype]
    close(gx, ref, bound, "grad_hidden")
    xz = torch.where(kept[:, None], x.double(), 0.0)
    sums = (n if dtype != "f32" else 6 * n + 16) + 64
    # the weight's copy of d is also scaled by g / max g before its rounding
    top = float((gd[:, 0] * kept).max())
    ew = gd * ed + (gd * d.abs()) * (ud + 4 * U32) + top * TINY[dtype] / 16384
    ref = (gd * d).t().contiguous() @ xz
    bound = ew.t().contiguous() @ xz.abs() + sums * U32 * ((gd * d.abs()).t().contiguous() @ xz.abs())
    close(gw, ref, bound + ref.abs() * (U[dtype] + 4 * U32) + TINY[dtype], "grad_weight")
    assert margins_untouched(gx) and margins_untouched(gw)
    # the same bits again, and each alone
    for both in ((gx, None), (None, gw)):
        out = [None if b is None else torch.full_like(b, float("nan")) for b in both]
        ar.ar_linear_cross_entropy_backward(comm, x, w, y, lse, gl, *out, n, vocab, width, dtype, ignore_index=ignore)
        assert all(a is None or torch.equal(a, b) for a, b in zip(out, both))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,vocab,width", [(1, 1, 1), (1, 300, 64), (3, 257, 128), (16, 1000, 72), (17, 255, 64),
                                           (64, 2000, 320), (65, 513, 33), (255, 256, 64), (300, 3001, 192),
                                           (513, 777, 520)])
def test_loss_and_gradients(comms, dtype, n, vocab, width):
    check_loss(comms, n, vocab, width, dtype, 20)


@pytest.mark.parametrize("dtype,pitch,offset", [("bf16", 8, 0), ("bf16", 3, 0), ("f16", 0, 1), ("f32", 5, 1), ("f16", 64, 8)])
def test_loss_of_strided_rows(comms, dtype, pitch, offset):
    check_loss(comms, 130, 700, 128, dtype, 21, pitch=pitch, offset=offset, index="i32")


@pytest.mark.parametrize("ignored", [0.0, 0.5, 1.0])
def test_loss_of_ignored_tokens(comms, ignored):
    check_loss(comms, 70, 400, 64, "bf16", 22, ignored=ignored)


@pytest.mark.parametrize("n,vocab,width,dtype", [(4096, 60_001, 64, "bf16"), (2000, 30_000, 96, "f32"), (9000, 40_000, 64, "f16")])
def test_loss_in_pieces(comms, n, vocab, width, dtype):
    """Sizes whose buffers take several pieces of the vocabulary."""
    check_loss(comms, n, vocab, width, dtype, 23)


def test_loss_forward_of_packed_pieces(comms):
    check_loss(comms, 20, 130_000, 1000, "f32", 24, grads=False)


def test_loss_of_large_logits(comms):
    """Logits of several hundred, and equal ones."""
    n, vocab, width = 40, 900, 64
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "bf16"))
    x, w, y, _ = loss_inputs(n, vocab, width, "bf16", 25, ignored=0.0)
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    for factor in (300.0, -300.0, 0.0):
        xs = x * factor
        z, ez, rl, el, rloss, eloss, kept, at = loss_ref(xs, w, y, -100)
        ar.ar_linear_cross_entropy(comm, xs, w, y, losses, lse, n, vocab, width, "bf16")
        close(lse, rl, el + 1e-300)
        close(losses, rloss, eloss + 1e-300)


def test_loss_of_numbers_that_are_none(comms):
    n, vocab, width = 33, 500, 64
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "f16"))
    x, w, y, _ = loss_inputs(n, vocab, width, "f16", 26, ignored=0.0)
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    x[7, 3] = float("nan")
    x[9, 5] = float("inf")
    y[11] = -100
    ar.ar_linear_cross_entropy(comm, x, w, y, losses, lse, n, vocab, width, "f16")
    bad = torch.isnan(losses)
    assert bad[7] and bad[9] and int(bad.sum()) == 2 and losses[11] == 0


def test_loss_of_no_tokens(comms):
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(0, 300, 64, "bf16", backward=True))
    w = normal(gen(1), 300, 64, dtype="bf16")
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    ar.ar_linear_cross_entropy(comm, 0, w, t, 0, 0, 0, 300, 64, "bf16")
    gw = nan_like(300, 64, dtype="bf16")
    ar.ar_linear_cross_entropy_backward(comm, 0, w, t, 0, 0, None, gw, 0, 300, 64, "bf16")
    assert (gw == 0).all()


def test_small_gradients_do_not_underflow(comms):
    """fp16 with the mean over many tokens: every probability times 1/n is far
    below fp16's range, their sums are not."""
    n, vocab, width = 2048, 4096, 64
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "f16", backward=True))
    x, w, y, _ = loss_inputs(n, vocab, width, "f16", 27, ignored=0.0)
    gl = torch.full((n,), 2.0 ** -20, device="cuda")
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    gw, gx = nan_like(vocab, width, dtype="f16"), nan_like(n, width, dtype="f16")
    ar.ar_linear_cross_entropy(comm, x, w, y, losses, lse, n, vocab, width, "f16")
    ar.ar_linear_cross_entropy_backward(comm, x, w, y, lse, gl * 2 ** 10, gx, gw, n, vocab, width, "f16")
    p = torch.softmax(x.double() @ w.double().t(), 1)
    p[torch.arange(n), y] -= 1
    ref = (p * 2.0 ** -10).t().contiguous() @ x.double()
    assert float((gw.double() - ref).norm() / ref.norm()) < 4 * U["f16"]


def test_loss_gradient_by_differences(comms):
    """Central differences of the fp32 loss along random directions. The
    truncation error is bounded by h^2/6 times the third derivative, whose size
    is bounded by that of the logits' changes cubed."""
    n, vocab, width = 12, 150, 20
    comm = comms(1, ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "f32", backward=True))
    x, w, y, gl = loss_inputs(n, vocab, width, "f32", 28, ignored=0.2)
    g = gen(29)
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    gx, gw = torch.empty_like(x), torch.empty_like(w)

    def total(xx, ww):
        ar.ar_linear_cross_entropy(comm, xx, ww, y, losses, lse, n, vocab, width, "f32")
        return float((losses.double() * gl.double()).sum()), float((losses.double().abs() + lse.double().abs()).sum())

    h = 2.0 ** -6
    base, size = total(x, w)
    ar.ar_linear_cross_entropy_backward(comm, x, w, y, lse, gl, gx, gw, n, vocab, width, "f32")
    for _ in range(3):
        ex, ew = normal(g, n, width) / math.sqrt(width), normal(g, vocab, width) / width
        up, _ = total(x + h * ex, w + h * ew)
        down, _ = total(x - h * ex, w - h * ew)
        left = float((gx.double() * ex.double()).sum() + (gw.double() * ew.double()).sum())
        dz = float(((ex.double() @ w.double().t()).abs() + (x.double() @ ew.double().t()).abs()).max()) + 1
        truncation = float(gl.sum()) * h * h * dz ** 3
        rounding = float(gl.max()) * size * 600 * U32 / h
        assert abs((up - down) / (2 * h) - left) <= truncation + rounding


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
def test_on_another_stream_and_in_a_graph(comms):
    """All calls captured into one graph and replayed between eager work, each
    replay against the eager result on the same inputs."""
    n, vocab, width = 200, 900, 64
    need = max(ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "bf16", backward=True),
               ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, "bf16"),
               ar.ar_embedding_workspace_bytes(n, vocab, width), ar.ar_clip_workspace_bytes())
    comm = comms(2, need)
    x, w, y, gl = loss_inputs(n, vocab, width, "bf16", 30)
    t = torch.randint(0, vocab, (n,), generator=gen(31), device="cuda")
    h, gx = torch.empty_like(x), torch.empty_like(x)
    gw, ge = torch.empty(vocab, width, dtype=torch.bfloat16, device="cuda"), torch.empty(vocab, width,
                                                                                       dtype=torch.bfloat16, device="cuda")
    losses, lse, norm = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(1, device="cuda")
    outs = [[torch.empty_like(gw) for _ in range(2)] for _ in range(2)]
    results = [h, losses, lse, gx, gw, ge, norm] + outs[0] + outs[1]

    def step(stream):
        s = {"stream": stream}
        ar.ar_embedding(comm, w, t, h, n, vocab, width, "bf16", scale=2.0, **s)
        ar.ar_linear_cross_entropy(comm, h, w, y, losses, lse, n, vocab, width, "bf16", **s)
        ar.ar_linear_cross_entropy_backward(comm, h, w, y, lse, gl, gx, gw, n, vocab, width, "bf16", **s)
        ar.ar_embedding_backward(comm, gx, t, ge, n, vocab, width, "bf16", scale=2.0, **s)
        ar.ar_all_reduce_clip(comm, [[gw, ge]], outs[:1], [vocab * width], 1e-3, norm, "bf16", **s)
        ar.ar_clip_grads(comm, [[gw, ge]], outs[1:], [vocab * width], 1e-3, norm, "bf16", "sharded", **s)

    def fill(seed):
        w.copy_(normal(gen(seed), vocab, width, dtype="bf16", std=0.2))
        for r in results:
            r.fill_(float("nan"))

    side = torch.cuda.Stream()
    fill(40)
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for seed in (41, 42, 43, 44):
        fill(seed)
        torch.cuda.synchronize()
        step(None)
        torch.cuda.synchronize()
        want = [r.clone() for r in results]
        fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(results, want):
            assert not torch.isnan(a.float()).any() and torch.equal(a, b)
