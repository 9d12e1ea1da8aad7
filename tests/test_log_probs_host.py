"""The log probabilities under a linear head without a GPU: workspace sizes and
refusals, which come before the first HIP call."""
import random

import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_lm_host import BAD, NOT_SERVED, at, host_comm, refused

SIZE = ar.ar_linear_log_probs_workspace_bytes


def test_workspace_sizes():
    for dtype in ("f32", "f16", "bf16"):
        f, b, t = SIZE(1000, 50_000, 512, dtype), SIZE(1000, 50_000, 512, dtype, backward=True), SIZE(1000, 50_000, 512, dtype, top=5)
        assert 0 < f < t and 0 < f < b < 4 << 30
    # the logits of a GiB worth of tokens at most
    assert SIZE(65_536, 262_144, 1024, "bf16", top=20) < SIZE(65_536, 262_144, 1024, "bf16") + (1 << 30) + (1 << 20)
    for bad, kw in (((10, 10, 0, "f32"), {}), ((1 << 31, 10, 8, "f32"), {}), ((10, 1 << 31, 8, "bf16"), {}),
                    ((10, 10, 8, "i32"), {}), ((10, 100, 8, "f32"), {"top": 65}), ((10, 100, 8, "f32"), {"top": -1}),
                    ((10, 1 << 24, 8, "f32"), {"top": 1})):
        with pytest.raises(ValueError):
            SIZE(*bad, **kw)


def test_refusals():
    def call(code, x=at(0), w=at(1), y=at(2), lp=at(3), h=at(4), lse=at(5), top=0, tl=None, ti=None, comm=None, n=4,
             vocab=8, width=16, dtype="bf16", **kw):
        refused(code, ar.ar_linear_log_probs, comm or host_comm(), x, w, y, lp, h, lse, n, vocab, width, dtype, top=top,
                top_log_probs=tl, top_ids=ti, **{"index": "i64", **kw})

    call(NOT_SERVED, dtype="i32")
    call(BAD, dtype=9)
    call(BAD, index=5)
    call(BAD, vocab=0)
    call(BAD, width=0)
    call(BAD, n=1 << 24)
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        call(BAD, scale=scale)
    call(BAD, x=0)
    call(BAD, w=at(1) + 1)
    call(BAD, y=at(2) + 4)
    call(BAD, lp=0)
    call(BAD, lse=0)
    call(BAD, h=at(4) + 2)
    call(BAD, lp=at(5) + 8)  # log_probs over lse
    call(BAD, h=at(3))
    call(BAD, lse=at(0) + 4)
    call(BAD, top=-1)
    call(BAD, top=9, tl=at(6), ti=at(7))       # more than the vocabulary
    call(BAD, top=65, tl=at(6), ti=at(7), vocab=100)
    call(BAD, top=2, vocab=1 << 24, tl=at(6), ti=1 << 43, w=1 << 42)
    call(BAD, top=2, ti=at(7))
    call(BAD, top=2, tl=at(6))
    call(BAD, top=2, tl=at(6), ti=at(6) + 28)
    call(BAD, top=2, tl=at(6), ti=at(3) - 4)
    call(BAD, top=2, tl=at(6) + 1, ti=at(7))
    call(BAD, top=2, tl=at(6), ti=at(7), lp=1 << 44)
    call(BAD, ld_hidden=8)
    call(BAD, ld_weight=8)
    call(BAD, comm=host_comm(1, SIZE(4, 8, 16, "bf16") - 1))
    call(BAD, top=1, tl=at(6), ti=at(7), comm=host_comm(1, SIZE(4, 8, 16, "bf16", top=1) - 1))
    with pytest.raises(TypeError):
        call(BAD, top=1, tl=at(6), ti=torch.zeros(4, 1, dtype=torch.int64))

    def grad(code, gx=at(7), gw=at(8), lse=at(3), h=at(4), a=at(5), b=at(6), comm=None, n=4, **kw):
        refused(code, ar.ar_linear_log_probs_backward, comm or host_comm(), at(0), at(1), at(2), lse, h, a, b, gx, gw, n, 8,
                16, "bf16", **{"index": "i64", **kw})

    grad(BAD, gx=None, gw=None)
    grad(BAD, gx=at(8))
    grad(BAD, gx=at(0))
    grad(BAD, gw=at(1) + 2)
    grad(BAD, gw=1 << 44)
    grad(BAD, lse=0)
    grad(BAD, a=0)
    grad(BAD, h=0)
    grad(BAD, h=None)
    grad(BAD, b=at(6) + 1)
    grad(BAD, gx=at(6))
    grad(BAD, gx=at(4))
    grad(BAD, scale=0.0)
    grad(BAD, ld_grad_hidden=3)
    grad(BAD, ld_grad_weight=3)
    grad(BAD, comm=host_comm(1, SIZE(4, 8, 16, "bf16", backward=True) - 1))


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses are not for a GPU")
def test_a_workspace_serves_fewer_tokens_and_alternatives():
    rng = random.Random(2)

    def passes(fn, *args, **kw):
        with pytest.raises(ar.ArError) as e:
            fn(*args, **kw, stream=0)
        assert e.value.code == ar.AR_ERR_HIP, str(e.value)

    far = [(1 << 45) * k for k in range(1, 11)]
    for _ in range(150):
        n, vocab, width = (int(2 ** rng.uniform(0, k)) for k in (14, 18, 13))
        dtype, top = rng.choice(["f32", "f16", "bf16"]), rng.choice([0, 1, 5, 64])
        top = min(top, vocab)
        ws = [SIZE(n, vocab, width, dtype, top=top), SIZE(n, vocab, width, dtype, backward=True)]
        for m in {n, max(1, n - 1), (n + 1) // 2, min(n, 64), min(n, 65), min(n, 16), min(n, 17), 1, rng.randint(1, n)}:
            passes(ar.ar_linear_log_probs, host_comm(ws_bytes=ws[0]), *far[:3], *far[3:6], m, vocab, width, dtype,
                   top=min(top, 1) if m % 2 else top, top_log_probs=far[6], top_ids=far[7], index="i64")
            passes(ar.ar_linear_log_probs_backward, host_comm(ws_bytes=ws[1]), *far[:9], m, vocab, width, dtype,
                   index="i64")
