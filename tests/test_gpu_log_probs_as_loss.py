"""At scale 1 and without entropy the log probabilities are the cross entropy
with its sign turned: both operators' lse and gradients, one against the other."""
import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_gpu_lm import TINY, U, U32, comms, loss_inputs, nan_like  # noqa: F401
from test_gpu_log_probs import forward, head_ref, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,vocab,width", [(5, 900, 64), (40, 900, 72), (300, 3001, 192), (700, 20_000, 64)])
def test_gradients(comms, dtype, n, vocab, width):  # noqa: F811
    x, w, y, gl = loss_inputs(n, vocab, width, dtype, 90)
    comm = comms(1, max(workspace(n, vocab, width, dtype),
                        ar.ar_linear_cross_entropy_workspace_bytes(n, vocab, width, dtype, backward=True)))
    got = forward(comm, x, w, y, n, vocab, width, dtype, entropy=False)
    losses, lse = nan_like(n, dtype="f32"), nan_like(n, dtype="f32")
    ar.ar_linear_cross_entropy(comm, x, w, y, losses, lse, n, vocab, width, dtype, ignore_index=5)
    r = head_ref(x, w, y, 5, 1.0)
    kept = r["kept"]
    assert ((got["lse"].double() - lse.double()).abs() <= 2 * r["el"]).all()
    assert ((got["log_probs"].double() + losses.double()).abs() <= 2 * r["elp"]).all()
    mine, loss = ((nan_like(n, width, dtype=dtype), nan_like(vocab, width, dtype=dtype)) for _ in range(2))
    ar.ar_linear_log_probs_backward(comm, x, w, y, got["lse"], None, -gl, None, *mine, n, vocab, width, dtype, ignore_index=5)
    ar.ar_linear_cross_entropy_backward(comm, x, w, y, lse, gl, *loss, n, vocab, width, dtype, ignore_index=5)
    # each side's d: the logits' and lse's errors, its own few roundings, and one to the
    # operands' type (in pieces of fp32 four of fp32), with what is left of a subnormal
    g = gl.double()[:, None] * kept[:, None]
    ud = U[dtype] if dtype != "f32" else 4 * U32
    size = r["p"].clone().scatter_add_(1, r["at"], torch.ones_like(g))  # p, and 1 at the target
    d = g * (r["p"] - torch.zeros_like(r["p"]).scatter_add_(1, r["at"], torch.ones_like(g)))
    ed = g * (r["p"] * (r["ez"] + r["el"][:, None]) * 1.01 + size * 16 * U32) + d.abs() * ud + g * TINY[dtype] / 4096
    wd, xz = w.double().abs(), torch.where(kept[:, None], x.double(), 0.0).abs()
    sums = (vocab if dtype != "f32" else 6 * vocab + 16) + 64
    ref = d @ w.double()
    bound = ed @ wd + sums * U32 * (d.abs() @ wd) + ref.abs() * (U[dtype] + 4 * U32) + TINY[dtype]
    assert ((mine[0].double() - loss[0].double()).abs() <= 2 * bound).all()
    # the weight's copy of d is rounded over the largest gradient once more
    sums = (n if dtype != "f32" else 6 * n + 16) + 64
    ew = ed + d.abs() * (ud + 8 * U32) + float(g.max()) * TINY[dtype] / 4096
    ref = d.t().contiguous() @ torch.where(kept[:, None], x.double(), 0.0)
    bound = (ew.t().contiguous() @ xz + sums * U32 * (d.abs().t().contiguous() @ xz) + ref.abs() * (U[dtype] + 4 * U32) +
             TINY[dtype])
    assert ((mine[1].double() - loss[1].double()).abs() <= 2 * bound).all()
    assert (mine[0][~kept] == 0).all() and (loss[0][~kept] == 0).all()
