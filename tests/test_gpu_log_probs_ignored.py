"""Gradients of ignored tokens are zeros, whatever the weight holds, for few
tokens (both gradients in one pass) and for many."""
import math

import pytest
import torch

import ring_all_reduce_ar_amd as ar
from test_gpu_lm import comms, gen, loss_inputs, nan_like  # noqa: F401
from test_gpu_log_probs import forward, workspace

pytestmark = pytest.mark.gpu

COUNTS = [1, 6, 16, 17, 40]


def gradients(comm, x, w, y, got, a, b, dtype):
    n, width, vocab = x.shape[0], x.shape[1], w.shape[0]
    gx, gw = nan_like(n, width, dtype=dtype), nan_like(vocab, width, dtype=dtype)
    ar.ar_linear_log_probs_backward(comm, x, w, y, got["lse"], got["entropy"], a, b, gx, gw, n, vocab, width, dtype,
                                    ignore_index=5)
    return gx, gw


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", COUNTS)
@pytest.mark.parametrize("width", [64, 77])
def test_of_a_masked_vocabulary(comms, dtype, n, width):  # noqa: F811
    """Rows of the vocabulary masked by -infinity: 0 times that is no zero."""
    vocab = 300
    x, w, y, a = loss_inputs(n, vocab, width, dtype, 80, ignored=0.0)
    x[:, 0] = 1.0
    w[::3, 0] = -math.inf
    y = (y.clamp(0, vocab - 1) // 3) * 3 + 1  # open rows
    y[y == 5] = 4
    y[n // 2] = 5
    kept = y != 5
    comm = comms(1, workspace(n, vocab, width, dtype))
    got = forward(comm, x, w, y, n, vocab, width, dtype)
    gx, gw = gradients(comm, x, w, y, got, a, 0.5 * a, dtype)
    assert (gx[~kept] == 0).all()
    assert torch.isfinite(gx[kept][:, 1:].float()).all()  # (column 0 takes the masks)
    assert torch.isfinite(gw.float()).all() and (gw[::3] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", COUNTS)
def test_of_ignored_tokens_alone(comms, dtype, n):  # noqa: F811
    """No token that counts: zeros, of infinities and NaN too."""
    vocab, width = 300, 64
    x, w, y, a = loss_inputs(n, vocab, width, dtype, 81)
    y.fill_(5)
    w[3], w[70, 9], w[299, 63] = math.inf, float("nan"), -math.inf
    x[0] = float("nan")
    comm = comms(1, workspace(n, vocab, width, dtype))
    got = forward(comm, x, w, y, n, vocab, width, dtype)
    assert (got["log_probs"] == 0).all()
    gx, gw = gradients(comm, x, w, y, got, a, a, dtype)
    assert (gx == 0).all() and (gw == 0).all()
