"""examples/bigram_lm.py: the language-model operators together, against the
same training in plain torch operations."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "bigram_lm.py")


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("bigram_lm", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_steps(trainer, steps_of_batches):
    """The same steps in 64 bits: losses, and the weights at the end."""
    emb, head = (row[0].double().clone() for row in trainer.weights)
    losses = []
    for step in steps_of_batches:
        grads = [torch.zeros_like(emb), torch.zeros_like(head)]
        mean = 0.0
        for inputs, targets in step:
            kept = targets != -100
            x = emb[inputs] * trainer.scale
            z = x @ head.t()
            lse = torch.logsumexp(z, 1)
            n = int(kept.sum())
            at = targets.clamp(min=0)[:, None]
            mean += float(((lse - z.gather(1, at)[:, 0]) * kept).sum()) / n / len(step)
            d = torch.exp(z - lse[:, None])
            d.scatter_add_(1, at, torch.full_like(lse[:, None], -1.0))
            d *= kept[:, None] / n
            grads[1] += d.t().contiguous() @ x / len(step)
            grads[0].index_add_(0, inputs, d @ head * (trainer.scale / len(step)))
        total = float(torch.sqrt(sum((g * g).sum() for g in grads)))
        scale = min(1.0, trainer.max_norm / (total + 1e-6))
        emb -= trainer.lr * scale * grads[0]
        head -= trainer.lr * scale * grads[1]
        losses.append(mean)
    return losses, (emb, head)


def test_training_is_the_plain_one(lm):
    """Six fp32 steps. Each step's gradients are off by a few hundred roundings
    of 2^-24 of their norm (sums of up to 512 x 6 products), the norm is clipped
    to 0.4, and the learning rate is 2: after six steps the weights differ by less
    than 6 * 2 * 1000 * 2^-24 of the clip, and the losses by that times the
    largest change of a loss with a weight, |scale * x| < 30."""
    data = lm.corpus(301, 5000, 2).cuda()
    trainer = lm.Trainer(3, 301, 72, 130, "f32")
    steps = [lm.batches(data, 3, 130, k) for k in range(6)]
    want, weights = plain_steps(trainer, steps)
    got = [float(trainer.step(s)) for s in steps]
    off = 6 * 2 * 1000 * 2.0 ** -24
    assert all(abs(a - b) <= 30 * off for a, b in zip(got, want)), (got, want)
    for row, ref in zip(trainer.weights, weights):
        assert all(float((w.double() - ref).abs().max()) <= off for w in row)
        assert all(torch.equal(w, row[0]) for w in row)
    trainer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_training_learns(lm, dtype):
    data = lm.corpus(200, 20_000, 3).cuda()
    trainer = lm.Trainer(2, 200, 64, 512, dtype)
    losses = [float(trainer.step(lm.batches(data, 2, 512, k))) for k in range(60)]
    # from about log 200 = 5.3 towards the chain's log 4 = 1.39
    assert losses[0] > 4.0 and losses[-1] < 2.5, losses
    trainer.close()
