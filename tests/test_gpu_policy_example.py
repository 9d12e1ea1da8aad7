"""examples/policy_lm.py: the operators of a policy-gradient step together, against
the same step in 64 bits."""
import importlib.util
import os

import pytest
import torch

from test_gpu_orthogonalize import error_bound, iterate

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "policy_lm.py")
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("policy_lm", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_gradients(trainer, batches):
    """Both gradients' means over the ranks and the objective, by autograd in 64 bits."""
    emb, head = (row[0].double().clone().requires_grad_() for row in trainer.weights)
    total = 0.0
    for inputs, actions, advantages in batches:
        log_p = torch.log_softmax((emb[inputs] * trainer.scale) @ head.t(), 1)
        chosen = log_p.gather(1, actions[:, None])[:, 0]
        entropy = -(log_p.exp() * log_p).sum(1)
        total = total - (advantages.double() * chosen + trainer.bonus * entropy).mean() / len(batches)
    return torch.autograd.grad(total, (emb, head))


def test_a_step_is_the_plain_one(lm):
    """fp32: the gradients are off by a few hundred roundings of 2^-24 of their
    norm, and orthogonalising lets what is off grow by at most 4 in each of its
    five steps, beside its own error."""
    trainer = lm.Trainer(3, 301, 72, 130, "f32")
    allowed = lm.chain(301, 5).cuda()
    g = torch.Generator(device="cuda").manual_seed(6)
    batches = [lm.batch(trainer, allowed, r, g)[0] for r in range(3)]
    for _, actions, _ in batches:
        assert actions.dtype == torch.int64 and int(actions.min()) >= 0 and int(actions.max()) < 301
    before = [row[0].double() for row in trainer.weights]
    grads = plain_gradients(trainer, batches)
    trainer.learn(batches)
    total = float(torch.sqrt(sum((x * x).sum() for x in grads)))
    assert abs(float(trainer.norm) - total) <= 500 * U32 * total
    clip = min(1.0, trainer.max_norm / (total + 1e-6))
    for grad, row, reduced, momentum, old in zip(grads, trainer.weights, trainer.grads, trainer.momentum, before):
        grad = grad * clip
        off = float((reduced[0].double() - grad).norm() / grad.norm())
        assert off <= 500 * U32
        assert float((momentum.double() - 0.05 * grad).norm()) <= 600 * U32 * 0.05 * float(grad.norm())
        want = old - trainer.lr * iterate(grad)  # momentum and its look ahead are multiples of the first gradient
        allowed_off = trainer.lr * (error_bound(301, 72) + 4 ** 5 * 600 * U32) + 4 * U32 * float(want.norm())
        assert float((row[0].double() - want).norm()) <= allowed_off
        assert all(torch.equal(w, row[0]) for w in row)
    trainer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_it_runs(lm, dtype):
    trainer = lm.Trainer(2, 200, 64, 256, dtype)
    allowed = lm.chain(200, 3).cuda()
    g = torch.Generator(device="cuda").manual_seed(4)
    for _ in range(5):
        trainer.learn([lm.batch(trainer, allowed, r, g)[0] for r in range(2)])
    assert all(torch.isfinite(w.float()).all() for row in trainer.weights for w in row)
    assert all(torch.equal(w, row[0]) for row in trainer.weights for w in row)
    assert (trainer.entropy > 0).all() and (trainer.log_probs < 0).all()
    trainer.close()
