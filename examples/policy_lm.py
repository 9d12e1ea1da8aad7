"""Policy-gradient training of the smallest language model over several ranks:
logits = head @ (scale * embedding[token]), rewarded for tokens that a chain
allows after the given one.

Each rank samples its actions among the likeliest tokens of its own inputs, and
learns from log p(action) times the advantage plus an entropy bonus. A step is
what a large model's step has around its trunk: the embedding lookup, the log
probabilities with entropy and alternatives, their gradients, one call that
averages the gradients over the ranks and clips them, and one that updates both
weights of every rank by orthogonalised momentum.

    python examples/policy_lm.py --ranks 4 --steps 100
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_all_reduce_ar_amd as ar  # noqa: E402

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def chain(vocab, seed, likely=16):
    """The tokens that may follow each token."""
    g = torch.Generator().manual_seed(seed)
    return torch.stack([torch.randperm(vocab, generator=g)[:likely] for _ in range(vocab)])


class Trainer:
    def __init__(self, ranks, vocab, width, tokens, dtype="bf16", top=16, lr=0.02, bonus=0.01, max_norm=1.0, scale=4.0,
                 seed=0):
        self.ranks, self.vocab, self.width, self.tokens, self.dtype = ranks, vocab, width, tokens, dtype
        self.top, self.lr, self.bonus, self.max_norm, self.scale = top, lr, bonus, max_norm, scale
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = DTYPES[dtype]
        first = [(torch.randn(vocab, width, generator=g, device="cuda") / width ** 0.5).to(t) for _ in range(2)]
        self.weights = [[w.clone() for _ in range(ranks)] for w in first]  # [embedding, head][rank]
        self.grads = [[torch.empty_like(w) for w in row] for row in self.weights]
        self.momentum = [torch.zeros(vocab, width, device="cuda") for _ in first]
        self.hidden = torch.empty(tokens, width, dtype=t, device="cuda")
        self.grad_hidden = torch.empty_like(self.hidden)
        self.log_probs, self.entropy, self.lse = (torch.empty(tokens, device="cuda") for _ in range(3))
        self.top_log_probs = torch.empty(tokens, top, device="cuda")
        self.top_ids = torch.empty(tokens, top, dtype=torch.int32, device="cuda")
        self.norm = torch.zeros(1, device="cuda")
        self.comm = ar.Comm(ranks, 0)
        need = max(ar.ar_embedding_workspace_bytes(tokens, vocab, width), ar.ar_clip_workspace_bytes(),
                   ar.ar_orthogonalize_workspace_bytes(2, vocab, width),
                   ar.ar_linear_log_probs_workspace_bytes(tokens, vocab, width, dtype, top=top),
                   ar.ar_linear_log_probs_workspace_bytes(tokens, vocab, width, dtype, backward=True))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        ar.ar_comm_set_workspace(self.comm, self.workspace)

    def evaluate(self, r, inputs, targets, top=0):
        """Rank r's log probabilities, entropies and lse of the targets, and with
        `top` their likeliest tokens, into the trainer's buffers."""
        n, vocab, width = self.tokens, self.vocab, self.width
        ar.ar_embedding(self.comm, self.weights[0][r], inputs, self.hidden, n, vocab, width, self.dtype, scale=self.scale)
        ar.ar_linear_log_probs(self.comm, self.hidden, self.weights[1][r], targets, self.log_probs, self.entropy, self.lse,
                               n, vocab, width, self.dtype, top=top, top_log_probs=self.top_log_probs if top else None,
                               top_ids=self.top_ids if top else None)

    def sample(self, r, inputs, noise):
        """Actions among the alternatives, by Gumbel noise [tokens][top]."""
        self.evaluate(r, inputs, torch.full_like(inputs, -100), self.top)
        return self.top_ids.gather(1, (self.top_log_probs + noise).argmax(1, keepdim=True))[:, 0].to(inputs.dtype)

    def rank_gradients(self, r, inputs, actions, advantages):
        """Of -mean(advantage * log p(action) + bonus * entropy)."""
        n, vocab, width, dtype, comm = self.tokens, self.vocab, self.width, self.dtype, self.comm
        self.evaluate(r, inputs, actions)
        ar.ar_linear_log_probs_backward(comm, self.hidden, self.weights[1][r], actions, self.lse, self.entropy,
                                        -advantages / n, torch.full_like(advantages, -self.bonus / n), self.grad_hidden,
                                        self.grads[1][r], n, vocab, width, dtype)
        ar.ar_embedding_backward(comm, self.grad_hidden, inputs, self.grads[0][r], n, vocab, width, dtype,
                                 scale=self.scale)

    def learn(self, batches):
        """One step over (inputs, actions, advantages) of every rank."""
        for r, batch in enumerate(batches):
            self.rank_gradients(r, *batch)
        counts = [w[0].numel() for w in self.weights]
        ar.ar_all_reduce_clip(self.comm, self.grads, self.grads, counts, self.max_norm, self.norm, self.dtype, "avg")
        ar.ar_muon_update(self.comm, [row[0] for row in self.grads], self.momentum, self.momentum,
                          [row[0] for row in self.weights], self.weights, self.vocab, self.width, self.dtype, lr=self.lr)

    def close(self):
        torch.cuda.synchronize()
        self.comm.close()


def batch(trainer, allowed, r, g):
    """Inputs, sampled actions and their advantages; the mean reward."""
    n = trainer.tokens
    inputs = torch.randint(0, trainer.vocab, (n,), generator=g, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(n, trainer.top, generator=g, device="cuda")))
    actions = trainer.sample(r, inputs, noise)
    reward = (allowed[inputs] == actions[:, None]).any(1).float()
    return (inputs, actions, reward - reward.mean()), reward.mean()


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--steps", type=int, default=100)
    p.add_argument("--vocab", type=int, default=200)
    p.add_argument("--width", type=int, default=128)
    p.add_argument("--tokens", type=int, default=512, help="per rank and step")
    p.add_argument("--dtype", choices=list(DTYPES), default="bf16")
    a = p.parse_args()
    allowed = chain(a.vocab, 1).cuda()
    trainer = Trainer(a.ranks, a.vocab, a.width, a.tokens, a.dtype)
    g = torch.Generator(device="cuda").manual_seed(2)
    for k in range(a.steps):
        batches, rewards = zip(*(batch(trainer, allowed, r, g) for r in range(a.ranks)))
        trainer.learn(batches)
        if k % 10 == 0 or k == a.steps - 1:
            print(f"step {k:4d}  reward {float(sum(rewards)) / a.ranks:.4f}  entropy {float(trainer.entropy.mean()):.4f}  "
                  f"gradient norm {float(trainer.norm):.4f}", flush=True)
    trainer.close()


if __name__ == "__main__":
    main()
