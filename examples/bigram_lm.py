"""Data-parallel training of the smallest language model, the next token from
the current one:  logits = head @ (scale * embedding[token]).

Each of N ranks holds a replica of both weights and its own part of the batch.
A step is what a large model's step has at its two ends and after its backward
pass: the embedding lookup, the cross entropy of the linear head without its
logits, both gradients, and one call that averages all gradients over the ranks
and clips them to a global norm.

    python examples/bigram_lm.py --ranks 4 --steps 100
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_all_reduce_ar_amd as ar  # noqa: E402

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def corpus(vocab, length, seed):
    """Tokens of a chain in which each token has four likely successors; the
    successors' own successors follow from the seed alone."""
    g = torch.Generator().manual_seed(seed)
    after = torch.randint(0, vocab, (vocab, 4), generator=g)
    pick = torch.randint(0, 4, (length,), generator=g)
    out = torch.empty(length, dtype=torch.int64)
    t = 0
    for i in range(length):
        t = int(after[t, pick[i]])
        out[i] = t
    return out


class Trainer:
    def __init__(self, ranks, vocab, width, tokens, dtype="bf16", lr=2.0, max_norm=0.4, scale=8.0, seed=0):
        self.ranks, self.vocab, self.width, self.tokens = ranks, vocab, width, tokens
        self.dtype, self.lr, self.max_norm, self.scale = dtype, lr, max_norm, scale
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = DTYPES[dtype]
        first = [(torch.randn(vocab, width, generator=g, device="cuda") / width ** 0.5).to(t) for _ in range(2)]
        self.weights = [[w.clone() for _ in range(ranks)] for w in first]  # [embedding, head][rank]
        self.grads = [[torch.empty_like(w) for w in row] for row in self.weights]
        self.hidden = torch.empty(tokens, width, dtype=t, device="cuda")
        self.grad_hidden = torch.empty_like(self.hidden)
        self.losses, self.lse = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.norm = torch.zeros(1, device="cuda")
        self.comm = ar.Comm(ranks, 0)
        need = max(ar.ar_embedding_workspace_bytes(tokens, vocab, width), ar.ar_clip_workspace_bytes(),
                   *(ar.ar_linear_cross_entropy_workspace_bytes(tokens, vocab, width, dtype, backward=b)
                     for b in (False, True)))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        ar.ar_comm_set_workspace(self.comm, self.workspace)

    def rank_gradients(self, r, inputs, targets):
        """Rank r's mean loss (a device number) and its gradients."""
        n, vocab, width, dtype, comm = self.tokens, self.vocab, self.width, self.dtype, self.comm
        embedding, head = self.weights[0][r], self.weights[1][r]
        counted = (targets != -100).sum()
        grad_losses = (1.0 / counted.clamp(min=1)).expand(n).contiguous()
        ar.ar_embedding(comm, embedding, inputs, self.hidden, n, vocab, width, dtype, scale=self.scale)
        ar.ar_linear_cross_entropy(comm, self.hidden, head, targets, self.losses, self.lse, n, vocab, width, dtype)
        ar.ar_linear_cross_entropy_backward(comm, self.hidden, head, targets, self.lse, grad_losses, self.grad_hidden,
                                            self.grads[1][r], n, vocab, width, dtype)
        ar.ar_embedding_backward(comm, self.grad_hidden, inputs, self.grads[0][r], n, vocab, width, dtype,
                                 scale=self.scale)
        return (self.losses * grad_losses).sum()

    def step(self, batches):
        """One step over (inputs, targets) of every rank; the mean loss."""
        losses = [self.rank_gradients(r, *batch) for r, batch in enumerate(batches)]
        counts = [w[0].numel() for w in self.weights]
        ar.ar_all_reduce_clip(self.comm, self.grads, self.grads, counts, self.max_norm, self.norm, self.dtype, "avg")
        for weights, grads in zip(self.weights, self.grads):
            for w, g in zip(weights, grads):
                w.add_(g, alpha=-self.lr)
        return torch.stack(losses).mean()

    def close(self):
        torch.cuda.synchronize()
        self.comm.close()


def batches(data, ranks, tokens, step, drop=16):
    """Each rank's next tokens and their successors; every `drop`-th one is not counted."""
    out = []
    for r in range(ranks):
        at = ((step * ranks + r) * tokens) % (len(data) - tokens - 1)
        targets = data[at + 1:at + tokens + 1].clone()
        targets[::drop] = -100
        out.append((data[at:at + tokens].contiguous(), targets))
    return out


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--steps", type=int, default=100)
    p.add_argument("--vocab", type=int, default=1000)
    p.add_argument("--width", type=int, default=128)
    p.add_argument("--tokens", type=int, default=512, help="per rank and step")
    p.add_argument("--dtype", choices=list(DTYPES), default="bf16")
    a = p.parse_args()
    data = corpus(a.vocab, 50_000, 1).cuda()
    trainer = Trainer(a.ranks, a.vocab, a.width, a.tokens, a.dtype)
    for k in range(a.steps):
        loss = trainer.step(batches(data, a.ranks, a.tokens, k))
        if k % 10 == 0 or k == a.steps - 1:
            print(f"step {k:4d}  loss {float(loss):.4f}  gradient norm {float(trainer.norm):.4f}", flush=True)
    trainer.close()


if __name__ == "__main__":
    main()
