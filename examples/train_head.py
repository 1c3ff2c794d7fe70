"""Train a small tied-embedding language model with the vocabulary losses and
the ZeRO step, then distill it into a narrower student.

N simulated data-parallel ranks share one GPU. Each rank runs its own
micro-batch: the body (embedding, one mixing layer) with PyTorch, the loss with
``zero_sharded_optimizer_gb300.losses``, whose gradient of the head goes
straight into the rank's flat gradient buffer -- on top of the embedding's,
since the two matrices are one -- and the fused ZeRO step updates every rank's
replica. The student learns from the teacher's top logits, mixed with the
labels.

    python examples/train_head.py [--steps 60] [--ranks 4]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from zero_sharded_optimizer_gb300 import abi, losses  # noqa: E402
from zero_sharded_optimizer_gb300.optimizer import ZeroOptimizer  # noqa: E402


class Ranks:
    """N replicas of one flat bf16 parameter vector: wte [V, D], then mix [D, D]."""

    def __init__(self, ranks: int, vocab: int, width: int, seed: int, lr: float):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.V, self.D, self.n = vocab, width, vocab * width + width * width
        init = torch.cat([0.5 * torch.randn(vocab * width, generator=g, device="cuda") / width ** 0.5,
                          torch.randn(width * width, generator=g, device="cuda") / width ** 0.5])
        self.params = [init.bfloat16() for _ in range(ranks)]
        self.grads = [torch.empty_like(p) for p in self.params]
        self.opt = ZeroOptimizer(self.n, ranks, abi.ZERO_BF16_MIXED, lr=lr, betas=(0.9, 0.95),
                                 master_init=init, max_grad_norm=1.0)

    def split(self, flat):
        cut = self.V * self.D
        return flat[:cut].view(self.V, self.D), flat[cut:].view(self.D, self.D)

    def hidden(self, rank: int, tokens):
        wte, mix = self.split(self.params[rank])
        x = torch.nn.functional.embedding(tokens, wte)
        return (x + torch.tanh(x @ mix)) * 2.0

    def step(self, batches, loss) -> float:
        """``loss(rank, hidden, wte, dweight)`` -> losses.Losses, the gradient of
        the head added to ``dweight``. Returns the mean loss."""
        total = 0.0
        for r, tokens in enumerate(batches):
            wte, mix = (w.detach().requires_grad_() for w in self.split(self.params[r]))
            x = torch.nn.functional.embedding(tokens[:, :-1].reshape(-1), wte)
            hidden = (x + torch.tanh(x @ mix)) * 2.0
            dwte, dmix = self.split(self.grads[r])
            dwte.zero_()
            out = loss(r, hidden.detach(), wte.detach(), dwte)
            hidden.backward(out.dhidden)
            dwte += wte.grad            # the embedding's share of the tied matrix
            dmix.copy_(mix.grad)
            total += float(out.reduced)
        self.opt.step(self.params, self.grads)
        return total / len(batches)


def text(generator, vocab: int, rows: int, length: int):
    """Token sequences that a model can learn: each token follows from the one
    before, with noise."""
    tokens = torch.empty(rows, length, dtype=torch.int64, device="cuda")
    tokens[:, 0] = torch.randint(0, vocab, (rows,), generator=generator, device="cuda")
    for i in range(1, length):
        tokens[:, i] = (tokens[:, i - 1] * 7 + 3) % vocab
        noise = torch.rand(rows, generator=generator, device="cuda") < 0.1
        tokens[:, i] = torch.where(noise, torch.randint(0, vocab, (rows,), generator=generator,
                                                        device="cuda"), tokens[:, i])
    return tokens


def run(steps: int = 60, ranks: int = 4, vocab: int = 2000, width: int = 128, student_width: int = 64,
        top: int = 16, temperature: float = 2.0, quiet: bool = True) -> dict:
    """Mean losses per step: {"teacher": [...], "student": [...]}."""
    g = torch.Generator(device="cuda").manual_seed(1)
    teacher = Ranks(ranks, vocab, width, 2, 2e-2)
    student = Ranks(ranks, vocab, student_width, 3, 2e-2)
    history = {"teacher": [], "student": []}
    for step in range(steps):
        batches = [text(g, vocab, 16, 65) for _ in range(ranks)]

        def xent(r, hidden, wte, dweight):
            labels = batches[r][:, 1:].reshape(-1)
            return losses.xent_step(hidden, wte, labels, dweight=dweight, accumulate=True)

        history["teacher"].append(teacher.step(batches, xent))
        if not quiet and step % 10 == 0:
            print(f"teacher step {step}: {history['teacher'][-1]:.3f}")
    for step in range(steps):
        batches = [text(g, vocab, 16, 65) for _ in range(ranks)]

        def distill(r, hidden, wte, dweight):
            tokens, labels = batches[r][:, :-1].reshape(-1), batches[r][:, 1:].reshape(-1)
            big, _ = teacher.split(teacher.params[r])
            logits, ids = (teacher.hidden(r, tokens) @ big.t()).float().topk(top, dim=1)
            return losses.distill_step(hidden, wte, ids, logits, temperature=temperature, labels=labels,
                                       alpha=0.7, dweight=dweight, accumulate=True)

        history["student"].append(student.step(batches, distill))
        if not quiet and step % 10 == 0:
            print(f"student step {step}: {history['student'][-1]:.3f}")
    for model in (teacher, student):
        assert all(torch.equal(p, model.params[0]) for p in model.params), "replicas differ"
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--ranks", type=int, default=4)
    a = ap.parse_args()
    h = run(a.steps, a.ranks, quiet=False)
    print({k: (round(v[0], 3), round(v[-1], 3)) for k, v in h.items()})
