"""Train a small tied-embedding language model with the vocabulary losses and
the ZeRO step, distill it into a narrower student, and tune the student on
preferences and on rewards.

N simulated data-parallel ranks share one GPU. Each rank runs its own
micro-batch: the embedding with ``zero_sharded_optimizer_gb300.embedding``, one
mixing layer with PyTorch, the loss with ``zero_sharded_optimizer_gb300.losses``,
whose gradient of the head goes straight into the rank's flat gradient buffer;
the embedding's is added on top, since the two matrices are one, and the fused
ZeRO step updates every rank's replica. The student learns from the teacher's
top logits, mixed with the labels; then to prefer sequences that follow the rule
of the text over others, near its own state before; then from rewards for tokens
that it sampled.

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

from zero_sharded_optimizer_gb300 import abi, embedding, losses  # noqa: E402
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

    def learning_rate(self, lr: float):
        self.opt.lr = lr

    def hidden(self, rank: int, tokens, flat=None):
        wte, mix = self.split(self.params[rank] if flat is None else flat)
        x = embedding.embedding_forward(tokens, wte)
        return (x + torch.tanh(x @ mix)) * 2.0

    def step(self, batches, loss) -> float:
        """``loss(rank, hidden, wte, dweight)`` -> the losses of ``batches``' tokens but for each
        sequence's last, the gradient of the head written to ``dweight``. Returns the mean loss."""
        total = 0.0
        for r, tokens in enumerate(batches):
            wte, mix = self.split(self.params[r])
            inputs = tokens[:, :-1].reshape(-1)
            x = embedding.embedding_forward(inputs, wte).requires_grad_()
            mix = mix.detach().requires_grad_()
            hidden = (x + torch.tanh(x @ mix)) * 2.0
            dwte, dmix = self.split(self.grads[r])
            out = loss(r, hidden.detach(), wte, dwte)
            hidden.backward(out.dhidden)
            # the embedding's share of the tied matrix
            embedding.embedding_backward(inputs, x.grad, dweight=dwte, accumulate=True)
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


def masked(tokens):
    """The tokens to be predicted, without those of each sequence's first quarter."""
    labels = tokens[:, 1:].clone()
    labels[:, :labels.shape[1] // 4] = -100
    return labels


def run(steps: int = 60, ranks: int = 4, vocab: int = 2000, width: int = 128, student_width: int = 64,
        top: int = 16, temperature: float = 2.0, tune: int = 10, quiet: bool = True) -> dict:
    """Mean losses per step: {"teacher": [...], "student": [...], "preference": [...],
    "policy": [...]}, the last two of ``tune`` steps each."""
    g = torch.Generator(device="cuda").manual_seed(1)
    teacher = Ranks(ranks, vocab, width, 2, 2e-2)
    student = Ranks(ranks, vocab, student_width, 3, 2e-2)
    history = {"teacher": [], "student": [], "preference": [], "policy": []}
    for step in range(steps):
        batches = [text(g, vocab, 16, 65) for _ in range(ranks)]

        def xent(r, hidden, wte, dweight):
            labels = batches[r][:, 1:].reshape(-1)
            return losses.xent_step(hidden, wte, labels, dweight=dweight)

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
                                       alpha=0.7, dweight=dweight)

        history["student"].append(student.step(batches, distill))
        if not quiet and step % 10 == 0:
            print(f"student step {step}: {history['student'][-1]:.3f}")
    student.learning_rate(1e-3)
    state = student.params[0].clone()      # the preferences' reference
    before, _ = student.split(state)
    for step in range(tune):
        # eight pairs a rank: texts, and the same beginnings gone astray; all but the first
        # quarter counts
        batches, refs = [], []
        for r in range(ranks):
            good = text(g, vocab, 8, 33)
            bad = good.clone()
            bad[:, 9:] = torch.randint(0, vocab, bad[:, 9:].shape, generator=g, device="cuda")
            batches.append(torch.cat([good, bad]))
            labels = masked(batches[r])
            refs.append(losses.preference_forward(student.hidden(r, batches[r][:, :-1], state), before,
                                                  labels).logps)

        def preference(r, hidden, wte, dweight):
            rows = hidden.view(16, 32, -1)
            out = losses.preference_step(rows, wte, masked(batches[r]), ref_logps=refs[r], dweight=dweight)
            return out._replace(dhidden=out.dhidden.view_as(hidden))

        history["preference"].append(student.step(batches, preference))
    for step in range(tune):
        # one token sampled after each: the reward is whether it follows the rule, against the
        # mean reward; two steps on the same samples
        batches = [text(g, vocab, 16, 33) for _ in range(ranks)]
        sampled = []
        for r in range(ranks):
            tokens = batches[r][:, :-1].reshape(-1)
            wte, _ = student.split(student.params[r])
            hidden = student.hidden(r, tokens)
            choice = torch.multinomial((hidden @ wte.t()).float().softmax(1), 1, generator=g)[:, 0]
            reward = (choice == (tokens * 7 + 3) % vocab).float()
            old = losses.xent_forward(hidden, wte, choice, reduction="none").loss.neg_()
            sampled.append((choice, old, reward - reward.mean()))

        def policy(r, hidden, wte, dweight):
            choice, old, advantages = sampled[r]
            return losses.policy_step(hidden, wte, choice, old, advantages, ref_logps=old, kl_weight=0.01,
                                      dweight=dweight)

        for _ in range(2):
            history["policy"].append(student.step(batches, policy))
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
