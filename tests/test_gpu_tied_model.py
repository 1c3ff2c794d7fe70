"""The embedding and the losses together, as a model whose embedding and head are
one matrix uses them: lookup, body, loss with the head's gradient in a rank's
flat gradient buffer, the embedding's on top, and the ZeRO step; and the example
that trains so.

fp32 storage: the losses are off by a few 2^-20 of themselves and the gradients by
2^-21 of their terms (test_gpu_policy and test_gpu_embedding bound each value); the
body in between is PyTorch's in fp32, with sums of 64 terms. 1e-4 of the whole
gradient, in 2-norm, holds all of it with a factor of ten to spare."""

import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
V, D, B, L, N = 301, 64, 8, 20, 2

pytestmark = pytest.mark.gpu


def body(x, mix):
    return (x + torch.tanh(x @ mix)) * 2.0


def batch(seed, device):
    g = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, V, (B, L + 1), generator=g)
    labels = tokens[:, 1:].clone()
    labels[:, :5] = -100
    adv = torch.randn(B, L, generator=g)
    adv[2] = 0.0
    return tokens[:, :-1].contiguous().to(device), labels.to(device), adv.to(device)


def exact_logps(hidden, wte, labels):
    z = torch.log_softmax(hidden @ wte.t(), -1)
    return torch.where(labels >= 0, z.gather(-1, labels.clamp(min=0).unsqueeze(-1))[..., 0], 0.0)


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_gradient_of_the_tied_matrix(abi, cuda, kind):
    from zero_sharded_optimizer_gb300 import embedding, losses
    from zero_sharded_optimizer_gb300.optimizer import ZeroOptimizer
    g = torch.Generator().manual_seed(1)
    flat = torch.cat([torch.randn(V * D, generator=g) * 0.5 / 8, torch.randn(D * D, generator=g) / 8]).to(cuda)
    params = [flat.clone() for _ in range(N)]
    grads = [torch.full_like(flat, float("nan")) for _ in range(N)]    # every value is written
    for r in range(N):
        tokens, labels, adv = batch(r, cuda)
        wte, mix = params[r][:V * D].view(V, D), params[r][V * D:].view(D, D)
        dwte, dmix = grads[r][:V * D].view(V, D), grads[r][V * D:].view(D, D)
        # in 64 bits
        wd, md = wte.double().requires_grad_(), mix.double().requires_grad_()
        l = exact_logps(body(3.0 * wd[tokens], md), wd, labels)
        old = (l.detach() - 0.1).float()
        if kind == "policy":
            count = (labels >= 0).sum()
            want = torch.where(labels >= 0, -adv.double() * torch.exp(l - old.double()), 0.0).sum() / count
        else:
            s = l.sum(1)
            want = torch.nn.functional.softplus(-0.1 * (s[:B // 2] - s[B // 2:])).mean()
        want.backward()
        # and with the library
        x = embedding.embedding_forward(tokens, wte, scale=3.0).requires_grad_()
        m = mix.clone().requires_grad_()
        hidden = body(x, m)
        if kind == "policy":
            out = losses.policy_step(hidden.detach(), wte, labels, old, adv, dweight=dwte)
        else:
            out = losses.preference_step(hidden.detach(), wte, labels, dweight=dwte)
        hidden.backward(out.dhidden)
        embedding.embedding_backward(tokens, x.grad, scale=3.0, dweight=dwte, accumulate=True)
        dmix.copy_(m.grad)
        assert float(out.reduced) == pytest.approx(float(want.detach()), rel=1e-5)
        for got, exact in ((dwte, wd.grad), (dmix, md.grad)):
            assert float((got.double() - exact).norm() / exact.norm()) < 1e-4
        # the same by autograd alone
        wa, ma = wte.clone().requires_grad_(), mix.clone().requires_grad_()
        hidden = body(embedding.embedding(tokens, wa, 3.0), ma)
        if kind == "policy":
            loss = losses.linear_policy(hidden, wa, labels, old, adv)
        else:
            loss = losses.linear_preference(hidden, wa, labels)
        loss.backward()
        for got, exact in ((wa.grad, wd.grad), (ma.grad, md.grad)):
            assert float((got.double() - exact).norm() / exact.norm()) < 1e-4
    opt = ZeroOptimizer(flat.numel(), N, abi.ZERO_FP32, lr=1e-3)
    opt.step(params, grads)
    assert torch.equal(params[0], params[1]) and bool(params[0].isfinite().all())
    assert not torch.equal(params[0], flat)


def test_train_head_example_tunes(abi, cuda):
    spec = importlib.util.spec_from_file_location("train_head", os.path.join(ROOT, "examples", "train_head.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    h = module.run(steps=3, ranks=2, tune=2)
    assert len(h["preference"]) == 2 and len(h["policy"]) == 4
    assert all(x == x and abs(x) < 100 for part in h.values() for x in part)
