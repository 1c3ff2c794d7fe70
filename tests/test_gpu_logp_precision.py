"""How exact the policy and the preference loss are beyond the bounds of a single value
(test_gpu_policy): rows whose labels are all but certain, errors of one sign over many
rows, and gradients beside the rounding of their own type."""

import math

import pytest
import torch

from logp_util import policy
from test_gpu_losses import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def losses(abi, cuda):
    from zero_sharded_optimizer_gb300 import losses as module
    return module


def policy_logps(losses, h, w, y):
    one = torch.ones(len(y), device=h.device)
    return losses.policy_forward(h, w, y, torch.zeros_like(one), one)


@pytest.mark.parametrize("T", [3, 70, 300])
@pytest.mark.parametrize("kind", TYPES)
def test_a_vocabulary_of_one_token(losses, cuda, kind, T):
    """Its probability is one: nothing is lost, and nothing is to be learned."""
    dt, g = TYPES[kind], torch.Generator().manual_seed(T)
    h, w = torch.randn(T, 64, generator=g).to(dt).to(cuda), torch.randn(1, 64, generator=g).to(dt).to(cuda)
    y, one = torch.zeros(T, dtype=torch.int64, device=cuda), torch.ones(T, device=cuda)
    got = losses.policy_step(h, w, y, torch.zeros_like(one), one)
    assert not got.logps.any() and bool((got.loss == -1).all())
    assert not got.dhidden.any() and not got.dweight.any()
    got = losses.preference_step(h, w, y, torch.tensor([0, 1, T], device=cuda), nll_weight=0.5)
    assert not got.logps.any() and float(got.reduced) == pytest.approx(math.log(2), rel=2.0 ** -23)
    assert not got.dhidden.any() and not got.dweight.any()


@pytest.mark.parametrize("T", [4, 70, 300])
@pytest.mark.parametrize("kind", TYPES)
def test_sure_rows_are_off_in_proportion_to_what_is_left(losses, cuda, kind, T):
    """1 - p from 1e-3 to 1e-13: l is -(1 - p) there, a sum over the other tokens, and off by what each of them
    is off by: 4 dz of the logits, 2^-20 of the exponentials and their sum. A column of weights that are all one
    makes its element of dhidden the sum of the row's gradient, zero: there the others are also off by 2^-23 |lse|
    of lse and V 2^-23 of their sum, and by 2^-8 each where G is bf16."""
    dt, V, D = TYPES[kind], 300, 64
    g = torch.Generator().manual_seed(59 + T)
    w = torch.randn(V, D, generator=g)
    w[:, 0] = 1.0
    y = torch.randint(V, (T,), generator=g)
    size = torch.linspace(20.0, 45.0, T).unsqueeze(1)
    h = size * w[y] / w[y].square().sum(1, keepdim=True)
    h[:, 0] = 0.0
    h, w, y = h.to(dt).to(cuda), w.to(dt).to(cuda), y.to(cuda)
    adv = torch.ones(T, device=cuda)
    r = policy(h, w, y, torch.zeros_like(adv), adv, reduction="sum")
    z = h.double() @ w.double().T
    others = torch.exp(torch.logsumexp(z.scatter(1, y.unsqueeze(1), -math.inf), 1) - z.gather(1, y.unsqueeze(1))[:, 0])
    assert float(others.min()) < 1e-9
    exact = -torch.log1p(others)
    got = losses.policy_step(h, w, y, exact.float(), adv, clip=0.5, reduction="sum")
    off = others * (4 * r["dz"] + 2.0 ** -20)
    assert bool(((got.logps.double() - exact).abs() <= 1.01 * off).all())
    off = others * (4 * r["dz"] + 2.0 ** -20 + 2.0 ** -23 * (r["lse"].abs() + V) + (2.0 ** -8 if kind == "bf16" else 0.0))
    assert bool((got.dhidden[:, 0].double().abs() <= 1.01 * off).all())


@pytest.mark.parametrize("top", [2 ** 33 + 1024 * 5, 2 ** 33 + 1024 * 8, 2 ** 33 + 1024 * 34])
@pytest.mark.parametrize("T", [1, 3, 16])
def test_logits_beyond_a_billion(losses, cuda, T, top):
    """Few rows of fp32, whose logits are whole numbers that fp32 holds, 2^20 apart: nothing but the largest counts, and
    every difference is exact. (Times log2(e) they are off by up to 512 in fp32: no exponent.)"""
    V = 40
    z = top - 2.0 ** 20 * torch.arange(V, dtype=torch.float64)
    assert torch.equal(z.float().double(), z)
    w, h = torch.zeros(V, 4), torch.zeros(T, 4)
    w[:, 0], h[:, 0] = z.float() * 2.0 ** -20, 2.0 ** 20
    y = torch.arange(T) * 2 % V
    got = policy_logps(losses, h.to(cuda), w.to(cuda), y.to(cuda))
    assert torch.equal(got.logps.cpu().double(), z[y] - top)
    assert bool((got.lse == float(top)).all())


@pytest.mark.parametrize("T", [3, 20, 300])
@pytest.mark.parametrize("kind", TYPES)
def test_rows_without_a_slope_beside_an_infinite_factor(losses, cuda, kind, T):
    """The gradient of the reduced loss is infinite: rows that have no part in it stay at zero."""
    dt, g = TYPES[kind], torch.Generator().manual_seed(T)
    h, w = torch.randn(T, 64, generator=g).to(dt).to(cuda), torch.randn(500, 64, generator=g).to(dt).to(cuda)
    y, adv = torch.arange(T, device=cuda), torch.ones(T, device=cuda)
    adv[::3] = 0.0
    old = policy_logps(losses, h, w, y).logps
    for factor in (math.inf, math.nan):
        got = losses.policy_step(h, w, y, old, adv, dloss=torch.tensor(factor, device=cuda))
        assert not got.dhidden[::3].any()
        assert not got.dhidden[1::3].isfinite().any() and not got.dhidden[2::3].isfinite().any()
