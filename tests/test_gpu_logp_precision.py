"""How exact the policy and the preference loss are beyond the bounds of a single value
(test_gpu_policy): rows whose labels are all but certain, errors of one sign over many
rows, and gradients beside the rounding of their own type."""

import math

import pytest
import torch

from logp_util import IGNORE, policy
from test_gpu_losses import TYPES, empty_matrix, gaps_untouched, matrix

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


def favoured(T, V, D, dt, favour, other, g, device):
    """Hidden states that favour a token by `favour`: their label, or another one."""
    w = torch.randn(V, D, generator=g) * 0.6 / math.sqrt(D)
    y, f = torch.randint(V, (T,), generator=g), torch.randint(V, (T,), generator=g)
    h = torch.randn(T, D, generator=g) + favour / 0.36 * w[f if other else y]
    return h.to(dt).to(device), w.to(dt).to(device), y.to(device)


def exact_logps(h, w, y):
    out = []
    for a in range(0, len(y), 1024):
        z = h[a:a + 1024].double() @ w.double().T
        out.append(z.gather(1, y[a:a + 1024, None])[:, 0] - torch.logsumexp(z, 1))
    return torch.cat(out)


@pytest.mark.parametrize("favour,other", [(0.0, False), (9.0, False), (14.0, False), (9.0, True), (14.0, True)])
@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("kind", TYPES)
def test_errors_of_one_sign(losses, cuda, kind, few, favour, other):
    """Over thousands of rows the mean error is what the arithmetic loses one way, and the loss and the sums
    over a sequence have all of it. What rounds, evens out: l of 8 to 16 is rounded by steps of 2^-20, 2.8e-7 as
    rms; two logits of size 14 are sums of 3 rounded products each in 256 chains and 8 halvings, of a partial
    sum's step 2^-20 at most: sqrt(8) 2.8e-7 would be all of them at the largest, and most are far below. 1e-6
    holds them together. What does not even out: sums on the tensor cores, cut off at each of 24 instructions of
    a segment, half a step of 2^-24 of a partial sum: 8e-6 at a logit of 14. That is corrected for the label and for the
    largest logit beside it; what is left is that of the other columns, whose logits are 5 at most and
    share their mass: 24 2^-25 of 2.5 as a mean, 1.8e-6, were all of it there, and a tenth of that
    for the logits around 0 to 2 that have most of the mass. 2.5e-7 holds it, and 1e-7 of chance for 200 rows."""
    dt, g = TYPES[kind], torch.Generator().manual_seed(int(favour) + 2 * other)
    T, V, D, calls = 6000, 5000, 768, 1
    if few:
        T, calls = (16 if kind == "fp32" else 4), 50
    off = []
    for _ in range(calls):
        h, w, y = favoured(T, V, D, dt, favour, other, g, cuda)
        off.append(policy_logps(losses, h, w, y).logps.double() - exact_logps(h, w, y))
    off = torch.cat(off)
    assert abs(float(off.mean())) < (3.5e-7 if few and kind == "bf16" else 2.5e-7)
    assert float(off.square().mean().sqrt()) < 1e-6


@pytest.mark.parametrize("kind", TYPES)
def test_mean_error_of_many_exponentials(losses, cuda, kind):
    """Log-probabilities of labels that nothing favours are log-sum-exps of 5000 exponentials, beside which nothing is
    off one way: the logits are sums of 16 products, one instruction of the tensor cores. Exponentials that are
    cut off take 4.3e-8 of the sum, and half as much again where they are rescaled. l is rounded by steps of 2^-20,
    an rms of 2.8e-7, or 4e-9 as a mean of 6000; 3e-8 is beyond chance and below what the exponentials would take."""
    dt, g = TYPES[kind], torch.Generator().manual_seed(12)
    for T, calls in ((6000, 1), (8 if kind == "bf16" else 16, 400)):
        off = []
        for _ in range(calls):
            h, w, y = favoured(T, 4931, 16, dt, 0.0, False, g, cuda)
            off.append(policy_logps(losses, h, w, y).logps.double() - exact_logps(h, w, y))
        assert abs(float(torch.cat(off).mean())) < 3e-8, T


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("T", [16, 100, 600])
def test_gradients_of_rows_that_expect_a_token(losses, cuda, T, other):
    """fp32: the rows of dhidden beside 64 bits, as means over the rows. Sums on the tensor cores are cut off at
    each of a segment's 32 instructions, half a step of 2^-24 of a partial sum: 1e-6 of a sum of one sign; slopes
    and probabilities are off by 2^-22 of themselves each, 2.4e-7. 2.5e-6 holds twice that."""
    V, D, g = 5000, 768, torch.Generator().manual_seed(T + other)
    h, w, y = favoured(T, V, D, torch.float32, 14.0, other, g, cuda)
    z = h.double() @ w.double().T
    l = torch.log_softmax(z, 1)
    ly = l.gather(1, y[:, None])[:, 0]
    G = torch.exp(l)
    G[torch.arange(T), y] = torch.expm1(ly)
    if not other:       # what a sure row leaves to the others, without the cancellation
        G[torch.arange(T), y] = -G.scatter(1, y[:, None], 0.0).sum(1)
    old = ly.float()
    want = G * torch.exp(ly - old.double())[:, None] @ w.double()
    got = losses.policy_step(h, w, y, old, torch.ones(T, device=cuda), clip=0.5, reduction="sum")
    off = (got.dhidden.double() - want).norm(dim=1) / want.norm(dim=1)
    assert float(off.mean()) < 2.5e-6


def labelled(T, V, D, labels, g, device):
    """bf16 rows that favour their labels, a tenth without one."""
    w = torch.randn(V, D, generator=g) * 0.6 / math.sqrt(D)
    y = {"any": lambda: torch.randint(V, (T,), generator=g), "one": lambda: torch.full((T,), V // 3),
         "frequent": lambda: (torch.rand(T, generator=g) * math.log(V)).exp().long().sub_(1).clamp_(0, V - 1)}[labels]()
    h = torch.randn(T, D, generator=g) + 10.0 * torch.rand(T, 1, generator=g) * w[y]
    y[torch.rand(T, generator=g) < 0.1] = IGNORE
    return h.bfloat16().to(device), w.bfloat16().to(device), y.to(device)


def exact_gradients(h, w, y, slope):
    """Of the sum of slopes times log-probabilities, in 64 bits, a block of rows at a time."""
    dh, dw = torch.zeros(h.shape, dtype=torch.float64, device=h.device), torch.zeros(w.shape, dtype=torch.float64, device=h.device)
    for a in range(0, len(y), 2048):
        k = a + torch.nonzero(slope[a:a + 2048]).squeeze(1)
        G = torch.softmax(h[k].double() @ w.double().T, 1).neg_()
        G[torch.arange(len(k)), y[k]] += 1.0
        G *= slope[k, None]
        dh[k] = G @ w.double()
        dw += G.T @ h[k].double()
    return dh, dw


def as_near_as_rounded(got, want, what):
    """Off by little more than what the result's own rounding makes it, in 2-norm."""
    own = (want.bfloat16().double() - want).norm()
    assert float((got.double() - want).norm()) <= 1.05 * float(own), what


@pytest.mark.parametrize("T,V,D,labels", [
    (300, 2000, 72, "any"), (500, 3000, 70, "one"), (512, 3000, 264, "frequent"), (513, 3000, 64, "frequent"), (1000, 6000, 97, "frequent"), (3000, 5000, 256, "frequent"), (3000, 5000, 64, "one"),
    (2100, 300001, 16, "frequent"), (33000, 3000, 40, "frequent"), (40000, 1500, 33, "any")])
@pytest.mark.parametrize("op", ["policy", "preference"])
def test_bf16_gradients_are_as_near_as_their_rounding(losses, cuda, op, T, V, D, labels):
    """More than 256 rows, whose G is bf16. The labels' entries, which are most of both gradients, get their rounding
    back, so what is left of G's is that of entries p of columns that are not the label's: the rows' other
    99.9 % of columns, each off by 2^-9 of a p that is a thousandth of 1 - p, and many together where a row has
    no more than that. 5 % holds them (with the labels' rounding: 20 to 45 %)."""
    g = torch.Generator().manual_seed(T + V)
    h, w, y = labelled(T, V, D, labels, g, cuda)
    l = exact_logps(h, w, torch.where(y >= 0, y, 0))
    if op == "policy":
        adv = torch.randn(T, generator=g).to(cuda)
        adv[torch.arange(T, device=cuda) % 5 == 0] = 0.0
        old = l.float()
        slope = torch.where(y >= 0, -adv.double() * torch.exp(l - old.double()), 0.0)

        def step(h, w, **more):
            return losses.policy_step(h, w, y, old, adv, clip=0.5, reduction="sum", **more)
    else:
        cuts = [0, T // 5, T // 2, T - 7, T]
        offsets = torch.tensor(cuts, device=cuda)
        S = torch.stack([torch.where(y >= 0, l, 0.0)[a:b].sum() for a, b in zip(cuts, cuts[1:])])
        ref = S.float()
        u = 0.1 * ((S[:2] - S[2:]) - (ref[:2].double() - ref[2:].double()))
        du = -0.1 / (1.0 + torch.exp(u))
        per = torch.cat([du, -du])
        slope = torch.where(y >= 0, torch.repeat_interleave(per, offsets.diff()), 0.0)

        def step(h, w, **more):
            return losses.preference_step(h, w, y, offsets, ref_logps=ref, reduction="sum", **more)
    dh, dw = exact_gradients(h, w, y, slope)
    got = step(h, w)
    as_near_as_rounded(got.dhidden, dh, "dhidden")
    as_near_as_rounded(got.dweight, dw, "dweight")
    # rows off 16 bytes, and without dhidden, where the labels' sums need a place of their own
    for pad in (0, 1, 3):
        to, buf = empty_matrix(V, D, torch.bfloat16, cuda, pad)
        dh_to, dh_buf = empty_matrix(T, D, torch.bfloat16, cuda, pad)
        step(matrix(h, cuda, pad), matrix(w, cuda, pad), dhidden=dh_to, dweight=to)
        as_near_as_rounded(to, dw, f"dweight {pad}")
        as_near_as_rounded(dh_to, dh, f"dhidden {pad}")
        gaps_untouched(buf, V, D, pad)
        gaps_untouched(dh_buf, T, D, pad)
        to.fill_(math.nan)
        step(matrix(h, cuda, pad), matrix(w, cuda, pad), dhidden=False, dweight=to)
        as_near_as_rounded(to, dw, f"dweight alone {pad}")
        before = torch.randn(V, D, generator=g).bfloat16().to(cuda) * dw.abs().max().float().bfloat16()
        to.copy_(before)
        step(matrix(h, cuda, pad), matrix(w, cuda, pad), dweight=to, accumulate=True)
        as_near_as_rounded(to, before.double() + dw, f"dweight added {pad}")
    only = step(h, w, dweight=False)
    as_near_as_rounded(only.dhidden, dh, "dhidden alone")


def test_labels_sums_with_rows_that_are_not_numbers(losses, cuda):
    """Rows without a slope, and without a label, bring nothing into the labels' sums."""
    T, V, D, g = 700, 900, 64, torch.Generator().manual_seed(5)
    h, w, y = labelled(T, V, D, "frequent", g, cuda)
    adv = torch.randn(T, generator=g).to(cuda)
    old = exact_logps(h, w, torch.where(y >= 0, y, 0)).float()
    adv[::3] = 0.0
    good = losses.policy_step(h, w, y, old, adv, reduction="sum")
    bad = h.clone()
    bad[::3], bad[y < 0] = math.nan, math.inf
    got = losses.policy_step(bad, w, y, old, adv, reduction="sum")
    assert torch.equal(got.dweight, good.dweight) and torch.equal(got.dhidden, good.dhidden)


@pytest.mark.parametrize("T", [300, 900])
def test_labels_sums_leave_out_an_ignored_id(losses, cuda, T):
    """An ignore_index inside the vocabulary: its rows are as those without a label."""
    V, D, g = 700, 48, torch.Generator().manual_seed(T)
    h, w, y = labelled(T, V, D, "frequent", g, cuda)
    adv, old = torch.randn(T, generator=g).to(cuda), torch.full((T,), -5.0, device=cuda)
    for ignored in (0, 3):
        want = losses.policy_step(h, w, torch.where(y == ignored, IGNORE, y), old, adv, reduction="sum")
        got = losses.policy_step(h, w, torch.where(y < 0, ignored, y), old, adv, reduction="sum", ignore_index=ignored)
        for a, b in zip(got, want):
            assert a is None and b is None or torch.equal(a, b)
