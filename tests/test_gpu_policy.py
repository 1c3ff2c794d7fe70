"""The policy and the preference loss on the GPU against their definitions in 64
bits, within bounds derived from their arithmetic (logp_util)."""

import math

import pytest
import torch

from logp_util import IGNORE, check, policy, preference
from test_gpu_losses import SIZES, TYPES, apart, empty_matrix, gaps_untouched, inputs, matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def losses(abi, cuda):
    from zero_sharded_optimizer_gb300 import losses as module
    return module


def parts_of(dtype, T):
    return 2 if dtype == torch.bfloat16 and T <= 256 else 1


def exact_logps(h, w, y):
    z = h.double() @ w.double().T
    has = (y >= 0) & (y < w.shape[0])
    return torch.where(has, z.gather(1, torch.where(has, y, 0).unsqueeze(1))[:, 0] - torch.logsumexp(z, 1), 0.0)


def sampled(h, w, y, g, clip=(0.2, 0.2), still=0.0):
    """Old log-probabilities whose ratios lie a hundredth from the bounds at least, advantages
    and a reference's log-probabilities."""
    T, dev = h.shape[0], h.device
    moved = 0.3 * torch.randn(T, generator=g, dtype=torch.float64)
    for bound in (1 - clip[0], 1 + clip[1]):
        near = (moved.exp() - bound).abs() < 0.01
        moved = torch.where(near, moved + 0.04, moved)
    l = exact_logps(h, w, y)
    adv = torch.randn(T, generator=g)
    adv[torch.rand(T, generator=g) < still] = 0.0
    ref = l + 0.3 * torch.randn(T, generator=g).to(dev)
    return (l - moved.to(dev)).float(), adv.to(dev), ref.float()


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("kind", TYPES)
def test_policy_step(losses, cuda, kind, T, V, D):
    dt = TYPES[kind]
    h, w, y, g = inputs(T, V, D, dt, 2000 + T + V + D, cuda, masked=0.2 if T > 2 else 0.0)
    for clip, kl, reduction in (((0.2, 0.2), 0.0, "mean"), ((0.1, 0.28), 0.05, "sum"), ((0.2, 0.3), 0.1, "none")):
        old, adv, ref = sampled(h, w, y, g, clip, still=0.2)
        dloss = torch.rand(T, generator=g).to(cuda) if reduction == "none" else None
        r = policy(h, w, y, old, adv, ref if kl else None, clip, kl, reduction, dloss)
        got = losses.policy_step(matrix(h, cuda), matrix(w, cuda), y, old, adv, ref_logps=ref if kl else None,
                                 clip=clip, kl_weight=kl, reduction=reduction, dloss=dloss)
        check(got, r, dt, f"{kind} {clip} {kl} {reduction}", parts_of(dt, T))
        assert torch.equal(got.dhidden[r["slopes"] == 0], torch.zeros_like(h)[r["slopes"] == 0])


@pytest.mark.parametrize("T", [4, 5, 8, 9, 16, 17, 31, 32, 33, 64, 65])
@pytest.mark.parametrize("kind", TYPES)
def test_around_what_counts_as_few_rows(losses, cuda, kind, T):
    """Rows on both sides of the limits and of the groups of eight, small and larger vocabularies and
    widths, columns off the blocks of four, 32 and 64; rows without a label or a slope between."""
    dt = TYPES[kind]
    for n, (V, D) in enumerate([(97, 33), (1027, 264), (5000, 520), (20001, 96), (130, 5200), (67, 10300)]):
        h, w, y, g = inputs(T, V, D, dt, 40 + T + V, cuda, masked=0.2)
        old, adv, ref = sampled(h, w, y, g, still=0.3)
        kl, reduction = (0.05, "none") if n % 2 else (0.0, "mean")
        dloss = torch.rand(T, generator=g).to(cuda) if n % 2 else None
        r = policy(h, w, y, old, adv, ref if kl else None, (0.2, 0.2), kl, reduction, dloss)
        for pad in (0, 3):
            before = torch.randn(V, D, generator=g).to(dt).to(cuda)
            dw, buf = empty_matrix(V, D, dt, cuda, pad)
            dh, dh_buf = empty_matrix(T, D, dt, cuda, pad)
            got = losses.policy_step(matrix(h, cuda, pad), matrix(w, cuda, pad), y, old, adv, clip=0.2, kl_weight=kl,
                                     ref_logps=ref if kl else None, reduction=reduction, dloss=dloss, dhidden=dh,
                                     dweight=dw)
            check(got, r, dt, f"{kind} {V} {D} {pad}", 2)
            gaps_untouched(buf, V, D, pad)
            gaps_untouched(dh_buf, T, D, pad)
            alone = dw.double()
            dw.copy_(before)
            losses.policy_step(matrix(h, cuda, pad), matrix(w, cuda, pad), y, old, adv, clip=0.2, kl_weight=kl,
                               ref_logps=ref if kl else None, reduction=reduction, dloss=dloss, dweight=dw,
                               accumulate=True)
            # as far as the gradient alone, which is rounded too, and one rounding
            unit = 2.0 ** -24 if kind == "fp32" else 2.0 ** -8
            want = before.double() + r["dweight"]
            off = (dw.double() - want).abs()
            assert bool((off <= (alone - r["dweight"]).abs() + 1.01 * unit * (alone.abs() + want.abs()) + 1e-7).all())


@pytest.mark.parametrize("T", [3, 20, 300])
@pytest.mark.parametrize("kind", TYPES)
def test_rows_without_a_slope_bring_nothing_in(losses, cuda, kind, T):
    """A hidden state that is not a number, in a row of advantage zero."""
    dt = TYPES[kind]
    h, w, y, g = inputs(T, 300, 64, dt, 50 + T, cuda)
    old, adv, _ = sampled(h, w, y, g)
    adv[1] = 0.0
    r = policy(h, w, y, old, adv, reduction="sum")
    bad = h.clone()
    bad[1] = math.nan
    got = losses.policy_step(bad, w, y, old, adv, reduction="sum")
    assert math.isnan(float(got.logps[1])) and float(got.loss[1]) == 0.0 and not got.dhidden[1].any()
    check(got._replace(logps=None, row_logps=None), r, dt, "", parts_of(dt, T))


@pytest.mark.parametrize("T", [8, 300])
@pytest.mark.parametrize("kind", TYPES)
def test_gradients_of_sure_rows_sum_to_zero(losses, cuda, kind, T):
    """Rows that are all but certain of their labels. A column of weights that are all one makes its
    element of dhidden the sum of the row's gradient, which is zero: the label's p - 1 cancels the others'
    p, 1 - p of it. The others' share of the error is in proportion to 1 - p: 4 dz of the logits, 2^-20 of
    their exponentials, 2^-23 |lse| of lse, V 2^-23 of their sum, 2^-8 where G is bf16. The label's own is
    that of a sum of exponentials that is 1 and little more: some roundings of 2^-24 and the mean of what
    the tensor cores' sums lose that is put back (1.1e-7), 2^-21 in all."""
    dt, V, D = TYPES[kind], 300, 64
    g = torch.Generator().manual_seed(58 + T)
    w = torch.randn(V, D, generator=g)
    w[:, 0] = 1.0
    y = torch.randint(V, (T,), generator=g)
    size = torch.linspace(20.0, 60.0, T).unsqueeze(1)
    h = size * w[y] / w[y].square().sum(1, keepdim=True)
    h[:, 0] = 0.0
    h, w, y = h.to(dt).to(cuda), w.to(dt).to(cuda), y.to(cuda)
    adv = torch.ones(T, device=cuda)
    r = policy(h, w, y, torch.zeros_like(adv), adv, reduction="sum")
    got = losses.policy_step(h, w, y, r["l"].float(), adv, clip=0.5, reduction="sum")
    others = -torch.expm1(r["l"])
    off = others * (4 * r["dz"] + 2.0 ** -20 + 2.0 ** -23 * (r["lse"].abs() + V) +
                    (2.0 ** -8 if kind == "bf16" else 0.0)) + 2.0 ** -21
    assert bool((got.dhidden[:, 0].double().abs() <= 1.01 * off).all())


def test_policy_clip_of_one_number(losses, cuda):
    h, w, y, g = inputs(50, 300, 64, torch.bfloat16, 1, cuda)
    old, adv, _ = sampled(h, w, y, g)
    a = losses.policy_forward(h, w, y, old, adv, clip=0.2)
    b = losses.policy_forward(h, w, y, old, adv, clip=(0.2, 0.2))
    assert torch.equal(a.loss, b.loss)


@pytest.mark.parametrize("T", [300, 1500, 3000])
@pytest.mark.parametrize("kind", TYPES)
def test_policy_most_rows_without_a_slope(losses, cuda, kind, T):
    """Advantages of zero and clipped ratios: the products take the other rows alone."""
    dt = TYPES[kind]
    V, D = 600, 72
    h, w, y, g = inputs(T, V, D, dt, T, cuda, masked=0.1)
    for still in (0.5, 0.95, 1.0):
        old, adv, _ = sampled(h, w, y, g, still=still)
        r = policy(h, w, y, old, adv)
        check(losses.policy_step(h, w, y, old, adv), r, dt, f"{still}", parts_of(dt, T))
        out = losses.policy_forward(h, w, y, old, adv)
        got = losses.policy_backward(h, w, y, out.lse, out.row_logps, out.slopes)
        check(got, r, dt, f"{still} backward", parts_of(dt, T))
    assert not got.dhidden.any() and not got.dweight.any()


@pytest.mark.parametrize("kind", TYPES)
def test_policy_edges(losses, cuda, kind):
    """Ratios that overflow or vanish, and advantages of zero beside them; values that are not numbers."""
    dt = TYPES[kind]
    T, V, D = 300, 500, 64
    h, w, y, g = inputs(T, V, D, dt, 8, cuda, masked=0.1)
    old, adv, _ = sampled(h, w, y, g)
    old[0::10], adv[0::10] = -math.inf, 1.0          # ratio inf: clipped
    old[1::10], adv[1::10] = -math.inf, 0.0          # without a part in the loss
    old[2::10], adv[2::10] = math.inf, 1.0           # ratio 0: free, without a slope
    old[3::10], adv[3::10] = math.inf, -1.0          # held at the lower bound
    there = y != IGNORE
    got = losses.policy_step(h, w, y, old, adv, reduction="none")
    want = {0: -1.2, 1: 0.0, 2: 0.0, 3: 0.8}
    for k, value in want.items():
        rows = there & (torch.arange(T, device=cuda) % 10 == k)
        assert torch.allclose(got.loss[rows].double(), torch.tensor(value, dtype=torch.float64, device=cuda), atol=1e-7)
        assert not got.slopes[rows].any() and not got.dhidden[rows].any()
    usual = torch.arange(T, device=cuda) % 10 > 3
    r = policy(h, w, torch.where(usual, y, IGNORE), old, adv, reduction="none")
    check(got._replace(logps=None, row_logps=None, slopes=None, dhidden=None,
                       loss=torch.where(usual, got.loss, 0.0)), r, dt)
    # not a number: it shows in its row, and in no other
    for name in ("old", "adv", "ref"):
        o, a, ref = sampled(h, w, y, g)
        k = int(torch.nonzero(there)[5])
        {"old": o, "adv": a, "ref": ref}[name][k] = math.nan
        got = losses.policy_step(h, w, y, o, a, ref_logps=ref, kl_weight=0.1, reduction="none")
        rest = torch.arange(T, device=cuda) != k
        assert math.isnan(float(got.loss[k])) and math.isnan(float(got.slopes[k])) and bool(got.dhidden[k].isnan().all())
        assert bool(got.loss[rest].isfinite().all()) and bool(got.dhidden[rest].isfinite().all())
    # what belongs to empty rows is not read
    o, a, ref = sampled(h, w, y, g)
    r = policy(h, w, y, o, a, ref, kl=0.1)
    bad = h.clone()
    for x in (o, a, ref, bad):
        x[~there] = math.nan
    got = losses.policy_step(bad, w, y, o, a, ref_logps=ref, kl_weight=0.1)
    check(got, r, dt, "", 1)
    assert not got.loss[~there].any() and not got.logps[~there].any() and not got.slopes[~there].any()


def pairs_of(T, P, g, empty=0.0):
    """Offsets of 2 P ragged sequences in T rows, some empty."""
    cuts = torch.randint(0, T + 1, (2 * P - 1,), generator=g).sort().values.tolist()
    bounds = [0] + cuts + [T]
    for k in range(1, 2 * P):
        if empty and float(torch.rand(1, generator=g)) < empty:
            bounds[k] = bounds[k - 1]
    return bounds


OPTIONS = [dict(), dict(beta=0.5, smoothing=0.1, margin=0.3), dict(kind="squared", beta=1.0, margin=0.5, average=True),
           dict(average=True, beta=2.0, nll=0.3), dict(kind="squared", beta=0.1, margin=-0.5, nll=0.2)]


def own(options):
    return {{"nll": "nll_weight"}.get(k, k): v for k, v in options.items()}


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("kind", TYPES)
def test_preference_step(losses, cuda, kind, T, V, D):
    dt = TYPES[kind]
    h, w, y, g = inputs(T, V, D, dt, 3000 + T + V + D, cuda, masked=0.2 if T > 2 else 0.0)
    l = exact_logps(h, w, y)
    for n, options in enumerate(OPTIONS):
        P = max(1, min(T // 2, (1, 3, 8)[n % 3]))
        bounds = pairs_of(T, P, g, 0.1)
        offsets = torch.tensor(bounds, device=cuda)
        reduction = ("mean", "sum", "none")[n % 3]
        dloss = torch.rand(P, generator=g).to(cuda) if reduction == "none" else None
        ref = None
        if n != 3:
            # a reference near the sums or the means
            ref = torch.stack([l[a:b].sum() for a, b in zip(bounds, bounds[1:])])
            if options.get("average"):
                has = y != IGNORE
                ref = ref / torch.stack([has[a:b].sum().clamp(min=1) for a, b in zip(bounds, bounds[1:])])
            ref = (ref + 2.0 * torch.randn(2 * P, generator=g).to(cuda)).float()
        r = preference(h, w, y, bounds, ref, reduction=reduction, dloss=dloss, **options)
        got = losses.preference_step(matrix(h, cuda), matrix(w, cuda), y, offsets, ref_logps=ref,
                                     reduction=reduction, dloss=dloss, **own(options))
        check(got, r, dt, f"{kind} {options}", parts_of(dt, T))


@pytest.mark.parametrize("kind", TYPES)
def test_preference_of_a_padded_batch(losses, cuda, kind):
    dt, P, L, V, D = TYPES[kind], 3, 37, 300, 40
    h, w, y, g = inputs(2 * P * L, V, D, dt, 5, cuda, masked=0.3)
    bounds = list(range(0, 2 * P * L + 1, L))
    r = preference(h, w, y, bounds)
    a = losses.preference_step(h.view(2 * P, L, D), w, y.view(2 * P, L))
    b = losses.preference_step(h, w, y, torch.tensor(bounds, device=cuda))
    check(a, r, dt, "", parts_of(dt, 2 * P * L))
    assert a.dhidden.shape == (2 * P, L, D)
    for x, z in zip(a, b):
        assert torch.equal(x.flatten(), z.flatten())


@pytest.mark.parametrize("kind", TYPES)
def test_preference_empty_sequences(losses, cuda, kind):
    """Pairs of which one sequence, or both, have no labelled row; rows outside all sequences;
    what belongs to nothing is not read."""
    dt, V, D = TYPES[kind], 400, 48
    T = 120
    h, w, y, g = inputs(T, V, D, dt, 6, cuda)
    bounds = [10, 30, 30, 50, 70, 70, 70, 90, 100]     # pairs (0,4) (1,5) (2,6) (3,7)
    y[30:50] = IGNORE                                  # sequence 2 without labels, 1 and 5 empty
    outside = torch.ones(T, dtype=torch.bool, device=cuda)
    outside[10:100] = False
    ref = torch.randn(8, generator=g).to(cuda)
    empty_pair = 1
    ref_bad = ref.clone()
    ref_bad[empty_pair] = ref_bad[empty_pair + 4] = math.nan
    for options in OPTIONS:
        for reduction in ("mean", "none"):
            dloss = None
            if reduction == "none":
                dloss = torch.rand(4, generator=g).to(cuda)
                dloss[empty_pair] = math.nan
            r = preference(h, w, y, bounds, ref, reduction=reduction, dloss=dloss, **options)
            got = losses.preference_step(h, w, y, torch.tensor(bounds, device=cuda), ref_logps=ref_bad,
                                         reduction=reduction, dloss=dloss, **own(options))
            check(got, r, dt, f"{options}", 2)
            assert not got.dhidden[outside].any() and float(got.loss[empty_pair]) == 0.0
    # no pair has a labelled row, and none is given
    none = torch.full_like(y, IGNORE)
    got = losses.preference_step(torch.full_like(h, math.nan), w, none, torch.tensor(bounds, device=cuda))
    assert float(got.reduced) == 0.0 and not got.loss.any() and not got.dhidden.any() and not got.dweight.any()
    got = losses.preference_step(h, w, y, torch.tensor([0], device=cuda))
    assert got.loss.shape == (0,) and float(got.reduced) == 0.0 and not got.dhidden.any() and not got.dweight.any()


@pytest.mark.parametrize("kind", TYPES)
def test_preference_offsets_that_do_not_ascend(losses, cuda, kind):
    """They are not followed: everything becomes NaN, and the next call is right."""
    dt = TYPES[kind]
    h, w, y, _ = inputs(60, 300, 40, dt, 7, cuda, masked=0.2)
    there = y != IGNORE
    good = losses.preference_step(h, w, y, torch.tensor([0, 10, 60], device=cuda))
    for bounds in ([0, 61, 61], [-1, 10, 60], [0, 30, 20], [2 ** 40, 5, 60], [0, -2 ** 62, 60], [0, 10, 2 ** 62]):
        offsets = torch.tensor(bounds, device=cuda)
        for got in (losses.preference_step(h, w, y, offsets), losses.preference_forward(h, w, y, offsets),
                    losses.preference_backward(h, w, y, good.lse, good.row_logps, good.slopes, offsets)):
            if got.loss is not None:
                assert bool(got.loss.isnan().all()) and bool(got.reduced.isnan())
                assert bool(got.logps.isnan().all()) and bool(got.slopes.isnan().all())
                for rows in (got.lse, got.row_logps):
                    assert bool(rows[there].isnan().all()) and not rows[~there].any()
                assert not got.counts.any()
            if got.dhidden is not None:
                assert bool(got.dhidden[there].isnan().all()) and not got.dhidden[~there].any()
                assert bool(got.dweight.isnan().all())
    again = losses.preference_step(h, w, y, torch.tensor([0, 10, 60], device=cuda))
    assert all(torch.equal(a, b) for a, b in zip(again, good))


def test_preference_many_pairs(losses, cuda):
    """More pairs than the kernel has blocks, and more offsets than a block has threads."""
    T, P, V, D = 4000, 1500, 300, 32
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 9, cuda, masked=0.2)
    bounds = pairs_of(T, P, g)
    ref = -5.0 * torch.rand(2 * P, generator=g).to(cuda)
    for reduction in ("mean", "none"):
        dloss = torch.rand(P, generator=g).to(cuda) if reduction == "none" else None
        r = preference(h, w, y, bounds, ref, reduction=reduction, dloss=dloss)
        got = losses.preference_step(h, w, y, torch.tensor(bounds, device=cuda), ref_logps=ref, reduction=reduction,
                                     dloss=dloss)
        check(got, r, torch.bfloat16)


def test_preference_saturates(losses, cuda):
    """Log-ratios far beyond what an exponential of fp32 holds."""
    T, V, D = 200, 300, 32
    h, w, y, g = inputs(T, V, D, torch.float32, 10, cuda)
    bounds = [0, 50, 100, 150, 200]
    for sign in (1.0, -1.0):
        ref = torch.tensor([-9000.0, 50.0, 9000.0, 0.0], device=cuda) * sign
        for options in (dict(), dict(smoothing=0.2)):
            r = preference(h, w, y, bounds, ref, beta=1.0, **options)
            got = losses.preference_step(h, w, y, torch.tensor(bounds, device=cuda), ref_logps=ref, beta=1.0, **options)
            check(got, r, torch.float32, f"{sign} {options}")


@pytest.mark.parametrize("kind", TYPES)
def test_no_rows(losses, cuda, kind):
    dt = TYPES[kind]
    h, w = torch.empty(0, 40, dtype=dt, device=cuda), torch.ones(300, 40, dtype=dt, device=cuda)
    y, none = torch.empty(0, dtype=torch.int64, device=cuda), torch.empty(0, device=cuda)
    got = losses.policy_step(h, w, y, none, none)
    assert got.loss.shape == (0,) and float(got.reduced) == 0.0 and not got.dweight.any()
    got = losses.preference_step(h, w, y, torch.zeros(5, dtype=torch.int64, device=cuda))
    assert got.loss.shape == (2,) and not got.loss.any() and float(got.reduced) == 0.0 and not got.dweight.any()


def both(losses, T, V, D, dt, seed, device, masked=0.2):
    """[(step, forward, backward, arguments, further arguments of the backward call, reference)]"""
    h, w, y, g = inputs(T, V, D, dt, seed, device, masked)
    old, adv, ref = sampled(h, w, y, g, still=0.3)
    bounds = pairs_of(T, 3, g)
    offsets = torch.tensor(bounds, device=device)
    return [(losses.policy_step, losses.policy_forward, losses.policy_backward, (h, w, y, old, adv),
             dict(ref_logps=ref, kl_weight=0.0), (), lambda **m: policy(h, w, y, old, adv, **m)),
            (losses.preference_step, losses.preference_forward, losses.preference_backward, (h, w, y, offsets),
             dict(nll_weight=0.1), (offsets,), lambda **m: preference(h, w, y, bounds, nll=0.1, **m))]


@pytest.mark.parametrize("T,V,D", [(3, 1000, 72), (20, 1001, 200), (200, 1000, 72), (1200, 3000, 64), (8200, 21000, 64)])
@pytest.mark.parametrize("kind", TYPES)
def test_backward_alone_equals_step(losses, cuda, kind, T, V, D):
    dt = TYPES[kind]
    if kind == "fp32" and T > 8000:
        T, V = 4100, 13000
    for step, forward, backward, args, more, extra, _ in both(losses, T, V, D, dt, 21, cuda):
        for reduction in ("mean", "none"):
            whole = step(*args, reduction=reduction, grad_scale=0.5, **more)
            first = forward(*args, reduction=reduction, **more)
            for name in ("loss", "reduced", "logps", "slopes", "lse", "row_logps", "counts"):
                a, b = getattr(whole, name), getattr(first, name)
                assert a is None and b is None or torch.equal(a, b), name
            saved = (first.lse, first.row_logps, first.slopes)
            then = backward(*args[:3], *saved, *extra, reduction=reduction, grad_scale=0.5)
            assert torch.equal(then.dhidden, whole.dhidden) and torch.equal(then.dweight, whole.dweight)
            for left in ("dhidden", "dweight"):
                then = backward(*args[:3], *saved, *extra, reduction=reduction, grad_scale=0.5, **{left: False})
                assert getattr(then, left) is None
                if left == "dhidden":
                    assert torch.equal(then.dweight, whole.dweight)
                else:       # summed in other parts where dweight's tiles leave it the machine
                    a, b = then.dhidden.double(), whole.dhidden.double()
                    assert float((a - b).norm()) <= 2 * (2.0 ** -8 if kind == "bf16" else 2.0 ** -20) * float(b.norm())


@pytest.mark.parametrize("kind", TYPES)
def test_gradients_of_the_reduced_loss(losses, cuda, kind):
    """dloss of one value, grad_scale, accumulation, strided outputs."""
    dt, T, V, D = TYPES[kind], 300, 515, 67
    scale = torch.tensor(0.7, device=cuda)
    for step, _, _, args, more, _, exact in both(losses, T, V, D, dt, 22, cuda):
        r = exact(dloss=0.7, grad_scale=3.0)
        for pad in (0, 5):
            dh, dh_buf = empty_matrix(T, D, dt, cuda, pad)
            dw, dw_buf = empty_matrix(V, D, dt, cuda, pad)
            got = step(*args, dloss=scale, grad_scale=3.0, dhidden=dh, dweight=dw, **more)
            check(got, r, dt, f"{kind} {pad}")
            gaps_untouched(dh_buf, T, D, pad)
            gaps_untouched(dw_buf, V, D, pad)
        before = torch.randn(V, D, device=cuda).to(dt)
        dw = before.clone()
        step(*args, dloss=scale, grad_scale=3.0, dweight=dw, accumulate=True, **more)
        unit = 2.0 ** -24 if kind == "fp32" else 2.0 ** -8
        sum_ = before.double() + r["dweight"]
        off = (dw.double() - sum_).abs()
        alone = step(*args, dloss=scale, grad_scale=3.0, **more).dweight.double()
        # as far as the gradient alone, which is rounded too, and one rounding
        assert bool((off <= (alone - r["dweight"]).abs() + unit * 1.01 * (alone.abs() + sum_.abs()) + 1e-7).all())


@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("kind", TYPES)
def test_strides_and_alignment(losses, cuda, kind, pad, offset):
    """The label's logit is summed from the caller's rows, however they lie."""
    dt, T, V, D = TYPES[kind], 70, 315, 205
    for step, _, _, args, more, _, exact in both(losses, T, V, D, dt, 23, cuda):
        h, w = matrix(args[0], cuda, pad, offset, "hidden"), matrix(args[1], cuda, pad, offset, "weight")
        check(step(h, w, *args[2:], **more), exact(), dt, f"{kind} {pad} {offset}", 2)


def test_label_logits_are_rounded_not_truncated(losses, cuda):
    """Rows whose label has a large logit, which the tensor cores' sums truncate: the mean error
    of many rows. The label's logit is a sum of 32 * 8 chains of three products each and eight
    halvings, each addition off by half a step of 2^-24 of a partial sum at most, in either
    direction; over 2048 rows those even out to a small part of the bound of one row, 11 2^-24
    times the sum of |h w| < 40 (4e-7 as mean where it were all of one sign). Truncation alone
    would make the mean larger than 2e-6."""
    T, V, D = 2048, 5000, 768
    g = torch.Generator().manual_seed(24)
    w = torch.randn(V, D, generator=g) * 0.6 / math.sqrt(D)
    y = torch.randint(0, V, (T,), generator=g)
    h = torch.randn(T, D, generator=g) + 25.0 * w[y]
    h, w, y = h.bfloat16().to(cuda), w.bfloat16().to(cuda), y.to(cuda)
    got = losses.policy_forward(h, w, y, torch.zeros(T, device=cuda), torch.ones(T, device=cuda))
    off = got.logps.double() - exact_logps(h, w, y)
    assert abs(float(off.mean())) < 1e-6


def test_equal_inputs_give_equal_bits(losses, cuda):
    for step, _, _, args, more, _, _ in both(losses, 1500, 9000, 72, torch.bfloat16, 25, cuda):
        first = step(*args, **more)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        a, b = step(*args, stream=side, **more), step(*args, **more)
        torch.cuda.current_stream().wait_stream(side)
        for again in (a, b):
            for x, z in zip(first, again):
                assert x is None and z is None or torch.equal(x, z)


@pytest.mark.parametrize("kind", TYPES)
def test_in_a_graph(losses, cuda, kind):
    dt = TYPES[kind]
    for T, n in ((700, 0), (700, 1), (20, 0), (20, 1)):
        step, _, _, args, more, _, _ = both(losses, T, 2000, 72, dt, 26, cuda)[n]
        args = tuple(t.clone() for t in args)
        step(*args, **more)
        torch.cuda.synchronize()
        graphs, outs = [], []
        for _ in range(2):                          # two graphs of one pool share their workspaces
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, pool=graphs[0].pool() if graphs else None):
                outs.append(step(*args, **more))
            graphs.append(graph)
        for seed in (27, 28):
            _, _, _, new, _, _, exact = both(losses, T, 2000, 72, dt, seed, cuda)[n]
            for a, b in zip(args, new):
                a.copy_(b)
            for graph, out in zip(graphs, outs):
                graph.replay()
                torch.cuda.synchronize()
                check(out, exact(), dt, f"{T} {seed}", parts_of(dt, T))


def test_another_stream(losses, cuda, monkeypatch):
    """A raw handle keeps the workspace and the results while its work is queued."""
    T, V, D = 300, 3000, 128
    for n, name in enumerate(("policy", "preference")):
        step, _, _, args, more, _, exact = both(losses, T, V, D, torch.bfloat16, 29, cuda)[n]
        seen, call = [], getattr(losses.abi, f"zero_{name}_step")

        def spy(p, q, stream=None):
            seen.append((p.workspace, p.workspace_bytes))
            return call(p, q, stream)

        monkeypatch.setattr(losses.abi, f"zero_{name}_step", spy)
        side = torch.cuda.Stream()
        step(*args, **more)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)
        got = step(*args, stream=side.cuda_stream, **more)
        at, size = seen[-1]
        fresh = [torch.empty(k, dtype=torch.uint8, device=cuda) for k in (size, size // 2, 4096) for _ in range(4)]
        assert not side.query(), "the work is still queued"
        assert all(apart(t, at, size) for t in fresh)
        side.synchronize()
        check(got, exact(), torch.bfloat16)


@pytest.mark.parametrize("kind", TYPES)
def test_a_wait_that_runs_out(losses, cuda, kind):
    """As for the other losses: all that the call writes is NaN but what belongs to empty rows."""
    abi, dt = losses.abi, TYPES[kind]

    def nan(x):
        return bool(x.isnan().all())

    for step, forward, backward, args, more, extra, _ in both(losses, 600, 9000, 72, dt, 30, cuda):
        there = args[2] != IGNORE
        rows = step is losses.policy_step
        good = step(*args, **more)
        for passes, call, a, m in ((1, forward, args, more), (1, step, args, more), (2, step, args, more),
                                   (3, step, args, more), (2, step, args, dict(more, dhidden=False)),
                                   (2, backward, (*args[:3], good.lse, good.row_logps, good.slopes, *extra), {})):
            torch.cuda.synchronize()
            abi.zero_debug_withhold_head_loss(passes, 50_000_000)
            r = call(*a, **m)
            torch.cuda.synchronize()
            if r.loss is not None:
                assert nan(r.reduced) and nan(r.lse[there]) and nan(r.row_logps[there])
                for x in (r.loss, r.logps, r.slopes):
                    assert nan(x[there] if rows else x)
                    assert not rows or not x[~there].any()
            if r.dhidden is not None:
                assert nan(r.dhidden[there]) and not r.dhidden[~there].any()
            assert r.dweight is None or nan(r.dweight)
        again = step(*args, **more)
        for a, b in zip(again, good):
            assert a is None and b is None or torch.equal(a, b)


@pytest.mark.parametrize("op", ["policy", "preference"])
def test_gradient_against_differences(losses, cuda, op):
    """The reduced loss's central difference along a direction, in fp32 storage, against the
    gradient along it. With steps of t = 2^-6 the difference is off by the third derivative,
    O(t^2) of the gradient's size, and by twice the loss's own error over 2 t: 2^-20 of a
    loss near one, so 2^-15 absolute; 2 % and 1e-3 hold both."""
    T, V, D = 60, 200, 48
    h, w, y, g = inputs(T, V, D, torch.float32, 31, cuda, masked=0.2)
    old, adv, ref = sampled(h, w, y, g)
    offsets = torch.tensor([0, 20, 30, 41, 60], device=cuda)

    def call(a, b, name):
        if op == "policy":
            # no clipping: the bounds are a kink
            return getattr(losses, f"policy_{name}")(a, b, y, old, adv, ref_logps=ref, clip=(0.99, 50.0), kl_weight=0.1)
        return getattr(losses, f"preference_{name}")(a, b, y, offsets, beta=0.2, nll_weight=0.3)

    r = call(h, w, "step")
    t = 2.0 ** -6
    for what in ("hidden", "weight"):
        for _ in range(3):
            x = h if what == "hidden" else w
            grad = r.dhidden if what == "hidden" else r.dweight
            d = torch.randn(x.shape, generator=g).to(cuda)
            d = 0.5 * d / d.norm() + 0.5 * grad / grad.norm()
            ends = [call(*((x + s * t * d, w) if what == "hidden" else (h, x + s * t * d)), "forward").reduced.double()
                    for s in (1, -1)]
            along = float((grad.double() * d.double()).sum())
            assert float(ends[0] - ends[1]) / (2 * t) == pytest.approx(along, rel=2e-2, abs=1e-3)


def test_autograd(losses, cuda):
    T, V, D = 200, 500, 64
    h, w, y, g = inputs(T, V, D, torch.float32, 32, cuda, masked=0.2)
    old, adv, ref = sampled(h, w, y, g)
    bounds = pairs_of(T, 3, g)
    offsets = torch.tensor(bounds, device=cuda)
    row, pair = torch.rand(T, generator=g).to(cuda), torch.rand(3, generator=g).to(cuda)
    for reduction in ("mean", "sum", "none"):
        for name, dloss in (("policy", row), ("preference", pair)):
            a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
            if name == "policy":
                loss = losses.linear_policy(a, b, y, old, adv, ref, (0.1, 0.2), 0.05, reduction)
                r = policy(h, w, y, old, adv, ref, (0.1, 0.2), 0.05, reduction, dloss if reduction == "none" else 2.0)
            else:
                loss = losses.linear_preference(a, b, y, offsets, beta=0.3, reduction=reduction)
                r = preference(h, w, y, bounds, beta=0.3, reduction=reduction,
                               dloss=dloss if reduction == "none" else 2.0)
            total = (loss * dloss).sum() if reduction == "none" else 2.0 * loss
            gh, gw = torch.autograd.grad(total, (a, b), create_graph=True)
            check(losses.LogpLosses(*[None] * 7, gh.detach(), gw.detach()), r, torch.float32,
                  f"{name} {reduction}")
            with pytest.raises(RuntimeError, match="no second derivatives"):
                gh.square().sum().backward()
            only, = torch.autograd.grad(losses.linear_policy(h, b, y, old, adv) if name == "policy" else
                                        losses.linear_preference(h, b, y, offsets), b)
            assert only.shape == w.shape


@pytest.mark.parametrize("T", [20, 500])
def test_autograd_in_a_graph(losses, cuda, T):
    """A tied model's forward and backward pass, captured while an eager graph of the same storage lives:
    replays on new values give what eager calls give."""
    from zero_sharded_optimizer_gb300.embedding import embedding
    V, D = 1500, 96
    _, w, y, g = inputs(T, V, D, torch.bfloat16, 34, cuda, masked=0.2)
    ids = torch.randint(V, (T,), generator=g).to(cuda)
    old, adv = torch.full((T,), -7.0, device=cuda), torch.randn(T, generator=g).to(cuda)
    offsets = torch.tensor([0, T // 5, T // 2, T - 3, T], device=cuda)

    def gradients():
        wte = w.detach().requires_grad_()
        x = embedding(ids, wte)
        total = losses.linear_policy(x, wte, y, old, adv) + losses.linear_preference(x, wte, y, offsets, beta=0.5)
        return total.detach(), *torch.autograd.grad(total, wte)

    leaf = w.detach().requires_grad_()
    alive = losses.linear_policy(embedding(ids, leaf), leaf, y, old, adv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gradients()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gradients()
    assert alive.requires_grad
    for _ in range(2):
        w.copy_(torch.randn(V, D, generator=g))
        ids.copy_(torch.randint(V, (T,), generator=g))
        adv.copy_(torch.randn(T, generator=g))
        offsets[1:4] = torch.randint(T + 1, (3,), generator=g).sort().values.to(cuda)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, gradients()):
            assert torch.equal(a, b)


def test_refusals_of_the_binding(losses, cuda):
    h, w, y, g = inputs(12, 100, 32, torch.bfloat16, 33, cuda)
    old = torch.zeros(12, device=cuda)
    offsets = torch.tensor([0, 6, 12], device=cuda)
    for a, b in ((old.double(), old), (old, old.cpu()), (None, old), (old, None)):
        with pytest.raises(TypeError):
            losses.policy_forward(h, w, y, a, b)
    for a, b in ((old[:5], old), (old, old.expand(2, 12)), (old.view(3, 4), old.view(4, 3))):
        with pytest.raises(ValueError):
            losses.policy_forward(h, w, y, a, b)
    with pytest.raises(ValueError):
        losses.policy_forward(h, w, y, old, old, kl_weight=0.1)
    for clip in (-0.1, (0.2, -0.1), (math.nan, 0.2), (0.2, math.inf)):
        with pytest.raises(RuntimeError):
            losses.policy_forward(h, w, y, old, old, clip=clip)
    with pytest.raises(RuntimeError):
        losses.policy_step(h, w, y, old, old, dhidden=False, dweight=False)
    with pytest.raises(RuntimeError):
        losses.policy_step(h, w, y, old, old, dhidden=h)
    with pytest.raises(TypeError):
        losses.policy_forward(h, w, None, old, old)
    for bad in (offsets[:2], offsets.view(1, 3), [0, 6, 12]):
        with pytest.raises(ValueError):
            losses.preference_forward(h, w, y, bad)
    with pytest.raises(TypeError):
        losses.preference_forward(h, w, y, offsets.int())
    for batch in (h.view(3, 4, 32), h, h.view(1, 2, 6, 32)):
        with pytest.raises(ValueError):
            losses.preference_forward(batch, w, y)
    with pytest.raises(ValueError):
        losses.preference_forward(h, w, y, offsets, kind="hinge")
    with pytest.raises(ValueError):
        losses.preference_forward(h, w, y, offsets, ref_logps=torch.zeros(3, device=cuda))
    with pytest.raises(ValueError):
        losses.preference_step(h, w, y, offsets, reduction="none", dloss=old)
    for more in (dict(smoothing=1.5), dict(smoothing=0.1, kind="squared"), dict(beta=math.inf), dict(margin=math.nan),
                 dict(nll_weight=math.inf)):
        with pytest.raises(RuntimeError):
            losses.preference_forward(h, w, y, offsets, **more)
