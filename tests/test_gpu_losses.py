"""The vocabulary losses on the GPU against their definition in 64 bits, within
bounds derived from their arithmetic (loss_util). Matrices sit between guard
regions, with sentinels in the gaps of their rows: a read past a row's end
brings a NaN into the result, a write past it is found afterwards."""

import math

import pytest
import torch

import parity_util
from loss_util import IGNORE, bounds, check, reference

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def losses(abi, cuda):
    from zero_sharded_optimizer_gb300 import losses as module
    return module


def matrix(values, device, pad=0, offset=0, what="matrix"):
    """`values` in a guarded buffer of rows `pad` elements apart."""
    n, d = values.shape
    buf = parity_util.guarded_empty(max(n * (d + pad), 1), values.dtype, device, offset, what)
    m = torch.as_strided(buf, (n, d), (d + pad, 1), buf.storage_offset())
    m.copy_(values)
    return m


def empty_matrix(n, d, dtype, device, pad=0, offset=0, what="output"):
    buf = parity_util.guarded_empty(max(n * (d + pad), 1), dtype, device, offset, what)
    return torch.as_strided(buf, (n, d), (d + pad, 1), buf.storage_offset()), buf


def gaps_untouched(buf, n, d, pad):
    """The gaps between an output's rows still hold the sentinel."""
    if pad == 0 or n < 2:
        return
    bits = buf.view(torch.int32 if buf.dtype == torch.float32 else torch.int16)
    s = 0x7FA5A5A5 if buf.dtype == torch.float32 else 0x7FA5
    assert bool((bits[:n * (d + pad)].view(n, d + pad)[:, d:] == s).all())


def inputs(T, V, D, dtype, seed, device, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    labels = torch.randint(0, V, (T,), generator=g)
    w = torch.randn(V, D, generator=g) * 0.7 / math.sqrt(D)
    h = torch.randn(T, D, generator=g) + 4.0 * torch.rand(T, 1, generator=g) * w[labels]
    labels[torch.rand(T, generator=g) < masked] = IGNORE
    return h.to(dtype).to(device), w.to(dtype).to(device), labels.to(device), g


def teacher(T, V, K, g, device, absent=0.0):
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)]) if T else \
        torch.zeros(0, K, dtype=torch.int64)
    logits = 3.0 * torch.randn(T, K, generator=g)
    ids[torch.rand(T, K, generator=g) < absent] = -1
    return ids.to(device), logits.to(device)


# One to a few tiles in each direction, on and around their edges.
SIZES = [(1, 1, 1), (1, 257, 64), (2, 255, 7), (3, 256, 8), (127, 300, 65), (128, 512, 64),
         (129, 513, 128), (300, 1000, 96), (257, 2049, 192), (64, 700, 513), (130, 259, 1032)]


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("kind", TYPES)
def test_xent_step(losses, cuda, kind, T, V, D):
    dt = TYPES[kind]
    h, w, y, _ = inputs(T, V, D, dt, 1000 + T + V + D, cuda, masked=0.2 if T > 2 else 0.0)
    h, w = matrix(h, cuda), matrix(w, cuda)
    for reduction in ("mean", "sum"):
        r = reference(h, w, y, reduction=reduction)
        got = losses.xent_step(h, w, y, reduction=reduction)
        check(got, r, dt, f"{kind} {reduction}")


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 0), (8, 8), (5, 3), (5, 0), (13, 0)])
@pytest.mark.parametrize("kind", TYPES)
def test_strides_and_alignment(losses, cuda, kind, pad, offset):
    dt = TYPES[kind]
    for T, V, D in [(70, 515, 72), (33, 300, 67), (40, 300, 201)]:
        h, w, y, g = inputs(T, V, D, dt, 7 + pad + offset, cuda, masked=0.3)
        h = matrix(h, cuda, pad, offset, "hidden")
        w = matrix(w, cuda, pad, offset, "weight")
        dh, dh_buf = empty_matrix(T, D, dt, cuda, pad, offset, "dhidden")
        dw, dw_buf = empty_matrix(V, D, dt, cuda, pad, offset, "dweight")
        dloss = torch.rand(T, generator=g).to(cuda)
        got = losses.xent_step(h, w, y, reduction="none", dloss=dloss, dhidden=dh, dweight=dw)
        check(got, reference(h, w, y, reduction="none", dloss=dloss), dt, f"{kind} {pad} {offset}")
        gaps_untouched(dh_buf, T, D, pad)
        gaps_untouched(dw_buf, V, D, pad)


@pytest.mark.parametrize("kind", TYPES)
def test_empty_rows_are_not_read(losses, cuda, kind):
    """Rows without a target hold NaN and infinities, in the hidden states and
    in dloss; an ignore index inside the vocabulary; labels out of range."""
    dt = TYPES[kind]
    T, V, D = 200, 777, 80
    h, w, y, g = inputs(T, V, D, dt, 5, cuda)
    gone = torch.rand(T, generator=g).to(cuda) < 0.5
    for mark, ignore in [(IGNORE, IGNORE), (0, 0), (V, IGNORE), (-1, IGNORE), (2 ** 40, IGNORE)]:
        labels = torch.where(gone, mark, y.clamp(min=1))
        bad = h.clone()
        bad[gone] = math.nan
        bad[torch.nonzero(gone)[::2, 0]] = math.inf
        dloss = torch.where(gone, math.nan, torch.rand(T, generator=g).to(cuda))
        r = reference(bad, w, labels, ignore_index=ignore, reduction="none", dloss=dloss)
        got = losses.xent_step(bad, w, labels, ignore_index=ignore, reduction="none", dloss=dloss)
        check(got, r, dt, f"{kind} {mark}")
        assert bool((got.loss[gone] == 0).all()) and bool((got.dhidden[gone] == 0).all())
        mean = losses.xent_forward(bad, w, labels, ignore_index=ignore)
        assert float(mean.reduced) == pytest.approx(float(got.loss.double().sum()) / int((~gone).sum()), rel=1e-6)


@pytest.mark.parametrize("kind", TYPES)
def test_no_row_has_a_target(losses, cuda, kind):
    dt = TYPES[kind]
    h, w, _, _ = inputs(5, 300, 40, dt, 3, cuda)
    y = torch.full((5,), IGNORE, device=cuda)
    got = losses.xent_step(torch.full_like(h, math.nan), w, y)
    assert float(got.reduced) == 0.0 and not got.loss.any()
    assert not got.dhidden.any() and not got.dweight.any()
    ids = torch.full((5, 3), -1, device=cuda)
    got = losses.distill_step(torch.full_like(h, math.nan), w, ids, torch.zeros(5, 3, device=cuda))
    assert float(got.reduced) == 0.0 and not got.dhidden.any() and not got.dweight.any()


@pytest.mark.parametrize("kind", TYPES)
def test_no_rows(losses, cuda, kind):
    dt = TYPES[kind]
    w = torch.ones(300, 40, dtype=dt, device=cuda)
    got = losses.xent_step(torch.empty(0, 40, dtype=dt, device=cuda), w,
                           torch.empty(0, dtype=torch.int64, device=cuda))
    assert got.loss.shape == (0,) and got.dhidden.shape == (0, 40)
    assert float(got.reduced) == 0.0 and not got.dweight.any()
    before = torch.randn(300, 40, device=cuda).to(dt)
    dw = before.clone()
    losses.xent_step(torch.empty(0, 40, dtype=dt, device=cuda), w,
                     torch.empty(0, dtype=torch.int64, device=cuda), dweight=dw, accumulate=True)
    assert torch.equal(dw, before)


@pytest.mark.parametrize("kind", TYPES)
def test_no_rows_and_a_weight_that_is_not_trained(losses, cuda, kind):
    """The gradient of the hidden states alone, of an empty batch."""
    dt = TYPES[kind]
    h = torch.empty(0, 40, dtype=dt, device=cuda, requires_grad=True)
    w = torch.ones(300, 40, dtype=dt, device=cuda)
    y = torch.empty(0, dtype=torch.int64, device=cuda)
    ids, logits = torch.empty(0, 3, dtype=torch.int64, device=cuda), torch.empty(0, 3, device=cuda)
    for loss in (losses.linear_cross_entropy(h, w, y), losses.linear_distillation(h, w, ids, logits, 2.0)):
        got, = torch.autograd.grad(loss, h)
        assert float(loss.detach()) == 0.0 and got.shape == (0, 40)
    got = losses.xent_step(h.detach(), w, y, dweight=False)
    assert got.dhidden.shape == (0, 40) and got.dweight is None and float(got.reduced) == 0.0


@pytest.mark.parametrize("kind", TYPES)
def test_no_rows_of_distillation_mixed_with_labels(losses, cuda, kind):
    dt = TYPES[kind]
    h, w = torch.empty(0, 40, dtype=dt, device=cuda), torch.ones(300, 40, dtype=dt, device=cuda)
    y = torch.empty(0, dtype=torch.int64, device=cuda)
    ids, logits = torch.empty(0, 3, dtype=torch.int64, device=cuda), torch.empty(0, 3, device=cuda)
    got = losses.distill_step(h, w, ids, logits, temperature=2.0, labels=y, alpha=0.5)
    assert float(got.reduced) == 0.0 and got.loss.shape == (0,) and got.dhidden.shape == (0, 40)
    assert not got.dweight.any()


@pytest.mark.parametrize("kind", TYPES)
def test_a_row_that_is_not_finite_shows(losses, cuda, kind):
    """A NaN in a row with a target makes that row's loss NaN, and no other's."""
    dt = TYPES[kind]
    h, w, y, _ = inputs(140, 600, 72, dt, 11, cuda)
    h[3, 5] = math.nan
    got = losses.xent_forward(h, w, y, reduction="none")
    assert math.isnan(float(got.loss[3]))
    rest = torch.arange(140, device=cuda) != 3
    assert bool(torch.isfinite(got.loss[rest]).all())


@pytest.mark.parametrize("K,absent", [(1, 0.0), (5, 0.4), (32, 0.0), (64, 0.2), (200, 0.1)])
@pytest.mark.parametrize("kind", TYPES)
def test_distill_step(losses, cuda, kind, K, absent):
    dt = TYPES[kind]
    for T, V, D, tau, alpha, with_labels in [(150, 1000, 96, 2.0, 0.5, True), (37, 300, 33, 1.0, 1.0, False),
                                             (130, 513, 64, 0.5, 0.25, True), (64, 400, 64, 4.0, 1.0, True),
                                             (20, 400, 64, 4.0, 0.0, True)]:
        h, w, y, g = inputs(T, V, D, dt, K + T, cuda, masked=0.3)
        ids, logits = teacher(T, V, K, g, cuda, absent)
        ids[::9] = -1
        labels = y if with_labels else None
        for reduction in ("mean", "none"):
            dloss = torch.rand(T, generator=g).to(cuda) if reduction == "none" else None
            more = dict(tau=tau, alpha=alpha, reduction=reduction, dloss=dloss)
            r = reference(h, w, labels, ids, logits, **more)
            got = losses.distill_step(h, w, ids, logits, temperature=tau, labels=labels, alpha=alpha,
                                      reduction=reduction, dloss=dloss)
            check(got, r, dt, f"{kind} {T} {reduction}")


@pytest.mark.parametrize("kind", TYPES)
def test_teacher_entries_at_their_edges(losses, cuda, kind):
    """Equal ids, ids out of range, logits of minus infinity and of the type's
    lowest value, the label inside and outside the list, ids at tile edges."""
    dt = TYPES[kind]
    T, V, D, K = 140, 700, 64, 6
    h, w, y, g = inputs(T, V, D, dt, 21, cuda)
    ids, logits = teacher(T, V, K, g, cuda)
    lowest = torch.finfo(torch.float32).min
    ids[0] = 7                                    # one id six times
    ids[1] = torch.tensor([255, 256, 511, 512, 699, 0])
    ids[2] = torch.tensor([-1, V, 2 ** 33, 5, 5, 9])
    logits[3] = -math.inf                         # all absent, but a label
    logits[4, 1:] = -math.inf
    logits[5] = lowest                            # uniform
    logits[6, 1:] = lowest                        # one entry has everything
    ids[7, 0] = y[7]
    ids[8, :3] = y[8]
    y[9] = IGNORE
    y[10] = IGNORE
    ids[10] = -1                                  # neither: empty
    h[10] = math.nan
    for labels, alpha in [(y, 0.5), (None, 1.0)]:
        bad = h.clone()
        if labels is None:
            bad[3] = math.nan
        r = reference(bad, w, labels, ids, logits, tau=1.5, alpha=alpha, reduction="sum")
        got = losses.distill_step(bad, w, ids, logits, temperature=1.5, labels=labels, alpha=alpha,
                                  reduction="sum")
        check(got, r, dt, f"{kind} {alpha}")


@pytest.mark.parametrize("tau", [0.5, 0.25, 1.0])
@pytest.mark.parametrize("logits_type", TYPES)
@pytest.mark.parametrize("kind", TYPES)
def test_teacher_logits_at_the_end_of_the_range(losses, cuda, kind, logits_type, tau):
    """Logits near the type's lowest and largest value, which the division by a temperature
    below one takes out of fp32: they are present, and only -inf is absent."""
    dt, lt = TYPES[kind], TYPES[logits_type]
    T, V, D, K = 12, 300, 64, 5
    h, w, y, g = inputs(T, V, D, dt, 22, cuda)
    ids, logits = teacher(T, V, K, g, cuda)
    logits = logits.to(lt)
    lowest = torch.finfo(lt).min
    logits[0] = lowest                            # uniform
    logits[1, 1:] = lowest                        # one entry has everything
    logits[2], logits[2, 0] = lowest, -math.inf   # four, uniform
    logits[3] = -lowest                           # uniform
    logits[4], logits[4, :2] = lowest, -lowest    # two share it
    logits[5] = -math.inf                         # absent
    logits[6, 1:] = 0.9 * lowest
    for labels, alpha in [(y, 0.5), (None, 1.0)]:
        r = reference(h, w, labels, ids, logits, tau=tau, alpha=alpha, reduction="sum")
        got = losses.distill_step(h, w, ids, logits, temperature=tau, labels=labels, alpha=alpha, reduction="sum")
        check(got, r, dt, f"{kind} {alpha}", parts=2)


def test_entries_of_equal_id_are_entries_of_their_own(losses, cuda):
    """The loss that the formula gives for them, written out for one row: six entries of one id
    and equal logits have q = 1/6 each, so log q is -log 6 in every term."""
    V, D, K, tau = 40, 16, 6, 2.0
    h, w, _, _ = inputs(1, V, D, torch.float32, 23, cuda)
    z = (h.double() @ w.double().T)[0] / tau
    got = losses.distill_step(h, w, torch.full((1, K), 7, device=cuda), torch.zeros(1, K, device=cuda), temperature=tau)
    want = tau * tau * (-math.log(K) - float(z[7]) + float(torch.logsumexp(z, 0)))
    assert float(got.loss[0]) == pytest.approx(want, rel=1e-5, abs=1e-5)
    p = torch.softmax(z, 0)
    p[7] -= 1.0                             # the six add their q
    assert torch.allclose(got.dhidden[0].double(), tau * (p @ w.double()), rtol=1e-4, atol=1e-6)


def test_distill_many_entries(losses, cuda):
    T, V, D, K = 9, 5000, 64, 1024
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 2, cuda)
    ids, logits = teacher(T, V, K, g, cuda)
    r = reference(h, w, y, ids, logits, tau=2.0, alpha=0.5)
    check(losses.distill_step(h, w, ids, logits, temperature=2.0, labels=y, alpha=0.5), r,
          torch.bfloat16)


@pytest.mark.parametrize("K", [184, 187, 188, 191, 192, 255])
def test_distill_many_rows_around_what_a_block_holds(losses, cuda, K):
    """Lists of K entries on both sides of what a block of 16 rows keeps in shared memory, and
    enough rows (16 for each of 152 SMs) that a block would take as many."""
    T, V, D = 2435, 300, 16
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 300 + K, cuda, masked=0.1)
    ids, logits = teacher(T, V, K, g, cuda, absent=0.1)
    r = reference(h, w, y, ids, logits, tau=2.0, alpha=0.5)
    check(losses.distill_step(h, w, ids, logits, temperature=2.0, labels=y, alpha=0.5), r, torch.bfloat16)


@pytest.mark.parametrize("kind", TYPES)
def test_backward_alone_equals_step(losses, cuda, kind):
    dt = TYPES[kind]
    T, V, D = 190, 900, 104
    h, w, y, g = inputs(T, V, D, dt, 8, cuda, masked=0.2)
    ids, logits = teacher(T, V, 12, g, cuda, 0.1)
    dloss = torch.tensor(0.37, device=cuda)
    a = losses.xent_step(h, w, y, dloss=dloss, grad_scale=0.5)
    f = losses.xent_forward(h, w, y)
    b = losses.xent_backward(h, w, y, f.lse, dloss=dloss, grad_scale=0.5)
    assert torch.equal(a.loss, f.loss) and torch.equal(a.reduced, f.reduced)
    assert torch.equal(a.dhidden, b.dhidden) and torch.equal(a.dweight, b.dweight)
    check(b, reference(h, w, y, dloss=dloss, grad_scale=0.5), dt)
    a = losses.distill_step(h, w, ids, logits, temperature=2.0, labels=y, alpha=0.3)
    f = losses.distill_forward(h, w, ids, logits, temperature=2.0, labels=y, alpha=0.3)
    b = losses.distill_backward(h, w, ids, logits, f.lse, f.lse_tau, temperature=2.0, labels=y, alpha=0.3)
    assert torch.equal(a.loss, f.loss)
    assert torch.equal(a.dhidden, b.dhidden) and torch.equal(a.dweight, b.dweight)
    # one gradient alone, and equal inputs give equal bits
    only = losses.xent_step(h, w, y, dloss=dloss, grad_scale=0.5, dweight=False)
    again = losses.xent_step(h, w, y, dloss=dloss, grad_scale=0.5, dhidden=False)
    both = losses.xent_step(h, w, y, dloss=dloss, grad_scale=0.5)
    assert only.dweight is None and again.dhidden is None
    assert torch.equal(only.dhidden, both.dhidden) and torch.equal(again.dweight, both.dweight)


@pytest.mark.parametrize("kind", TYPES)
def test_accumulate_adds_with_one_rounding(losses, cuda, kind):
    dt = TYPES[kind]
    T, V, D = 100, 530, 72
    h, w, y, g = inputs(T, V, D, dt, 31, cuda)
    r = reference(h, w, y)
    before = (torch.randn(V, D, generator=g) * 1e-2).to(dt).to(cuda)
    dw = before.clone()
    losses.xent_step(h, w, y, dweight=dw, accumulate=True)
    want = before.double() + r["dweight"]
    unit = 2.0 ** -24 if dt == torch.float32 else 2.0 ** -8
    allowed = bounds(r, dt)["dweight"] + unit * 1.01 * want.abs()
    assert bool(((dw.double() - want).abs() <= allowed).all())


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("kind,T,V,D", [("bf16", 8200, 21000, 64), ("fp32", 4100, 13000, 72)])
def test_accumulate_over_several_pieces(losses, cuda, kind, T, V, D, pad):
    """As above, with dweight's rows in several pieces of the vocabulary, on 16 bytes and off them."""
    dt = TYPES[kind]
    h, w, y, g = inputs(T, V, D, dt, 32, cuda, masked=0.1)
    r = reference(h, w, y)
    before = (torch.randn(V, D, generator=g) * 1e-4).to(dt).to(cuda)
    dw, buf = empty_matrix(V, D, dt, cuda, pad)
    dw.copy_(before)
    got = losses.xent_step(h, w, y, dweight=dw, accumulate=True)
    want = before.double() + r["dweight"]
    unit = 2.0 ** -24 if dt == torch.float32 else 2.0 ** -8
    allowed = bounds(r, dt)["dweight"] + unit * 1.01 * want.abs()
    assert bool(((dw.double() - want).abs() <= allowed).all())
    gaps_untouched(buf, V, D, pad)
    check(got._replace(dweight=None), r, dt)


def test_another_stream(losses, cuda):
    """Inputs made and outputs used on a side stream, named or current."""
    side = torch.cuda.Stream()
    T, V, D = 300, 3000, 128
    h, w, y, _ = inputs(T, V, D, torch.bfloat16, 4, cuda)
    r = reference(h, w, y)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        x = h * 1.0
        got = losses.xent_step(x, w, y)
    side.synchronize()
    check(got, r, torch.bfloat16)
    side.wait_stream(torch.cuda.current_stream())
    got = losses.xent_step(h, w, y, stream=side)
    side.synchronize()
    check(got, r, torch.bfloat16)


def spy_on(monkeypatch, losses, name):
    """The problems passed to the library's call `name`, as (address, bytes) of their workspace."""
    seen, call = [], getattr(losses.abi, name)

    def spy(p, stream=None):
        seen.append((p.workspace, p.workspace_bytes))
        return call(p, stream)

    monkeypatch.setattr(losses.abi, name, spy)
    return seen


def test_a_handle_keeps_its_workspace(losses, cuda, monkeypatch):
    """A stream given as a raw handle: while its work is still queued, no new tensor of the
    current stream gets the workspace."""
    T, V, D = 300, 3000, 128
    h, w, y, _ = inputs(T, V, D, torch.bfloat16, 65, cuda)
    seen = spy_on(monkeypatch, losses, "zero_xent_step")
    for side in (torch.cuda.Stream(), torch.cuda.Stream()):
        losses.xent_step(h, w, y)          # memory to hand out again is there
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)
        got = losses.xent_step(h, w, y, stream=side.cuda_stream)
        at, size = seen[-1]
        fresh = [torch.empty(n, dtype=torch.uint8, device=cuda) for n in (size, size // 2, 4096) for _ in range(4)]
        assert not side.query(), "the work is still queued"
        for t in fresh:
            assert t.data_ptr() + t.numel() <= at or at + size <= t.data_ptr()
        side.synchronize()
        check(got, reference(h, w, y), torch.bfloat16)


def apart(t, at, size):
    return t.data_ptr() + t.numel() * t.element_size() <= at or at + size <= t.data_ptr()


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_memory_that_the_current_stream_still_uses(losses, cuda, monkeypatch, op):
    """A call on another stream gets neither its workspace nor its results from memory whose
    last use is still queued on the current stream; nor does a later call there from results
    that the current stream still reads."""
    T, V, D = 300, 3000, 128
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 67, cuda)
    ids, logits = teacher(T, V, 5, g, cuda)
    args = (h, w, y) if op == "xent" else (h, w, ids, logits)
    step = getattr(losses, op + "_step")
    r = reference(h, w, y) if op == "xent" else reference(h, w, None, ids, logits)
    seen = spy_on(monkeypatch, losses, f"zero_{op}_step")
    side = torch.cuda.Stream()
    step(*args)                            # the sizes that a call asks for
    size = seen[-1][1]
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    freed = []
    for n in (size, V * D * 2, T * D * 2, T * 4, T * 4, T * 4, 4):
        t = torch.empty(n, dtype=torch.uint8, device=cuda)
        t.fill_(1)
        freed.append((t.data_ptr(), n))
        del t
    got = step(*args, stream=side)
    assert not torch.cuda.current_stream().query(), "the memory's last use is still queued"
    for at, n in freed:
        assert seen[-1][0] + size <= at or at + n <= seen[-1][0]
        assert all(apart(t, at, n) for t in got if t is not None)
    side.synchronize()
    check(got, r, torch.bfloat16)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    used = [(t.data_ptr(), t.numel() * t.element_size()) for t in got if t is not None]
    sums = [t.double().sum() for t in got if t is not None]
    del got
    again = step(*args, stream=side)
    assert not torch.cuda.current_stream().query(), "the results' last use is still queued"
    for at, n in used:
        assert seen[-1][0] + size <= at or at + n <= seen[-1][0]
        assert all(apart(t, at, n) for t in again if t is not None)
    side.synchronize()
    check(again, r, torch.bfloat16)
    torch.cuda.synchronize()
    assert [float(x) for x in sums] == [float(t.double().sum()) for t in again if t is not None]


def test_bf16_teacher_logits(losses, cuda):
    """They give the bits of the same values in float32 -- also on a named stream while the
    current one is busy, when they come from work on that stream that is still queued."""
    T, V, D, K = 140, 700, 64, 6
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 68, cuda, masked=0.1)
    ids, logits = teacher(T, V, K, g, cuda, absent=0.1)
    logits = logits.bfloat16()
    more = dict(temperature=2.0, labels=y, alpha=0.5)
    want = losses.distill_step(h, w, ids, logits.float(), **more)
    r = reference(h, w, y, ids, logits.float(), tau=2.0, alpha=0.5)
    got = losses.distill_step(h, w, ids, logits, **more)
    check(got, r, torch.bfloat16)
    torch.cuda.synchronize()
    for side in (torch.cuda.Stream(), torch.cuda.Stream()):
        for stream in (side, side.cuda_stream):
            with torch.cuda.stream(side):
                late = torch.full_like(logits, -50.0)
            side.synchronize()
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
                late.copy_(logits)
            torch.cuda._sleep(400_000_000)
            got = losses.distill_step(h, w, ids, late, stream=stream, **more)
            side.synchronize()
            assert not torch.cuda.current_stream().query(), "nothing of the call waits for the current stream"
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            torch.cuda.synchronize()


def test_the_default_stream_by_its_handles(losses, cuda):
    T, V, D = 70, 500, 64
    h, w, y, _ = inputs(T, V, D, torch.bfloat16, 66, cuda)
    for handle in (0, 1):
        got = losses.xent_step(h, w, y, stream=handle)
        torch.cuda.synchronize()
        check(got, reference(h, w, y), torch.bfloat16)


@pytest.mark.parametrize("T,V,D", [(90, 700, 64), (600, 9000, 72)])
@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("kind", TYPES)
def test_a_wait_that_runs_out(losses, cuda, kind, op, T, V, D):
    """A word that nothing sets: the waits give up at their limit, everything that the call
    writes is NaN (but what belongs to empty rows), and the next call is right."""
    import time
    abi, dt = losses.abi, TYPES[kind]
    h, w, y, g = inputs(T, V, D, dt, 71, cuda, masked=0.2)
    ids, logits = teacher(T, V, 5, g, cuda)
    ids[y == IGNORE] = -1
    there = y != IGNORE
    args = (h, w, y) if op == "xent" else (h, w, ids, logits)
    more = {} if op == "xent" else dict(temperature=2.0, labels=y, alpha=0.5)
    forward, backward, step = (getattr(losses, f"{op}_{name}") for name in ("forward", "backward", "step"))

    def nan(x):
        return bool(torch.isnan(x).all())

    def withheld(passes, call, *a, **m):
        torch.cuda.synchronize()
        abi.zero_debug_withhold_head_loss(passes, 50_000_000)
        begin = time.perf_counter()
        r = call(*a, **m)
        torch.cuda.synchronize()
        took = time.perf_counter() - begin
        assert 0.05 <= took < 10.0, took
        if r.loss is not None:
            assert nan(r.loss[there]) and nan(r.reduced) and not r.loss[~there].any()
            assert nan(r.lse[there]) and (r.lse_tau is None or nan(r.lse_tau[there]))
        if r.dhidden is not None:
            assert nan(r.dhidden[there]) and not r.dhidden[~there].any()
        assert r.dweight is None or nan(r.dweight)
        return r

    good = step(*args, **more)
    stats = (good.lse,) if op == "xent" else (good.lse, good.lse_tau)
    failed = withheld(1, forward, *args, **more)
    # a backward call from it shows it
    bad = backward(*args, *((failed.lse,) if op == "xent" else (failed.lse, failed.lse_tau)), **more)
    assert nan(bad.dhidden[there]) and nan(bad.dweight)
    for passes in (1, 2, 3):
        withheld(passes, step, *args, **more)
    withheld(2, step, *args, dhidden=False, **more)
    withheld(2, backward, *args, *stats, **more)
    withheld(2, backward, *args, *stats, dhidden=False, **more)
    withheld(2, backward, *args, *stats, dweight=False, **more)
    for pad, accumulate in ((0, True), (1, False), (1, True)):
        dw, buf = empty_matrix(V, D, dt, cuda, pad)
        dw.fill_(1.0)
        withheld(2, step, *args, dweight=dw, accumulate=accumulate, **more)
        gaps_untouched(buf, V, D, pad)
    abi.zero_debug_withhold_head_loss(3, 50_000_000)
    abi.zero_debug_withhold_head_loss(0)       # cleared
    again = step(*args, **more)
    for a, b in zip(again, good):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("kind", TYPES)
def test_gradient_against_differences(losses, cuda, kind):
    """The losses' own central difference along a direction, against the
    gradient along it. What the difference itself is off by comes from the
    definition in 64 bits; what is left is the losses' error over the step."""
    dt = torch.float32
    T, V, D = 40, 600, 48
    h, w, y, g = inputs(T, V, D, dt, 17, cuda)
    ids, logits = teacher(T, V, 9, g, cuda, 0.2)
    u = torch.randn(T, D, generator=g).to(cuda)
    x = (torch.randn(V, D, generator=g) / math.sqrt(D)).to(cuda)
    eps = 2.0 ** -5
    if kind == "bf16":     # the same with the gradient taken in the mixed mode
        h, w = h.bfloat16().float(), w.bfloat16().float()
    for own, args in [("xent", (y,)), ("distill", (ids, logits))]:
        more = {} if own == "xent" else dict(tau=2.0, alpha=0.6, ids=ids, logits=logits)
        call = {} if own == "xent" else dict(temperature=2.0, alpha=0.6, labels=y)
        fwd = getattr(losses, own + "_forward")
        step = getattr(losses, own + "_step")
        store = TYPES[kind]
        got = step(h.to(store), w.to(store), *args, reduction="sum", **call)
        for dh, dw in [(u, torch.zeros_like(w)), (torch.zeros_like(h), x)]:
            ends, exact, allowed = [], [], 0.0
            for sign in (1, -1):
                a, b = h + sign * eps * dh, w + sign * eps * dw
                ends.append(float(fwd(a, b, *args, reduction="sum", **call).loss.double().sum()))
                r = reference(a, b, y, reduction="sum", **more)
                exact.append(float(r["loss"].sum()))
                allowed += float(bounds(r, dt)["loss"].sum())
            r = reference(h, w, y, reduction="sum", **more)
            along = float((r["dhidden"] * dh.double()).sum() + (r["dweight"] * dw.double()).sum())
            b = bounds(r, store)
            allowed = allowed / (2 * eps) + float((b["dhidden"] * dh.abs()).sum() + (b["dweight"] * dw.abs()).sum())
            curve = (exact[0] - exact[1]) / (2 * eps) - along
            mine = float((got.dhidden.double() * dh).sum() + (got.dweight.double() * dw).sum())
            assert abs((ends[0] - ends[1]) / (2 * eps) - curve - mine) <= allowed, own


def test_autograd(losses, cuda):
    T, V, D = 60, 500, 64
    h, w, y, g = inputs(T, V, D, torch.float32, 41, cuda, masked=0.2)
    ids, logits = teacher(T, V, 6, g, cuda)
    scale = 0.3
    a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
    (scale * losses.linear_cross_entropy(a.view(4, 15, D), b, y)).backward()
    r = reference(h, w, y, dloss=scale)
    lim = bounds(r, torch.float32)
    assert bool(((a.grad.double() - r["dhidden"]).abs() <= lim["dhidden"]).all())
    assert bool(((b.grad.double() - r["dweight"]).abs() <= lim["dweight"]).all())
    a, b = h.clone().requires_grad_(), w.clone()
    per_row = losses.linear_distillation(a, b, ids, logits, 2.0, y, 0.5, reduction="none")
    rows = torch.rand(T, generator=g).to(cuda)
    (per_row * rows).sum().backward()
    r = reference(h, w, y, ids, logits, tau=2.0, alpha=0.5, reduction="none", dloss=rows)
    assert bool(((a.grad.double() - r["dhidden"]).abs() <= bounds(r, torch.float32)["dhidden"]).all())


def test_a_graph_of_the_gradients(losses, cuda):
    """Under create_graph the gradients are those without; to differentiate them again raises."""
    T, V, D = 60, 500, 64
    x, w, y, g = inputs(T, V, D, torch.float32, 42, cuda, masked=0.2)
    ids, logits = teacher(T, V, 6, g, cuda)
    for loss in (lambda h: losses.linear_cross_entropy(h, w, y),
                 lambda h: losses.linear_distillation(h, w, ids, logits, 2.0, y, 0.5)):
        a = x.clone().requires_grad_()
        plain, = torch.autograd.grad(loss(a * a), a)
        once, = torch.autograd.grad(loss(a * a), a, create_graph=True)
        assert torch.equal(plain, once)
        with pytest.raises(RuntimeError, match="no second derivatives"):
            once.square().sum().backward()


@pytest.mark.parametrize("kind,T,V,D", [("bf16", 8200, 21000, 64), ("fp32", 4100, 13000, 64)])
def test_several_pieces_of_the_vocabulary(losses, cuda, kind, T, V, D):
    """Enough rows that the gradient of the logits is formed in several pieces."""
    dt = TYPES[kind]
    h, w, y, g = inputs(T, V, D, dt, 51, cuda, masked=0.1)
    r = reference(h, w, y)
    got = losses.xent_step(h, w, y)
    check(got, r, dt)


@pytest.mark.parametrize("kind,T,V,D", [("bf16", 8200, 21000, 64), ("fp32", 4100, 13000, 64)])
def test_distillation_over_several_pieces(losses, cuda, kind, T, V, D):
    dt = TYPES[kind]
    h, w, y, g = inputs(T, V, D, dt, 52, cuda, masked=0.1)
    ids = (torch.randint(0, V - 4000, (T, 1), generator=g) + torch.arange(0, 4000, 500)).to(cuda)
    logits = 3.0 * torch.randn(T, 8, generator=g).to(cuda)
    ids[::7] = -1
    r = reference(h, w, y, ids, logits, tau=2.0, alpha=0.5)
    got = losses.distill_step(h, w, ids, logits, temperature=2.0, labels=y, alpha=0.5)
    check(got, r, dt)


@pytest.mark.parametrize("T,V,D", [(1, 31, 64), (1, 50257, 96), (3, 1009, 65), (16, 2000, 448),
                                   (64, 41217, 200), (200, 300, 771), (256, 777, 128)])
@pytest.mark.parametrize("op", ["xent", "distill", "both"])
def test_few_rows_lose_nothing_to_the_logits_gradient(losses, cuda, op, T, V, D):
    """Up to 256 rows of bf16 the gradients' error is the rounding of the results: the
    logits' gradient is kept in two bf16 parts."""
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 41 * T + D, cuda, masked=0.0)
    hm, wm = matrix(h, cuda), matrix(w, cuda)
    if op == "xent":
        got = losses.xent_step(hm, wm, y)
        r = reference(h, w, y)
    else:
        ids, logits = teacher(T, V, min(V, 12), g, cuda, absent=0.2)
        labels, alpha = (y, 0.5) if op == "both" else (None, 1.0)
        got = losses.distill_step(hm, wm, ids, logits, temperature=2.0, labels=labels, alpha=alpha)
        r = reference(h, w, labels, ids, logits, tau=2.0, alpha=alpha)
    check(got, r, torch.bfloat16, f"{op} {T}x{V}x{D}", parts=2)


@pytest.mark.parametrize("T", [1023, 1024, 1025, 2049])
def test_around_the_rows_that_one_kernel_prepares(losses, cuda, T):
    V, D = 300, 40
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 72, cuda, masked=0.3)
    bad = h.clone()
    bad[y == IGNORE] = math.nan
    check(losses.xent_step(bad, w, y), reference(bad, w, y), torch.bfloat16)


def test_many_rows_few_of_them_labelled(losses, cuda):
    """More rows than the numbering takes at a time, most without a label."""
    T, V, D = 40_003, 300, 24
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 61, cuda, masked=0.97)
    y[:17_000] = IGNORE
    r = reference(h, w, y)
    check(losses.xent_step(h, w, y), r, torch.bfloat16)
    ids, logits = torch.randint(-1, V, (T, 3), generator=g).to(cuda), torch.randn(T, 3, generator=g).to(cuda)
    ids[:, 0] = torch.where(y == IGNORE, -1, ids[:, 0])
    ids[:, 1:] = torch.where((y == IGNORE).unsqueeze(1), -1, ids[:, 1:])
    r = reference(h, w, None, ids, logits, reduction="sum")
    check(losses.distill_step(h, w, ids, logits, reduction="sum"), r, torch.bfloat16)


def test_equal_inputs_give_equal_bits(losses, cuda):
    """Several pieces and split sums, four times over, on two streams at once."""
    T, V, D = 5000, 20_000, 96
    h, w, y, _ = inputs(T, V, D, torch.bfloat16, 62, cuda, masked=0.1)
    first = losses.xent_step(h, w, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    again = [losses.xent_step(h, w, y, stream=streams[i % 2]) for i in range(4)]
    torch.cuda.synchronize()
    for r in again:
        for name in ("loss", "reduced", "lse", "dhidden", "dweight"):
            assert torch.equal(getattr(r, name), getattr(first, name)), name


def test_beside_other_launches_of_other_priorities(losses, cuda):
    """Steps that compete for the SMs with each other and with other kernels: their pairs of
    blocks begin at different times, and some only after others have worked for a while."""
    T, V, D = 3000, 9_000, 96
    h, w, y, _ = inputs(T, V, D, torch.bfloat16, 63, cuda, masked=0.1)
    busy = torch.randn(1 << 26, device=cuda)
    first = losses.xent_step(h, w, y)
    torch.cuda.synchronize()
    other, streams = torch.cuda.Stream(), [torch.cuda.Stream(priority=p) for p in (0, -1, 0, -1)]
    again = []
    for i in range(16):
        with torch.cuda.stream(other):
            busy.mul_(0.5)
        again.append(losses.xent_step(h, w, y, stream=streams[i % 4]))
    torch.cuda.synchronize()
    for r in again:
        for name in ("loss", "dhidden", "dweight"):
            assert torch.equal(getattr(r, name), getattr(first, name)), name


def test_in_a_graph(losses, cuda):
    """Captured once and replayed on new values of the same tensors."""
    T, V, D = 90, 700, 64
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 63, cuda)
    losses.xent_step(h, w, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = losses.xent_step(h, w, y)
    h2, w2, y2, _ = inputs(T, V, D, torch.bfloat16, 64, cuda, masked=0.3)
    h.copy_(h2), w.copy_(w2), y.copy_(y2)
    graph.replay()
    torch.cuda.synchronize()
    check(got, reference(h2, w2, y2), torch.bfloat16)


@pytest.mark.parametrize("kind", TYPES)
def test_distillation_in_a_graph(losses, cuda, kind):
    """Captured once, in both storage types, and replayed on new values of the same tensors."""
    dt = TYPES[kind]
    T, V, D, K = 90, 700, 64, 6
    h, w, y, g = inputs(T, V, D, dt, 73, cuda)
    ids, logits = teacher(T, V, K, g, cuda)
    more = dict(temperature=2.0, labels=y, alpha=0.5)
    losses.distill_step(h, w, ids, logits, **more)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = losses.distill_step(h, w, ids, logits, **more)
    for seed in (74, 75):
        h2, w2, y2, g = inputs(T, V, D, dt, seed, cuda, masked=0.3)
        ids2, logits2 = teacher(T, V, K, g, cuda, absent=0.3)
        for to, value in ((h, h2), (w, w2), (y, y2), (ids, ids2), (logits, logits2)):
            to.copy_(value)
        graph.replay()
        torch.cuda.synchronize()
        check(got, reference(h2, w2, y2, ids2, logits2, tau=2.0, alpha=0.5), dt)


def test_offsets_beyond_32_bits(losses, cuda):
    """A weight whose last rows lie more than 2^32 bytes from its first."""
    V, D, stride = 600, 64, 4_000_000
    buf = torch.empty((V - 1) * stride + D, dtype=torch.bfloat16, device=cuda)
    w = torch.as_strided(buf, (V, D), (stride, 1))
    h, values, y, _ = inputs(50, V, D, torch.bfloat16, 6, cuda)
    w.copy_(values)
    dbuf = torch.empty((V - 1) * stride + D, dtype=torch.bfloat16, device=cuda)
    dw = torch.as_strided(dbuf, (V, D), (stride, 1))
    got = losses.xent_step(h, w, y, dweight=dw)
    check(got, reference(h, values, y), torch.bfloat16)


def test_refusals_of_the_binding(losses, cuda):
    h, w, y, _ = inputs(10, 50, 16, torch.bfloat16, 1, cuda)
    with pytest.raises(TypeError):
        losses.xent_forward(h.half(), w.half(), y)
    with pytest.raises(TypeError):
        losses.xent_forward(h, w.float(), y)
    with pytest.raises(TypeError):
        losses.xent_forward(h, w, y.int())
    with pytest.raises(TypeError):
        losses.xent_forward(h.cpu(), w, y)
    with pytest.raises(ValueError):
        losses.xent_forward(h, w[:, :8], y)
    with pytest.raises(ValueError):
        losses.xent_forward(h.t().contiguous().t(), w, y)
    with pytest.raises(ValueError):
        losses.xent_forward(h, w, y[:5])
    with pytest.raises(ValueError):
        losses.xent_forward(h, w, y, reduction="average")
    with pytest.raises(ValueError):
        losses.xent_step(h, w, y, accumulate=True)
    with pytest.raises(ValueError):
        losses.distill_forward(h, w, y.view(10, 1), torch.zeros(10, 2, device=cuda))
    from zero_sharded_optimizer_gb300 import abi
    for bad in (dict(dhidden=h), dict(dweight=w)):                 # an output over an input
        with pytest.raises(abi.ZeroError) as e:
            losses.xent_step(h, w, y, **bad)
        assert e.value.code == abi.ZERO_EINVAL and "overlap" in str(e.value)
    wide = torch.zeros(10, 32, dtype=torch.bfloat16, device=cuda)  # column blocks of one buffer
    wide[:, :16] = h
    got = losses.xent_step(wide[:, :16], w, y, dhidden=wide[:, 16:])
    check(got, reference(h, w, y), torch.bfloat16)


def test_shapes_that_do_not_fit_the_rows(losses, cuda):
    """As many elements in another order are refused; the rows' own dimensions, the rows in one
    dimension, dimensions of one element, and any dimensions beside rows in one are not."""
    B, S, V, D, K = 4, 6, 50, 16, 3
    T = B * S
    h, w, y, g = inputs(T, V, D, torch.bfloat16, 69, cuda)
    ids, logits = teacher(T, V, K, g, cuda)
    r = reference(h, w, y, ids, logits, alpha=0.5)
    h3, dloss = h.view(B, S, D), torch.rand(T, generator=g).to(cuda)

    def distill(y=y, ids=ids, logits=logits, h=h3, **more):
        return losses.distill_step(h, w, ids, logits, labels=y, alpha=0.5, **more)

    for shape in ((T,), (B, S), (T, 1), (1, T), (B, 1, S), (B, S, 1)):
        for rows in ((T,), (B, S)):
            check(distill(y.view(shape), ids.view(*rows, K), logits.view(B, S, K)), r, torch.bfloat16)
    more = dict(reduction="none")
    each = losses.xent_step(h3, w, y, dloss=dloss.view(B, S), **more)
    for bad in ((S, B), (B // 2, 2 * S), (B, 2, S // 2)):
        with pytest.raises(ValueError, match="labels"):
            losses.xent_forward(h3, w, y.view(bad))
        with pytest.raises(ValueError, match="labels"):
            distill(y.view(bad))
        with pytest.raises(ValueError, match="dloss"):
            losses.xent_step(h3, w, y, dloss=dloss.view(bad), **more)
        with pytest.raises(ValueError, match="lse"):
            losses.xent_backward(h3, w, y, each.lse.view(bad), dloss=dloss, **more)
        with pytest.raises(ValueError, match="teacher_ids"):
            distill(ids=ids.view(*bad, K))
        with pytest.raises(ValueError, match="teacher_logits"):
            distill(logits=logits.view(*bad, K))
    for rows in ((B, S), (S, B), (2, 2, S)):
        check(distill(y.view(rows), ids.view(*rows, K), logits.view(*rows, K), h), r, torch.bfloat16)
        check(distill(y.view(rows), ids, logits.view(*rows, K), h), r, torch.bfloat16)
    with pytest.raises(ValueError, match="teacher_logits"):
        distill(y, ids.view(B, S, K), logits.view(S, B, K), h)
    with pytest.raises(ValueError, match="teacher_ids"):
        distill(y.view(B, S), ids.view(S, B, K), logits, h)
    with pytest.raises(ValueError, match="teacher_logits"):
        distill(logits=logits.t().contiguous())
    with pytest.raises(ValueError, match="teacher_logits"):
        distill(logits=logits.view(B, S, K).transpose(1, 2).contiguous())
    with pytest.raises(ValueError, match="teacher_ids"):
        distill(ids=ids.t().contiguous())
