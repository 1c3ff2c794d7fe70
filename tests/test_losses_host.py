"""The vocabulary losses without a GPU: the binding's struct, the workspace
query, and every argument check (each before any device work)."""

import ctypes
import math
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def problem(abi, distill=False, **changes):
    p = abi.HeadLoss()
    p.T, p.V, p.D = 10, 100, 32
    p.precision, p.reduction = abi.ZERO_BF16_MIXED, abi.ZERO_REDUCE_MEAN
    p.hidden_stride = p.weight_stride = p.dhidden_stride = p.dweight_stride = 32
    p.ignore_index, p.grad_scale = -100, 1.0
    at = 1 << 20
    for name in ("hidden", "weight", "labels", "loss", "lse", "reduced", "dhidden", "dweight",
                 "workspace"):
        setattr(p, name, at)
        at += 1 << 20
    p.workspace_bytes = 1 << 30
    if distill:
        p.teacher_ids, p.teacher_logits, p.lse_tau = 1 << 32, 1 << 33, 1 << 34
        p.teacher_k, p.temperature, p.alpha = 4, 2.0, 0.5
    for k, v in changes.items():
        setattr(p, k, v)
    return p


def refused(abi, kind, name, p, code, text):
    rc = abi.raw_call(f"zero_{kind}_{name}", None if p is None else ctypes.byref(p), None)
    assert rc == code, (rc, abi.zero_last_error())
    assert text in abi.zero_last_error(), abi.zero_last_error()


def test_struct_matches_the_header(abi, tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in abi.HeadLoss._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "zero_gb300.h"\nint main(void) {\n'
                   'printf("%zu\\n", sizeof(zero_head_loss_t));\n' +
                   "".join(f'printf("%zu\\n", offsetof(zero_head_loss_t, {f}));\n' for f in fields) +
                   "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    seen = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                           text=True).stdout.split()]
    assert seen == [ctypes.sizeof(abi.HeadLoss)] + [getattr(abi.HeadLoss, f).offset for f in fields]


@pytest.mark.parametrize("change,text", [
    (dict(T=-1), "T="), (dict(T=2 ** 31), "T="), (dict(V=0), "V="), (dict(V=2 ** 31), "V="),
    (dict(D=0), "D="), (dict(precision=2), "precision"), (dict(reduction=3), "reduction"),
    (dict(hidden_stride=31), "hidden_stride"), (dict(weight_stride=31), "weight_stride"),
    (dict(weight_stride=2 ** 62), "weight_stride"), (dict(dhidden_stride=0), "dhidden_stride"),
    (dict(dweight_stride=-32), "dweight_stride"), (dict(hidden=None), "hidden is NULL"),
    (dict(weight=None), "weight is NULL"), (dict(labels=None), "labels is NULL"),
    (dict(loss=None), "loss is NULL"), (dict(lse=None), "lse is NULL"),
    (dict(reduced=None), "reduced is NULL"), (dict(grad_scale=math.nan), "grad_scale"),
    (dict(dhidden=None, dweight=None), "neither"), (dict(workspace=None), "workspace"),
    (dict(workspace_bytes=1000), "are needed"), (dict(teacher_k=3), "teacher fields"),
    (dict(teacher_ids=4096), "teacher fields"), (dict(lse_tau=4096), "teacher fields"),
    (dict(dhidden=1 << 20), "overlap"), (dict(dweight=2 << 20), "overlap"),
    (dict(workspace=1 << 20), "overlap"), (dict(loss=(1 << 20) + 16), "overlap"),
    (dict(lse=4 << 20), "overlap")])
def test_xent_refusals(abi, change, text):
    refused(abi, "xent", "step", problem(abi, **change), abi.ZERO_EINVAL, text)


@pytest.mark.parametrize("change,text", [
    (dict(teacher_k=0), "teacher_k"), (dict(teacher_k=1025), "teacher_k"),
    (dict(temperature=0.0), "temperature"), (dict(temperature=-1.0), "temperature"),
    (dict(temperature=math.inf), "temperature"), (dict(temperature=math.nan), "temperature"),
    (dict(temperature=1e-60), "temperature"), (dict(alpha=-0.1), "alpha"),
    (dict(alpha=1.1), "alpha"), (dict(alpha=math.nan), "alpha"),
    (dict(labels=None), "without labels"), (dict(teacher_ids=None), "teacher_ids is NULL"),
    (dict(teacher_logits=None), "teacher_logits is NULL"), (dict(lse_tau=None), "lse_tau is NULL"),
    (dict(lse=None), "lse is NULL")])
def test_distill_refusals(abi, change, text):
    refused(abi, "distill", "step", problem(abi, True, **change), abi.ZERO_EINVAL, text)


@pytest.mark.parametrize("change,text", [
    (dict(hidden=(1 << 20) + 1), "hidden"), (dict(weight=(2 << 20) + 1), "weight"),
    (dict(labels=(3 << 20) + 4), "labels"), (dict(loss=(4 << 20) + 2), "loss"),
    (dict(dhidden=(7 << 20) + 1), "dhidden"), (dict(dweight=(8 << 20) + 1), "dweight"),
    (dict(workspace=(9 << 20) + 128), "workspace")])
def test_misaligned_pointers(abi, change, text):
    refused(abi, "xent", "step", problem(abi, **change), abi.ZERO_EALIGN, text)


def test_an_empty_dhidden_may_be_null(abi):
    """Without rows dhidden has no elements: a backward call for it alone has nothing to do, a
    step needs what a forward call does."""
    changes = dict(T=0, dhidden=None, dweight=None, workspace_bytes=1000)
    p = problem(abi, **changes)
    assert abi.raw_call("zero_xent_backward", ctypes.byref(p), None) == abi.ZERO_OK
    refused(abi, "xent", "step", p, abi.ZERO_EINVAL, f"{abi.zero_xent_workspace_bytes(p)} are needed")


def test_empty_labels_may_be_null(abi):
    """Without rows the labels have no elements either, whatever alpha."""
    p = problem(abi, True, T=0, labels=None, workspace_bytes=1000)
    refused(abi, "distill", "step", p, abi.ZERO_EINVAL, "are needed")


def test_empty_buffers_overlap_nothing(abi):
    """Without rows, a pointer into another buffer (an arena's) shares no byte with it."""
    for change in (dict(labels=(8 << 20) + 64), dict(loss=(8 << 20) + 64), dict(lse=(9 << 20) + 64)):
        refused(abi, "xent", "step", problem(abi, T=0, workspace_bytes=1000, **change), abi.ZERO_EINVAL, "are needed")
    change = dict(teacher_ids=(8 << 20) + 64, teacher_logits=(8 << 20) + 64)
    refused(abi, "distill", "step", problem(abi, True, T=0, workspace_bytes=1000, **change), abi.ZERO_EINVAL,
            "are needed")


def test_withholding_is_checked(abi):
    for passes, limit in ((-1, 1), (4, 1), (1, 0), (1, -5), (1, 10_000_000_001)):
        assert abi.raw_call("zero_debug_withhold_head_loss", passes, ctypes.c_int64(limit)) == abi.ZERO_EINVAL
    abi.zero_debug_withhold_head_loss(3, 1)
    abi.zero_debug_withhold_head_loss(0)


def test_null_problem_and_output(abi):
    for kind in ("xent", "distill"):
        for name in ("forward", "backward", "step"):
            refused(abi, kind, name, None, abi.ZERO_EINVAL, "NULL")
    p = problem(abi)
    assert abi.raw_call("zero_xent_workspace_bytes", ctypes.byref(p), None) == abi.ZERO_EINVAL


def test_workspace_sizes(abi):
    """It does not grow with T x V: the logits are never kept."""
    def size(**changes):
        return abi.zero_xent_workspace_bytes(problem(abi, **changes))

    big = dict(T=8192, V=50257, D=768, hidden_stride=768, weight_stride=768, dhidden_stride=768,
               dweight_stride=768)
    assert size(**big) < 8192 * 50257 * 2 / 4
    forward = size(**dict(big, dhidden=None, dweight=None))
    assert forward < size(**big)
    # packed rows, and 8 bytes of statistics for each half tile of 128 columns
    assert forward < 8192 * 768 * 2 + 8192 * 400 * 8 + (1 << 20)
    # rows that 16-byte copies cannot read are packed first
    assert size(**dict(big, weight_stride=769)) >= size(**big) + 50257 * 768 * 2
    assert size(T=0) > 0
    with pytest.raises(abi.ZeroError):
        size(**dict(big, D=2 ** 30, hidden_stride=2 ** 30, weight_stride=2 ** 30, dhidden_stride=2 ** 30,
                    dweight_stride=2 ** 30, V=2 ** 31 - 2000, T=2 ** 31 - 2000, precision=0))


@pytest.fixture
def on_the_cpu(abi, monkeypatch):
    """losses, with its four autograd calls replaced by the definition on CPU tensors."""
    import torch
    from zero_sharded_optimizer_gb300 import losses

    def value(h, w, y, ids=None, u=None, temperature=1.0, alpha=1.0, reduction="mean", ignore_index=-100):
        z = h @ w.T
        loss = torch.zeros(h.shape[0], dtype=h.dtype)
        if y is not None:
            ce = torch.nn.functional.cross_entropy(z, y, reduction="none", ignore_index=ignore_index)
            loss = loss + (ce if ids is None else (1 - alpha) * ce)
        if ids is not None:
            logq = torch.log_softmax(u / temperature, 1)
            logp = torch.log_softmax(z / temperature, 1).gather(1, ids)
            loss = loss + alpha * temperature ** 2 * (logq.exp() * (logq - logp)).sum(1)
        return loss, (loss.mean() if reduction == "mean" else loss.sum())

    def result(loss, reduced, distill, **grads):
        lse = torch.zeros(loss.shape[0])
        return losses.Losses(loss.detach(), reduced.detach(), lse, lse if distill else None, **grads)

    def gradients(h, w, distill, dloss, dhidden, dweight, *args, **more):
        with torch.enable_grad():
            a, b = h.detach().requires_grad_(), w.detach().requires_grad_()
            loss, reduced = value(a, b, *args, **more)
            total = loss @ dloss if more["reduction"] == "none" else reduced * dloss
            gh, gw = torch.autograd.grad(total, (a, b))
        return result(loss, reduced, distill, dhidden=None if dhidden is False else gh,
                      dweight=None if dweight is False else gw)

    monkeypatch.setattr(losses, "xent_forward", lambda h, w, y, **m: result(*value(h, w, y, **m), False))
    monkeypatch.setattr(losses, "distill_forward", lambda h, w, ids, u, labels, **m:
                        result(*value(h, w, labels, ids, u, **m), True))
    monkeypatch.setattr(losses, "xent_backward", lambda h, w, y, lse, dloss, dhidden, dweight, **m:
                        gradients(h, w, False, dloss, dhidden, dweight, y, **m))
    monkeypatch.setattr(losses, "distill_backward",
                        lambda h, w, ids, u, lse, lse_tau, labels, dloss, dhidden, dweight, **m:
                        gradients(h, w, True, dloss, dhidden, dweight, labels, ids, u, **m))
    return losses, value


@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("reduction", ["mean", "none"])
@pytest.mark.parametrize("wrt", ["hidden", "weight", "both"])
def test_second_derivatives_raise(on_the_cpu, op, reduction, wrt):
    """Gradients with a graph are the right ones; a penalty on them, whose gradient runs
    through the losses' own second derivatives, raises instead of losing that part."""
    import torch
    losses, value = on_the_cpu
    g = torch.Generator().manual_seed(5)
    T, V, D, K = 6, 20, 4, 3

    def fresh():
        p = [torch.randn(T, D, generator=g, dtype=torch.float64), torch.randn(V, D, generator=g, dtype=torch.float64)]
        return [x.requires_grad_(wrt in (name, "both")) for x, name in zip(p, ("hidden", "weight"))]

    a, b = fresh()
    taken = [x for x in (a, b) if x.requires_grad]
    y = torch.randint(0, V, (T,), generator=g)
    ids, u = torch.randint(0, V, (T, K), generator=g), torch.randn(T, K, generator=g, dtype=torch.float64)
    rows = torch.randn(T, generator=g, dtype=torch.float64)
    h, w = a * a, b * b + b          # what the penalty's gradient also runs through
    if op == "xent":
        got = losses.linear_cross_entropy(h, w, y, reduction=reduction)
        loss, reduced = value(h, w, y)
    else:
        got = losses.linear_distillation(h, w, ids, u, 2.0, y, 0.5, reduction=reduction)
        loss, reduced = value(h, w, y, ids, u, 2.0, 0.5)
    got, want = (got @ rows, loss @ rows) if reduction == "none" else (got, reduced)
    once = torch.autograd.grad(got, taken, create_graph=True)
    exact = torch.autograd.grad(want, taken)
    for x, e in zip(once, exact):
        assert torch.allclose(x, e, rtol=1e-9, atol=1e-12)
    penalty = sum(x.square().sum() for x in once)
    with pytest.raises(RuntimeError, match="no second derivatives"):
        penalty.backward()
    # through the incoming gradient alone, too
    scale = torch.ones((), dtype=torch.float64, requires_grad=True)
    h = a.detach().requires_grad_()
    loss = losses.linear_cross_entropy(h, b.detach(), y)
    d, = torch.autograd.grad(loss * scale, h, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivatives"):
        d.sum().backward()
