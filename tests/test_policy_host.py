"""The policy and the preference loss without a GPU: the binding's structs, the
workspace queries, and every argument check (each before any device work)."""

import ctypes
import math
import os
import shutil
import subprocess

import pytest

from test_losses_host import problem

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def policy(abi, **changes):
    q = abi.Policy()
    q.clip_low = q.clip_high = 0.2
    at = 1 << 32
    for name in ("old_logps", "advantages", "logps", "slopes"):
        setattr(q, name, at)
        at += 1 << 20
    for k, v in changes.items():
        setattr(q, k, v)
    return q


def preference(abi, **changes):
    q = abi.Preference()
    q.pairs, q.beta = 5, 0.1
    at = 1 << 33
    for name in ("offsets", "logps", "row_logps", "slopes", "counts"):
        setattr(q, name, at)
        at += 1 << 20
    for k, v in changes.items():
        setattr(q, k, v)
    return q


def refused(abi, kind, name, p, q, code, text):
    rc = abi.raw_call(f"zero_{kind}_{name}", None if p is None else ctypes.byref(p),
                      None if q is None else ctypes.byref(q), None)
    assert rc == code, (rc, abi.zero_last_error())
    assert text in abi.zero_last_error(), abi.zero_last_error()


@pytest.mark.parametrize("name", ["Policy", "Preference"])
def test_structs_match_the_header(abi, tmp_path, name):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    struct, ctype = getattr(abi, name), f"zero_{name.lower()}_t"
    fields = [f for f, _ in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "zero_gb300.h"\nint main(void) {\n'
                   f'printf("%zu\\n", sizeof({ctype}));\n' +
                   "".join(f'printf("%zu\\n", offsetof({ctype}, {f}));\n' for f in fields) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    seen = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                           text=True).stdout.split()]
    assert seen == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]


@pytest.mark.parametrize("change,text", [
    (dict(T=-1), "T="), (dict(V=0), "V="), (dict(D=0), "D="), (dict(precision=2), "precision"),
    (dict(reduction=3), "reduction"), (dict(hidden_stride=31), "hidden_stride"), (dict(labels=None), "labels is NULL"),
    (dict(loss=None), "loss is NULL"), (dict(lse=None), "lse is NULL"), (dict(reduced=None), "reduced is NULL"),
    (dict(grad_scale=math.nan), "grad_scale"), (dict(dhidden=None, dweight=None), "neither"),
    (dict(workspace_bytes=1000), "are needed"), (dict(teacher_k=3), "teacher fields"),
    (dict(dhidden=1 << 20), "overlap")])
def test_refusals_of_the_common_part(abi, change, text):
    for kind, q in (("policy", policy(abi)), ("preference", preference(abi))):
        refused(abi, kind, "step", problem(abi, **change), q, abi.ZERO_EINVAL, text)


@pytest.mark.parametrize("change,text", [
    (dict(clip_low=-0.1), "clip_low"), (dict(clip_low=math.nan), "clip_low"), (dict(clip_high=math.inf), "clip_high"),
    (dict(kl_weight=math.inf), "kl_weight"), (dict(kl_weight=0.1), "ref_logps is NULL"),
    (dict(old_logps=None), "old_logps is NULL"), (dict(advantages=None), "advantages is NULL"),
    (dict(logps=None), "logps is NULL"), (dict(slopes=None), "slopes is NULL"),
    (dict(logps=1 << 20), "overlap"), (dict(slopes=1 << 32), "overlap"), (dict(logps=(1 << 32) + 16), "overlap"),
    (dict(old_logps=9 << 20), "overlap")])
def test_policy_refusals(abi, change, text):
    refused(abi, "policy", "step", problem(abi), policy(abi, **change), abi.ZERO_EINVAL, text)


@pytest.mark.parametrize("change,text", [
    (dict(pairs=-1), "pairs="), (dict(pairs=2 ** 30), "pairs="), (dict(pairs=3, offsets=None), "equal length"),
    (dict(pairs=0, offsets=None), "equal length"), (dict(kind=2), "kind"), (dict(beta=math.inf), "beta"),
    (dict(smoothing=-0.1), "smoothing"), (dict(smoothing=1.1), "smoothing"), (dict(smoothing=math.nan), "smoothing"),
    (dict(smoothing=0.1, kind=1), "smoothing"), (dict(margin=math.nan), "margin"),
    (dict(nll_weight=math.inf), "nll_weight"), (dict(logps=None), "logps is NULL"),
    (dict(slopes=None), "slopes is NULL"), (dict(counts=None), "counts is NULL"),
    (dict(row_logps=None), "row_logps is NULL"), (dict(row_logps=(1 << 33) + 40), "overlap"),
    (dict(counts=(1 << 33) + 40), "overlap"), (dict(ref_logps=(1 << 33) + (1 << 20)), "overlap")])
def test_preference_refusals(abi, change, text):
    refused(abi, "preference", "step", problem(abi), preference(abi, **change), abi.ZERO_EINVAL, text)


def test_misaligned_pointers(abi):
    for change in (dict(old_logps=(1 << 32) + 2), dict(slopes=(1 << 34) + 1)):
        refused(abi, "policy", "step", problem(abi), policy(abi, **change), abi.ZERO_EALIGN, "aligned")
    for change in (dict(offsets=(1 << 33) + 4), dict(counts=(1 << 34) + 2)):
        refused(abi, "preference", "step", problem(abi), preference(abi, **change), abi.ZERO_EALIGN, "aligned")


def test_null_problem_and_output(abi):
    for kind, q in (("policy", policy(abi)), ("preference", preference(abi))):
        for name in ("forward", "backward", "step"):
            refused(abi, kind, name, None, q, abi.ZERO_EINVAL, "NULL")
            refused(abi, kind, name, problem(abi), None, abi.ZERO_EINVAL, "NULL")
        p = problem(abi)
        assert abi.raw_call(f"zero_{kind}_workspace_bytes", ctypes.byref(p), ctypes.byref(q), None) == abi.ZERO_EINVAL


def test_a_backward_call_needs_little(abi):
    """lse, the rows' log-probabilities, the slopes and, for pairs, their number and offsets."""
    p = problem(abi, loss=None, reduced=None, workspace_bytes=1000)
    refused(abi, "policy", "backward", p, policy(abi, old_logps=None, advantages=None), abi.ZERO_EINVAL, "are needed")
    refused(abi, "policy", "backward", p, policy(abi, logps=None), abi.ZERO_EINVAL, "logps is NULL")
    refused(abi, "preference", "backward", p, preference(abi, logps=None, counts=None), abi.ZERO_EINVAL, "are needed")


def test_workspaces_are_near_the_cross_entropys(abi):
    big = dict(T=8192, V=50257, D=768, hidden_stride=768, weight_stride=768, dhidden_stride=768, dweight_stride=768)
    p = problem(abi, **big)
    size = abi.zero_xent_workspace_bytes(p)
    for other in (abi.zero_policy_workspace_bytes(p, policy(abi)),
                  abi.zero_preference_workspace_bytes(p, preference(abi))):
        assert size <= other <= size + 8192 * 12 + 1024


@pytest.mark.parametrize("f32,T,V,D,pad,few", [
    (0, 8, 50257, 768, 0, True), (0, 16, 50257, 768, 0, False), (0, 8, 131072, 4096, 0, False),
    (0, 4, 131072, 4096, 0, True), (0, 32, 8000, 512, 0, True), (0, 16, 50257, 64, 0, False),
    (0, 32, 50257, 8, 0, False), (0, 1, 50257, 769, 0, False), (0, 1, 50257, 768, 1, False), (0, 8, 8000, 513, 0, True),
    (0, 32, 1009, 97, 0, True), (1, 16, 131072, 4096, 0, True), (1, 32, 50257, 64, 0, False),
    (1, 32, 8000, 512, 0, True), (1, 64, 8000, 512, 0, False), (1, 8, 50257, 769, 0, True),
    (1, 16, 50257, 769, 0, False), (1, 64, 1009, 96, 0, True)])
def test_few_rows_go_by_their_own_work(abi, f32, T, V, D, pad, few):
    """Which calls are worked on without the tensor cores: those that gain by it, as measured. Their logits are kept,
    in groups of eight rows; else the packed hidden states, the pieces of G and, for fp32, the weight's parts."""
    more = dict(T=T, V=V, D=D, precision=abi.ZERO_FP32 if f32 else abi.ZERO_BF16_MIXED, hidden_stride=D,
                weight_stride=D + pad, dhidden_stride=D, dweight_stride=D)
    kept = (T + 7) // 8 * 8 * 4 * V
    parts = 304 * 4 * D + T * 4 * D * 304 + (1 << 20)         # at most: dhidden's sums, statistics, rows
    for own in (abi.zero_policy_workspace_bytes(problem(abi, **more), policy(abi)),
                abi.zero_preference_workspace_bytes(problem(abi, **more), preference(abi))):
        other = abi.zero_xent_workspace_bytes(problem(abi, **more))
        if few:
            assert own != other and kept <= own <= kept + parts
        else:
            assert other <= own <= other + 16 * T + V // 2 + 4096


@pytest.mark.parametrize("op", ["policy", "preference"])
@pytest.mark.parametrize("wrt", ["hidden", "weight", "both"])
def test_second_derivatives_raise(abi, monkeypatch, op, wrt):
    """Gradients with a graph are the right ones; to differentiate them again raises. (The
    calls replaced by the definition on CPU tensors.)"""
    import torch
    from zero_sharded_optimizer_gb300 import losses
    g = torch.Generator().manual_seed(5)
    T, V, D = 6, 20, 4
    y = torch.randint(0, V, (T,), generator=g)
    weights = torch.randn(T, generator=g, dtype=torch.float64)

    def value(h, w):
        return (torch.log_softmax(h @ w.T, 1).gather(1, y.unsqueeze(1))[:, 0] * weights).sum()

    def forward(h, w, *a, **m):
        none = torch.zeros(T)
        return losses.LogpLosses(none, value(h, w).detach(), none, none, none, none)

    def backward(h, w, *a, dloss, dhidden, dweight, **m):
        with torch.enable_grad():
            x, z = h.detach().requires_grad_(), w.detach().requires_grad_()
            gh, gw = torch.autograd.grad(value(x, z) * dloss, (x, z))
        return losses.LogpLosses(*[None] * 7, None if dhidden is False else gh, None if dweight is False else gw)

    monkeypatch.setattr(losses, f"{op}_forward", forward)
    monkeypatch.setattr(losses, f"{op}_backward", backward)
    p = [torch.randn(T, D, generator=g, dtype=torch.float64), torch.randn(V, D, generator=g, dtype=torch.float64)]
    a, b = [x.requires_grad_(wrt in (name, "both")) for x, name in zip(p, ("hidden", "weight"))]
    taken = [x for x in (a, b) if x.requires_grad]
    none = torch.zeros(T)
    got = losses.linear_policy(a * a, b, y, none, none) if op == "policy" else \
        losses.linear_preference(a * a, b, y, torch.tensor([0, 3, 6]))
    once = torch.autograd.grad(got, taken, create_graph=True)
    exact = torch.autograd.grad(value(a * a, b), taken)
    for x, e in zip(once, exact):
        assert torch.allclose(x, e, rtol=1e-9, atol=1e-12)
    with pytest.raises(RuntimeError, match="no second derivatives"):
        sum(x.square().sum() for x in once).backward()
