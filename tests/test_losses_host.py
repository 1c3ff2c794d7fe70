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
