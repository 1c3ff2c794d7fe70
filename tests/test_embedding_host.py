"""The embedding without a GPU: the binding's struct, the workspace query, and
every argument check (each before any device work)."""

import ctypes
import math
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def problem(abi, **changes):
    p = abi.Embedding()
    p.T, p.V, p.D = 10, 100, 32
    p.precision, p.scale, p.padding_id = abi.ZERO_BF16_MIXED, 1.0, -1
    p.weight_stride = p.out_stride = p.dout_stride = p.dweight_stride = 32
    at = 1 << 20
    for name in ("ids", "weight", "out", "dout", "dweight", "workspace"):
        setattr(p, name, at)
        at += 1 << 20
    p.workspace_bytes = 1 << 19
    for k, v in changes.items():
        setattr(p, k, v)
    return p


def refused(abi, name, p, code, text):
    rc = abi.raw_call(f"zero_embedding_{name}", None if p is None else ctypes.byref(p), None)
    assert rc == code, (rc, abi.zero_last_error())
    assert text in abi.zero_last_error(), abi.zero_last_error()


def test_struct_matches_the_header(abi, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in abi.Embedding._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "zero_gb300.h"\nint main(void) {\n'
                   'printf("%zu\\n", sizeof(zero_embedding_t));\n' +
                   "".join(f'printf("%zu\\n", offsetof(zero_embedding_t, {f}));\n' for f in fields) +
                   "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    seen = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                           text=True).stdout.split()]
    assert seen == [ctypes.sizeof(abi.Embedding)] + [getattr(abi.Embedding, f).offset for f in fields]


BOTH = [(dict(T=-1), "T="), (dict(T=2 ** 31), "T="), (dict(V=0), "V="), (dict(V=2 ** 31), "V="),
        (dict(D=0), "D="), (dict(precision=2), "precision"), (dict(scale=math.nan), "scale"),
        (dict(scale=1e300), "scale"), (dict(ids=None), "ids is NULL")]


@pytest.mark.parametrize("change,text", BOTH + [
    (dict(weight_stride=31), "weight_stride"), (dict(out_stride=0), "out_stride"),
    (dict(out_stride=2 ** 62), "out_stride"), (dict(weight=None), "weight is NULL"),
    (dict(out=None), "out is NULL"), (dict(out=2 << 20), "overlap"), (dict(out=(1 << 20) + 16), "overlap")])
def test_forward_refusals(abi, change, text):
    refused(abi, "forward", problem(abi, **change), abi.ZERO_EINVAL, text)


@pytest.mark.parametrize("change,text", BOTH + [
    (dict(dout_stride=31), "dout_stride"), (dict(dweight_stride=-32), "dweight_stride"),
    (dict(dout=None), "dout is NULL"), (dict(dweight=None), "dweight is NULL"),
    (dict(dweight=4 << 20), "overlap"), (dict(workspace=5 << 20), "overlap"),
    (dict(workspace=None), "are needed"), (dict(workspace_bytes=1000), "are needed")])
def test_backward_refusals(abi, change, text):
    refused(abi, "backward", problem(abi, **change), abi.ZERO_EINVAL, text)


@pytest.mark.parametrize("name,change,text", [
    ("forward", dict(ids=(1 << 20) + 4), "ids"), ("forward", dict(weight=(2 << 20) + 1), "weight"),
    ("forward", dict(out=(3 << 20) + 1), "out"), ("backward", dict(dout=(4 << 20) + 1), "dout"),
    ("backward", dict(dweight=(5 << 20) + 1), "dweight"),
    ("backward", dict(workspace=(6 << 20) + 128), "workspace")])
def test_misaligned_pointers(abi, name, change, text):
    refused(abi, name, problem(abi, **change), abi.ZERO_EALIGN, text)


def test_nothing_to_do(abi):
    """Without tokens a lookup writes nothing, and an accumulated gradient adds nothing: the
    buffers that have no elements may be NULL."""
    p = problem(abi, T=0, ids=None, out=None, dout=None, accumulate=1)
    for name in ("forward", "backward"):
        assert abi.raw_call(f"zero_embedding_{name}", ctypes.byref(p), None) == abi.ZERO_OK


def test_null_problem_and_output(abi):
    for name in ("forward", "backward"):
        refused(abi, name, None, abi.ZERO_EINVAL, "NULL")
    p = problem(abi)
    assert abi.raw_call("zero_embedding_workspace_bytes", ctypes.byref(p), None) == abi.ZERO_EINVAL


def test_workspace_sizes(abi):
    """Some bytes a token beside the sums of the runs, whatever the vocabulary."""
    def size(**changes):
        return abi.zero_embedding_workspace_bytes(problem(abi, **changes))

    assert size(T=0) >= 0
    big = size(T=131072, D=4096, V=50257)
    assert big < 131072 * 4096 * 2 / 4
    assert size(T=131072, D=4096, V=131072) < 1.1 * big


def test_refusals_of_the_binding(abi):
    """Tensors that are not on a GPU are refused before anything else."""
    import torch
    from zero_sharded_optimizer_gb300 import embedding
    ids, w = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 4)
    with pytest.raises(TypeError):
        embedding.embedding_forward(ids, w)
    with pytest.raises(TypeError):
        embedding.embedding_backward(ids, torch.zeros(3, 4), 5)
    with pytest.raises(TypeError):
        embedding.embedding_backward(None, None, 5)
    with pytest.raises(ValueError):
        embedding.embedding_backward(ids, torch.zeros(4, 4), 5)
