"""The embedding on the GPU against its definition in 64 bits.

A lookup is one product with the scale as fp32 (2^-24 of itself), rounded in
fp32 and then to its type. A gradient is a sum of n terms in fp32, in any order
off by at most n 2^-24 of the sum of their sizes, times the scale, rounded to
its type, after an addition where it accumulates. Matrices sit between guard
regions, with sentinels in the gaps of their rows: a read past a row's end
brings a NaN into the result, a write past it is found afterwards."""

import math

import pytest
import torch

import parity_util

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}     # half a step


@pytest.fixture(scope="module")
def embedding(abi, cuda):
    from zero_sharded_optimizer_gb300 import embedding as module
    return module


def matrix(values, pad=0, offset=0, what="matrix"):
    """`values` in a guarded buffer of rows `pad` elements apart."""
    n, d = values.shape
    buf = parity_util.guarded_empty(max(n * (d + pad), 1), values.dtype, values.device, offset, what)
    m = torch.as_strided(buf, (n, d), (d + pad, 1), buf.storage_offset())
    m.copy_(values)
    return m, buf


def gaps_untouched(buf, n, d, pad):
    if pad == 0 or n < 2:
        return
    bits = buf.view(torch.int32 if buf.dtype == torch.float32 else torch.int16)
    s = 0x7FA5A5A5 if buf.dtype == torch.float32 else 0x7FA5
    assert bool((bits[:n * (d + pad)].view(n, d + pad)[:, d:] == s).all())


def close(got, want, error, dtype, what=""):
    """`error`: what the result may be off by before its last rounding."""
    bound = 1.01 * (error + UNIT[dtype] * (want.abs() + error)) + 2.0 ** -126
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((off / bound).max())} of the bound"


def check_gradient(got, ids, dout, V, scale, before=None, padding_id=-1, what=""):
    ids = ids.flatten()
    keep = (ids >= 0) & (ids < V) & (ids != padding_id)
    at, rows = ids[keep], dout.reshape(len(ids), dout.shape[-1])[keep].double()
    zero = torch.zeros(V, rows.shape[1], dtype=torch.float64, device=rows.device)
    total, size = zero.index_add(0, at, rows), zero.index_add(0, at, rows.abs())
    n = torch.zeros(V, dtype=torch.float64, device=rows.device).index_add(0, at, torch.ones_like(at, dtype=torch.float64))
    want = scale * total
    error = abs(scale) * size * (n + 2).unsqueeze(1) * 2.0 ** -24
    if before is not None:
        want = want + before.double()
        error = error + 2.0 ** -24 * want.abs()
    close(got, want, error, got.dtype, what)
    absent = n == 0
    if before is not None:
        assert torch.equal(got[absent], before[absent]), what
    else:
        assert not got[absent].any(), what


def tokens(T, V, g, kind="frequent"):
    if kind == "frequent":       # low ids are frequent, as in a vocabulary in order of frequency
        return (torch.rand(T, generator=g) * math.log(V)).exp().long().sub_(1).clamp_(0, V - 1)
    if kind == "any":
        return torch.randint(0, V, (T,), generator=g)
    if kind == "one":
        return torch.full((T,), V // 2)
    if kind == "two":
        return torch.where(torch.rand(T, generator=g) < 0.5, 0, V - 1)
    return torch.randperm(V, generator=g)[:T]     # distinct


SIZES = [(1, 1, 1), (1, 50257, 768), (7, 3, 5), (8, 100, 256), (9, 100, 257), (31, 64, 129), (33, 1000, 96),
         (256, 256, 64), (257, 511, 72), (1000, 512, 513), (4095, 513, 40), (4097, 1009, 33), (8193, 50257, 24)]


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("kind", TYPES)
def test_forward(embedding, cuda, kind, T, V, D):
    dt, g = TYPES[kind], torch.Generator().manual_seed(T + V + D)
    w, _ = matrix(torch.randn(V, D, generator=g).to(dt).to(cuda))
    ids = tokens(T, V, g, "any").to(cuda)
    ids[::5] = torch.tensor([-1, V, 2 ** 40, -2 ** 40, V + 7], device=cuda)[torch.arange(len(ids[::5])) % 5]
    there = (ids >= 0) & (ids < V)
    for scale in (1.0, math.sqrt(D), -0.3):
        got = embedding.embedding_forward(ids, w, scale=scale)
        want = torch.where(there.unsqueeze(1), w[torch.where(there, ids, 0)].double() * scale, 0.0)
        close(got, want, 2.0 ** -23 * want.abs(), dt, f"{kind} {scale}")
        assert not got[~there].any()
        if scale == 1.0:
            assert torch.equal(got[there], w[ids[there]])


@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("kind", TYPES)
def test_backward(embedding, cuda, kind, T, V, D):
    dt, g = TYPES[kind], torch.Generator().manual_seed(T + V + D)
    dout, _ = matrix(torch.randn(T, D, generator=g).to(dt).to(cuda))
    for order in ("frequent", "any", "one", "two") + (("distinct",) if T <= V else ()):
        ids = tokens(T, V, g, order).to(cuda)
        got = embedding.embedding_backward(ids, dout, V, scale=0.5)
        check_gradient(got, ids, dout, V, 0.5, what=f"{kind} {order}")
        before = torch.randn(V, D, generator=g).to(dt).to(cuda)
        dw = before.clone()
        assert embedding.embedding_backward(ids, dout, dweight=dw, accumulate=True, scale=3.0) is dw
        check_gradient(dw, ids, dout, V, 3.0, before, what=f"{kind} {order} accumulated")


@pytest.mark.parametrize("V", [1, 2, 255, 256, 511, 512, 513, 65535, 65536, 131072, 262143, 262144, 300000])
@pytest.mark.parametrize("T", [5000, 20000])
def test_digits_of_the_sort(embedding, cuda, V, T):
    """Vocabularies on both sides of the digits' ends, ids outside them among the tokens."""
    g = torch.Generator().manual_seed(V)
    ids = torch.randint(-1, V + 1, (T,), generator=g)
    ids[::7] = V - 1
    ids = ids.to(cuda)
    dout = torch.randn(T, 16, generator=g).to(cuda)
    got = embedding.embedding_backward(ids, dout, V)
    check_gradient(got, ids, dout, V, 1.0, what=str(V))


@pytest.mark.parametrize("V", [1024, 131072, 131073, 262144, 262145])
@pytest.mark.parametrize("T", [1023, 1024, 1025, 16384, 32767, 32768, 32769, 33000])
def test_around_what_one_kernel_sorts(embedding, cuda, T, V):
    """Numbers of tokens and sizes of the vocabulary on both sides of the sorts' limits."""
    g = torch.Generator().manual_seed(T + V)
    dout = torch.randn(T, 12, generator=g).to(cuda)
    for order in ("frequent", "any", "one"):
        ids = tokens(T, V, g, order)
        ids[::17] = -1
        ids[3::29] = V - 1
        ids = ids.to(cuda)
        got = torch.full((V, 12), math.nan, device=cuda)
        embedding.embedding_backward(ids, dout, dweight=got, padding_id=0)
        check_gradient(got, ids, dout, V, 1.0, padding_id=0, what=order)


@pytest.mark.parametrize("V,D,dt", [(300000, 128, torch.float32), (5, 20000, torch.bfloat16), (700, 40001, torch.float32)])
def test_zeros_of_many_tokens(embedding, cuda, V, D, dt):
    """More rows than the sort has the time to clear, and rows of which it clears few or one."""
    g = torch.Generator().manual_seed(V)
    T = 40000 if V > 1000 else 33000
    ids = tokens(T, V, g)
    ids[::2] = V // 3
    ids[1::4] = V - 1 - (torch.arange(len(ids[1::4])) % 3) * (V // 5)
    ids = ids.to(cuda)
    if V < 1000:        # few tokens with a gradient, of long rows
        ids[200:] = -1
    dout = torch.randn(200 if V < 1000 else T, D, generator=g).to(dt).to(cuda)
    if V < 1000:
        dout = torch.cat([dout, torch.zeros(1, D, dtype=dt, device=cuda).expand(T - 200, D)])
    got = torch.full((V, D), math.nan, dtype=dt, device=cuda)
    embedding.embedding_backward(ids, dout, dweight=got)
    kept = torch.nonzero(ids >= 0)[:, 0]
    check_gradient(got, ids[kept], dout[kept], V, 1.0)


@pytest.mark.parametrize("T", [5, 33000])
@pytest.mark.parametrize("kind", TYPES)
def test_zeros_of_rows_without_gaps(embedding, cuda, kind, T):
    """Rows off 16 bytes side by side are cleared as one array, from any address to any."""
    g = torch.Generator().manual_seed(35)
    for V, D in [(1, 1), (2, 1), (2, 3), (5, 7), (40, 37), (3000, 257)]:
        ids = (torch.randint(V, (T,), generator=g) if V < 5 else torch.randint(2, V - 2, (T,), generator=g)).to(cuda)
        dout = torch.randn(T, D, generator=g).to(TYPES[kind]).to(cuda)
        nan = torch.full((V, D), math.nan, dtype=TYPES[kind], device=cuda)
        for offset in range(9):
            dw, _ = matrix(nan, 0, offset, "dweight")
            embedding.embedding_backward(ids, dout, dweight=dw)
            check_gradient(dw, ids, dout, V, 1.0, what=f"{V} {D} {offset}")


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 0), (8, 8), (5, 3), (4, 4), (13, 0)])
@pytest.mark.parametrize("kind", TYPES)
def test_strides_and_alignment(embedding, cuda, kind, pad, offset):
    dt = TYPES[kind]
    for T, V, D in [(70, 115, 72), (333, 40, 67), (40, 300, 264), (90, 50, 259)]:
        g = torch.Generator().manual_seed(T + pad + offset)
        ids = tokens(T, V, g).to(cuda)
        w, _ = matrix(torch.randn(V, D, generator=g).to(dt).to(cuda), pad, offset, "weight")
        out, out_buf = matrix(torch.zeros(T, D, dtype=dt, device=cuda), pad, offset, "out")
        assert embedding.embedding_forward(ids, w, out=out) is out
        assert torch.equal(out, w[ids])
        gaps_untouched(out_buf, T, D, pad)
        dout, _ = matrix(torch.randn(T, D, generator=g).to(dt).to(cuda), pad, offset, "dout")
        before = torch.randn(V, D, generator=g).to(dt).to(cuda)
        for accumulate in (False, True):
            dw, buf = matrix(before, pad, offset, "dweight")
            embedding.embedding_backward(ids, dout, dweight=dw, accumulate=accumulate)
            check_gradient(dw, ids, dout, V, 1.0, before if accumulate else None, what=f"{kind} {pad} {offset}")
            gaps_untouched(buf, V, D, pad)


@pytest.mark.parametrize("kind", TYPES)
def test_tokens_without_a_gradient_are_not_read(embedding, cuda, kind):
    """Padding and ids outside the vocabulary: their rows hold NaN."""
    dt, g = TYPES[kind], torch.Generator().manual_seed(3)
    T, V, D = 3000, 400, 80
    ids = tokens(T, V, g).to(cuda)
    ids[::3], ids[1::11], ids[2::13] = 7, V, -5
    gone = (ids < 0) | (ids >= V)
    dout = torch.randn(T, D, generator=g).to(dt).to(cuda)
    dout[gone] = math.nan
    check_gradient(embedding.embedding_backward(ids, dout, V), ids, dout, V, 1.0)
    dout[ids == 7] = math.inf
    got = embedding.embedding_backward(ids, dout, V, padding_id=7)
    check_gradient(got, ids, dout, V, 1.0, padding_id=7)
    assert not got[7].any()
    none = torch.full((T,), V, device=cuda)
    assert not embedding.embedding_backward(none, torch.full_like(dout, math.nan), V).any()
    before = torch.randn(V, D, generator=g).to(dt).to(cuda)
    dw = before.clone()
    embedding.embedding_backward(none, torch.full_like(dout, math.nan), dweight=dw, accumulate=True)
    assert torch.equal(dw, before)


@pytest.mark.parametrize("kind", TYPES)
def test_a_value_that_is_not_finite_shows(embedding, cuda, kind):
    dt = TYPES[kind]
    dout = torch.ones(100, 24, dtype=dt, device=cuda)
    dout[50, 3], dout[60, 4], dout[61, 4] = math.nan, math.inf, -math.inf
    ids = torch.arange(100, device=cuda) // 10
    got = embedding.embedding_backward(ids, dout, 20)
    assert math.isnan(float(got[5, 3])) and math.isnan(float(got[6, 4]))
    got[5, 3] = got[6, 4] = 10.0
    assert bool((got[:10] == 10).all()) and not got[10:].any()


@pytest.mark.parametrize("kind", TYPES)
def test_no_tokens(embedding, cuda, kind):
    dt = TYPES[kind]
    ids = torch.empty(0, dtype=torch.int64, device=cuda)
    w = torch.ones(30, 40, dtype=dt, device=cuda)
    assert embedding.embedding_forward(ids, w).shape == (0, 40)
    dout = torch.empty(0, 40, dtype=dt, device=cuda)
    assert not embedding.embedding_backward(ids, dout, 30).any()
    dw = w.clone()
    embedding.embedding_backward(ids, dout, dweight=dw, accumulate=True)
    assert torch.equal(dw, w)
    assert not embedding.embedding_backward(ids, dout, dweight=dw).any()


def test_shapes_of_ids(embedding, cuda):
    g = torch.Generator().manual_seed(1)
    w = torch.randn(50, 16, generator=g).to(cuda)
    for shape in ((), (1,), (3, 4), (2, 3, 5), (2, 0, 5)):
        ids = torch.randint(0, 50, shape, generator=g).to(cuda)
        out = embedding.embedding_forward(ids, w)
        assert out.shape == (*shape, 16) and torch.equal(out, w[ids])
        got = embedding.embedding_backward(ids, out, 50)
        check_gradient(got, ids, out, 50, 1.0)


def test_equal_inputs_give_equal_bits(embedding, cuda):
    g = torch.Generator().manual_seed(2)
    for T, V, D in [(3000, 50, 72), (70000, 3000, 64)]:
        ids = tokens(T, V, g).to(cuda)
        dout = torch.randn(T, D, generator=g).to(cuda)
        first = embedding.embedding_backward(ids, dout, V)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            assert torch.equal(embedding.embedding_backward(ids, dout, V), first)
        other = embedding.embedding_backward(ids, dout, V, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other, first)


def test_many_tokens(embedding, cuda):
    """Tiles of the sort longer than the shortest; a segment over thousands of runs."""
    g = torch.Generator().manual_seed(4)
    T, V, D = 1_500_007, 5000, 8
    ids = tokens(T, V, g)
    ids[torch.rand(T, generator=g) < 0.3] = 17
    ids, dout = ids.to(cuda), torch.randn(T, D, generator=g).to(cuda)
    check_gradient(embedding.embedding_backward(ids, dout, V), ids, dout, V, 1.0)


def test_offsets_beyond_32_bits(embedding, cuda):
    """Rows more than 2^32 bytes from the first."""
    V, D = 1_100_000, 2100
    w = torch.zeros(V, D, dtype=torch.bfloat16, device=cuda)
    ids = torch.tensor([V - 1, 5, V - 2, V - 1], device=cuda)
    w[V - 1], w[V - 2] = 3.0, 4.0
    out = embedding.embedding_forward(ids, w)
    assert bool((out[0] == 3).all()) and bool((out[2] == 4).all()) and not out[1].any()
    dout = torch.ones(4, D, dtype=torch.bfloat16, device=cuda)
    w[7] = 1.0
    embedding.embedding_backward(ids, dout, dweight=w)
    assert bool((w[V - 1] == 2).all()) and bool((w[V - 2] == 1).all()) and bool((w[5] == 1).all())
    assert float(w.float().sum()) == 4 * D


def test_in_a_graph(embedding, cuda):
    """Captured calls replay on new inputs; two graphs of one pool share their workspaces."""
    g = torch.Generator().manual_seed(6)
    T, V, D = 2000, 700, 48
    w = torch.randn(V, D, generator=g).to(cuda)
    ids, dout = tokens(T, V, g).to(cuda), torch.randn(T, D, generator=g).to(cuda)
    embedding.embedding_backward(ids, embedding.embedding_forward(ids, w), V)
    torch.cuda.synchronize()
    graphs, results = [], []
    for scale in (1.0, 2.0):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=graphs[0].pool() if graphs else None):
            results.append((embedding.embedding_forward(ids, w, scale=scale),
                            embedding.embedding_backward(ids, dout, V, scale=scale)))
        graphs.append(graph)
    for seed in (7, 8):
        g = torch.Generator().manual_seed(seed)
        ids.copy_(tokens(T, V, g))
        dout.copy_(torch.randn(T, D, generator=g))
        for graph, (out, dw), scale in zip(graphs, results, (1.0, 2.0)):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w[ids] * scale)
            check_gradient(dw, ids, dout, V, scale)


def test_another_stream(embedding, cuda):
    """A result on another stream, and memory given back while that stream still works."""
    g = torch.Generator().manual_seed(9)
    T, V, D = 20000, 3000, 128
    ids, dout = tokens(T, V, g).to(cuda), torch.randn(T, D, generator=g).to(cuda)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = embedding.embedding_backward(ids, dout, V, stream=stream)
        again = dout.clone()
        out = embedding.embedding_forward(ids, got, stream=stream)
        del again
        torch.empty(T, D, device=cuda).fill_(math.nan)
        torch.cuda.current_stream().wait_stream(side)
        check_gradient(got, ids, dout, V, 1.0)
        assert torch.equal(out, got[ids])


def test_autograd(embedding, cuda):
    g = torch.Generator().manual_seed(10)
    V, D = 60, 12
    ids = torch.randint(0, V, (3, 40), generator=g).to(cuda)
    w = torch.randn(V, D, generator=g).to(cuda).requires_grad_()
    target = torch.randn(3, 40, D, generator=g).to(cuda)
    loss = (embedding.embedding(ids, w, 0.5, padding_id=4) - target).square().sum()
    got, = torch.autograd.grad(loss, w, create_graph=True)
    keep = (ids != 4).unsqueeze(-1)
    x = w.detach().double().requires_grad_()
    row = 0.5 * x[ids]
    row = torch.where(keep, row, row.detach())
    exact, = torch.autograd.grad((row - target.double()).square().sum(), x, create_graph=True)
    assert torch.allclose(got.double(), exact, rtol=1e-5, atol=1e-5)
    # the gradient's own gradient
    second, = torch.autograd.grad(got.square().sum(), w)
    want, = torch.autograd.grad(exact.square().sum(), x)
    assert torch.allclose(second.double(), want, rtol=1e-4, atol=1e-4)
    # an expanded gradient, and a table that is not trained
    embedding.embedding(ids, w).sum().backward()
    count = torch.zeros(V, device=cuda).index_add_(0, ids.flatten(), torch.ones(120, device=cuda))
    assert torch.equal(w.grad, count.unsqueeze(1).expand(V, D))
    assert not embedding.embedding(ids, w.detach()).requires_grad


def test_gradient_against_differences(embedding, cuda):
    g = torch.Generator().manual_seed(11)
    T, V, D = 50, 9, 6
    ids = torch.randint(0, V, (T,), generator=g).to(cuda)
    dout = torch.randint(-8, 9, (T, D), generator=g).float().to(cuda)
    w = torch.randint(-8, 9, (V, D), generator=g).float().to(cuda)
    grad = embedding.embedding_backward(ids, dout, V, scale=0.5)

    def value(x):       # of small whole numbers: exact
        return float((embedding.embedding_forward(ids, x, scale=0.5).double() * dout.double()).sum())

    for v in range(V):
        for d in range(D):
            up, down = w.clone(), w.clone()
            up[v, d] += 1
            down[v, d] -= 1
            assert (value(up) - value(down)) / 2 == float(grad[v, d])


def test_refusals_of_the_binding(embedding, cuda):
    ids = torch.zeros(6, dtype=torch.int64, device=cuda)
    w = torch.zeros(10, 8, device=cuda)
    dout = torch.zeros(6, 8, device=cuda)
    for bad in (ids.int(), ids.cpu(), [0, 1]):
        with pytest.raises(TypeError):
            embedding.embedding_forward(bad, w)
    with pytest.raises(ValueError):
        embedding.embedding_forward(ids.expand(2, 6).t(), w)
    for bad in (w.half(), w.cpu()):
        with pytest.raises(TypeError):
            embedding.embedding_forward(ids, bad)
    for bad in (w.t(), w[0]):
        with pytest.raises(ValueError):
            embedding.embedding_forward(ids, bad)
    with pytest.raises(ValueError):
        embedding.embedding_forward(ids, w, out=dout[:5])
    with pytest.raises(TypeError):
        embedding.embedding_forward(ids, w, out=dout.bfloat16())
    with pytest.raises(ValueError):
        embedding.embedding_backward(ids, dout[:5], 10)
    with pytest.raises(ValueError):
        embedding.embedding_backward(ids, dout)
    with pytest.raises(ValueError):
        embedding.embedding_backward(ids, dout, 10, accumulate=True)
    with pytest.raises(ValueError):
        embedding.embedding_backward(ids, dout, 11, dweight=w)
    with pytest.raises(ValueError):
        embedding.embedding_backward(ids, dout, dweight=w[:, :7])
    with pytest.raises(RuntimeError):
        embedding.embedding_backward(ids, dout, 10, scale=math.inf)
    with pytest.raises(RuntimeError):
        embedding.embedding_backward(ids, w[:6], dweight=w)       # the gradient over its own input
