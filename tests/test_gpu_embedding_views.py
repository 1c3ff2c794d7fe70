"""Token ids that are a view of something else, as a batch's tokens but for each sequence's last."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def embedding(abi, cuda):
    from zero_sharded_optimizer_gb300 import embedding as module
    return module


VIEWS = {"shifted": lambda t: t[:, :-1], "turned": lambda t: t.t(), "every other": lambda t: t[::2, 1::3],
         "one column": lambda t: t[:, 4], "permuted": lambda t: t.view(4, 2, 10).permute(2, 0, 1)}


@pytest.mark.parametrize("view", VIEWS)
def test_views_give_what_their_copies_give(embedding, cuda, view):
    g = torch.Generator().manual_seed(3)
    V, D = 90, 24
    whole = torch.randint(-1, V + 1, (8, 10), generator=g).to(cuda)
    ids = VIEWS[view](whole)
    assert not ids.is_contiguous()
    w = torch.randn(V, D, generator=g).to(cuda)
    dout = torch.randn(*ids.shape, D, generator=g).to(cuda)
    out, dw = embedding.embedding_forward(ids.contiguous(), w), embedding.embedding_backward(ids.contiguous(), dout, V)
    assert torch.equal(embedding.embedding_forward(ids, w), out)
    assert torch.equal(embedding.embedding_backward(ids, dout, V), dw)
    into = torch.empty_like(out)
    assert embedding.embedding_forward(ids, w, out=into) is into and torch.equal(into, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        a, b = embedding.embedding_forward(ids, w, stream=stream), embedding.embedding_backward(ids, dout, V, stream=stream)
        torch.empty(ids.numel(), dtype=torch.int64, device=cuda).fill_(-1)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, out) and torch.equal(b, dw)
    leaf = w.clone().requires_grad_()
    got = embedding.embedding(ids, leaf)
    whole.fill_(0)                      # the function has its own copy
    got.backward(dout)
    assert torch.equal(got, out) and torch.equal(leaf.grad, dw)


def test_expanded_ids(embedding, cuda):
    """The positions of a batch: the differentiable function takes them, the calls refuse them."""
    w = torch.randn(12, 8, device=cuda).requires_grad_()
    at = torch.arange(10, device=cuda).expand(3, 10)
    out = embedding.embedding(at, w)
    assert torch.equal(out, w[at])
    out.backward(torch.ones_like(out))
    assert bool((w.grad[:10] == 3).all()) and not w.grad[10:].any()
    with pytest.raises(ValueError, match="expanded"):
        embedding.embedding_forward(at, w.detach())


def test_a_view_in_a_graph(embedding, cuda):
    g = torch.Generator().manual_seed(4)
    V, D = 60, 16
    whole, w = torch.randint(0, V, (6, 9), generator=g).to(cuda), torch.randn(V, D, generator=g).to(cuda)
    dout = torch.randn(6, 8, D, generator=g).to(cuda)
    embedding.embedding_backward(whole[:, 1:], embedding.embedding_forward(whole[:, :-1], w), V)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, dw = embedding.embedding_forward(whole[:, :-1], w), embedding.embedding_backward(whole[:, 1:], dout, V)
    for _ in range(2):
        whole.copy_(torch.randint(0, V, (6, 9), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w[whole[:, :-1]])
        assert torch.equal(dw, embedding.embedding_backward(whole[:, 1:].contiguous(), dout, V))
