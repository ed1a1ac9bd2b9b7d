"""Chunks, windows and log probabilities where calls meet: offsets past 32 bits, graphs that share a workspace, requests that share
pages, gradients inside graphs and of gradients."""
import numpy as np
import pytest

from tests._rows_ref import Rows
from tests.test_gpu_kv_attention import handle, lqm  # noqa: F401
from tests.test_gpu_logprobs import check, gradient64, rows

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_a_cache_past_32_bits(lqm, handle, window, sinks):  # noqa: F811
    """The same pages behind 4 GiB of others."""
    c = Rows(lqm, [4, 4], [700, 90], hq=8, hkv=8, bits=8, window=window, sinks=sinks, seed=1)
    want, one = c.chunk(handle), c.decode(handle)
    small, total = c.cache.pages, c.cache.pages.shape[0]
    before = 2 ** 32 // small[0].numel() + 1
    pages = torch.zeros((before + total,) + small.shape[1:], dtype=small.dtype, device="cuda")
    pages[before:] = small
    c.cache = lqm.KVCache(pages, page_size=c.page, kv_heads=8, head_dim=128, bits=8)
    c.dev["bt"] += before
    got, other = c.chunk(handle), c.decode(handle)
    for a, b in zip(want + one, got + other):
        assert torch.equal(a, b)
    c.check(*got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_past_32_bits(lqm, handle, dtype):  # noqa: F811
    x, t = rows(2, 1000, dtype, seed=2)
    far = 2 ** 31 + 8
    wide = torch.zeros(far + 1000, dtype=x.dtype, device="cuda")
    y = wide.as_strided((2, 1000), (far, 1))
    y.copy_(x)
    check(x, t, handle.token_logprobs(y, t, top=3), 3)
    leaf = y.requires_grad_()
    logprob, entropy, _, _ = handle.token_logprobs(leaf, t)
    one = torch.ones(2, device="cuda")
    d, = torch.autograd.grad([logprob, entropy], [leaf], [one, one])
    want, bound = gradient64(x, t, one, one)
    assert torch.all((d.cpu().double() - want).abs() <= bound)


def test_requests_that_share_pages(lqm, handle):  # noqa: F811
    c = Rows(lqm, [40, 40], [600, 600], seed=3, poison=False)
    c.dev["bt"][1] = c.dev["bt"][0]
    c.bt[1] = c.bt[0]
    c.q[40:] = c.q[:40]
    out, lse = c.chunk(handle)
    c.check(out, lse)


def test_graphs_that_share_a_workspace(lqm, handle):  # noqa: F811
    """Three captured calls that leave partial sums, replayed in every order."""
    a, b = Rows(lqm, [20], [9000], hq=2, hkv=2, seed=4), Rows(lqm, [1] * 3, [5000, 70, 800], window=900, sinks=4, seed=5)
    x, t = rows(2, 60000, "bf16", seed=6)
    calls = [lambda: a.chunk(handle), lambda: b.decode(handle), lambda: handle.token_logprobs(x, t, top=4)]
    want = [[o.clone() for o in f()] for f in calls]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = f()
        graphs.append((g, got))
    for order in ([0, 1, 2], [2, 1, 0], [1, 0, 2], [0, 0, 2, 2, 1, 1]):
        for _, got in graphs:
            for o in got:
                o.zero_()
        for k in order:
            graphs[k][0].replay()
        torch.cuda.synchronize()
        for (_, got), w in zip(graphs, want):
            assert all(torch.equal(o, p) for o, p in zip(got, w))
    handle.sync()


def test_a_captured_gradient(lqm, handle):  # noqa: F811
    x, t = rows(3, 20000, "bf16", seed=7)
    y, u = rows(3, 20000, "bf16", seed=8)
    one = torch.ones(3, device="cuda")

    def step(leaf):
        logprob, entropy, _, _ = handle.token_logprobs(leaf, t)
        return torch.autograd.grad([logprob, entropy], [leaf], [one, one])[0]
    leaf = x.clone().requires_grad_()
    step(leaf)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        d = step(leaf)
    for a, b in ((x, t.clone()), (y, u)):
        leaf.data.copy_(a)
        t.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        want, bound = gradient64(a, b, one, one)
        assert torch.all((d.cpu().double() - want).abs() <= bound)


def test_no_second_derivative(lqm, handle):  # noqa: F811
    x, t = rows(2, 50, "f32", seed=9)
    leaf = x.requires_grad_()
    logprob, _, _, _ = handle.token_logprobs(leaf, t)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(logprob.sum(), leaf, create_graph=True)


def test_alternatives_carry_no_gradient(lqm, handle):  # noqa: F811
    x, t = rows(2, 50, "f32", seed=10)
    _, _, ids, best = handle.token_logprobs(x.requires_grad_(), t, top=3)
    assert not ids.requires_grad and not best.requires_grad


def test_rows_that_are_one(lqm, handle):  # noqa: F811
    """Broadcast rows: their gradients come one by one, and torch sums them."""
    x, t = rows(1, 300, "f32", seed=11)
    leaf = x.requires_grad_()
    tokens = torch.tensor([3, 5, 3, 299], device="cuda")
    logprob, entropy, _, _ = handle.token_logprobs(leaf.expand(4, 300), tokens)
    d, = torch.autograd.grad(logprob.sum(), leaf)
    many = x.detach().expand(4, 300).contiguous()
    want, bound = gradient64(many, tokens, torch.ones(4), torch.zeros(4))
    assert torch.all((d.cpu().double() - want.sum(0)).abs() <= bound.sum(0) + 4 * 2.0 ** -24 * want.abs().sum(0))
