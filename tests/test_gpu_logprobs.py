"""token_logprobs and its gradient against a 64-bit evaluation.

Bounds, with d_i = x_i - max x, p the probabilities, M1 = sum p |d|, M2 = sum p d^2 and k = V / 256 + 40 additions one after
another at most (a thread's, then those that join threads and blocks):
* a term e^d is off by (|d| + 1) 2^-21 relatively (the rounding of d and of d log2 e, and the exponential's own 2^-22), so
  s by e_s = (M1 + 1) 2^-21 + k 2^-24, ln s and with it lse and a log probability by that and their own roundings;
* w = sum e^d d by (M2 + M1) 2^-21 + M1 k 2^-24 relative to s, so the entropy ln s - w / s by that and (1 + M1) e_s;
* a gradient p (-g - h (ln p + H)) + g: p by (|ln p| + 2) 2^-21 + e_lse, H by e_H, and half a step of the type.
"""
import ctypes

import numpy as np
import pytest

from tests.test_gpu_kv_attention import handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rows(n, V, dtype, pad=0, seed=0, sigma=3.0, banned=0.0, lead=0):
    g = torch.Generator().manual_seed(seed * 1000 + V)
    x = torch.randn(n, V + pad, generator=g) * sigma
    if banned:
        x[torch.rand(x.shape, generator=g) < banned] = -np.inf
    flat = torch.empty(n * (V + pad) + lead, dtype=DT[dtype], device="cuda")
    flat[lead:] = x.flatten().to(DT[dtype])
    t = torch.randint(0, V, (n,), generator=g)
    return flat[lead:].view(n, V + pad)[:, :V], t.cuda()


def exact(x, t):
    x = x.double().cpu()
    V = x.shape[1]
    m = x.amax(1, keepdim=True)
    d = torch.where(torch.isinf(x), torch.zeros_like(x), x - m)
    p = torch.where(torch.isinf(x), torch.zeros_like(x), torch.exp(x - m))
    s = p.sum(1, keepdim=True)
    p /= s
    M1, M2 = (p * d.abs()).sum(1), (p * d * d).sum(1)
    lse = (m + s.log())[:, 0]
    H = s.log()[:, 0] + M1
    k = V / 256 + 40
    es = (M1 + 1) * 2.0 ** -21 + k * 2.0 ** -24
    e_lse = es + 2.0 ** -23 * (lse.abs() + m[:, 0].abs() + s.log()[:, 0].abs())
    e_H = (M2 + M1) * 2.0 ** -21 + M1 * k * 2.0 ** -24 + (2 + M1) * es + 2.0 ** -22 * (s.log()[:, 0] + M1)
    t = t.cpu()
    lp = torch.where(t >= 0, torch.gather(x, 1, t.clamp(min=0)[:, None])[:, 0] - lse, 0.0)
    return lp, H, lse, p, e_lse, e_H


def check(x, t, out, top):
    lp, H, lse, p, e_lse, e_H = exact(x, t)
    logprob, entropy, ids, best = out
    assert torch.all((logprob.cpu().double() - lp).abs() <= e_lse + 2.0 ** -23 * (lp.abs() + 1)), (logprob.cpu().double() - lp).abs().max()
    assert torch.all((entropy.cpu().double() - H).abs() <= e_H), (entropy.cpu().double() - H).abs().max()
    if not top:
        assert ids is None and best is None
        return
    v, order = torch.sort(x.float().cpu(), dim=1, descending=True, stable=True)
    assert torch.equal(ids.cpu(), order[:, :top])
    want = v[:, :top].double() - lse[:, None]
    err = (best.cpu().double() - want).abs()
    live = ~torch.isinf(want)
    assert torch.equal(torch.isneginf(best.cpu()), ~live)
    assert torch.all(err[live] <= (e_lse[:, None] + 2.0 ** -23 * (want.abs() + 1))[live])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 255, 1000, 4097, 8191, 8193, 32000, 50021])
@pytest.mark.parametrize("n,top", [(1, 0), (1, 5), (3, 1), (5, 20), (2, 64)])
def test_rows_of_any_length(lqm, handle, dtype, V, n, top):  # noqa: F811
    x, t = rows(n, V, dtype, seed=top)
    top = min(top, V)
    check(x, t, handle.token_logprobs(x, t, top=top), top)
    handle.sync()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,lead", [(0, 1), (3, 0), (8, 5), (1, 7), (64, 2)])
@pytest.mark.parametrize("V", [5, 997, 16390])
def test_strides_and_starts_of_any_alignment(lqm, handle, dtype, pad, lead, V):  # noqa: F811
    x, t = rows(6, V, dtype, pad=pad, lead=lead, seed=pad)
    check(x, t, handle.token_logprobs(x, t, top=5), 5)


@pytest.mark.parametrize("n,V,top", [(700, 5000, 3), (3000, 300, 0), (1300, 9000, 9), (40, 131072, 10)])
def test_many_rows(lqm, handle, n, V, top):  # noqa: F811
    x, t = rows(n, V, "bf16", seed=1)
    a, b = handle.token_logprobs(x, t, top=top), handle.token_logprobs(x, t, top=top)
    assert all(u is None or torch.equal(u, w) for u, w in zip(a, b))
    check(x, t, a, top)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("how", ["constant", "few values", "up", "down", "negative", "zeros of both signs", "one thread", "by thread",
                                 "subnormal"])
@pytest.mark.parametrize("top", [1, 8, 9, 64])
def test_equal_logits_go_to_the_lower_id(lqm, handle, dtype, how, top):  # noqa: F811
    V, n = 150011, 3
    g = torch.Generator().manual_seed(5)
    j = torch.arange(V).float()
    x = {"constant": torch.full((V,), -2.5), "few values": torch.randint(-3, 3, (V,), generator=g).float(), "up": j / 64,
         "down": -j / 64, "negative": -torch.randint(1, 30, (V,), generator=g).float(),
         "zeros of both signs": torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0),
         "one thread": torch.where(j % 2048 < 8, 9.0, -torch.rand(V, generator=g)),
         "by thread": -(j // 8 % 512 * 64 + j // 4096 * 8 + j % 8) / 64.0,
         "subnormal": torch.randint(-5, 6, (V,), generator=g).float() * 2.0 ** -24}[how]
    x = x.expand(n, V).to(DT[dtype]).contiguous().cuda()
    t = torch.tensor([0, V - 1, 77], device="cuda")
    check(x, t, handle.token_logprobs(x, t, top=top), top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_banned_tokens(lqm, handle, dtype):  # noqa: F811
    x, t = rows(6, 30000, dtype, banned=0.5, seed=3)
    x[torch.arange(6), t] = 1.0
    check(x, t, handle.token_logprobs(x, t, top=20), 20)
    # fewer possible tokens than alternatives asked for; and one only
    x[0] = -np.inf
    x[0, 7], x[0, 29000], t[0] = 2.0, 2.0, 7
    x[1] = -np.inf
    x[1, 123], t[1] = -50.0, 123
    out = handle.token_logprobs(x, t, top=20)
    check(x, t, out, 20)
    assert float(out[0][1]) == 0.0 and float(out[1][1]) == 0.0
    # a banned token was given
    t[0] = 8
    assert float(handle.token_logprobs(x, t)[0][0]) == -np.inf


def test_rows_that_are_no_distribution(lqm, handle):  # noqa: F811
    x, t = rows(4, 9000, "f32", seed=4)
    x[0] = -np.inf
    x[1, 8888] = np.nan
    x[2, 5] = np.inf
    for n in (4, 1):
        logprob, entropy, ids, best = handle.token_logprobs(x[:n], t[:n], top=3)
        assert float(logprob[0]) == -np.inf and float(entropy[0]) == 0 and bool((best[0] == -np.inf).all())
        assert ids[0].tolist() == [0, 1, 2]
    logprob, entropy, ids, best = handle.token_logprobs(x, t, top=3)
    assert bool(logprob[1:3].isnan().all()) and bool(entropy[1:3].isnan().all()) and bool(best[1:3].isnan().all())
    assert int(ids[1, 0]) == 8888 and int(ids[2, 0]) == 5
    check(x[3:], t[3:], tuple(o[3:] for o in (logprob, entropy, ids, best)), 3)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bad", [np.inf, np.nan, -np.nan])
@pytest.mark.parametrize("n", [1, 400])
def test_ids_among_many_that_are_no_numbers(lqm, handle, dtype, bad, n):  # noqa: F811
    """NaN counts as the largest, infinity comes next, equal ones by id."""
    x, t = rows(n, 30000, dtype, seed=15)
    x[:, 1000:29000:3] = bad
    x[:, 17], x[:, 29999] = np.inf, np.nan
    logprob, entropy, ids, best = handle.token_logprobs(x, t, top=40)
    assert bool(logprob.isnan().all()) and bool(entropy.isnan().all()) and bool(best.isnan().all())
    key = torch.where(x[0].isnan(), 2, torch.where(x[0] == np.inf, 1, 0)).cpu()
    want = torch.sort(key, descending=True, stable=True)[1][:40]
    assert key[want].min() > 0
    assert bool((ids.cpu() == want).all())


def test_large_logits(lqm, handle):  # noqa: F811
    x, t = rows(3, 5000, "f32", sigma=1e4, seed=6)
    x[1] += 3e38
    check(x, t, handle.token_logprobs(x, t, top=4), 4)


def test_tokens_left_out(lqm, handle):  # noqa: F811
    x, t = rows(5, 3000, "bf16", seed=7)
    t[1], t[3] = -1, -(2 ** 63)
    check(x, t, handle.token_logprobs(x, t), 0)
    handle.sync()
    t[2] = 3000
    u = t.clone()
    u[2] = -1
    got = handle.token_logprobs(x, t)
    with pytest.raises(lqm.LQError) as e:
        handle.sync()
    assert e.value.status == lqm.LQ_ERR_INDEX
    check(x, u, got, 0)


def gradient64(x, t, g, h):
    """The formula in 64 bits, and the bound of its fp32 evaluation."""
    lp, H, lse, p, e_lse, e_H = exact(x, t)
    t, g, h = t.cpu(), g.cpu().double(), h.cpu().double()
    g = torch.where(t >= 0, g, 0.0)
    ln = torch.where(p > 0, x.double().cpu() - lse[:, None], 0.0)
    inner = g[:, None].abs() + h[:, None].abs() * (ln.abs() + H[:, None])
    d = -p * (g[:, None] + h[:, None] * (ln + H[:, None]))
    d[torch.arange(len(t)), t.clamp(min=0)] += g
    err = p * inner * ((ln.abs() + 4) * 2.0 ** -21 + e_lse[:, None]) + p * h[:, None].abs() * e_H[:, None] + 2.0 ** -23 * g[:, None].abs() * p
    err[torch.arange(len(t)), t.clamp(min=0)] += 2.0 ** -23 * g.abs()
    eps = torch.finfo(x.dtype)
    return d, err + eps.eps / 2 * (d.abs() + err) + eps.smallest_normal * eps.eps


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,V,pad,lead", [(1, 1, 0, 0), (1, 7, 0, 0), (3, 1000, 0, 0), (5, 8193, 3, 1), (2, 50021, 8, 0), (700, 2000, 0, 0)])
def test_gradient(lqm, handle, dtype, n, V, pad, lead):  # noqa: F811
    x, t = rows(n, V, dtype, pad=pad, lead=lead, seed=8, banned=0.1 if V > 100 else 0.0)
    x[torch.arange(n), t] = 1.0
    if n > 2:
        t[1] = -1
    g, h = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    leaf = x.detach().requires_grad_()
    logprob, entropy, ids, best = handle.token_logprobs(leaf, t, top=min(3, V))
    assert logprob.requires_grad and entropy.requires_grad and not best.requires_grad and not ids.requires_grad
    d, = torch.autograd.grad([logprob, entropy], [leaf], [g, h])
    assert d.dtype is x.dtype and d.shape == x.shape
    want, bound = gradient64(x, t, g, h)
    err = (d.cpu().double() - want).abs()
    assert torch.all(err <= bound), float((err / bound).max())
    assert torch.all(d.cpu()[torch.isneginf(x.cpu())] == 0)
    # one of the outputs only; gradients that are broadcast
    for i, other in ((0, torch.zeros_like(h)), (1, torch.zeros_like(g))):
        out = handle.token_logprobs(leaf, t)[i]
        d, = torch.autograd.grad(out.sum(), leaf)
        one = torch.ones_like(g)
        want, bound = gradient64(x, t, one if i == 0 else other, one if i == 1 else other)
        assert torch.all((d.cpu().double() - want).abs() <= bound)


def test_gradient_against_differences(lqm, handle):  # noqa: F811
    """Along random directions: central differences of the definition in 64 bits (their own error: e^2 / 6 times a third
    derivative, below 30 |u|^3 here)."""
    x, t = rows(4, 500, "f32", seed=9, sigma=1.0)
    leaf = x.detach().requires_grad_()
    logprob, entropy, _, _ = handle.token_logprobs(leaf, t)
    a, b = torch.randn(4), torch.randn(4)
    d, = torch.autograd.grad([logprob, entropy], [leaf], [a.cuda(), b.cuda()])

    def loss(y):
        lp = torch.log_softmax(y, 1)
        return (a.double() * lp[torch.arange(4), t.cpu()]).sum() - (b.double() * (lp.exp() * lp).sum(1)).sum()
    for k in range(5):
        u = torch.randn(4, 500, generator=torch.Generator().manual_seed(k)).double()
        u /= u.norm()
        e = 1e-3
        diff = (loss(x.cpu().double() + e * u) - loss(x.cpu().double() - e * u)) / (2 * e)
        want, bound = gradient64(x, t, a, b)
        assert abs(float((d.cpu().double() * u).sum() - diff)) <= float((bound * u.abs()).sum()) + 30 * e * e / 6


def test_gradient_over_the_logits(lqm, handle):  # noqa: F811
    """The C call may write the gradient over the logits."""
    from bit_weight_quantized_dequant_gb300 import _lq
    x, t = rows(5, 4099, "bf16", pad=5, seed=10)
    g, h = torch.randn(5, device="cuda"), torch.randn(5, device="cuda")
    want, bound = gradient64(x, t, g, h)
    logprob, entropy, lse, _, _ = handle._token_logprobs(x, t, 0, None)
    a = _lq.lq_logprobs_grad_args(x.data_ptr(), x.data_ptr(), _lq.BF16, 5, 4099, 4104, 4104, t.data_ptr(), lse.data_ptr(), entropy.data_ptr(),
                                  g.data_ptr(), h.data_ptr())
    assert handle._lib.lq_logprobs_grad(handle.raw, ctypes.byref(a), None) == 0
    torch.cuda.synchronize()
    assert torch.all((x.cpu().double() - want).abs() <= bound)


def test_gradient_of_a_row_of_nothing(lqm, handle):  # noqa: F811
    x, t = rows(2, 300, "f32", seed=11)
    x[0] = -np.inf
    leaf = x.detach().requires_grad_()
    logprob, entropy, _, _ = handle.token_logprobs(leaf, t)
    d, = torch.autograd.grad([logprob, entropy], [leaf], [torch.zeros(2, device="cuda"), torch.ones(2, device="cuda")])
    assert bool((d[0] == 0).all()) and bool(d[1].isfinite().all())


def test_captured_calls(lqm, handle):  # noqa: F811
    x, t = rows(3, 40000, "bf16", seed=12)
    y, u = rows(3, 40000, "bf16", seed=13)
    handle.token_logprobs(x, t, top=5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = handle.token_logprobs(x, t, top=5)
    for a, b in ((x.clone(), t.clone()), (y, u)):
        x.copy_(a)
        t.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        check(x, t, out, 5)


def test_another_stream(lqm, handle):  # noqa: F811
    x, t = rows(3, 40000, "bf16", seed=14)
    want = handle.token_logprobs(x, t, top=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = handle.token_logprobs(x, t, top=5, stream=s)
    leaf = x.detach().requires_grad_()
    logprob = handle.token_logprobs(leaf, t, stream=s)[0]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(logprob, want[0])
    d, = torch.autograd.grad(logprob.sum(), leaf)
    one = torch.ones(3, device="cuda")
    grad, bound = gradient64(x, t, one, torch.zeros_like(one))
    assert torch.all((d.cpu().double() - grad).abs() <= bound)


def test_no_rows(lqm, handle):  # noqa: F811
    x = torch.empty(0, 100, device="cuda")
    out = handle.token_logprobs(x, torch.empty(0, dtype=torch.int64, device="cuda"), top=2)
    assert [tuple(o.shape) for o in out] == [(0,), (0,), (0, 2), (0, 2)]
