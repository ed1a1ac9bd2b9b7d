"""The gradient of log probabilities and entropy of logits far from zero: a distribution does not depend on where its
logits lie, and neither may the gradient's accuracy.

The bound is that of tests/test_gpu_logprobs.py without any |lse|.  lse and its rest are m + ln s without an error of their own,
so what p is off by comes from s (e_s), ln s (2^-23 of it), and ln p = (x - lse) - rest.  x - lse is exact where x lies between lse / 2
and 2 lse; elsewhere |x - lse| >= |lse| / 2, the rest is below 2^-22 of that, and the rounding below 2^-23 |ln p|.  The rest is no
larger than ln s (m is an fp32 number), so its own product with log2 e and the sum's rounding are below 2^-23 (|ln p| + ln s):
(|ln p| + 4) 2^-21 with the exponential's 2^-22, and 2^-22 ln s.
"""
import ctypes

import numpy as np
import pytest

from tests.test_gpu_kv_attention import handle, lqm  # noqa: F401
from tests.test_gpu_logprobs import DT, exact

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
MOST = float(np.finfo(np.float32).max)


def gradient(x, t, g, h):
    """The formula in 64 bits and its bound; x are logits of any size."""
    x = x.double().cpu()
    t, g, h = t.cpu(), g.cpu().double()[:, None], h.cpu().double()[:, None]
    y = x - x.amax(1, keepdim=True)                    # (exact: the values of a row lie on one grid here, or far apart)
    _, H, lse, p, _, e_H = exact(y, t)
    H, e_H, ln = H[:, None], e_H[:, None], torch.where(p > 0, y - lse[:, None], 0.0)
    M1, k = (p * y.abs()).sum(1, keepdim=True), x.shape[1] / 256 + 40
    e_p = (M1 + 1) * 2.0 ** -21 + k * 2.0 ** -24 + 2.0 ** -22 * lse[:, None].abs() + (ln.abs() + 4) * 2.0 ** -21
    d = -p * (g + h * (ln + H))
    at = torch.arange(len(t)), t
    d[at] += g[:, 0]
    inner = g.abs() + h.abs() * (ln.abs() + H)
    err = p * inner * e_p + p * h.abs() * e_H + 2.0 ** -23 * g.abs() * p
    err[at] += 2.0 ** -23 * g[:, 0].abs()
    return d, err


def run(handle, x, t, g, h):  # noqa: F811
    leaf = x.detach().requires_grad_()
    logprob, entropy, _, _ = handle.token_logprobs(leaf, t)
    d, = torch.autograd.grad([logprob, entropy], [leaf], [g, h])
    want, err = gradient(x, t, g, h)
    eps = torch.finfo(x.dtype)
    bound = err + eps.eps / 2 * (want.abs() + err) + eps.smallest_normal * eps.eps
    off = (d.double().cpu() - want).abs()
    assert torch.all(off <= bound), float((off / bound).max())
    # the gradient of a log probability sums to 0 over its row, within what each of its terms may be off by
    one = torch.ones_like(g)
    d, = torch.autograd.grad(handle.token_logprobs(leaf, t)[0].sum(), leaf)
    want, err = gradient(x, t, one, torch.zeros_like(one))
    bound = (err + eps.eps / 2 * (want.abs() + err) + eps.smallest_normal * eps.eps).sum(1)
    assert torch.all(d.double().cpu().sum(1).abs() <= bound)


def weights(n, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda()


@pytest.mark.parametrize("offset", [0.0, 1e4, -1e4, 1e6, -1e6, 1e8, -1e8, 1e12])
@pytest.mark.parametrize("n,V", [(3, 1000), (2, 32000)])
def test_rows_about_an_offset(lqm, handle, offset, n, V):  # noqa: F811
    """Small logits, moved by what fp32 represents: steps of the offset's last place."""
    step = max(float(np.spacing(np.float32(abs(offset)))) * 2, 2.0 ** -12)
    g = torch.Generator().manual_seed(V)
    x = ((torch.randn(n, V, generator=g, dtype=torch.float64) * 3 / step).round() * step + float(np.float32(offset)))
    assert torch.equal(x.float().double(), x)
    t = torch.randint(0, V, (n,), generator=g).cuda()
    run(handle, x.float().cuda(), t, *weights(n))


@pytest.mark.parametrize("dtype,value", [("f32", -MOST), ("f32", MOST), ("f32", 1e9), ("f32", 1e4), ("bf16", -float(torch.finfo(torch.bfloat16).max)),
                                         ("bf16", 1e4), ("f16", -65504.0), ("f16", 3e4)])
@pytest.mark.parametrize("V", [2, 1000, 30011])
def test_rows_of_one_value(lqm, handle, dtype, value, V):  # noqa: F811
    """A mask by the type's lowest value that leaves nothing, and others: every token is as likely as the next."""
    x = torch.full((3, V), value).to(DT[dtype]).cuda()
    t = torch.tensor([0, V - 1, V // 2], device="cuda")
    run(handle, x, t, *weights(3))


def test_masks_by_the_lowest_value(lqm, handle):  # noqa: F811
    """Some tokens possible, the others at the lowest value: those have no part."""
    g = torch.Generator().manual_seed(3)
    x = torch.full((4, 5000), -MOST)
    keep = torch.rand(4, 5000, generator=g) < 0.1
    x[keep] = torch.randn(int(keep.sum()), generator=g) * 3
    t = keep.float().argmax(1)
    run(handle, x.cuda(), t.cuda(), *weights(4))


def test_both_ends_of_the_range(lqm, handle):  # noqa: F811
    x = torch.full((2, 300), -MOST)
    x[0, 7] = x[0, 9] = MOST
    x[1] = 3e38
    x[1, 5:9] = -3e38
    run(handle, x.cuda(), torch.tensor([7, 0]).cuda(), *weights(2))


def test_rows_cut_into_parts(lqm, handle):  # noqa: F811
    """One long row, which many blocks share: its statistics are joined."""
    x = torch.randint(-4, 4, (1, 200003), generator=torch.Generator().manual_seed(4)).float() * 8 + 1e8
    run(handle, x.cuda(), torch.tensor([11]).cuda(), *weights(1))


def test_the_gradient_follows_the_rest(lqm, handle):  # noqa: F811
    """The C calls: lse and its rest add up to the log-sum-exp; without a rest lse counts as it is."""
    from bit_weight_quantized_dequant_gb300 import _lq
    n, V = 4, 3000
    x = (torch.randint(-4, 4, (n, V), generator=torch.Generator().manual_seed(5)).float() * 8 + 1e8).cuda()
    t = torch.tensor([1, 2, -1, 5], device="cuda")
    lse, rest, logprob = (torch.zeros(n, device="cuda") for _ in range(3))
    a = _lq.lq_logprobs_args(x.data_ptr(), _lq.F32, n, V, V, t.data_ptr(), logprob.data_ptr(), None, lse.data_ptr(), 0, None, None,
                             rest.data_ptr())
    assert handle._lib.lq_logprobs(handle.raw, ctypes.byref(a), None) == 0
    torch.cuda.synchronize()
    want = torch.logsumexp(x.double().cpu() - 1e8, 1)
    _, _, _, _, e_lse, _ = exact(x.double().cpu() - 1e8, t)
    assert torch.all((lse.cpu().double() - 1e8 + rest.cpu().double() - want).abs() <= e_lse)
    one = torch.ones(n, device="cuda")
    for given, total in ((rest, lse.cpu().double() + rest.cpu().double()), (None, lse.cpu().double())):
        d = torch.zeros_like(x)
        b = _lq.lq_logprobs_grad_args(x.data_ptr(), d.data_ptr(), _lq.F32, n, V, V, V, t.data_ptr(), lse.data_ptr(), None, one.data_ptr(), None,
                                      given.data_ptr() if given is not None else None)
        assert handle._lib.lq_logprobs_grad(handle.raw, ctypes.byref(b), None) == 0
        torch.cuda.synchronize()
        ln = x.cpu().double() - total[:, None]
        p = ln.exp()
        w = -p
        w[2] = 0
        w[torch.arange(n), t.cpu().clamp(min=0)] += torch.tensor([1.0, 1.0, 0.0, 1.0]).double()
        bound = p * ((ln.abs() + 4) * 2.0 ** -21) + 2.0 ** -23 * (p + (w + p).abs())
        assert torch.all((d.cpu().double() - w).abs() <= bound)
