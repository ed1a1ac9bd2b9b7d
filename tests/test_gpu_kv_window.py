"""kv_attention through a sliding window with sinks, against a 64-bit evaluation (bounds: tests/_rows_ref.py)."""
import numpy as np
import pytest

from tests._rows_ref import Rows
from tests.test_gpu_kv_attention import SHAPES, handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,window,sinks", [(1, 1, 0), (300, 1, 0), (300, 1, 5), (300, 16, 0), (300, 17, 1), (300, 100, 4), (300, 100, 16),
                                            (300, 284, 15), (300, 299, 0), (300, 300, 3), (300, 5000, 7), (2049, 130, 33), (17, 16, 1)])
def test_one_token(lqm, handle, bits, D, dtype, n, window, sinks):  # noqa: F811
    c = Rows(lqm, [1], [n], D=D, bits=bits, dtype=dtype, window=window, sinks=sinks, seed=n + window)
    c.check(*c.decode(handle), dense=False)
    handle.sync()


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("T,hq,hkv", [(2, 4, 4), (4, 8, 2), (7, 6, 2), (16, 2, 1), (33, 4, 2), (64, 5, 5), (3, 24, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (40, 0), (65, 20), (1000, 4)])
def test_several_tokens(lqm, handle, bits, D, T, hq, hkv, window, sinks):  # noqa: F811
    """Every row has a window of its own; rows of requests shorter than T see nothing."""
    c = Rows(lqm, [T] * 6, [T, 1, 0, T - 1, 100 + T, 257], hq=hq, hkv=hkv, D=D, bits=bits, window=window, sinks=sinks, seed=T)
    c.check(*c.decode(handle), dense=False)


@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("window,sinks", [(48, 0), (200, 49), (1, 1000)])
def test_batches_of_ragged_lengths(lqm, handle, page, window, sinks):  # noqa: F811
    lens = [int(n) for n in np.random.default_rng(page).integers(1, 1500, 40)]
    c = Rows(lqm, [1] * 40, lens, hq=8, hkv=4, page=page, window=window, sinks=sinks, seed=page)
    c.check(*c.decode(handle), dense=False)


@pytest.mark.parametrize("T,hq", [(1, 8), (4, 8), (16, 4)])
def test_long_context_is_split_over_blocks(lqm, handle, T, hq):  # noqa: F811
    c = Rows(lqm, [T] * 2, [20000, 9001], hq=hq, hkv=2, window=6000, sinks=100, seed=T)
    a, b = c.decode(handle), c.decode(handle)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a, dense=False)


def test_a_window_of_everything_is_no_window(lqm, handle):  # noqa: F811
    c = Rows(lqm, [3] * 4, [700, 5, 64, 3], seed=4)
    want = c.decode(handle)
    for window, sinks in ((700, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 700)):
        c.window, c.sinks = window, sinks
        got = c.decode(handle)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_pages_outside_the_window_need_not_exist(lqm, handle):  # noqa: F811
    c = Rows(lqm, [2], [1000], window=100, sinks=10, seed=9)
    want = c.decode(handle)
    c.dev["bt"][0, 1:(1000 - 101) // 64] = -7        # pages between the sinks' and the windows'
    got = c.decode(handle)
    handle.sync()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.dev["bt"][0, 0] = -7
    c.decode(handle)
    with pytest.raises(lqm.LQError) as e:
        handle.sync()
    assert e.value.status == lqm.LQ_ERR_INDEX


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_that_are_no_numbers_stay_with_the_rows_that_see_them(lqm, handle, bits, D, dtype):  # noqa: F811
    """Token j is NaN: rows whose window has passed it answer as if it were not there."""
    T, n, window, sinks = 8, 90, 30, 2
    c = Rows(lqm, [T], [n], hq=4, hkv=2, D=D, bits=bits, dtype=dtype, window=window, sinks=sinks, seed=3)
    good = c.decode(handle)
    clean = [m.copy() for m in c.meta]
    for j in (n - T + 3 - window, n - T + 4, 1, n - 1):
        sees = np.array([(j <= p and j > p - window) or j < sinks for p in range(n - T, n)])
        assert sees.any()
        s = torch.from_numpy(sees).cuda()
        page, tile, at = c.where(0, j)
        for which in (3, 1):                             # Z of the values, of the keys
            c.meta = [m.copy() for m in clean]
            c.meta[which][page, :, tile, at, 1] = np.nan
            c.repack()
            out, lse = c.decode(handle)
            assert torch.equal(out[~s], good[0][~s]) and torch.equal(lse[~s], good[1][~s])
            if which == 3:
                assert torch.equal(lse, good[1])
                assert bool(out[s][..., 32:64].isnan().all()) and not bool(out[s][..., :32].isnan().any())
            else:
                assert bool(out[s].isnan().all()) and bool(lse[s].isnan().all())


def test_captured_calls_follow_the_lengths(lqm, handle):  # noqa: F811
    c = Rows(lqm, [1] * 3, [900, 300, 70], window=128, sinks=4, seed=5, poison=False)
    out, lse = c.decode(handle)
    q = c.q.view(3, 1, c.hq, c.D)
    o = torch.empty_like(q)
    l = torch.empty(3, 1, c.hq, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        handle.kv_attention(q, c.cache, c.dev["bt"], c.dev["lens"], scale=c.scale, window=128, sinks=4, out=o, lse=l)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o.view_as(out), out) and torch.equal(l.view_as(lse), lse)
    c.lens = [901, 17, 0]
    c.dev["lens"].copy_(torch.tensor(c.lens))
    g.replay()
    torch.cuda.synchronize()
    c.check(o.view_as(out), l.view_as(lse), dense=False)


def test_another_stream(lqm, handle):  # noqa: F811
    c = Rows(lqm, [1] * 5, [500] * 5, window=77, sinks=1, seed=6)
    want = c.decode(handle)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.decode(handle, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
