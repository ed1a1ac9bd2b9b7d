"""kv_attention_chunk against a 64-bit evaluation over the cache's own values (bounds: tests/_rows_ref.py)."""
import numpy as np
import pytest

from tests._rows_ref import Rows
from tests.test_gpu_kv_attention import SHAPES, handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fresh,n", [(1, 1), (1, 17), (2, 130), (16, 16), (65, 65), (100, 300), (128, 128), (129, 513), (300, 1000)])
def test_one_request(lqm, handle, bits, D, dtype, fresh, n):  # noqa: F811
    c = Rows(lqm, [fresh], [n], D=D, bits=bits, dtype=dtype, seed=n)
    c.check(*c.chunk(handle))
    handle.sync()


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (8, 1), (12, 4), (7, 1), (40, 2), (130, 1)])
def test_head_groups(lqm, handle, bits, D, hq, hkv):  # noqa: F811
    c = Rows(lqm, [40, 3, 77], [300, 3, 500], hq=hq, hkv=hkv, D=D, bits=bits, seed=hq)
    c.check(*c.chunk(handle))


def test_ragged_batches(lqm, handle):  # noqa: F811
    """Empty requests, single tokens among chunks, requests shorter than their new rows, lengths past the page list."""
    c = Rows(lqm, [0, 1, 200, 0, 33, 5, 64, 0], [50, 700, 260, 0, 20, 0, 5000, 9], hq=8, hkv=2, seed=1, extra_pages=1)
    c.check(*c.chunk(handle))
    handle.sync()


def test_lengths_past_the_page_list_and_below_zero(lqm, handle):  # noqa: F811
    c = Rows(lqm, [0, 1, 200, 0, 33], [50, 700, 2 ** 31 - 1, -(2 ** 31), -5], seed=2, pages=12)
    c.check(*c.chunk(handle))
    handle.sync()


@pytest.mark.parametrize("page", [16, 32, 48, 128, 256])
def test_page_sizes(lqm, handle, page):  # noqa: F811
    c = Rows(lqm, [100, 3, 128, 61], [1000, 3, 511, 777], page=page, seed=page, extra_pages=2)
    c.check(*c.chunk(handle))


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 3), (128, 0), (128, 128), (129, 130), (300, 4), (100, 600), (5000, 2)])
def test_windows(lqm, handle, bits, D, window, sinks):  # noqa: F811
    c = Rows(lqm, [300, 1, 65, 0, 140], [1100, 900, 65, 40, 141], hq=6, hkv=2, D=D, bits=bits, window=window, sinks=sinks, seed=window)
    c.check(*c.chunk(handle))


def test_many_requests(lqm, handle):  # noqa: F811
    g = np.random.default_rng(3)
    fresh = [int(x) for x in g.integers(0, 12, 700)]
    lens = [int(f + x) for f, x in zip(fresh, g.integers(0, 200, 700))]
    c = Rows(lqm, fresh, lens, hq=2, hkv=1, D=64, page=16, seed=4)
    c.check(*c.chunk(handle))


@pytest.mark.parametrize("hq,hkv", [(8, 1), (2, 2)])
def test_long_contexts_are_cut_and_joined(lqm, handle, hq, hkv):  # noqa: F811
    """Few units of many key blocks: most are cut between blocks, and the joined sums repeat bit for bit."""
    c = Rows(lqm, [20, 70], [30000, 11111], hq=hq, hkv=hkv, seed=7)
    a, b = c.chunk(handle), c.chunk(handle)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a)


@pytest.mark.parametrize("spread", [1e-4, 0.01, 30.0, 2000.0])
def test_scales_far_from_one(lqm, handle, spread):  # noqa: F811
    c = Rows(lqm, [50], [400], spread=spread, seed=8)
    c.check(*c.chunk(handle))


def test_queries_far_from_one(lqm, handle):  # noqa: F811
    for f in (1e-30, 1e-6, 300.0):
        c = Rows(lqm, [50], [400], seed=8)
        c.q.mul_(f)
        c.check(*c.chunk(handle))


def test_agrees_with_the_decode_kernel(lqm, handle):  # noqa: F811
    """The same rows by kv_attention, within both kernels' bounds."""
    c = Rows(lqm, [4] * 3, [300, 77, 1000], window=90, sinks=3, seed=2)
    c.check(*c.chunk(handle))
    c.check(*c.decode(handle), dense=False)


def test_rows_of_no_request_are_left_alone(lqm, handle):  # noqa: F811
    c = Rows(lqm, [30, 0, 100], [90, 5, 100], lead=7, tail=20, seed=11)
    out, lse = torch.full_like(c.q, 3.0), torch.full(c.q.shape[:2], 5.0, device="cuda")
    o, l = c.chunk(handle, out=out, lse=lse)
    assert o is out and l is lse
    c.check(out, lse)
    for r in (slice(0, 7), slice(137, 157)):
        assert bool((out[r] == 3).all()) and bool((lse[r] == 5).all())
    handle.sync()


def test_strided_rows_and_out_over_q(lqm, handle):  # noqa: F811
    c = Rows(lqm, [30, 100], [90, 100], hq=4, hkv=2, seed=12)
    want = c.chunk(handle)
    wide = torch.zeros(130, 4 * 128 + 72, device="cuda", dtype=c.q.dtype)
    q = wide[:, 8:8 + 512].unflatten(1, (4, 128))
    q.copy_(c.q)
    got = c.chunk(handle, q=q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.chunk(handle, q=q, out=q)
    assert torch.equal(q, want[0]) and bool((wide[:, :8] == 0).all()) and bool((wide[:, 520:] == 0).all())


def test_bad_starts_are_moved_and_reported(lqm, handle):  # noqa: F811
    for bad in ([0, -3, 60, 100], [0, 40, 30, 100], [0, 40, 5000, 100], [50, 60, 70, 2 ** 31 - 1], [-2 ** 31, 0, 0, 0]):
        c = Rows(lqm, [40, 30, 30], [90, 80, 70], seed=13, poison=False)
        c.dev["starts"].copy_(torch.tensor(bad))
        out, lse = torch.zeros_like(c.q), torch.zeros(c.q.shape[:2], device="cuda")
        c.chunk(handle, out=out, lse=lse)
        with pytest.raises(lqm.LQError) as e:
            handle.sync()
        assert e.value.status == lqm.LQ_ERR_INDEX
    c = Rows(lqm, [40, 30, 30], [90, 80, 70], seed=13)
    c.check(*c.chunk(handle))
    handle.sync()


def test_pages_outside_the_cache_hide_their_tokens(lqm, handle):  # noqa: F811
    c = Rows(lqm, [100], [400], page=16, seed=14, poison=False)
    for page, j in ((-1, 3), (10 ** 6, 24), (-2 ** 31, 7)):
        c.dev["bt"][0, j] = page
    out, lse = c.chunk(handle)
    with pytest.raises(lqm.LQError) as e:
        handle.sync()
    assert e.value.status == lqm.LQ_ERR_INDEX
    # the same as if those tokens' keys scored nothing: evaluate over what is left
    from tests import _rows_ref as RR
    keep = np.ones(400, bool)
    for j in (3, 24, 7):
        keep[16 * j:16 * j + 16] = False
    j = np.arange(400)
    seen = RR.visible(400, 100, 0, 0) & keep
    q = c.q.float().cpu().numpy()
    for h in range(2):
        k, v = c.k[c.bt[0][j // 16], h, j % 16], c.v[c.bt[0][j // 16], h, j % 16]
        o, s, mass, size = RR.attend(q[:, 4 * h:4 * h + 4], k, v, seen, c.scale)
        assert np.abs(lse[:, 4 * h:4 * h + 4].cpu().numpy() - s).max() < 2.0 ** -18
        assert np.all(np.abs(out[:, 4 * h:4 * h + 4].float().cpu().numpy() - o) <= 2.0 ** -9 * mass + 2.0 ** -8 * np.abs(o) + 2.0 ** -22)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("T", [1, 60, 300])
def test_pages_outside_the_window_need_not_exist(lqm, handle, page, T):  # noqa: F811
    n, window, sinks = 2000, 150, 20
    c = Rows(lqm, [T, 5], [n, 40], page=page, window=window, sinks=sinks, seed=T)
    want = c.chunk(handle)
    handle.sync()
    first = (n - T - window + 1) // page                # the first page with a token in some row's window
    c.dev["bt"][0, -(-sinks // page):first] = -5
    c.dev["bt"][1, -(-40 // page):] = 2 ** 31 - 1
    got = c.chunk(handle)
    handle.sync()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(*got)


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
@pytest.mark.parametrize("n", [40, 300, 3000])
def test_values_that_are_no_numbers_stay_with_the_rows_that_see_them(lqm, handle, bits, D, window, sinks, n):  # noqa: F811
    T = 40
    c = Rows(lqm, [T, 10], [n, 60], hq=4, hkv=2, D=D, bits=bits, window=window, sinks=sinks, seed=n)
    good = c.chunk(handle)
    clean = [m.copy() for m in c.meta]
    for j in (n - 1, n - T + 7, n - T, 2, max(0, n - T - 60)):
        sees = np.array([j <= p and (not window or j > p - window or j < sinks) for p in range(n - T, n)])
        if not sees.any():
            continue
        s = torch.from_numpy(np.concatenate([sees, np.zeros(10, bool)])).cuda()
        page, tile, at = c.where(0, j)
        for which, bad in ((3, np.nan), (2, np.nan), (3, np.inf), (1, np.nan), (0, np.nan)):
            c.meta = [m.copy() for m in clean]
            c.meta[which][page, :, tile, at, 1] = bad
            c.repack()
            out, lse = c.chunk(handle)
            assert torch.equal(out[~s], good[0][~s]) and torch.equal(lse[~s], good[1][~s])
            if which >= 2:
                assert torch.equal(lse, good[1])
                hit, rest = out[s][..., 32:64], torch.cat([out[s][..., :32], out[s][..., 64:]], -1)
                assert bool((~hit.isfinite()).all())
                assert torch.equal(rest, torch.cat([good[0][s][..., :32], good[0][s][..., 64:]], -1))
            else:
                assert bool(out[s].isnan().all()) and bool(lse[s].isnan().all())
    handle.sync()


@pytest.mark.parametrize("bits,D", SHAPES)
def test_a_value_that_is_no_number_among_many_blocks(lqm, handle, bits, D):  # noqa: F811
    """As many units as there are pairs of CTAs, each of many key blocks: what a block's values are is looked at while
    later blocks' are under way."""
    n, T = 2048, 1024
    c = Rows(lqm, [T], [n], hq=20, hkv=20, D=D, bits=bits, seed=3, poison=False)
    good = c.chunk(handle)
    clean = [m.copy() for m in c.meta]
    for k in range(8):
        c.meta = [m.copy() for m in clean]
        page, tile, at = c.where(0, 128 * k + 127)          # the last key of block k, which all rows see
        c.meta[3][page, :, tile, at, 1] = np.nan
        c.repack()
        out, lse = c.chunk(handle)
        assert torch.equal(lse, good[1])
        assert bool(out[..., 32:64].isnan().all()), int((~out[..., 32:64].isnan()).sum())
        assert torch.equal(out[..., :32], good[0][..., :32]) and torch.equal(out[..., 64:], good[0][..., 64:])
    handle.sync()


def test_captured_calls_follow_lengths_and_rows(lqm, handle):  # noqa: F811
    c = Rows(lqm, [60, 40], [900, 300], seed=5, poison=False)
    want = c.chunk(handle)
    out, lse = torch.zeros_like(c.q), torch.zeros(c.q.shape[:2], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.chunk(handle, out=out, lse=lse)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    c.fresh, c.lens, c.starts = [5, 70], [17, 290], np.array([0, 5, 75], np.int32)
    c.dev["lens"].copy_(torch.tensor(c.lens))
    c.dev["starts"].copy_(torch.from_numpy(c.starts))
    out.fill_(9.0)
    g.replay()
    torch.cuda.synchronize()
    c.check(out, lse)
    assert bool((out[75:] == 9).all())


def test_another_stream(lqm, handle):  # noqa: F811
    c = Rows(lqm, [60, 40], [900, 300], seed=5)
    want = c.chunk(handle)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.chunk(handle, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_small_workspace_is_refused(lqm):  # noqa: F811
    with lqm.Handle(0, 2 << 20) as h:
        c = Rows(lqm, [3], [9], seed=1)
        with pytest.raises(lqm.LQError) as e:
            c.chunk(h)
        assert e.value.status == lqm.LQ_ERR_WORKSPACE


def test_no_rows(lqm, handle):  # noqa: F811
    c = Rows(lqm, [0, 0], [5, 7], seed=1)
    out, lse = c.chunk(handle)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    handle.sync()
