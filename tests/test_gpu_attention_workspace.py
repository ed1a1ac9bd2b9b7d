"""lq_kv_attention takes what its workspace has room for: another kernel for the shared prefix, or the requests in turns.
Only where a single request does not fit it answers LQ_ERR_WORKSPACE, and then it has written nothing."""
import numpy as np
import pytest

from tests.test_gpu_kv_attention import Case, handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _lens(B, top, seed=1):
    return [int(x) for x in np.random.default_rng(seed).integers(0, top, B)]


def test_many_rows_over_a_short_prefix_on_the_default_workspace(lqm, handle):  # noqa: F811
    """1024 requests of 8 tokens, 64 query heads over 8: 65536 rows of a kv head, whose prefix sums alone are 270 MB."""
    c = Case(lqm, _lens(1024, 17), T=8, hq=64, hkv=8, prefix=256, page=16, seed=3)
    c.check(*c.run(handle), requests=[0, 1, 77, 511, 512, 513, 900, 1023])
    handle.sync()


@pytest.mark.parametrize("megabytes", [16, 12, 8])
@pytest.mark.parametrize("B,T,hq,hkv,prefix", [(20, 1, 8, 8, 1000), (5, 4, 8, 8, 1000), (64, 8, 64, 8, 700), (64, 8, 64, 8, 200),
                                               (1024, 1, 4, 4, 390), (300, 2, 40, 40, 0)])
def test_small_workspaces(lqm, handle, megabytes, B, T, hq, hkv, prefix):  # noqa: F811
    """20 rows over 1000 tokens: the dense kernel's slots are 20 MB, the other's records 80 KB.  64 x 8 x 64 heads: the
    records are 17 MB, so the requests come in turns."""
    c = Case(lqm, _lens(B, 33), T=T, hq=hq, hkv=hkv, prefix=prefix, page=16, seed=B)
    h = lqm.Handle(0, workspace_bytes=megabytes << 20)
    try:
        out, lse = c.run(h)
        c.check(out, lse, requests=sorted({0, 1, B // 4, B // 2 - 1, B // 2, B // 2 + 1, B - 1}))
        h.sync()
        # in turns or at once: the same within the sums' rounding
        ref, _ = c.run(handle)
        assert (out.float() - ref.float()).abs().max() <= 2.0 ** -7 * ref.float().abs().max()
    finally:
        h.close()


def test_without_room_for_one_request_nothing_is_written(lqm):  # noqa: F811
    c = Case(lqm, [300], T=4, hq=32, hkv=4, prefix=500, seed=2)
    h = lqm.Handle(0, workspace_bytes=1 << 16)
    out, lse = torch.full_like(c.q, 7.0), torch.full(c.q.shape[:3], 7.0, device="cuda")
    with pytest.raises(lqm.LQError) as e:
        c.run(h, out=out, lse=lse)
    assert e.value.status == lqm.LQ_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and bool((lse == 7).all())
    h.close()


def test_more_tiles_than_an_index_counts(lqm, handle):  # noqa: F811
    """1024 requests of 64 tokens, 64 query heads over 8, page lists that reach 128 Ki tokens: every limit of the header is
    kept, and the tiles that the lists could hold, counted for every 16 rows, pass 2^31.  In turns."""
    c = Case(lqm, _lens(1024, 81), T=64, hq=64, hkv=8, D=64, page=80, seed=5)
    c.bt = np.ascontiguousarray(np.repeat(c.bt, 1639, 1))        # (tokens past a length are never looked up)
    assert (1639 * 80 // 16) * 1024 * 8 * 32 > 2 ** 31
    c.check(*c.run(handle), requests=[0, 255, 511, 512, 1023])
    handle.sync()
