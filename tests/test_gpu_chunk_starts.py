"""Divisions of a call's rows that are out of order or out of range: an entry counts as the nearer end, a request that ends before it
begins has no rows, either is reported, and rows of no request stay as they were."""
import numpy as np
import pytest

from tests._rows_ref import Rows
from tests.test_gpu_kv_attention import handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("starts,parts", [
    ([0, -3, 60, 100], [(0, 0), (0, 60), (60, 100)]),
    ([0, 40, 30, 30], [(0, 40), (40, 40), (30, 30)]),
    ([0, 40, 5000, 100], [(0, 40), (40, 100), (100, 100)]),
    ([50, 60, 70, 2 ** 31 - 1], [(50, 60), (60, 70), (70, 100)]),
    ([-2 ** 31, 0, 0, 0], [(0, 0), (0, 0), (0, 0)]),
    ([2 ** 31 - 1, 0, 10, 30], [(100, 100), (0, 10), (10, 30)])])
def test_moved_starts(lqm, handle, starts, parts):  # noqa: F811
    c = Rows(lqm, [40, 30, 30], [90, 80, 70], seed=13, poison=False)
    c.dev["starts"].copy_(torch.tensor(starts))
    out, lse = torch.full_like(c.q, 3.0), torch.full(c.q.shape[:2], 5.0, device="cuda")
    c.chunk(handle, out=out, lse=lse)
    if starts != [50, 60, 70, 100]:
        with pytest.raises(lqm.LQError) as e:
            handle.sync()
        assert e.value.status == lqm.LQ_ERR_INDEX
    nobodys = np.ones(100, bool)
    for b, (r0, r1) in enumerate(parts):
        nobodys[r0:r1] = False
        c.fresh[b], c.starts = r1 - r0, np.array([r0, r1] if b == 0 else list(c.starts[:b]) + [r0, r1])
        c.check(out, lse, requests=[b])
    n = torch.from_numpy(nobodys).cuda()
    assert bool((out[n] == 3).all()) and bool((lse[n] == 5).all())
