"""lq_sync reports each condition that a kernel raised, one a call, the gravest first, and loses none."""
import numpy as np
import pytest

from tests._util import quantized_2bit, x_for
from tests.test_gpu_kv_attention import handle, lqm  # noqa: F401
from tests.test_gpu_operand_domain import with_big_group

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _index(lqm, h):  # noqa: F811
    table = h.rope_table(8, 32)
    h.rope(torch.zeros(1, 1, 32, device="cuda"), torch.tensor([99], dtype=torch.int32, device="cuda"), table)


def _range(lqm, h):  # noqa: F811
    p, outl = quantized_2bit(96, 256, seed=5)
    anchors = set(p["anchor_idx"].tolist())
    g = next(i for i in range(8) if not anchors & set(range(32 * i, 32 * i + 32)))
    w = lqm.QuantWeights.from_host(with_big_group(p, 17, g, 50000.0), lqm.FMT_2BIT)
    h.gemv(w, torch.from_numpy(x_for(1, 256, "f16", outl, seed=5)).view(torch.float16).cuda())


def _timeout(lqm, h):  # noqa: F811
    h.selftest_wait(20_000)


def _reported(lqm, h):  # noqa: F811
    out = []
    for _ in range(4):
        try:
            h.sync()
            return out
        except lqm.LQError as e:
            out.append(e.status)
    return out


@pytest.mark.parametrize("order", [("index", "timeout"), ("timeout", "index"), ("range", "index"), ("index", "range"),
                                   ("index", "range", "timeout"), ("index", "index"), ("timeout", "range")])
def test_every_condition_is_reported_once(lqm, handle, order):  # noqa: F811
    raise_ = {"index": _index, "range": _range, "timeout": _timeout}
    handle.sync()
    for what in order:
        raise_[what](lqm, handle)
    status = {"timeout": lqm.LQ_ERR_TIMEOUT, "range": lqm.LQ_ERR_RANGE, "index": lqm.LQ_ERR_INDEX}
    assert _reported(lqm, handle) == [status[w] for w in ("timeout", "range", "index") if w in order]
    # and the handle is as new
    q = torch.randn(3, 2, 32, device="cuda")
    table = handle.rope_table(8, 32)
    got = handle.rope(q, torch.arange(3, dtype=torch.int32, device="cuda"), table)
    assert torch.equal(got[0], q[0]) and np.isfinite(got.cpu().numpy()).all()
    handle.sync()
