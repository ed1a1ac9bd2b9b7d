"""Rows without alternatives that many blocks share: one lane of the last block learns that all parts are there, and all of its warp's
lanes read them.  Each call's parts are another row's than the last call's, so that a part read too early is a wrong answer."""
import pytest

from tests.test_gpu_kv_attention import handle, lqm  # noqa: F401
from tests.test_gpu_logprobs import check, rows

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,V", [(1, 200003), (4, 131072), (20, 40000)])
def test_parts_of_other_rows(lqm, handle, n, V):  # noqa: F811
    x, t = rows(n, V, "bf16", seed=1)
    y, u = rows(n, V, "bf16", seed=2, sigma=1.0)
    first, second = handle.token_logprobs(x, t), handle.token_logprobs(y, u)
    check(x, t, first, 0)
    check(y, u, second, 0)
    got = []
    for _ in range(200):
        got += [handle.token_logprobs(x, t)[:2], handle.token_logprobs(y, u)[:2]]
    for k, (logprob, entropy) in enumerate(got):
        want = second if k % 2 else first
        assert torch.equal(logprob, want[0]) and torch.equal(entropy, want[1]), k
    handle.sync()
