"""What lq_logprobs leaves of lse's rounding: its pointer is optional and of fp32's alignment.  No GPU: refusals come before the
handle is read."""
from bit_weight_quantized_dequant_gb300 import _lq
from tests.test_long_prompt_refusals_cpu import A16, ALN, INV, L, grad, score  # noqa: F401


def test_the_rest_of_lse(L):  # noqa: F811
    assert score(L, lse_rest=A16 + 2) == ALN and grad(L, lse_rest=A16 + 1) == ALN
    assert score(L, n=0, lse_rest=None) == _lq.LQ_OK and score(L, n=0, lse_rest=A16 + 4) == _lq.LQ_OK
    assert grad(L, n=0, lse_rest=None) == _lq.LQ_OK and grad(L, n=0, lse_rest=A16 + 4) == _lq.LQ_OK
    assert grad(L, lse=None, lse_rest=A16) == INV
