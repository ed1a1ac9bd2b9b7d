"""The scoring example: projections, cache, chunk and window attention and log probabilities as one program.

Its logits are checked against a 64-bit evaluation over the values that the cache holds and the weights that lq_dequant gives.
Every rounding on the way, relative to the magnitudes that meet in it (E: the product of absolute values):
* o is within the attention's bound, 2^-10 of sum p |v| and 2^-8 of itself for bfloat16 (d_o);
* y = x + o Wo': the product within 4e-3 E for bfloat16 operands, its output and the sum rounded to bfloat16, 2^-8 each;
* logits: what that moves through |H|, and 4e-3 E again.
"""
import os
import sys

import numpy as np
import pytest

from tests import _rows_ref as RR

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import bit_weight_quantized_dequant_gb300 as lq
    lq.build()
    import score_prompt
    return score_prompt


@pytest.mark.parametrize("window,sinks", [(None, 0), (50, 3)])
@pytest.mark.parametrize("before,n", [(0, 200), (333, 64), (130, 1)])
def test_logits_and_log_probabilities(example, window, sinks, before, n):
    import bit_weight_quantized_dequant_gb300 as lq
    with lq.Handle(0) as h:
        s = example.Scorer(h, vocab=1024, window=window, sinks=sinks)
        tokens = torch.randint(0, 1024, (before + n,), generator=torch.Generator().manual_seed(n)).cuda()
        if before:
            s.logits(tokens[:before])
        part = tokens[before:]
        logits = s.logits(part)
        x = s.embedding[part]
        at = torch.arange(before + n, device="cuda")
        slots = s.block_table[0][at // 64].long() * 64 + at % 64
        k, v = (t.cpu().numpy() for t in h.kv_read(s.cache, slots, dtype=torch.float32))
        q = h.rope(s.project(s.wq, x).view(n, 8, 128), at[before:].int(), s.table).float().cpu().numpy()
        seen = RR.visible(before + n, n, window or 0, sinks)
        o, mass = np.zeros((n, 8, 128)), np.zeros((n, 8, 128))
        for head in range(2):
            hs = slice(4 * head, 4 * head + 4)
            o[:, hs], _, mass[:, hs], _ = RR.attend(q[:, hs], k[:, head], v[:, head], seen, 128 ** -0.5)
        o, mass = o.reshape(n, -1), mass.reshape(n, -1)
        wo, hd = (h.dequant(w, out_dtype=torch.float32).cpu().numpy().astype(np.float64) for w in (s.wo, s.head))
        x = x.float().cpu().numpy().astype(np.float64)
        d_o = 2.0 ** -10 * 2 * mass + 2.0 ** -8 * np.abs(o)
        y = x + o @ wo.T
        d_y = d_o @ np.abs(wo).T + (4e-3 + 2.0 ** -8) * ((np.abs(o) + d_o) @ np.abs(wo).T) + 2.0 ** -8 * np.abs(y)
        want = y @ hd.T
        bound = d_y @ np.abs(hd).T + 4e-3 * ((np.abs(y) + d_y) @ np.abs(hd).T)
        got = logits.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= bound)
        t = torch.randint(0, 1024, (n,), generator=torch.Generator().manual_seed(1)).cuda()
        logprob = h.token_logprobs(logits, t)[0].double().cpu()
        exact = torch.log_softmax(logits.double().cpu(), -1)[torch.arange(n), t.cpu()]
        assert torch.all((logprob - exact).abs() <= 2.0 ** -17 * (1 + exact.abs()))
        h.sync()


def test_example_runs(example, capsys):
    logprob, tokens = example.main(length=300, chunk=100, steps=3)
    assert logprob.shape == (299,) and bool(logprob.isfinite().all()) and tokens.shape == (3,)
    assert "300 tokens in chunks of 100" in capsys.readouterr().out
