"""The decode-step example: projections, rotation, cache and attention as one program, against a 64-bit evaluation
over the values that the cache holds.

The output projection is a decode GEMV of the attention's bfloat16 output: |y - y_ref| <= 1e-3 * E for the output it
was given.  That output is within the attention's bound of the 64-bit attention (2^-11 of the values' magnitude mass
plus bfloat16's 2^-8 of the output; the mass is at most 4 here per unit of value): both go through |Wo|.
"""
import os
import sys

import numpy as np
import pytest

from tests import _kv_ref as R

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
    import decode_step
    return decode_step


def test_steps_against_the_cache_in_64_bits(example):
    import bit_weight_quantized_dequant_gb300 as lq
    batch, hidden, hq, hkv, D, prefix = 3, 512, 8, 2, 128, 130
    g = torch.Generator(device="cuda").manual_seed(2)
    with lq.Handle(0) as h:
        b = example.AttentionBlock(h, hidden, hq, hkv, D, batch, pages_each=2, prefix_pages=3)
        b.write_prefix(*(torch.randn(prefix, hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2)))
        for step in range(70):                       # past a page's end
            x = torch.randn(batch, hidden, generator=g, device="cuda").bfloat16()
            y = b.step(x)
        assert b.lens.tolist() == [70] * batch
        # the last step again, from what the cache holds now
        q = h.gemv(b.wq, x, y_dtype=torch.bfloat16).view(batch, hq, D)
        q = h.rope(q, torch.full((batch,), 69 + prefix, dtype=torch.int32, device="cuda"), b.table)
        at = torch.arange(prefix, device="cuda")
        shared = h.kv_read(b.cache, b.prefix_table[at // 64].long() * 64 + at % 64, dtype=torch.float32)
        wo = h.dequant(b.wo, out_dtype=torch.float32).cpu().numpy().astype(np.float64)
        for r in range(batch):
            at = torch.arange(70, device="cuda")
            own = h.kv_read(b.cache, b.block_table[r][at // 64].long() * 64 + at % 64, dtype=torch.float32)
            k, v = (torch.cat([s, o]).cpu().numpy() for s, o in zip(shared, own))
            ref, mass = [], []
            for head in range(hkv):
                qs = q[r, head * 4:head * 4 + 4][None].float().cpu().numpy()
                o, _, m, _ = R.attend(qs, k[:, head], v[:, head], [prefix + 70], D ** -0.5)
                ref.append(o[0]), mass.append(m[0])
            ref, mass = np.concatenate(ref).reshape(-1), np.concatenate(mass).reshape(-1)
            off = 2.0 ** -11 * 5 * mass + 2.0 ** -8 * np.abs(ref)      # of the attention's output
            want = wo @ ref
            bound = np.abs(wo) @ off + 1e-3 * (np.abs(wo) @ (np.abs(ref) + off)) + 2.0 ** -8 * np.abs(want)
            assert np.all(np.abs(y[r].float().cpu().numpy() - want) <= bound * 1.01)
        h.sync()


def test_example_runs(example, capsys):
    y = example.main(steps=3)
    assert y.shape == (4, 1024) and bool(y.isfinite().all())
    assert "3 of their own" in capsys.readouterr().out
