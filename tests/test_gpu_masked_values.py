"""lq_kv_attention: what a row does not see leaves it alone, whatever is cached there."""
import numpy as np
import pytest

from tests.test_gpu_kv_attention import SHAPES, Case, handle, lqm  # noqa: F401
from tests.test_gpu_value_scales import Edit

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,hq,hkv,n", [(4, 4, 2, 61), (2, 8, 1, 17), (7, 4, 2, 300), (64, 2, 2, 64), (3, 24, 2, 130), (16, 2, 2, 16)])
def test_nan_of_a_later_token_stays_with_the_rows_that_see_it(lqm, handle, bits, D, dtype, T, hq, hkv, n):  # noqa: F811
    """Draft tokens whose keys or values are NaN or infinite: the tokens before them answer as if they were not there, and
    a NaN value reaches its own group of dimensions only."""
    c = Case(lqm, [n, n + 5], T=T, hq=hq, hkv=hkv, D=D, bits=bits, dtype=dtype, seed=n)
    good, good_lse = c.run(handle)
    first = T - T // 2                                    # query token from which on the rows see bad ones
    for what in ("value", "value z", "value inf", "value z inf", "key"):
        e = Edit(c)
        keep = c.cache.pages.clone()

        def spoil(ko, vo, t):
            if what.startswith("value"):
                vo[2 if "z" in what else 1][t, 1] = np.inf if "inf" in what else np.nan
                if what == "value":
                    vo[2][t, 1] = np.nan                  # (as a cached NaN has it)
            else:
                ko[1][t, 0] = np.nan
        for j in range(n - T + first, n):
            for h in range(hkv):
                e.token(0, j, h, spoil)
        e.done()
        out, lse = c.run(handle)
        assert torch.equal(out[0, :first], good[0, :first]) and torch.equal(lse[0, :first], good_lse[0, :first]), what
        assert torch.equal(out[1], good[1])
        if what == "key":
            assert bool(out[0, first:].isnan().all()) and bool(lse[0, first:].isnan().all())
        else:
            hit = out[0, first:, :, 32:64]
            assert bool((~hit.isfinite()).all()) if "inf" not in what else bool((~hit.isfinite()).any())
            rest = torch.cat([out[0, first:, :, :32], out[0, first:, :, 64:]], -1)
            want = torch.cat([good[0, first:, :, :32], good[0, first:, :, 64:]], -1)
            assert torch.equal(rest, want) and torch.equal(lse, good_lse)
        c.cache.pages.copy_(keep)
    handle.sync()
