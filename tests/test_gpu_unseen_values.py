"""What lies in slots that no row sees, finite extremes among it: large scales of either sign under the largest code, offsets at the
ends of binary16's range, NaN and infinities, in turn within one tile.  Answers are those of a cache without them
(bounds: tests/_rows_ref.py)."""
import numpy as np
import pytest

from tests._rows_ref import Rows, visible
from tests.test_gpu_kv_attention import SHAPES, handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
# S and Z of a slot, for keys and values alike
FINITE = [(-60000.0, -65504.0), (60000.0, 65504.0), (-65504.0, 65504.0), (65504.0, -65504.0), (-5000.0, 0.0), (1.0, -65504.0)]
OTHERS = [(np.nan, 1.0), (1.0, np.nan), (np.inf, -1.0), (-np.inf, 0.0), (0.0, np.inf)]


def spoil(c, kinds, seed=0):
    """Every slot that no row of any request sees gets one of the kinds, codes at their largest."""
    shape = c.codes[0].shape[:4]                       # pages, heads, tiles, tokens
    used = np.zeros((shape[0], c.page), bool)
    for b in range(len(c.lens)):
        j = np.nonzero(visible(c.length(b), c.fresh[b], c.window, c.sinks).any(0))[0]
        used[c.bt[b][j // c.page], j % c.page] = True
    free = np.broadcast_to(~used.reshape(shape[0], 1, *shape[2:]), shape)
    which = np.random.default_rng(seed).integers(0, len(kinds), shape)
    table = np.array(kinds, np.float32).astype(np.float16)
    for i, m in enumerate(c.meta):
        m[free] = table[which[free], i % 2][:, None]
    for codes in c.codes:
        codes[free] = 2 ** c.bits - 1
    c.repack()


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("window,sinks", [(70, 3), (133, 0), (5, 20), (1, 0), (0, 0)])
@pytest.mark.parametrize("kinds", [FINITE, FINITE[:1], FINITE + OTHERS], ids=["finite", "one kind", "all"])
def test_chunks(lqm, handle, bits, D, dtype, window, sinks, kinds):  # noqa: F811
    c = Rows(lqm, [40, 1, 7, 300], [703, 301, 90, 1500], hq=4, hkv=2, D=D, bits=bits, dtype=dtype, window=window, sinks=sinks, seed=1,
             poison=False)
    want = c.chunk(handle)
    spoil(c, kinds)
    got = c.chunk(handle)
    c.check(*got)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    handle.sync()


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("window,sinks", [(70, 3), (5, 20), (1, 0), (0, 0)])
@pytest.mark.parametrize("T", [1, 7])
def test_decode_steps(lqm, handle, bits, D, dtype, window, sinks, T):  # noqa: F811
    c = Rows(lqm, [T] * 4, [703, 301, 90, 1500], hq=4, hkv=2, D=D, bits=bits, dtype=dtype, window=window, sinks=sinks, seed=2,
             poison=False)
    for kinds in (FINITE, FINITE + OTHERS):
        spoil(c, kinds)
        c.check(*c.decode(handle), dense=False)
    handle.sync()
