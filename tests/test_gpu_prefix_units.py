"""A shared prefix under many rows: more (kv head, 128 rows) units than the device has SMs, so that a block of the dense
kernel has several units and parts of units.  Requests are sampled so that every unit is checked, against 64 bits."""
import numpy as np
import pytest

from tests.test_gpu_kv_attention import Case, handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,hq,hkv,D,bits,prefix,dtype", [
    (400, 1, 40, 40, 128, 4, 400, "bf16"),     # 160 units
    (64, 8, 64, 8, 128, 4, 400, "f16"),        # 256
    (1000, 1, 32, 4, 64, 8, 385, "bf16"),      # 252
    (16, 64, 32, 32, 64, 4, 500, "bf16"),      # 256
    (1024, 2, 16, 16, 64, 8, 390, "f16"),      # 256, rows end a tile
    (700, 3, 24, 12, 64, 4, 386, "bf16"),      # 396: two units and a part in a block
])
def test_more_units_than_blocks(lqm, handle, B, T, hq, hkv, D, bits, prefix, dtype):  # noqa: F811
    g = np.random.default_rng(B)
    c = Case(lqm, [int(x) for x in g.integers(0, 17, B)], T=T, hq=hq, hkv=hkv, D=D, bits=bits, prefix=prefix, page=16, seed=B,
             dtype=dtype)
    rows = T * (hq // hkv)                     # of a request and kv head
    tiles = -(-B * rows // 128)
    assert tiles * hkv > torch.cuda.get_device_properties(0).multi_processor_count
    sample = sorted({min(B - 1, (128 * t + 64) // rows) for t in range(tiles)} | {0, B - 1})
    c.check(*c.run(handle), requests=sample)
    handle.sync()
