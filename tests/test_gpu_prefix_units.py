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


@pytest.mark.parametrize("B,T,hq,hkv,D,bits,prefix", [
    (1024, 1, 4, 4, 128, 4, 390),              # two key blocks a share
    (300, 1, 12, 12, 64, 8, 520),              # five
    (130, 1, 8, 2, 128, 8, 2000),
    (40, 2, 40, 40, 128, 4, 700),
])
def test_first_calls_with_nothing_in_the_caches(lqm, B, T, hq, hkv, D, bits, prefix):  # noqa: F811
    """Values that come late, in a workspace that nothing has written: the sums are read when they are done, so a first
    call answers what later ones do, bit for bit, and right in every unit."""
    g = np.random.default_rng(B)
    c = Case(lqm, [int(x) for x in g.integers(0, 33, B)], T=T, hq=hq, hkv=hkv, D=D, bits=bits, prefix=prefix, page=16, seed=B)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(12):
        h = lqm.Handle(0)
        flush.fill_(i)
        out, lse = c.run(h)
        h.sync()
        if first is None:
            first = out, lse
            rows = T * (hq // hkv)
            tiles = -(-B * rows // 128)
            c.check(out, lse, requests=sorted({min(B - 1, (128 * t + 64) // rows) for t in range(tiles)}))
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        h.close()
