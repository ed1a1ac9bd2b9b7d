"""The low-bit KV cache on the GPU: lq_kv_append's stored bytes and lq_kv_read's values are the definition's bits
(every fp32 step is correctly rounded, so there is one right answer), with and without the rotation of k and q."""
import numpy as np
import pytest

from tests import _kv_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TDT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def lqm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_weight_quantized_dequant_gb300 as lq
    lq.build()
    return lq


@pytest.fixture(scope="module")
def handle(lqm):
    h = lqm.Handle(0)
    yield h
    h.close()


def _expected(pages, page, bits, D, k, v, slots):
    """The pages after the definition's append of k, v (fp32 [n][hkv][D], already of the input type)."""
    pages = pages.copy()
    hkv = k.shape[1]
    for i, s in enumerate(slots):
        if s < 0:
            continue
        p, off = divmod(int(s), page)
        for h in range(hkv):
            tile = pages[p, h, off // 16]
            _, _, kk, vv = R.unpack(tile, bits, D)
            for old, new in ((kk, R.quantize(k[i, h], bits)), (vv, R.quantize(v[i, h], bits))):
                for a, b in zip(old, new):
                    a[off % 16] = b
            pages[p, h, off // 16] = R.pack(*kk, *vv, bits)
    return pages


def _values(n, hkv, D, dtype, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, hkv, D)).astype(np.float32)
    x[:, :, ::19] *= 9.0
    x[0, 0, :32] = 0.5                                   # a flat group
    if n > 2:
        x[1, 0, :32] = 0.0
        x[2, -1, 32:64] *= 1e-6                          # a group whose scale is subnormal or zero
    return torch.from_numpy(x).to(TDT[dtype]).cuda()


@pytest.mark.parametrize("bits,D", [(4, 64), (4, 128), (8, 64), (8, 128)])
@pytest.mark.parametrize("n,hkv,page,dtype", [(1, 1, 16, "bf16"), (45, 3, 48, "f16"), (70, 8, 32, "bf16"), (33, 2, 128, "f32")])
def test_append_and_read_are_bit_exact(lqm, handle, bits, D, n, hkv, page, dtype):
    k, v = _values(n, hkv, D, dtype, n), _values(n, hkv, D, dtype, n + 1)
    pages_n = -(-n // page) + 2
    start = np.random.default_rng(3).integers(0, 256, (pages_n, hkv, page // 16, lqm.load_library().lq_kv_tile_bytes(bits, D)),
                                              dtype=np.uint8)
    cache = lqm.KVCache(torch.from_numpy(start).cuda(), page_size=page, kv_heads=hkv, head_dim=D, bits=bits)
    slots = torch.randperm(pages_n * page, generator=torch.Generator().manual_seed(n))[:n]
    if n > 5:
        slots[4] = -1
    assert handle.kv_append(cache, k, v, slots.cuda()) is None
    want = _expected(start, page, bits, D, k.float().cpu().numpy(), v.float().cpu().numpy(), slots.numpy())
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    handle.sync()
    for odt in ("f32", "f16", "bf16"):
        ko, vo = handle.kv_read(cache, slots.cuda(), dtype=TDT[odt])
        for got, src in ((ko, k), (vo, v)):
            ref = R.dequantize(*R.quantize(src.float().cpu().numpy(), bits))
            ref[slots.numpy() < 0] = 0.0
            assert torch.equal(got.cpu(), torch.from_numpy(ref).to(TDT[odt]))


@pytest.mark.parametrize("bits,D,rot", [(4, 128, 128), (8, 128, 64), (4, 64, 32), (8, 64, 64), (4, 64, 16), (8, 128, 96)])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_fused_rotation_equals_rotation_then_append(lqm, handle, bits, D, rot, layout, dtype):
    n, hq, hkv, page = 41, 6, 2, 32
    g = torch.Generator().manual_seed(rot)
    row = torch.randn(n, hq + 2 * hkv, D, generator=g).to(TDT[dtype]).cuda()
    q, k, v = row.split([hq, hkv, hkv], 1)
    table = handle.rope_table(300, rot)
    pos = torch.randint(0, 300, (n,), generator=g, dtype=torch.int32).cuda()
    slots = torch.randperm(96, generator=g)[:n].cuda()
    a, b = (lqm.KVCache(num_pages=3, page_size=page, kv_heads=hkv, head_dim=D, bits=bits) for _ in range(2))
    qo = handle.kv_append(a, k, v, slots, q=q, table=table, positions=pos, layout=layout)
    assert torch.equal(qo, handle.rope(q, pos, table, layout=layout))
    handle.kv_append(b, handle.rope(k, pos, table, layout=layout), v, slots)
    assert torch.equal(a.pages, b.pages) and bool(a.pages.any())
    # in place, and q alone copied without a table
    q2 = q.contiguous()
    handle.kv_append(b, k, v, slots, q=q2, table=table, positions=pos, layout=layout, q_out=q2)
    assert torch.equal(q2, qo) and torch.equal(a.pages, b.pages)
    assert torch.equal(handle.kv_append(b, k, v, slots, q=q), q)
    handle.sync()


@pytest.mark.parametrize("bits", [4, 8])
def test_nan_and_infinity(lqm, handle, bits):
    k, v = _values(20, 2, 64, "bf16", 1), _values(20, 2, 64, "bf16", 2)
    k[3, 1, 5], k[4, 0, 40], v[5, 1, 63], v[6, 0, 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    k[7, 0, 9] = 1e38
    cache = lqm.KVCache(num_pages=1, page_size=32, kv_heads=2, head_dim=64, bits=bits)
    slots = torch.arange(20, device="cuda")
    handle.kv_append(cache, k, v, slots)
    ko, vo = handle.kv_read(cache, slots, dtype=torch.float32)
    for got, src in ((ko, k), (vo, v)):
        ref = R.dequantize(*R.quantize(src.float().cpu().numpy(), bits))
        assert np.array_equal(got.cpu().numpy(), ref, equal_nan=True)
    assert bool(ko[3, 1, :32].isnan().all()) and bool(ko[3, 1, 32:].isfinite().all()) and bool(ko[4].isfinite().all())


def test_slots_past_the_cache(lqm, handle):
    k, v = _values(4, 1, 64, "f16", 1), _values(4, 1, 64, "f16", 2)
    cache = lqm.KVCache(num_pages=2, page_size=16, kv_heads=1, head_dim=64, bits=4)
    handle.kv_append(cache, k, v, torch.tensor([0, 32, 2 ** 62, 31], device="cuda"))
    with pytest.raises(lqm.LQError) as e:
        handle.sync()
    assert e.value.status == lqm.LQ_ERR_INDEX
    ko, _ = handle.kv_read(cache, torch.tensor([0, 32, -5, 31], device="cuda"))
    with pytest.raises(lqm.LQError):
        handle.sync()
    assert bool(ko[0].any()) and bool(ko[3].any()) and not bool(ko[1:3].any())
    handle.sync()


def test_offsets_past_32_bits(lqm, handle):
    """A cache of 4.6 GB: the last page's tokens land in the last page."""
    tile = lqm.load_library().lq_kv_tile_bytes(8, 128)
    pages = 2 ** 32 // (tile * 4) + 20000
    cache = lqm.KVCache(num_pages=pages, page_size=64, kv_heads=1, head_dim=128, bits=8)
    k, v = _values(3, 1, 128, "bf16", 5), _values(3, 1, 128, "bf16", 6)
    slots = torch.tensor([pages * 64 - 1, pages * 64 - 33, 7], device="cuda")
    handle.kv_append(cache, k, v, slots)
    ko, vo = handle.kv_read(cache, slots, dtype=torch.float32)
    assert np.array_equal(ko.cpu().numpy(), R.dequantize(*R.quantize(k.float().cpu().numpy(), 8)))
    assert np.array_equal(vo.cpu().numpy(), R.dequantize(*R.quantize(v.float().cpu().numpy(), 8)))
    assert bool(cache.pages[-1].any()) and bool(cache.pages[0].any())
    handle.sync()


def test_empty_and_refusals(lqm, handle):
    cache = lqm.KVCache(num_pages=2, page_size=16, kv_heads=2, head_dim=64, bits=4)
    k = torch.zeros(3, 2, 64, device="cuda", dtype=torch.float16)
    slots = torch.arange(3, device="cuda")
    handle.kv_append(cache, k[:0], k[:0], slots[:0])
    assert handle.kv_read(cache, slots[:0])[0].shape == (0, 2, 64)
    for bad in (lambda: handle.kv_append(cache, k, k.float(), slots), lambda: handle.kv_append(cache, k, k, slots.int()),
                lambda: handle.kv_append(cache, k, k[:2], slots), lambda: handle.kv_append(cache, k[..., :32], k, slots),
                lambda: handle.kv_append(cache, k, k, slots, q=k[:2]), lambda: handle.kv_append(cache, k.cpu(), k, slots),
                lambda: handle.kv_read(cache, slots.cpu()), lambda: lqm.KVCache(num_pages=1, page_size=24, kv_heads=1, head_dim=64, bits=4),
                lambda: lqm.KVCache(num_pages=1, page_size=16, kv_heads=1, head_dim=96, bits=4),
                lambda: lqm.KVCache(torch.zeros(2, 2, 1, 5, dtype=torch.uint8), page_size=16, kv_heads=2, head_dim=64, bits=4)):
        with pytest.raises(ValueError):
            bad()
    shifted = torch.zeros(3 * 128 + 4, device="cuda", dtype=torch.float16)[4:].view(3, 2, 64)
    with pytest.raises(lqm.LQError) as e:
        handle.kv_append(cache, shifted, k, slots)
    assert e.value.status == lqm.LQ_ERR_ALIGNMENT
