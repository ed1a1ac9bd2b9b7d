"""Rotary positions on the GPU against their definition.

* lq_rope_table: within 4e-7 of the 64-bit cos and sin at every position tried (the angle's fixed-point error is
  1.5e-9 rad, its fp32 rounding at most pi * 2^-25 = 9.4e-8, and sincospi's error 1 to 2 ulp of 1, 2^-24 each), up to
  positions near 2^31;
* lq_rope: bit for bit the definition's fp32 roundings, every layout, type, part of the head, stride and alignment; the
  inverse is the transpose (checked as an adjoint and against differences).
"""
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


@pytest.mark.parametrize("rot", [2, 6, 32, 64, 128, 200, 256])
@pytest.mark.parametrize("first,count", [(0, 1), (0, 777), (131000, 300), (2 ** 31 - 1000, 999)])
def test_table(handle, rot, first, count):
    for kw in (dict(), dict(factor=4.0), dict(factor=16.0, original=8192.0), dict(factor=8.0, original=4096.0, low=0.5, high=4.0, base=5e5)):
        got = handle.rope_table(count, rot, base=kw.get("base", 10000.0), first=first, factor=kw.get("factor", 1.0),
                                original_length=kw.get("original", 0.0), low_rotations=kw.get("low", 1.0),
                                high_rotations=kw.get("high", 32.0), mscale=1.25)
        # positions near 2^31 times a frequency rounded in its last (53rd) bit: 2^31 * 2^-53 = 2.4e-7 rad
        ref = R.table64(first, count, rot, mscale=1.25, **kw)
        tol = 1.25 * (4e-7 + 4 * 2.0 ** -53 * (first + count))
        assert got.shape == (count, rot) and np.abs(got.cpu().numpy() - ref).max() <= tol


def _case(n, heads, D, rot, dtype, seed, pad=0, head_pad=0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(n, heads * (D + head_pad) + pad, generator=g).to(TDT[dtype]).cuda()
    x = wide[:, pad:].unflatten(1, (heads, D + head_pad))[..., :D]
    table = torch.from_numpy(R.table64(0, 500, rot).astype(np.float32)).cuda()
    pos = torch.randint(0, 500, (n,), generator=g, dtype=torch.int32).cuda()
    return x, table, pos


def _same(got, x, table, pos, layout, inverse, dtype):
    ref = R.rotate(x.float().cpu().numpy(), table.cpu().numpy(), pos.cpu().numpy(), layout, inverse)
    assert torch.equal(got.cpu(), torch.from_numpy(ref).to(TDT[dtype])), "not the definition's bits"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("n,heads,D,rot,pad,head_pad", [
    (1, 1, 64, 64, 0, 0), (1, 40, 128, 128, 0, 0), (37, 5, 128, 64, 0, 0), (3, 33, 256, 256, 0, 0), (200, 8, 96, 96, 16, 0),
    (5, 3, 80, 32, 0, 8),                                                    # rows of 10 vectors, heads apart
    (7, 3, 64, 64, 3, 0), (4, 2, 64, 48, 0, 1), (5, 2, 10, 6, 0, 0), (2, 1, 2, 2, 1, 0), (3, 2, 66, 20, 0, 0), (2, 3, 320, 64, 0, 0),
])
def test_rotation_is_the_definition_bit_for_bit(handle, dtype, layout, inverse, n, heads, D, rot, pad, head_pad):
    x, table, pos = _case(n, heads, D, rot, dtype, n + D, pad, head_pad)
    _same(handle.rope(x, pos, table, layout=layout, inverse=inverse), x, table, pos, layout, inverse, dtype)


def test_out_strides_and_in_place(handle):
    x, table, pos = _case(19, 6, 128, 128, "bf16", 4)
    wide = torch.full((19, 6, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    handle.rope(x, pos, table, out=wide[..., :128])
    _same(wide[..., :128], x, table, pos, 0, False, "bf16")
    assert bool((wide[..., 128:] == 7).all())
    y = x.clone()
    handle.rope(y, pos, table, layout=1, out=y)
    _same(y, x, table, pos, 1, False, "bf16")
    odd = torch.randn(19, 6, 131, device="cuda")[..., 2:130]       # the narrow path, in place
    keep = odd.clone()
    handle.rope(odd, pos, table, out=odd)
    _same(odd, keep, table, pos, 0, False, "f32")


@pytest.mark.parametrize("layout", [0, 1])
def test_inverse_is_the_gradient(handle, layout):
    """<rope(x), u> = <x, inverse(u)>, and the inverse equals central differences of <rope(x), u>, in fp32: each
    output carries 3 roundings of 2^-24, so a sum of N products is off by at most 4 * 2^-24 * sum |terms|."""
    x, table, pos = _case(3, 2, 32, 16, "f32", 9)
    u = torch.randn(x.shape, generator=torch.Generator().manual_seed(1)).cuda()
    fwd = lambda z: handle.rope(z, pos, table, layout=layout).double()  # noqa: E731
    grad = handle.rope(u, pos, table, layout=layout, inverse=True).double()
    lhs, rhs = (fwd(x) * u).sum(), (x * grad).sum()
    assert abs(lhs - rhs) <= 8 * 2.0 ** -24 * ((fwd(x) * u).abs().sum() + (x * grad).abs().sum())
    step = 0.5                                                       # (the map is linear: any step does)
    for i in range(0, x.numel(), 7):
        d = torch.zeros_like(x).view(-1)
        d[i] = step
        d = d.view(x.shape)
        diff = ((fwd(x + d) - fwd(x - d)) * u).sum() / (2 * step)
        scale = ((fwd(x + d).abs() + fwd(x - d).abs()) * u.abs()).sum() / (2 * step)
        assert abs(diff - grad.view(-1)[i]) <= 8 * 2.0 ** -24 * scale


def test_position_outside_the_table(lqm, handle):
    x, table, pos = _case(6, 2, 64, 64, "f16", 2)
    bad = pos.clone()
    bad[1], bad[4] = -1, 500
    for t in (x, x[..., :62]):
        got = handle.rope(t, bad, table[:, :60].contiguous() if t is not x else table)
        with pytest.raises(lqm.LQError) as e:
            handle.sync()
        assert e.value.status == lqm.LQ_ERR_INDEX
        assert torch.equal(got[1], t[1]) and torch.equal(got[4], t[4]) and not torch.equal(got[0], t[0])
    handle.sync()


def test_empty_and_refusals(handle):
    x, table, pos = _case(4, 2, 64, 64, "f16", 2)
    assert handle.rope(x[:0], pos[:0], table).shape == (0, 2, 64)
    with pytest.raises(ValueError):
        handle.rope(x, pos[:3], table)
    with pytest.raises(ValueError):
        handle.rope(x, pos.long(), table)
    with pytest.raises(ValueError):
        handle.rope(x.transpose(1, 2), pos, table)
    with pytest.raises(ValueError):
        handle.rope(x, pos, table.double())
    with pytest.raises(ValueError):
        handle.rope(x.to(torch.int16), pos, table)
    with pytest.raises(ValueError):
        handle.rope(x.cpu(), pos, table)


def test_other_stream(handle):
    x, table, pos = _case(2000, 32, 128, 128, "bf16", 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = handle.rope(x, pos, table, stream=s)
    s.synchronize()
    _same(got, x, table, pos, 0, False, "bf16")
