"""The cache's tile layout and quantizer definition (plain restatement), and the host-side refusals of the
rotary, cache and attention entry points.  No GPU."""
import ctypes
import itertools
import os
import re

import numpy as np
import pytest

import bit_weight_quantized_dequant_gb300 as lq
from bit_weight_quantized_dequant_gb300 import _lq
from tests import _kv_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPES = list(itertools.product((4, 8), (64, 128)))


@pytest.fixture(scope="module")
def L():
    lq.build()
    return _lq.load_library(build_if_missing=False)


@pytest.mark.parametrize("bits,D", SHAPES)
def test_layout_is_a_permutation(bits, D):
    """Every code has bits of its own and every S and Z bytes of its own; together they fill the tile."""
    G = D // 32
    pk, pv, ks, vs = R.places(bits, D)
    region = 16 * D * bits // 8
    for p, lo in ((pk, 0), (pv, region)):
        assert np.array_equal(np.sort(p.ravel()), 8 * lo + bits * np.arange(16 * D))
    meta = np.concatenate([(o + z).ravel() for o in (ks, vs) for z in (0, 32 * G)])
    assert np.array_equal(np.sort(meta), 2 * region + 2 * np.arange(4 * 16 * G))


@pytest.mark.parametrize("bits,D", SHAPES)
def test_pack_and_unpack_are_inverse(bits, D):
    g = np.random.default_rng(bits + D)
    c = [g.integers(0, 2 ** bits, (3, 16, D), dtype=np.uint8) for _ in range(2)]
    m = [g.standard_normal((3, 16, D // 32)).astype(np.float16) for _ in range(4)]
    tiles = R.pack(c[0], m[0], m[1], c[1], m[2], m[3], bits)
    k, v, (kc, ks, kz), (vc, vs, vz) = R.unpack(tiles, bits, D)
    assert np.array_equal(kc, c[0]) and np.array_equal(vc, c[1])
    for a, b in zip((ks, kz, vs, vz), m):
        assert np.array_equal(a, b)
    assert np.array_equal(k, R.dequantize(c[0], m[0], m[1])) and np.array_equal(v, R.dequantize(c[1], m[2], m[3]))


@pytest.mark.parametrize("bits", [4, 8])
def test_quantizer_error_and_edges(bits):
    """Half a step of error plus the rounding of S and Z; constant, zero, huge and NaN groups."""
    g = np.random.default_rng(7)
    x = (g.standard_normal((200, 64)) * np.exp(g.uniform(-3, 3, (200, 1)))).astype(np.float32)
    c, S, Z = R.quantize(x, bits)
    y = R.dequantize(c, S, Z)
    s = np.repeat(S.astype(np.float64), 32, -1)
    top = 2 ** bits - 1
    # half a step; the top code may fall short by top * (rounding of S), and Z moves by half an ulp
    bound = s * 0.5 + top * s * 2.0 ** -11 + np.abs(np.repeat(Z.astype(np.float64), 32, -1)) * 2.0 ** -11 + 1e-6
    assert np.all(np.abs(y.astype(np.float64) - x) <= bound)
    flat = np.full((1, 32), 0.75, np.float32)
    assert np.array_equal(R.dequantize(*R.quantize(flat, bits)), flat)
    big = np.zeros((1, 64), np.float32)
    big[0, :2], big[0, 40] = (np.inf, -1e30), np.nan
    c, S, Z = R.quantize(big, bits)
    assert np.isfinite(S[0, 0]) and Z[0, 0] == -65504 and np.isnan(S[0, 1]) and np.isnan(Z[0, 1]) and not c[0, 32:].any()


def test_header_tile_bytes(L):
    for bits, D in itertools.product((0, 2, 4, 8, 16), (0, 32, 64, 96, 128, 256)):
        want = 16 * (2 * D * bits // 8 + D // 32 * 8) if bits in (4, 8) and D in (64, 128) else 0
        assert L.lq_kv_tile_bytes(bits, D) == want


def test_struct_fields_follow_the_header():
    """The binding's structures name the header's fields in the header's order."""
    src = open(os.path.join(ROOT, "include", "lq.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    for st in (_lq.lq_rope_config, _lq.lq_rope_args, _lq.lq_kv_cache, _lq.lq_kv_append_args, _lq.lq_kv_attention_args):
        body = re.search(r"typedef struct %s \{(.*?)\}" % st.__name__, src, re.S).group(1)
        names = [re.search(r"(\w+)\s*$", n).group(1) for line in body.split(";") if line.strip() for n in line.split(",")]
        assert names == [f[0] for f in st._fields_], st.__name__


H = ctypes.c_void_p(0x1000)     # only with arguments that fail before the handle is read
A16 = 0x10000
INV, UNS, ALN = _lq.LQ_ERR_INVALID_ARG, _lq.LQ_ERR_UNSUPPORTED, _lq.LQ_ERR_ALIGNMENT


def _with(_base, **kw):
    a = type(_base).from_buffer_copy(_base)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_rope_table_refusals(L):
    ok = _lq.lq_rope_config(64, 10000.0, 1.0, 0.0, 1.0, 32.0, 1.0)
    call = lambda c, h=H, first=0, count=4, t=A16: L.lq_rope_table(h, ctypes.byref(c), first, count, t, None)  # noqa: E731
    assert call(ok, h=None) == INV and call(ok, t=None) == INV and call(ok, t=A16 + 4) == ALN
    assert call(ok, first=-1) == INV and call(ok, count=0) == INV and call(ok, first=2 ** 31 - 2) == INV
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(base=1.0), dict(base=float("nan")), dict(factor=0.0),
               dict(original_length=-1.0), dict(original_length=4096.0, high_rotations=1.0)):
        assert call(_with(ok, **kw)) == INV, kw
    assert call(_with(ok, rot_dim=258)) == UNS and call(_with(ok, factor=0.5)) == UNS


def test_rope_refusals(L):
    ok = _lq.lq_rope_args(A16, A16 + 0x1000, 2, 3, 4, 64, 64, 256, 64, 256, 64, A16, 100, A16, 0, 0)
    call = lambda a, h=H: L.lq_rope(h, ctypes.byref(a), None)  # noqa: E731
    assert call(ok, h=None) == INV
    for kw in (dict(x=None), dict(y=None), dict(table=None), dict(positions=None), dict(dtype=5), dict(n=-1), dict(heads=0),
               dict(rot_dim=3), dict(rot_dim=66), dict(rot_dim=0), dict(table_rows=0), dict(layout=2),
               dict(y=A16, y_token_stride=512)):
        assert call(_with(ok, **kw)) == INV, kw
    assert call(_with(ok, x=A16 + 1)) == ALN and call(_with(ok, positions=A16 + 2)) == ALN
    assert call(_with(ok, heads=1 << 26)) == UNS


def test_cache_refusals(L):
    ok = _lq.lq_kv_cache(A16, 10, 64, 8, 128, 4)
    a = _lq.lq_kv_append_args(A16, A16, A16, A16, 2, 3, 16, 1024, 1024, 2048, 2048, A16, A16, 100, A16, 128, 0)
    call = lambda c, a=a: L.lq_kv_append(H, ctypes.byref(c), ctypes.byref(a), None)  # noqa: E731
    for kw in (dict(pages=None), dict(num_pages=0), dict(page_size=0), dict(page_size=24), dict(kv_heads=0)):
        assert call(_with(ok, **kw)) == INV, kw
    for kw in (dict(bits=2), dict(bits=16), dict(head_dim=96), dict(head_dim=256)):
        assert call(_with(ok, **kw)) == UNS, kw
    assert call(_with(ok, pages=A16 + 8)) == ALN
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(dtype=3), dict(n=-1), dict(q_out=None), dict(q_heads=0),
               dict(positions=None), dict(rot_dim=0), dict(rot_dim=144), dict(layout=-1), dict(table_rows=0),
               dict(q_out_token_stride=4096)):
        assert call(ok, _with(a, **kw)) == INV, kw
    assert call(ok, _with(a, rot_dim=24)) == UNS
    for kw in (dict(k=A16 + 8), dict(v_token_stride=1028), dict(q_token_stride=2052, q_out=A16 * 2), dict(slots=A16 + 4),
               dict(table=A16 + 4)):
        assert call(ok, _with(a, **kw)) == ALN, kw
    read = lambda slots=A16, n=3, k=A16, v=A16, dt=2: L.lq_kv_read(H, ctypes.byref(ok), slots, n, k, v, dt, None)  # noqa: E731
    assert read(slots=None) == INV and read(n=-1) == INV and read(k=None, v=None) == INV and read(dt=7) == INV
    assert read(k=A16 + 8) == ALN and read(slots=A16 + 4) == ALN
    assert L.lq_kv_read(None, ctypes.byref(ok), A16, 3, A16, A16, 2, None) == INV


def test_attention_refusals(L):
    c = _lq.lq_kv_cache(A16, 10, 64, 8, 128, 4)
    ok = _lq.lq_kv_attention_args(A16, A16, A16, 2, 3, 2, 32, 4096, 4096, A16, 5, 5, A16, A16, 100, 0.1)
    call = lambda a, h=H, c=c: L.lq_kv_attention(h, ctypes.byref(c), ctypes.byref(a), None)  # noqa: E731
    assert call(ok, h=None) == INV and call(ok, c=_with(c, page_size=8)) == INV
    for kw in (dict(q=None), dict(out=None), dict(block_table=None), dict(lens=None), dict(prefix_table=None), dict(dtype=0),
               dict(batch=0), dict(tokens=0), dict(q_heads=0), dict(q_heads=12), dict(max_pages=0), dict(max_pages=6),
               dict(prefix_len=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(_with(ok, **kw)) == INV, kw
    for kw in (dict(batch=1025), dict(tokens=65), dict(max_pages=1 << 26, block_table_stride=1 << 26)):
        assert call(_with(ok, **kw)) == UNS, kw
    for kw in (dict(q=A16 + 8), dict(out_token_stride=4100), dict(lens=A16 + 2), dict(lse=A16 + 1)):
        assert call(_with(ok, **kw)) == ALN, kw
