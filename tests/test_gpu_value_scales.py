"""lq_kv_attention where the values' scales differ widely: a wide group (a clamped infinity) among ordinary ones.

Bound of an output over n visible tokens, with u = 2^-11 and p a token's probability relative to the row's largest:
* probabilities, and probabilities times S, are rounded by u / 2 each:  u * sum p (|v| + 2 |Z|), as everywhere;
* a product of a probability and an ordinary S is held with 2^11 in front in binary16, so it is off by 2^-36 at least:
  at most 255 * 2^-36 < 2^-28 a token after its code;
* for a token whose group has S > 3.9, span = S * (2^bits - 1): a probability below 2^-25 is off by 2^-36, and the wide S is
  multiplied after a power of two that leaves at most 2 of the tile's largest.  With |Z| <= span together at most
  2^-36 * 3 span < 2^-34 span; and neither rounding moves a product by more than itself, so at most 4 p span.
Sums of p are at least 1, so dividing by them makes nothing larger.
"""
import numpy as np
import pytest

from tests import _kv_ref as R
from tests.test_gpu_kv_attention import SHAPES, Case, handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
WIDE = {4: 8734.0, 8: 513.5}          # S of a group from -65504 to 65504


class Edit:
    """Change cached tokens of a case: keys' and values' codes, S and Z of one token of one head at a time."""

    def __init__(self, case):
        self.c, self.pages = case, case.cache.pages.cpu().numpy()

    def token(self, b, j, head, fn):
        c = self.c
        page, off = c.bt[b][j // c.page], j % c.page
        _, _, ko, vo = R.unpack(self.pages[page, head, off // 16], c.bits, c.D)
        fn(ko, vo, off % 16)
        self.pages[page, head, off // 16] = R.pack(*ko, *vo, c.bits)
        with np.errstate(all="ignore"):
            c.k[page, head, off] = R.dequantize(*ko)[off % 16]
            c.v[page, head, off] = R.dequantize(*vo)[off % 16]
        c.z[page, head, off] = np.repeat(np.abs(vo[2][off % 16].astype(np.float32)), 32, -1)

    def done(self):
        self.c.cache.pages.copy_(torch.from_numpy(self.pages))


def _hide(c, b, j, head):
    """Token j's key as far below the others as a score gets: its probability is below 2^-38."""
    x = c.q.float().cpu().numpy()[b, 0, head * (c.hq // c.hkv)]
    kk, S, Z = R.quantize((-3.6 * x / np.linalg.norm(x) * np.sqrt(c.D)).astype(np.float32), c.bits)

    def fn(ko, vo, t):
        ko[0][t], ko[1][t], ko[2][t] = kk, S, Z
    return fn


def _set_value(groups, S, Z):
    def fn(ko, vo, t):
        for g in groups:
            vo[1][t, g], vo[2][t, g] = S, Z
    return fn


def _tight(c, out, lse, spans):
    """spans: of the tokens of each request, [n] or a number: S * (2^bits - 1) of the widest group where that S > 3.9."""
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    ulp = 2.0 ** -8 if c.q.dtype == torch.bfloat16 else 2.0 ** -11
    q = c.q.float().cpu().numpy()
    gsz = c.hq // c.hkv
    for b, n in enumerate(c.lens):
        pages, offs = c.tokens(c.bt[b], n)
        for h in range(c.hkv):
            hs = slice(h * gsz, (h + 1) * gsz)
            k, v, z = c.k[pages, h, offs], c.v[pages, h, offs], c.z[pages, h, offs]
            o, s, mass, size = R.attend(q[b][:, hs], k, v, [n], c.scale)
            zmass = R.attend(q[b][:, hs], k, z, [n], c.scale)[0]
            size = size * c.scale
            score = q[b][:, hs].astype(np.float64) @ k.T.astype(np.float64) * c.scale
            p = np.exp(score - score.max(-1, keepdims=True))
            wide = (np.minimum(2.0 ** -34, 4 * p) * spans[b]).sum(-1)[..., None]
            assert np.all(np.abs(lse[b][:, hs] - s) <= 2.0 ** -20 * size + 2.0 ** -19)
            bound = (2.0 ** -11 + 2.0 ** -18 * (1 + size[..., None])) * (mass + 2 * zmass) + ulp * np.abs(o) + 2.0 ** -28 * n + wide
            err = np.abs(out[b][:, hs] - o)
            assert np.all(err <= bound), (b, h, float((err / bound).max()))


def _spans(c, of):
    """of: (request, token) -> S."""
    out = [np.zeros(n) for n in c.lens]
    for (b, j), S in of.items():
        out[b][j] = S * (2 ** c.bits - 1) if S > 3.9 else 0.0
    return out


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hidden", [False, True])
@pytest.mark.parametrize("where,vscale", [(0, 1.0), (3, 0.1), (200, 0.01), (599, 0.1), (0, 0.01)])
def test_one_wide_value(lqm, handle, bits, D, dtype, hidden, where, vscale):  # noqa: F811
    """One group of one token spans binary16's range.  The other groups keep their precision, and where the token has no
    probability its own group does too."""
    c = Case(lqm, [600, 40, 9], hq=2, hkv=2, D=D, bits=bits, dtype=dtype, seed=where, vscale=vscale, poison=False)
    e = Edit(c)
    at = ((0, where), (1, where % 40), (2, where % 9))
    for b, j in at:
        for h in range(2):
            e.token(b, j, h, _set_value([1], WIDE[bits], -65504.0))
            if hidden:
                e.token(b, j, h, _hide(c, b, j, h))
    e.done()
    _tight(c, *c.run(handle), _spans(c, {i: WIDE[bits] for i in at}))


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("S,vscale", [(4.0, 0.01), (60.0, 0.1), (513.5, 1.0), (513.5, 0.01)])
def test_first_tile_wide_and_hidden(lqm, handle, bits, D, S, vscale):  # noqa: F811
    """The tokens that a warp meets first have wide values and no probability; the rest are ordinary."""
    c = Case(lqm, [256], hq=2, hkv=2, D=D, bits=bits, dtype="f16", seed=int(S), vscale=vscale, poison=False)
    e = Edit(c)
    for j in range(128):
        for h in range(2):
            e.token(0, j, h, _set_value(range(D // 32), S, -0.5 * (2 ** bits - 1) * S))
            e.token(0, j, h, _hide(c, 0, j, h))
    e.done()
    _tight(c, *c.run(handle), _spans(c, {(0, j): S for j in range(128)}))


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("first,rest", [(0.0, 1.0), (2.0 ** -14, 1.0), (1.0, 2.0 ** -12), (2.0 ** -14, 300.0), (300.0, 1.0), (300.0, 500.0)])
def test_scales_that_change_along_the_context(lqm, handle, bits, D, first, rest):  # noqa: F811
    c = Case(lqm, [400], hq=2, hkv=2, D=D, bits=bits, dtype="f16", seed=1, poison=False)
    e, top = Edit(c), 2 ** bits - 1          # (S times the largest code stays finite: 500 * 255 / 2)
    for j in range(400):
        S = np.float16(first if j < 128 else rest)
        for h in range(2):
            e.token(0, j, h, _set_value(range(D // 32), S, np.float16(-0.5 * top) * S))
    e.done()
    _tight(c, *c.run(handle), _spans(c, {(0, j): first if j < 128 else rest for j in range(400)}))


@pytest.mark.parametrize("bits,D", SHAPES)
def test_groups_and_tokens_of_many_sizes(lqm, handle, bits, D):  # noqa: F811
    """S spread over 2^-14 .. 2^9, from token to token and from group to group, under ordinary probabilities."""
    c = Case(lqm, [700], hq=4, hkv=2, D=D, bits=bits, dtype="f16", seed=2, poison=False)
    e, top, g = Edit(c), 2 ** bits - 1, np.random.default_rng(4)
    for j in range(700):
        for h in range(2):
            for grp in range(D // 32):
                S = np.float16(2.0 ** g.uniform(-14, 9 if grp == 0 and j % 50 == 7 else 1 - 4 * grp))
                e.token(0, j, h, _set_value([grp], S, np.float16(-0.5 * top) * S))
    e.done()
    _tight(c, *c.run(handle), _spans(c, {(0, j): 512.0 for j in range(7, 700, 50)}))


@pytest.mark.parametrize("bits,D", SHAPES)
def test_small_values_of_a_wide_group_come_out_small(lqm, handle, bits, D):  # noqa: F811
    """A wide group whose codes make S c + Z zero: with the token's probability rounded the same against both parts they cancel,
    to fp32's rounding of sums as large as p |Z| (2^-24 a step, below 2^-20 in all), beside the ordinary bound of the rest."""
    c = Case(lqm, [90], hq=2, hkv=2, D=D, bits=bits, dtype="f16", seed=9, poison=False)
    e, S, code = Edit(c), np.float16(512.0 if bits == 8 else 4096.0), 100 if bits == 8 else 7
    for h in range(2):
        def fn(ko, vo, t):
            vo[0][t, 32:64], vo[1][t, 1], vo[2][t, 1] = code, S, np.float16(-float(S) * code)
        e.token(0, 20, h, fn)
    e.done()
    assert not c.v[c.bt[0][0], :, 20, 32:64].any()
    out, lse = c.run(handle)
    pages, offs = c.tokens(c.bt[0], 90)
    for h in range(2):
        k, v, z = (a[pages, h, offs].copy() for a in (c.k, c.v, c.z))
        big = float(z[20, 32])
        z[20, 32:64] = 0.0
        q = c.q[0][:, h:h + 1].float().cpu().numpy()
        o, s, mass, size = R.attend(q, k, v, [90], c.scale)
        zmass, size = R.attend(q, k, z, [90], c.scale)[0], size * c.scale
        p20 = np.exp((q.astype(np.float64) @ k[20].astype(np.float64)) * c.scale - s)[..., None]
        bound = (2.0 ** -11 + 2.0 ** -18 * (1 + size[..., None])) * (mass + 2 * zmass) + 2.0 ** -11 * np.abs(o) + 2.0 ** -28 * 90
        bound = bound + np.where((np.arange(D) // 32 == 1)[None, None], p20 * big * 2.0 ** -20, 0.0)
        assert np.all(np.abs(out[0][:, h:h + 1].float().cpu().numpy() - o) <= bound)
