"""The shared prefix's dense kernel (17 rows per kv head and 385 tokens on) at its edges: binary16, pages outside
the cache in the prefix's page list, wide groups.  Bounds as in test_gpu_kv_attention.py."""
import numpy as np
import pytest

from tests import _kv_ref as R
from tests.test_gpu_kv_attention import SHAPES, Case, handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("B,T,hq,hkv,prefix", [(20, 1, 8, 2, 600), (33, 2, 4, 2, 385), (150, 1, 8, 2, 1000)])
def test_binary16(lqm, handle, bits, D, B, T, hq, hkv, prefix):  # noqa: F811
    g = np.random.default_rng(B)
    c = Case(lqm, [int(x) for x in g.integers(0, 60, B)], T=T, hq=hq, hkv=hkv, D=D, bits=bits, prefix=prefix, page=48, dtype="f16",
             seed=B)
    c.check(*c.run(handle), requests=[0, 1, B // 2, B - 1])
    handle.sync()


def _hidden(c, pages):
    """The case with these entries of the prefix's page list outside the cache, and the prefix tokens that are left."""
    pt = c.pt.copy()
    pt[pages] = [(-1, 10 ** 6, c.cache.num_pages)[i % 3] for i in range(len(pages))]
    j = np.arange(c.prefix)
    return pt, ~np.isin(j // c.page, pages)


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,pages", [(20, [1]), (20, [0, 3, 4, 8]), (20, list(range(4, 11))), (20, list(range(11))), (140, [2, 10]),
                                     (3, [1, 5]), (3, list(range(11)))])
def test_prefix_pages_outside_the_cache(lqm, handle, bits, D, dtype, B, pages):  # noqa: F811
    """Their tokens are hidden from every row and LQ_ERR_INDEX reported, also where nothing is left of the prefix; 3 requests
    take the other kernel."""
    c = Case(lqm, [int(x) for x in np.random.default_rng(B).integers(0, 40, B)], hq=2, hkv=2, D=D, bits=bits, prefix=700, page=64,
             dtype=dtype, seed=len(pages))
    c.lens[1] = 0                                     # (a row that may see nothing at all)
    good = c.run(handle)                              # (what lies in shared memory from before is not zero)
    handle.sync()
    kept, (c.pt, left) = c.pt, _hidden(c, pages)
    out, lse = c.run(handle)
    with pytest.raises(lqm.LQError) as e:
        handle.sync()
    assert e.value.status == lqm.LQ_ERR_INDEX
    ulp = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    pp, po = (a[left] for a in c.tokens(kept, c.prefix))
    for b in {0, 1, 2, B - 1}:
        bp, bo = c.tokens(c.bt[b], c.lens[b])
        pg, of = np.concatenate([pp, bp]), np.concatenate([po, bo])
        for h in range(2):
            q = c.q[b][:, h:h + 1].float().cpu().numpy()
            o, s, mass, size = R.attend(q, c.k[pg, h, of], c.v[pg, h, of], [len(pg)], c.scale)
            zmass = R.attend(q, c.k[pg, h, of], c.z[pg, h, of], [len(pg)], c.scale)[0]
            got, l = out[b, :, h:h + 1].float().cpu().numpy(), lse[b, :, h:h + 1].cpu().numpy()
            if len(pg) == 0:
                assert not got.any() and np.isneginf(l).all()
                continue
            size = size * c.scale
            assert np.all(np.abs(l - s) <= 2.0 ** -20 * size + 2.0 ** -19)
            bound = (2.0 ** -11 + 2.0 ** -18 * (1 + size[..., None])) * (mass + 2 * zmass) + ulp * np.abs(o) + 2.0 ** -24 * np.abs(c.v[pg, h, of]).max()
            assert np.all(np.abs(got - o) <= bound)
    c.pt = kept
    again = c.run(handle)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
    handle.sync()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_group_of_both_infinities_leaves_the_others_alone(lqm, handle, bits, dtype):  # noqa: F811
    """A value token whose group 0 holds both infinities (clamped when cached), under 70 rows: groups 1 to 3 keep the
    ordinary bound; group 0 has the token's share of binary16's range in its mass."""
    hkv, D, n, B = 1, 128, 450, 70
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float16
    cache = lqm.KVCache(num_pages=-(-n // 64) + B, page_size=64, kv_heads=hkv, head_dim=D, bits=bits)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(n, hkv, D, generator=g, device="cuda").to(tdt) for _ in range(2))
    v[77, 0, 0], v[77, 0, 1] = -float("inf"), float("inf")
    at = torch.arange(n, device="cuda")
    handle.kv_append(cache, k, v, at)
    q = torch.randn(B, 1, 1, D, generator=g, device="cuda").to(tdt)
    shared = -(-n // 64)
    bt = torch.arange(shared, shared + B, device="cuda", dtype=torch.int32)[:, None]
    out, lse = handle.kv_attention(q, cache, bt, torch.zeros(B, dtype=torch.int32, device="cuda"),
                                   prefix_table=torch.arange(shared, device="cuda", dtype=torch.int32), prefix_len=n)
    kk, vv = (x[:, 0].cpu().numpy() for x in handle.kv_read(cache, at, dtype=torch.float32))
    # |Z| of a value's group is at most the largest |v| of the group
    z = np.repeat(np.abs(vv).reshape(n, D // 32, 32).max(-1), 32, -1)
    ulp = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    for b in range(0, B, 7):
        qs = q[b].float().cpu().numpy()
        o, s, mass, size = R.attend(qs, kk, vv, [n], D ** -0.5)
        zmass, size = R.attend(qs, kk, z, [n], D ** -0.5)[0], size * D ** -0.5
        assert np.all(np.abs(lse[b].cpu().numpy() - s) <= 2.0 ** -20 * size + 2.0 ** -19)
        bound = (2.0 ** -11 + 2.0 ** -18 * (1 + size[..., None])) * (mass + 2 * zmass) + ulp * np.abs(o) + \
            2.0 ** -24 * np.repeat(np.abs(vv).reshape(n, 4, 32).max((0, 2)), 32)
        assert np.all(np.abs(out[b].float().cpu().numpy() - o) <= bound)
    handle.sync()
