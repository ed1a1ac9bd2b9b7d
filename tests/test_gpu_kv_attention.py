"""lq_kv_attention against a 64-bit evaluation over the cache's own values.

Bounds, with u = 2^-11 (the kernels multiply probabilities, and probabilities times a group's scale, as 16-bit
floats with fp32 sums; keys, queries and scores keep fp32 precision):
* a score is off by at most 2^-20 * scale * sum_d |q_d k_d| (fp32 sums of D products and the exponential's 2^-22), so
  lse by the largest such amount plus 2^-19, and each probability by twice that, relatively;
* each probability is rounded at most twice, by u / 2 each, against S c and once against Z: with |S c| <= |v| + |Z|
  an output is off by at most (u + 2^-18 * (1 + size)) * sum_j p_j (|v_j| + 2 |Z_j|), and by its own rounding (2^-8
  of it for bfloat16, 2^-11 for binary16), with 2^-24 of the largest value for probabilities that vanish.
"""
import numpy as np
import pytest

from tests import _kv_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TDT = {"f16": torch.float16, "bf16": torch.bfloat16}


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


class Case:
    """A cache with random pages, block tables of shuffled pages, poisoned slots past every length."""

    def __init__(self, lqm, lens, T=1, hq=8, hkv=2, D=128, bits=4, page=64, prefix=0, dtype="bf16", seed=0, extra_pages=0,
                 spread=1.0, vscale=1.0, poison=True):
        g = np.random.default_rng(seed)
        self.lens, self.T, self.hq, self.hkv, self.D, self.bits, self.page, self.prefix = lens, T, hq, hkv, D, bits, page, prefix
        B = len(lens)
        each = max(1, -(-max(lens) // page)) + extra_pages
        shared = -(-prefix // page)
        total = B * each + shared + 1
        G = D // 32
        top = 2 ** bits - 1
        shape = (total, hkv, page // 16, 16)
        codes = [g.integers(0, top + 1, shape + (D,), dtype=np.uint8) for _ in range(2)]
        meta = []
        for scale in (spread, vscale):
            S = ((g.random(shape + (G,)) + 3.0) * scale / top).astype(np.float16)
            Z = (-0.5 * top * S.astype(np.float32) + 0.3 * scale * g.standard_normal(shape + (G,))).astype(np.float16)
            meta += [S, Z]
        order = g.permutation(total).astype(np.int32)
        self.bt, self.pt = order[:B * each].reshape(B, each), order[B * each:B * each + shared]
        if poison:      # what lies past a length (and in pages nobody has) is NaN or infinite
            used = np.zeros((total, page), bool)
            for b, n in enumerate(lens):
                j = np.arange(min(n, each * page))
                used[self.bt[b][j // page], j % page] = True
            j = np.arange(prefix)
            used[self.pt[j // page], j % page] = True
            free = ~used.reshape(total, 1, page // 16, 16)
            for i, m in enumerate(meta):
                m[np.broadcast_to(free, shape)] = [np.nan, np.inf, np.nan, -np.inf][i]
        tiles = R.pack(codes[0], meta[0], meta[1], codes[1], meta[2], meta[3], bits)
        with np.errstate(all="ignore"):
            self.k = R.dequantize(codes[0], meta[0], meta[1]).reshape(total, hkv, page, D)
            self.v = R.dequantize(codes[1], meta[2], meta[3]).reshape(total, hkv, page, D)
        self.z = np.repeat(np.abs(meta[3].astype(np.float32)), 32, -1).reshape(total, hkv, page, D)
        self.cache = lqm.KVCache(torch.from_numpy(tiles).cuda(), page_size=page, kv_heads=hkv, head_dim=D, bits=bits)
        self.q = torch.from_numpy(g.standard_normal((B, T, hq, D)).astype(np.float32)).to(TDT[dtype]).cuda()
        self.scale = D ** -0.5

    def run(self, handle, **kw):
        return handle.kv_attention(self.q, self.cache, torch.from_numpy(self.bt).cuda(),
                                   torch.tensor(self.lens, dtype=torch.int32, device="cuda"), scale=self.scale,
                                   prefix_table=torch.from_numpy(self.pt).cuda() if self.prefix else None,
                                   prefix_len=self.prefix, **kw)

    def tokens(self, table, n):
        j = np.arange(n)
        return table[j // self.page], j % self.page

    def check(self, out, lse, requests=None):
        out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        ulp = 2.0 ** -8 if self.q.dtype == torch.bfloat16 else 2.0 ** -11
        gsz = self.hq // self.hkv
        q = self.q.float().cpu().numpy()
        worst = 0.0
        for b in (range(len(self.lens)) if requests is None else requests):
            n = min(max(self.lens[b], 0), self.bt.shape[1] * self.page)
            pp, po = self.tokens(self.pt, self.prefix)
            bp, bo = self.tokens(self.bt[b], n)
            pages, offs = np.concatenate([pp, bp]), np.concatenate([po, bo])
            visible = [self.prefix + max(0, n - self.T + 1 + t) for t in range(self.T)]
            for h in range(self.hkv):
                hs = slice(h * gsz, (h + 1) * gsz)
                k, v, z = self.k[pages, h, offs], self.v[pages, h, offs], self.z[pages, h, offs]
                o, s, mass, size = R.attend(q[b][:, hs], k, v, visible, self.scale)
                zmass = R.attend(q[b][:, hs], k, z, visible, self.scale)[0]
                size = size * self.scale
                assert np.array_equal(np.isneginf(lse[b][:, hs]), np.isneginf(s))
                live = ~np.isneginf(s)
                e = np.abs(lse[b][:, hs][live] - s[live])
                assert np.all(e <= 2.0 ** -20 * size[live] + 2.0 ** -19), (b, h, e.max())
                bound = (2.0 ** -11 + 2.0 ** -18 * (1 + size[..., None])) * (mass + 2 * zmass) + ulp * np.abs(o) + \
                    2.0 ** -24 * (np.abs(v).max() if len(v) else 0.0)
                err = np.abs(out[b][:, hs] - o)
                worst = max(worst, float((err / (bound + 1e-30)).max()))
                assert np.all(err <= bound + 1e-30), (b, h, float((err / (bound + 1e-30)).max()))
                assert np.all(out[b][:, hs][~live] == 0)
        return worst


SHAPES = [(4, 64), (4, 128), (8, 64), (8, 128)]


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 500, 2049])
def test_one_token(lqm, handle, bits, D, dtype, n):
    c = Case(lqm, [n], D=D, bits=bits, dtype=dtype, seed=n)
    c.check(*c.run(handle))
    handle.sync()


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (8, 1), (12, 4), (16, 1), (24, 1), (40, 2), (64, 8)])
def test_head_groups(lqm, handle, bits, D, hq, hkv):
    c = Case(lqm, [300, 0, 77], hq=hq, hkv=hkv, D=D, bits=bits, seed=hq)
    c.check(*c.run(handle))


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("T", [2, 3, 4, 7, 16, 33, 64])
def test_several_tokens_are_causal(lqm, handle, bits, D, T):
    """The last T tokens see what precedes them; rows of requests shorter than T see nothing."""
    c = Case(lqm, [T, 1, 0, T - 1, 100 + T, 257], T=T, hq=6, hkv=2, D=D, bits=bits, seed=T)
    c.check(*c.run(handle))


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 256])
def test_page_sizes(lqm, handle, page):
    c = Case(lqm, [1000, 3, 511, 512, 513], page=page, seed=page, extra_pages=2)
    c.check(*c.run(handle))


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("prefix", [1, 16, 63, 64, 700])
@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 2), (3, 4, 4), (1, 32, 1), (2, 24, 2)])
def test_shared_prefix(lqm, handle, bits, D, prefix, T, hq, hkv):
    c = Case(lqm, [0, 1, 200, 64, 5], T=T, hq=hq, hkv=hkv, D=D, bits=bits, prefix=prefix, seed=prefix)
    c.check(*c.run(handle))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,T,hq,hkv,prefix", [(40, 1, 16, 2, 1500), (150, 1, 4, 4, 333), (9, 5, 8, 1, 2000), (70, 2, 8, 2, 130)])
def test_shared_prefix_many_rows(lqm, handle, bits, B, T, hq, hkv, prefix):
    g = np.random.default_rng(B)
    c = Case(lqm, [int(x) for x in g.integers(0, 90, B)], T=T, hq=hq, hkv=hkv, bits=bits, prefix=prefix, seed=B, page=32)
    c.check(*c.run(handle), requests=list(g.integers(0, B, 6)) + [0, B - 1])


@pytest.mark.parametrize("bits,D", SHAPES)
@pytest.mark.parametrize("spread,vscale,mult", [(0.01, 1.0, 100.0), (1e-4, 1.0, 1e4), (1.0, 0.02, 1.0), (1.0, 2e-3, 1.0),
                                               (3000.0, 3000.0, 1e-3)])
def test_shared_prefix_scales_far_from_one(lqm, handle, bits, D, spread, vscale, mult):
    """Small keys under large queries (scales of the keys down to binary16's subnormals), small and large values."""
    c = Case(lqm, [5] * 20, hq=8, hkv=2, D=D, bits=bits, prefix=600, spread=spread, vscale=vscale, seed=17, page=48)
    c.q = (c.q.float() * mult).to(torch.bfloat16)
    c.check(*c.run(handle), requests=[0, 7, 19])


@pytest.mark.parametrize("bits", [4, 8])
def test_shared_prefix_groups_that_span_the_range(lqm, handle, bits):
    """Keys and values of which a group holds both infinities (clamped when cached): the dense product stays finite."""
    hkv, D, n, B = 1, 128, 320, 70
    cache = lqm.KVCache(num_pages=n // 64 + B, page_size=64, kv_heads=hkv, head_dim=D, bits=bits)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(n, hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    k[9, 0, 32], k[9, 0, 40], v[77, 0, 0], v[77, 0, 1] = float("inf"), -float("inf"), -float("inf"), float("inf")
    at = torch.arange(n, device="cuda")
    handle.kv_append(cache, k, v, at)
    q = torch.randn(B, 1, 1, D, generator=g, device="cuda").bfloat16() * 1e-4
    bt = torch.arange(n // 64, n // 64 + B, device="cuda", dtype=torch.int32)[:, None]
    out, lse = handle.kv_attention(q, cache, bt, torch.zeros(B, dtype=torch.int32, device="cuda"),
                                   prefix_table=torch.arange(n // 64, device="cuda", dtype=torch.int32), prefix_len=n)
    kk, vv = handle.kv_read(cache, at, dtype=torch.float32)
    kk, vv = kk[:, 0].cpu().numpy(), vv[:, 0].cpu().numpy()
    for b in (0, 35, 69):
        o, s, mass, size = R.attend(q[b].float().cpu().numpy(), kk, vv, [n], D ** -0.5)
        # the group's keys are c S / 2 twice, each rounded by 2^-11: an error of 2^-11 of its share of the score
        tol = 2.0 ** -11 * size[0] * D ** -0.5 + 2.0 ** -19
        assert abs(float(lse[b, 0, 0]) - s[0, 0]) <= tol
        assert np.all(np.abs(out[b, 0].float().cpu().numpy() - o[0]) <= (2.0 ** -10 + 2 * tol) * mass[0] + 2.0 ** -8 * np.abs(o[0]) + 2.0 ** -11 * 65504 / n)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B", [33, 200, 1024])
def test_many_requests(lqm, handle, bits, B):
    g = np.random.default_rng(B)
    c = Case(lqm, [int(x) for x in g.integers(0, 120, B)], hq=4, hkv=2, bits=bits, D=64, page=32, seed=B)
    c.check(*c.run(handle), requests=list(g.integers(0, B, 8)) + [0, B - 1])


@pytest.mark.parametrize("bits", [4, 8])
def test_long_context_split_over_the_device(lqm, handle, bits):
    c = Case(lqm, [40007, 13], hq=8, hkv=1, bits=bits, seed=5, poison=False)
    out, lse = c.run(handle)
    c.check(out, lse)
    again = c.run(handle)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])      # the joins have one order


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("spread,vscale", [(8.0, 1.0), (0.01, 1.0), (1.0, 1e-4), (1.0, 3000.0), (30.0, 0.01)])
def test_scales_far_from_one(lqm, handle, dtype, spread, vscale):
    """Peaked and flat scores, values that are tiny or near binary16's limit: the 16-bit products keep their precision."""
    for bits in (4, 8):
        c = Case(lqm, [700, 40], bits=bits, dtype=dtype, spread=spread, vscale=vscale, seed=11)
        c.check(*c.run(handle))


def test_one_key_far_above_many(lqm, handle):
    """One key takes most of the softmax, 30000 others share the rest: their small probabilities still count."""
    c = Case(lqm, [30000], hq=4, hkv=1, bits=8, seed=3, poison=False)
    x = c.q.float().cpu().numpy()[0, 0].mean(0)
    k = (3.5 * x / np.linalg.norm(x) * np.sqrt(128)).astype(np.float32)
    kk, S, Z = R.quantize(k, 8)
    page, off = c.bt[0][77 // 64], 77 % 64
    tile = c.cache.pages[page, 0, off // 16].cpu().numpy()
    _, _, ko, vo = R.unpack(tile, 8, 128)
    for a, b in zip(ko, (kk, S, Z)):
        a[off % 16] = b
    c.cache.pages[page, 0, off // 16] = torch.from_numpy(R.pack(*ko, *vo, 8)).cuda()
    c.k[page, 0, off] = R.dequantize(kk, S, Z)
    c.check(*c.run(handle))


@pytest.mark.parametrize("mult", [1e-20, 1e-3, 1e3, 1e20])
def test_query_magnitudes(lqm, handle, mult):
    """bfloat16 queries of any finite size (scores scaled back by `scale`)."""
    c = Case(lqm, [300], seed=2)
    c.q = (c.q.float() * mult).to(torch.bfloat16)
    c.scale = 128 ** -0.5 / mult
    c.check(*c.run(handle))


def test_nan_and_infinite_rows_stay_alone(lqm, handle):
    c = Case(lqm, [300, 200], hq=8, hkv=2, seed=6)
    good, _ = c.run(handle)
    c.q[0, 0, 3, 5] = float("nan")
    out, lse = c.run(handle)
    assert bool(out[0, 0, 3].isnan().all()) and bool(lse[0, 0, 3].isnan())
    keep = torch.ones(8, dtype=torch.bool)
    keep[3] = False
    assert torch.equal(out[0, 0, keep], good[0, 0, keep]) and torch.equal(out[1], good[1])
    c.cache.pages[c.bt[1][0], 1, 0] = 255                      # a cached NaN: everyone who sees it is NaN
    out, _ = c.run(handle)
    assert bool(out[1, 0, 4:].isnan().all()) and bool(out[1, 0, :4].isfinite().all()) and bool(out[0, 0, keep].isfinite().all())


def test_strides_out_and_lse(lqm, handle):
    c = Case(lqm, [90, 300], T=2, hq=4, hkv=2, seed=8)
    wide = torch.zeros(2, 2, 12, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 4:8] = c.q
    ref, rl = c.run(handle)
    c.q = wide[:, :, 4:8]
    dst = torch.full((2, 2, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 2, 4, device="cuda")
    c.run(handle, out=dst[:, :, :4], lse=lse)
    assert torch.equal(dst[:, :, :4], ref) and torch.equal(lse, rl) and bool((dst[:, :, 4:] == 3).all())
    c.bt = np.concatenate([c.bt, c.bt], 1)[:, :c.bt.shape[1]]   # a block table that is a slice of a wider one
    c.check(*c.run(handle))


def test_bad_pages_hide_their_tokens(lqm, handle):
    c = Case(lqm, [200], hq=4, hkv=2, seed=9)
    c.bt = c.bt.copy()
    ref = Case(lqm, [200], hq=4, hkv=2, seed=9)
    for bad in (-1, 10 ** 6):
        c.bt[0, 1] = bad
        out, lse = c.run(handle)
        with pytest.raises(lqm.LQError) as e:
            handle.sync()
        assert e.value.status == lqm.LQ_ERR_INDEX
    keep = np.r_[0:64, 128:200]
    pages, offs = ref.tokens(ref.bt[0], 200)
    for h in range(2):
        hs = slice(2 * h, 2 * h + 2)
        k, v = ref.k[pages, h, offs][keep], ref.v[pages, h, offs][keep]
        o, s, mass, _ = R.attend(c.q.float().cpu().numpy()[0][:, hs], k, v, [len(keep)], c.scale)
        assert np.abs(lse[0].cpu().numpy()[:, hs] - s).max() < 1e-4
        assert np.abs(out[0].float().cpu().numpy()[:, hs] - o).max() < 0.02
    handle.sync()


def test_lens_are_clamped(lqm, handle):
    c = Case(lqm, [128, 128], seed=4)
    ref = c.run(handle)
    c.lens = [10 ** 6, -3]
    out, lse = c.run(handle)
    assert torch.equal(out[0], ref[0][0]) and torch.equal(lse[0], ref[1][0])
    assert not bool(out[1].any()) and bool(torch.isneginf(lse[1]).all())
    handle.sync()


def test_refusals(lqm, handle):
    c = Case(lqm, [90], seed=8)
    bt, ln = torch.from_numpy(c.bt).cuda(), torch.tensor([90], dtype=torch.int32, device="cuda")
    for bad in (lambda: handle.kv_attention(c.q[..., :64], c.cache, bt, ln), lambda: handle.kv_attention(c.q, c.cache, bt.long(), ln),
                lambda: handle.kv_attention(c.q, c.cache, bt, ln.long()), lambda: handle.kv_attention(c.q, c.cache, bt, ln.cpu()),
                lambda: handle.kv_attention(c.q, c.cache, bt[0], ln), lambda: handle.kv_attention(c.q.transpose(2, 3), c.cache, bt, ln),
                lambda: handle.kv_attention(c.q, c.cache, bt, ln, prefix_table=bt[0], prefix_len=10 ** 6),
                lambda: handle.kv_attention(c.q, c.cache, bt, ln, lse=torch.empty(1, 1, 8, dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: handle.kv_attention(c.q.float(), c.cache, bt, ln), lqm.LQ_ERR_INVALID_ARG),
                        (lambda: handle.kv_attention(c.q[:, :, :7].contiguous(), c.cache, bt, ln), lqm.LQ_ERR_INVALID_ARG),
                        (lambda: handle.kv_attention(c.q, c.cache, bt, ln, scale=-1.0), lqm.LQ_ERR_INVALID_ARG)):
        with pytest.raises(lqm.LQError) as e:
            bad()
        assert e.value.status == status


def test_small_workspace(lqm):
    """A handle whose workspace holds little: the call answers LQ_ERR_WORKSPACE or the right result."""
    c = Case(lqm, [5000, 300], hq=32, hkv=4, T=4, seed=2, prefix=500)
    h = lqm.Handle(0, workspace_bytes=1 << 16)
    try:
        out, lse = c.run(h)
        c.check(out, lse, requests=[1])
    except lqm.LQError as e:
        assert e.status == lqm.LQ_ERR_WORKSPACE
    h.close()


def test_captured_in_a_graph_with_new_lengths(lqm, handle):
    """One captured call serves other lengths, pages and queries: nothing of a call is kept on the host."""
    c, d = Case(lqm, [500, 30, 77], seed=1, prefix=100), Case(lqm, [12, 512, 400], seed=1, prefix=100)
    bt, ln = torch.from_numpy(c.bt).cuda(), torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    pt = torch.from_numpy(c.pt).cuda()
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device="cuda")
    call = lambda: handle.kv_attention(c.q, c.cache, bt, ln, scale=c.scale, prefix_table=pt, prefix_len=100, out=out, lse=lse)  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    c.check(out, lse)
    for dst, src in ((bt, torch.from_numpy(d.bt)), (pt, torch.from_numpy(d.pt)), (ln, torch.tensor(d.lens, dtype=torch.int32)),
                     (c.cache.pages, d.cache.pages), (c.q, d.q)):
        dst.copy_(src)
    g.replay()
    d.check(out, lse)
