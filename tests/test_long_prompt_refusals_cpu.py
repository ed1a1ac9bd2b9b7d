"""Refusals of the chunk and window attention and of the log probabilities: at the C boundary and in the binding.  No GPU:
every call fails before the handle is read."""
import ctypes
import types

import pytest

import bit_weight_quantized_dequant_gb300 as lq
from bit_weight_quantized_dequant_gb300 import _lq
from tests.test_binding_refusals_cpu import _OnDevice, handle  # noqa: F401

torch = pytest.importorskip("torch")
H, A16 = ctypes.c_void_p(0x1000), 0x10000
INV, UNS, ALN = _lq.LQ_ERR_INVALID_ARG, _lq.LQ_ERR_UNSUPPORTED, _lq.LQ_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def L():
    lq.build()
    return _lq.load_library(build_if_missing=False)


def chunk(L, cache=(A16, 10, 64, 8, 128, 4), h=H, **kw):
    c = _lq.lq_kv_cache(*cache)
    a = _lq.lq_kv_chunk_args(A16, A16, A16, _lq.BF16, 3, 100, 32, 4096, 4096, A16, A16, 5, 5, A16, 0, 0, 0.1)
    for k, v in kw.items():
        setattr(a, k, v)
    return L.lq_kv_attention_chunk(h, ctypes.byref(c), ctypes.byref(a), None)


def test_chunk(L):
    assert chunk(L, tokens=0) == _lq.LQ_OK                      # nothing to do, nothing launched
    assert chunk(L, h=None) == INV
    for name in ("q", "out", "starts", "block_table", "lens"):
        assert chunk(L, **{name: None}) == INV, name
    for kw in (dict(dtype=_lq.F32), dict(dtype=9), dict(batch=0), dict(tokens=-1), dict(q_heads=0), dict(q_heads=33), dict(max_pages=0),
               dict(block_table_stride=4), dict(window=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(scale=2.4e38)):
        assert chunk(L, **kw) == INV, kw
    for kw in (dict(batch=1025), dict(max_pages=2 ** 25, block_table_stride=2 ** 25), dict(q_heads=2 ** 24), dict(tokens=2 ** 30)):
        assert chunk(L, **kw) == UNS, kw
    for kw in (dict(q=A16 + 8), dict(out=A16 + 8), dict(q_token_stride=4092), dict(out_token_stride=4097), dict(lens=A16 + 2), dict(starts=A16 + 1),
               dict(block_table=A16 + 2), dict(lse=A16 + 2)):
        assert chunk(L, **kw) == ALN, kw
    assert chunk(L, cache=(A16, 0, 64, 8, 128, 4)) == INV
    assert chunk(L, cache=(A16, 10, 24, 8, 128, 4)) == INV
    assert chunk(L, cache=(A16, 10, 64, 8, 96, 4)) == UNS
    assert chunk(L, cache=(A16 + 8, 10, 64, 8, 128, 4)) == ALN


def test_window(L):
    c = _lq.lq_kv_cache(A16, 10, 64, 8, 128, 4)
    a = _lq.lq_kv_attention_args(A16 + 8, A16, A16, 2, 3, 2, 32, 4096, 4096, A16, 5, 5, A16, None, 0, 0.1)
    call = lambda w, s, h=H: L.lq_kv_attention_window(h, ctypes.byref(c), ctypes.byref(a), w, s, None)  # noqa: E731
    assert call(1, 0) == ALN and call(2 ** 31 - 1, 2 ** 31 - 1) == ALN      # (only q's alignment is wrong)
    assert call(0, 0) == INV and call(-5, 0) == INV and call(4, -1) == INV and call(4, 0, None) == INV
    a.prefix_len, a.prefix_table = 5, A16
    assert call(4, 0) == UNS
    a.prefix_len = -1
    assert call(4, 0) == INV
    assert L.lq_kv_attention_window(H, ctypes.byref(c), None, 4, 0, None) == INV


def score(L, h=H, **kw):
    a = _lq.lq_logprobs_args(A16, _lq.BF16, 4, 100, 100, A16, A16, A16, A16, 5, A16, A16)
    for k, v in kw.items():
        setattr(a, k, v)
    return L.lq_logprobs(h, ctypes.byref(a), None)


def grad(L, h=H, **kw):
    a = _lq.lq_logprobs_grad_args(A16, 2 * A16, _lq.BF16, 4, 100, 100, 100, A16, A16, A16, A16, A16)
    for k, v in kw.items():
        setattr(a, k, v)
    return L.lq_logprobs_grad(h, ctypes.byref(a), None)


def test_logprobs(L):
    assert score(L, n=0) == _lq.LQ_OK
    assert score(L, h=None) == INV
    for kw in (dict(logits=None), dict(tokens=None), dict(logprob=None), dict(dtype=3), dict(n=-1), dict(vocab=0), dict(top=-1), dict(top=101),
               dict(top_ids=None), dict(top_logprobs=None)):
        assert score(L, **kw) == INV, kw
    assert score(L, top=65) == UNS and score(L, vocab=0x7fff0001) == UNS
    for kw in (dict(logits=A16 + 1), dict(tokens=A16 + 4), dict(logprob=A16 + 2), dict(entropy=A16 + 1), dict(lse=A16 + 2), dict(top_ids=A16 + 4),
               dict(top_logprobs=A16 + 2), dict(logits=A16 + 2, dtype=_lq.F32)):
        assert score(L, **kw) == ALN, kw


def test_logprobs_gradient(L):
    assert grad(L, n=0) == _lq.LQ_OK
    assert grad(L, h=None) == INV
    for kw in (dict(logits=None), dict(d_logits=None), dict(tokens=None), dict(lse=None), dict(entropy=None), dict(dtype=3), dict(n=-1),
               dict(vocab=0), dict(d_row_stride=99), dict(d_logits=A16, row_stride=101)):
        assert grad(L, **kw) == INV, kw
    assert grad(L, vocab=0x7fff0001) == UNS
    for kw in (dict(logits=A16 + 1), dict(d_logits=A16 + 1), dict(tokens=A16 + 4), dict(lse=A16 + 2), dict(entropy=A16 + 1), dict(d_logprob=A16 + 2),
               dict(d_entropy=A16 + 3)):
        assert grad(L, **kw) == ALN, kw


def test_more_rows_than_count(L):
    assert score(L, n=0x7fff0001) == UNS and grad(L, n=0x7fff0001) == UNS


def test_the_binding_of_chunks(handle):  # noqa: F811
    cache = types.SimpleNamespace(head_dim=64, kv_heads=2, page_size=16)
    D = _OnDevice
    q, bt = D((10, 4, 64), torch.float16), D((2, 5), torch.int32)
    lens, starts = D((2,), torch.int32), D((3,), torch.int32)

    def refused(match, *a, **kw):
        with pytest.raises(ValueError, match=match):
            handle.kv_attention_chunk(*a, **kw)
    refused("tokens", D((10, 64), torch.float16), cache, bt, lens, starts)
    refused("heads", D((10, 4, 128), torch.float16), cache, bt, lens, starts)
    refused("2.31", D((2 ** 31, 1, 64), torch.float16), cache, bt, lens, starts)
    refused("out", q, cache, bt, lens, starts, out=D((10, 4, 64), torch.bfloat16), lse=D((10, 4), torch.float32))
    out, lse = D((10, 4, 64), torch.float16), D((10, 4), torch.float32)
    refused("lse", q, cache, bt, lens, starts, out=out, lse=D((4, 10), torch.float32))
    refused("block_table", q, cache, D((2, 5), torch.int64), lens, starts, out=out, lse=lse)
    refused("starts", q, cache, bt, lens, D((2,), torch.int32), out=out, lse=lse)
    refused("starts", q, cache, bt, lens, D((3,), torch.int64), out=out, lse=lse)
    refused("starts", q, cache, bt, lens, None, out=out, lse=lse)
    refused("lens", q, cache, bt, D((3,), torch.int32), starts, out=out, lse=lse)
    refused("sinks", q, cache, bt, lens, starts, out=out, lse=lse, sinks=4)
    for window, sinks in ((0, 0), (-1, 0), (2 ** 31, 0), (4, -1), (4, 2 ** 31)):
        refused("window", q, cache, bt, lens, starts, out=out, lse=lse, window=window, sinks=sinks)
    refused("float32", D((10, 4, 64), torch.float64), cache, bt, lens, starts, out=D((10, 4, 64), torch.float64), lse=lse)


def test_the_binding_of_windows(handle):  # noqa: F811
    cache = types.SimpleNamespace(head_dim=64, kv_heads=2, page_size=16, _on=lambda device: None)
    D = _OnDevice
    q, bt, lens = D((2, 1, 4, 64), torch.float16), D((2, 5), torch.int32), D((2,), torch.int32)
    kw = dict(out=D((2, 1, 4, 64), torch.float16), lse=D((2, 1, 4), torch.float32))
    handle._lib = types.SimpleNamespace(lq_kv_attention=None, lq_kv_attention_window=None)
    with pytest.raises(ValueError, match="sinks"):
        handle.kv_attention(q, cache, bt, lens, sinks=3, **kw)
    for window, sinks in ((0, 0), (-1, 0), (2 ** 31, 0), (4, -1)):
        with pytest.raises(ValueError, match="window"):
            handle.kv_attention(q, cache, bt, lens, window=window, sinks=sinks, **kw)


def test_the_binding_of_logprobs(handle):  # noqa: F811
    D = _OnDevice

    def refused(match, *a, **kw):
        with pytest.raises(ValueError, match=match):
            handle.token_logprobs(*a, **kw)
    x, t = D((4, 100), torch.float32), D((4,), torch.int64)
    refused("logits", D((4, 10, 10), torch.float32), t)
    refused("2.31", D((4, 2 ** 31), torch.float32), t)
    refused("tokens", x, D((4,), torch.int32))
    refused("tokens", x, D((5,), torch.int64))
    refused("tokens", x, None)
    refused("top", x, t, top=101)
    refused("top", x, t, top=-1)
    strided = D((4, 100), torch.float32)
    strided.stride = lambda: (1, 4)
    refused("contiguous", strided, t)
