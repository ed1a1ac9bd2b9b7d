"""Host-side refusals at the ends of 32-bit sizes, which the kernels' token counts (rounded up to tiles) must not pass.
No GPU: every call fails before the handle is read."""
import ctypes

import pytest

import bit_weight_quantized_dequant_gb300 as lq
from bit_weight_quantized_dequant_gb300 import _lq

H, A16 = ctypes.c_void_p(0x1000), 0x10000


@pytest.fixture(scope="module")
def L():
    lq.build()
    return _lq.load_library(build_if_missing=False)


@pytest.mark.parametrize("prefix_len", [0x7fffff01, 2 ** 31 - 16, 2 ** 31 - 15, 2 ** 31 - 1])
def test_prefix_of_almost_2_to_the_31_tokens(L, prefix_len):
    c = _lq.lq_kv_cache(A16, 10, 64, 8, 128, 4)
    a = _lq.lq_kv_attention_args(A16, A16, A16, 2, 3, 2, 32, 4096, 4096, A16, 5, 5, A16, A16, prefix_len, 0.1)
    a.q = A16 + 8       # (misaligned: what a call that gets past the sizes is refused for)
    assert L.lq_kv_attention(H, ctypes.byref(c), ctypes.byref(a), None) == _lq.LQ_ERR_UNSUPPORTED
    a.prefix_len = 0x7fffff00
    assert L.lq_kv_attention(H, ctypes.byref(c), ctypes.byref(a), None) == _lq.LQ_ERR_ALIGNMENT


@pytest.mark.parametrize("scale", [2.4e38, 2.9e38])
def test_scale_whose_base_2_form_is_infinite(L, scale):
    c = _lq.lq_kv_cache(A16, 10, 64, 8, 128, 4)
    a = _lq.lq_kv_attention_args(A16 + 8, A16, A16, 2, 3, 2, 32, 4096, 4096, A16, 5, 5, A16, A16, 100, scale)
    assert L.lq_kv_attention(H, ctypes.byref(c), ctypes.byref(a), None) == _lq.LQ_ERR_INVALID_ARG
    a.scale = 2.3e38
    assert L.lq_kv_attention(H, ctypes.byref(c), ctypes.byref(a), None) == _lq.LQ_ERR_ALIGNMENT
