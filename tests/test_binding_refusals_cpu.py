"""Arguments that a binding call needs and was not given are refused as ValueError, like every other wrong one.  No GPU:
the checks run before anything is read from the device."""
import pytest

import bit_weight_quantized_dequant_gb300 as lq

torch = pytest.importorskip("torch")


class _OnDevice:
    """What the checks look at of a tensor on cuda:0."""

    requires_grad = False

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, "cuda:0"

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def stride(self):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s)


@pytest.fixture()
def handle():
    h = lq.Handle.__new__(lq.Handle)
    h.device, h._device, h._lib, h._h = 0, "cuda:0", None, None
    return h


def test_a_table_without_positions(handle):
    class Cache:
        head_dim, kv_heads = 64, 2
    k, slots, table = _OnDevice((3, 2, 64), torch.float16), _OnDevice((3,), torch.int64), _OnDevice((9, 64), torch.float32)
    with pytest.raises(ValueError, match="positions"):
        handle.kv_append(Cache(), k, k, slots, table=table)
    with pytest.raises(ValueError, match="positions"):
        handle.rope(k, None, table, out=k)
    with pytest.raises(ValueError, match="slots"):
        handle.kv_append(Cache(), k, k, None)


def test_sizes_past_31_bits(handle):
    """Numbers that the C boundary would cut to 32 bits: 2^32 + 5 rows are not 5."""
    for first, count in ((2 ** 32 + 5, 4), (0, 2 ** 32 + 4), (5 - 2 ** 32, 4), (2 ** 31, 4)):
        with pytest.raises(ValueError, match="2.31"):
            handle.rope_table(count, 2, first=first, out=_OnDevice((count, 2), torch.float32))
    table = _OnDevice((9, 2), torch.float32)
    for shape in ((2 ** 32 + 5, 1, 2), (1, 2 ** 32 + 5, 2), (1, 1, 2 ** 32 + 6)):
        x = _OnDevice(shape, torch.float16)
        with pytest.raises(ValueError, match="2.31"):
            handle.rope(x, _OnDevice((shape[0],), torch.int32), table, out=x)
