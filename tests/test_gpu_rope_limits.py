"""lq_rope at the ends of its sizes."""
import pytest

from tests.test_gpu_kv_attention import handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_a_head_of_almost_2_to_the_31_dimensions(handle):  # noqa: F811
    """The largest row that is taken (4.3 GB): a thread's next index after its last stays above all of them."""
    D = 0x7fffff00
    x = torch.empty((1, 1, D), dtype=torch.float16, device="cuda").fill_(0.5)
    x[0, 0, :4] = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda")
    x[0, 0, -3:] = torch.tensor([5.0, 6.0, 7.0], device="cuda")
    table = torch.tensor([[0.0, 1.0]], device="cuda")            # a quarter turn
    y = handle.rope(x, torch.zeros(1, dtype=torch.int32, device="cuda"), table)
    handle.sync()
    assert y[0, 0, :4].tolist() == [-2.0, 1.0, 3.0, 4.0]
    step = 1 << 28
    assert all(torch.equal(y[..., a:a + step], x[..., a:a + step]) for a in range(2, D, step))


@pytest.mark.parametrize("heads,D", [(65536, 16), (100000, 16), (140003, 16), (70001, 8), (300000, 32)])
@pytest.mark.parametrize("n", [1, 3])
def test_many_narrow_heads(handle, heads, D, n):  # noqa: F811
    """More chunks of heads than a grid has rows."""
    g = torch.Generator(device="cuda").manual_seed(heads)
    x = torch.randn(n, heads, D, generator=g, device="cuda").half()
    table, pos = handle.rope_table(50, D), torch.arange(n, dtype=torch.int32, device="cuda")
    y = handle.rope(x, pos, table)
    handle.sync()
    for a in range(0, heads, 1000):              # the same heads a few at a time
        assert torch.equal(y[:, a:a + 1000], handle.rope(x[:, a:a + 1000], pos, table))
