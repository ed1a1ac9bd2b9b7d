"""Handle.rope of a tensor that requires a gradient: the gradient arrives, and is the transpose, bit for bit."""
import pytest

from tests.test_gpu_kv_attention import handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _case(dtype, n=37, heads=6, D=64, rot=32, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, D, generator=g).to(dtype).cuda()
    u = torch.randn(n, heads, D, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 90, (n,), generator=g, dtype=torch.int32).cuda()
    return x, u, pos, rot


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradient_is_the_transpose(handle, dtype, layout, inverse):  # noqa: F811
    x, u, pos, rot = _case(dtype)
    table = handle.rope_table(90, rot)
    want = handle.rope(x, pos, table, layout=layout, inverse=inverse)
    x.requires_grad_()
    y = handle.rope(x, pos, table, layout=layout, inverse=inverse)
    assert y.requires_grad and torch.equal(y, want)
    y.backward(u)
    assert torch.equal(x.grad, handle.rope(u, pos, table, layout=layout, inverse=not inverse))
    with torch.no_grad():
        assert not handle.rope(x, pos, table, layout=layout, inverse=inverse).requires_grad
    handle.sync()


def test_inside_a_graph_of_operations(handle):  # noqa: F811
    """q rotated out of a fused projection, a sum whose gradient is expanded, and differences: the loss is linear in x
    up to fp32 roundings (3 per output of 2^-24, and the sum's own, below 2^-16 of the terms together)."""
    x, u, pos, rot = _case(torch.float32, n=5, heads=4)
    table = handle.rope_table(90, rot)
    wide = torch.cat([x, x], 1).requires_grad_()
    loss = lambda w: (handle.rope(w[:, 4:], pos, table) * u).double().sum()  # noqa: E731
    loss(wide).backward()
    assert not bool(wide.grad[:, :4].any())
    for i in (0, 17, 40, 63):
        step = torch.zeros_like(x)
        step[3, 2, i] = 1.0
        diff = (loss(torch.cat([x, x + step], 1)) - loss(torch.cat([x, x - step], 1))) / 2
        scale = 2 * ((x.abs() + 1) * u.abs()).double().sum()
        assert abs(diff - wide.grad[3, 6, i]) <= 2.0 ** -16 * scale
    x.requires_grad_()
    handle.rope(x, pos, table).sum().backward()             # (a gradient of ones without strides)
    assert torch.equal(x.grad, handle.rope(torch.ones_like(x), pos, table, inverse=True))


def test_out_and_gradient_exclude_each_other(handle):  # noqa: F811
    x, _, pos, rot = _case(torch.float32)
    table = handle.rope_table(90, rot)
    x.requires_grad_()
    with pytest.raises(ValueError):
        handle.rope(x, pos, table, out=torch.empty_like(x))
    with torch.no_grad():
        handle.rope(x, pos, table, out=torch.empty_like(x))
