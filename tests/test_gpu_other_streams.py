"""Calls on another stream than the current one: a result made by the call lies in that stream's memory, not in a
block that the current stream has freed and may still be reading."""
import pytest

from tests import _kv_ref as R
from tests.test_gpu_kv_attention import Case, handle, lqm  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _fresh(shape, dtype):
    """The address that the current stream's allocator would hand out next for such a tensor."""
    torch.cuda.synchronize()
    t = torch.empty(shape, dtype=dtype, device="cuda")
    at = t.data_ptr()
    del t
    return at


def _calls(lqm, h):  # noqa: F811
    x = torch.randn(700, 16, 128, device="cuda").bfloat16()
    table = h.rope_table(900, 128)
    pos = torch.arange(700, dtype=torch.int32, device="cuda")
    cache = lqm.KVCache(num_pages=20, page_size=64, kv_heads=4, head_dim=128, bits=4)
    kv, slots = x[:, :4].contiguous(), torch.arange(700, device="cuda")
    c = Case(lqm, [300] * 40, hq=64, hkv=4, seed=1)
    return {
        "rope_table": ((5000, 128), torch.float32, lambda s: [h.rope_table(5000, 128, stream=s)]),
        "rope": (x.shape, x.dtype, lambda s: [h.rope(x, pos, table, stream=s)]),
        "kv_append": (x.shape, x.dtype, lambda s: [h.kv_append(cache, kv, kv, slots, q=x, table=table, positions=pos, stream=s)]),
        "kv_read": (kv.shape, kv.dtype, lambda s: list(h.kv_read(cache, slots, stream=s))),
        "kv_attention": (c.q.shape, c.q.dtype, lambda s: list(c.run(h, stream=s))),
    }


@pytest.mark.parametrize("name", ["rope_table", "rope", "kv_append", "kv_read", "kv_attention"])
def test_results_do_not_lie_in_the_current_streams_blocks(lqm, handle, name):  # noqa: F811
    shape, dtype, call = _calls(lqm, handle)[name]
    want = call(None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    at = _fresh(shape, dtype)
    got = call(s)
    assert all(t.data_ptr() != at for t in got)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # freed, it is not handed to `s` again while the current stream may still read it
    torch.cuda.synchronize()
    del got
    handle.sync()


def test_a_block_that_the_current_stream_still_reads(lqm, handle):  # noqa: F811
    """The current stream is busy with a long copy out of a tensor that is freed at once; a call on another stream, which
    waits only for its inputs, leaves that copy alone."""
    x = torch.randn(4096, 32, 128, device="cuda").bfloat16()
    table = handle.rope_table(4096, 128)
    pos = torch.arange(4096, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    src = torch.full(x.shape, 3.0, dtype=x.dtype, device="cuda")
    dst = [torch.zeros_like(src) for _ in range(20)]
    torch.cuda.synchronize()
    for d in dst:
        d.copy_(src)
    del src
    got = handle.rope(x, pos, table, stream=s)
    torch.cuda.synchronize()
    assert all(bool((d == 3).all()) for d in dst)
    ref = R.rotate(x[:64].float().cpu().numpy(), table.cpu().numpy(), pos[:64].cpu().numpy(), 0)
    assert torch.equal(got[:64].cpu(), torch.from_numpy(ref).bfloat16())
