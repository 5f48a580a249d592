"""GPU: calls that are given a stream take the memory of their results and workspaces from that stream, so
that nothing which other streams have yet to do with it is disturbed."""
import pytest

from tests._gpu_util import D

pytestmark = pytest.mark.gpu


def calls(cuda, tq):
    """(elements of the result in bf16, call) on inputs that are ready."""
    n, hq, hkv = 512, 16, 4
    rope = tq.Rope()
    layer = tq.Layer(n // 16, hkv)
    q, k = cuda.randn(n, hq, D, device="cuda").bfloat16(), cuda.randn(n, hkv, D, device="cuda").bfloat16()
    at = cuda.arange(n, device="cuda")
    layer.append(k, k, at)
    blocks = cuda.arange(n // 16, dtype=cuda.int32, device="cuda")
    lens = cuda.ones(n, dtype=cuda.int32, device="cuda")
    size = n * hq * D
    return [(size, lambda s: tq.apply_rope(rope, at, q, stream=s)[0]),
            (size, lambda s: layer.rope_append(rope, k, k, at, at, q=q, stream=s)),
            (size, lambda s: layer.prefix_decode(q, blocks, n, stream=s)),
            (size, lambda s: layer.decode(q, blocks.view(n // 16, 1).repeat(16, 1), lens, stream=s)),
            (n * hkv * D, lambda s: layer.dequantize(0, at, out_dtype=cuda.bfloat16, stream=s))]


@pytest.mark.parametrize("which", range(5))
def test_results_do_not_take_memory_that_is_still_read(cuda, tqlib, which):
    size, call = calls(cuda, tqlib)[which]
    side = cuda.cuda.Stream()
    want = call(side)
    x, copy = cuda.randn(size, device="cuda").bfloat16(), cuda.empty(size, dtype=cuda.bfloat16, device="cuda")
    keep = x.cpu()
    cuda.cuda.synchronize()
    cuda.cuda._sleep(200_000_000)  # (about a tenth of a second: the copy of x comes after it)
    copy.copy_(x)
    del x
    got = call(side)  # on the side stream, at once
    side.synchronize()
    cuda.cuda.synchronize()
    assert cuda.equal(got, want)
    assert cuda.equal(copy.cpu(), keep)
    assert tqlib.get_device_status() == 0
