"""The split count that tq_auto_splits names for int8 layers is the one that the automatic choice uses."""
import ctypes

import numpy as np
import pytest

from tests.test_gpu_int8_long import D, layer_with

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,heads,group,ctx", [(1, 1, 4, 30000), (163, 8, 4, 700), (70, 8, 17, 100), (2, 2, 8, 20), (300, 8, 1, 333)])
def test_auto_splits(cuda, tqlib, batch, heads, group, ctx):
    g = np.random.default_rng(batch)
    layer = layer_with(cuda, tqlib, *g.standard_normal((2, 40 * 16, heads, D)))
    width, hq = -(-ctx // 16), heads * group
    table = cuda.from_numpy(g.integers(0, 40, (batch, width)).astype(np.int32)).cuda()
    lens = cuda.full((batch,), ctx, dtype=cuda.int32, device="cuda")
    q = cuda.randn(batch, hq, D, device="cuda")
    splits = tqlib.lib().tq_auto_splits(ctypes.byref(layer.desc), batch, hq, width)
    assert 1 <= splits <= width
    assert cuda.equal(layer.decode(q, table, lens, num_splits=splits), layer.decode(q, table, lens))
    assert tqlib.get_device_status() == 0


def test_no_heads(tqlib):
    layer = tqlib.Layer(4, 2, kv_format="int8")
    assert tqlib.lib().tq_auto_splits(ctypes.byref(layer.desc), 3, 1, 4) == 1  # (fewer query heads than KV heads)
