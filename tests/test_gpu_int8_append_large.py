"""Appends of more tokens x heads than the small CTAs take (32,768), bit by bit: CTAs of 16, 32 and 64 tokens."""
import numpy as np
import pytest

from tests import _int8_ref as ref
from tests.test_gpu_int8 import BLOCK, assert_pages, blank, data, host, layer_of, orders

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,heads,kind", [(33001, 1, "sequence"), (32769, 1, "time"), (32800, 1, "any"), (16400, 2, "time"),
                                          (16385, 2, "any"), (10950, 3, "sequence"), (10923, 3, "any"), (4097, 8, "time"),
                                          (4113, 8, "sequence")])
def test_append_large(cuda, tqlib, n, heads, kind):
    """One call, slots given twice and skipped ones among them, keys and values."""
    blocks = n // BLOCK + 10
    slots = orders(kind, 5 * n, n, blocks)
    g = np.random.default_rng(n)
    slots[g.integers(0, n, n // 9)] = -1
    slots[n // 2 :: 7] = slots[1 : n - n // 2 + 1 : 7]
    layer, want = layer_of(tqlib, blocks, heads), [blank(blocks, heads), blank(blocks, heads)]
    k, v = data(cuda, n, n, heads), data(cuda, n + 1, n, heads)
    layer.append(k, v, cuda.from_numpy(slots.astype(np.int64)).cuda())
    touched = np.unique(slots[slots >= 0] // BLOCK)
    for w, x in ((0, k), (1, v)):
        ref.append(*want[w], host(x), slots)
        assert_pages(layer, want[w], w, touched)
    assert tqlib.get_device_status() == 0


def test_append_large_twice(cuda, tqlib):
    """A second large call into blocks that the first left partly filled, fp32, larger values: codes are rounded again."""
    n, heads = 34000, 1
    blocks = n // BLOCK + 10
    slots = orders("time", 1, n, blocks)
    layer, want = layer_of(tqlib, blocks, heads), blank(blocks, heads)
    first = np.arange(n) % 40 < 1  # (a small one)
    for part, grow in ((first, 1.0), (~first, 1.7)):
        k = data(cuda, 3, int(part.sum()), heads, "f32") * grow
        layer.append(k, None, cuda.from_numpy(slots[part].astype(np.int64)).cuda())
        ref.append(*want, host(k), slots[part])
    assert_pages(layer, want, 0, np.unique(slots // BLOCK))
    assert tqlib.get_device_status() == 0
