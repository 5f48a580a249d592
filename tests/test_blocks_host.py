"""Refusals and workspaces of the block calls, before anything reaches a GPU."""
import ctypes

import torch


def test_pairs_bounded(tqlib):
    """Every pair is held against all others: lists that would take seconds are refused."""
    layer = tqlib.Layer(4, 2, kv_format="int8", device="cpu")
    descs = (ctypes.POINTER(tqlib.CacheDesc) * 1)(ctypes.pointer(layer.desc))
    ids = torch.zeros(16, dtype=torch.int32)
    for n in ((1 << 16) + 1, 10 ** 6, 1 << 40):
        assert tqlib.lib().tq_copy_blocks(descs, 1, ids.data_ptr(), ids.data_ptr(), n, None) == tqlib.TQ_ERR_UNSUPPORTED
    assert "65536" in tqlib.last_error()
