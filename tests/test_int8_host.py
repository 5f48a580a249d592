"""Refusals of the int8 layer's calls and of the block calls, before anything reaches a GPU."""
import ctypes

import pytest
import torch

D = 128


@pytest.fixture(scope="module")
def layer(tqlib):
    return tqlib.Layer(4, 2, kv_format="int8", device="cpu")


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_layer(tqlib, layer):
    assert layer.page_bytes_k == layer.page_bytes_v == 16 * D + 16
    assert layer.image_bytes(2) == 64 + 2 * 2 * 2 * (16 * D + 16)
    with pytest.raises(ValueError, match="kv_format"):
        tqlib.Layer(4, 2, kv_format="int9", device="cpu")
    desc = tqlib.CacheDesc.from_buffer_copy(layer.desc)
    for name, value in (("bits_k", 4), ("bits_v", 7), ("qjl_k", 1)):
        bad = tqlib.CacheDesc.from_buffer_copy(desc)
        setattr(bad.fmt, name, value)
        assert tqlib.lib().tq_page_bytes(ctypes.byref(bad), 0) == 0


def status(tq, name, *args):
    return getattr(tq.lib(), name)(*args)


@pytest.mark.parametrize("rot", [0, 1, 2])
def test_calls_of_other_layers(tqlib, layer, rot):
    """What an int8 layer does not do is refused, whatever stands in the fields that it does not use."""
    bad = tqlib.CacheDesc.from_buffer_copy(layer.desc)
    bad.fmt.rot_kind = rot
    ref, x = ctypes.byref(bad), torch.zeros(4, 2, D)
    p = ctypes.c_void_p(x.data_ptr())
    heads = tqlib.Heads(x.data_ptr(), x.data_ptr(), 2, 2 * D, D, 2 * D, D)
    rope = tqlib.Rope()
    assert status(tqlib, "tq_rope_append", ref, rope.ref, None, ctypes.byref(heads), None, 0, p, p, 4, None) == tqlib.TQ_ERR_UNSUPPORTED
    assert status(tqlib, "tq_prefix_decode", ref, p, 0, 4, 2, p, 16, None, 0, None, 1.0, p, 0, p, 1 << 20, None) == tqlib.TQ_ERR_UNSUPPORTED
    assert status(tqlib, "tq_decode_step", ref, p, p, 0, p, 0, 4, 2, p, 1, p, 1.0, p, 0, p, 1 << 20, 0, None) == tqlib.TQ_ERR_UNSUPPORTED
    assert status(tqlib, "tq_quantize_rotated", ref, 0, p, p, p, 4, None) == tqlib.TQ_ERR_INVALID_ARG
    assert status(tqlib, "tq_quantize_append", ref, p, None, 0, p, 1 << 28, None) == tqlib.TQ_ERR_UNSUPPORTED


def test_attend_refusals(tqlib, layer):
    x = torch.zeros(4, 2, D)
    p = ctypes.c_void_p(x.data_ptr())

    def call(desc=layer.desc, heads=2, dtype=0, out_dtype=0, n=4, starts=p, batch=1, table=p, width=1, lens=p, scale=1.0, out=x.data_ptr(),
             inp=x.data_ptr()):
        rows = tqlib.Heads(inp, out, heads, 2 * D, D, 2 * D, D)
        return status(tqlib, "tq_attend", ctypes.byref(desc), ctypes.byref(rows), dtype, out_dtype, n, starts, batch, table, width, lens, scale,
                      p, 1 << 20, None)

    other = tqlib.Layer(4, 2, device="cpu")
    assert call(desc=other.desc) == tqlib.TQ_ERR_UNSUPPORTED
    for bad in (dict(heads=3), dict(heads=0), dict(dtype=2), dict(out_dtype=-1), dict(n=-1), dict(batch=-1), dict(starts=None),
                dict(table=None), dict(width=0), dict(lens=None), dict(scale=float("nan")), dict(out=None), dict(inp=None),
                dict(out=x.data_ptr() + 2), dict(inp=x.data_ptr() + 1)):
        assert call(**bad) == tqlib.TQ_ERR_INVALID_ARG, bad
    for big in (dict(n=(1 << 26) + 1), dict(batch=65536), dict(heads=(1 << 16) + 2), dict(n=1 << 20, heads=1 << 12), dict(width=(1 << 26) + 1)):
        assert call(**big) == tqlib.TQ_ERR_UNSUPPORTED, big
    assert call(n=0) == tqlib.TQ_OK and call(batch=0) == tqlib.TQ_OK
    assert tqlib.lib().tq_attend_workspace_bytes(ctypes.byref(other.desc), 4, 1, 2, 1) == 0


@pytest.mark.parametrize("bad", [dict(q=torch.zeros(4, 2, 64)), dict(q=torch.zeros(4, 2 * D)), dict(out=torch.zeros(4, 1, D)),
                                 dict(starts=ints(3)), dict(table=ints(4)), dict(lens=ints(2)), dict(lens=torch.zeros(1, dtype=torch.int64))])
def test_attend_sizes(layer, bad):
    args = dict(q=torch.zeros(4, 2, D), starts=ints(2), table=ints(1, 1), lens=ints(1), out=torch.zeros(4, 2, D))
    args.update(bad)
    with pytest.raises((ValueError, TypeError)):
        layer.attend(args["q"], args["starts"], args["table"], args["lens"], out=args["out"], workspace=torch.zeros(1 << 20, dtype=torch.uint8))


def test_block_refusals(tqlib, layer):
    lib, TQ = tqlib.lib(), tqlib
    from turboquant_quantized_kv_gb300._binding import BlockPool, BlockRows
    buf = torch.zeros(1 << 16, dtype=torch.uint8)
    at = (buf.data_ptr() + 255) // 256 * 256
    size = lib.tq_blocks_workspace_bytes(4, 8)
    assert 0 < size < 1 << 15
    assert lib.tq_blocks_workspace_bytes(0, 1) == 0 and lib.tq_blocks_workspace_bytes(4, -1) == 0
    assert lib.tq_blocks_workspace_bytes((1 << 30) + 1, 1) == 0
    pool = BlockPool(4, at, at + 4096, size)
    rows, other = BlockRows(at, at + 1024, 4, 8), BlockRows(at + 2048, at + 2560, 8, 8)
    descs = (ctypes.POINTER(TQ.CacheDesc) * 2)(ctypes.pointer(layer.desc), ctypes.pointer(layer.desc))
    ref = ctypes.byref
    small = BlockPool(4, at, at + 4096, size - 1)
    assert lib.tq_blocks_extend(ref(small), ref(other), at, None) == TQ.TQ_ERR_WORKSPACE
    for pool2 in (BlockPool(0, at, at + 4096, size), BlockPool(4, None, at + 4096, size), BlockPool(4, at, None, size), BlockPool(4, at, at + 4, size)):
        assert lib.tq_blocks_extend(ref(pool2), ref(rows), at, None) == TQ.TQ_ERR_INVALID_ARG
        assert lib.tq_blocks_release(ref(pool2), ref(rows), None, None) == TQ.TQ_ERR_INVALID_ARG
    for bad in (BlockRows(None, at, 4, 8), BlockRows(at, None, 4, 8), BlockRows(at, at + 1024, -1, 8), BlockRows(at, at + 1024, 4, 0)):
        assert lib.tq_blocks_extend(ref(pool), ref(bad), at, None) == TQ.TQ_ERR_INVALID_ARG
        assert lib.tq_blocks_release(ref(pool), ref(bad), None, None) == TQ.TQ_ERR_INVALID_ARG
        assert lib.tq_blocks_reorder(ref(pool), None, 0, ref(rows), at, ref(bad), None) == TQ.TQ_ERR_INVALID_ARG
        assert lib.tq_blocks_compact(ref(pool), None, 0, ref(bad), 1, None, None, None) == TQ.TQ_ERR_INVALID_ARG
    huge = BlockRows(at, at + 1024, 1 << 16, 1 << 15)
    pool_huge = BlockPool(4, at, at + 4096, lib.tq_blocks_workspace_bytes(4, 1 << 16))
    assert lib.tq_blocks_extend(ref(pool_huge), ref(huge), at, None) == TQ.TQ_ERR_UNSUPPORTED
    assert lib.tq_blocks_reorder(ref(pool_huge), None, 0, ref(huge), at, ref(rows), None) == TQ.TQ_ERR_UNSUPPORTED
    assert lib.tq_blocks_extend(ref(pool), ref(rows), None, None) == TQ.TQ_ERR_INVALID_ARG
    # old and new rows in the same memory, tables of other widths, a cache twice, a layer of another size
    assert lib.tq_blocks_reorder(ref(pool), None, 0, ref(rows), at, ref(rows), None) == TQ.TQ_ERR_INVALID_ARG
    assert lib.tq_blocks_reorder(ref(pool), None, 0, ref(rows), None, ref(other), None) == TQ.TQ_ERR_INVALID_ARG
    assert lib.tq_blocks_reorder(ref(pool), None, 0, ref(rows), at, ref(BlockRows(at + 2048, at + 2560, 8, 7)), None) == TQ.TQ_ERR_INVALID_ARG
    assert lib.tq_blocks_reorder(ref(pool), descs, 2, ref(rows), at, ref(other), None) == TQ.TQ_ERR_INVALID_ARG
    pool5 = BlockPool(5, at, at + 4096, lib.tq_blocks_workspace_bytes(5, 8))
    assert lib.tq_blocks_reorder(ref(pool5), descs, 1, ref(rows), at, ref(other), None) == TQ.TQ_ERR_INVALID_ARG
    assert lib.tq_blocks_compact(ref(pool), descs, -1, ref(rows), 1, None, None, None) == TQ.TQ_ERR_INVALID_ARG
    two = (BlockRows * 2)(rows, rows)
    assert lib.tq_blocks_compact(ref(pool), descs, 1, two, 2, None, None, None) == TQ.TQ_ERR_INVALID_ARG
    assert lib.tq_copy_blocks(descs, 0, at, at, 1, None) == TQ.TQ_ERR_INVALID_ARG
    assert lib.tq_copy_blocks(descs, 2, at, at, 1, None) == TQ.TQ_ERR_INVALID_ARG
    assert lib.tq_copy_blocks(descs, 1, None, at, 1, None) == TQ.TQ_ERR_INVALID_ARG
    assert lib.tq_copy_blocks(descs, 1, at, at, -1, None) == TQ.TQ_ERR_INVALID_ARG
    assert lib.tq_copy_blocks(descs, 1, None, None, 0, None) == TQ.TQ_OK


def test_block_tensors(tqlib):
    blocks = tqlib.Blocks(10, device="cpu")
    for call in (lambda: blocks.extend(ints(2), ints(2), ints(2)), lambda: blocks.extend(ints(2, 3), ints(3), ints(2)),
                 lambda: blocks.extend(ints(2, 3).long(), ints(2), ints(2)), lambda: blocks.reorder([], ints(2, 3), ints(2), ints(2, 1)),
                 lambda: blocks.release(ints(2, 3), ints(2), ints(2)), lambda: blocks.compact([], ints(2, 3), ints(2), ints(2, 3))):
        with pytest.raises((ValueError, TypeError)):
            call()
