"""Block calls that run out of blocks, of many rows, of many layers and tables, against plain loops."""
import numpy as np
import pytest

from tests.test_gpu_blocks import BLOCK, FORMATS, Model, check, dev, host_pages, layers_of

pytestmark = pytest.mark.gpu


def test_short(cuda, tqlib):
    """Calls that take the last block, and calls that lack one or two: -1 in the entries that got none, and the bit for it."""
    num_blocks, none = 11, tqlib.TQ_DEV_NO_BLOCK
    layers = layers_of(cuda, tqlib, num_blocks, 1, FORMATS[:2])
    model, blocks = Model(num_blocks, host_pages(layers, num_blocks)), tqlib.Blocks(num_blocks)
    table, lens = np.full((3, 6), -1, np.int32), np.zeros(3, np.int32)
    t = dev(cuda, table)

    def extend(new, status):
        nonlocal lens
        blocks.extend(t, dev(cuda, lens), dev(cuda, new))
        model.extend(table, lens, new)
        assert np.array_equal(t.cpu().numpy(), table)
        assert np.array_equal(blocks.refs.cpu().numpy(), model.refs)
        assert tqlib.get_device_status() == status
        lens = new

    extend(np.array([20, 33, 5], np.int32), 0)
    extend(np.array([40, 60, 50], np.int32), 0)  # eleven blocks: all there are
    assert (model.refs == 1).all() and (table[:, 3:] == [[-1, -1, -1], [table[1, 3], -1, -1], [table[2, 3], -1, -1]]).all()
    keep = table.copy(), lens.copy()
    extend(np.array([40, 65, 50], np.int32), none)
    assert table[1, 4] == -1
    table[:], lens = keep
    t = dev(cuda, table)

    def reorder(parents, status):
        nonlocal table, lens, t
        parents = np.array(parents, np.int32)
        t, n = blocks.reorder(layers, t, dev(cuda, lens), dev(cuda, parents))
        table, lens = model.reorder(table, lens, parents)
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(n.cpu().numpy(), lens)
        check(cuda, blocks, layers, model)
        assert tqlib.get_device_status() == status

    reorder([0, 1, 1], 0)  # the third row's four blocks are given up, the second's last is copied
    assert (model.refs <= 0).sum() == 3
    reorder([0, 0, 1, 1, 2], 0)  # two copies
    assert (model.refs <= 0).sum() == 1
    reorder([0, 2, 0, 4, 3, 0, 1], none)  # two copies of row 0's last block, one block
    assert (model.refs > 0).all() and table[5, 2] == -1 and table[2, 2] >= 0
    reorder([5, 1, 5], tqlib.TQ_DEV_BAD_BLOCK)  # (an entry that got no block is left as it is, and recorded)


@pytest.mark.parametrize("old,new", [(4097, 300), (300, 4100), (5000, 5000), (4096, 4096)])
def test_many_rows(cuda, tqlib, old, new):
    """More rows than one CTA holds: children are counted by a kernel of their own from 4097 rows on, old or new."""
    num_blocks, width = 30011, 3
    g = np.random.default_rng(old + new)
    layers = layers_of(cuda, tqlib, num_blocks, 1, [dict(bits_k=2, bits_v=2)])
    model, blocks = Model(num_blocks, host_pages(layers, num_blocks)), tqlib.Blocks(num_blocks)
    table, lens = np.full((old, width), -1, np.int32), g.integers(0, width * BLOCK + 1, old).astype(np.int32)
    t, zero = dev(cuda, table), np.zeros(old, np.int32)
    blocks.extend(t, dev(cuda, zero), dev(cuda, lens))
    model.extend(table, zero, lens)
    parents = g.integers(-1, old, new).astype(np.int32)
    parents[:: 50] = parents[0]
    n, nl = blocks.reorder(layers, t, dev(cuda, lens), dev(cuda, parents))
    mt, ml = model.reorder(table, lens, parents)
    assert np.array_equal(n.cpu().numpy(), mt) and np.array_equal(nl.cpu().numpy(), ml)
    check(cuda, blocks, layers, model)
    which = g.random(new) < 0.5
    blocks.release(n, nl, dev(cuda, which))
    model.release(mt, ml, which)
    grown = np.minimum(ml + g.integers(0, 30, new), width * BLOCK).astype(np.int32)
    blocks.extend(n, nl, dev(cuda, grown))
    model.extend(mt, ml, grown)
    assert np.array_equal(n.cpu().numpy(), mt)
    live = blocks.compact(layers, n, dev(cuda, grown))
    assert int(live) == model.compact([(mt, grown)])[0] and np.array_equal(n.cpu().numpy(), mt)
    check(cuda, blocks, layers, model)
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("layers_n,tables_n", [(70, 9), (3, 17), (130, 1), (64, 8), (0, 9)])
def test_many_layers(cuda, tqlib, layers_n, tables_n):
    """More layers than a launch moves (64) and more tables (8), in one reordering and one compaction."""
    num_blocks, width = 200, 4
    g = np.random.default_rng(layers_n)
    layers = layers_of(cuda, tqlib, num_blocks, 1, [FORMATS[i % 4] for i in range(layers_n)])
    model, blocks = Model(num_blocks, host_pages(layers, num_blocks)), tqlib.Blocks(num_blocks)
    host, on_gpu = [], []
    for k in range(tables_n):
        table, lens = np.full((3, width), -1, np.int32), g.integers(1, width * BLOCK, 3).astype(np.int32)
        t, zero = dev(cuda, table), np.zeros(3, np.int32)
        blocks.extend(t, dev(cuda, zero), dev(cuda, lens))
        model.extend(table, zero, lens)
        host.append((table, lens))
        on_gpu.append((t, dev(cuda, lens)))
    parents = np.array([1, 1, 1, 0], np.int32)  # the last row's blocks are given up: holes
    on_gpu[0] = blocks.reorder(layers, *on_gpu[0], dev(cuda, parents))
    host[0] = model.reorder(*host[0], parents)
    check(cuda, blocks, layers, model)
    for (t, n), (table, lens) in list(zip(on_gpu, host))[1::2]:
        blocks.release(t, n, dev(cuda, np.array([True, False, True])))
        model.release(table, lens, [1, 0, 1])
    live = blocks.compact(layers, *[x for pair in on_gpu for x in pair])
    assert int(live) == model.compact(host)[0]
    for (t, n), (table, lens) in zip(on_gpu, host):
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(n.cpu().numpy(), lens)
    check(cuda, blocks, layers, model)
    assert tqlib.get_device_status() == 0
