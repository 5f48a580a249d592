"""Workspaces of the block calls: what an object and the graphs that captured its calls keep."""
import numpy as np
import pytest

from tests.test_gpu_blocks import BLOCK, Model, dev

pytestmark = pytest.mark.gpu


def test_captured_calls_share(cuda, tqlib):
    """Twelve steps captured in one graph, of an object without a workspace: their workspaces (11.5 MB each) follow one another
    in the graph's memory, and every replay gives the steps' results."""
    num_blocks, rows, width = 1 << 20, 6, 8
    g = np.random.default_rng(0)
    blocks = tqlib.Blocks(num_blocks)
    size = tqlib.lib().tq_blocks_workspace_bytes(num_blocks, 1024)
    lens = g.integers(1, 40, rows).astype(np.int32)
    table, model = np.full((rows, width), -1, np.int32), Model(num_blocks, [])
    model.extend(table, np.zeros(rows, np.int32), lens)
    d = dict(t=dev(cuda, table), lens=dev(cuda, lens), refs=dev(cuda, model.refs))
    parents = [g.integers(0, rows, rows).astype(np.int32) for _ in range(12)]
    on_gpu = [dev(cuda, p) for p in parents]
    cuda.cuda.synchronize()
    before = cuda.cuda.memory_reserved()
    graph = cuda.cuda.CUDAGraph()
    with cuda.cuda.graph(graph):
        blocks.refs.copy_(d["refs"])
        t, n = d["t"], d["lens"]
        for p in on_gpu:
            t, n = blocks.reorder([], t, n, p)
            blocks.extend(t, n, n + 3)
            n = n + 3
    assert cuda.cuda.memory_reserved() - before < 4 * size
    for p in parents:
        table, lens = model.reorder(table, lens, p)
        model.extend(table, lens, lens + 3)
        lens = lens + 3
    for _ in range(2):
        graph.replay()
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(n.cpu().numpy(), lens)
        assert np.array_equal(blocks.refs.cpu().numpy(), model.refs)
    assert tqlib.get_device_status() == 0


def test_growing_calls(cuda, tqlib):
    """Calls of ever more rows do not leave a workspace each."""
    num_blocks = 1 << 18
    blocks = tqlib.Blocks(num_blocks)
    size = tqlib.lib().tq_blocks_workspace_bytes(num_blocks, 1024)
    cuda.cuda.synchronize()
    before = cuda.cuda.memory_allocated()
    for rows in range(1, 60):
        t, n = cuda.full((rows, 1), -1, dtype=cuda.int32, device="cuda"), cuda.zeros(rows, dtype=cuda.int32, device="cuda")
        blocks.extend(t, n, n + BLOCK)
    assert np.array_equal(t.cpu().numpy()[:, 0], np.arange(rows) + rows * (rows - 1) // 2)
    assert cuda.cuda.memory_allocated() - before < 2 * size
    assert tqlib.get_device_status() == 0
