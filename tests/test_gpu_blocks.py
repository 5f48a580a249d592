"""Blocks that sequences share: copies, forks, extension, release and compaction against plain loops."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
BLOCK = 16


class Model:
    """The same calls in plain Python on host arrays; pages[p] [num_blocks, bytes]."""

    def __init__(self, num_blocks, pages):
        self.refs, self.pages = np.zeros(num_blocks, np.int32), pages

    def take(self, count):
        free = [int(i) for i in np.nonzero(self.refs <= 0)[0][:count]]
        self.refs[free] = 1
        return free + [-1] * (count - len(free))

    def valid(self, i):
        return 0 <= i < self.refs.size

    def extend(self, table, lens, new):
        spots = [(b, j) for b in range(len(lens)) for j in range(-(-lens[b] // BLOCK), -(-new[b] // BLOCK))]
        for (b, j), i in zip(spots, self.take(len(spots))):
            table[b, j] = i

    def release(self, table, lens, which):
        for b in np.nonzero(which)[0]:
            for j in range(-(-lens[b] // BLOCK)):
                if self.valid(table[b, j]):
                    self.refs[table[b, j]] -= 1
                table[b, j] = -1
            lens[b] = 0

    def reorder(self, table, lens, parents):
        n, width = table.shape
        new, out = np.full((len(parents), width), -1, np.int32), np.zeros(len(parents), np.int32)
        for b in range(n):
            for j in range(-(-lens[b] // BLOCK)):
                if self.valid(table[b, j]):
                    self.refs[table[b, j]] -= 1
        seen, copies = set(), []
        for i, p in enumerate(parents):
            if not 0 <= p < n:
                continue
            out[i] = lens[p]
            used = -(-lens[p] // BLOCK)
            new[i, :used] = table[p, :used]
            if p in seen and lens[p] % BLOCK and self.valid(table[p, used - 1]):
                copies.append((i, used - 1, int(table[p, used - 1])))
                new[i, used - 1] = -1
            seen.add(p)
            for j in range(used):
                if self.valid(new[i, j]):
                    self.refs[new[i, j]] += 1
        for (i, j, src), dst in zip(copies, self.take(len(copies))):
            new[i, j] = dst
            if dst >= 0:
                for p in self.pages:
                    p[dst] = p[src]
        return new, out

    def compact(self, tables):
        live = int((self.refs > 0).sum())
        holes = [i for i in range(live) if self.refs[i] <= 0]
        movers = [i for i in range(live, self.refs.size) if self.refs[i] > 0]
        to = np.arange(self.refs.size, dtype=np.int32)
        for d, s in zip(holes, movers):
            to[s] = d
            self.refs[d], self.refs[s] = self.refs[s], 0
            for p in self.pages:
                p[d] = p[s]
        for table, lens in tables:
            for b in range(len(lens)):
                for j in range(-(-lens[b] // BLOCK)):
                    if self.valid(table[b, j]):
                        table[b, j] = to[table[b, j]]
        return live, to


FORMATS = [dict(bits_k=4, bits_v=4), dict(kv_format="int8"), dict(bits_k=2, bits_v=3, qjl=True), dict(kv_format="bf16")]


def layers_of(cuda, tq, blocks, heads, formats, seed=0):
    g = cuda.Generator(device="cuda").manual_seed(seed)
    out = [tq.Layer(blocks, heads, layer=i, **f) for i, f in enumerate(formats)]
    for ly in out:
        for pool in (ly.k_cache, ly.v_cache):
            pool.copy_(cuda.randint(0, 256, pool.shape, generator=g, dtype=cuda.uint8, device="cuda"))
    return out


def host_pages(layers, blocks):
    return [pool.cpu().numpy().reshape(blocks, -1).copy() for ly in layers for pool in (ly.k_cache, ly.v_cache)]


def dev(cuda, x):
    return cuda.from_numpy(np.ascontiguousarray(x)).cuda()


def check(cuda, blocks, layers, model):
    assert np.array_equal(blocks.refs.cpu().numpy(), model.refs)
    for got, want in zip(host_pages(layers, blocks.num_blocks), model.pages):
        assert np.array_equal(got, want)


def start(cuda, tq, seed, rows, width, num_blocks, formats, heads=2, lens=None):
    g = np.random.default_rng(seed)
    layers = layers_of(cuda, tq, num_blocks, heads, formats, seed)
    model, blocks = Model(num_blocks, host_pages(layers, num_blocks)), tq.Blocks(num_blocks)
    # some blocks are somebody else's
    other = g.random(num_blocks) < 0.3
    model.refs[other] = 1
    blocks.refs.copy_(dev(cuda, model.refs))
    table = np.full((rows, width), -1, np.int32)
    new = g.integers(0, width * BLOCK + 1, rows).astype(np.int32) if lens is None else np.array(lens, np.int32)
    t, zero = dev(cuda, table), np.zeros(rows, np.int32)
    blocks.extend(t, dev(cuda, zero), dev(cuda, new))
    model.extend(table, zero, new)
    assert np.array_equal(t.cpu().numpy(), table)
    return g, layers, model, blocks, table, new, t


@pytest.mark.parametrize("rows,width,num_blocks,children", [(1, 1, 5, 1), (1, 3, 40, 7), (9, 5, 200, 9), (33, 17, 3000, 70),
                                                            (1500, 3, 12000, 2100), (6, 600, 9001, 4)])
def test_steps(cuda, tqlib, rows, width, num_blocks, children):
    """Extension, forks, appended room, release, compaction, in a row."""
    formats = FORMATS[:1] if num_blocks > 5000 else FORMATS
    g, layers, model, blocks, table, lens, t = start(cuda, tqlib, rows, rows, width, num_blocks, formats)
    parents = g.integers(-1, rows, children).astype(np.int32)
    n, nl = blocks.reorder(layers, t, dev(cuda, lens), dev(cuda, parents))
    mt, ml = model.reorder(table, lens, parents)
    assert np.array_equal(n.cpu().numpy(), mt) and np.array_equal(nl.cpu().numpy(), ml)
    check(cuda, blocks, layers, model)
    grown = np.minimum(ml + g.integers(0, 40, children), width * BLOCK).astype(np.int32)
    blocks.extend(n, nl, dev(cuda, grown))
    model.extend(mt, ml, grown)
    assert np.array_equal(n.cpu().numpy(), mt)
    nl = dev(cuda, grown)
    which = g.random(children) < 0.5
    blocks.release(n, nl, dev(cuda, which))
    model.release(mt, grown, which)
    assert np.array_equal(n.cpu().numpy(), mt) and np.array_equal(nl.cpu().numpy(), grown)
    check(cuda, blocks, layers, model)
    moved = cuda.empty(num_blocks, dtype=cuda.int32, device="cuda")
    live = blocks.compact(layers, n, nl, moved=moved)
    want, to = model.compact([(mt, grown)])
    assert int(live) == want and np.array_equal(moved.cpu().numpy(), to) and np.array_equal(n.cpu().numpy(), mt)
    check(cuda, blocks, layers, model)
    blocks.release(n, nl)
    model.release(mt, grown, np.ones(children, bool))
    check(cuda, blocks, layers, model)
    assert not nl.any() and tqlib.get_device_status() == 0


def test_no_blocks_left(cuda, tqlib):
    g, layers, model, blocks, table, lens, t = start(cuda, tqlib, 3, 4, 4, 24, FORMATS[:1], lens=[20, 33, 16, 5])
    for _ in range(2):
        new = np.minimum(lens + 30, 64).astype(np.int32)
        blocks.extend(t, dev(cuda, lens), dev(cuda, new))
        model.extend(table, lens, new)
        assert np.array_equal(t.cpu().numpy(), table)
        status = tqlib.get_device_status()
        assert status == (tqlib.TQ_DEV_NO_BLOCK if (table[:, :2] == -1).any() or (model.refs > 0).all() and -1 in table[1, :4] else status)
        lens = new
    assert (model.refs > 0).all() and np.array_equal(blocks.refs.cpu().numpy(), model.refs)
    parents = np.array([0, 0, 0, 1], np.int32)
    lens = np.array([20, 33, 16, 5], np.int32)
    n, nl = blocks.reorder(layers, t, dev(cuda, lens), dev(cuda, parents))
    mt, ml = model.reorder(table, lens, parents)
    assert np.array_equal(n.cpu().numpy(), mt) and np.array_equal(nl.cpu().numpy(), ml)
    check(cuda, blocks, layers, model)
    tqlib.get_device_status()


def test_bad_entries(cuda, tqlib):
    g, layers, model, blocks, table, lens, t = start(cuda, tqlib, 5, 5, 4, 60, FORMATS[:2], lens=[20, 33, 16, 64, 0])
    table[0, 1], table[3, 0] = 60, -7
    t = dev(cuda, table)
    parents = np.array([0, 0, 3, 9, -2, -1, 4], np.int32)
    n, nl = blocks.reorder(layers, t, dev(cuda, lens), dev(cuda, parents))
    mt, ml = model.reorder(table, lens, parents)
    assert np.array_equal(n.cpu().numpy(), mt) and np.array_equal(nl.cpu().numpy(), ml)
    check(cuda, blocks, layers, model)
    assert tqlib.get_device_status() == tqlib.TQ_DEV_BAD_BLOCK | tqlib.TQ_DEV_BAD_ROW
    live = blocks.compact(layers, n, nl)
    assert int(live) == model.compact([(mt, ml)])[0] and np.array_equal(n.cpu().numpy(), mt)
    assert tqlib.get_device_status() == tqlib.TQ_DEV_BAD_BLOCK
    # lengths outside a row
    bad = np.array([-3, 1000, 0, 0, 0, 0, 0], np.int32)
    blocks.extend(n, nl, dev(cuda, bad))
    model.extend(mt, ml, np.clip(bad, 0, 64))
    assert np.array_equal(n.cpu().numpy(), mt)
    assert tqlib.get_device_status() == tqlib.TQ_DEV_BAD_CONTEXT
    check(cuda, blocks, layers, model)


def test_two_tables_compacted(cuda, tqlib):
    g, layers, model, blocks, table, lens, t = start(cuda, tqlib, 8, 6, 5, 100, FORMATS[:1])
    prefix, plen = np.full((1, 3), -1, np.int32), np.array([48], np.int32)
    p, zero = dev(cuda, prefix), np.zeros(1, np.int32)
    blocks.extend(p, dev(cuda, zero), dev(cuda, plen))
    model.extend(prefix, zero, plen)
    blocks.release(t, dev(cuda, lens), dev(cuda, np.array([True, False, True, False, False, True])))
    model.release(table, lens.copy(), [1, 0, 1, 0, 0, 1])
    lens[[0, 2, 5]] = 0
    live = blocks.compact(layers, t, dev(cuda, lens), p, dev(cuda, plen))
    assert int(live) == model.compact([(table, lens), (prefix, plen)])[0]
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(p.cpu().numpy(), prefix)
    check(cuda, blocks, layers, model)


@pytest.mark.parametrize("layers_n,heads", [(1, 1), (5, 3), (70, 1)])
def test_copy_blocks(cuda, tqlib, layers_n, heads):
    nb = 50
    layers = layers_of(cuda, tqlib, nb, heads, [FORMATS[i % 4] for i in range(layers_n)])
    pages = host_pages(layers, nb)
    src, dst = np.array([3, 4, 5, -1, 7, 7, 9], np.int32), np.array([10, 11, 12, -1, 13, 14, 9], np.int32)
    tqlib.copy_blocks(layers, dev(cuda, src), dev(cuda, dst))
    for p in pages:
        for s, d in zip(src, dst):
            if s >= 0:
                p[d] = p[s]
    for got, want in zip(host_pages(layers, nb), pages):
        assert np.array_equal(got, want)
    assert tqlib.get_device_status() == 0
    # two sources for one block: the later pair counts; a source that another pair writes, ids outside
    src, dst = np.array([1, 2, 20, 21, 50, 5, -1], np.int32), np.array([30, 30, 21, 31, 32, -1, 33], np.int32)
    tqlib.copy_blocks(layers, dev(cuda, src), dev(cuda, dst))
    for p in pages:
        p[30], p[21] = p[2], p[20]
    for got, want in zip(host_pages(layers, nb), pages):
        assert np.array_equal(got, want)
    assert tqlib.get_device_status() == tqlib.TQ_DEV_BAD_BLOCK


def test_captured_and_other_stream(cuda, tqlib):
    """A reordering and an extension captured once and replayed twice; the same calls given a stream."""
    g, layers, model, blocks, table, lens, t = start(cuda, tqlib, 13, 12, 6, 400, FORMATS[:2])
    lens = np.minimum(lens, 70).astype(np.int32)
    refs0 = np.zeros(400, np.int32)
    for b in range(12):
        for j in range(-(-lens[b] // BLOCK)):
            refs0[table[b, j]] += 1
    parents = g.integers(0, 12, 20).astype(np.int32)
    blocks.refs.copy_(dev(cuda, refs0))
    d = dict(t=t, lens=dev(cuda, lens), parents=dev(cuda, parents), refs=dev(cuda, refs0))
    side = cuda.cuda.Stream()
    side.wait_stream(cuda.cuda.current_stream())
    with cuda.cuda.stream(side):  # (workspaces of this size exist before the capture)
        blocks.reorder(layers, d["t"], d["lens"], d["parents"])
    cuda.cuda.current_stream().wait_stream(side)
    pages = host_pages(layers, 400)
    graph = cuda.cuda.CUDAGraph()
    with cuda.cuda.graph(graph):
        blocks.refs.copy_(d["refs"])
        n, nl = blocks.reorder(layers, d["t"], d["lens"], d["parents"])
        blocks.extend(n, nl, nl + 1)
    model = Model(400, pages)
    for _ in range(2):
        graph.replay()
        model.refs[:] = refs0
        mt, ml = model.reorder(table, lens, parents)
        model.extend(mt, ml, ml + 1)
        assert np.array_equal(n.cpu().numpy(), mt) and np.array_equal(nl.cpu().numpy(), ml)
        check(cuda, blocks, layers, model)
    blocks.refs.copy_(d["refs"])
    side.wait_stream(cuda.cuda.current_stream())
    n, nl = blocks.reorder(layers, d["t"], d["lens"], d["parents"], stream=side)
    side.synchronize()
    model.refs[:] = refs0
    mt, ml = model.reorder(table, lens, parents)
    assert np.array_equal(n.cpu().numpy(), mt)
    check(cuda, blocks, layers, model)
    assert tqlib.get_device_status() == 0


def test_captured_before_any_call(cuda, tqlib):
    """The first calls of an object are captured, in memory that an earlier graph left full of other bytes: calls outside the
    graph, before its first replay and after it, have a workspace of their own."""
    g, layers, model, blocks, table, lens, t = start(cuda, tqlib, 17, 8, 5, 200, FORMATS[:1])
    blocks = tqlib.Blocks(200)  # (without a workspace yet)
    lens = np.minimum(lens, 60).astype(np.int32)
    refs0 = np.zeros(200, np.int32)
    for b in range(8):
        for j in range(-(-lens[b] // BLOCK)):
            refs0[table[b, j]] += 1
    parents = g.integers(0, 8, 16).astype(np.int32)
    d = dict(t=t, lens=dev(cuda, lens), parents=dev(cuda, parents), refs=dev(cuda, refs0))
    cuda.cuda.synchronize()
    first, graph = cuda.cuda.CUDAGraph(), cuda.cuda.CUDAGraph()
    with cuda.cuda.graph(first):
        full = [cuda.full((8192,), 0x55, dtype=cuda.uint8, device="cuda") for _ in range(240)]
        del full
    first.replay()
    with cuda.cuda.graph(graph, pool=first.pool()):
        blocks.refs.copy_(d["refs"])
        n, nl = blocks.reorder(layers, d["t"], d["lens"], d["parents"])
        blocks.extend(n, nl, nl + 1)
    pages = host_pages(layers, 200)
    model = Model(200, pages)

    def want():
        model.refs[:] = refs0
        mt, ml = model.reorder(table, lens, parents)
        model.extend(mt, ml, ml + 1)
        return mt, ml

    for replay in (False, True, False):
        if replay:
            graph.replay()
            got = n, nl
        else:
            blocks.refs.copy_(d["refs"])
            got = blocks.reorder(layers, d["t"], d["lens"], d["parents"])
            blocks.extend(got[0], got[1], got[1] + 1)
        mt, ml = want()
        assert np.array_equal(got[0].cpu().numpy(), mt) and np.array_equal(got[1].cpu().numpy(), ml)
        check(cuda, blocks, layers, model)
    assert tqlib.get_device_status() == 0
