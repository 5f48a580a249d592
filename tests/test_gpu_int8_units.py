"""Attention of several tokens over int8 layers where every CTA has several units of the line of tiles: short ones one after
another, of one stream and of two, whole and cut, beside sequences that the decode kernel takes."""
import math

import numpy as np
import pytest

from tests import _int8_ref as ref

pytestmark = pytest.mark.gpu
D, BLOCK = 128, 16
SCALE = 1.0 / math.sqrt(D)


def drawn(seed, seqs, new, past, empty=0):
    """Ragged lengths: new tokens and tokens before them of so many sequences; every `empty`-th has none before."""
    g = np.random.default_rng(seed)
    n, p = g.integers(*new, seqs), g.integers(*past, seqs)
    if empty:
        p[::empty] = 0
    return [int(x) for x in n], [int(x) for x in p]


# heads, group, (new tokens, tokens before them); of 152 CTAs' parts: most units in one, cut units, parts cut at both ends
CASES = {
    "short": (8, 4, drawn(0, 64, (6, 61), (0, 200))),  # 4, 0, 0: units of 1 to 3 steps
    "mixed": (8, 8, drawn(1, 40, (3, 70), (0, 1500), 7)),  # 7, 54, 18: of 1 to 12, both streams or one
    "one_head": (4, 1, drawn(2, 70, (21, 260), (0, 900))),  # 4, 14, 0
    "beside_decode": (8, 3, ([700, 3, 90, 1, 260, 33] * 3, [0, 500, 2100, 40, 0, 900] * 3)),  # 5, 36, 16
    "cut": (4, 5, ([1000, 400], [1500, 9000])),  # 3, 222, 33: of 13 to 74
    "one_long": (8, 8, ([33] * 30, [20000] + [40] * 29)),  # 8, 160, 8: of 157 among short ones
}


def places(new, past, heads, group):
    """Length of the line: steps of all units, and three a unit."""
    per, total = 256 // group, 0
    for n, p in zip(new, past):
        if n * group > 24:
            total += sum(max(1, -(-(p + min(n, (k + 1) * per)) // 128)) + 3 for k in range(-(-n // per))) * heads
    return total


def attention(cuda, q, k, v, past, scale):
    """(out [n, Hq, D], largest sum of a logit's magnitudes [n, Hq]) of q [n, Hq, D] after `past` tokens, k and v
    [tokens, heads, D], in 64 bits."""
    n, hq, heads = q.shape[0], q.shape[1], k.shape[1]
    out, size = cuda.empty(q.shape, dtype=cuda.float64, device="cuda"), cuda.empty((n, hq), dtype=cuda.float64, device="cuda")
    ahead = cuda.arange(past + n, device="cuda") > past + cuda.arange(n, device="cuda")[:, None]
    for h in range(hq):
        kh, vh = k[:past + n, h // (hq // heads)], v[:past + n, h // (hq // heads)]
        s = (q[:, h] @ kh.T * scale).masked_fill(ahead, -math.inf)
        w = cuda.exp(s - s.amax(1, keepdim=True))
        out[:, h] = w @ vh / w.sum(1, keepdim=True)
        size[:, h] = (q[:, h].abs() @ kh.abs().T * abs(scale)).masked_fill(ahead, 0.0).amax(1)
    return out, size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", CASES)
def test_attend_units(cuda, tqlib, name, dtype):
    heads, group, (new, past) = CASES[name]
    hq, lens = heads * group, [a + b for a, b in zip(new, past)]
    assert places(new, past, heads, group) > 14 * cuda.cuda.get_device_properties(0).multi_processor_count
    gen = cuda.Generator(device="cuda").manual_seed(len(name))
    used = [-(-n // BLOCK) for n in lens]
    blocks = sum(used) + 2
    layer = tqlib.Layer(blocks, heads, kv_format="int8")
    x = [cuda.randn(blocks * BLOCK, heads, D, device="cuda", generator=gen) for _ in "kv"]
    layer.append(*x, cuda.arange(blocks * BLOCK, device="cuda"))
    ids = cuda.randperm(blocks, device="cuda", generator=gen).int()
    table = cuda.full((len(lens), max(used)), -1, dtype=cuda.int32, device="cuda")
    for b, n in enumerate(used):
        table[b, :n] = ids[sum(used[:b]):sum(used[:b]) + n]
    starts = [sum(new[:b]) for b in range(len(new) + 1)]
    q = cuda.randn(starts[-1] + 2, hq, D, device="cuda", generator=gen).to(cuda.bfloat16 if dtype == "bf16" else cuda.float32)
    args = (cuda.tensor(starts, dtype=cuda.int32, device="cuda"), table, cuda.tensor(lens, dtype=cuda.int32, device="cuda"))
    ws = cuda.zeros(layer.attend_workspace_bytes(q.shape[0], len(new), hq, table.shape[1]), dtype=cuda.uint8, device="cuda")
    out = cuda.full(q.shape, 7.0, dtype=cuda.float32, device="cuda")
    layer.attend(q, *args, out=out, workspace=ws)
    assert tqlib.get_device_status() == 0 and not ws[:65536].any()
    assert (out[starts[-1]:] == 7.0).all()
    for _ in range(3):  # the same bits, whatever the CTAs do first
        again = layer.attend(q, *args, out_dtype=cuda.float32, workspace=ws)
        assert cuda.equal(again[:starts[-1]], out[:starts[-1]])
    k, v = (cuda.from_numpy(ref.values(*ref.split(pool.cpu().numpy(), blocks, heads))).cuda() for pool in (layer.k_cache, layer.v_cache))
    # what a call over few tokens may be off by (_int8_ref.attention), and what the accumulators cut off: 2^-20 of a sum a
    # step, of up to 128 steps for bf16 queries and 8 for fp32 ones
    weights, span = (2.0 ** -11, 128) if dtype == "bf16" else (0.0, 8)
    for b, n in enumerate(new):
        at = table[b, :used[b]].long()
        kb, vb = (t[at].transpose(1, 2).reshape(-1, heads, D)[:lens[b]] for t in (k, v))
        want, size = attention(cuda, q[starts[b]:starts[b + 1]].double(), kb, vb, past[b], SCALE)
        cut = min(span, -(-lens[b] // 128)) * 2.0 ** -20
        room = (2 * 2.0 ** -19 * size + 2.0 ** -20 + weights + cut) * vb.abs().max()
        err = (out[starts[b]:starts[b + 1]] - want).abs().amax(-1)
        assert (err <= room).all(), (b, float((err / room).max()))
    assert tqlib.get_device_status() == 0


def small_case(cuda, tqlib, dtype, seed=0):
    """60 ragged sequences over a layer of 4 heads in groups of four, some for the decode kernel: (layer, q, call)."""
    new, past = drawn(seed, 60, (1, 120), (0, 300), 5)
    heads, hq, lens = 4, 16, [a + b for a, b in zip(new, past)]
    gen = cuda.Generator(device="cuda").manual_seed(seed)
    used = [-(-n // BLOCK) for n in lens]
    blocks = sum(used)
    layer = tqlib.Layer(blocks, heads, kv_format="int8")
    layer.append(*(cuda.randn(blocks * BLOCK, heads, D, device="cuda", generator=gen) for _ in "kv"), cuda.arange(blocks * BLOCK, device="cuda"))
    table = cuda.full((len(lens), max(used)), -1, dtype=cuda.int32, device="cuda")
    for b, n in enumerate(used):
        table[b, :n] = cuda.arange(sum(used[:b]), sum(used[:b]) + n, device="cuda")
    starts = cuda.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=cuda.int32, device="cuda")
    lens = cuda.tensor(lens, dtype=cuda.int32, device="cuda")
    q = cuda.randn(sum(new), hq, D, device="cuda", generator=gen).to(dtype)
    return layer, q, (starts, table, lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_rows_anywhere(cuda, tqlib, dtype):
    """Rows that begin at any element, heads and tokens in any order, in place: the same bits as contiguous ones."""
    dtype = cuda.bfloat16 if dtype == "bf16" else cuda.float32
    layer, q, args = small_case(cuda, tqlib, dtype)
    want = layer.attend(q, *args)
    n, hq = q.shape[0], q.shape[1]

    def views():
        odd = cuda.full((n * (hq * 131 + 7) + 3,), 5.0, dtype=dtype, device="cuda")
        yield odd, odd.as_strided((n, hq, D), (hq * 131 + 7, 131, 1), 3)  # no row is aligned to more than an element
        turned = cuda.full((hq + 1, n, D + 4), 5.0, dtype=dtype, device="cuda")
        yield turned, turned[1:, :, 4:].transpose(0, 1)  # head by head

    for _, rows in views():
        rows.copy_(q)
        assert cuda.equal(layer.attend(rows, *args), want)
    for whole, rows in views():
        layer.attend(q, *args, out=rows)
        assert cuda.equal(rows, want)
        rows.fill_(5.0)
        assert (whole == 5.0).all()  # nothing between the rows was written
    for _, rows in views():
        rows.copy_(q)
        assert layer.attend(rows, *args, out=rows) is rows and cuda.equal(rows, want)
    assert tqlib.get_device_status() == 0


def test_attend_replayed(cuda, tqlib):
    """A captured call over several units a CTA, replayed with other lengths, queries and tables; calls on two streams at once, each
    with a workspace of its own."""
    layer, q, (starts, table, lens) = small_case(cuda, tqlib, cuda.bfloat16)
    other = small_case(cuda, tqlib, cuda.bfloat16, 1)
    ws = cuda.zeros(layer.attend_workspace_bytes(q.shape[0], 60, 16, table.shape[1]), dtype=cuda.uint8, device="cuda")
    out = cuda.zeros_like(q)
    side = cuda.cuda.Stream()
    side.wait_stream(cuda.cuda.current_stream())
    with cuda.cuda.stream(side):
        layer.attend(q, starts, table, lens, out=out, workspace=ws)
    cuda.cuda.current_stream().wait_stream(side)
    graph = cuda.cuda.CUDAGraph()
    with cuda.cuda.graph(graph):
        layer.attend(q, starts, table, lens, out=out, workspace=ws)
    g = np.random.default_rng(5)
    for turn in range(4):
        lens.copy_(cuda.from_numpy(np.maximum(lens.cpu().numpy() - g.integers(0, 20, 60), 0).astype(np.int32)))
        table.copy_(table[cuda.randperm(60, device="cuda")])
        q.mul_(-1.0)
        graph.replay()
        got = out.clone()
        tqlib.get_device_status()  # (rows whose tables have become shorter than their lengths name blocks that are not there)
        assert cuda.equal(got, layer.attend(q, starts, table, lens, out=cuda.zeros_like(q)))
    want = other[0].attend(other[1], *other[2])
    tqlib.get_device_status()
    for _ in range(5):
        side.wait_stream(cuda.cuda.current_stream())
        graph.replay()
        with cuda.cuda.stream(side):
            second = other[0].attend(other[1], *other[2])
        cuda.cuda.current_stream().wait_stream(side)
        assert cuda.equal(second, want) and cuda.equal(out, got)
    tqlib.get_device_status()
