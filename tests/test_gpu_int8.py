"""int8 layers: appends bit by bit, decode and attention of several tokens, against 64-bit arithmetic."""
import math

import numpy as np
import pytest

from tests import _int8_ref as ref

pytestmark = pytest.mark.gpu
D, BLOCK = 128, 16
SCALE = 1.0 / math.sqrt(D)


def layer_of(tq, blocks, heads, **kw):
    return tq.Layer(blocks, heads, kv_format="int8", **kw)


def pages(layer, which):
    pool = (layer.k_cache, layer.v_cache)[which]
    return ref.split(pool.cpu().numpy(), layer.num_blocks, layer.num_kv_heads)


def assert_pages(layer, want, which, touched=None):
    got = pages(layer, which)
    for g, w, what in zip(got, want, ("codes", "steps", "bits")):
        if touched is not None:
            g, w = g[touched], w[touched]
        assert np.array_equal(g, w), what


def data(cuda, seed, n, heads, dtype="bf16", spread=1.0):
    g = np.random.default_rng(seed)
    x = (g.standard_normal((n, heads, D)) * np.exp(spread * g.standard_normal((1, heads, D)))).astype(np.float32)
    t = cuda.from_numpy(x).cuda()
    return t.to(cuda.bfloat16) if dtype == "bf16" else t


def host(t):
    return t.float().cpu().numpy()


def blank(blocks, heads):
    return np.full((blocks, heads, BLOCK, D), -128, np.int8), np.zeros((blocks, heads), np.float32), np.zeros((blocks, heads), np.uint32)


def orders(kind, seed, n, blocks):
    """Slots of n tokens: one sequence from a slot inside a block on, sequences token by token, or any order."""
    g = np.random.default_rng(seed)
    ids = g.permutation(blocks)
    if kind == "sequence":
        at = 5 + np.arange(n)
        return ids[at // BLOCK] * BLOCK + at % BLOCK
    if kind == "time":  # as many sequences as fit, each with a block row of its own
        per = max(1, blocks // 7)
        seqs = min(7, -(-n // (per * BLOCK - 3))) + 1
        t, b = np.divmod(np.arange(n), seqs)
        at = 3 + t
        return ids[(b * per + at // BLOCK) % blocks] * BLOCK + at % BLOCK
    return g.permutation(blocks * BLOCK)[:n]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,heads,kind", [(1, 1, "sequence"), (1, 8, "any"), (16, 3, "sequence"), (37, 2, "sequence"),
                                          (300, 1, "time"), (700, 2, "any"), (1500, 2, "sequence"), (8192, 1, "time"),
                                          (8193, 1, "sequence"), (8209, 2, "time"), (9000, 1, "any")])
def test_append_bit_by_bit(cuda, tqlib, n, heads, kind, dtype):
    """Two appends in a row: the second into blocks that the first left partly filled, with larger and smaller values."""
    blocks = n // BLOCK + 10
    slots = orders(kind, n, n, blocks)
    layer = layer_of(tqlib, blocks, heads)
    want = [blank(blocks, heads), blank(blocks, heads)]
    first = np.arange(n) % 3 != 1
    for part, grow in ((first, 1.0), (~first, 1.7)):
        s = slots[part]
        if s.size == 0:
            continue
        k, v = (data(cuda, 7 * n + i, s.size, heads, dtype) * g for i, g in ((0, grow), (1, 1.0 / grow)))
        layer.append(k, v, cuda.from_numpy(s.astype(np.int64)).cuda())
        for w, x in ((0, k), (1, v)):
            ref.append(*want[w], host(x), s)
    touched = np.unique(slots // BLOCK)
    for w in (0, 1):
        assert_pages(layer, want[w], w, touched)
    rest = np.setdiff1d(np.arange(blocks), touched)  # other blocks are as they were
    assert not layer.k_cache.view(blocks, -1)[cuda.from_numpy(rest).cuda()].any()
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("n,heads,kind", [(1024, 2, "time"), (1025, 4, "time"), (1030, 1, "any"), (4096, 5, "time"),
                                          (4097, 4, "time"), (4100, 2, "sequence")])
def test_append_at_once(cuda, tqlib, n, heads, kind):
    """One call of tokens around the sizes where tokens go to CTAs in other numbers, slots given twice and skipped ones among them."""
    blocks = n // BLOCK + 10
    slots = orders(kind, 3 * n, n, blocks)
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


def test_append_token_by_token(cuda, tqlib):
    """Sixteen decode steps into one block a sequence: the step grows, earlier codes are rounded again."""
    B, H = 5, 2
    layer = layer_of(tqlib, B, H)
    want = [blank(B, H), blank(B, H)]
    for t in range(BLOCK):
        k, v = data(cuda, 100 + t, B, H) * (1.0 + 0.3 * t), data(cuda, 200 + t, B, H) * (2.0 - 0.1 * t)
        s = np.arange(B) * BLOCK + t
        layer.append(k, v, cuda.from_numpy(s).cuda())
        for w, x in ((0, k), (1, v)):
            ref.append(*want[w], host(x), s)
    for w in (0, 1):
        assert_pages(layer, want[w], w)


@pytest.mark.parametrize("n", [40, 9001])
def test_append_borders(cuda, tqlib, n):
    """Values that lie in the middle between two codes, and next to it, go where the exact quotient goes."""
    blocks, H = n // BLOCK + 1, 1
    g = np.random.default_rng(n)
    top = np.float32(3.0)
    step = np.float32(top / np.float32(127))
    mid = (g.integers(-126, 126, (n, H, D)) + 0.5) * np.float64(step)
    x = mid.astype(np.float32)
    near = g.integers(-2, 3, x.shape)
    for k in (1, 2):
        x = np.where(near >= k, np.nextafter(x, np.float32(np.inf)), x)
        x = np.where(near <= -k, np.nextafter(x, np.float32(-np.inf)), x)
    x[::16, :, 0] = top
    layer, want = layer_of(tqlib, blocks, H), [blank(blocks, H), blank(blocks, H)]
    s = np.arange(n)
    t = cuda.from_numpy(x).cuda()
    layer.append(t, t, cuda.from_numpy(s).cuda())
    # steps of a power of two, whose middles are exact: ties go to even codes
    ref.append(*want[0], x, s)
    assert_pages(layer, want[0], 0)
    y = ((g.integers(-126, 126, (n, H, D)) + 0.5) * 0.25).astype(np.float32)
    y[::16, :, 3] = 127 * 0.25
    t = cuda.from_numpy(y).cuda()
    layer.append(None, t, cuda.from_numpy(s).cuda())
    ref.append(*want[1], y, s)
    assert_pages(layer, want[1], 1)
    # and the rounding of codes that are there: twice the step, codes that are odd
    if n < 100:
        big = np.zeros((2, H, D), np.float32)
        big[:, :, 1] = 127 * 0.5
        s2 = np.array([15, 16 + 15])
        layer.append(None, cuda.from_numpy(big).cuda(), cuda.from_numpy(s2).cuda())
        ref.append(*want[1], big, s2)
        assert_pages(layer, want[1], 1)


def test_append_extremes(cuda, tqlib):
    """Zeros, values below the least step, the largest ones; tokens with infinities and NaN among others."""
    blocks, H = 6, 2
    x = host(data(cuda, 3, blocks * BLOCK, H))
    x[0:16] = 0.0
    x[16:32] *= 1e-40
    x[32:48] *= np.float32(1e38) / np.abs(x[32:48]).max() * 3
    x[50, 0, 3], x[51, 1, 5], x[52, 0, 7] = np.nan, np.inf, -np.inf
    x[64:80] = np.nan
    s = np.arange(blocks * BLOCK)
    layer, want = layer_of(tqlib, blocks, H, fill=0xA5), blank(blocks, H)
    want[1][:] = np.frombuffer(b"\xa5\xa5\xa5\xa5", np.float32)[0]
    t = cuda.from_numpy(x).cuda()
    layer.append(t, t, cuda.from_numpy(s).cuda())
    ref.append(*want, x, s)
    for w in (0, 1):
        assert_pages(layer, want, w)
    # what is read back: the others' values stay, the marked tokens are NaN whole
    got = layer.dequantize(0, cuda.from_numpy(s).cuda()).cpu().numpy()
    exact = ref.values(*want).transpose(0, 2, 1, 3).reshape(-1, H, D)
    assert np.array_equal(np.isnan(got), np.isnan(exact))
    with np.errstate(over="ignore"):
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(exact.astype(np.float32)))
    # a marked token that is written again is a number again
    y = host(data(cuda, 4, 1, H))
    layer.append(cuda.from_numpy(y).cuda(), None, cuda.tensor([50], device="cuda"))
    ref.append(*want, y, [50])
    assert_pages(layer, want, 0)
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("n", [50, 9000])
def test_append_slots(cuda, tqlib, n):
    """Skipped tokens, a slot given twice (the later token stays), slots past the pool (recorded), keys alone."""
    blocks, H = n // BLOCK + 2, 2
    g = np.random.default_rng(n)
    s = g.permutation(blocks * BLOCK)[:n].astype(np.int64)
    s[::7] = -1
    s[5::11] = s[4::11][:s[5::11].size]
    s[3] = blocks * BLOCK
    s[8] = 1 << 40
    k = data(cuda, n, n, H)
    layer, want = layer_of(tqlib, blocks, H), blank(blocks, H)
    layer.append(k, None, cuda.from_numpy(s).cuda())
    assert tqlib.get_device_status() == tqlib.TQ_DEV_BAD_SLOT
    ref.append(*want, host(k), s)
    assert_pages(layer, want, 0, np.unique(s[(s >= 0) & (s < blocks * BLOCK)] // BLOCK))
    assert not layer.v_cache.any()


def filled(cuda, tq, seed, blocks, heads, spread=1.0):
    layer = layer_of(tq, blocks, heads)
    k, v = (data(cuda, seed + i, blocks * BLOCK, heads, spread=spread) for i in (0, 1))
    layer.append(k, v, cuda.arange(blocks * BLOCK, device="cuda"))
    return layer


def dev(cuda, x, dtype=None):
    t = cuda.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def check_rows(out, wants, half=0.0):
    """out [rows, Hq, D] against (value, bound) a row; `half`: half a step of the output's type."""
    for i, (want, bound) in enumerate(wants):
        fine = ~np.isnan(want)
        assert np.array_equal(np.isnan(out[i]), ~fine), i
        room = bound[:, None] + half * np.abs(want) + 1e-37
        err = np.abs(out[i] - want)
        assert (err[fine] <= room[fine]).all(), (i, float((err[fine] / room[fine]).max()))


def tables(seed, lens, blocks):
    g = np.random.default_rng(seed)
    width = max(1, -(-max(lens) // BLOCK))
    ids = np.stack([g.permutation(blocks)[:width] for _ in lens]).astype(np.int32)
    return ids


LENS = [[1], [16, 17], [0, 5, 300, 15], [33, 0, 700, 64, 1, 1000]]


@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (8, 4), (1, 5), (2, 8), (3, 12), (1, 17)])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode(cuda, tqlib, heads, group, lens, dtype):
    blocks, hq = 70, heads * group
    layer = filled(cuda, tqlib, 11, blocks, heads)
    table, g = tables(5, lens, blocks), np.random.default_rng(hq)
    q = dev(cuda, g.standard_normal((len(lens), hq, D)).astype(np.float32) * 2, cuda.bfloat16 if dtype == "bf16" else None)
    k, v = (ref.values(*pages(layer, w)) for w in (0, 1))
    wants = [ref.attention(host(q)[i].astype(np.float64), k, v, table[i], n, SCALE) for i, n in enumerate(lens)]
    ws = cuda.zeros(layer.workspace_bytes(len(lens), hq, table.shape[1]), dtype=cuda.uint8, device="cuda")
    first = None
    for splits in (0, 1, 5, 0):
        out = layer.decode(q, dev(cuda, table), dev(cuda, np.array(lens, np.int32)), out_dtype=cuda.float32, num_splits=splits, workspace=ws)
        check_rows(out.cpu().numpy().astype(np.float64), wants)
        if splits == 0:
            assert first is None or cuda.equal(out, first)  # the same call, the same bits
            first = out
    half = layer.decode(q, dev(cuda, table), dev(cuda, np.array(lens, np.int32)), out_dtype=cuda.bfloat16, workspace=ws)
    assert cuda.equal(half, first.to(cuda.bfloat16))
    assert not ws[:65536].any() and tqlib.get_device_status() == 0


def test_decode_many_rows(cuda, tqlib):
    """More rows than threads, most of them short or empty: units inside a warp's range, and across warps."""
    rows, heads, hq, blocks = 700, 2, 6, 90
    g = np.random.default_rng(1)
    lens = g.integers(0, 40, rows)
    lens[3], lens[699], lens[500] = 800, 0, 900
    layer, table = filled(cuda, tqlib, 21, blocks, heads), tables(6, list(lens), blocks)
    q = g.standard_normal((rows, hq, D)).astype(np.float32)
    k, v = (ref.values(*pages(layer, w)) for w in (0, 1))
    out = layer.decode(dev(cuda, q), dev(cuda, table), dev(cuda, lens.astype(np.int32))).cpu().numpy()
    check_rows(out, [ref.attention(q[i].astype(np.float64), k, v, table[i], int(n), SCALE) for i, n in enumerate(lens)])
    assert tqlib.get_device_status() == 0


def test_decode_bad_entries(cuda, tqlib):
    """Block ids outside the pool count as no tokens, contexts outside the table are cut; both are recorded."""
    layer, hq = filled(cuda, tqlib, 31, 20, 2), 8
    table = tables(7, [80, 80, 80], 20)
    table[0, 1], table[1, :], table[2, 4] = -1, 20, 1 << 30
    lens = np.array([70, 33, 5 * BLOCK + 9], np.int32)
    q = np.random.default_rng(2).standard_normal((3, hq, D)).astype(np.float32)
    k, v = (ref.values(*pages(layer, w)) for w in (0, 1))
    out = layer.decode(dev(cuda, q), dev(cuda, table), dev(cuda, lens)).cpu().numpy()
    check_rows(out, [ref.attention(q[i].astype(np.float64), k, v, table[i], min(int(n), 80), SCALE) for i, n in enumerate(lens)])
    assert not out[1].any()
    assert tqlib.get_device_status() == tqlib.TQ_DEV_BAD_BLOCK | tqlib.TQ_DEV_BAD_CONTEXT
    lens[:] = -5
    assert not layer.decode(dev(cuda, q), dev(cuda, table), dev(cuda, lens)).any()
    assert tqlib.get_device_status() == tqlib.TQ_DEV_BAD_CONTEXT


@pytest.mark.parametrize("hq", [4, 8])
def test_decode_ranges(cuda, tqlib, hq):
    """Values of a block far above or below the others', tiny and huge queries, logits of thousands, NaN tokens
    behind the context and inside it, a query that is not finite: each row only pays for itself."""
    heads, blocks, n = 1, 24, 24 * BLOCK
    g = np.random.default_rng(hq)
    k, v = g.standard_normal((n, heads, D)).astype(np.float32), g.standard_normal((n, heads, D)).astype(np.float32)
    v[32:48] *= 2.0 ** 60
    k[32:48] = -np.abs(k[32:48])
    v[200:216] *= 2.0 ** -70
    k[300, 0, 5], v[310, 0, 9] = np.nan, np.inf
    layer = layer_of(tqlib, blocks, heads)
    layer.append(dev(cuda, k), dev(cuda, v), cuda.arange(n, device="cuda"))
    q = g.standard_normal((7, hq, D)).astype(np.float32)
    q[0] = np.abs(q[0]) * 20   # the block of large values has weights far below 2^-60
    q[1] *= 1e-30
    q[2] *= 1000.0
    q[3, 1, 4] = np.inf
    lens = np.array([200, 200, 290, 100, 300, 301, 320], np.int32)
    table = np.tile(np.arange(blocks, dtype=np.int32), (7, 1))
    kk, vv = (ref.values(*pages(layer, w)) for w in (0, 1))
    out = layer.decode(dev(cuda, q), dev(cuda, table), dev(cuda, lens)).cpu().numpy()
    with np.errstate(all="ignore"):
        wants = [ref.attention(q[i].astype(np.float64), kk, vv, table[i], int(m), SCALE) for i, m in enumerate(lens)]
    wants[3][0][1] = np.nan
    wants[3][1][1] = 0.0
    # (a row whose weights on the large values vanish is held to the values that it does attend)
    s = (kk.reshape(-1, D)[:200] @ q[0].astype(np.float64).T) * SCALE
    w = np.exp(s - s.max(0))
    assert (w[32:48] < 2.0 ** -90).all()
    keep = np.abs(np.delete(vv.reshape(-1, D)[:200], slice(32, 48), 0)).max()
    wants[0] = (wants[0][0], wants[0][1] / np.abs(vv.reshape(-1, D)[:200]).max() * keep)
    assert np.isfinite(wants[4][0]).all() and np.isnan(wants[5][0]).all() and np.isnan(wants[6][0]).all()
    check_rows(out, wants)


ATTEND = [(2, 4, [1], [0]), (1, 8, [5, 0, 17, 1], [0, 30, 100, 15]), (2, 3, [40, 33], [0, 7]), (1, 1, [130], [20]),
          (1, 12, [3, 64], [250, 1]),
          # tiles: one row past a stream, past a tile; groups that do not divide one; several tiles and steps
          (1, 4, [33], [0]), (1, 4, [64, 65], [0, 300]), (2, 8, [100, 3, 33], [50, 20, 0]), (1, 3, [300], [200]),
          (3, 5, [60, 0, 52], [1000, 8, 3]), (1, 1, [257, 40], [0, 128]), (1, 7, [37], [400]), (1, 128, [5], [77]),
          (1, 300, [2], [40])]


def attend_case(cuda, tqlib, seed, heads, group, new, past, dtype, change=None, scale=SCALE, pool=None):
    """One call over a filled layer (`change`: of its keys and values first); rows against 64 bits."""
    hq, lens = heads * group, [a + b for a, b in zip(new, past)]
    blocks = -(-max(lens) // BLOCK) + 3
    g = np.random.default_rng(seed)
    n = blocks * BLOCK
    k, v = (g.standard_normal((n, heads, D)).astype(np.float32) for _ in "kv")
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rows = int(starts[-1]) + 3
    q = g.standard_normal((rows, hq + 2, D)).astype(np.float32)
    table = tables(seed, lens, blocks)
    if change is not None:
        change(k, v, q, table)
    layer = layer_of(tqlib, blocks, heads)
    layer.append(dev(cuda, k), dev(cuda, v), cuda.arange(n, device="cuda"))
    q = dev(cuda, q, dtype)[:, 1:hq + 1]  # a view of a fused projection
    out = cuda.full((rows, hq, D), 7.0, dtype=cuda.float32, device="cuda")
    ws = cuda.zeros(layer.attend_workspace_bytes(rows, len(new), hq, table.shape[1]), dtype=cuda.uint8, device="cuda")
    args = (dev(cuda, starts), dev(cuda, table), dev(cuda, np.array(lens, np.int32)))
    assert layer.attend(q, *args, out=out, workspace=ws, sm_scale=scale) is out
    got = out.cpu().numpy()
    assert (got[starts[-1]:] == 7.0).all()  # rows behind the last sequence
    assert not ws[:65536].any()
    again = layer.attend(q, *args, out=out.clone(), workspace=ws, sm_scale=scale)
    assert np.array_equal(again.cpu().numpy(), got, equal_nan=True)  # the same bits
    half = layer.attend(q, *args, out_dtype=cuda.bfloat16, workspace=ws, sm_scale=scale)[:starts[-1]]
    assert cuda.equal(half.nan_to_num(3e4), out[:starts[-1]].to(cuda.bfloat16).nan_to_num(3e4))
    kk, vv = (ref.values(*pages(layer, w)) for w in (0, 1))
    weights = 2.0 ** -11 if dtype == cuda.bfloat16 else 0.0
    qh = host(q).astype(np.float64)
    with np.errstate(all="ignore"):
        wants = [ref.attention(qh[starts[b] + i], kk, vv, table[b], past[b] + i + 1, scale, weights)
                 for b, m in enumerate(new) for i in range(m)]
    return got[:starts[-1]], wants, kk, vv


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(cuda, tqlib, case, dtype):
    got, wants, _, _ = attend_case(cuda, tqlib, case, *ATTEND[case], cuda.bfloat16 if dtype == "bf16" else cuda.float32,
                                   scale=SCALE if case % 3 else -0.2)
    check_rows(got, wants)
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_ranges(cuda, tqlib, dtype):
    """Blocks of values far above and below the others', NaN tokens that only later rows see, tiny, large and
    infinite queries, bad block ids, in tiles: each row only pays for itself."""
    def change(k, v, q, table):
        v[32:48] *= 2.0 ** 40
        v[96:112] *= 2.0 ** -60
        k[130, 0, 5], v[160, 0, 9] = np.nan, np.inf
        table[0] = np.arange(table.shape[1])  # (these blocks are tokens of the first sequence in order)
        table[0, 3] = -1
        table[1, 2] = 1 << 28
        q[5] *= 1e-30
        q[6] *= 200.0
        q[7, 2] = np.inf
        table[1][table[1] == 2] = 5
        table[1][table[1] == 8] = 6
        table[1][table[1] == 10] = 7

    got, wants, kk, vv = attend_case(cuda, tqlib, 99, 1, 4, [180, 50], [10, 100], cuda.bfloat16 if dtype == "bf16" else cuda.float32, change)
    wants[7][0][1] = np.nan
    assert np.abs(vv[2]).max() > 1e9
    for i, (want, _) in enumerate(wants[:180]):  # row i of the first sequence sees tokens 0 .. 10 + i
        assert np.isnan(want).all() == (i >= 130 - 10), i
    check_rows(got, wants)
    assert tqlib.get_device_status() == tqlib.TQ_DEV_BAD_BLOCK


def test_attend_lengths(cuda, tqlib):
    """Contexts shorter than the queries (zero rows), outside the table, empty sequences."""
    heads, group = 1, 4
    layer = filled(cuda, tqlib, 61, 12, heads)
    new, lens = [40, 20, 10, 3], [25, 0, 400, -3]
    table = np.tile(np.arange(8, dtype=np.int32), (4, 1))
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = np.random.default_rng(4).standard_normal((int(starts[-1]), 4, D)).astype(np.float32)
    out = layer.attend(dev(cuda, q), dev(cuda, starts), dev(cuda, table), dev(cuda, np.array(lens, np.int32))).cpu().numpy()
    k, v = (ref.values(*pages(layer, w)) for w in (0, 1))
    wants = []
    for b, n in enumerate(new):
        ctx = min(max(lens[b], 0), 128)
        wants += [ref.attention(q[starts[b] + i].astype(np.float64), k, v, table[b], max(0, ctx - n + i + 1), SCALE) for i in range(n)]
    check_rows(out, wants)
    assert not out[:15].any() and not out[40:60].any()
    assert tqlib.get_device_status() == tqlib.TQ_DEV_BAD_CONTEXT
