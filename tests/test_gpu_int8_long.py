"""int8 layers over long contexts, which a table gets by naming the same few blocks many times: sums of many steps."""
import math

import numpy as np
import pytest

from tests import _int8_ref as ref

pytestmark = pytest.mark.gpu
D, BLOCK = 128, 16
SCALE = 1.0 / math.sqrt(D)


def layer_with(cuda, tq, k, v):
    """A layer of the blocks that hold k and v [tokens, heads, D] from block 0 on."""
    layer = tq.Layer(k.shape[0] // BLOCK, k.shape[1], kv_format="int8")
    layer.append(*(cuda.from_numpy(np.ascontiguousarray(x, np.float32)).cuda() for x in (k, v)), cuda.arange(k.shape[0], device="cuda"))
    return layer


def values(layer):
    """Keys and values [blocks, heads, 16, D] in 64 bits."""
    return (ref.values(*ref.split(pool.cpu().numpy(), layer.num_blocks, layer.num_kv_heads)) for pool in (layer.k_cache, layer.v_cache))


def attend(cuda, layer, q, new, row, ctx, seqs):
    """`seqs` equal sequences of `new` query tokens each (the same rows q [new, Hq, D] for all) over the table row `row`."""
    starts = cuda.arange(seqs + 1, dtype=cuda.int32, device="cuda") * new
    table = cuda.from_numpy(row.astype(np.int32)).cuda().expand(seqs, -1).contiguous()
    lens = cuda.full((seqs,), ctx, dtype=cuda.int32, device="cuda")
    out = layer.attend(q.repeat(seqs, 1, 1), starts, table, lens, out_dtype=cuda.float32)
    return out.view(seqs, new, *q.shape[1:]).cpu().numpy().astype(np.float64)


def counted(q, k, v, row, lim):
    """Attention of q [Hq, D] over the first lim tokens of `row` in 64 bits, each token of the pool counted as often as
    it is named; with the largest sum of the magnitudes of a logit's products and the largest value."""
    blocks, heads = k.shape[0], k.shape[1]
    count = np.zeros((blocks, BLOCK))
    np.add.at(count, row[:lim // BLOCK], 1.0)
    if lim % BLOCK:
        count[row[lim // BLOCK], :lim % BLOCK] += 1.0
    out = np.zeros(q.shape)
    count, group, size = count.reshape(-1), q.shape[0] // heads, 0.0
    for h in range(q.shape[0]):
        kh, vh = k[:, h // group].reshape(-1, D)[count > 0], v[:, h // group].reshape(-1, D)[count > 0]
        s = kh @ q[h] * SCALE
        w = count[count > 0] * np.exp(s - s.max())
        out[h] = w @ vh / w.sum()
        size = max(size, (np.abs(kh) @ np.abs(q[h])).max() * SCALE)
    return out, size


def seqs_for(cuda, heads):
    """Sequences whose units of one tile are as many as the SMs, or more: each then is one CTA's alone."""
    return -(-cuda.cuda.get_device_properties(0).multi_processor_count // heads)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctx", [1 << 20, 30011, 5000])
def test_attend_sums(cuda, tqlib, ctx, dtype):
    """Units of up to 8192 steps.  Queries of zero attend to all tokens alike and the steps are powers of two, so that
    weights, products and the denominator are whole numbers without a rounding, and only the sums of values lose:
    an accumulator of the tensor cores what it cuts off, each fp32 addition outside half a step.  Values of 1 to
    127 grow steadily, so the half of all steps counts.  An accumulator takes at most 2^10 products (16 tokens
    each) of less than 2^-23 of its size, half of that; additions outside are at most ctx / 1024 of 2^-24, half of
    that; then the division and the last product, 2^-23 together."""
    heads, group, new = 8, 8, 32
    g = np.random.default_rng(ctx)
    k = g.standard_normal((2 * BLOCK, heads, D))
    v = g.integers(1, 128, (2 * BLOCK, heads, D)) * 0.25
    v[::BLOCK, :, 0] = 127 * 0.25
    layer = layer_with(cuda, tqlib, k, v)
    row = g.integers(0, 2, -(-ctx // BLOCK))
    q = cuda.zeros((new, heads * group, D), dtype=cuda.bfloat16 if dtype == "bf16" else cuda.float32, device="cuda")
    got = attend(cuda, layer, q, new, row, ctx, seqs_for(cuda, heads))
    kk, vv = values(layer)
    assert np.array_equal(vv.transpose(0, 2, 1, 3).reshape(v.shape), v)
    room = 2.0 ** 10 * 2.0 ** -24 + ctx / 1024 * 2.0 ** -25 + 2.0 ** -23
    for i in (0, 7, new - 1):
        want, _ = counted(np.zeros((heads * group, D)), kk, vv, row, ctx - new + i + 1)
        err = np.abs(got[:, i] - want) / want
        assert err.max() <= room, (i, err.max(), room)
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("group,new", [(8, 32), (4, 30)])  # both streams of a unit, one of them
def test_attend_sums_f32(cuda, tqlib, group, new):
    """fp32 queries over 150,000 tokens.  Logits lose what the short contexts' bound says (2^-19 of the magnitudes of
    their products, weights twice as much relatively and 2^-20); values' sums 2^7 products a span of 2^-23 each at
    most, and a span's addition, of at most ctx / 1024 of 2^-24; relative to the largest value."""
    heads, ctx = 8, 150001
    g = np.random.default_rng(group)
    layer = layer_with(cuda, tqlib, g.standard_normal((6 * BLOCK, heads, D)), 1.0 + 0.3 * g.standard_normal((6 * BLOCK, heads, D)))
    row = g.integers(0, 6, -(-ctx // BLOCK))
    q = g.standard_normal((new, heads * group, D)).astype(np.float32)
    got = attend(cuda, layer, cuda.from_numpy(q).cuda(), new, row, ctx, seqs_for(cuda, heads))
    kk, vv = values(layer)
    for i in (0, new - 1):
        want, size = counted(q[i].astype(np.float64), kk, vv, row, ctx - new + i + 1)
        room = (2 * 2.0 ** -19 * size + 2.0 ** -20 + 2.0 ** 7 * 2.0 ** -23 + ctx / 1024 * 2.0 ** -24) * np.abs(vv).max()
        err = np.abs(got[:, i] - want).max()
        assert err <= room, (i, err, room)
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("group", [4, 8])
def test_decode_long(cuda, tqlib, group):
    """One row over 200,000 tokens: parts of many warps joined."""
    heads, ctx = 2, 200003
    g = np.random.default_rng(group)
    layer = layer_with(cuda, tqlib, g.standard_normal((5 * BLOCK, heads, D)), 1.0 + 0.3 * g.standard_normal((5 * BLOCK, heads, D)))
    row = g.integers(0, 5, -(-ctx // BLOCK))
    q = g.standard_normal((1, heads * group, D)).astype(np.float32)
    table = cuda.from_numpy(row.astype(np.int32)).cuda().view(1, -1)
    got = layer.decode(cuda.from_numpy(q).cuda(), table, cuda.tensor([ctx], dtype=cuda.int32, device="cuda")).cpu().numpy().astype(np.float64)
    kk, vv = values(layer)
    want, size = counted(q[0].astype(np.float64), kk, vv, row, ctx)
    # (a block's products inside the tensor cores, then at most 12,501 blocks of half a step each in fp32, in parts)
    room = (2 * 2.0 ** -19 * size + 2.0 ** -20 + 2.0 ** -19 + 12501 * 2.0 ** -25) * np.abs(vv).max()
    assert np.abs(got[0] - want).max() <= room
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("below", [27.5, 20.0])
def test_attend_values_of_zero(cuda, tqlib, below, dtype):
    """Tokens without values (zeros, whose step is the least there is) count in the denominator however far their logits
    lie below the largest one: 2^20 of them, 27.5 binary orders below, take 0.5% of a row's result.  Room: half a step of a
    weight's type on either side of it, and the logits' and sums' of the other tests."""
    heads, group, new, ctx = 8, 8, 32, 1 << 20
    k, v = np.zeros((2 * BLOCK, heads, D)), np.zeros((2 * BLOCK, heads, D))
    k[0, :, 0] = 127.0 / 128  # the one token that counts, with a logit of 60 binary orders
    v[0] = np.random.default_rng(3).integers(64, 128, (heads, D)) * 0.25
    v[0, :, 0] = 127 * 0.25
    scale = SCALE * math.log2(math.e)
    q = np.zeros((new, heads * group, D), np.float32)
    q[..., 0] = 474.0
    k[BLOCK:, :, 0] = k[0, 0, 0] - below / (474.0 * scale)
    layer = layer_with(cuda, tqlib, k, v)
    row = np.ones(ctx // BLOCK, np.int64)
    row[0] = 0
    got = attend(cuda, layer, cuda.from_numpy(q).cuda().to(cuda.bfloat16 if dtype == "bf16" else cuda.float32), new, row, ctx, seqs_for(cuda, heads))
    kk, vv = values(layer)
    for i in (0, new - 1):
        want, size = counted(q[i].astype(np.float64), kk, vv, row, ctx - new + i + 1)
        alone = vv[0, :, 0].repeat(group, 0)
        assert (want / alone).max() < 1 - (4e-3 if below == 27.5 else 0.4)
        room = 2 * 2.0 ** -19 * size + 2.0 ** -15 + (2.0 ** -11 if dtype == "bf16" else 0.0)
        err = np.abs(got[:, i] / want - 1)
        assert err.max() <= room, (i, err.max(), room)
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("dtype,span", [("bf16", 128), ("f32", 8)])
def test_attend_growing(cuda, tqlib, dtype, span):
    """Values that grow by 2^3 with every `span` steps of the tiles, and queries that like later tokens more: the references
    of a row move after sums of earlier steps have been put aside.  Room as above, with a span's 2^-20 a step."""
    heads, group, new = 2, 8, 32
    ctx = 6 * span * 128 + 77
    n = -(-ctx // BLOCK) * BLOCK
    g = np.random.default_rng(span)
    k, v = g.standard_normal((n, heads, D)), 1.0 + 0.3 * g.standard_normal((n, heads, D))
    at = np.arange(n)[:, None, None] // BLOCK * BLOCK / (128.0 * span)
    v *= 2.0 ** (3 * at)
    k[:, :, :1] = 4 * at
    layer = layer_with(cuda, tqlib, k, v)
    q = g.standard_normal((new, heads * group, D)).astype(np.float32)
    q[..., 0] = np.arange(heads * group) % 5 * 2.0  # (logits grow by up to 2.8 a span)
    t = cuda.from_numpy(q).cuda().to(cuda.bfloat16 if dtype == "bf16" else cuda.float32)
    row = g.permutation(n // BLOCK)
    order = np.argsort(row)  # (block row[j] holds tokens 16 j ..)
    for pool in (layer.k_cache, layer.v_cache):
        pool.copy_(pool.view(n // BLOCK, -1)[cuda.from_numpy(order).cuda()].reshape(-1))
    seqs = seqs_for(cuda, heads)
    got = attend(cuda, layer, t, new, row, ctx, seqs)
    kk, vv = values(layer)
    th = t.double().cpu().numpy()
    for i in (0, new - 1):
        want, size = counted(th[i], kk, vv, row, ctx - new + i + 1)
        big = np.abs(vv).max()
        assert (np.abs(want).max(1) > big / 40).all()
        room = (2 * 2.0 ** -19 * size + 2.0 ** -20 + span * 2.0 ** -20 + (2.0 ** -11 if dtype == "bf16" else 0.0)) * big
        err = np.abs(got[:, i] - want).max()
        assert err <= room, (i, err / big, room / big)
        assert np.array_equal(got[0], got[-1])
    assert tqlib.get_device_status() == 0
