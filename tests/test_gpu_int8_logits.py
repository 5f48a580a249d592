"""int8 layers with large logits: rows whose weights go to one token give that token's value, whatever the size of the logits."""
import numpy as np
import pytest

from tests.test_gpu_int8_long import BLOCK, D, SCALE, attend, layer_with, seqs_for, values

pytestmark = pytest.mark.gpu


def inputs(cuda, tq, seed, heads, group, new, ctx, dtype, power, least):
    """A layer, queries (times 2^power) and rows [new, Hq, D] that one token decides, NaN for the others: its logit is the
    largest by 2^-12 of the row's largest sum of magnitudes (what fp32 sums leave of a logit is well within), and by `least`."""
    g = np.random.default_rng(seed)
    n = -(-ctx // BLOCK) * BLOCK
    v = g.standard_normal((n, heads, D)) * 2.0 ** g.integers(-3, 4, (n // BLOCK, 1, 1)).repeat(BLOCK, 0)
    layer = layer_with(cuda, tq, g.standard_normal((n, heads, D)), v)
    q = cuda.from_numpy((g.standard_normal((new, heads * group, D)) * 2.0 ** power).astype(np.float32)).cuda().to(dtype)
    kk, vv = (x.transpose(1, 0, 2, 3).reshape(heads, n, D) for x in values(layer))
    qh, want = q.double().cpu().numpy(), np.full((new, heads * group, D), np.nan)
    for i in range(new):
        lim = ctx - new + i + 1
        for h in range(heads * group):
            s = kk[h // group, :lim] @ qh[i, h] * SCALE
            size = (np.abs(kk[h // group, :lim]) @ np.abs(qh[i, h])).max() * SCALE
            top = np.argsort(s)[-2:]
            if s[top[1]] - s[top[0]] > max(2.0 ** -12 * size, least):
                want[i, h] = vv[h // group, top[1]]
    return layer, q, want


def check(got, want, half):
    fine = ~np.isnan(want[..., 0])
    assert fine.mean() > 0.6
    err = np.abs(got - want).max(-1) / np.abs(want).max(-1)
    assert (err[fine] <= half).all(), float(np.nanmax(np.where(fine, err, 0.0)))  # (a result that is NaN fails)


POWERS = [9, 12, 16, 18, 20, 24, 30, 60, 110]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("power", POWERS)
def test_decode(cuda, tqlib, power, group, dtype):
    """Room: two parts of a weight, and the rest as above."""
    t = cuda.bfloat16 if dtype == "bf16" else cuda.float32
    heads, ctx = 3, 700
    layer, q, want = inputs(cuda, tqlib, 50 + power, heads, group, 1, ctx, t, power, 30.0)
    seqs = 5
    table = cuda.arange(layer.num_blocks, dtype=cuda.int32, device="cuda").expand(seqs, -1).contiguous()
    lens = cuda.full((seqs,), ctx, dtype=cuda.int32, device="cuda")
    got = layer.decode(q.expand(seqs, -1, -1).contiguous(), table, lens, out_dtype=cuda.float32).cpu().numpy()
    for b in range(seqs):
        check(got[b:b + 1], want, 2.0 ** -15)
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", POWERS)
def test_attend(cuda, tqlib, power, dtype):
    """Room: half a step of a weight's type, 2^-11 in fp16 or 2^-22 in two parts; for steps by logarithms 2^-13 more (references
    below 2^11); 2^-15 for what the accumulators cut off and the weights of 2^-22 and less that others keep."""
    heads, group, new = 4, 8, 32
    t = cuda.bfloat16 if dtype == "bf16" else cuda.float32
    layer, q, want = inputs(cuda, tqlib, power, heads, group, new, 700, t, power, 30.0)
    row = np.arange(layer.num_blocks)
    got = attend(cuda, layer, q, new, row, 700, seqs_for(cuda, heads))
    assert np.array_equal(got[0], got[-1])
    check(got[0], want, 2.0 ** -15 + (2.0 ** -11 + 2.0 ** -13 if dtype == "bf16" else 2.0 ** -22))
    assert tqlib.get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [12, 17, 19, 40])
def test_attend_repeats(cuda, tqlib, power, dtype):
    """The same blocks three times over: copies of the token that decides stand in later steps too, whose references have been
    found by then.  Room as above."""
    heads, group, new, n = 4, 8, 32, 12 * BLOCK
    t = cuda.bfloat16 if dtype == "bf16" else cuda.float32
    layer, q, want = inputs(cuda, tqlib, 90 + power, heads, group, 1, n, t, power, 30.0)
    row = np.tile(np.arange(n // BLOCK), 30)
    got = attend(cuda, layer, q.expand(new, -1, -1).contiguous(), new, row, 30 * n - 3, seqs_for(cuda, heads))
    room = 2.0 ** -15 + (2.0 ** -11 + 2.0 ** -13 if dtype == "bf16" else 2.0 ** -22)
    for i in (0, new - 1):
        check(got[0, i:i + 1], want, room)
    assert tqlib.get_device_status() == 0
