"""GPU: rotary positions and the rotated append against their fp64 definitions.

Tolerances.  The angle is exact to 2^-64 turns a position, rounded once to fp32 (at most
2^-25 half turns, 9.4e-8 rad); sine, cosine, their product with the amplitude and the two
products and the sum of a pair add a few fp32 half steps (6e-8 each): ROT = 8e-7 of the
pair's length covers them.  Results rounded to bf16 add half a step, 2^-8 of the value
(taken as finfo.eps / 2), FP8 E4M3 2^-4 of it and 2^-10 below its normal range."""
import numpy as np
import pytest

import workloads
from oracle import codebook as ocb, fp8 as ofp8, quantize as oq
from tests._gpu_util import D, oracle_pi, page_fields, slot_fields, tie_band_ok
from tests._rope_ref import frequencies, pair_norm, rotate

pytestmark = pytest.mark.gpu

ROT = 8e-7
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}
YARN = {"kind": "yarn", "factor": 16.0, "low": 1.0, "high": 32.0, "length": 4096}


def draw(cuda, shape, dtype, seed):
    x = cuda.from_numpy(workloads.rng(seed).standard_normal(shape, dtype=np.float32)).cuda()
    return x if dtype == "f32" else x.to(cuda.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def check_rows(got, x, pos, f, amp, layout, rotary, dtype, transpose=False):
    want = rotate(x, pos, f, amp, layout, transpose)
    bound = HALF[dtype] * np.abs(want) * (1 + ROT) + ROT * amp * pair_norm(x, rotary, layout)
    bound[..., rotary:] = 0.0  # what passes through is copied
    bad = np.abs(got - want) > bound
    assert not bad.any(), (np.argwhere(bad)[:4], np.max(np.abs(got - want)))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rotary", [2, 32, 62, 96, 126, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_apply_matches_definition(cuda, tqlib, layout, rotary, dtype):
    tq = tqlib
    rope = tq.Rope(rotary, 10000.0, layout=layout, scaling=YARN)
    f, amp = frequencies(rotary, 10000.0, YARN)
    n, hq, hk = 37, 5, 2
    qkv = draw(cuda, (n, hq + 2 * hk, D), dtype, rotary)  # q and k are views of one projection
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    pos = cuda.from_numpy(workloads.rng(3).integers(-5, 1 << 20, n)).cuda()
    before = qkv.clone()
    for transpose in (False, True):
        qo, ko = tq.apply_rope(rope, pos, q, k, transpose=transpose)
        for got, x in ((qo, q), (ko, k)):
            assert got.is_contiguous() and got.dtype == x.dtype
            check_rows(f64(got), f64(x), pos.cpu().numpy(), f, amp, layout, rotary, dtype, transpose)
    assert cuda.equal(qkv, before)


@pytest.mark.parametrize("n,hq,hk", [(0, 4, 2), (1, 1, 1), (3, 64, 8), (700, 3, 1), (2500, 32, 8)])
def test_apply_sizes_and_single_tensors(cuda, tqlib, n, hq, hk):
    tq = tqlib
    rope = tq.Rope()
    f, amp = frequencies(128, 10000.0)
    q, k = draw(cuda, (n, hq, D), "bf16", n + 1), draw(cuda, (n, hk, D), "bf16", n + 2)
    pos = cuda.arange(n, device="cuda") * 3
    qo, ko = tq.apply_rope(rope, pos, q, k)
    only_q, none = tq.apply_rope(rope, pos, q)
    assert none is None and cuda.equal(only_q, qo)
    assert cuda.equal(tq.apply_rope(rope, pos, None, k)[1], ko)
    check_rows(f64(qo), f64(q), pos.cpu().numpy(), f, amp, "half", 128, "bf16")
    check_rows(f64(ko), f64(k), pos.cpu().numpy(), f, amp, "half", 128, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout,rotary", [("half", 128), ("half", 64), ("half", 126), ("interleaved", 128),
                                           ("interleaved", 50)])
def test_apply_strides_alignment_and_in_place(cuda, tqlib, layout, rotary, dtype):
    """Rows one element off alignment, heads before tokens, and the rotation in place give what
    contiguous rows give, bit for bit."""
    tq = tqlib
    rope = tq.Rope(rotary, 500.0, layout=layout)
    n, h = 41, 3
    x = draw(cuda, (n, h, D), dtype, 5)
    pos = cuda.from_numpy(workloads.rng(4).integers(0, 100000, n)).cuda()
    want = tq.apply_rope(rope, pos, x)[0]
    odd = cuda.zeros(n * h * (D + 1) + 1, dtype=x.dtype, device="cuda")[1:].view(n, h, D + 1)[..., :D]
    odd.copy_(x)
    turned = cuda.zeros((h, n, D), dtype=x.dtype, device="cuda").transpose(0, 1)
    turned.copy_(x)
    for src in (odd, turned):
        assert cuda.equal(tq.apply_rope(rope, pos, src)[0], want)
        dst = cuda.zeros_like(odd)
        tq.apply_rope(rope, pos, x, q_out=dst)
        assert cuda.equal(dst.contiguous(), want)
        tq.apply_rope(rope, pos, src, q_out=src)
        assert cuda.equal(src.contiguous(), want)


def test_apply_far_positions(cuda, tqlib):
    """Positions past 2^31 keep the precision of near ones: the definition in exact arithmetic."""
    tq = tqlib
    rope = tq.Rope(128, 10000.0)
    pos = np.array([0, 1, 2 ** 24 + 1, 2 ** 31 + 7, 2 ** 40 + 3, -(2 ** 33)], np.int64)
    x = draw(cuda, (len(pos), 2, D), "f32", 8)
    got = f64(tq.apply_rope(rope, cuda.from_numpy(pos).cuda(), x)[0])
    turns = np.array([[(int(p) * int(t)) % 2 ** 64 / 2.0 ** 64 for t in rope.desc.turns] for p in pos])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    xs = f64(x)
    want = np.concatenate([xs[..., :64] * c - xs[..., 64:] * s, xs[..., 64:] * c + xs[..., :64] * s], -1)
    assert np.all(np.abs(got - want) <= ROT * pair_norm(xs, 128, "half"))


@pytest.mark.parametrize("layout,rotary", [("half", 128), ("half", 96), ("interleaved", 64)])
def test_transpose_is_the_gradient(cuda, tqlib, layout, rotary):
    """<g, R(x + d) - R(x - d)> / 2 = <R^T g, d> (R is linear: the central difference is exact up to
    rounding), and R^T R = A^2 on the rotated coordinates."""
    tq = tqlib
    rope = tq.Rope(rotary, 10000.0, layout=layout, scaling=YARN)
    n, h = 9, 4
    pos = cuda.arange(n, device="cuda") * 1237
    x, d, g = (draw(cuda, (n, h, D), "f32", s) for s in (1, 2, 3))
    run = lambda t, tr=False: tq.apply_rope(rope, pos, t, transpose=tr)[0].double()
    left = (g.double() * (run(x + d) - run(x - d))).sum(-1) / 2
    right = (run(g, True) * d.double()).sum(-1)
    # each of 128 products is off by ROT of the pairs' lengths and the inputs' sums by 2^-24
    scale = (g.double().abs().sum(-1) * (x.double().abs() + d.double().abs()).amax(-1)) * rope.amplitude
    assert bool(((left - right).abs() <= 4 * ROT * scale).all())
    back = run(run(x).float(), True)
    want = x.double() * cuda.where(cuda.arange(D, device="cuda") < rotary, rope.amplitude ** 2, 1.0)
    assert bool(((back - want).abs() <= 4 * ROT * rope.amplitude ** 2 * cuda.from_numpy(pair_norm(f64(x), rotary, layout)).cuda()).all())


def test_apply_nan_and_inf_stay_in_their_pairs(cuda, tqlib):
    tq = tqlib
    for layout in ("half", "interleaved"):
        rope = tq.Rope(64, layout=layout)
        x = draw(cuda, (4, 2, D), "bf16", 3)
        x[1, 0, 100] = float("nan")  # passes through
        x[2, 1, 70] = float("inf")
        x[3, 0, 5] = float("nan")  # in a pair
        y = tq.apply_rope(rope, cuda.arange(4, device="cuda") + 11, x)[0]
        bad = cuda.nonzero(~cuda.isfinite(y)).tolist()
        pair = [[3, 0, 5], [3, 0, 37]] if layout == "half" else [[3, 0, 4], [3, 0, 5]]
        assert bad == [[1, 0, 100], [2, 1, 70]] + pair
        assert float(y[2, 1, 70]) == float("inf")


# ------------------------------------------------------------- rotated append

FORMATS = [("bf16", 4, 4), ("k8v4", 8, 4), ("k8v4", 8, 2), ("packed", 4, 4), ("packed", 3, 4), ("packed", 2, 2),
           ("packed", 4, 3)]


def append_case(cuda, tq, fmt, bk, bv, *, n, hq, hkv, layout, rotary, dtype, skip=0, seed=0, scale=1.0):
    blocks = -(-n // 16) + 3
    layer = tq.Layer(blocks, hkv, kv_format=fmt, bits_k=bk, bits_v=bv, seed=seed + 2, layer=1, fill=0xA5)
    rope = tq.Rope(rotary, 10000.0, layout=layout)
    qkv = draw(cuda, (n, hq + 2 * hkv, D), dtype, seed) * scale
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    g = workloads.rng(seed + 1)
    pos = g.integers(0, 1 << 17, n)
    slots = g.permutation(blocks * 16)[:n].astype(np.int64)
    slots[g.permutation(n)[:skip]] = -1
    pos_d, slots_d = cuda.from_numpy(pos).cuda(), cuda.from_numpy(slots).cuda()
    k_out = cuda.full((n, hkv, D), 7.0, dtype=q.dtype, device="cuda")
    n0 = tq.launch_count()
    q_out = layer.rope_append(rope, k, v, pos_d, slots_d, q=q if hq else None, k_out=k_out)
    assert tq.launch_count() - n0 == (1 if n else 0)
    cuda.cuda.synchronize()
    assert tq.get_device_status() == 0
    return layer, rope, q, k, v, pos, slots, q_out, k_out


def check_stored(cuda, tq, layer, which, x, slots, exact_in):
    """x fp64 [n, hkv, D]: what the records at the live slots were made of; every other byte of the
    pool keeps its fill."""
    pool = (layer.k_cache if which == 0 else layer.v_cache).cpu().numpy()
    live = slots >= 0
    sl = slots[live]
    blk, off = sl // 16, sl % 16
    hkv = layer.num_kv_heads
    if layer.kv_format == "bf16" or (layer.k8v4 and which == 0):
        wide = layer.kv_format == "bf16"
        pages = pool.view(np.uint16 if wide else np.uint8).reshape(-1, hkv, 16, D)
        got = pages[blk, :, off]
        want = x[live]
        if wide:
            val, step, tiny = oq.bf16_bits_to_f64(got), 2.0 ** -8, 0.0
        else:
            val, step, tiny = ofp8.decode(got), 2.0 ** -4, 2.0 ** -10
            want = np.clip(want, -448, 448)
        slack = 0.0 if exact_in else ROT * 2 * np.max(np.abs(x), axis=-1, keepdims=True)[live]
        assert np.all(np.abs(val - want) <= step * np.abs(want) * (1 + ROT) + tiny + slack)
        mask = np.ones(pages.shape[:3], bool)
        mask[blk, :, off] = False
        assert np.all(pages[mask] == (0xA5A5 if wide else 0xA5))
        return
    bits = layer.bits_k if which == 0 else layer.bits_v
    c, b = ocb.codebook_fp32(D, bits)
    codes, gamma = page_fields(layer, which, pool)[:2]
    pi = oracle_pi(layer)
    for h in range(hkv):
        got, gam = codes[blk, h, off], gamma[blk, h, off]
        idx, _, y = oq.quantize(x[live][:, h], pi, c, b)
        ok, _ = tie_band_ok(y, got, idx, b, 1e-5)
        assert ok
        n = np.linalg.norm(x[live][:, h], axis=-1)
        cn = np.linalg.norm(np.asarray(c, np.float64)[got], axis=-1)
        # n and |c| from fp32 sums of 128 squares, a square root and a division each
        assert np.all(np.abs(gam - n / cn) <= 4e-6 * n / cn)
    mask = np.ones(codes.shape[:3], bool)
    mask[blk, :, off] = False
    assert np.all(gamma[mask].astype(np.float32).view(np.uint32) == 0xA5A5A5A5)


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
@pytest.mark.parametrize("layout,rotary", [("half", 128), ("half", 64), ("half", 34), ("interleaved", 128),
                                           ("interleaved", 30)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_matches_definition(cuda, tqlib, fmt, bk, bv, layout, rotary, dtype):
    tq = tqlib
    layer, rope, q, k, v, pos, slots, q_out, k_out = append_case(
        cuda, tq, fmt, bk, bv, n=75, hq=6, hkv=3, layout=layout, rotary=rotary, dtype=dtype, skip=9, seed=rotary)
    f, amp = frequencies(rotary, 10000.0)
    check_rows(f64(q_out), f64(q), pos, f, amp, layout, rotary, dtype)
    check_rows(f64(k_out), f64(k), pos, f, amp, layout, rotary, dtype)
    check_stored(cuda, tq, layer, 0, rotate(f64(k), pos, f, amp, layout), slots, False)
    check_stored(cuda, tq, layer, 1, f64(v), slots, True)


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (1, 8, 8), (17, 0, 1), (130, 12, 1), (1000, 4, 2), (3000, 16, 12)])
def test_append_sizes(cuda, tqlib, fmt, bk, bv, n, hq, hkv):
    tq = tqlib
    layer, rope, q, k, v, pos, slots, q_out, k_out = append_case(
        cuda, tq, fmt, bk, bv, n=n, hq=hq, hkv=hkv, layout="half", rotary=128, dtype="bf16", skip=n // 5, seed=n)
    f, amp = frequencies(128, 10000.0)
    if hq:
        check_rows(f64(q_out), f64(q), pos, f, amp, "half", 128, "bf16")
    check_rows(f64(k_out), f64(k), pos, f, amp, "half", 128, "bf16")
    check_stored(cuda, tq, layer, 0, rotate(f64(k), pos, f, amp, "half"), slots, False)
    check_stored(cuda, tq, layer, 1, f64(v), slots, True)


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
def test_append_alone_in_place_and_unaligned(cuda, tqlib, fmt, bk, bv):
    """Keys alone, values alone, unaligned strided rows and rotation of q and k in place write the
    same bytes as the whole call."""
    tq = tqlib
    layer, rope, q, k, v, pos, slots, q_out, k_out = append_case(
        cuda, tq, fmt, bk, bv, n=90, hq=5, hkv=2, layout="half", rotary=64, dtype="bf16", seed=3)
    p, s = cuda.from_numpy(pos).cuda(), cuda.from_numpy(slots).cuda()
    want = layer.k_cache.clone(), layer.v_cache.clone()

    def fresh():
        layer.k_cache.fill_(0xA5)
        layer.v_cache.fill_(0xA5)

    def off(x):
        o = cuda.zeros((x.shape[0], x.shape[1], D + 1), dtype=x.dtype, device="cuda")
        o[..., 1:] = x
        return o[..., 1:]

    fresh()
    layer.rope_append(rope, k, None, p, s)
    assert cuda.equal(layer.k_cache, want[0]) and bool((layer.v_cache == 0xA5).all())
    layer.rope_append(rope, None, v, p, s)
    assert cuda.equal(layer.v_cache, want[1])
    fresh()
    assert cuda.equal(layer.rope_append(rope, off(k), off(v), p, s, q=off(q)), q_out)
    assert cuda.equal(layer.k_cache, want[0]) and cuda.equal(layer.v_cache, want[1])
    fresh()
    q2, k2 = q.clone(), k.clone()
    layer.rope_append(rope, k2, v, p, s, q=q2, q_out=q2, k_out=k2)
    assert cuda.equal(q2, q_out) and cuda.equal(k2, k_out)
    assert cuda.equal(layer.k_cache, want[0]) and cuda.equal(layer.v_cache, want[1])


def test_append_bad_slots_are_skipped_and_flagged(cuda, tqlib):
    tq = tqlib
    for fmt, bk, bv in FORMATS:
        layer = tq.Layer(2, 2, kv_format=fmt, bits_k=bk, bits_v=bv, fill=0xA5)
        x = draw(cuda, (3, 2, D), "bf16", 1)
        pos = cuda.arange(3, device="cuda")
        slots = cuda.tensor([32, 1 << 40, -7], device="cuda")
        layer.rope_append(tq.Rope(), x, x, pos, slots)
        assert tq.get_device_status() == tq.TQ_DEV_BAD_SLOT
        assert bool((layer.k_cache == 0xA5).all()) and bool((layer.v_cache == 0xA5).all())


def test_append_zero_vectors_and_large_values(cuda, tqlib):
    """A zero vector has norm 0 and the middle codes; FP8 keys saturate at 448."""
    tq = tqlib
    layer = tq.Layer(1, 1, bits_k=4, bits_v=3)
    z = cuda.zeros((2, 1, D), dtype=cuda.bfloat16, device="cuda")
    layer.rope_append(tq.Rope(), z, z, cuda.tensor([5, 9], device="cuda"), cuda.tensor([0, 3], device="cuda"))
    for which, mid in ((0, 8), (1, 4)):
        codes, gamma = page_fields(layer, which, (layer.k_cache, layer.v_cache)[which].cpu().numpy())[:2]
        assert np.all(codes[0, 0, [0, 3]] == mid) and np.all(gamma[0, 0, [0, 3]] == 0.0)
    k8 = tq.Layer(1, 1, kv_format="k8v4")
    x = cuda.full((1, 1, D), 1e4, dtype=cuda.bfloat16, device="cuda")
    k8.rope_append(tq.Rope(), x, x, cuda.zeros(1, dtype=cuda.int64, device="cuda"), cuda.zeros(1, dtype=cuda.int64, device="cuda"))
    assert bool((k8.k_cache[:D].view(cuda.float8_e4m3fn).float() == 448).all())


def test_calls_follow_their_stream(cuda, tqlib):
    """On a side stream, and captured into a graph that is replayed on new inputs."""
    tq = tqlib
    rope = tq.Rope(layout="interleaved")
    layer = tq.Layer(4, 2, bits_k=3)
    q, k, v = (draw(cuda, (20, h, D), "bf16", h) for h in (4, 2, 2))
    pos = cuda.arange(20, device="cuda")
    slots = cuda.arange(20, device="cuda") + 7
    q_out, k_out = cuda.empty_like(q), cuda.empty_like(k)
    side = cuda.cuda.Stream()
    side.wait_stream(cuda.cuda.current_stream())
    with cuda.cuda.stream(side):
        graph = cuda.cuda.CUDAGraph()
        tq.apply_rope(rope, pos, q, k, q_out=q_out, k_out=k_out)
        side.synchronize()
        with cuda.cuda.graph(graph, stream=side):
            layer.rope_append(rope, k, v, pos, slots, q=q, q_out=q_out, k_out=k_out)
    q.copy_(draw(cuda, q.shape, "bf16", 77))
    pos += 1000
    cuda.cuda.synchronize()
    graph.replay()
    cuda.cuda.synchronize()
    want = tq.apply_rope(rope, pos, q, k)
    assert cuda.equal(q_out, want[0]) and cuda.equal(k_out, want[1])


def test_binding_refuses_wrong_tensors(cuda, tqlib):
    tq = tqlib
    rope = tq.Rope()
    x = draw(cuda, (4, 2, D), "bf16", 1)
    pos = cuda.arange(4, device="cuda")
    for args, kw, err in (((pos.int(), x), {}, TypeError), ((pos[:3], x), {}, ValueError),
                          ((pos, x[..., :64]), {}, ValueError), ((pos, x.half()), {}, TypeError),
                          ((pos, x.cpu()), {}, ValueError), ((pos, x, x.float()), {}, TypeError),
                          ((pos, None), {}, ValueError), ((pos, x), {"q_out": x.float()}, ValueError),
                          ((pos, x.transpose(1, 2).contiguous().transpose(1, 2)), {}, ValueError)):
        with pytest.raises(err):
            tq.apply_rope(rope, *args, **kw)
    layer = tq.Layer(1, 2)
    with pytest.raises(tq.TQError):
        layer.rope_append(rope, x[:, :1], x[:, :1], pos, pos)
