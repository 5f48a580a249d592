"""GPU: decode attention over a shared prefix against fp64 softmax attention over the
values the cache stands for.

Tolerance: max over rows of the largest error over the row's largest value, 5e-3, the
bound of the decode kernels with bf16 data: the output is rounded to bf16 (half a step, 2^-8 of
the value, 3.9e-3); the code tables and the values are held in fp16 (half a step 2^-11 each,
with random signs over coordinates and tokens), and so are the weights; the queries in two
fp16 parts (2^-22)."""
import math

import numpy as np
import pytest

import workloads
from oracle import codebook as ocb, fp8 as ofp8, quantize as oq
from tests._gpu_util import D, max_rel_err, oracle_pi, page_fields
from tests._rope_ref import prefix_attention

pytestmark = pytest.mark.gpu

TOL = 5e-3
FORMATS = [("bf16", 4, 4), ("k8v4", 8, 4), ("k8v4", 8, 3), ("packed", 4, 4), ("packed", 3, 4), ("packed", 2, 2),
           ("packed", 3, 3), ("packed", 4, 2), ("packed", 2, 4)]


def stands_for(layer):
    """fp64 keys and values [blocks, Hkv, 16, D] (garbage where nothing was stored)."""
    out = []
    pi = oracle_pi(layer) if layer.kv_format != "bf16" else None
    for which, pool in enumerate((layer.k_cache, layer.v_cache)):
        host = pool.cpu().numpy()
        if layer.kv_format == "bf16":
            x = oq.bf16_bits_to_f64(host.view(np.uint16)).reshape(-1, layer.num_kv_heads, 16, D)
        elif layer.k8v4 and which == 0:
            x = ofp8.decode(host).reshape(-1, layer.num_kv_heads, 16, D)
        else:
            c = np.asarray(ocb.codebook_fp32(D, layer.bits_k if which == 0 else layer.bits_v)[0], np.float64)
            codes, gamma = page_fields(layer, which, host)[:2]
            x = (c[codes] * gamma[..., None].astype(np.float64)) @ pi
        out.append(x)
    return out


def build(cuda, tq, fmt, bk, bv, *, B, hq, hkv, P, lens, seed=0, q_dtype="bf16", heavy=False, width=None):
    lens = np.asarray(lens, np.int32)
    pb = -(-P // 16)
    width = (int(lens.max()) + 15) // 16 if width is None else width
    ids = workloads.rng(seed).permutation(pb + B * width + 3).astype(np.int32)
    ptab, table = ids[:pb], ids[pb:pb + B * width].reshape(B, width)
    # bytes that were never written are NaN in every format
    layer = tq.Layer(len(ids), hkv, kv_format=fmt, bits_k=bk, bits_v=bv, seed=seed + 5, layer=2, fill=0xFF)
    slots = [ptab[np.arange(P) // 16].astype(np.int64) * 16 + np.arange(P) % 16]
    slots += [table[b, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16 for b, n in enumerate(lens)]
    slots = np.concatenate(slots)
    if len(slots):
        kv = (workloads.heavy_tail_kv if heavy else workloads.lognormal_channel_kv)(seed + 1, len(slots), hkv, D)
        k, v = (cuda.from_numpy(x.view(np.int16)).cuda().view(cuda.bfloat16) for x in kv)
        layer.append(k, v, cuda.from_numpy(slots).cuda())
    q = cuda.from_numpy(workloads.queries(seed + 3, B, hq, D, dtype="f32")).cuda()
    return layer, (q if q_dtype == "f32" else q.to(cuda.bfloat16)), ptab, table, lens


def run(cuda, tq, case, P, out_dtype=None, **kw):
    layer, q, ptab, table, lens = case
    own = (None, None) if table.shape[1] == 0 else (cuda.from_numpy(table).cuda(), cuda.from_numpy(lens).cuda())
    out = layer.prefix_decode(q, cuda.from_numpy(ptab).cuda(), P, *own, out_dtype=out_dtype, **kw)
    cuda.cuda.synchronize()
    assert tq.get_device_status() == 0
    return out


def check(cuda, tq, case, P, out_dtype=None):
    layer, q, ptab, table, lens = case
    out = run(cuda, tq, case, P, out_dtype)
    ref = prefix_attention(q.double().cpu().numpy(), *stands_for(layer), ptab, P, table, lens, 1 / math.sqrt(D))
    got = out.float().cpu().numpy()
    empty = (lens == 0) & (P == 0)
    assert np.all(got[empty] == 0.0)
    if not empty.all():
        err = max_rel_err(got[~empty], ref[~empty])
        print("max rel err %.3e" % err)
        assert err <= TOL


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
@pytest.mark.parametrize("P", [1, 15, 16, 17, 127, 128, 129, 333, 1000])
def test_prefix_lengths(cuda, tqlib, fmt, bk, bv, P):
    case = build(cuda, tqlib, fmt, bk, bv, B=3, hq=8, hkv=2, P=P, lens=[40, 0, 7], seed=P)
    check(cuda, tqlib, case, P)


@pytest.mark.parametrize("fmt,bk,bv", [("bf16", 4, 4), ("k8v4", 8, 4), ("packed", 4, 4), ("packed", 3, 4)])
@pytest.mark.parametrize("B,hq,hkv", [(1, 1, 1), (1, 32, 8), (5, 7, 1), (9, 24, 2), (33, 16, 4), (64, 5, 1), (70, 16, 2),
                                      (130, 12, 1)])
def test_rows_and_groups(cuda, tqlib, fmt, bk, bv, B, hq, hkv):
    """From one row a KV head over odd groups to several tiles of rows with a ragged last one."""
    lens = workloads.rng(B).integers(0, 30, B)
    case = build(cuda, tqlib, fmt, bk, bv, B=B, hq=hq, hkv=hkv, P=300, lens=lens, seed=B + hq)
    check(cuda, tqlib, case, 300)


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
@pytest.mark.parametrize("q_dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_types(cuda, tqlib, fmt, bk, bv, q_dtype, out):
    case = build(cuda, tqlib, fmt, bk, bv, B=4, hq=8, hkv=2, P=210, lens=[3, 50, 0, 17], seed=9, q_dtype=q_dtype,
                 heavy=True)
    check(cuda, tqlib, case, 210, getattr(cuda, {"f32": "float32", "bf16": "bfloat16"}[out]))


@pytest.mark.parametrize("fmt,bk,bv", [("bf16", 4, 4), ("k8v4", 8, 4), ("packed", 3, 4)])
def test_without_prefix_or_own_tokens(cuda, tqlib, fmt, bk, bv):
    tq = tqlib
    for P, lens in ((0, [20, 0, 1]), (100, [0, 0, 0]), (0, [0, 0, 0])):
        for width in (None, 2):
            case = build(cuda, tq, fmt, bk, bv, B=3, hq=4, hkv=2, P=P, lens=lens, seed=4, width=width if max(lens) == 0 else None)
            check(cuda, tq, case, P)


def test_long_prefix_over_many_splits(cuda, tqlib):
    case = build(cuda, tqlib, "packed", 4, 4, B=2, hq=8, hkv=2, P=20011, lens=[100, 3], seed=11)
    check(cuda, tqlib, case, 20011)
    case = build(cuda, tqlib, "bf16", 4, 4, B=40, hq=8, hkv=1, P=9000, lens=[5] * 40, seed=12)
    check(cuda, tqlib, case, 9000)


@pytest.mark.parametrize("fmt,bk,bv", [("bf16", 4, 4), ("k8v4", 8, 4), ("packed", 4, 4)])
def test_sharp_and_graded_logits(cuda, tqlib, fmt, bk, bv):
    """Keys that grow along the prefix, so that the running maximum moves in every tile, and value
    norms over seven decades: the rows' sums are rescaled again and again."""
    tq = tqlib
    P, B, hq, hkv = 700, 2, 4, 1
    layer = tq.Layer(60, hkv, kv_format=fmt, bits_k=bk, bits_v=bv, seed=1, fill=0xFF)
    g = workloads.rng(2)
    base = g.standard_normal(D)
    k = base[None] * np.linspace(0.05, 3.0, P)[:, None] + 0.1 * g.standard_normal((P, D))
    v = g.standard_normal((P, D)) * 10.0 ** np.linspace(-4, 3, P)[:, None]
    ids = g.permutation(60).astype(np.int32)
    pb = -(-P // 16)
    slots = ids[np.arange(P) // 16].astype(np.int64) * 16 + np.arange(P) % 16
    to = lambda x: cuda.from_numpy(x[:, None].astype(np.float32)).cuda()
    layer.append(to(k), to(v), cuda.from_numpy(slots).cuda())
    for sign in (1.0, -1.0):
        q = cuda.from_numpy((sign * base * np.ones((B, hq, 1)) + 0.05 * g.standard_normal((B, hq, D))).astype(np.float32)).cuda()
        q = q.to(cuda.bfloat16)
        case = layer, q, ids[:pb], np.zeros((B, 0), np.int32), np.zeros(B, np.int32)
        check(cuda, tq, case, P, cuda.float32)


def test_agrees_with_decode_over_the_joined_table(cuda, tqlib):
    """A prefix of whole blocks is what decode computes with the prefix's blocks in every row."""
    tq = tqlib
    for fmt, bk, bv in FORMATS:
        P = 160
        case = build(cuda, tq, fmt, bk, bv, B=5, hq=8, hkv=2, P=P, lens=[33, 1, 16, 40, 2], seed=6)
        layer, q, ptab, table, lens = case
        out = run(cuda, tq, case, P, cuda.float32)
        joined = np.concatenate([np.tile(ptab, (5, 1)), table], 1)
        ref = layer.decode(q, cuda.from_numpy(joined).cuda(), cuda.from_numpy(lens + P).cuda(), out_dtype=cuda.float32)
        assert max_rel_err(out.cpu().numpy(), ref.cpu().numpy()) <= 2 * TOL


def test_workspace_serves_both_calls_and_repeats(cuda, tqlib):
    """One workspace through prefix calls of several sizes and plain decodes, each result the same
    bits as with a workspace of its own; and the same call twice gives the same bits."""
    tq = tqlib
    big = cuda.zeros(64 << 20, dtype=cuda.uint8, device="cuda")
    for fmt, bk, bv, B, P, lens in (("packed", 4, 4, 4, 500, [9, 0, 60, 31]), ("packed", 3, 4, 2, 90, [0, 0]),
                                    ("bf16", 4, 4, 40, 200, [3] * 40), ("k8v4", 8, 4, 3, 2000, [100, 5, 0])):
        case = build(cuda, tq, fmt, bk, bv, B=B, hq=8, hkv=2, P=P, lens=lens, seed=P)
        layer, q, ptab, table, lens = case
        one = run(cuda, tq, case, P, workspace=big)
        assert cuda.equal(one, run(cuda, tq, case, P))
        assert cuda.equal(one, run(cuda, tq, case, P, workspace=big))
        if table.shape[1]:
            args = (q, cuda.from_numpy(table).cuda(), cuda.from_numpy(lens).cuda())
            assert cuda.equal(layer.decode(*args, workspace=big), layer.decode(*args))


@pytest.mark.parametrize("fmt,bk,bv", [("bf16", 4, 4), ("k8v4", 8, 4), ("packed", 4, 4), ("packed", 3, 4)])
@pytest.mark.parametrize("width", [127, 128, 129, 200])
def test_wide_block_tables(cuda, tqlib, fmt, bk, bv, width):
    """Block tables around the width from which the decode kernel takes the own tokens, with a full, a
    short and an empty sequence."""
    case = build(cuda, tqlib, fmt, bk, bv, B=3, hq=8, hkv=1, P=150, lens=[16 * width - 3, 20, 0], seed=width,
                 width=width)
    check(cuda, tqlib, case, 150)


@pytest.mark.parametrize("fmt,bk,bv", [("bf16", 4, 4), ("k8v4", 8, 4), ("packed", 4, 4)])
@pytest.mark.parametrize("scale", [-0.05, 0.0, 0.3])
def test_scales_of_any_sign(cuda, tqlib, fmt, bk, bv, scale):
    P = 200
    case = build(cuda, tqlib, fmt, bk, bv, B=3, hq=8, hkv=2, P=P, lens=[20, 0, 33], seed=3, heavy=True)
    layer, q, ptab, table, lens = case
    out = run(cuda, tqlib, case, P, cuda.float32, sm_scale=scale)
    ref = prefix_attention(q.double().cpu().numpy(), *stands_for(layer), ptab, P, table, lens, scale)
    assert max_rel_err(out.cpu().numpy(), ref) <= TOL


def test_bad_context_lengths_are_clamped_and_flagged(cuda, tqlib):
    """As in decode: a negative length counts as none, one past the table as the whole table."""
    tq = tqlib
    for fmt, bk, bv in FORMATS:
        layer, q, ptab, table, lens = build(cuda, tq, fmt, bk, bv, B=3, hq=4, hkv=2, P=40, lens=[32, 32, 5], seed=8)
        out = layer.prefix_decode(q, cuda.from_numpy(ptab).cuda(), 40, cuda.from_numpy(table).cuda(),
                                  cuda.tensor([-4, 1000, 5], dtype=cuda.int32, device="cuda"), out_dtype=cuda.float32)
        cuda.cuda.synchronize()
        assert tq.get_device_status() == tq.TQ_DEV_BAD_CONTEXT
        ref = prefix_attention(q.double().cpu().numpy(), *stands_for(layer), ptab, 40, table, np.array([0, 32, 5]),
                               1 / math.sqrt(D))
        assert max_rel_err(out.cpu().numpy(), ref) <= TOL


def test_bad_own_blocks_are_skipped_and_flagged(cuda, tqlib):
    tq = tqlib
    for fmt, bk, bv in FORMATS:
        layer, q, ptab, table, lens = build(cuda, tq, fmt, bk, bv, B=2, hq=4, hkv=2, P=40, lens=[48, 20], seed=8)
        bad = table.copy()
        bad[0, 1], bad[1, 0] = layer.num_blocks + 7, -2
        out = layer.prefix_decode(q, cuda.from_numpy(ptab).cuda(), 40, cuda.from_numpy(bad).cuda(),
                                  cuda.from_numpy(lens).cuda(), out_dtype=cuda.float32)
        cuda.cuda.synchronize()
        assert tq.get_device_status() == tq.TQ_DEV_BAD_BLOCK
        left = np.stack([table[0, [0, 2, 2]], table[1, [1, 1, 1]]])
        ref = prefix_attention(q.double().cpu().numpy(), *stands_for(layer), ptab, 40, left, np.array([32, 4]),
                               1 / math.sqrt(D))
        assert max_rel_err(out.cpu().numpy(), ref) <= TOL


def test_unaligned_output_and_raw_norms(cuda, tqlib):
    tq = tqlib
    P = 100
    layer, q, ptab, table, lens = case = build(cuda, tq, "packed", 4, 4, B=3, hq=4, hkv=2, P=P, lens=[9, 0, 17], seed=2)
    for dtype in (cuda.bfloat16, cuda.float32):
        want = run(cuda, tq, case, P, dtype)
        flat = cuda.zeros(q.numel() + 1, dtype=dtype, device="cuda")
        out = flat[1:].view(q.shape)
        run(cuda, tq, case, P, out=out)
        assert cuda.equal(out, want)
    raw = tq.Layer(10, 1, bits_k=3, bits_v=2, norm_mode=tq.TQ_NORM_RAW, seed=4, fill=0xFF)
    k, v = (cuda.from_numpy(x.view(np.int16)).cuda().view(cuda.bfloat16) for x in workloads.lognormal_channel_kv(3, 70, 1, D))
    pos = cuda.arange(70, device="cuda")
    raw.rope_append(tq.Rope(), k, v, pos, pos)
    q1 = cuda.from_numpy(workloads.queries(5, 2, 3, D, dtype="f32")).cuda()
    ids = cuda.arange(5, dtype=cuda.int32, device="cuda")
    out = raw.prefix_decode(q1, ids, 70)
    ref = prefix_attention(q1.double().cpu().numpy(), *stands_for(raw), np.arange(5), 70, np.zeros((2, 0), np.int32),
                           np.zeros(2, np.int32), 1 / math.sqrt(D))
    assert max_rel_err(out.cpu().numpy(), ref) <= TOL


def test_example_runs_the_operators_together(cuda, tqlib):
    from examples import shared_prefix
    assert shared_prefix.main(batch=3, prompt=120, steps=3, verbose=False) <= 2 * TOL


def test_bad_prefix_blocks_are_skipped_and_flagged(cuda, tqlib):
    tq = tqlib
    for fmt, bk, bv in FORMATS:
        layer, q, ptab, table, lens = build(cuda, tq, fmt, bk, bv, B=2, hq=4, hkv=2, P=64, lens=[5, 0], seed=8)
        bad = ptab.copy()
        bad[1], bad[2] = -1, layer.num_blocks
        out = layer.prefix_decode(q, cuda.from_numpy(bad).cuda(), 64, cuda.from_numpy(table).cuda(),
                                  cuda.from_numpy(lens).cuda(), out_dtype=cuda.float32)
        cuda.cuda.synchronize()
        assert tq.get_device_status() == tq.TQ_DEV_BAD_BLOCK
        ref = prefix_attention(q.double().cpu().numpy(), *stands_for(layer), ptab[[0, 3]], 32, table, lens,
                               1 / math.sqrt(D))
        assert max_rel_err(out.cpu().numpy(), ref) <= TOL


@pytest.mark.parametrize("fmt,bk,bv", [("bf16", 4, 4), ("k8v4", 8, 4), ("packed", 4, 4), ("packed", 3, 2)])
@pytest.mark.parametrize("B,P", [(24, 3000), (80, 900)])
def test_many_own_tokens_beside_the_prefix(cuda, tqlib, fmt, bk, bv, B, P):
    """Enough CTAs of own tokens that the prefix is cut into fewer splits and both kernels run at
    once: right, the same bits in calls that follow one another without a pause, and the
    workspace serves the call without own tokens."""
    tq = tqlib
    lens = workloads.rng(B).integers(0, 1500, B)
    lens[:3] = 0, 1500, 1
    case = build(cuda, tq, fmt, bk, bv, B=B, hq=16, hkv=4, P=P, lens=lens, seed=B)
    check(cuda, tq, case, P)
    layer, q, ptab, table, lens = case
    p, t, n = (cuda.from_numpy(x).cuda() for x in (ptab, table, lens))
    ws = cuda.zeros(layer.prefix_workspace_bytes(B, 16, P, table.shape[1]), dtype=cuda.uint8, device="cuda")
    outs = [layer.prefix_decode(q, p, P, t, n, workspace=ws) for _ in range(20)]
    alone = layer.prefix_decode(q, p, P, workspace=ws)
    cuda.cuda.synchronize()
    assert tq.get_device_status() == 0
    assert all(cuda.equal(o, outs[0]) for o in outs[1:])
    none = np.zeros((B, 0), np.int32)
    ref = prefix_attention(q.double().cpu().numpy(), *stands_for(layer), ptab, P, none, np.zeros(B, np.int32),
                           1 / math.sqrt(D))
    assert max_rel_err(alone.float().cpu().numpy(), ref) <= TOL


def test_capture_on_a_side_stream(cuda, tqlib):
    tq = tqlib
    case = build(cuda, tq, "packed", 4, 4, B=6, hq=8, hkv=2, P=333, lens=[1, 2, 3, 40, 0, 9], seed=21)
    layer, q, ptab, table, lens = case
    dev = [cuda.from_numpy(x).cuda() for x in (ptab, table, lens)]
    ws = cuda.zeros(layer.prefix_workspace_bytes(6, 8, 333, table.shape[1]), dtype=cuda.uint8, device="cuda")
    out = cuda.empty_like(q)
    cuda.cuda.synchronize()
    side = cuda.cuda.Stream()
    graph = cuda.cuda.CUDAGraph()
    with cuda.cuda.stream(side):
        layer.prefix_decode(q, dev[0], 333, dev[1], dev[2], out=out, workspace=ws)
        side.synchronize()
        with cuda.cuda.graph(graph, stream=side):
            layer.prefix_decode(q, dev[0], 333, dev[1], dev[2], out=out, workspace=ws)
    q.copy_(-q)
    cuda.cuda.synchronize()
    graph.replay()
    cuda.cuda.synchronize()
    assert cuda.equal(out, run(cuda, tq, case, 333))


def test_binding_refuses_wrong_tensors(cuda, tqlib):
    tq = tqlib
    layer, q, ptab, table, lens = build(cuda, tq, "packed", 4, 4, B=2, hq=4, hkv=2, P=64, lens=[5, 20], seed=8)
    p, t, n = (cuda.from_numpy(x).cuda() for x in (ptab, table, lens))
    for args, err in (((q, p[:3], 64, t, n), ValueError), ((q, p.long(), 64, t, n), TypeError),
                      ((q, p, 64, t.long(), n), TypeError), ((q, p, 64, t[:1], n), ValueError),
                      ((q, p, 64, t, n[:1]), ValueError), ((q, p, 64, t), ValueError), ((q.half(), p, 64, t, n), TypeError)):
        with pytest.raises(err):
            layer.prefix_decode(*args)
    small = cuda.zeros(1024, dtype=cuda.uint8, device="cuda")
    with pytest.raises(tq.TQError) as e:
        layer.prefix_decode(q, p, 64, t, n, workspace=small)
    assert e.value.status == tq.TQ_ERR_WORKSPACE
