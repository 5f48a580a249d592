"""GPU: rotated appends large enough that the rows (queries, FP8 keys) go in a kernel of their own before the
codes: 2^17 rows of heads and more.  Tolerances as in test_gpu_rope.py."""
import numpy as np
import pytest

import workloads
from tests._gpu_util import D
from tests._rope_ref import frequencies, rotate
from tests.test_gpu_rope import check_rows, check_stored, draw, f64

pytestmark = pytest.mark.gpu

CODED = [("packed", 4, 4), ("packed", 3, 2), ("k8v4", 8, 4), ("k8v4", 8, 3)]


def make(cuda, tq, fmt, bk, bv, n, hq, hkv, rotary, layout, dtype, skip):
    blocks = -(-n // 16) + 3
    layer = tq.Layer(blocks, hkv, kv_format=fmt, bits_k=bk, bits_v=bv, seed=2, layer=1, fill=0xA5)
    qkv = draw(cuda, (n, hq + 2 * hkv, D), dtype, n)
    g = workloads.rng(n + 1)
    pos = g.integers(0, 1 << 17, n)
    slots = g.permutation(blocks * 16)[:n].astype(np.int64)
    slots[g.permutation(n)[:skip]] = -1
    return layer, tq.Rope(rotary, 10000.0, layout=layout), qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, slots


@pytest.mark.parametrize("fmt,bk,bv", CODED)
@pytest.mark.parametrize("n,hq,hkv,rotary,layout,dtype", [
    (4097, 32, 2, 128, "half", "bf16"),           # just past the threshold
    (9001, 32, 2, 128, "half", "bf16"),
    (5003, 64, 2, 96, "half", "f32"),
    (140003, 2, 1, 64, "interleaved", "bf16"),    # tiles of eight tokens
    (4100, 64, 1, 34, "half", "bf16"),            # one pair an item
])
def test_rows_apart_match_the_definition(cuda, tqlib, fmt, bk, bv, n, hq, hkv, rotary, layout, dtype):
    tq = tqlib
    layer, rope, q, k, v, pos, slots = make(cuda, tq, fmt, bk, bv, n, hq, hkv, rotary, layout, dtype, 300)
    p, s = cuda.from_numpy(pos).cuda(), cuda.from_numpy(slots).cuda()
    k_out = cuda.full((n, hkv, D), 7.0, dtype=q.dtype, device="cuda")
    n0 = tq.launch_count()
    q_out = layer.rope_append(rope, k, v, p, s, q=q, k_out=k_out)
    assert tq.launch_count() - n0 == 2
    cuda.cuda.synchronize()
    assert tq.get_device_status() == 0
    f, amp = frequencies(rotary, 10000.0)
    check_rows(f64(q_out), f64(q), pos, f, amp, layout, rotary, dtype)
    check_rows(f64(k_out), f64(k), pos, f, amp, layout, rotary, dtype)
    check_stored(cuda, tq, layer, 0, rotate(f64(k), pos, f, amp, layout), slots, False)
    check_stored(cuda, tq, layer, 1, f64(v), slots, True)


@pytest.mark.parametrize("fmt,bk,bv", CODED)
def test_rows_apart_in_place_repeated_and_captured(cuda, tqlib, fmt, bk, bv):
    """The pair of kernels in place; its records read at once by the call behind it, again and again; and
    captured into a graph that is replayed on other inputs: the same bits each time."""
    tq = tqlib
    n, hq, hkv = 9001, 32, 2
    layer, rope, q, k, v, pos, slots = make(cuda, tq, fmt, bk, bv, n, hq, hkv, 128, "half", "bf16", 0)
    p, s = cuda.from_numpy(pos).cuda(), cuda.from_numpy(slots).cuda()
    q_out = layer.rope_append(rope, k, v, p, s, q=q)
    want = layer.k_cache.clone(), layer.v_cache.clone()
    read = layer.dequantize(1, s, out_dtype=cuda.bfloat16)
    for _ in range(5):
        layer.k_cache.fill_(0xA5)
        layer.v_cache.fill_(0xA5)
        q2, k2 = q.clone(), k.clone()
        layer.rope_append(rope, k2, v, p, s, q=q2, q_out=q2, k_out=k2)
        again = layer.dequantize(1, s, out_dtype=cuda.bfloat16)
        assert cuda.equal(again, read) and cuda.equal(q2, q_out)
        assert cuda.equal(layer.k_cache, want[0]) and cuda.equal(layer.v_cache, want[1])
    side, graph = cuda.cuda.Stream(), cuda.cuda.CUDAGraph()
    out = cuda.empty_like(q_out)
    side.wait_stream(cuda.cuda.current_stream())
    with cuda.cuda.stream(side):
        layer.rope_append(rope, k, v, p, s, q=q, q_out=out)
        side.synchronize()
        with cuda.cuda.graph(graph, stream=side):
            layer.rope_append(rope, k, v, p, s, q=q, q_out=out)
            got = layer.dequantize(1, s, out_dtype=cuda.bfloat16)
    v.neg_()
    p += 5
    cuda.cuda.synchronize()
    graph.replay()
    cuda.cuda.synchronize()
    assert cuda.equal(out, tq.apply_rope(rope, p, q)[0])
    replayed = layer.k_cache.clone(), layer.v_cache.clone()
    layer.rope_append(rope, k, v, p, s, q=q)
    assert cuda.equal(layer.k_cache, replayed[0]) and cuda.equal(layer.v_cache, replayed[1])
    assert cuda.equal(got, layer.dequantize(1, s, out_dtype=cuda.bfloat16))
