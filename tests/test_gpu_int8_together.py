"""int8 layers and shared blocks in use: captured and replayed, on streams of their own, beside the calls that other
layers have too (append_decode, append_layers, offload, the call without a workspace), and together."""
import ctypes

import numpy as np
import pytest

from tests import _int8_ref as ref
from tests.test_gpu_int8 import BLOCK, D, SCALE, assert_pages, check_rows, data, dev, filled, host, layer_of, pages, tables

pytestmark = pytest.mark.gpu


def test_example(cuda, tqlib):
    """Weights of 16-bit queries in tiles go to fp16 (2^-11 of the largest value attended, which is up to some eight times
    a row's largest: values average out over up to 200 tokens); the rest is smaller."""
    from examples import forked_answers
    assert forked_answers.main(verbose=False) < 2.0 ** -11 * 16


def wants_of(q, layer, table, lens):
    k, v = (ref.values(*pages(layer, w)) for w in (0, 1))
    return [ref.attention(host(q)[i].astype(np.float64), k, v, table[i], int(n), SCALE) for i, n in enumerate(lens)]


def test_append_decode_and_layers(cuda, tqlib):
    B, H, hq = 6, 2, 8
    lens = np.array([1, 16, 17, 33, 70, 300], np.int32)
    table = np.arange(B * 20, dtype=np.int32).reshape(B, 20)
    layers = [filled(cuda, tqlib, 5 + i, B * 20, H) for i in range(2)]
    slots = table[np.arange(B), (lens - 1) // BLOCK].astype(np.int64) * BLOCK + (lens - 1) % BLOCK
    ks, vs = [data(cuda, 30 + i, B, H) * 3 for i in range(2)], [data(cuda, 40 + i, B, H) for i in range(2)]
    want = [[list(pages(ly, w)) for w in (0, 1)] for ly in layers]
    tqlib.append_layers(layers, ks, vs, dev(cuda, slots))
    q = data(cuda, 50, B, hq)
    for i, ly in enumerate(layers):
        for w, x in ((0, ks[i]), (1, vs[i])):
            ref.append(*want[i][w], host(x), slots)
            assert_pages(ly, want[i][w], w)
    # the next token by the call that appends and decodes
    slots, lens = slots + 0, lens.copy()
    lens[[1, 3]] -= 1  # (two rows write a token again)
    out = layers[0].append_decode(ks[1], vs[1], dev(cuda, slots), q, dev(cuda, table), dev(cuda, lens), out_dtype=cuda.float32)
    for w, x in ((0, ks[1]), (1, vs[1])):
        ref.append(*want[0][w], host(x), slots)
        assert_pages(layers[0], want[0][w], w)
    check_rows(out.cpu().numpy(), wants_of(q, layers[0], table, lens))
    assert tqlib.get_device_status() == 0


def test_offload_and_restore(cuda, tqlib):
    layer, other = filled(cuda, tqlib, 3, 12, 3), layer_of(tqlib, 12, 3)
    ids = [7, 2, 11]
    image = layer.offload(ids)
    cuda.cuda.synchronize()
    other.restore([0, 1, 2], image)
    for a, b in ((layer.k_cache, other.k_cache), (layer.v_cache, other.v_cache)):
        assert cuda.equal(a.view(12, -1)[ids], b.view(12, -1)[:3])
    with pytest.raises(tqlib.TQError):
        tqlib.Layer(12, 3, kv_format="bf16").restore([0, 1, 2], image)


def test_decode_without_workspace(cuda, tqlib):
    layer, lens = filled(cuda, tqlib, 9, 30, 2), [100, 0, 333]
    table = tables(3, lens, 30)
    q = data(cuda, 2, 3, 6)
    args = (dev(cuda, table), dev(cuda, np.array(lens, np.int32)))
    want = layer.decode(q, *args, out_dtype=cuda.float32)
    fn = tqlib.lib().tq_decode_attention_static
    fn.restype, fn.argtypes = ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p] + [ctypes.c_int] * 3 + [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                             ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    out = cuda.empty_like(want)
    st = cuda.cuda.current_stream().cuda_stream
    assert fn(ctypes.addressof(layer.desc), q.data_ptr(), tqlib.TQ_BF16, 3, 6, args[0].data_ptr(), table.shape[1], args[1].data_ptr(),
              SCALE, out.data_ptr(), tqlib.TQ_F32, 0, st) == tqlib.TQ_OK
    assert cuda.equal(out, want)


def test_captured_steps(cuda, tqlib):
    """A step -- append, decode, attention of several tokens -- captured and replayed over inputs that change, and beside
    it the same calls on another stream with a workspace of their own."""
    B, H, hq, width = 5, 2, 8, 12
    layer = layer_of(tqlib, B * width, H)
    table = np.random.default_rng(0).permutation(B * width).astype(np.int32).reshape(B, width)
    fill = (table.reshape(-1)[:, None].astype(np.int64) * BLOCK + np.arange(BLOCK)).reshape(-1)
    layer.append(data(cuda, 1, fill.size, H), data(cuda, 2, fill.size, H), dev(cuda, fill))
    t = dev(cuda, table)
    k, v, q = data(cuda, 3, B, H), data(cuda, 4, B, H), data(cuda, 5, B, hq)
    qs = data(cuda, 6, 90, hq)
    starts = dev(cuda, np.array([0, 40, 41, 41, 60, 90], np.int32))
    slots, lens = cuda.zeros(B, dtype=cuda.int64, device="cuda"), cuda.zeros(B, dtype=cuda.int32, device="cuda")
    ws = cuda.zeros(max(layer.workspace_bytes(B, hq, width), layer.attend_workspace_bytes(90, B, hq, width)), dtype=cuda.uint8, device="cuda")
    out, outs = cuda.empty(B, hq, D, device="cuda"), cuda.empty(90, hq, D, device="cuda")

    def step(w, o, os):
        layer.append(k, v, slots)
        layer.decode(q, t, lens, out=o, workspace=w)
        layer.attend(qs, starts, t, lens, out=os, workspace=w)

    side = cuda.cuda.Stream()
    side.wait_stream(cuda.cuda.current_stream())
    with cuda.cuda.stream(side):
        lens.fill_(60)
        step(ws, out, outs)
    cuda.cuda.current_stream().wait_stream(side)
    graph = cuda.cuda.CUDAGraph()
    with cuda.cuda.graph(graph):
        step(ws, out, outs)
    ws2, o2, os2 = cuda.zeros_like(ws), cuda.empty_like(out), cuda.empty_like(outs)
    for n in ([100, 41, 17, 192, 64], [101, 42, 18, 96, 65]):
        n = np.array(n, np.int32)
        lens.copy_(dev(cuda, n))
        slots.copy_(dev(cuda, table[np.arange(B), (n - 1) // BLOCK].astype(np.int64) * BLOCK + (n - 1) % BLOCK))
        k.copy_(data(cuda, int(n[0]), B, H))
        graph.replay()
        check_rows(out.cpu().numpy(), wants_of(q, layer, table, n))
        kk, vv = (ref.values(*pages(layer, w)) for w in (0, 1))
        new, qh = [40, 1, 0, 19, 30], host(qs).astype(np.float64)
        first = np.concatenate([[0], np.cumsum(new)])
        check_rows(outs.cpu().numpy(), [ref.attention(qh[first[b] + i], kk, vv, table[b], max(0, int(n[b]) - m + i + 1), SCALE, 2.0 ** -11)
                                        for b, m in enumerate(new) for i in range(m)])
        # both at once: the replay and the same reads on the other stream
        side.wait_stream(cuda.cuda.current_stream())
        layer.decode(q, t, lens, out=o2, workspace=ws2, stream=side)
        layer.attend(qs, starts, t, lens, out=os2, workspace=ws2, stream=side)
        side.synchronize()
        assert cuda.equal(o2, out) and cuda.equal(os2, outs)
    assert tqlib.get_device_status() == 0


def test_results_on_a_given_stream(cuda, tqlib):
    """Results and workspaces of calls that are given a stream belong to it: what the current stream still does with freed
    memory does not reach them."""
    layer, lens = filled(cuda, tqlib, 19, 20, 2), [100, 50]
    table = tables(3, lens, 20)
    args = (dev(cuda, table), dev(cuda, np.array(lens, np.int32)))
    q, starts = data(cuda, 2, 60, 8), dev(cuda, np.array([0, 40, 60], np.int32))
    want = layer.attend(q, starts, *args)
    side = cuda.cuda.Stream()
    cuda.cuda.synchronize()
    for _ in range(3):
        junk = cuda.full((1 << 26,), 1.0, device="cuda")
        for _ in range(20):
            junk.mul_(1.5)
        del junk
        got = layer.attend(q, starts, *args, stream=side)
        side.synchronize()
        assert cuda.equal(got, want)
    cuda.cuda.synchronize()
