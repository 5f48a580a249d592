"""GPU: rotated appends of several host threads at once, of kinds that need different amounts of shared
memory of the same kernel (keys alone or keys and values, one KV head or many)."""
import ctypes
import threading

import pytest

from tests._gpu_util import D

pytestmark = pytest.mark.gpu


def test_threads_do_not_take_each_others_shared_memory(cuda, tqlib):
    tq = tqlib
    rope = tq.Rope()
    errors = []
    start = threading.Barrier(4)

    def work(hkv, values, n):
        layer = tq.Layer(4, hkv)
        x = cuda.randn(n, hkv, D, device="cuda").to(cuda.bfloat16)
        at = cuda.arange(n, device="cuda")
        heads = tq.Heads(x.data_ptr(), None, hkv, hkv * D, D, 0, 0)
        stream = cuda.cuda.Stream()
        call = (ctypes.byref(layer.desc), rope.ref, None, ctypes.byref(heads), ctypes.byref(heads) if values else None,
                tq.TQ_BF16, at.data_ptr(), at.data_ptr(), n, stream.cuda_stream)
        append = tq.lib().tq_rope_append
        cuda.cuda.synchronize()
        append(*call)
        cuda.cuda.synchronize()
        want = layer.k_cache.clone()
        start.wait()
        bad = sum(append(*call) != tq.TQ_OK for _ in range(20000))
        stream.synchronize()
        if bad or not cuda.equal(layer.k_cache, want):
            errors.append((hkv, values, bad, tq.last_error()))

    threads = [threading.Thread(target=work, args=a) for a in ((1, True, 40), (16, False, 2), (8, False, 3), (1, True, 64))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert tq.get_device_status() == 0
