"""GPU: the shared-prefix decode gives the same bits whatever ran on the GPU before it."""
import pytest

import workloads
from tests.test_gpu_prefix import FORMATS, build, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
@pytest.mark.parametrize("B,hq,hkv", [(2, 8, 8), (5, 7, 1), (33, 4, 1), (33, 16, 4), (70, 8, 2)])
def test_bits_do_not_hang_on_what_ran_before(cuda, tqlib, fmt, bk, bv, B, hq, hkv):
    """Few rows a KV head, or a ragged last tile of them, between calls of other sizes of queries, whose
    operands stay in shared memory."""
    lens = workloads.rng(B).integers(0, 40, B)
    case = build(cuda, tqlib, fmt, bk, bv, B=B, hq=hq, hkv=hkv, P=2600, lens=lens, seed=B)
    others = [build(cuda, tqlib, *f, B=64, hq=32, hkv=8, P=2600, lens=[0] * 64, seed=1) for f in FORMATS[:1] + FORMATS[3:4]]
    outs = []
    for size in (1.0, 1e-20, 1e6, 1e20):
        for other in others:
            other[1].copy_(size * cuda.randn(other[1].shape, device="cuda"))
            run(cuda, tqlib, other, 2600)
            outs.append(run(cuda, tqlib, case, 2600, cuda.float32))
    assert all(cuda.equal(o, outs[0]) for o in outs[1:])
