"""GPU: the workspace of the shared-prefix decode: one made for a prefix and a width of block tables serves
every shorter prefix and every narrower table of the same batch and heads."""
import numpy as np
import pytest

import workloads
from tests.test_gpu_prefix import build, check, run

pytestmark = pytest.mark.gpu

LENGTHS = [0, 1, 100, 129, 1000, 2400, 2433, 5000, 20000, 131072, 524288, 600000]
WIDTHS = [0, 1, 16, 17, 100, 128, 129, 200, 513, 8192]


@pytest.mark.parametrize("B,hq,hkv", [(1, 1, 1), (16, 32, 8), (32, 32, 8), (64, 32, 8), (64, 64, 8), (512, 32, 8),
                                      (100, 12, 3), (300, 64, 64)])
def test_bytes_grow_with_length_and_width(cuda, tqlib, B, hq, hkv):
    layer = tqlib.Layer(1, hkv)
    size = np.array([[layer.prefix_workspace_bytes(B, hq, p, w) for w in WIDTHS] for p in LENGTHS])
    assert np.all(np.diff(size, axis=0) >= 0) and np.all(np.diff(size, axis=1) >= 0)


@pytest.mark.parametrize("fmt,bk,bv", [("packed", 4, 4), ("bf16", 4, 4)])
@pytest.mark.parametrize("B,hq,hkv", [(64, 16, 4), (2, 8, 8)])
def test_one_workspace_serves_narrower_tables_and_shorter_prefixes(cuda, tqlib, fmt, bk, bv, B, hq, hkv):
    """From 200 blocks (whose splits the batch decides) down to 128 (eight splits) and to none, and over
    prefixes whose splits grow as they get shorter."""
    tq = tqlib
    lens = workloads.rng(B).integers(0, 40, B)
    case = build(cuda, tq, fmt, bk, bv, B=B, hq=hq, hkv=hkv, P=2600, lens=lens, seed=B, width=200)
    layer, q, ptab, table, lens = case
    ws = cuda.zeros(layer.prefix_workspace_bytes(B, hq, 2600, 200), dtype=cuda.uint8, device="cuda")
    for P in (2600, 2432, 129, 0):
        for width in (200, 129, 128, 3, 0):
            part = layer, q, ptab, table[:, :width].copy(), lens if width else np.zeros(B, np.int32)
            one = run(cuda, tq, part, P, workspace=ws)
            assert cuda.equal(one, run(cuda, tq, part, P))
    check(cuda, tq, case, 2600)


def test_more_units_than_the_counter_region_holds(cuda, tqlib):
    """2,100 sequences of 8 KV heads with a wide table: the own tokens' partials take no counters, so no pass
    zeroes them, and the workspace serves decode calls before and after."""
    tq = tqlib
    B, P, width = 2100, 40, 129
    lens = workloads.rng(7).integers(0, 5, B)
    case = build(cuda, tq, "packed", 4, 4, B=B, hq=8, hkv=8, P=P, lens=lens, seed=7, width=1)
    layer, q, ptab, table, lens = case
    wide = layer, q, ptab, np.repeat(table, width, 1), lens
    ws = cuda.zeros(layer.prefix_workspace_bytes(B, 8, P, width), dtype=cuda.uint8, device="cuda")
    n0 = tq.launch_count()
    one = run(cuda, tq, wide, P, workspace=ws)
    assert tq.launch_count() - n0 == 3
    args = q[:4].contiguous(), cuda.from_numpy(table[:4]).cuda(), cuda.from_numpy(lens[:4]).cuda()
    plain = layer.decode(*args)
    for _ in range(3):
        assert cuda.equal(layer.decode(*args, workspace=ws), plain)
        assert cuda.equal(run(cuda, tq, wide, P, workspace=ws), one)
    check(cuda, tq, wide, P)
