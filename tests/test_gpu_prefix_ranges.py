"""GPU: decode attention over a shared prefix where the sizes of queries, keys or values differ by
many powers of two, or are not finite, within one call: no row answers for another.

Tolerance: as in test_gpu_prefix.py (5e-3 of a row's largest value), against the same fp64
definition."""
import math

import numpy as np
import pytest

import workloads
from tests._gpu_util import D, max_rel_err
from tests._rope_ref import prefix_attention
from tests.test_gpu_prefix import FORMATS, TOL, build, run, stands_for

pytestmark = pytest.mark.gpu


def reference(case, P, q=None):
    layer, q0, ptab, table, lens = case
    q = (q0 if q is None else q).double().cpu().numpy()
    return prefix_attention(q, *stands_for(layer), ptab, P, table, lens, 1 / math.sqrt(D))


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
@pytest.mark.parametrize("q_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,hq", [(3, 8), (70, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1e30, 3e38, 2.0 ** 14, 2.0 ** 20])
def test_one_query_row_leaves_the_others_alone(cuda, tqlib, fmt, bk, bv, q_dtype, B, hq, bad):
    """A row of NaN, of infinities or of large values among rows of ordinary ones and rows of zeros (the
    unused slots of a padded batch): the others' results are those of a call without it.  (3, 8):
    one tile of rows a KV head; (70, 8): two, ragged."""
    P = 300
    case = build(cuda, tqlib, fmt, bk, bv, B=B, hq=hq, hkv=2, P=P, lens=[5, 0, 33] + [0] * (B - 3), seed=B, q_dtype=q_dtype)
    q = case[1]
    q[1, 3] = 0.0
    ref = reference(case, P)
    q[B - 2, 1] = bad * q[B - 2, 1].sign() if math.isfinite(bad) else bad
    out = run(cuda, tqlib, case, P, cuda.float32).cpu().numpy()
    others = np.ones((B, hq), bool)
    others[B - 2, 1] = False
    assert max_rel_err(out[others], ref[others]) <= TOL


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
def test_query_rows_of_every_size(cuda, tqlib, fmt, bk, bv):
    """Rows from 2^-100 to 2^3 of the ordinary size: the small ones attend evenly, as their logits say."""
    B, hq, P = 40, 8, 300
    case = build(cuda, tqlib, fmt, bk, bv, B=B, hq=hq, hkv=2, P=P, lens=[7] * B, seed=3, q_dtype="f32")
    q = case[1]
    e = workloads.rng(5).integers(-100, 4, (B, hq, 1))
    q *= cuda.from_numpy((2.0 ** e).astype(np.float32)).cuda()
    out = run(cuda, tqlib, case, P, cuda.float32).cpu().numpy()
    assert max_rel_err(out, reference(case, P)) <= TOL


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
@pytest.mark.parametrize("P,width", [(300, None), (0, None), (300, 0), (300, 140)])
def test_rows_that_are_not_finite_say_so(cuda, tqlib, fmt, bk, bv, P, width):
    """The softmax of NaN logits is NaN, not an empty row's zeros: by the prefix kernel, the own tokens'
    and both, next to a sequence without any token."""
    lens = [0, 0, 0] if width == 0 else [9, 40, 0]
    case = build(cuda, tqlib, fmt, bk, bv, B=3, hq=4, hkv=2, P=P, lens=lens, seed=4, width=width)
    q = case[1]
    q[0, 1], q[1, 2, 77] = float("nan"), float("inf")
    out = run(cuda, tqlib, case, P, cuda.float32)
    assert bool(out[0, 1].isnan().all()) and bool(out[1, 2].isnan().all())
    out[0, 1], out[1, 2] = 0.0, 0.0
    assert bool(out.isfinite().all())
    assert P > 0 or bool((out[2] == 0).all())
