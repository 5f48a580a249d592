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


def graded(cuda, tq, fmt, bk, bv, *, P, own, outlier, small=False, B=3, hq=4, seed=0):
    """Two kinds of tokens in every block: ordinary ones, and every fifth with values `outlier` times as
    large that no query attends (logits 60 below); small: those are the ones attended (logits 60
    above), and the ordinary ones' values the large ones.  P prefix tokens, `own` of each sequence."""
    g = workloads.rng(seed)
    pb, width = -(-P // 16), -(-own // 16)
    ids = g.permutation(pb + B * width + 1).astype(np.int32)
    ptab, table = ids[:pb], ids[pb:pb + B * width].reshape(B, width)
    layer = tq.Layer(len(ids), 1, kv_format=fmt, bits_k=bk, bits_v=bv, seed=seed, fill=0xFF)
    slots = [ptab[np.arange(P) // 16].astype(np.int64) * 16 + np.arange(P) % 16]
    slots = np.concatenate(slots + [t[np.arange(own) // 16].astype(np.int64) * 16 + np.arange(own) % 16 for t in table])
    base = g.standard_normal(D)
    rare = np.arange(len(slots)) % 5 == 2
    k = 0.1 * g.standard_normal((len(slots), D)) + np.where(rare, 5.5 if small else -5.5, 0.0)[:, None] * base
    v = g.standard_normal((len(slots), D)) * np.where(rare ^ small, outlier, 1.0)[:, None]
    to = lambda x: cuda.from_numpy(x.astype(np.float32)).cuda()
    layer.append(to(k[:, None]), to(v[:, None]), cuda.from_numpy(slots).cuda())
    q = to(base + 0.1 * g.standard_normal((B, hq, D))).to(cuda.bfloat16)
    return layer, q, ptab, table, np.full(B, own, np.int32)


@pytest.mark.parametrize("P,own", [(300, 0), (300, 40), (0, 40)])
@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("outlier", [2.0 ** 10, 2.0 ** 17, 2.0 ** 24, 2.0 ** 80])
def test_bf16_values_of_every_size(cuda, tqlib, P, own, small, outlier):
    case = graded(cuda, tqlib, "bf16", 4, 4, P=P, own=own, outlier=outlier, small=small)
    out = run(cuda, tqlib, case, P, cuda.float32).cpu().numpy()
    assert max_rel_err(out, reference(case, P)) <= TOL


@pytest.mark.parametrize("B", [2, 70])
def test_bf16_channels_of_every_size(cuda, tqlib, B):
    """Channels from 2^-60 to 1, and one with an infinite element: each keeps its own precision."""
    P, hq = 400, 4
    layer, q, ptab, table, lens = case = build(cuda, tqlib, "bf16", 4, 4, B=B, hq=hq, hkv=1, P=P, lens=[0] * B, seed=8)
    size = cuda.from_numpy(2.0 ** -workloads.rng(1).integers(0, 61, D).astype(np.float32)).cuda()
    pool = layer.v_cache.view(cuda.bfloat16).view(-1, D)
    pool.copy_(cuda.where(pool.isfinite(), pool * size, pool))
    ref = reference(case, P)
    pool[int(ptab[3]) * 16 + 2, 17] = float("inf")
    out = run(cuda, tqlib, case, P, cuda.float32).cpu().numpy()
    assert not np.any(np.isfinite(out[..., 17]))
    rest = np.arange(D) != 17
    # of a channel's largest result: weights to 2^-16, sums in fp32
    err = np.abs(out - ref)[..., rest].max((0, 1)) / np.abs(ref)[..., rest].max((0, 1))
    assert err.max() <= TOL


@pytest.mark.parametrize("fmt,bk,bv", FORMATS[1:])
@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("B", [3, 70])
@pytest.mark.parametrize("outlier", [2.0 ** 10, 2.0 ** 17, 2.0 ** 24, 2.0 ** 60])
def test_coded_values_of_every_size(cuda, tqlib, fmt, bk, bv, small, B, outlier):
    case = graded(cuda, tqlib, fmt, bk, bv, P=300, own=0, outlier=outlier, small=small, B=B)
    out = run(cuda, tqlib, case, 300, cuda.float32).cpu().numpy()
    assert max_rel_err(out, reference(case, 300)) <= TOL


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("P,own", [(0, 40), (300, 40), (0, 300), (20, 2100)])
@pytest.mark.parametrize("outlier", [2.0 ** 17, 2.0 ** 60])
def test_own_values_of_every_size(cuda, tqlib, fmt, bk, bv, small, P, own, outlier):
    """(20, 2100): a block table for the decode kernel."""
    case = graded(cuda, tqlib, fmt, bk, bv, P=P, own=own, outlier=outlier, small=small)
    out = run(cuda, tqlib, case, P, cuda.float32).cpu().numpy()
    assert max_rel_err(out, reference(case, P)) <= TOL


@pytest.mark.parametrize("fmt,bk,bv", FORMATS)
@pytest.mark.parametrize("P,own,at", [(300, 0, 150), (300, 40, 150), (300, 40, 310), (0, 40, 10), (20, 2100, 100)])
def test_logits_of_every_size(cuda, tqlib, fmt, bk, bv, P, own, at):
    """Rows whose largest logit is from 2^6 to 2^110, more than an fp32 of the size of 2^24 can tell apart
    in units: token `at` (of the first sequence's tokens, its own behind the prefix's) has it by far, and
    the result is its value."""
    B, hq = 3, 24
    layer, q, ptab, table, lens = case = graded(cuda, tqlib, fmt, bk, bv, P=P, own=own, outlier=1.0, B=B, hq=hq)
    q0 = q[:, :1].double().mean(0, keepdim=True)
    slots = [int(ptab[at // 16]) * 16 + at % 16] if at < P else [int(t[(at - P) // 16]) * 16 + (at - P) % 16 for t in table]
    k = (4.0 * q0).float().expand(len(slots), 1, D).contiguous()
    layer.append(k, cuda.randn(len(slots), 1, D, device="cuda"), cuda.tensor(slots, device="cuda"))
    e = np.linspace(0, 104, hq).astype(int)
    q = (q0 * cuda.from_numpy(2.0 ** e[:, None]).cuda()).expand(B, hq, D).float().contiguous()
    case = layer, q, ptab, table, lens
    out = run(cuda, tqlib, case, P, cuda.float32).cpu().numpy()
    assert max_rel_err(out, reference(case, P)) <= TOL


def long_prefix_error(cuda, tq, fmt, P):
    """Lengths up to the last that is accepted, by a table that names one block again and again: what the
    block alone gives (a last, partial block changes it by 2^-20).  The values have a mean, so that an
    accumulator that loses a little at each addition shows."""
    layer = tq.Layer(2, 1, kv_format=fmt, bits_k=2, bits_v=2, fill=0xFF)
    g = workloads.rng(5)
    to = lambda x: cuda.from_numpy(x.astype(np.float32)).cuda()
    layer.append(to(g.standard_normal((16, 1, D))), to(g.standard_normal((16, 1, D)) + 2.0), cuda.arange(16, 32, device="cuda"))
    q = to(0.5 * g.standard_normal((1, 2, D)))
    table = cuda.ones((P + 15) // 16, dtype=cuda.int32, device="cuda")
    out = layer.prefix_decode(q, table, P, out_dtype=cuda.float32)
    cuda.cuda.synchronize()
    assert tq.get_device_status() == 0
    ref = prefix_attention(q.double().cpu().numpy(), *stands_for(layer), np.array([1]), 16, np.zeros((1, 0), np.int32),
                           np.zeros(1, np.int32), 1 / math.sqrt(D))
    return max_rel_err(out.cpu().numpy(), ref)


@pytest.mark.parametrize("fmt", ["bf16", "packed"])
@pytest.mark.parametrize("P", [2 ** 31 - 128, 2 ** 24 + 5])
def test_long_prefixes_keep_their_sums(cuda, tqlib, fmt, P):
    assert long_prefix_error(cuda, tqlib, fmt, P) <= TOL


@pytest.mark.parametrize("fmt", ["bf16", "packed"])
@pytest.mark.parametrize("P", [2 ** 31 - 1, 2 ** 31 - 127])
def test_the_longest_prefixes(cuda, tqlib, fmt, P):
    assert long_prefix_error(cuda, tqlib, fmt, P) <= TOL


@pytest.mark.parametrize("fmt,bk,bv", FORMATS[:2])
@pytest.mark.parametrize("own", [0, 40])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 30])
def test_a_key_that_is_not_a_number_shows(cuda, tqlib, fmt, bk, bv, own, size):
    """In the prefix, or among a sequence's own tokens, under ordinary logits and under large ones: every row
    that attends it is NaN, the other sequences are not."""
    P, B = 300, 3
    layer, q, ptab, table, lens = graded(cuda, tqlib, fmt, bk, bv, P=P, own=own, outlier=1.0, B=B)
    q = q.float() * size
    bad = cuda.full((1, 1, D), float("nan"), device="cuda")
    slot = int(table[1, 1]) * 16 + 3 if own else int(ptab[7]) * 16 + 3
    layer.append(bad, None, cuda.tensor([slot], device="cuda"))
    out = run(cuda, tqlib, (layer, q, ptab, table, lens), P, cuda.float32)
    nan = out.isnan().all(-1).all(-1).tolist()
    assert nan == ([False, True, False] if own else [True] * 3)
    assert bool(out[~cuda.tensor(nan, device="cuda")].isfinite().all())
