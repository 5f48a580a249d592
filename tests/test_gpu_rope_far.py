"""GPU: rotary positions far out against angles in exact integer arithmetic, none of them from libtq.

Tolerance: ROT of test_gpu_rope.py for the angle's rounding to fp32 and the arithmetic behind it, and
the 2^-65 turns a position that a frequency of 64 bits may be off."""
import numpy as np
import pytest

from tests._gpu_util import D
from tests._rope_ref import pair_norm
from tests.test_gpu_rope import ROT, draw, f64
from tests.test_rope_host import exact_turns

pytestmark = pytest.mark.gpu


def test_far_positions_by_exact_angles(cuda, tqlib):
    f = 10000.0 ** (-np.arange(64) / 64.0)
    rope = tqlib.Rope(128, inv_freq=f)
    pos = np.array([0, 1, 2 ** 24 + 1, 2 ** 31 + 7, 2 ** 40 + 3, -(2 ** 33), -(2 ** 40) + 1], np.int64)
    x = draw(cuda, (len(pos), 2, D), "f32", 8)
    got = f64(tqlib.apply_rope(rope, cuda.from_numpy(pos).cuda(), x)[0])
    turns = np.array([[exact_turns(w, int(p)) / 2.0 ** 64 for w in f] for p in pos])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    xs = f64(x)
    want = np.concatenate([xs[..., :64] * c - xs[..., 64:] * s, xs[..., 64:] * c + xs[..., :64] * s], -1)
    slack = ROT + 2 * np.pi * np.abs(pos)[:, None, None] * 2.0 ** -65
    assert np.all(np.abs(got - want) <= slack * pair_norm(xs, 128, "half"))


@pytest.mark.parametrize("heads", [6640020, 8388607, 12000001])
def test_millions_of_heads_at_one_position(cuda, tqlib, heads):
    """One token whose head count is past the integers that an fp32 quotient tells apart (heads of many
    sequences at the same position, taken as one token): as rows of a token each."""
    tq = tqlib
    rope = tq.Rope()
    x = cuda.randn(1, heads, D, device="cuda", dtype=cuda.bfloat16)
    at = cuda.tensor([77], device="cuda")
    got = tq.apply_rope(rope, at, x)[0]
    for lo in (0, heads // 2, heads - 5000):
        rows = x[0, lo:lo + 5000].view(-1, 1, D)
        want = tq.apply_rope(rope, at.expand(rows.shape[0]).contiguous(), rows)[0]
        assert cuda.equal(got[0, lo:lo + 5000].view(-1, 1, D), want)
