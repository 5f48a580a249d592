"""Host parts of the rotary positions, the rotated append and the shared-prefix decode:
frequencies against their formulas, and refusals that launch nothing (no GPU needed)."""
import ctypes

import numpy as np
import pytest

from tests._rope_ref import frequencies
from tests.test_abi_host import fake_desc

BANDED = {"kind": "banded", "factor": 8.0, "low": 1.0, "high": 4.0, "length": 8192}
YARN = {"kind": "yarn", "factor": 16.0, "low": 1.0, "high": 32.0, "length": 4096}


@pytest.mark.parametrize("rotary_dim", [2, 62, 64, 128])
@pytest.mark.parametrize("scaling", [None, {"kind": "linear", "factor": 4.0}, {"kind": "ntk", "factor": 8.0}, BANDED, YARN])
def test_frequencies_follow_their_formulas(tqlib, rotary_dim, scaling):
    """turns_i = f_i / (2 pi) to 2^-53 of a turn and the roundings of its fp64 evaluation."""
    rope = tqlib.Rope(rotary_dim, 10000.0, scaling=scaling)
    f, amplitude = frequencies(rotary_dim, 10000.0, scaling)
    assert np.max(np.abs(rope.turns() - f / (2 * np.pi))) <= 1e-15
    assert rope.amplitude == np.float32(amplitude)


def test_explicit_frequencies_wrap_to_a_turn(tqlib):
    f = np.array([0.0, 2 * np.pi * 1.25, -2 * np.pi * 0.25, 1e-9])
    t = tqlib.Rope(8, inv_freq=f).turns()
    assert np.max(np.abs(t - np.array([0.0, 0.25, 0.75, 1e-9 / (2 * np.pi)]))) <= 1e-15


@pytest.mark.parametrize("kw,word", [
    (dict(rotary_dim=3), "rotary_dim"), (dict(rotary_dim=0), "rotary_dim"), (dict(rotary_dim=130), "rotary_dim"),
    (dict(base=1.0), "base"), (dict(base=float("nan")), "base"), (dict(base=float("inf")), "base"),
    (dict(scaling={"kind": "linear", "factor": 0.5}), "factor"),
    (dict(scaling={"kind": "ntk", "factor": float("nan")}), "factor"),
    (dict(scaling={"kind": "banded", "factor": 2.0, "low": 4.0, "high": 1.0, "length": 8192}), "low"),
    (dict(scaling={"kind": "yarn", "factor": 2.0, "low": 1.0, "high": 32.0}), "length"),
    (dict(rotary_dim=4, inv_freq=[1.0, float("inf")]), "finite"),
    (dict(rotary_dim=4, inv_freq=[1.0, 0.5], scaling={"kind": "linear", "factor": 2.0}), "scaling"),
])
def test_make_rope_refusals(tqlib, kw, word):
    with pytest.raises(tqlib.TQError) as e:
        tqlib.Rope(**kw)
    assert e.value.status == tqlib.TQ_ERR_INVALID_ARG and word in str(e.value)


def test_rope_class_refusals(tqlib):
    for kw in (dict(layout="other"), dict(scaling={"kind": "other", "factor": 2.0}), dict(rotary_dim=4, inv_freq=[1.0])):
        with pytest.raises(ValueError):
            tqlib.Rope(**kw)


def heads(tq, inp=0x10000, out=0x20000, n=8):
    h = tq.Heads()
    h.inp, h.out, h.num_heads = inp, out, n
    h.in_token_stride = h.out_token_stride = n * 128
    h.in_head_stride = h.out_head_stride = 128
    return h


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_rope_apply_refusals(tqlib):
    tq = tqlib
    rope = tq.Rope().desc
    n0 = tq.launch_count()

    def call(rope, q, k, dtype=tq.TQ_BF16, pos=0x30000, n=4):
        return tq.lib().tq_rope_apply(ref(rope), 0, ref(q), ref(k), dtype, ctypes.c_void_p(pos), n, None)

    good = heads(tq)
    broken = tq.Rope().desc
    broken.rotary_dim = 5
    wild = tq.Rope().desc
    wild.amplitude = float("inf")
    for args, word in (((None, good, None), "rope"), ((broken, good, None), "rotary_dim"), ((wild, good, None), "amplitude"),
                       ((rope, None, None), "null"), ((rope, good, None, 7), "dtype"),
                       ((rope, heads(tq, inp=None), None), "null"), ((rope, good, heads(tq, out=None)), "null"),
                       ((rope, heads(tq, n=0), None), "num_heads"), ((rope, heads(tq, inp=0x10001), None), "aligned"),
                       ((rope, heads(tq, out=0x10002), None, tq.TQ_F32), "aligned"),
                       ((rope, good, None, tq.TQ_BF16, None), "positions"),
                       ((rope, good, None, tq.TQ_BF16, 0x30000, -1), "n_tokens")):
        assert call(*args) == tq.TQ_ERR_INVALID_ARG, word
        assert word in tq.last_error()
    assert call(rope, good, None, n=0) == tq.TQ_OK
    assert tq.launch_count() == n0


def test_rope_append_refusals(tqlib):
    tq = tqlib
    rope = tq.Rope().desc
    n0 = tq.launch_count()
    good = fake_desc(tq)

    def call(desc, q, k, v, dtype=tq.TQ_BF16, pos=0x30000, slots=0x40000, n=4, rope=rope):
        return tq.lib().tq_rope_append(ref(desc), ref(rope), ref(q), ref(k), ref(v), dtype, ctypes.c_void_p(pos),
                                       ctypes.c_void_p(slots), n, None)

    q, k, v = heads(tq, n=32), heads(tq, out=None), heads(tq, out=None)
    for desc in (fake_desc(tq, rot_kind=tq.TQ_ROT_DENSE), fake_desc(tq, qjl_k=1, qjl_proj=0x50000),
                 fake_desc(tq, kv_format=tq.TQ_KV_POLAR)):
        assert call(desc, q, k, v) == tq.TQ_ERR_UNSUPPORTED
        assert "tq_rope_append" in tq.last_error()
    for args, word in (((good, q, None, None), "null"), ((good, heads(tq, out=None), k, v), "null"),
                       ((good, q, heads(tq, n=4), v), "heads"), ((good, q, k, heads(tq, n=16, out=None)), "heads"),
                       ((good, q, k, heads(tq)), "output"), ((good, q, k, v, 9), "dtype"),
                       ((good, q, k, v, tq.TQ_BF16, None), "null"), ((good, q, k, v, tq.TQ_BF16, 8, None), "null"),
                       ((good, q, k, v, tq.TQ_BF16, 8, 8, -2), "n_tokens"),
                       ((fake_desc(tq, head_dim=64), q, k, v), "head_dim")):
        assert call(*args) in (tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED), word
        assert word in tq.last_error()
    assert call(good, q, k, v, rope=None) == tq.TQ_ERR_INVALID_ARG
    assert call(good, q, k, v, n=0) == tq.TQ_OK
    assert tq.launch_count() == n0


def test_prefix_decode_refusals(tqlib):
    tq = tqlib
    n0 = tq.launch_count()
    good = fake_desc(tq)

    def call(desc, batch=2, hq=8, ptab=0x1000, plen=100, bt=0x2000, mb=4, ctx=0x3000, q=0x4000, out=0x5000, qd=1, od=1,
             scale=0.1):
        return tq.lib().tq_prefix_decode(ref(desc), ctypes.c_void_p(q), qd, batch, hq, ctypes.c_void_p(ptab), plen,
                                         ctypes.c_void_p(bt), mb, ctypes.c_void_p(ctx), scale, ctypes.c_void_p(out), od,
                                         ctypes.c_void_p(0x40000), 1 << 20, None)

    for desc in (fake_desc(tq, rot_kind=tq.TQ_ROT_DENSE), fake_desc(tq, qjl_k=1, qjl_proj=0x50000),
                 fake_desc(tq, kv_format=tq.TQ_KV_POLAR)):
        assert call(desc) == tq.TQ_ERR_UNSUPPORTED
    for kw, word in ((dict(plen=-1), "prefix_len"), (dict(plen=1 << 31), "prefix_len"), (dict(ptab=None), "prefix_table"),
                     (dict(mb=-1), "max_blocks"), (dict(bt=None), "block_table"), (dict(ctx=None), "context_lens"),
                     (dict(batch=-1), "batch"), (dict(hq=12), "num_q_heads"), (dict(hq=0), "num_q_heads"),
                     (dict(q=None), "null"), (dict(out=None), "null"), (dict(qd=5), "q_dtype"), (dict(od=5), "out_dtype"),
                     (dict(scale=float("nan")), "NaN"), (dict(q=0x4008), "aligned")):
        assert call(good, **kw) == tq.TQ_ERR_INVALID_ARG, kw
        assert word in tq.last_error(), kw
    assert call(good, batch=70000) == tq.TQ_ERR_UNSUPPORTED
    assert call(good, batch=0) == tq.TQ_OK
    assert tq.lib().tq_prefix_workspace_bytes(ref(good), 2, 12, 100, 4) == 0
    assert tq.lib().tq_prefix_workspace_bytes(ref(good), 2, 8, -1, 4) == 0
    assert tq.launch_count() == n0


def exact_turns(f, p=1):
    """p f / (2 pi) modulo one turn, in units of 2^-64 rounded to nearest: integers, pi by Machin's formula."""
    from fractions import Fraction

    def atan_inverse(n, bits):
        x = total = (1 << bits) // n
        k, sign = 1, -1
        while x:
            x, k = x // (n * n), k + 2
            total, sign = total + sign * (x // k), -sign
        return total

    pi = Fraction(16 * atan_inverse(5, 512) - 4 * atan_inverse(239, 512), 1 << 512)
    return round(Fraction(float(f)) * p / (2 * pi) * 2 ** 64) % 2 ** 64


def test_turns_hold_64_bits_of_the_frequency(tqlib):
    """turns_i is the nearest 64-bit fraction of the frequency, a double: of one, of powers of the base, of
    large, small and negative ones."""
    f = [1.0, -1.0, 1e-8, 2.0 ** -64, 2.0 ** -70, 1e-300, 0.0, 3.0, 2.0 ** 63 * 1.9, -1e19, 1e6 + 1 / 3, np.pi, 2 * np.pi]
    f += list(10000.0 ** (-np.arange(30) / 30.0)) + list(np.random.default_rng(1).standard_normal(21))
    rope = tqlib.Rope(128, inv_freq=f)
    assert [int(t) for t in rope.desc.turns] == [exact_turns(x) for x in f]
    assert int(tqlib.Rope().desc.turns[0]) == exact_turns(1.0)
    with pytest.raises(tqlib.TQError):
        tqlib.Rope(2, inv_freq=[2.0 ** 64])


def test_more_heads_than_a_token_can_have_are_refused(tqlib):
    tq = tqlib
    h = heads(tq, n=(1 << 28) + 1)
    assert tq.lib().tq_rope_apply(ref(tq.Rope().desc), 0, ref(h), None, tq.TQ_BF16, ctypes.c_void_p(0x30000), 1, None) == tq.TQ_ERR_INVALID_ARG
    assert "num_heads" in tq.last_error()
