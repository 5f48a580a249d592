"""Plain fp64 definitions of the rotary positions and of attention over a shared
prefix, for the operator tests.  Nothing here comes from libtq."""
import math

import numpy as np

D = 128


def frequencies(rotary_dim, base, scaling=None):
    """(radians a position [rotary_dim / 2], amplitude)."""
    s = scaling or {"kind": None}
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    if s["kind"] == "ntk" and rotary_dim > 2:
        base = base * s["factor"] ** (rotary_dim / (rotary_dim - 2.0))
    f = base ** (-2.0 * i / rotary_dim)
    if s["kind"] == "linear":
        return f / s["factor"], 1.0
    if s["kind"] == "banded":
        keep = np.clip((s["length"] * f / (2 * math.pi) - s["low"]) / (s["high"] - s["low"]), 0, 1)
        return (1 - keep) * f / s["factor"] + keep * f, 1.0
    if s["kind"] == "yarn":
        at = lambda t: rotary_dim * math.log(s["length"] / (2 * math.pi * t)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(s["high"])), 0), min(math.ceil(at(s["low"])), rotary_dim - 1)
        keep = 1 - np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return (1 - keep) * f / s["factor"] + keep * f, 0.1 * math.log(s["factor"]) + 1.0
    return f, 1.0


def rotate(x, positions, freqs, amplitude, layout, transpose=False):
    """x fp64 [n, heads, D] turned by positions [n] (integers)."""
    r = 2 * len(freqs)
    ang = np.asarray(positions, np.float64)[:, None] * freqs
    c, s = np.cos(ang)[:, None] * amplitude, np.sin(ang)[:, None] * amplitude * (-1 if transpose else 1)
    y = np.array(x, np.float64)
    ia = np.arange(r // 2) if layout == "half" else 2 * np.arange(r // 2)
    ib = ia + r // 2 if layout == "half" else ia + 1
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def pair_norm(x, rotary_dim, layout):
    """|(x_a, x_b)| at both coordinates of every pair (|x| elsewhere)."""
    n = np.abs(np.array(x, np.float64))
    h = rotary_dim // 2
    ia = np.arange(h) if layout == "half" else 2 * np.arange(h)
    ib = ia + h if layout == "half" else ia + 1
    n[..., ia] = n[..., ib] = np.hypot(x[..., ia], x[..., ib])
    return n


def prefix_attention(q, keys, values, prefix_ids, prefix_len, table, lens, sm_scale):
    """q [B, Hq, D]; keys, values [num_blocks, Hkv, 16, D] (what the cache stands for);
    rows without any token are zero."""
    bsz, hq, _ = q.shape
    hkv = keys.shape[1]
    g = hq // hkv
    out = np.zeros((bsz, hq, D))
    flat = lambda x, ids, n: x[ids].transpose(1, 0, 2, 3).reshape(hkv, -1, D)[:, :n]
    for b in range(bsz):
        k, v = (np.concatenate([flat(x, prefix_ids, prefix_len), flat(x, table[b], lens[b])], 1) for x in (keys, values))
        if k.shape[1] == 0:
            continue
        s = np.einsum("hgd,htd->hgt", q[b].reshape(hkv, g, D), k) * sm_scale
        w = np.exp(s - s.max(-1, keepdims=True))
        out[b] = np.einsum("hgt,htd->hgd", w / w.sum(-1, keepdims=True), v).reshape(hq, D)
    return out
