"""int8 layers in plain 64-bit arithmetic: pages, appends and attention, for the parity tests.

A page: 16 records of 128 bytes (code + 128), fp32 step, uint32 bits of records that are not numbers,
8 bytes without meaning.  Codes and steps as include/tq.h defines them."""
import math

import numpy as np

D, BLOCK, PAGE = 128, 16, 16 * 128 + 16
TINY = np.float32(2.0 ** -126)


def split(pool, blocks, heads):
    """(codes int8 [blocks, heads, 16, D], steps fp32 [blocks, heads], bits uint32 [blocks, heads])."""
    pages = np.ascontiguousarray(pool).reshape(blocks, heads, PAGE)
    codes = (pages[..., :BLOCK * D].astype(np.int16) - 128).astype(np.int8).reshape(blocks, heads, BLOCK, D)
    tail = np.ascontiguousarray(pages[..., BLOCK * D:])
    return codes, tail[..., :4].copy().view(np.float32)[..., 0], tail[..., 4:8].copy().view(np.uint32)[..., 0]


def append(codes, steps, bits, x, slots):
    """One append of x [n, heads, D] (fp32 values) in place; the last token of a slot stays."""
    by_block = {}
    for t, s in enumerate(slots):
        if 0 <= s < codes.shape[0] * BLOCK:
            by_block.setdefault(int(s) // BLOCK, {})[int(s) % BLOCK] = t
    for b, rows in by_block.items():
        for h in range(x.shape[1]):
            new = {r: x[t, h].astype(np.float64) for r, t in rows.items()}
            finite = {r: np.isfinite(v).all() for r, v in new.items()}
            top = max([np.abs(v).max() for r, v in new.items() if finite[r]], default=0.0)
            step = max(np.float32(np.float32(top) / np.float32(127)), TINY)
            old = steps[b, h]
            begins = 0 in rows or not (old >= TINY and np.isfinite(old))
            if begins:
                codes[b, h], bits[b, h] = 0, 0
            else:
                step = max(step, old)
                if step != old:
                    codes[b, h] = np.rint(codes[b, h].astype(np.float64) * np.float64(old) / np.float64(step))
            steps[b, h] = step
            for r, v in new.items():
                v = v if finite[r] else np.zeros(D)
                codes[b, h, r] = np.clip(np.rint(v / np.float64(step)), -127, 127)
                bits[b, h] = (int(bits[b, h]) & ~(1 << r)) | (0 if finite[r] else 1 << r)


def values(codes, steps, bits):
    """[blocks, heads, 16, D] in 64 bits, NaN for records that are not numbers."""
    v = codes.astype(np.float64) * steps.astype(np.float64)[..., None, None]
    return np.where(((bits[..., None] >> np.arange(BLOCK, dtype=np.uint32)) & 1).astype(bool)[..., None], np.nan, v)


def attention(q, k, v, table, ctx, scale, weights=0.0):
    """(out [Hq, D], bound [Hq]) of one query token: q [Hq, D]; k, v [blocks, heads, 16, D]; `bound` is what
    fp32 sums and 22-bit parts may cost: the products of a logit lose at most 2^-19 of the sum of their
    magnitudes (2^-22 the two parts of a query, 2^-23 each of 8 sums and the last scalings, with room for a
    tensor core that cuts off instead of rounding), a weight as much and 2^-20 for its own two parts,
    exponential and the denominator; relative to the largest value attended.  `weights`: half a step of the type
    that weights are rounded to."""
    hq, heads = q.shape[0], k.shape[1]
    out, bound = np.zeros((hq, D)), np.zeros(hq)
    ids = [(int(table[p // BLOCK]), p % BLOCK) for p in range(ctx)]
    ids = [(b, r) for b, r in ids if 0 <= b < k.shape[0]]
    if not ids:
        return out, bound
    bs, rs = np.array([b for b, _ in ids]), np.array([r for _, r in ids])
    for h in range(hq):
        kh, vh = k[bs, h // (hq // heads), rs], v[bs, h // (hq // heads), rs]
        s = (kh @ q[h]) * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        out[h] = w @ vh
        delta = 2.0 ** -19 * (np.abs(kh) @ np.abs(q[h])).max() * abs(scale)
        bound[h] = (2 * delta + 2.0 ** -20 + weights) * np.abs(vh).max()
    return out, bound
