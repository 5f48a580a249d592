"""Rotary positions, rotated appends and shared-prefix attention: cases, inputs, plain forms.

Three operators that a server of the paged KV cache calls one after another:

* rope    -- rotary positions of the query and key heads of a batch of tokens
             (views of one fused projection), half or interleaved pairs, all or
             part of the head, scaled frequencies, and the transposed rotation
             (the gradient of the rotation);
* append  -- the same rotation applied on the way into the paged cache: keys are
             rotated, keys and values stored in the layer's format (bf16, FP8 keys
             with 4-bit values, 2/3/4-bit Lloyd-Max codes), queries rotated in the
             same call;
* prefix  -- decode attention of a batch whose sequences share one long prefix in
             the cache: the prefix is read once for the whole batch, each
             sequence's own tokens follow from its block table.

`own` chooses between the plain forms (elementary torch operations) and the
package's entry points.
"""

import math

import numpy as np
import torch

own = False

D = 128  # head dimension of every cache layer
BLOCK = 16  # tokens a page


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of a batch of 16: the smallest call, a view of the fused projection
        {"name": "rope_step", "op": "rope", "tokens": 16, "hq": 32, "hkv": 8, "dtype": "bf16", "layout": "half",
         "rotary": 128, "scaling": "none", "far": 8192, "transpose": False},
        # a prompt batch of ragged sequences, interleaved pairs in half of the head, long-context bands
        {"name": "rope_prompt", "op": "rope", "tokens": 12345, "hq": 32, "hkv": 8, "dtype": "bf16",
         "layout": "interleaved", "rotary": 64, "scaling": "banded", "far": 131072, "transpose": False},
        # the gradient of a training batch's rotation in fp32, positions far out
        {"name": "rope_gradient", "op": "rope", "tokens": 4001, "hq": 64, "hkv": 8, "dtype": "f32", "layout": "half",
         "rotary": 128, "scaling": "yarn", "far": 1000000, "transpose": True},
        # one decode step into a full-precision boundary layer
        {"name": "append_step_bf16", "op": "append", "tokens": 16, "hq": 32, "hkv": 8, "fmt": "bf16", "bits_k": 0,
         "bits_v": 0, "layout": "half", "rotary": 128, "scaling": "none", "far": 8192, "skip": 0},
        # a prompt of ragged sequences into a layer of FP8 keys and 4-bit values, a tail of padding
        {"name": "append_prompt_k8v4", "op": "append", "tokens": 4099, "hq": 64, "hkv": 8, "fmt": "k8v4", "bits_k": 8,
         "bits_v": 4, "layout": "interleaved", "rotary": 64, "scaling": "linear", "far": 32768, "skip": 37},
        # the prefill burst of a prompt into a 4-bit layer
        {"name": "append_prompt_4bit", "op": "append", "tokens": 11000, "hq": 32, "hkv": 8, "fmt": "packed",
         "bits_k": 4, "bits_v": 4, "layout": "half", "rotary": 128, "scaling": "ntk", "far": 16384, "skip": 0},
        # a long prompt into the layout of the long-context workload, 3-bit keys and 4-bit values
        {"name": "append_long_3bit", "op": "append", "tokens": 65536, "hq": 64, "hkv": 8, "fmt": "packed",
         "bits_k": 3, "bits_v": 4, "layout": "half", "rotary": 128, "scaling": "yarn", "far": 131072, "skip": 0},
        # two answers to one short system prompt, one of them without tokens of its own
        {"name": "prefix_pair", "op": "prefix", "batch": 2, "hq": 32, "hkv": 8, "fmt": "bf16", "bits_k": 0,
         "bits_v": 0, "prefix": 333, "own": 40},
        # a batch of chats behind one instruction prompt, 4-bit layer
        {"name": "prefix_chat", "op": "prefix", "batch": 16, "hq": 32, "hkv": 8, "fmt": "packed", "bits_k": 4,
         "bits_v": 4, "prefix": 8192, "own": 1024},
        # questions about one document, groups of eight query heads, FP8 keys
        {"name": "prefix_k8v4", "op": "prefix", "batch": 24, "hq": 64, "hkv": 8, "fmt": "k8v4", "bits_k": 8,
         "bits_v": 4, "prefix": 5003, "own": 700},
        # many samples of one prompt in a full-precision boundary layer
        {"name": "prefix_many", "op": "prefix", "batch": 128, "hq": 32, "hkv": 8, "fmt": "bf16", "bits_k": 0,
         "bits_v": 0, "prefix": 16384, "own": 256},
        # a batch over one long document, 3-bit keys and 4-bit values, groups of eight: the largest
        {"name": "prefix_long", "op": "prefix", "batch": 64, "hq": 64, "hkv": 8, "fmt": "packed", "bits_k": 3,
         "bits_v": 4, "prefix": 100000, "own": 500},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "prefix"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
    turn = {"layout": rng.choice(["half", "interleaved"]), "rotary": rng.choice([128, 128, 64, 32, 96, 126, 2]),
            "scaling": rng.choice(["none", "linear", "ntk", "banded", "yarn"]), "far": _log_int(rng, 128, 1 << 20)}
    if op == "rope":
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "hq": hq, "hkv": hkv, "dtype": rng.choice(["bf16", "f32"]),
                **turn, "transpose": rng.random() < 0.4}
    fmt, bits_k, bits_v = rng.choice([("bf16", 0, 0), ("k8v4", 8, 4), ("k8v4", 8, 3), ("packed", 4, 4), ("packed", 3, 4),
                                      ("packed", 3, 3), ("packed", 2, 4), ("packed", 2, 2), ("packed", 4, 2)])
    kind = {"hq": hq, "hkv": hkv, "fmt": fmt, "bits_k": bits_k, "bits_v": bits_v}
    if op == "append":
        n = _log_int(rng, 1, 65536 * 8 // max(hkv, hq // 8))
        n = min(n, 65536)
        return {"op": op, "tokens": n, **kind, **turn, "skip": rng.randint(0, n // 3)}
    batch = _log_int(rng, 1, 256)
    most = 64 * 64 * 100000 // (batch * hq)
    prefix = _log_int(rng, 1, min(131072, most))
    return {"op": op, "batch": batch, **kind, "prefix": prefix, "own": _log_int(rng, 1, max(1, min(1024, 32768 // batch)))}


def work(case):
    """Bytes and operations one pass cannot do without."""
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "rope":
        n, e = case["tokens"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * (hq + hkv) * D * e + 8 * n, "flops": 3 * n * (hq + hkv) * case["rotary"]}
    if case["fmt"] == "bf16":
        kb = vb = 2 * D
    else:
        kb = D if case["fmt"] == "k8v4" else case["bits_k"] * D // 8 + 4
        vb = case["bits_v"] * D // 8 + 4
    if case["op"] == "append":
        n, live = case["tokens"], case["tokens"] - case["skip"]
        # q read and written, k and v read, rotated k written, records written; coded records are
        # read back as bf16 values (bf16 and FP8 pools are returned as they are)
        byt = 2 * n * hq * D * 2 + 3 * n * hkv * D * 2 + live * hkv * (kb + vb) + 16 * n
        flops = 3 * n * (hq + hkv) * case["rotary"]
        for coded, b in ((case["fmt"] == "packed", kb), (case["fmt"] != "bf16", vb)):
            if coded:
                byt += live * hkv * b + n * hkv * D * 2
                flops += 2 * live * hkv * D * 7 + 8 * live * hkv * D  # two butterflies, norms, cells
        return {"bytes": byt, "flops": flops}
    b, p = case["batch"], case["prefix"]
    lens = _own_lens(b, case["own"])
    tokens = p + int(lens.sum())
    pairs = b * p + int(lens.sum())
    return {"bytes": tokens * hkv * (kb + vb) + 2 * b * hq * D * 2 + 4 * (tokens // BLOCK + b), "flops": 4 * pairs * hq * D}


# ---------------------------------------------------- rotations and code tables

def _frequencies(rotary, scaling, base=500000.0):
    """(radians a position of each pair in 64 bits, amplitude) of the named scaling.

    Plain f_i = base^(-2 i / rotary).  linear: f / 8.  ntk: the base grows by
    8^(r / (r - 2)).  banded: wavelengths under L / 4 are kept, over L are divided by
    8, between them interpolated in L / wavelength, L = 8192.  yarn: a ramp between
    the pairs that turn 32 times and once in L, factor 16, amplitude 0.1 ln 16 + 1."""
    i = np.arange(rotary // 2, dtype=np.float64)
    if scaling == "ntk" and rotary > 2:
        base = base * 8.0 ** (rotary / (rotary - 2.0))
    f = base ** (-2.0 * i / rotary)
    if scaling == "linear":
        return f / 8.0, 1.0
    if scaling == "banded":
        turns = 8192.0 * f / (2.0 * math.pi)
        s = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return (1.0 - s) * f / 8.0 + s * f, 1.0
    if scaling == "yarn":
        at = [rotary * math.log(8192.0 / (2.0 * math.pi * turns)) / (2.0 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / 16.0 * ramp + f * (1.0 - ramp), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


_rope_arguments = {"none": None, "linear": {"kind": "linear", "factor": 8.0}, "ntk": {"kind": "ntk", "factor": 8.0},
                   "banded": {"kind": "banded", "factor": 8.0, "low": 1.0, "high": 4.0, "length": 8192},
                   "yarn": {"kind": "yarn", "factor": 16.0, "low": 1.0, "high": 32.0, "length": 8192}}

_tables = {}


def _codebook(bits):
    """Lloyd-Max centroids and boundaries (fp32) of one coordinate of a uniform unit
    vector in 128 dimensions, density ~ (1 - t^2)^62.5: each centroid is the mean of its
    cell, each boundary the midpoint of its neighbours."""
    if bits not in _tables:
        x, w = np.polynomial.legendre.leggauss(80)
        half = 1 << (bits - 1)
        c = np.linspace(0.02, 0.24, half)
        for _ in range(100000):
            lo = np.concatenate([[0.0], 0.5 * (c[1:] + c[:-1])])
            hi = np.concatenate([lo[1:], [1.0]])
            t = 0.5 * (hi - lo)[:, None] * x + 0.5 * (hi + lo)[:, None]
            mass = 0.5 * (hi - lo) * ((1.0 - t * t) ** 62.5 @ w)
            new = ((1.0 - lo * lo) ** 63.5 - (1.0 - hi * hi) ** 63.5) / 127.0 / mass
            done = np.max(np.abs(new - c)) < 1e-15
            c = new
            if done:
                break
        c = c.astype(np.float32)
        c = np.concatenate([-c[::-1], c])
        _tables[bits] = c, (c[1:] + c[:-1]) * np.float32(0.5)
    return _tables[bits]


def _hadamard():
    h = torch.ones(1, 1, dtype=torch.float64)
    for _ in range(7):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(D)


def _rotation(signs, dtype):
    """Pi = H diag(signs) / sqrt(128), as a matrix."""
    return (_hadamard().to(signs.device) * signs.double()).to(dtype)


# ------------------------------------------------------------------- the inputs

def _own_lens(batch, most):
    """Own tokens of each sequence: spread over 0 .. most, the first has most, the last none
    where there are two sequences at least."""
    if batch == 1:
        return np.array([most])
    return np.array([most - (i * most + batch - 2) // (batch - 1) for i in range(batch)])


def _channel_normal(shape, gen, dtype):
    """N(0, 1) with lognormal scales for each head and channel, as keys and values come."""
    scale = torch.exp(torch.randn(shape[-2:], generator=gen, device="cuda"))
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _layer(case, blocks, signs):
    import turboquant_quantized_kv_gb300 as tq
    if case["fmt"] == "bf16":
        return tq.Layer(blocks, case["hkv"], kv_format="bf16")
    return tq.Layer(blocks, case["hkv"], kv_format=case["fmt"], bits_k=case["bits_k"], bits_v=case["bits_v"],
                    rotation=signs.cpu().numpy())


def _positions(case, gen):
    n, far = case["tokens"], case["far"]
    if n <= 256:  # a decode step: every sequence somewhere else
        return torch.randint(0, far, (n,), generator=gen, device="cuda")
    # a prompt batch: three ragged sequences one after another
    cut = [n // 2, n // 2 + n // 3, n]
    at = torch.arange(n, device="cuda")
    start = torch.where(at < cut[0], 0, torch.where(at < cut[1], cut[0], cut[1]))
    return at - start + max(0, far - n)


def _write_pages(codes, gamma, bits):
    """Pages [blocks][heads][page bytes]: sixteen LSB-first records, then sixteen fp32 norms."""
    nb, h = codes.shape[:2]
    c = codes.to(torch.int32)
    if bits == 3:
        c = c.view(nb, h, BLOCK, D // 8, 8)
        word = (c << (3 * torch.arange(8, device=c.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
        rec = torch.stack([word & 255, (word >> 8) & 255, (word >> 16) & 255], -1)
    else:
        per = 8 // bits
        c = c.view(nb, h, BLOCK, D // per, per)
        rec = (c << (bits * torch.arange(per, device=c.device, dtype=torch.int32))).sum(-1)
    rec = rec.reshape(nb, h, -1).to(torch.uint8)
    return torch.cat([rec, gamma.contiguous().view(torch.uint8).view(nb, h, -1)], -1)


def _stored(case, which, blocks, gen, signs):
    """A pool full of stored keys (0) or values (1), as bytes in the layer's page layout."""
    x = _channel_normal((blocks * BLOCK, case["hkv"], D), gen, torch.bfloat16)
    x = x.view(blocks, BLOCK, case["hkv"], D).transpose(1, 2).contiguous()
    if case["fmt"] == "bf16":
        return x.view(torch.uint8).reshape(-1)
    if which == 0 and case["fmt"] == "k8v4":
        return x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1)
    bits = case["bits_k"] if which == 0 else case["bits_v"]
    cents, bounds = (torch.from_numpy(t).cuda() for t in _codebook(bits))
    x = x.float() @ _rotation(signs, torch.float32).t()
    n = x.norm(dim=-1, keepdim=True)
    codes = torch.bucketize(x / n, bounds, right=True)
    gamma = n.squeeze(-1) / cents[codes].norm(dim=-1)
    return _write_pages(codes, gamma, bits).reshape(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    draws = np.random.default_rng(seed)
    state = {"case": dict(case)}
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] in ("rope", "append"):
        n = case["tokens"]
        kind = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
        qkv = _channel_normal((n, hq + 2 * hkv, D), gen, kind)  # the fused projection
        state["q"], state["k"], state["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        state["positions"] = _positions(case, gen)
        state["inv_freq"], state["amplitude"] = _frequencies(case["rotary"], case["scaling"])
        if own:
            import turboquant_quantized_kv_gb300 as tq
            state["rope"] = tq.Rope(case["rotary"], base=500000.0, layout=case["layout"],
                                    scaling=_rope_arguments[case["scaling"]])
    signs = torch.from_numpy(np.where(draws.random(D) < 0.5, -1.0, 1.0).astype(np.float32)).cuda()
    if case["op"] == "append":
        blocks = -(-n // BLOCK) + 3
        table = torch.from_numpy(draws.permutation(blocks)).cuda()
        at = torch.arange(n, device="cuda")
        slots = table[at // BLOCK] * BLOCK + at % BLOCK
        state["slots"] = torch.where(at < n - case["skip"], slots, -1)
        state["signs"], state["blocks"] = signs, blocks
        if own:
            state["layer"] = _layer(case, blocks, signs)
    if case["op"] == "prefix":
        b, p = case["batch"], case["prefix"]
        pb = -(-p // BLOCK)
        lens = _own_lens(b, case["own"])
        width = -(-int(lens.max()) // BLOCK)
        blocks = pb + b * width + 2
        ids = draws.permutation(blocks).astype(np.int32)
        state["prefix_table"] = torch.from_numpy(ids[:pb]).cuda()
        state["block_table"] = torch.from_numpy(ids[pb:pb + b * width].reshape(b, width)).cuda()
        state["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        state["q"] = torch.randn((b, hq, D), generator=gen, device="cuda").to(torch.bfloat16)
        state["signs"], state["blocks"] = signs, blocks
        pools = [_stored(case, which, blocks, gen, signs) for which in (0, 1)]
        if own:
            layer = state["layer"] = _layer(case, blocks, signs)
            layer.k_cache.copy_(pools[0])
            layer.v_cache.copy_(pools[1])
            state["workspace"] = torch.zeros(layer.prefix_workspace_bytes(b, hq, p, width), dtype=torch.uint8,
                                             device="cuda")
        else:
            state["k_pool"], state["v_pool"] = pools
    return state


# -------------------------------------------------------------- the plain forms

def _turn(x, cos, sin, layout, rotary):
    """x [tokens, heads, D] with its pairs turned by [tokens, rotary / 2] angles."""
    cos, sin = cos[:, None], sin[:, None]
    r = x[..., :rotary]
    if layout == "half":
        a, b = r[..., :rotary // 2], r[..., rotary // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rotary:]], -1)


def _cos_sin(state, dtype):
    case = state["case"]
    f = torch.from_numpy(state["inv_freq"]).cuda()
    angle = state["positions"].double()[:, None] * f
    sin = torch.sin(angle)
    if case.get("transpose"):
        sin = -sin
    return (torch.cos(angle) * state["amplitude"]).to(dtype), (sin * state["amplitude"]).to(dtype)


def _rope(state):
    case = state["case"]
    cos, sin = _cos_sin(state, torch.float32)
    out = [_turn(x.float(), cos, sin, case["layout"], case["rotary"]).to(x.dtype) for x in (state["q"], state["k"])]
    return {"q": out[0], "k": out[1]}


def _code_and_read(x, signs, bits, slots, blocks):
    """x [tokens, heads, D] in 64 bits -> codes and norms stored at the slots, read back as bf16."""
    cents, bounds = (torch.from_numpy(t).cuda().double() for t in _codebook(bits))
    pi = _rotation(signs, torch.float64)
    y = x @ pi.t()
    n = y.norm(dim=-1, keepdim=True)
    codes = torch.bucketize(torch.where(n > 0, y / n, torch.zeros_like(y)), bounds, right=True)
    gamma = (n.squeeze(-1) / cents[codes].norm(dim=-1)).float()
    pool = torch.zeros((blocks * BLOCK, x.shape[1], D), dtype=torch.uint8, device="cuda")
    norms = torch.zeros((blocks * BLOCK, x.shape[1]), device="cuda")
    live = slots >= 0
    pool[slots[live]] = codes[live].to(torch.uint8)
    norms[slots[live]] = gamma[live]
    at = slots.clamp(min=0)
    back = (cents[pool[at].long()] @ pi).float() * norms[at][..., None]
    return (back * live[:, None, None]).to(torch.bfloat16)


def _append(state):
    case, slots, blocks = state["case"], state["slots"], state["blocks"]
    cos, sin = _cos_sin(state, torch.float64 if case["fmt"] != "bf16" else torch.float32)
    q, k, v = (state[t] for t in "qkv")
    q = _turn(q.float(), cos.float(), sin.float(), case["layout"], case["rotary"]).to(torch.bfloat16)
    k = _turn(k.to(cos.dtype), cos, sin, case["layout"], case["rotary"])
    out = {"q": q, "k": k.to(torch.bfloat16)}
    live = slots >= 0

    def pool(x, dtype):
        p = torch.zeros((blocks, case["hkv"], BLOCK, D), dtype=dtype, device="cuda")
        p[slots[live] // BLOCK, :, slots[live] % BLOCK] = x[live].to(dtype)
        return p

    if case["fmt"] == "bf16":
        out["k_pool"], out["v_pool"] = pool(k, torch.bfloat16), pool(v, torch.bfloat16)
        return out
    if case["fmt"] == "k8v4":
        out["k_pool"] = pool(k.clamp(-448, 448), torch.float32).to(torch.float8_e4m3fn)
    else:
        out["k_stored"] = _code_and_read(k, state["signs"], case["bits_k"], slots, blocks)
    out["v_stored"] = _code_and_read(v.double(), state["signs"], case["bits_v"], slots, blocks)
    return out


def _read_pages(pool, ids, bits, hkv, table):
    """Codes and norms of the blocks `ids`: centroids fp32 [n, heads, 16, D], norms [n, heads, 16]."""
    rb = bits * D // 8
    pages = pool.view(-1, hkv, BLOCK * (rb + 4))[ids]
    rec = pages[..., :BLOCK * rb].reshape(*pages.shape[:2], BLOCK, rb)
    if bits == 3:
        b = rec.reshape(*rec.shape[:-1], D // 8, 3).to(torch.int32)
        word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        codes = (word[..., None] >> (3 * torch.arange(8, device="cuda"))) & 7
    else:
        codes = (rec[..., None] >> (bits * torch.arange(8 // bits, device="cuda", dtype=torch.uint8))) & ((1 << bits) - 1)
    codes = codes.reshape(*rec.shape[:3], D)
    gamma = pages[..., BLOCK * rb:].contiguous().view(torch.float32)
    return table[codes.long()], gamma


def _read(state, which, ids):
    """Keys or values of the blocks `ids` as the logits use them, fp32 [heads, n * 16, D]."""
    case = state["case"]
    pool = state["k_pool"] if which == 0 else state["v_pool"]
    hkv = case["hkv"]
    if case["fmt"] == "bf16":
        x = pool.view(torch.bfloat16).view(-1, hkv, BLOCK, D)[ids].float()
    elif which == 0 and case["fmt"] == "k8v4":
        x = pool.view(-1, hkv, BLOCK, D)[ids].view(torch.float8_e4m3fn).float()
    else:
        bits = case["bits_k"] if which == 0 else case["bits_v"]
        c, gamma = _read_pages(pool, ids, bits, hkv, torch.from_numpy(_codebook(bits)[0]).cuda())
        x = c * gamma[..., None]
    return x.transpose(0, 1).reshape(hkv, -1, D)


def _prefix(state):
    case = state["case"]
    b, hkv, p = case["batch"], case["hkv"], case["prefix"]
    g = case["hq"] // hkv
    pi = _rotation(state["signs"], torch.float32)
    q = state["q"].float() / math.sqrt(D)
    if case["fmt"] == "packed":
        q = q @ pi.t()
    q = q.view(b, hkv, g, D).transpose(0, 1)  # [hkv, b, g, D]
    table, lens = state["block_table"].long(), state["lens"]
    s1 = q.reshape(hkv, b * g, D) @ _read(state, 0, state["prefix_table"].long())[:, :p].transpose(1, 2)
    s1 = s1.view(hkv, b, g, p)
    width = table.shape[1] * BLOCK
    s2 = q @ _read(state, 0, table.view(-1)).view(hkv, b, width, D).transpose(2, 3)
    dead = torch.arange(width, device="cuda") >= lens[:, None, None]
    s2 = s2.masked_fill(dead, -math.inf)
    top = torch.maximum(s1.amax(-1, keepdim=True), s2.amax(-1, keepdim=True))
    s1, s2 = torch.exp(s1 - top), torch.exp(s2 - top)
    total = s1.sum(-1, keepdim=True) + s2.sum(-1, keepdim=True)
    o = (s1.view(hkv, b * g, p) @ _read(state, 1, state["prefix_table"].long())[:, :p]).view(hkv, b, g, D)
    o = o + s2 @ _read(state, 1, table.view(-1)).view(hkv, b, width, D)
    o = o / total
    if case["fmt"] != "bf16":
        o = o @ pi
    return o.transpose(0, 1).reshape(b, case["hq"], D).to(torch.bfloat16)


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if not own:
        return {"rope": _rope, "append": _append, "prefix": _prefix}[case["op"]](state)
    import turboquant_quantized_kv_gb300 as tq
    if case["op"] == "rope":
        q, k = tq.apply_rope(state["rope"], state["positions"], state["q"], state["k"], transpose=case["transpose"])
        return {"q": q, "k": k}
    layer = state["layer"]
    if case["op"] == "prefix":
        return layer.prefix_decode(state["q"], state["prefix_table"], case["prefix"], state["block_table"],
                                   state["lens"], workspace=state["workspace"])
    k_out = torch.empty(state["k"].shape, dtype=torch.bfloat16, device="cuda")
    q = layer.rope_append(state["rope"], state["k"], state["v"], state["positions"], state["slots"], q=state["q"],
                          k_out=k_out)
    out = {"q": q, "k": k_out}
    shape = (state["blocks"], case["hkv"], BLOCK, D)
    if case["fmt"] == "bf16":
        out["k_pool"] = layer.k_cache.view(torch.bfloat16).view(shape)
        out["v_pool"] = layer.v_cache.view(torch.bfloat16).view(shape)
        return out
    if case["fmt"] == "k8v4":
        out["k_pool"] = layer.k_cache.view(torch.float8_e4m3fn).view(shape)
    else:
        out["k_stored"] = layer.dequantize(0, state["slots"], out_dtype=torch.bfloat16)
    out["v_stored"] = layer.dequantize(1, state["slots"], out_dtype=torch.bfloat16)
    return out


# ------------------------------------------------- the definitions in 64 bits

def _exact_turn(x, positions, inv_freq, amplitude, layout, rotary, transpose):
    """Pairs as complex numbers, times amplitude e^{+-i position frequency}."""
    r = x[..., :rotary].double()
    z = torch.complex(r[..., :rotary // 2].contiguous(), r[..., rotary // 2:].contiguous()) if layout == "half" \
        else torch.view_as_complex(r.reshape(*r.shape[:-1], rotary // 2, 2).contiguous())
    # whole turns leave the angle before the sine is taken
    turns = positions.double()[:, None] * torch.from_numpy(inv_freq / (2.0 * math.pi)).to(x.device)
    angle = 2.0 * math.pi * (turns - torch.floor(turns))
    z = z * torch.polar(torch.full_like(angle, amplitude), -angle if transpose else angle)[:, None]
    r = torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).flatten(-2)
    return torch.cat([r, x[..., rotary:].double()], -1)


def _butterfly(x):
    """The orthonormal Walsh-Hadamard transform of the last axis, stage by stage."""
    shape = x.shape
    for bit in range(7):
        x = x.reshape(*shape[:-1], D >> (bit + 1), 2, 1 << bit)
        x = torch.stack([x[..., 0, :] + x[..., 1, :], x[..., 0, :] - x[..., 1, :]], -2)
    return x.reshape(shape) / math.sqrt(D)


def _exact_stored(x, signs, bits, slots):
    """The stored value of each token: nearest centroid of each rotated unit coordinate, the norm kept."""
    c, b = (torch.from_numpy(t).to(x.device).double() for t in _codebook(bits))
    out = torch.zeros_like(x)
    for lo in range(0, x.shape[0], 8192):
        y = _butterfly(x[lo:lo + 8192] * signs.double())
        n = y.square().sum(-1, keepdim=True).sqrt()
        unit = torch.where(n > 0, y / n.clamp(min=1e-300), 0.0)
        idx = sum((unit >= t).long() for t in b)
        v = c[idx]
        v = v * (n / v.square().sum(-1, keepdim=True).sqrt())
        out[lo:lo + 8192] = _butterfly(v) * signs.double()
    return out * (slots >= 0)[:, None, None]


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("rope", "append"):
        q, k = (_exact_turn(state[t], state["positions"], state["inv_freq"], state["amplitude"], case["layout"],
                            case["rotary"], case.get("transpose", False)) for t in "qk")
        if case["op"] == "rope":
            return {"q": q, "k": k}
        out = {"q": q, "k": k}
        slots, v = state["slots"], state["v"].double()
        live = slots >= 0

        def pool(x):
            p = torch.zeros((state["blocks"] * BLOCK, case["hkv"], D), dtype=torch.float64, device="cuda")
            p[slots[live]] = x[live]
            return p.view(state["blocks"], BLOCK, case["hkv"], D).transpose(1, 2).contiguous()

        if case["fmt"] == "bf16":
            out["k_pool"], out["v_pool"] = pool(k), pool(v)
            return out
        if case["fmt"] == "k8v4":
            out["k_pool"] = pool(k.clamp(-448, 448))
        else:
            out["k_stored"] = _exact_stored(k, state["signs"], case["bits_k"], slots)
        out["v_stored"] = _exact_stored(v, state["signs"], case["bits_v"], slots)
        return out
    # softmax attention of each sequence over its prefix and its own tokens, from the stored values
    b, hkv, p = case["batch"], case["hkv"], case["prefix"]
    g = case["hq"] // hkv
    pools = [state["k_pool"], state["v_pool"]] if not own else [state["layer"].k_cache, state["layer"].v_cache]

    def values(which, ids, count):
        bits = case["bits_k"] if which == 0 else case["bits_v"]
        pool = pools[which]
        if case["fmt"] == "bf16":
            x = pool.view(torch.bfloat16).view(-1, hkv, BLOCK, D)[ids].double()
        elif case["fmt"] == "k8v4" and which == 0:
            x = pool.view(torch.float8_e4m3fn).view(-1, hkv, BLOCK, D)[ids].double()
        else:
            size = BLOCK * (bits * D // 8)
            page = pool.view(-1, hkv, size + 4 * BLOCK)[ids]
            bit = (page[..., :size].reshape(*page.shape[:2], BLOCK, -1, 1) >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
            bit = bit.reshape(*bit.shape[:3], D, bits)
            idx = sum(bit[..., j].long() << j for j in range(bits))
            x = torch.from_numpy(_codebook(bits)[0]).cuda().double()[idx]
            x = x * page[..., size:].contiguous().view(torch.float32).double()[..., None]
            x = _butterfly(x) * state["signs"].double()
        return x.transpose(0, 1).reshape(hkv, -1, D)[:, :count]

    head = [values(w, state["prefix_table"].long(), p) for w in (0, 1)]
    out = torch.zeros((b, case["hq"], D), dtype=torch.float64, device="cuda")
    lens = state["lens"].tolist()
    for i in range(b):
        ids = state["block_table"][i].long()
        k, v = (torch.cat([head[w], values(w, ids, lens[i])], 1) for w in (0, 1))
        s = state["q"][i].double().view(hkv, g, D) @ k.transpose(1, 2) / math.sqrt(D)
        w = torch.exp(s - torch.logsumexp(s, -1, keepdim=True))
        out[i] = (w @ v).reshape(case["hq"], D)
    return out
