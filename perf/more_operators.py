"""A cache held in 8 bits and the blocks that sequences share: cases, inputs, plain forms.

Operators that a server of the paged KV cache calls one after another:

* append  -- keys and values of new tokens stored in 8 bits, one scale for each block of 16
             tokens and head: step = (largest magnitude of the block) / 127, code = x / step
             rounded to the nearest (ties to even); when new tokens of a block need a larger
             step, the codes that are there already are rounded to it; slot 0 begins a block;
* decode  -- attention of one token a sequence over such a cache;
* attend  -- attention of the last tokens of each sequence (a prompt, a chunk of one, some
             drafted tokens to verify), causal, over the same cache;
* fork    -- sequences of the cache in a new order, some several times, some not at all:
             whole blocks are shared by count, a block that is not full is copied for every
             row but the first; then room for one more token a row;
* compact -- the blocks in use moved to the low end of the pools, tables rewritten.

`own` chooses between the plain forms (elementary torch operations) and the package's entry
points.
"""

import math

import torch

own = False

D = 128  # head dimension of every cache layer
BLOCK = 16  # tokens a page
TINY = 2.0 ** -126  # the least step of a block


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of a batch of 64: a token each, most of them in the middle of a block
        {"name": "append_step", "op": "append", "batch": 64, "new": 1, "past": 1000, "ragged": False, "hkv": 8,
         "dtype": "bf16", "order": "sequence", "skip": 0},
        # ragged prompts of a batch, some of them behind earlier tokens, a tail of padding
        {"name": "append_prompts", "op": "append", "batch": 9, "new": 3001, "past": 333, "ragged": True, "hkv": 8,
         "dtype": "bf16", "order": "sequence", "skip": 37},
        # two short answers: the smallest attention, where latency counts
        {"name": "decode_pair", "op": "decode", "batch": 2, "ctx": 333, "ragged": True, "hq": 32, "hkv": 8,
         "dtype": "bf16"},
        # the decode step of a batch of 16 at 8192 tokens
        {"name": "decode_batch", "op": "decode", "batch": 16, "ctx": 8192, "ragged": False, "hq": 32, "hkv": 8,
         "dtype": "bf16"},
        # a batch of very different lengths, one of them empty, groups of eight query heads, fp32 queries
        {"name": "decode_ragged", "op": "decode", "batch": 64, "ctx": 15001, "ragged": True, "hq": 64, "hkv": 8,
         "dtype": "f32"},
        # few sequences of long contexts, groups of eight: the most memory
        {"name": "decode_long", "op": "decode", "batch": 4, "ctx": 131072, "ragged": False, "hq": 64, "hkv": 8,
         "dtype": "bf16"},
        # drafted tokens of a batch, verified at once
        {"name": "attend_verify", "op": "attend", "batch": 24, "new": 5, "past": 3000, "ragged": True, "hq": 32,
         "hkv": 8, "dtype": "bf16", "skip": 3},
        # ragged prompts from their first token on
        {"name": "attend_prompts", "op": "attend", "batch": 6, "new": 4097, "past": 0, "ragged": True, "hq": 32,
         "hkv": 8, "dtype": "bf16", "skip": 0},
        # a chunk of one long prompt, groups of eight: the most products
        {"name": "attend_chunk", "op": "attend", "batch": 1, "new": 2048, "past": 30000, "ragged": False, "hq": 64,
         "hkv": 8, "dtype": "bf16", "skip": 0},
        # a step of a search with four beams for eight requests, two layers: a few tails to copy
        {"name": "fork_beams", "op": "fork", "rows": 32, "group": 4, "times": 1, "ctx": 500, "layers": 2, "hkv": 8,
         "bits": 4},
        # 64 prompts answered eight times each: every answer's tail block is a copy
        {"name": "fork_samples", "op": "fork", "rows": 64, "group": 1, "times": 8, "ctx": 2000, "layers": 4, "hkv": 8,
         "bits": 4},
        # a pool half of whose sequences have gone
        {"name": "compact_pool", "op": "compact", "rows": 48, "ctx": 3000, "layers": 4, "hkv": 8, "bits": 4,
         "free": 0.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["append", "decode", "attend", "fork", "compact"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    ragged = rng.random() < 0.7
    if op == "append":
        batch = _log_int(rng, 1, 128)
        return {"op": op, "batch": batch, "new": _log_int(rng, 1, 20000 // batch), "past": rng.randint(0, 2000),
                "ragged": ragged, "hkv": hkv, "dtype": dtype, "order": rng.choice(["sequence", "time"]),
                "skip": rng.choice([0, 0, 1, 13, 100])}
    if op == "decode":
        batch = _log_int(rng, 1, 256)
        ctx = _log_int(rng, 1, min(131072, 500000 * 64 // (batch * max(8 * hkv, hq))))
        return {"op": op, "batch": batch, "ctx": ctx, "ragged": ragged, "hq": hq, "hkv": hkv, "dtype": dtype}
    if op == "attend":
        batch = _log_int(rng, 1, 32)
        new = _log_int(rng, 1, 4000 // batch)
        past = rng.choice([0, _log_int(rng, 1, min(30000, 2000 * 30000 * 64 // (batch * new * hq)))])
        return {"op": op, "batch": batch, "new": new, "past": past, "ragged": ragged, "hq": hq, "hkv": hkv,
                "dtype": "bf16", "skip": rng.choice([0, 0, 1, 7])}
    layers, bits = rng.randint(1, 4), rng.choice([2, 3, 4])
    if op == "fork":
        group = rng.choice([1, 2, 3, 4, 5, 8])
        rows = group * _log_int(rng, 1, 64 // group)
        return {"op": op, "rows": rows, "group": group, "times": rng.choice([1, 1, 2, 3, 8]), "ctx": _log_int(rng, 1, 2000),
                "layers": layers, "hkv": hkv, "bits": bits}
    return {"op": op, "rows": _log_int(rng, 1, 64), "ctx": _log_int(rng, 1, 2000), "layers": layers, "hkv": hkv,
            "bits": bits, "free": rng.choice([0.1, 0.5, 0.5, 0.9])}


def _lens(n, most, ragged, least=0):
    """Lengths of n sequences: the first the longest; ragged: of every size, the second the least."""
    if not ragged:
        return [most] * n
    part = [(0.31 + 0.6180339887 * i) % 1.0 for i in range(n)]
    out = [max(least, int(most * p * p)) for p in part]
    out[0] = most
    if n > 2:
        out[1] = least
    return out


def _new_past(case):
    """(new tokens, earlier tokens) of each sequence of an append or attend."""
    b = case["batch"]
    return _lens(b, case["new"], case["ragged"], 1), list(reversed(_lens(b, case["past"], case["ragged"] or case["new"] == 1)))


def _parents(case):
    """The old row of each new row: of every group about six tenths go on, some of them twice; then each row `times` times."""
    rows, group, times = case["rows"], case["group"], case["times"]
    base = [i - i % group + (i % group) * 6 // 10 for i in range(rows)]
    return [p for p in base for _ in range(times)]


def _row_lens(case):
    return _lens(case["rows"], case["ctx"], True, 1 if case["ctx"] > 0 else 0)


def work(case):
    """Bytes and operations one pass cannot do without."""
    op, hkv = case["op"], case["hkv"]
    record = 2 * hkv * (D + 4.0 / BLOCK)  # bytes a token has in the cache
    if op == "append":
        new, _ = _new_past(case)
        n, e = sum(new), 2 if case["dtype"] == "bf16" else 4
        # read and stored; the blocks touched are read back as fp32 values
        rows = sum((k + BLOCK - 1) // BLOCK for k in new) * BLOCK
        return {"bytes": n * 2 * hkv * D * e + n * record + 8 * n + rows * (record + 2 * hkv * D * 4),
                "flops": 6 * n * hkv * D}
    if op == "decode":
        lens, e = _lens(case["batch"], case["ctx"], case["ragged"]), 2 if case["dtype"] == "bf16" else 4
        return {"bytes": sum(lens) * record + 2 * case["batch"] * case["hq"] * D * e + sum(lens) // 4,
                "flops": 4 * sum(lens) * case["hq"] * D}
    if op == "attend":
        new, past = _new_past(case)
        pairs = sum(k * p + k * (k + 1) // 2 for k, p in zip(new, past))
        tokens = sum(new) + sum(past)
        return {"bytes": tokens * record + 2 * sum(new) * case["hq"] * D * 2 + tokens // 4,
                "flops": 4 * pairs * case["hq"] * D}
    block = 2 * hkv * BLOCK * (case["bits"] * D // 8 + 4) * case["layers"]
    lens = _row_lens(case)
    if op == "fork":
        parents = _parents(case)
        again = [p for i, p in enumerate(parents) if p in parents[:i] and lens[p] % BLOCK]
        entries = sum(-(-lens[p] // BLOCK) for p in parents)
        return {"bytes": 2 * len(again) * block + 8 * entries, "flops": 0}
    used = sum(-(-n // BLOCK) for n in lens)
    total = int(used / (1.0 - case["free"])) + 1
    return {"bytes": 2 * int(used * (1.0 - used / total)) * block + 8 * used + 4 * total, "flops": 0}


# ----------------------------------------------------------------- 8-bit blocks

def _store(codes, step, x, slots):
    """x [n, heads, D] stored at `slots` (negative: nowhere) of a pool of codes [blocks, heads, 16, D] with
    steps [blocks, heads], in place; in 64 bits, so that a code next to a border goes to its side."""
    live = slots >= 0
    x, at = x[live].double(), slots[live]
    block, row = at // BLOCK, at % BLOCK
    top = torch.zeros(step.shape, dtype=torch.float64, device=x.device)
    top.scatter_reduce_(0, block[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    touched = torch.zeros(step.shape[0], dtype=torch.bool, device=x.device)
    begun = touched.clone()
    touched[block] = True
    begun[block[row == 0]] = True
    old = torch.where(begun[:, None], 0.0, step.double())
    new = torch.maximum(old, (top / 127).float().double().clamp(min=TINY))
    ids = touched.nonzero()[:, 0]
    # codes that are there: rounded to the new step; a block that begins has none
    kept = torch.round(codes[ids].double() * old[ids, :, None, None] / new[ids, :, None, None])
    codes[ids] = kept.to(torch.int8)
    step[ids] = new[ids].float()
    codes[block, :, row] = torch.round(x / new[block][:, :, None]).clamp(-127, 127).to(torch.int8)


def _values(codes, step):
    """The values that codes [blocks, heads, 16, D] stand for, fp32 [blocks, heads, 16, D]."""
    return codes.float() * step[:, :, None, None]


def _table(gen, lens, width, blocks):
    """A block table of random distinct blocks, -1 behind each row's last; int32 [rows, width]."""
    ids = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    used = torch.tensor([-(-n // BLOCK) for n in lens], device="cuda")
    mask = torch.arange(width, device="cuda") < used[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[mask] = ids[:int(used.sum())]
    return table


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hkv = case["hkv"]
    state = {"case": case}
    if case["op"] in ("fork", "compact"):
        return _prepare_blocks(state, gen)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    scale = torch.exp(_normal(gen, (hkv, D), torch.float32))  # lognormal channels
    if case["op"] == "decode":
        lens = _lens(case["batch"], case["ctx"], case["ragged"])
        state["q"] = _normal(gen, (case["batch"], case["hq"], D), dtype)
    else:
        new, past = _new_past(case)
        lens = [a + b for a, b in zip(new, past)]
    width = max(1, -(-max(lens) // BLOCK))
    used = sum(-(-n // BLOCK) for n in lens)
    blocks = used + 3
    state["table"] = _table(gen, lens, width, blocks)
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if own:
        import turboquant_quantized_kv_gb300 as tq
        state["layer"] = tq.Layer(blocks, hkv, kv_format="int8")
    else:
        state["codes"] = [torch.zeros((blocks, hkv, BLOCK, D), dtype=torch.int8, device="cuda") for _ in "kv"]
        state["step"] = [torch.zeros((blocks, hkv), dtype=torch.float32, device="cuda") for _ in "kv"]

    def put(k, v, slots):
        if own:
            state["layer"].append(k, v, slots)
        else:
            for w, x in enumerate((k, v)):
                _store(state["codes"][w], state["step"][w], x, slots)

    if case["op"] == "append":
        # where the new tokens go; the tokens before them in the same block are there already
        where = [(b, p, p + n) for b, (n, p) in enumerate(zip(new, past))]
        slots, early = [], []
        for b, lo, hi in where:
            at = torch.arange(lo - lo % BLOCK, hi, device="cuda")
            at = state["table"][b, at // BLOCK].long() * BLOCK + at % BLOCK
            early.append(at[:lo % BLOCK])
            slots.append(at[lo % BLOCK:])
        if case["order"] == "time":  # token after token of all sequences
            turn = torch.cat([torch.arange(n) for n in new]).argsort(stable=True).cuda()
            slots = torch.cat(slots)[turn]
        else:
            slots = torch.cat(slots)
        early = torch.cat(early)
        if early.numel():
            put(*(_normal(gen, (early.numel(), hkv, D), dtype) * scale.to(dtype) for _ in "kv"), early)
        state["rows"] = ((slots // BLOCK).unique()[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).view(-1)
        state["slots"] = torch.cat([slots, torch.full((case["skip"],), -1, dtype=torch.int64, device="cuda")])
        n = state["slots"].numel()
        state["k"], state["v"] = (_normal(gen, (n, hkv, D), dtype) * scale.to(dtype) for _ in "kv")
        return state
    # a full cache: every block of the table from its first row on
    part = 1 << 15
    for lo in range(0, blocks, part):
        n = min(part, blocks - lo) * BLOCK
        put(*((_normal(gen, (n, hkv, D), torch.float32) * scale).to(torch.bfloat16) for _ in "kv"),
            torch.arange(lo * BLOCK, lo * BLOCK + n, device="cuda"))
    if case["op"] == "attend":
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        state["plan"] = list(zip(starts, new, past))
        state["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        state["q"] = _normal(gen, (starts[-1] + case["skip"], case["hq"], D), dtype)
        state["out"] = torch.zeros((starts[-1] + case["skip"], case["hq"], D), dtype=dtype, device="cuda")
    if own:
        layer, n = state["layer"], state["q"].shape[0]
        size = layer.workspace_bytes(n, case["hq"], width) if case["op"] == "decode" else \
            layer.attend_workspace_bytes(n, case["batch"], case["hq"], width)
        state["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return state


def _prepare_blocks(state, gen):
    case = state["case"]
    lens, hkv = _row_lens(case), case["hkv"]
    width = -(-max(lens) // BLOCK) + 1
    used = sum(-(-n // BLOCK) for n in lens)
    if case["op"] == "fork":
        blocks = used + len(_parents(case)) * 2 + 5
        state["parents"] = torch.tensor(_parents(case), dtype=torch.int32, device="cuda")
    else:
        blocks = int(used / (1.0 - case["free"])) + 1
    state["table"] = _table(gen, lens, width, blocks)
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "fork" and case["group"] > 1:
        # the rows of a group share the whole blocks of their first half, as beams of one request do
        first = torch.arange(case["rows"], device="cuda")
        first = first - first % case["group"]
        common = torch.minimum(state["lens"], state["lens"][first]) // (2 * BLOCK)
        state["table"] = torch.where(torch.arange(width, device="cuda") < common[:, None], state["table"][first], state["table"])
    held = state["table"][state["table"] >= 0].long()
    state["refs"] = torch.bincount(held, minlength=blocks).to(torch.int32)
    size = blocks * hkv * BLOCK * (case["bits"] * D // 8 + 4)
    pools = [torch.randint(0, 256, (size,), generator=gen, dtype=torch.uint8, device="cuda") for _ in range(2 * case["layers"])]
    if own:
        import turboquant_quantized_kv_gb300 as tq
        state["layers"] = [tq.Layer(blocks, hkv, bits_k=case["bits"], bits_v=case["bits"], layer=i) for i in range(case["layers"])]
        for i, layer in enumerate(state["layers"]):
            layer.k_cache.copy_(pools[2 * i])
            layer.v_cache.copy_(pools[2 * i + 1])
        state["pools"] = [p for layer in state["layers"] for p in (layer.k_cache, layer.v_cache)]
        state["blocks"] = tq.Blocks(blocks)
    else:
        state["pools"] = pools
    return state


# -------------------------------------------------------------- the plain forms

def _append(state):
    codes, step = ([t.clone() for t in state[name]] for name in ("codes", "step"))
    _store(codes[0], step[0], state["k"], state["slots"])
    _store(codes[1], step[1], state["v"], state["slots"])
    block, row = state["rows"] // BLOCK, state["rows"] % BLOCK
    k, v = (codes[w][block, :, row].float() * step[w][block][:, :, None] for w in (0, 1))
    return {"k_stored": k, "v_stored": v}


def _decode(state):
    case = state["case"]
    b, hkv = case["batch"], case["hkv"]
    g = case["hq"] // hkv
    ids = state["table"].long().clamp(min=0).view(-1)
    k, v = (_values(state["codes"][w][ids], state["step"][w][ids]).view(b, -1, hkv, BLOCK, D).transpose(1, 2)
            .reshape(b, hkv, -1, D) for w in (0, 1))
    q = state["q"].float().view(b, hkv, g, D) / math.sqrt(D)
    s = q @ k.transpose(2, 3)
    dead = torch.arange(k.shape[2], device="cuda") >= state["lens"][:, None, None, None]
    s = s.masked_fill(dead, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True)).masked_fill(dead, 0.0)
    o = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(b, case["hq"], D).to(state["q"].dtype)


def _attend(state):
    case = state["case"]
    hq, hkv = case["hq"], case["hkv"]
    out = torch.zeros_like(state["out"])
    for b, (lo, n, past) in enumerate(state["plan"]):
        ids = state["table"][b, :-(-(n + past) // BLOCK)].long()
        k, v = (_values(state["codes"][w][ids], state["step"][w][ids]).transpose(0, 1).reshape(hkv, 1, -1, D)[:, :, :n + past]
                for w in (0, 1))
        q = state["q"][lo:lo + n].float().transpose(0, 1).reshape(hkv, hq // hkv, n, D) / math.sqrt(D)
        s = q @ k.transpose(2, 3)
        ahead = torch.arange(n + past, device="cuda") > past + torch.arange(n, device="cuda")[:, None]
        s = s.masked_fill(ahead, -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = (p @ v) / p.sum(-1, keepdim=True)
        out[lo:lo + n] = o.reshape(hq, n, D).transpose(0, 1).to(out.dtype)
    return out


def _take(refs, count):
    """The `count` lowest blocks that nobody holds; they are held once from here on."""
    free = (refs == 0).nonzero()[:count, 0]
    refs[free] = 1
    return free


def _move(pools, blocks, src, dst):
    for pool in pools:
        pages = pool.view(blocks, -1)
        pages[dst] = pages[src]


def _fork(state):
    refs, table, lens = state["refs"].clone(), state["table"], state["lens"].long()
    parents = state["parents"].long()
    cols = torch.arange(table.shape[1], device="cuda")
    used = (lens + BLOCK - 1) // BLOCK
    refs.index_add_(0, table[cols < used[:, None]].long(), torch.full((int(used.sum()),), -1, dtype=torch.int32, device="cuda"))
    n, m = table.shape[0], parents.shape[0]
    order = torch.arange(m, device="cuda")
    first = torch.full((n,), m, device="cuda").scatter_reduce_(0, parents, order, "amin")
    lens, used = lens[parents], used[parents]
    table = torch.where(cols < used[:, None], table[parents], -1)
    again = (first[parents] != order) & (lens % BLOCK != 0)
    rows = again.nonzero()[:, 0]
    src = table[rows, used[rows] - 1].long()
    table[rows, used[rows] - 1] = -1
    kept = table[table >= 0].long()
    refs.index_add_(0, kept, torch.ones_like(kept, dtype=torch.int32))
    dst = _take(refs, rows.numel())
    table[rows, used[rows] - 1] = dst.to(torch.int32)
    _move(state["pools"], refs.numel(), src, dst)
    # room for one more token a row
    more = (cols >= used[:, None]) & (cols < ((lens + BLOCK) // BLOCK)[:, None])
    table[more] = _take(refs, int(more.sum())).to(torch.int32)
    return {"table": table, "lens": lens.to(torch.int32), "refs": refs, "pools": state["pools"]}


def _compact(state):
    refs, table = state["refs"].clone(), state["table"]
    held = refs > 0
    live = int(held.sum())
    holes, movers = (~held[:live]).nonzero()[:, 0], held[live:].nonzero()[:, 0] + live
    to = torch.arange(refs.numel(), device="cuda", dtype=torch.int32)
    to[movers] = holes.to(torch.int32)
    _move(state["pools"], refs.numel(), movers, holes)
    refs[holes] = refs[movers]
    refs[movers] = 0
    table = torch.where(table >= 0, to[table.clamp(min=0).long()], table)
    return {"table": table, "refs": refs, "live": torch.full((1,), live, dtype=torch.int32, device="cuda"), "pools": state["pools"]}


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if not own:
        return {"append": _append, "decode": _decode, "attend": _attend, "fork": _fork, "compact": _compact}[case["op"]](state)
    if case["op"] == "append":
        layer = state["layer"]
        layer.append(state["k"], state["v"], state["slots"])
        return {"k_stored": layer.dequantize(0, state["rows"]), "v_stored": layer.dequantize(1, state["rows"])}
    if case["op"] == "decode":
        return state["layer"].decode(state["q"], state["table"], state["lens"], workspace=state["workspace"])
    if case["op"] == "attend":
        return state["layer"].attend(state["q"], state["starts"], state["table"], state["lens"], out=state["out"],
                                     workspace=state["workspace"])
    blocks = state["blocks"]
    blocks.refs.copy_(state["refs"])
    if case["op"] == "fork":
        table, lens = blocks.reorder(state["layers"], state["table"], state["lens"], state["parents"])
        blocks.extend(table, lens, lens + 1)
        return {"table": table, "lens": lens, "refs": blocks.refs, "pools": state["pools"]}
    table = state["table"].clone()
    live = blocks.compact(state["layers"], table, state["lens"])
    return {"table": table, "refs": blocks.refs, "live": live, "pools": state["pools"]}


# ------------------------------------------------- the definitions in 64 bits

def _exact_stored(state, which, x):
    """The stored values of the touched blocks' rows: nearest multiples of the step by whole parts and what is left."""
    codes, step = state["codes"][which].clone(), state["step"][which].clone()
    slots = state["slots"]
    x, slots = x[slots >= 0].double(), slots[slots >= 0]
    ids, inverse = (slots // BLOCK).unique(return_inverse=True)
    fresh = torch.full((ids.numel(), BLOCK), -1, dtype=torch.int64, device="cuda")
    fresh[inverse, slots % BLOCK] = torch.arange(slots.numel(), device="cuda")
    taken = fresh >= 0
    rows = x[fresh.clamp(min=0)] * taken[:, :, None, None]  # [blocks, 16, heads, D]
    before = step[ids].double() * (~taken[:, 0])[:, None]
    after = torch.maximum(before, torch.clamp((rows.abs().amax((1, 3)) / 127).float().double(), min=TINY))
    old = codes[ids].double().transpose(1, 2) * before[:, None, :, None]
    rows = torch.where(taken[:, :, None, None], rows, old)

    def nearest(y, s):
        whole = torch.floor(y / s)
        whole = torch.where(y - whole * s < 0, whole - 1, torch.where(y - whole * s >= s, whole + 1, whole))
        left = 2 * (y - whole * s) - s
        return whole + ((left > 0) | ((left == 0) & (whole.remainder(2) == 1))).double()

    s = after[:, None, :, None]
    return (nearest(rows, s) * s).reshape(-1, *x.shape[1:])


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None
    state = prepare(case, seed)
    if own:  # (the same pages, as codes and steps)
        layer = state["layer"]
        every = torch.arange(layer.num_blocks * BLOCK, device="cuda")
        shape = (layer.num_blocks, BLOCK, case["hkv"], D)
        state["values"] = [layer.dequantize(w, every).double().view(shape).transpose(1, 2) for w in (0, 1)]
    else:
        state["values"] = [c.double() * s.double()[:, :, None, None] for c, s in zip(state["codes"], state["step"])]
    if case["op"] == "append":
        if own:
            return None
        return {"k_stored": _exact_stored(state, 0, state["k"]), "v_stored": _exact_stored(state, 1, state["v"])}
    lens, hkv, hq = state["lens"].tolist(), case["hkv"], case["hq"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    plan = state["plan"] if case["op"] == "attend" else [(b, 1, lens[b] - 1) for b in range(case["batch"])]
    for b, (lo, n, past) in enumerate(plan):
        if lens[b] == 0:
            continue
        ids = state["table"][b, :-(-lens[b] // BLOCK)].long()
        for h in range(hkv):
            k, v = (x[ids, h].reshape(-1, D)[:lens[b]] for x in state["values"])
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            s = torch.einsum("ngd,td->gnt", state["q"][lo:lo + n, heads].double(), k) * D ** -0.5
            seen = torch.ones((n, lens[b]), dtype=torch.bool, device="cuda").tril(past)
            w = torch.exp(s.masked_fill(~seen, -math.inf) - torch.logsumexp(s.masked_fill(~seen, -math.inf), -1, keepdim=True))
            out[lo:lo + n, heads] = torch.einsum("gnt,td->ngd", w, v)
    return out
