"""Several answers to each prompt over a cache held in 8 bits: prompts attended and appended, forked into
answers that share their blocks, grown token by token, some of them given up, the pool compacted.

One layer of a model with grouped-query attention:

  1. the prompts' keys and values go into an int8 layer and their queries attend causally, all prompts
     in one call (append, attend), a second part of each in a second call;
  2. every prompt is forked into `answers` rows (Blocks.reorder): whole blocks are shared, the last one of
     a prompt is copied for all answers but the first;
  3. each step every row gets room for a token (Blocks.extend), the token is appended, and the row's query
     attends to its context (append_decode);
  4. half way through, every second answer is given up (Blocks.release) and the others move together
     (Blocks.compact).

Every step is held against the same attention from the values that the cache gives back (dequantize).

    python -m examples.forked_answers
"""
import math

import torch

import turboquant_quantized_kv_gb300 as tq


def attention(layer, q, table, length):
    """Softmax attention in fp64 of q [n, heads, d], the last n of `length` tokens, over dequantized values."""
    at = torch.arange(length, device="cuda")
    slots = table[at // tq.TQ_BLOCK_SIZE].long() * tq.TQ_BLOCK_SIZE + at % tq.TQ_BLOCK_SIZE
    k, v = (layer.dequantize(w, slots).double() for w in (0, 1))
    n, heads, d = q.shape
    group = heads // layer.num_kv_heads
    s = torch.einsum("nhgd,thd->hgnt", q.double().view(n, -1, group, d), k) / math.sqrt(d)
    seen = torch.ones(n, length, dtype=torch.bool, device="cuda").tril(length - n)
    w = s.masked_fill(~seen, -math.inf).softmax(-1)
    return torch.einsum("hgnt,thd->nhgd", w, v).reshape(n, heads, d)


def main(prompts=3, answers=4, tokens=150, steps=24, heads=16, kv_heads=4, verbose=True):
    """Returns the largest difference from the 64-bit attention, relative to a row's largest value."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    dim, block = tq.TQ_HEAD_DIM, tq.TQ_BLOCK_SIZE
    lens = [tokens + 13 * i for i in range(prompts)]
    width = -(-(max(lens) + steps) // block)
    layer = tq.Layer(prompts * width + prompts * answers * (2 + steps // block) + 7, kv_heads, kv_format="int8")
    blocks = tq.Blocks(layer.num_blocks)
    worst = 0.0

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def project(n):
        qkv = torch.randn(n, heads + 2 * kv_heads, dim, device="cuda", generator=gen).to(torch.bfloat16)
        return qkv[:, :heads], qkv[:, heads:heads + kv_heads].contiguous(), qkv[:, heads + kv_heads:].contiguous()

    def check(got, want):
        nonlocal worst
        worst = max(worst, float(((got.double() - want).abs().amax(-1) / want.abs().amax(-1)).max()))

    # the prompts, in two parts
    table = torch.full((prompts, width), -1, dtype=torch.int32, device="cuda")
    done = [0] * prompts
    for part in (0, 1):
        upto = [n // 2 if part == 0 else n for n in lens]
        blocks.extend(table, ints(done), ints(upto))
        new = [b - a for a, b in zip(done, upto)]
        at = torch.cat([torch.arange(a, b, device="cuda") for a, b in zip(done, upto)])
        row = torch.repeat_interleave(torch.arange(prompts, device="cuda"), torch.tensor(new, device="cuda"))
        slots = table[row, at // block].long() * block + at % block
        q, k, v = project(sum(new))
        layer.append(k, v, slots)
        starts = [sum(new[:i]) for i in range(prompts + 1)]
        out = layer.attend(q, ints(starts), table, ints(upto), out_dtype=torch.float32)
        for b in range(prompts):
            check(out[starts[b]:starts[b + 1]], attention(layer, q[starts[b]:starts[b + 1]], table[b], upto[b]))
        done = upto

    # their answers
    parents = ints([p for p in range(prompts) for _ in range(answers)])
    table, length = blocks.reorder([layer], table, ints(lens), parents)
    rows = prompts * answers
    workspace = torch.zeros(layer.workspace_bytes(rows, heads, width), dtype=torch.uint8, device="cuda")
    for step in range(steps):
        if step == steps // 2:
            which = torch.arange(table.shape[0], device="cuda") % 2 == 1
            blocks.release(table, length, which)
            live = blocks.compact([layer], table, length)
            table, length = blocks.reorder([layer], table, length, ints(list(range(0, rows, 2))))
            rows = table.shape[0]
            if int(live) != int((blocks.refs > 0).sum()):
                raise RuntimeError("blocks were lost")
        blocks.extend(table, length, length + 1)
        slots = table[torch.arange(rows, device="cuda"), (length // block).long()].long() * block + length % block
        length = length + 1
        q, k, v = project(rows)
        q = q.contiguous()
        out = layer.append_decode(k, v, slots, q, table, length, out_dtype=torch.float32, workspace=workspace)
        counts = length.tolist()
        for b in range(0, rows, 5):
            check(out[b:b + 1], attention(layer, q[b:b + 1], table[b], counts[b]))
    status = tq.get_device_status()
    if status != 0:
        raise RuntimeError("device status %d" % status)
    if verbose:
        print("%d prompts, %d answers each, %d steps: largest difference from 64 bits %.1e of a row's largest value"
              % (prompts, answers, steps, worst))
    return worst


if __name__ == "__main__":
    main()
