"""Serving a batch behind one prompt: rotary positions, rotated appends and attention over
the shared prefix, used together.

One layer of a model with grouped-query attention answers `batch` requests that share a prompt:

  1. the prompt's keys and values go into the cache once, rotated on the way (rope_append);
  2. each step, every request's new query and key are rotated and its key and value appended to
     the request's own blocks in one call (rope_append), and the step's attention reads the
     prompt's blocks once for the whole batch (prefix_decode);
  3. for comparison the same step as a plain decode, whose block tables repeat the prompt's blocks
     in every row (a prompt of whole blocks only).

    python -m examples.shared_prefix
"""
import math

import torch

import turboquant_quantized_kv_gb300 as tq


def main(batch=16, prompt=4096, steps=8, heads=32, kv_heads=8, bits_k=4, bits_v=4, verbose=True):
    """Returns the largest difference between the two ways, relative to a row's largest value."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    dim, block = tq.TQ_HEAD_DIM, tq.TQ_BLOCK_SIZE
    prompt = prompt // block * block
    own_blocks = -(-steps // block)
    rope = tq.Rope(dim, base=500000.0, scaling={"kind": "banded", "factor": 8.0, "low": 1.0, "high": 4.0, "length": 8192})
    layer = tq.Layer(prompt // block + batch * own_blocks, kv_heads, bits_k=bits_k, bits_v=bits_v)

    def project(tokens):  # stands for the layer's fused projection: views of one buffer
        qkv = torch.randn(tokens, heads + 2 * kv_heads, dim, device="cuda", generator=gen).to(torch.bfloat16)
        return qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]

    # the prompt, once: block i of the prompt is block i of the pool
    prefix_table = torch.arange(prompt // block, dtype=torch.int32, device="cuda")
    _, k, v = project(prompt)
    at = torch.arange(prompt, device="cuda")
    layer.rope_append(rope, k, v, positions=at, slot_mapping=at)

    # the requests' own blocks follow
    block_table = (prompt // block + torch.arange(batch * own_blocks, device="cuda", dtype=torch.int32)).view(batch, -1)
    workspace = torch.zeros(layer.prefix_workspace_bytes(batch, heads, prompt, own_blocks), dtype=torch.uint8, device="cuda")
    joined = torch.cat([prefix_table.expand(batch, -1), block_table], 1).contiguous()
    worst = 0.0
    for step in range(steps):
        q, k, v = project(batch)
        positions = torch.full((batch,), prompt + step, dtype=torch.int64, device="cuda")
        slots = block_table[:, step // block].long() * block + step % block
        q = layer.rope_append(rope, k, v, positions, slots, q=q)
        lens = torch.full((batch,), step + 1, dtype=torch.int32, device="cuda")
        out = layer.prefix_decode(q, prefix_table, prompt, block_table, lens, out_dtype=torch.float32, workspace=workspace)
        plain = layer.decode(q, joined, lens + prompt, sm_scale=1.0 / math.sqrt(dim), out_dtype=torch.float32)
        worst = max(worst, float(((out - plain).abs().amax(-1) / plain.abs().amax(-1)).max()))
    status = tq.get_device_status()
    if status != 0:
        raise RuntimeError("device status %d" % status)
    if verbose:
        print("%d steps of %d requests behind %d tokens: largest difference from the plain decode %.1e of a row's "
              "largest value" % (steps, batch, prompt, worst))
    return worst


if __name__ == "__main__":
    main()
