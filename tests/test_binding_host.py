"""Refusals of the Python calls before anything reaches the library (no GPU needed): tensors of sizes that
the kernels would read or write past."""
import pytest
import torch

D = 128
SIZES = r"must be (\[batch|\(2, 4, 128\))"  # (not the refusal of CPU tensors)


@pytest.fixture(scope="module")
def layer(tqlib):
    return tqlib.Layer(4, 2, device="cpu")


def queries(b=2, h=4, d=D):
    return torch.zeros(b, h, d)


BAD = [dict(q=queries(d=64)), dict(q=queries(d=256)), dict(q=torch.zeros(2, 4 * D)), dict(out=queries(b=1)),
       dict(out=queries(h=2)), dict(out=queries(d=64)), dict(out=torch.zeros(2 * 4 * D)), dict(out=queries(b=4, h=2))]


@pytest.mark.parametrize("bad", BAD)
def test_prefix_decode_refuses_other_sizes(layer, bad):
    args = dict(q=queries(), out=queries())
    args.update(bad)
    table = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match=SIZES):
        layer.prefix_decode(args["q"], table, 20, out=args["out"], workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match=SIZES):
        layer.prefix_decode(args["q"], None, 0, table.view(2, 1), table, out=args["out"],
                            workspace=torch.zeros(1 << 20, dtype=torch.uint8))


def test_prefix_decode_refuses_a_missing_table(layer):
    with pytest.raises(ValueError):
        layer.prefix_decode(queries(), None, 20)


@pytest.mark.parametrize("bad", BAD)
def test_decode_calls_refuse_other_sizes(layer, bad):
    args = dict(q=queries(), out=queries())
    args.update(bad)
    kv = torch.zeros(2, 2, D)
    table, lens, slots = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: layer.decode(args["q"], table, lens, out=args["out"], workspace=ws),
                 lambda: layer.append_decode(kv, kv, slots, args["q"], table, lens, out=args["out"], workspace=ws),
                 lambda: layer.decode_step(kv, kv, args["q"], table, lens, out=args["out"], workspace=ws)):
        with pytest.raises(ValueError, match=SIZES):
            call()


def test_outputs_without_their_inputs_are_refused(layer, tqlib):
    """An output that nothing would be written to."""
    rope, x = tqlib.Rope(), torch.zeros(3, 2, D)
    at = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: tqlib.apply_rope(rope, at, None, x, q_out=x), lambda: tqlib.apply_rope(rope, at, x, k_out=x),
                 lambda: layer.rope_append(rope, None, x, at, at, k_out=x),
                 lambda: layer.rope_append(rope, x, x, at, at, q_out=x)):
        with pytest.raises(ValueError, match="_out is given without"):
            call()
