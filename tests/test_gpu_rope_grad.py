"""GPU: apply_rope under autograd.  Tolerances as in test_gpu_rope.py: ROT of the pair's length, half a step
of bf16 where the gradient is rounded to it."""
import numpy as np
import pytest

from tests._gpu_util import D
from tests._rope_ref import frequencies, pair_norm, rotate
from tests.test_gpu_rope import HALF, ROT, YARN, draw, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout,rotary", [("half", 128), ("half", 96), ("interleaved", 64)])
@pytest.mark.parametrize("transpose", [False, True])
def test_gradient_is_the_transposed_rotation(cuda, tqlib, dtype, layout, rotary, transpose):
    """Of views of one projection, by the formula; the part that is not rotated gets no gradient."""
    tq = tqlib
    rope = tq.Rope(rotary, 10000.0, layout=layout, scaling=YARN)
    f, amp = frequencies(rotary, 10000.0, YARN)
    n, hq, hk = 13, 5, 2
    qkv = draw(cuda, (n, hq + 2 * hk, D), dtype, 1).requires_grad_()
    w = draw(cuda, (n, hq + hk, D), dtype, 2)
    pos = cuda.arange(n, device="cuda") * 91
    q, k = tq.apply_rope(rope, pos, qkv[:, :hq], qkv[:, hq:hq + hk], transpose=transpose)
    assert q.requires_grad and k.requires_grad
    grad, = cuda.autograd.grad((q, k), qkv, (w[:, :hq], w[:, hq:]))
    got, ws = f64(grad), f64(w)
    want = rotate(ws, pos.cpu().numpy(), f, amp, layout, not transpose)
    bound = HALF[dtype] * np.abs(want) * (1 + ROT) + ROT * amp * pair_norm(ws, rotary, layout)
    assert np.all(np.abs(got[:, :hq + hk] - want) <= bound)
    assert np.all(got[:, hq + hk:] == 0.0)


def test_gradient_by_differences(cuda, tqlib):
    """<w, R(x + d) - R(x - d)> / 2 against <gradient, d> (the rotation is linear); w expanded, as sum() leaves it."""
    tq = tqlib
    rope = tq.Rope(128, 500.0)
    n, h = 7, 3
    x, d = draw(cuda, (n, h, D), "f32", 3).requires_grad_(), draw(cuda, (n, h, D), "f32", 4)
    pos = cuda.arange(n, device="cuda") * 1237
    tq.apply_rope(rope, pos, x)[0].sum().backward()
    with cuda.no_grad():
        left = ((tq.apply_rope(rope, pos, x + d)[0].double() - tq.apply_rope(rope, pos, x - d)[0].double()) / 2).sum(-1)
    right = (x.grad.double() * d.double()).sum(-1)
    scale = (x.detach().abs() + d.abs()).double().sum(-1) * 2
    assert bool(((left - right).abs() <= 4 * ROT * scale).all())


def test_which_inputs_take_gradients(cuda, tqlib):
    tq = tqlib
    rope = tq.Rope()
    pos = cuda.arange(4, device="cuda")
    q, k = draw(cuda, (4, 2, D), "bf16", 1), draw(cuda, (4, 1, D), "bf16", 2)
    plain = tq.apply_rope(rope, pos, q, k)
    assert not plain[0].requires_grad and plain[0].grad_fn is None
    kg = k.clone().requires_grad_()
    qo, ko = tq.apply_rope(rope, pos, q, kg)
    assert cuda.equal(qo, plain[0]) and cuda.equal(ko, plain[1])
    ko.float().square().sum().backward()
    assert kg.grad is not None and kg.grad.shape == kg.shape
    qg = q.clone().requires_grad_()
    only = tq.apply_rope(rope, pos, qg)
    assert only[1] is None
    only[0].sum().backward()
    none, only_k = tq.apply_rope(rope, pos, None, kg)
    assert none is None and only_k.requires_grad
    with cuda.no_grad():
        assert not tq.apply_rope(rope, pos, qg, kg)[0].requires_grad
        tq.apply_rope(rope, pos, qg.detach(), q_out=qg.detach())
    for kw in (dict(q_out=cuda.empty_like(q)), dict(k_out=cuda.empty_like(k))):
        with pytest.raises(ValueError):
            tq.apply_rope(rope, pos, qg, kg, **kw)


def test_second_derivative_and_side_stream(cuda, tqlib):
    """The gradient of the gradient is the rotation again; a call on a stream of its own."""
    tq = tqlib
    rope = tq.Rope(layout="interleaved")
    pos = cuda.arange(5, device="cuda") + 100
    x, w = draw(cuda, (5, 2, D), "f32", 1).requires_grad_(), draw(cuda, (5, 2, D), "f32", 2).requires_grad_()
    g, = cuda.autograd.grad(tq.apply_rope(rope, pos, x)[0], x, w, create_graph=True)
    gg, = cuda.autograd.grad(g, w, cuda.ones_like(g))
    assert cuda.equal(gg, tq.apply_rope(rope, pos, cuda.ones_like(g))[0])
    side = cuda.cuda.Stream()
    side.wait_stream(cuda.cuda.current_stream())
    y = tq.apply_rope(rope, pos, x, stream=side)[0]
    cuda.cuda.current_stream().wait_stream(side)
    assert cuda.equal(y, tq.apply_rope(rope, pos, x)[0])
    y.sum().backward()
    cuda.cuda.synchronize()
    assert bool(x.grad.isfinite().all())
