"""examples/own_router_step.py: the operators together, as a training step uses them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "own_router_step.py")


def _example():
    spec = importlib.util.spec_from_file_location("own_router_step", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_loss_falls_and_repeats():
    m = _example()
    losses = m.train(steps=6)
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert losses == m.train(steps=6)


def test_one_step_against_float64():
    """The whole step's gradients against autograd in float64 on the same weights and picks.  E4M3 keeps four bits (2.6%
    of a value at random) in each of the two operands of a product, 8 bits of the SwiGLU inputs: about 4% of a gradient
    that passes two of the FFN's products; 10% is asked of each."""
    m = _example()
    gen = torch.Generator("cuda").manual_seed(1)
    T, d, I = 200, 256, 128
    ffn, layer = m.DenseFfn(T, d, I, gen), m.Experts(T, d, 8, 2, 1, I, gen)
    x = torch.randn(T, d, device="cuda", generator=gen).bfloat16()
    dout = torch.randn(T, d, device="cuda", generator=gen).bfloat16()
    y = ffn.forward(x)
    layer.forward(y)
    dy = layer.backward(dout)
    dx = ffn.backward(dy)
    f = lambda t: t.double().requires_grad_()  # noqa: E731
    x64, w1, w2, r = f(x), f(ffn.w1), f(ffn.w2), f(layer.router)
    w = [f(t) for t in layer.w]
    a, b = (x64 @ w1.t()).chunk(2, dim=1)
    y64 = x64 + (torch.nn.functional.silu(a) * b) @ w2.t()
    s = torch.softmax(y64 @ r.t(), dim=1).gather(1, layer.idx.long())
    gate = s / s.sum(1, keepdim=True)
    ffns = [(torch.nn.functional.silu(y64 @ wg.t()) * (y64 @ wu.t())) @ wd.t() for k in (0, 3) for wg, wu, wd in
            zip(*w[k:k + 3])]
    out = y64 + ffns[-1]
    for k in range(2):
        out = out + gate[:, k:k + 1] * torch.stack(ffns[:8], 1)[torch.arange(T, device="cuda"), layer.idx[:, k].long()]
    (out * dout.double()).sum().backward()
    for got, ref in ((dx, x64.grad), (ffn.d_w1.out, w1.grad), (ffn.d_w2.out, w2.grad), (layer.d_router, r.grad),
                     *((g, t.grad) for g, t in zip(layer.g, w))):
        assert ((got.double() - ref).norm() / ref.norm()).item() < 0.1
