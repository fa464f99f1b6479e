"""moe_swiglu_forward8 and moe_swiglu_backward8 on the GPU against float64.

Codes and scales are compared bit for bit (fp32 products and correctly rounded quotients).  h, dA, dB are computed in fp32
and rounded once to bf16: 2^-8 of the value covers that rounding (2^-9) and the fp32 error of the sigmoid (2^-19 at |a| <
40); dA holds the difference 1 + a (1 - sg), so its fp32 error counts against |dh b| (1 + |a|): 2^-19 of that."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from oracle import operators as P  # noqa: E402


def forward(ab, with_h=True, stream=None):
    rows, inter = ab.shape[0], ab.shape[1] // 2
    h = torch.full((rows, inter), float("nan"), dtype=torch.bfloat16, device="cuda") if with_h else None
    q = torch.full((rows, 2 * inter), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows, 2 * inter // 128), float("nan"), device="cuda")
    moe.moe_swiglu_forward8(rows, inter, ab, h, q, s, stream)
    return h, q, s


def backward(dh, q, s, with_h=True):
    rows, inter = dh.shape
    d = torch.full((rows, 2 * inter), float("nan"), dtype=torch.bfloat16, device="cuda")
    h = torch.full_like(dh, float("nan")) if with_h else None
    moe.moe_swiglu_backward8(rows, inter, dh, q, s, d, h)
    return d, h


def inputs(rows, inter, seed, size=2.0):
    g = torch.Generator("cuda").manual_seed(seed)
    ab = (size * torch.randn(rows, 2 * inter, device="cuda", generator=g)).bfloat16()
    return ab, torch.randn(rows, inter, device="cuda", generator=g).bfloat16()


@pytest.mark.parametrize("rows,inter,size", [(1, 128, 1.0), (3, 256, 0.01), (255, 1408, 2.0), (17, 128, 10.0),
                                             (1000, 384, 1.0), (4, 8192, 3.0)])
def test_against_float64(rows, inter, size):
    ab, dh = inputs(rows, inter, rows + inter, size)
    ab[0, :128] = 0
    h, q, s = forward(ab)
    x = ab.float().cpu().numpy()
    codes, scales = P.codes8(x)
    assert np.array_equal(q.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), scales)
    ref = P.swiglu(x)
    assert (np.abs(h.float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-30).all()
    d, h2 = backward(dh, q, s)
    d_ref, h_ref = P.swiglu8_backward(dh.float().cpu().numpy(), codes, scales)
    assert (np.abs(h2.float().cpu().numpy() - h_ref) <= 2.0 ** -8 * np.abs(h_ref) + 1e-30).all()
    a, b = np.split(codes * np.repeat(scales.astype(np.float64), 128, 1), 2, axis=1)
    size = np.concatenate([np.abs(b) * (1 + np.abs(a)), np.abs(a)], axis=1) * np.tile(np.abs(dh.float().cpu().numpy()), 2)
    assert (np.abs(d.float().cpu().numpy() - d_ref) <= 2.0 ** -8 * np.abs(d_ref) + 2.0 ** -19 * size + 1e-30).all()


def test_gradients_near_those_of_the_inputs_themselves():
    """What 8 bits cost a gradient of normal inputs: the codes' error is at most amax / 254, about 0.6% of the inputs'
    size at random, so the gradient's relative error stays near 1% (2% is asked)."""
    ab, dh = inputs(300, 512, 1, 1.0)
    _, q, s = forward(ab, with_h=False)
    d, _ = backward(dh, q, s, with_h=False)
    x = ab.double().requires_grad_()
    a, b = x.chunk(2, dim=1)
    (a * torch.sigmoid(a) * b * dh.double()).sum().backward()
    assert ((d.double() - x.grad).norm() / x.grad.norm()).item() < 0.02


def test_extreme_and_not_finite_values():
    ab, dh = inputs(6, 256, 2)
    ab[0, :128] = 1e-39                       # subnormal: the scale is one too
    ab[0, 64] = -9e-39
    ab[1, 5] = 3e38                           # one value that hides its run
    ab[2, 130] = float("inf")                 # a's second run
    ab[3, 300] = float("nan")                 # b's first run
    ab[4, :256] = -100.0                      # sigmoid 0
    ab[5, :256] = 100.0
    _, q, s = forward(ab)
    codes, scales = P.codes8(ab.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), codes)
    assert np.array_equal(s.cpu().numpy(), scales, equal_nan=True)
    d, h = backward(dh, q, s)
    bad = torch.isnan(d)
    # dA and dB of a feature use both its a and its b
    assert bad[2, 128:256].all() and bad[2, 384:].all() and bad[3, :128].all()
    assert not bad[0].any() and not bad[2, :128].any() and not bad[3, 128:256].any() and not bad[4:].any()
    assert (h[4] == 0).all() and (d[4] == 0).all()


def test_without_h_the_rest_is_the_same():
    ab, dh = inputs(33, 640, 3)
    h, q, s = forward(ab)
    _, q2, s2 = forward(ab, with_h=False)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    d, _ = backward(dh, q, s)
    d2, _ = backward(dh, q, s, with_h=False)
    assert torch.equal(d, d2)


def test_no_rows_and_another_stream():
    ab, _ = inputs(700, 256, 4)
    first = forward(ab)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = forward(ab, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    moe.moe_swiglu_forward8(0, 256, None, None, None, None)
    moe.moe_swiglu_backward8(0, 256, None, None, None, None)


def test_offsets_past_32_bits():
    """More than 2^32 elements of ab: the last rows come out as they do alone."""
    rows, inter = (1 << 20) + 11, 2048
    block, dh = inputs(64, inter, 5)
    reps = rows // 64 + 1
    ab = block.repeat(reps, 1)[:rows]
    h, q, s = forward(ab)
    tail = ab[rows - 64:].contiguous()
    h2, q2, s2 = forward(tail)
    assert torch.equal(h[rows - 64:], h2) and torch.equal(q[rows - 64:], q2) and torch.equal(s[rows - 64:], s2)
    del ab, h
    big = dh.repeat(reps, 1)[:rows]
    d, g = backward(big, q, s)
    d2, g2 = backward(big[rows - 64:].contiguous(), q2, s2)
    assert torch.equal(d[rows - 64:], d2) and torch.equal(g[rows - 64:], g2)
