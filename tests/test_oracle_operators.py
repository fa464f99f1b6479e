"""The float64 statements of oracle/operators.py: hand values, special cases, and gradients against differences."""
import numpy as np
import pytest

from oracle import operators as P


def test_gate_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    idx, g, load, _ = P.gate(l, None, 2, True)
    assert idx.tolist() == [[2, 1]] and np.allclose(g, [[2 / 3, 1 / 3]]) and load.tolist() == [0, 1, 1, 0]
    idx, g, _, _ = P.gate(l, None, 3, True, renorm=False, scale=2.0)
    assert idx.tolist() == [[2, 1, 0]] and np.allclose(g, [[1.0, 0.5, 0.25]])   # the tie goes to the lower index
    # the bias ranks and does not weigh; sigmoid(log x) = x / (1 + x)
    idx, g, _, _ = P.gate(l, np.array([0.0, 0.0, -1.0, 1.0]), 2, False, renorm=False)
    assert idx.tolist() == [[3, 1]] and np.allclose(g, [[0.5, 2 / 3]])


def test_gate_groups_by_hand():
    l = np.array([[3.0, -9.0, 2.0, 2.0, 1.0, 1.0]])
    # best of a group: {0, 1} wins with the 3; sum of two: {2, 3} wins
    assert P.gate(l, None, 2, False, 3, 1, False)[0].tolist() == [[0, 1]]
    assert P.gate(l, None, 2, False, 3, 1, True)[0].tolist() == [[2, 3]]


def test_gate_masked_and_empty_rows():
    inf = np.inf
    l = np.array([[-inf, 1.0, -inf], [-inf, -inf, -inf], [0.0, 0.0, 0.0]])
    for softmax in (False, True):
        idx, g, load, _ = P.gate(l, None, 2, softmax)
        assert idx.tolist() == [[1, -1], [-1, -1], [0, 1]]
        assert np.array_equal(g, [[1, 0], [0, 0], [0.5, 0.5]]) and load.tolist() == [1, 2, 0]
    assert P.gate(l, np.array([-inf, 0.0, 0.0]), 2, True)[0].tolist() == [[1, -1], [-1, -1], [1, 2]]


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_backward_against_differences(softmax, renorm):
    rng = np.random.default_rng(7)
    l, dg = rng.standard_normal((5, 9)), rng.standard_normal((5, 3))
    idx = P.gate(l, None, 3, softmax)[0]
    idx[1, 2] = -1
    got = P.gate_backward(l, idx, dg, softmax, renorm, 1.5)
    f = lambda x: (dg * P.gate_values(P.gate_scores(x, softmax), idx, renorm, 1.5)).sum()  # noqa: E731
    h = 1e-5   # central differences: error about h^2 and 1e-16 / h
    for t in range(5):
        for i in range(9):
            e = np.zeros_like(l)
            e[t, i] = h
            assert abs((f(l + e) - f(l - e)) / (2 * h) - got[t, i]) < 1e-8


def test_matmul_blocks():
    rng = np.random.default_rng(1)
    a, b = rng.integers(-8, 8, (3, 256)).astype(float), rng.integers(-8, 8, (130, 256)).astype(float)
    sa, sb = rng.random((3, 2)), rng.random((2, 2))
    out, size = P.matmul_fp8("forward", a, sa, b, sb)
    want = sum(sa[2, k] * sb[1, k] * (a[2, 128 * k:128 * k + 128] * b[129, 128 * k:128 * k + 128]).sum() for k in (0, 1))
    assert np.isclose(out[2, 129], want) and (size >= np.abs(out) - 1e-9).all()
    assert np.allclose(P.matmul_fp8("input_grad", a, sa, b.T, sb.T)[0], out)
    assert np.allclose(P.matmul_fp8("weight_grad", a, sa, b, np.repeat(sb, 128, 0)[:130])[0], out)


def test_codes8():
    x = np.zeros((1, 256), np.float32)
    x[0, :4] = [127.0, -63.5, 0.5, 1.5]
    codes, scale = P.codes8(x)
    assert scale[0, 1] == 1.0 and np.isclose(scale[0, 0], 1.0, rtol=1e-6) and codes[0, 0] == 127
    assert codes[0, 128:].tolist() == [0] * 128
    x[0, 200] = np.inf
    assert np.isnan(P.codes8(x)[1][0, 1]) and np.isfinite(P.codes8(x)[1][0, 0])
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 512)).astype(np.float32)
    codes, scale = P.codes8(x)
    err = np.abs(codes * np.repeat(scale.astype(np.float64), 128, 1) - x)
    assert (err <= np.repeat(scale, 128, 1) * 0.501).all()


def test_swiglu8_backward_against_differences():
    rng = np.random.default_rng(3)
    codes, scales = P.codes8(rng.standard_normal((3, 256)).astype(np.float32))
    dh = rng.standard_normal((3, 128))
    d_ab, h = P.swiglu8_backward(dh, codes, scales)
    ab = codes * np.repeat(scales.astype(np.float64), 128, 1)
    assert np.allclose(h, P.swiglu(ab), rtol=1e-12)
    step = 1e-5
    for r, c in ((0, 0), (1, 77), (2, 127), (0, 128), (2, 255)):
        e = np.zeros_like(ab)
        e[r, c] = step
        assert abs(((P.swiglu(ab + e) - P.swiglu(ab - e)) * dh).sum() / (2 * step) - d_ab[r, c]) < 1e-8


def test_gate_of_an_empty_place_beside_a_nan():
    l = np.array([[0.5, np.nan, -np.inf, -np.inf]])
    for softmax in (False, True):
        idx, g, _, _ = P.gate(l, None, 3, softmax)
        assert idx.tolist() == [[0, 1, -1]] and np.isnan(g[0, 1]) and g[0, 2] == 0
