"""The float64 statements of oracle/block.py against independent ones: torch's autograd, differences, closed forms."""
import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import operators as P


def rng(seed):
    return np.random.default_rng(seed)


def test_bf16_against_torch():
    x = np.concatenate([rng(0).standard_normal(4000).astype(np.float32) * np.float32(10.0) ** rng(1).integers(-30, 30, 4000),
                        np.array([0, -0.0, np.inf, -np.inf, np.nan, 3.4e38, 1e-45], np.float32)]).astype(np.float32)
    assert np.array_equal(B.bf16(x), torch.from_numpy(x).bfloat16().float().numpy(), equal_nan=True)


@pytest.mark.parametrize("rows,cols,eps", [(3, 8, 1e-6), (5, 40, 0.1)])
def test_norm_and_gradient_against_autograd_and_differences(rows, cols, eps):
    g = rng(rows)
    h, w, d_y, d_s = g.standard_normal((rows, cols)), g.standard_normal(cols), g.standard_normal((rows, cols)), \
        g.standard_normal((rows, cols))
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = th / torch.sqrt(th.square().mean(1, keepdim=True) + eps) * tw
    got, rstd = B.norm(h, w, eps)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-13)
    np.testing.assert_allclose(got, h * rstd[:, None] * w, rtol=1e-13)
    ((y * torch.tensor(d_y)).sum() + (th * torch.tensor(d_s)).sum()).backward()
    d_x, d_w = B.norm_backward(h, w, eps, d_y, d_s)
    np.testing.assert_allclose(d_x, th.grad.numpy(), rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(d_w, tw.grad.numpy(), rtol=1e-11, atol=1e-13)
    step, (i, j) = 1e-6, (rows - 1, 3)
    hp, hm = h.copy(), h.copy()
    hp[i, j] += step
    hm[i, j] -= step
    slope = ((B.norm(hp, w, eps)[0] - B.norm(hm, w, eps)[0]) * d_y).sum() / (2 * step) + d_s[i, j]
    assert abs(slope - d_x[i, j]) < 1e-6 * (1 + abs(slope))


def test_norm_of_equal_values_and_the_sum():
    y, rstd = B.norm(np.full((1, 16), 3.0), np.full(16, 2.0), 0.0)
    assert np.allclose(y, 2.0) and np.allclose(rstd, 1 / 3)
    x, r = rng(2).standard_normal((2, 64)).astype(np.float32), rng(3).standard_normal((2, 64)).astype(np.float32)
    xb, rb = torch.from_numpy(x).bfloat16(), torch.from_numpy(r).bfloat16()
    assert np.array_equal(B.norm_sum(xb.float().numpy(), rb.float().numpy(), "bf16"), (xb + rb).float().numpy())
    assert np.array_equal(B.norm_sum(x, r, "f32"), x + r) and np.array_equal(B.norm_sum(x, None, "f32"), x)


def problem(seed, T=23, N=6, K=2):
    g = rng(seed)
    logits = g.standard_normal((T, N))
    idx = np.argsort(-logits, axis=1)[:, :K].copy()
    idx[4] = -1                     # padding
    idx[9, 1] = N + 3               # one pick that is none
    return logits, idx, np.array([0, 7, 7, 20, 23])


@pytest.mark.parametrize("softmax", [True, False])
def test_balance_gradient_against_differences(softmax):
    logits, idx, starts = problem(5)
    d_loss = np.array([1.0, -2.0, 0.5, 3.0])
    got = B.balance_backward(logits, idx, starts, softmax, 0.3, d_loss)
    f = lambda l: (B.balance(l, idx, starts, softmax, 0.3)[0] * d_loss).sum()  # noqa: E731
    for t, i in [(0, 0), (4, 2), (6, 5), (9, 1), (22, 3)]:
        p, m = logits.copy(), logits.copy()
        p[t, i] += 1e-6
        m[t, i] -= 1e-6
        assert abs((f(p) - f(m)) / 2e-6 - got[t, i]) < 1e-8
    assert (got[4] == 0).all() and np.abs(got.sum(axis=1)).max() < (1e-15 if softmax else 1)


def test_balance_closed_forms():
    """Equal scores and equal picks: every f_i P_i is 1/N of 1, so the loss is alpha.  All picks on one expert under a
    softmax that favours it alone: the loss nears alpha N / K ... (K = 1)."""
    N, T = 4, 8
    even = np.arange(T)[:, None] % N
    loss, counts, tokens, total = B.balance(np.zeros((T, N)), even, np.array([0, T]), True, 0.1)
    assert np.isclose(loss[0], 0.1) and (counts == 2).all() and tokens[0] == T and np.allclose(total, T / N)
    l = np.zeros((T, N))
    l[:, 2] = 60
    loss, *_ = B.balance(l, np.full((T, 1), 2), np.array([0, T]), True, 0.1)
    assert np.isclose(loss[0], 0.1 * N)


def test_balance_is_the_layers_statistic():
    """With centroids that give these logits, the routing's own balance statistic."""
    from oracle import moe_oracle as O
    logits, idx, _ = problem(6, T=20)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :2]
    s = P.sigmoid(logits)
    loss, *_ = B.balance(logits, idx, np.array([0, 10, 20]), False, 0.01)
    assert np.allclose(loss, O.seq_balance_loss(s, idx, 10, 0.01))


def test_shares_far_below_the_types_range():
    p = B.shares(np.array([[-200.0, -200.0], [-300.0, -300.0 + np.log(3.0)]]), False)
    assert np.allclose(p, [[0.5, 0.5], [0.25, 0.75]])
    assert (B.shares(np.array([[-np.inf, 0.0]]), True) == [[0, 1]]).all()


def test_counts_of_a_whole_job():
    """Two halves with their counts added up: the gradients of the whole batch."""
    logits, idx, _ = problem(7, T=20)
    whole = np.array([0, 20])
    _, counts, tokens, total = B.balance(logits, idx, whole, True, 0.2)
    parts = [B.balance(logits[r], idx[r], np.array([0, 10]), True, 0.2) for r in (slice(0, 10), slice(10, 20))]
    assert (parts[0][1] + parts[1][1] == counts).all() and parts[0][2] + parts[1][2] == tokens
    d = np.concatenate([B.balance_backward(logits[r], idx[r], np.array([0, 10]), True, 0.2, [1.0], counts, tokens)
                        for r in (slice(0, 10), slice(10, 20))])
    np.testing.assert_allclose(d, B.balance_backward(logits, idx, whole, True, 0.2, [1.0]), rtol=1e-12, atol=1e-18)


def test_adapters_against_merged_weights():
    g = rng(8)
    x, a, b, base = g.standard_normal((5, 16)), g.standard_normal((3, 8, 16)), g.standard_normal((3, 24, 8)), \
        g.standard_normal((5, 24))
    which, scale, ranks = np.array([2, -1, 0, 0, 3]), np.array([0.5, 1.0, 2.0]), np.array([8, 3, 5])
    out, size = B.adapters(x, which, a, b, scale, ranks, base)
    for t in range(5):
        e = which[t]
        w = np.zeros((24, 16)) if not 0 <= e < 3 else scale[e] * b[e][:, :ranks[e]] @ a[e][:ranks[e]]
        np.testing.assert_allclose(out[t], base[t] + x[t] @ w.T, rtol=1e-12, atol=1e-12)
        assert (np.abs(out[t] - base[t]) <= size[t] + 1e-12).all()
