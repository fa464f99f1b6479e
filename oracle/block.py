"""Float64 statements of the operators around the layer: the norm with the residual's addition and an E4M3 output, the
balance loss from logits with its gradient, and low-rank adapters.

Plain numpy on plain arrays, row by row or sequence by sequence.  `stream` says how the norm's sum is held ("f32", "bf16").
"""
from __future__ import annotations

import numpy as np

from . import operators as P


def bf16(x):
    """fp32 values rounded to bf16, to nearest even (as fp32)."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((b.astype(np.uint64) + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return np.where(np.isnan(x), np.float32(np.nan), r.view(np.float32))


# ---------------------------------------------------------------- norm

def norm_sum(x, residual, stream):
    """h as it is held, fp32 (of the stream's values)."""
    h = np.asarray(x, np.float32)
    if residual is not None:
        with np.errstate(invalid="ignore", over="ignore"):
            h = h + np.asarray(residual, np.float32)
    return bf16(h) if stream == "bf16" else h


def norm(h, weight, eps):
    """(y, rstd)."""
    h = np.asarray(h, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        rstd = 1 / np.sqrt((h * h).mean(axis=1) + eps)
        return h * rstd[:, None] * np.asarray(weight, np.float64), rstd


def norm_backward(h, weight, eps, d_y, d_sum=None):
    """(d_x, d_weight): the Jacobian of y with respect to h, row by row."""
    h, w, d_y = (np.asarray(v, np.float64) for v in (h, weight, d_y))
    n = h.shape[1]
    d_x = np.zeros_like(h)
    d_w = np.zeros(n)
    for r in range(h.shape[0]):
        size = np.sqrt((h[r] @ h[r]) / n + eps)
        v = w * d_y[r]
        d_x[r] = v / size - h[r] * (h[r] @ v) / (n * size ** 3)
        d_w += d_y[r] * h[r] / size
    return (d_x if d_sum is None else d_x + np.asarray(d_sum, np.float64)), d_w


# ---------------------------------------------------------------- balance loss

def shares(logits, softmax):
    """p [T, N] and dp's factor: the softmax, or the sigmoids over their sum (in logarithms, so that nothing is lost)."""
    l = np.asarray(logits, np.float64)
    a = l if softmax else -np.logaddexp(0, -l)
    top = a.max(axis=1, keepdims=True)
    e = np.exp(a - np.where(np.isneginf(top), 0, top))
    total = e.sum(axis=1, keepdims=True)
    return e / np.where(total == 0, 1, total)


def balance(logits, idx, starts, softmax, alpha):
    """(loss [S], counts [S, N], tokens [S], prob_sum [S, N])."""
    p = shares(logits, softmax)
    T, N = p.shape
    K, S = idx.shape[1], len(starts) - 1
    loss, tokens = np.zeros(S), np.zeros(S, np.int64)
    counts, total = np.zeros((S, N), np.int64), np.zeros((S, N))
    for s in range(S):
        for t in range(starts[s], starts[s + 1]):
            picks = [e for e in idx[t] if 0 <= e < N]
            if not picks:
                continue
            tokens[s] += 1
            total[s] += p[t]
            for e in picks:
                counts[s, e] += 1
        if tokens[s]:
            f = N * counts[s] / (K * tokens[s])
            loss[s] = alpha * (f * (total[s] / tokens[s])).sum()
    return loss, counts, tokens, total


def balance_backward(logits, idx, starts, softmax, alpha, d_loss, counts=None, tokens=None):
    """d_logits [T, N] through the Jacobian of each token's p; counts and tokens: given ones (a whole job's)."""
    own = balance(logits, idx, starts, softmax, alpha)
    counts, tokens = (own[1] if counts is None else counts), (own[2] if tokens is None else tokens)
    p = shares(logits, softmax)
    T, N = p.shape
    K = idx.shape[1]
    out = np.zeros((T, N))
    for s in range(len(starts) - 1):
        for t in range(starts[s], starts[s + 1]):
            if not any(0 <= e < N for e in idx[t]):
                continue
            dp = d_loss[s] * alpha * (N * counts[s] / (K * tokens[s])) / tokens[s]
            jac = np.diag(p[t]) - np.outer(p[t], p[t])            # of p by the scores' logarithms
            slope = np.ones(N) if softmax else P.sigmoid(-np.asarray(logits[t], np.float64))
            out[t] = (dp @ jac) * slope
    return out


# ---------------------------------------------------------------- adapters

def adapters(x, which, a, b, scale, ranks, base):
    """(out, size): size is the sum of the magnitudes that make up each low-rank term."""
    x, a, b = (np.asarray(v, np.float64) for v in (x, a, b))
    out = np.array(base, np.float64)
    size = np.zeros_like(out)
    for t, e in enumerate(which):
        if 0 <= e < a.shape[0]:
            r = a.shape[1] if ranks is None else min(max(int(ranks[e]), 0), a.shape[1])
            out[t] += scale[e] * (b[e, :, :r] @ (a[e, :r] @ x[t]))
            size[t] = abs(scale[e]) * (np.abs(b[e, :, :r]) @ (np.abs(a[e, :r]) @ np.abs(x[t])))
    return out, size
