"""Float64 statements of the operators beside the layer: routing from given logits, the FP8 product with one scale
per block of 128, and SwiGLU whose inputs are kept in 8 bits.

Plain numpy on plain arrays.  Codes and scales follow their formats bit for bit (the scales and quotients are fp32 by
definition); everything else is float64.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


# ---------------------------------------------------------------- routing

def gate_scores(logits, softmax):
    """s [T, N]; a row whose logits are all -inf has s = 0."""
    l = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if not softmax:
            return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
        top = np.max(l, axis=1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(top), 0, top))
        total = e.sum(axis=1, keepdims=True)
        return e / np.where(total == 0, 1, total)


def gate(logits, bias, top_k, softmax, groups=1, top_groups=1, top2=False, renorm=True, scale=1.0):
    """(idx [T, K], gates [T, K], load [N], gap [T]): gap is the smallest difference that decided a row (a pick
    against the next key, a kept group against the next one; equal keys of equal logits and biases do not count)."""
    l = np.asarray(logits, np.float64)
    T, N = l.shape
    b = np.zeros(N) if bias is None else np.asarray(bias, np.float64)
    s = gate_scores(l, softmax)
    key = s + b
    size = N // groups
    idx = np.full((T, top_k), -1, np.int64)
    gap = np.full(T, np.inf)
    for t in range(T):
        able = [i for i in range(N) if not np.isneginf(l[t, i]) and not np.isneginf(b[i])]
        rank = lambda i: (-np.inf if np.isnan(key[t, i]) else key[t, i])  # noqa: E731
        if top_groups < groups:
            score = []
            for g in range(groups):
                mine = sorted((rank(i) for i in able if i // size == g), reverse=True)
                if not mine:
                    score.append((-1, -np.inf))
                elif top2 and len(mine) > 1 and np.isfinite(mine[1]):
                    score.append((0, mine[0] + mine[1]))
                else:
                    score.append((0, mine[0]))
            order = sorted(range(groups), key=lambda g: (-score[g][0], -score[g][1], g))
            near = score[order[top_groups - 1]], score[order[top_groups]]
            if near[0][0] == near[1][0] == 0:
                gap[t] = min(gap[t], abs(near[0][1] - near[1][1]))
            able = [i for i in able if i // size in order[:top_groups]]
        order = sorted(able, key=lambda i: (-rank(i), i))
        for k in range(min(top_k, len(order))):
            idx[t, k] = order[k]
            if k + 1 < len(order):
                i, j = order[k], order[k + 1]
                if not (l[t, i] == l[t, j] and b[i] == b[j]):
                    gap[t] = min(gap[t], abs(rank(i) - rank(j))) if np.isfinite(rank(j)) else gap[t]
    return idx, gate_values(s, idx, renorm, scale), np.bincount(idx[idx >= 0], minlength=N), gap


def gate_values(s, idx, renorm=True, scale=1.0):
    on = idx >= 0
    sel = np.where(on, np.take_along_axis(s, np.where(on, idx, 0), 1), 0.0)
    if renorm:
        total = sel.sum(axis=1, keepdims=True)
        sel = np.where(on, sel / np.where(total == 0, 1, total), 0.0)
    return scale * sel


def gate_backward(logits, idx, d_gate, softmax, renorm=True, scale=1.0):
    """dL/dlogits through the gates of the picks idx, as the product of the Jacobians of s and of the gates."""
    l = np.asarray(logits, np.float64)
    T, N = l.shape
    s = gate_scores(l, softmax)
    out = np.zeros((T, N))
    for t in range(T):
        on = [k for k in range(idx.shape[1]) if 0 <= idx[t, k] < N]
        e = [int(idx[t, k]) for k in on]
        dg = scale * np.array([d_gate[t, k] for k in on], np.float64)
        ds = np.zeros(N)
        if renorm and s[t, e].sum() > 0:
            total = s[t, e].sum()
            jac = np.eye(len(e)) / total - np.outer(s[t, e], np.ones(len(e))) / total ** 2   # [gate, s]
            ds[e] = dg @ jac
        elif not renorm:
            ds[e] = dg
        if softmax:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
        else:
            out[t] = ds * s[t] * gate_scores(-l[t:t + 1], False)[0]
    return out


# ---------------------------------------------------------------- FP8 product

def _spread(scale, rows, cols, tall):
    s = np.repeat(np.asarray(scale, np.float64), BLOCK, axis=1)[:, :cols]
    return np.repeat(s, BLOCK, axis=0)[:rows] if tall else s


def matmul_fp8(form, a, a_scale, b, b_scale):
    """(out, size): the product in float64, and the sum of the products' magnitudes.  form: "forward" (b [n, k]),
    "input_grad" (b [k, n]) or "weight_grad" (b [n, k], a scale per row and block); a, b hold the codes' values."""
    x = np.asarray(a, np.float64) * _spread(a_scale, *a.shape, False)
    y = np.asarray(b, np.float64) * _spread(b_scale, *b.shape, form != "weight_grad")
    if form != "input_grad":
        y = y.T
    return x @ y, np.abs(x) @ np.abs(y)


def run_scales(x, largest):
    """fp32 scales of the runs of 128 along the rows: amax times fp32(1 / largest), 1 for a run of zeros, NaN for a
    run that is not finite."""
    v = np.asarray(x, np.float32).reshape(x.shape[0], -1, BLOCK)
    amax = np.abs(v).max(axis=2)
    scale = (amax * (np.float32(1) / np.float32(largest))).astype(np.float32)
    scale = np.where(amax == 0, np.float32(1), scale)
    return np.where(np.isfinite(v).all(axis=2), scale, np.float32(np.nan))


# ---------------------------------------------------------------- SwiGLU in 8 bits

def codes8(x):
    """(codes int8, scales fp32) of bf16 values x [rows, 2I]."""
    scale = run_scales(x, 127)
    v = np.asarray(x, np.float32).reshape(*scale.shape, BLOCK)
    with np.errstate(invalid="ignore"):
        q = np.clip(np.rint(v / scale[:, :, None]), -127, 127)
    return np.nan_to_num(q, nan=0.0).astype(np.int8).reshape(x.shape), scale


def sigmoid(x):
    return gate_scores(np.asarray(x, np.float64), False)


def swiglu(ab):
    ab = np.asarray(ab, np.float64)
    a, b = np.split(ab, 2, axis=1)
    return a * sigmoid(a) * b


def swiglu8_backward(dh, codes, scales):
    """(d_ab, h) from the codes."""
    ab = codes.astype(np.float64) * _spread(scales, *codes.shape, False)
    a, b = np.split(ab, 2, axis=1)
    dh = np.asarray(dh, np.float64)
    sg = sigmoid(a)
    return np.concatenate([dh * b * sg * (1 + a * sigmoid(-a)), dh * a * sg], axis=1), a * sg * b
