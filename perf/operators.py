"""Cases, plain forms and 64-bit values of the layer's operators: the gate, the FP8 product, the 8-bit checkpoint.

Three operators, each in the forms that a training or serving step calls:

* "gate": routing from given logits (softmax or sigmoid scores, balance bias, expert groups, top-k, gates
  renormalised or not), and its gradient with respect to the logits;
* "matmul": the product of E4M3 operands with one fp32 scale per block of 128: a forward product and an input
  gradient on quantised operands, and a weight gradient from the bf16 activations;
* "swiglu8": SwiGLU whose inputs are kept for the backward pass in 8 bits, forward and backward.

`run` computes a case in its plain form where `own` is false and through the package's entry points where it is true.
"""
import math

import torch

own = False
DEV = "cuda"
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ---------------------------------------------------------------- cases

def _gate(name, tokens, experts, top_k, score, groups, top_groups, group_score, renorm, bias, dtype, train, padding):
    return {"name": name, "op": "gate", "tokens": tokens, "experts": experts, "top_k": top_k, "score": score,
            "groups": groups, "top_groups": top_groups, "group_score": group_score, "renorm": renorm, "bias": bias,
            "dtype": dtype, "train": train, "padding": padding}


def _matmul(name, form, m, n, k, out):
    return {"name": name, "op": "matmul", "form": form, "m": m, "n": n, "k": k, "out": out}


def _swiglu(name, rows, inter):
    return {"name": name, "op": "swiglu8", "rows": rows, "inter": inter}


def listed():
    return [
        # one token of a served sequence, 256 experts in 8 groups: latency alone
        _gate("gate decode", 1, 256, 8, "sigmoid", 8, 4, "top2", True, True, "f32", False, 0),
        # a ragged training batch under a bf16 softmax router, gates not renormalised; its last rows are padding
        # tokens whose logits are all masked
        _gate("gate softmax odd", 1021, 60, 4, "softmax", 1, 1, "max", False, False, "bf16", True, 13),
        # a training step of the 64-expert layer, 6 active, renormalised softmax
        _gate("gate train 64", 32768, 64, 6, "softmax", 1, 1, "max", True, False, "f32", True, 0),
        # a training step of the 256-expert layer, 8 active, group-limited, with the balance bias
        _gate("gate train 256", 16384, 256, 8, "sigmoid", 8, 4, "top2", True, True, "f32", True, 0),
        # one decoded token through the stacked gate/up projection (weights read once: bandwidth)
        _matmul("fp8 one token", "forward", 1, 4096, 7168, "bf16"),
        # a small serving batch, ragged, through the down projection
        _matmul("fp8 77 tokens", "forward", 77, 7168, 2048, "bf16"),
        # a ragged prompt through the mid-size layer's stacked projection
        _matmul("fp8 1000 tokens", "forward", 1000, 2816, 2048, "bf16"),
        # a prefill batch through the stacked gate/up projection
        _matmul("fp8 prefill", "forward", 8192, 4096, 7168, "bf16"),
        # the input gradient of the down projection, weights as stored, one token over a tile
        _matmul("fp8 input grad", "input_grad", 4097, 2048, 7168, "bf16"),
        # the stacked projection's weight gradient over a ragged batch, kept in fp32
        _matmul("fp8 weight grad", "weight_grad", 4096, 7168, 8100, "f32"),
        # one ragged micro-batch of the mid-size layer's SwiGLU, forward and backward
        _swiglu("swiglu8 255", 255, 1408),
        # the permuted rows of a training batch of the large layer
        _swiglu("swiglu8 32768", 32768, 2048),
    ]


def _log(rng, lo, hi):
    """A size of the range, odd (the listed cases have the round ones)."""
    return (int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) - 1) | 1


def draw(rng):
    kind = rng.choice(("gate", "gate", "matmul", "matmul", "matmul", "swiglu8"))
    if kind == "gate":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * rng.randint(max(2, 8 // groups), 512 // groups)
        top_groups = rng.randint(1, groups)
        tokens = _log(rng, 1, 32768 if experts <= 128 else 16384)
        c = _gate("", tokens, experts, rng.randint(1, min(32, top_groups * (experts // groups))),
                  rng.choice(("sigmoid", "softmax")), groups, top_groups, rng.choice(("max", "top2")),
                  rng.random() < 0.6, rng.random() < 0.6, rng.choice(("f32", "bf16")), rng.random() < 0.6,
                  rng.choice((0, 0, tokens // 8)))
    elif kind == "matmul":
        form = rng.choice(("forward", "forward", "input_grad", "weight_grad"))
        n, wide = 16 * _log(rng, 8, 448), 128 * _log(rng, 1, 56)
        if form == "weight_grad":
            c = _matmul("", form, 16 * _log(rng, 8, 256), n, _log(rng, 1, 8192), rng.choice(("f32", "bf16")))
        else:
            c = _matmul("", form, _log(rng, 1, 4096), n, wide, rng.choice(("bf16", "bf16", "f32")))
    else:
        c = _swiglu("", _log(rng, 1, 16384), 128 * _log(rng, 1, 32))
    del c["name"]
    return c


def work(case):
    if case["op"] == "gate":
        t, n, k = case["tokens"], case["experts"], case["top_k"]
        es = 4 if case["dtype"] == "f32" else 2
        b = t * n * es + t * k * 8 + n * 4 + (n * 4 if case["bias"] else 0)
        if case["train"]:
            b += t * k * 4 + t * n * es
        return {"bytes": b, "flops": t * n * (12 if case["train"] else 6)}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        o = m * n * (4 if case["out"] == "f32" else 2)
        if case["form"] == "weight_grad":
            return {"bytes": 2 * k * (m + n) + o, "flops": 2 * m * n * k}
        kb = k // 128
        return {"bytes": m * k + n * k + 4 * (m * kb + -(-n // 128) * kb) + o, "flops": 2 * m * n * k}
    # reads [a b] and dh, writes h, the codes, [dA dB] and H, reads the codes back
    r, i = case["rows"], case["inter"]
    return {"bytes": r * i * 18 + 2 * 4 * r * (2 * i // 128), "flops": r * i * 40}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _keys(logits, bias, case, wide):
    """Scores and ranking keys in the type `wide` (masked experts: -inf)."""
    l = logits.to(wide)
    shut = l == -math.inf
    if bias is not None:
        shut = shut | (bias == -math.inf)
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        top = l.max(dim=1, keepdim=True).values
        e = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = e.sum(dim=1, keepdim=True)
        s = e / torch.where(total > 0, total, torch.ones_like(total))
    c = s if bias is None else s + bias.to(wide)
    return s, torch.where(shut, torch.full_like(c, -math.inf), c)


def _group_scores(c, case):
    t, n = c.shape
    g = c.reshape(t, case["groups"], n // case["groups"])
    best = g.max(dim=2).values
    if case["group_score"] == "max" or g.shape[2] == 1:
        return best
    two = torch.sort(g, dim=2, descending=True, stable=True).values[:, :, :2]
    return torch.where(two[:, :, 1] == -math.inf, two[:, :, 0], two.sum(dim=2))


def _limited(c, case):
    """The keys with every group outside the best `top_groups` masked."""
    if case["top_groups"] >= case["groups"]:
        return c
    score = _group_scores(c, case)
    order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
    keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order, True)
    keep = keep.repeat_interleave(c.shape[1] // case["groups"], dim=1)
    return torch.where(keep, c, torch.full_like(c, -math.inf))


def _clear(logits, bias, case):
    """Rows whose choice does not hang on the last bits of a score: either order of two keys that differ by less
    than 32-bit rounding is right, so such rows are no test of anything.  Equal keys (equal logits without a
    bias) stay: they go to the lower index."""
    _, c = _keys(logits, bias, case, torch.float64)
    plain = bias is None
    ok = torch.ones(c.shape[0], dtype=torch.bool, device=c.device)
    near = 2e-6 * torch.where(c == -math.inf, torch.zeros_like(c), c).abs().max(dim=1, keepdim=True).values

    def apart(v, rank, ties):
        gap = (v[:, :-1] - v[:, 1:])[:, rank]
        eps = near if not (plain and case["score"] == "softmax") else 4e-6 * v[:, 1:][:, rank].abs()
        eps = torch.where(eps < math.inf, eps, torch.zeros_like(eps))
        small = (gap <= eps) & ~torch.isnan(gap)
        return ~(small & ~((gap == 0) & ties)).any(dim=1)

    if case["top_groups"] < case["groups"]:
        score = torch.sort(_group_scores(c, case), dim=1, descending=True).values
        at = case["top_groups"] - 1
        ok &= apart(score, slice(at, at + 1), plain and case["group_score"] == "max")
    c = torch.sort(_limited(c, case), dim=1, descending=True).values
    return ok & apart(c, slice(0, case["top_k"]), plain)


def _logits(case, g):
    t, n = case["tokens"], case["experts"]
    dtype = F32 if case["dtype"] == "f32" else BF16
    liked = 0.5 * torch.randn(n, device=DEV, generator=g)          # some experts are liked more than others
    bias = None
    if case["bias"]:
        bias = (0.1 if case["score"] == "sigmoid" else 0.5 / n) * torch.randn(n, device=DEV, generator=g)

    def some(rows):
        return (torch.randn(rows, n, device=DEV, generator=g) + liked).to(dtype)

    logits = some(t)
    for _ in range(10):
        bad = torch.nonzero(~_clear(logits, bias, case)).flatten()
        if bad.numel() == 0:
            break
        logits[bad] = some(bad.numel())
    bad = ~_clear(logits, bias, case)
    if bool(bad.any()) and not bool(bad.all()):
        logits[bad] = logits[torch.nonzero(~bad).flatten()[0]]
    if case["padding"]:
        logits[t - case["padding"]:] = -math.inf
    return logits, bias


def _tiles(x):
    """Rows quantised per run of 128: E4M3 codes and fp32 scales."""
    v = x.to(F32).reshape(x.shape[0], -1, 128)
    amax = v.abs().amax(dim=2)
    scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    return (v / scale[:, :, None]).to(F8).reshape(x.shape), scale


def _blocks(w):
    """A matrix quantised per 128 x 128 block (the last blocks may be smaller)."""
    r, c = w.shape
    rb, cb = -(-r // 128), -(-c // 128)
    full = torch.zeros(rb * 128, cb * 128, device=w.device)
    full[:r, :c] = w
    v = full.reshape(rb, 128, cb, 128)
    amax = v.abs().amax(dim=(1, 3))
    scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    q = (v / scale[:, None, :, None]).to(F8).reshape(rb * 128, cb * 128)
    return q[:r, :c].contiguous(), scale


def _acts(rows, cols, g, size=1.0):
    """Activations: normal, with a few columns several times larger, in bf16."""
    col = torch.where(torch.rand(cols, device=DEV, generator=g) < 0.01, 8.0, 1.0)
    return (size * torch.randn(rows, cols, device=DEV, generator=g) * col).to(BF16)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "gate":
        t, n, k = case["tokens"], case["experts"], case["top_k"]
        s["logits"], s["bias"] = _logits(case, g)
        s["d_gate"] = torch.randn(t, k, device=DEV, generator=g)
        s["idx"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
        s["gate"] = torch.empty(t, k, device=DEV)
        s["load"] = torch.empty(n, dtype=torch.int32, device=DEV)
        s["d_logits"] = torch.empty_like(s["logits"])
    elif case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        if case["form"] == "weight_grad":
            s["dy"], s["x"] = _acts(k, m, g, 0.01), _acts(k, n, g)
            pad = -(-k // 128) * 128
            for name, w in (("dy", m), ("x", n)):
                s[name + "_q"] = torch.empty(w, pad, dtype=F8, device=DEV)
                s[name + "_s"] = torch.empty(w, pad // 128, device=DEV)
        else:
            s["a"], s["a_s"] = _tiles(_acts(m, k, g))
            shape = (n, k) if case["form"] == "forward" else (k, n)
            s["b"], s["b_s"] = _blocks(torch.randn(shape, device=DEV, generator=g) / math.sqrt(shape[1]))
        s["out"] = torch.empty(m, n, device=DEV, dtype=F32 if case["out"] == "f32" else BF16)
    else:
        r, i = case["rows"], case["inter"]
        s["ab"], s["dh"] = _acts(r, 2 * i, g), _acts(r, i, g, 0.01)
        s["h"], s["h_again"] = torch.empty_like(s["dh"]), torch.empty_like(s["dh"])
        s["d_ab"] = torch.empty_like(s["ab"])
        s["saved"] = torch.empty(r, 2 * i, dtype=torch.int8, device=DEV)
        s["saved_s"] = torch.empty(r, 2 * i // 128, device=DEV)
    return s


# ---------------------------------------------------------------- passes

def run(state):
    op = state["case"]["op"]
    if op == "gate":
        return _gate_own(state) if own else _gate_plain(state)
    if op == "matmul":
        return _matmul_own(state) if own else _matmul_plain(state)
    return _swiglu_own(state) if own else _swiglu_plain(state)


def _workspace(s, size):
    ws = s.get("workspace")
    if ws is None:
        ws = s["workspace"] = torch.empty(max(1, size), dtype=torch.uint8, device=DEV)
    return ws


def _gate_own(s):
    import mixture_experts_layer_adjusted_amd as moe
    c = s["case"]
    cfg = s.get("cfg")
    if cfg is None:
        cfg = s["cfg"] = moe.make_gate_config(
            c["tokens"], c["experts"], c["top_k"], moe.MOE_DTYPE_F32 if c["dtype"] == "f32" else moe.MOE_DTYPE_BF16,
            moe.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else moe.MOE_SCORE_SIGMOID, c["groups"], c["top_groups"],
            moe.MOE_GROUP_MAX if c["group_score"] == "max" else moe.MOE_GROUP_TOP2, c["renorm"], 1.0)
        _workspace(s, moe.moe_gate_workspace_size(cfg))
    moe.moe_gate(cfg, s["logits"], s["bias"], s["idx"], s["gate"], s["load"], s["workspace"])
    out = {"idx": s["idx"], "gate": s["gate"], "load": s["load"]}
    if c["train"]:
        moe.moe_gate_backward(cfg, s["logits"], s["idx"], s["d_gate"], s["d_logits"])
        out["d_logits"] = s["d_logits"]
    return out


def _gate_plain(s):
    c, logits, bias = s["case"], s["logits"], s["bias"]
    score, key = _keys(logits, bias, c, F32)
    key = _limited(key, c)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    taken = key.gather(1, order) > -math.inf
    idx = torch.where(taken, order, torch.full_like(order, -1)).to(torch.int32)
    chosen = torch.where(taken, score.gather(1, order), 0.0)
    total = chosen.sum(dim=1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total)) if c["renorm"] else torch.ones_like(total)
    gate = chosen / total
    load = torch.zeros(c["experts"], dtype=torch.int32, device=DEV)
    load.scatter_add_(0, order.flatten(), taken.flatten().to(torch.int32))
    out = {"idx": idx, "gate": gate, "load": load}
    if c["train"]:
        d = torch.where(taken, s["d_gate"], 0.0)
        if c["renorm"]:
            d = torch.where(taken, (d - (d * gate).sum(dim=1, keepdim=True)) / total, 0.0)
        ds = torch.zeros_like(score).scatter_(1, order, d)
        if c["score"] == "sigmoid":
            dl = ds * score * (1 - score)
        else:
            dl = score * (ds - (ds * score).sum(dim=1, keepdim=True))
        out["d_logits"] = dl.to(logits.dtype)
    return out


def _matmul_own(s):
    import mixture_experts_layer_adjusted_amd as moe
    c = s["case"]
    shape = s.get("shape")
    if shape is None:
        form = {"forward": moe.MOE_FP8_FORWARD, "input_grad": moe.MOE_FP8_INPUT_GRAD,
                "weight_grad": moe.MOE_FP8_WEIGHT_GRAD}[c["form"]]
        k = c["k"] if c["form"] != "weight_grad" else s["x_q"].shape[1]
        shape = s["shape"] = moe.make_matmul_shape(c["m"], c["n"], k, form,
                                                   moe.MOE_DTYPE_F32 if c["out"] == "f32" else moe.MOE_DTYPE_BF16)
        _workspace(s, moe.moe_matmul_fp8_workspace_size(shape))
    if c["form"] == "weight_grad":
        moe.moe_quantize_act_t(c["k"], c["m"], s["dy"], s["dy_q"], s["dy_s"])
        moe.moe_quantize_act_t(c["k"], c["n"], s["x"], s["x_q"], s["x_s"])
        a, a_s, b, b_s = s["dy_q"], s["dy_s"], s["x_q"], s["x_s"]
    else:
        a, a_s, b, b_s = s["a"], s["a_s"], s["b"], s["b_s"]
    moe.moe_matmul_fp8(shape, a, a_s, b, b_s, s["out"], s["workspace"])
    return s["out"]


def _spread(codes, scale, tall):
    """The fp32 values that codes stand for; `tall`: scales per 128 x 128 block."""
    if tall:
        scale = scale.repeat_interleave(128, dim=0)[:codes.shape[0]]
    return codes.to(F32) * scale.repeat_interleave(128, dim=1)[:, :codes.shape[1]]


def _matmul_plain(s):
    c = s["case"]
    if c["form"] == "weight_grad":
        pad = -c["k"] % 128
        pair = []
        for v in (s["dy"], s["x"]):
            v = torch.cat([v, v.new_zeros(pad, v.shape[1])]).t()
            pair.append(_spread(*_tiles(v), False))
        out = pair[0] @ pair[1].t()
    else:
        b = _spread(s["b"], s["b_s"], True)
        out = _spread(s["a"], s["a_s"], False) @ (b.t() if c["form"] == "forward" else b)
    return out.to(s["out"].dtype)


def _swiglu_own(s):
    import mixture_experts_layer_adjusted_amd as moe
    c = s["case"]
    moe.moe_swiglu_forward8(c["rows"], c["inter"], s["ab"], s["h"], s["saved"], s["saved_s"])
    moe.moe_swiglu_backward8(c["rows"], c["inter"], s["dh"], s["saved"], s["saved_s"], s["d_ab"], s["h_again"])
    return {"h": s["h"], "d_ab": s["d_ab"], "h_again": s["h_again"]}


def _swiglu_plain(s):
    r, i = s["case"]["rows"], s["case"]["inter"]
    ab = s["ab"].to(F32)
    a, b = ab[:, :i], ab[:, i:]
    h = a / (1 + torch.exp(-a)) * b
    v = ab.reshape(r, -1, 128)
    scale = v.abs().amax(dim=2, keepdim=True) / 127
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    codes = torch.round(v / scale).to(torch.int8)
    ab = (codes.to(F32) * scale).reshape(r, 2 * i)
    a, b, dh = ab[:, :i], ab[:, i:], s["dh"].to(F32)
    sig = 1 / (1 + torch.exp(-a))
    d_ab = torch.cat([dh * b * sig * (1 + a * (1 - sig)), dh * a * sig], dim=1)
    return {"h": h.to(BF16), "d_ab": d_ab.to(BF16), "h_again": (a * sig * b).to(BF16)}


# ---------------------------------------------------------------- values in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gate":
        return _gate_exact(case, s)
    if case["op"] == "matmul":
        return _matmul_exact(case, s)
    return _swiglu_exact(case, s)


def _gate_exact(case, s):
    """Rank by rank: each pick is the largest key left, the first of equals."""
    l = s["logits"].double()
    t, n = l.shape
    if case["score"] == "sigmoid":
        p = torch.special.expit(l)
    else:
        p = torch.nan_to_num(torch.softmax(l, dim=1), nan=0.0)
    key = p + (0 if s["bias"] is None else s["bias"].double())
    key = key.masked_fill(torch.isneginf(l), -math.inf)
    if case["top_groups"] < case["groups"]:
        size = n // case["groups"]
        grouped = key.view(t, case["groups"], size)
        score = grouped.amax(2)
        if case["group_score"] == "top2" and size > 1:
            second = grouped.topk(2, dim=2).values[:, :, 1]
            score = score + second.masked_fill(torch.isneginf(second), 0)
        # a group's rank: how many groups are above it, or equal and before it
        above = (score[:, None, :] > score[:, :, None]).sum(2)
        equal = (score[:, None, :] == score[:, :, None]).tril(-1).sum(2)
        key = grouped.masked_fill((above + equal >= case["top_groups"])[:, :, None], -math.inf).reshape(t, n)
    place = torch.arange(n, device=DEV)
    picks = []
    left = key.clone()
    for _ in range(case["top_k"]):
        best = left.amax(1, keepdim=True)
        at = torch.where((left == best) & torch.isfinite(best), place, n).amin(1)
        picks.append(at)
        left.masked_fill_(place == at[:, None], -math.inf)
    idx = torch.stack(picks, 1)
    real = idx < n
    mask = torch.zeros(t, n + 1, dtype=torch.float64, device=DEV).scatter_(1, idx, 1.0)[:, :n]
    sel = torch.cat([p, p.new_zeros(t, 1)], 1).gather(1, idx)
    total = sel.sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0) if case["renorm"] else torch.ones_like(total)
    out = {"idx": torch.where(real, idx, -1).to(torch.int32), "gate": sel / total,
           "load": mask.sum(0).to(torch.int32)}
    if case["train"]:
        dg = torch.zeros(t, n + 1, dtype=torch.float64, device=DEV).scatter_(1, idx, s["d_gate"].double())[:, :n] * mask
        # the gate of expert i is mask_i p_i / total; total is the selected sum, or 1
        dp = mask * dg / total
        if case["renorm"]:
            dp = dp - mask * (dg * mask * p).sum(1, keepdim=True) / total ** 2
        if case["score"] == "sigmoid":
            dl = dp * torch.special.expit(l) * torch.special.expit(-l)
        else:
            dl = p * dp - p * (p * dp).sum(1, keepdim=True)
        out["d_logits"] = torch.nan_to_num(dl, nan=0.0)
    return out


def _matmul_exact(case, s):
    """Block by block of the contraction, in 64 bits."""
    def runs(v):   # the format itself: one fp32 scale per run of 128, the code nearest to the fp32 quotient
        v = v.float().unflatten(1, (-1, 128))
        top = v.abs().amax(2, keepdim=True)
        sc = torch.where(top > 0, top / 448, 1.0)
        return (v / sc).to(F8).double() * sc.double()

    if case["form"] == "weight_grad":
        pad = -case["k"] % 128
        a, b = (runs(torch.nn.functional.pad(v, (0, 0, 0, pad)).t()) for v in (s["dy"], s["x"]))
    else:
        kb = case["k"] // 128
        a = s["a"].double().unflatten(1, (kb, 128)) * s["a_s"].double()[:, :, None]
        b = s["b"].double() if case["form"] == "forward" else s["b"].double().t()
        bs = s["b_s"].double() if case["form"] == "forward" else s["b_s"].double().t()
        row = torch.arange(case["n"], device=DEV) // 128
        b = b.unflatten(1, (kb, 128)) * bs[row][:, :, None]
    out = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
    for j in range(0, a.shape[1], 8):
        out += a[:, j:j + 8].flatten(1) @ b[:, j:j + 8].flatten(1).t().contiguous()
    return out


def _swiglu_exact(case, s):
    r, i = case["rows"], case["inter"]
    out = {"h": [], "d_ab": [], "h_again": []}
    for at in range(0, r, 4096):
        x = s["ab"][at:at + 4096].double()
        dh = s["dh"][at:at + 4096].double()
        out["h"].append(torch.nn.functional.silu(x[:, :i]) * x[:, i:])
        top = x.unflatten(1, (-1, 128)).abs().amax(2, keepdim=True)
        step = torch.where(top > 0, (top.float() / 127).double(), 1.0)   # the stored scale is fp32
        x = (torch.round(x.unflatten(1, (-1, 128)) / step) * step).flatten(1)
        a, b = x[:, :i], x[:, i:]
        up, down = torch.special.expit(a), torch.special.expit(-a)
        out["d_ab"].append(torch.cat([dh * b * (up + a * up * down), dh * a * up], 1))
        out["h_again"].append(a * up * b)
    return {k: torch.cat(v) for k, v in out.items()}
