"""Cases, plain forms and 64-bit values of the operators around the layer: the norm, the balance loss, the adapters.

Three operators, each in the forms that a training or serving step calls:

* "norm": the residual's addition and the root-mean-square norm behind it, with an E4M3 output (one fp32 scale per
  run of 128), and the gradients of input, residual and weight;
* "balance": the balance loss of a router from its logits and picks, the picks of each expert, and the gradient with
  respect to the logits, for sequences of different lengths packed one behind the other;
* "adapters": low-rank adapters of many requests added to a shared projection's output.

`run` computes a case in its plain form where `own` is false and through the package's entry points where it is true.
"""
import math

import torch

own = False
DEV = "cuda"
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6
ALPHA = 1e-4


# ---------------------------------------------------------------- cases

def _norm(name, rows, cols, dtype, residual, y, codes, train):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual, "y": y,
            "codes": codes, "train": train}


def _balance(name, tokens, experts, top_k, score, dtype, seqs, padding):
    return {"name": name, "op": "balance", "tokens": tokens, "experts": experts, "top_k": top_k, "score": score,
            "dtype": dtype, "seqs": seqs, "padding": padding}


def _adapters(name, rows, d_in, d_out, adapters, rank, mixed_ranks, order, out):
    return {"name": name, "op": "adapters", "rows": rows, "d_in": d_in, "d_out": d_out, "adapters": adapters,
            "rank": rank, "mixed_ranks": mixed_ranks, "order": order, "out": out}


def listed():
    return [
        # one decoded token before the FP8 projection: latency alone
        _norm("norm one token", 1, 7168, "bf16", True, True, True, False),
        # the mid-size layer's norm over a ragged serving batch
        _norm("norm 77 rows", 77, 2048, "bf16", True, False, True, False),
        # a training step of an fp32 residual stream, ragged, without 8-bit codes
        _norm("norm train fp32", 1021, 1408, "f32", True, True, False, True),
        # a prefill batch of the large layer: the sum and the codes, as the FP8 projection takes them
        _norm("norm prefill", 8192, 7168, "bf16", True, False, True, False),
        # a training batch of the large layer: y is kept too, for the weight gradient and the router
        _norm("norm train", 16384, 7168, "bf16", True, True, True, True),
        # a ragged micro-batch under a bf16 softmax router, seven packed sequences, its last rows padding
        _balance("balance odd", 1021, 60, 4, "softmax", "bf16", 7, 13),
        # a training batch of the 64-expert layer, one loss over the batch
        _balance("balance 64", 32768, 64, 6, "softmax", "f32", 1, 0),
        # a training batch of the 256-expert layer, a loss for each sequence
        _balance("balance 256", 16384, 256, 8, "sigmoid", "f32", 5, 100),
        # one decoded token of a request with an adapter, beside the stacked gate/up projection
        _adapters("adapters one token", 1, 7168, 4096, 8, 16, False, "mixed", "bf16"),
        # a decode batch, every request its own adapter of 32 resident ones, ranks up to 64, some rows without
        _adapters("adapters 64 requests", 64, 7168, 4096, 32, 64, True, "mixed", "bf16"),
        # ragged prompts through the mid-size layer's stacked projection, kept in fp32
        _adapters("adapters 1000 rows", 1000, 2048, 2816, 6, 32, False, "prompts", "f32"),
        # a prefill batch of several prompts through the large layer's stacked projection
        _adapters("adapters prefill", 8192, 7168, 4096, 8, 16, False, "prompts", "bf16"),
    ]


def _log(rng, lo, hi):
    """A size of the range, odd (the listed cases have the round ones)."""
    return (int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) - 1) | 1


def draw(rng):
    kind = rng.choice(("norm", "norm", "balance", "adapters", "adapters"))
    if kind == "norm":
        codes = rng.random() < 0.6
        cols = 128 * _log(rng, 1, 55) if codes else 8 * _log(rng, 4, 895)
        c = _norm("", _log(rng, 1, 16383), cols, rng.choice(("bf16", "bf16", "f32")), rng.random() < 0.7,
                  not codes or rng.random() < 0.5, codes, rng.random() < 0.5)
        if c["dtype"] == "f32":
            c["rows"] = max(1, c["rows"] // 2)
    elif kind == "balance":
        experts = rng.randint(8, 512)
        c = _balance("", _log(rng, 1, 32767 if experts <= 128 else 16383), experts, rng.randint(1, min(16, experts)),
                     rng.choice(("sigmoid", "softmax")), rng.choice(("f32", "bf16")), rng.choice((1, 1, _log(rng, 2, 64))), 0)
        c["padding"] = rng.choice((0, c["tokens"] // 9))
    else:
        rank = 8 * rng.choice((1, 2, 2, 3, 4, 8, 16))
        c = _adapters("", _log(rng, 1, 8191), 8 * _log(rng, 16, 895), 8 * _log(rng, 16, 511),
                      min(_log(rng, 1, 64), 2048 // rank), rank, rng.random() < 0.3,
                      rng.choice(("mixed", "prompts")), rng.choice(("bf16", "bf16", "f32")))
        if c["order"] == "mixed":   # rows of different requests side by side: a decode batch
            c["rows"] = min(c["rows"], 511)
    del c["name"]
    return c


def work(case):
    if case["op"] == "norm":
        n, es = case["rows"] * case["cols"], 4 if case["dtype"] == "f32" else 2
        b = es * (1 + 2 * case["residual"] + case["y"]) + 1.03125 * case["codes"]
        if case["train"]:
            b += es * (3 + case["residual"])
        return {"bytes": b * n + 4 * case["cols"] * (1 + case["train"]), "flops": n * (26 if case["train"] else 10)}
    if case["op"] == "balance":
        t, n, k = case["tokens"], case["experts"], case["top_k"]
        es = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * t * n * es + t * k * 4 + 8 * case["seqs"] * n, "flops": 16 * t * n}
    t, i, o, r = case["rows"], case["d_in"], case["d_out"], case["rank"]
    used = min(t, case["adapters"])
    es = 4 if case["out"] == "f32" else 2
    return {"bytes": 2 * t * i + 2 * es * t * o + 2 * used * r * (i + o), "flops": 2 * t * r * (i + o)}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 6151 + 29)


def _acts(rows, cols, g, dtype, size=1.0):
    """Activations: normal, with a few columns several times larger."""
    col = torch.where(torch.rand(cols, device=DEV, generator=g) < 0.01, 8.0, 1.0)
    return (size * torch.randn(rows, cols, device=DEV, generator=g) * col).to(dtype)


def _cuts(total, parts, g):
    """Borders of `parts` pieces of [0, total], some possibly empty (int32 [parts + 1])."""
    inner = torch.randint(0, total + 1, (parts - 1,), device=DEV, generator=g)
    ends = torch.tensor([0, total], device=DEV)
    return torch.sort(torch.cat([ends, inner])).values.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        dtype = F32 if case["dtype"] == "f32" else BF16
        s["x"] = _acts(r, c, g, dtype, 0.5)
        s["residual"] = _acts(r, c, g, dtype) if case["residual"] else None
        s["weight"] = 1 + 0.1 * torch.randn(c, device=DEV, generator=g)
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["y"] = torch.empty_like(s["x"]) if case["y"] else None
        if case["codes"]:
            s["codes"] = torch.empty(r, c, dtype=F8, device=DEV)
            s["scales"] = torch.empty(r, c // 128, device=DEV)
        if case["train"]:
            s["rstd"] = torch.empty(r, device=DEV)
            s["d_y"] = _acts(r, c, g, dtype, 0.01)
            s["d_sum"] = _acts(r, c, g, dtype, 0.01) if case["residual"] else None
            s["d_x"] = torch.empty_like(s["x"])
            s["d_weight"] = torch.empty(c, device=DEV)
    elif case["op"] == "balance":
        t, n, k, q = case["tokens"], case["experts"], case["top_k"], case["seqs"]
        liked = 0.5 * torch.randn(n, device=DEV, generator=g)      # some experts are liked more than others
        s["logits"] = (torch.randn(t, n, device=DEV, generator=g) + liked).to(F32 if case["dtype"] == "f32" else BF16)
        s["idx"] = torch.topk(s["logits"].to(F32), k, dim=1).indices.to(torch.int32)
        if case["padding"]:
            s["logits"][t - case["padding"]:] = -math.inf
            s["idx"][t - case["padding"]:] = -1
        s["start"] = _cuts(t, q, g)
        s["d_loss"] = 1 + 0.1 * torch.rand(q, device=DEV, generator=g)
        s["loss"] = torch.empty(q, device=DEV)
        s["counts"] = torch.empty(q, n, dtype=torch.int32, device=DEV)
        s["seq_tokens"] = torch.empty(q, dtype=torch.int32, device=DEV)
        s["prob_sum"] = torch.empty(q, n, device=DEV)
        s["d_logits"] = torch.empty_like(s["logits"])
    else:
        t, i, o, n, r = case["rows"], case["d_in"], case["d_out"], case["adapters"], case["rank"]
        out = F32 if case["out"] == "f32" else BF16
        s["x"] = _acts(t, i, g, BF16)
        s["base"] = torch.randn(t, o, device=DEV, generator=g).to(out)
        s["a"] = (torch.randn(n, r, i, device=DEV, generator=g) / math.sqrt(i)).to(BF16)
        s["b"] = (torch.randn(n, o, r, device=DEV, generator=g) / math.sqrt(r)).to(BF16)
        s["scale"] = 0.25 + torch.rand(n, device=DEV, generator=g)
        s["ranks"] = None
        if case["mixed_ranks"]:
            s["ranks"] = torch.randint(1, r + 1, (n,), device=DEV, generator=g).to(torch.int32)
        if case["order"] == "mixed":
            which = torch.randint(0, n, (t,), device=DEV, generator=g)
            if t > 1:   # a few requests have none
                which = torch.where(torch.rand(t, device=DEV, generator=g) < 0.05, -1, which)
        else:           # prompts behind one another, the adapters in any order, the last rows without one
            cuts = _cuts(t - t // 50, n, g)
            order = torch.randperm(n, device=DEV, generator=g)
            at = torch.searchsorted(cuts, torch.arange(t, device=DEV, dtype=torch.int32), right=True) - 1
            which = torch.where(at < n, order[at.clamp(max=n - 1)], -1)
        s["which"] = which.to(torch.int32)
        s["out"] = torch.empty(t, o, dtype=out, device=DEV)
    return s


# ---------------------------------------------------------------- passes

def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    if op == "balance":
        return _balance_own(state) if own else _balance_plain(state)
    return _adapters_own(state) if own else _adapters_plain(state)


def _workspace(size):
    return torch.empty(max(16, size), dtype=torch.uint8, device=DEV)


def _norm_own(s):
    import mixture_experts_layer_adjusted_amd as moe
    c = s["case"]
    if "shape" not in s:
        s["shape"] = moe.make_norm_shape(c["rows"], c["cols"], moe.MOE_DTYPE_F32 if c["dtype"] == "f32" else moe.MOE_DTYPE_BF16,
                                         EPS)
        s["workspace"] = _workspace(moe.moe_norm_workspace_size(s["shape"]) if c["train"] else 0)
    moe.moe_norm_forward(s["shape"], s["x"], s["residual"], s["weight"], s["sum"], s["y"], s.get("codes"), s.get("scales"),
                         s.get("rstd"))
    out = {k: s[k] for k in ("sum", "y", "codes", "scales") if s.get(k) is not None}
    if c["train"]:
        h = s["x"] if s["residual"] is None else s["sum"]
        moe.moe_norm_backward(s["shape"], s["d_y"], s["d_sum"], h, s["weight"], s["rstd"], s["d_x"], s["d_weight"],
                              s["workspace"])
        out |= {"d_x": s["d_x"], "d_weight": s["d_weight"]}
    return out


def _norm_plain(s):
    c, x = s["case"], s["x"]
    out = {}
    h = x.to(F32)
    if s["residual"] is not None:   # the sum is part of the stream: the norm is that of the kept value
        out["sum"] = (h + s["residual"].to(F32)).to(x.dtype)
        h = out["sum"].to(F32)
    rstd = 1 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    unit = h * rstd
    y = unit * s["weight"]
    if c["y"]:
        out["y"] = y.to(x.dtype)
    if c["codes"]:
        v = y.reshape(y.shape[0], -1, 128)
        amax = v.abs().amax(dim=2)
        out["scales"] = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        out["codes"] = (v / out["scales"][:, :, None]).clamp(-448, 448).to(F8).reshape(y.shape)
    if c["train"]:
        dy = s["d_y"].to(F32)
        g = dy * s["weight"]
        d = rstd * (g - unit * (g * unit).mean(dim=1, keepdim=True))
        if s["d_sum"] is not None:
            d = d + s["d_sum"].to(F32)
        out["d_x"] = d.to(x.dtype)
        out["d_weight"] = (dy * unit).sum(dim=0)
    return out


def _balance_own(s):
    import mixture_experts_layer_adjusted_amd as moe
    c = s["case"]
    if "cfg" not in s:
        s["cfg"] = moe.make_balance_config(
            c["tokens"], c["experts"], c["top_k"], moe.MOE_DTYPE_F32 if c["dtype"] == "f32" else moe.MOE_DTYPE_BF16,
            moe.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else moe.MOE_SCORE_SIGMOID, c["seqs"], ALPHA)
        s["workspace"] = _workspace(moe.moe_balance_workspace_size(s["cfg"]))
    moe.moe_balance_loss(s["cfg"], s["logits"], s["idx"], s["start"], s["loss"], s["counts"], s["seq_tokens"], s["prob_sum"],
                         s["workspace"])
    moe.moe_balance_backward(s["cfg"], s["logits"], s["idx"], s["start"], s["counts"], s["seq_tokens"], s["d_loss"],
                             s["d_logits"])
    return {k: s[k] for k in ("loss", "counts", "seq_tokens", "prob_sum", "d_logits")}


def _balance_plain(s):
    c, n, q = s["case"], s["case"]["experts"], s["case"]["seqs"]
    l, idx = s["logits"].to(F32), s["idx"].to(torch.int64)
    real = (idx >= 0).any(dim=1, keepdim=True)
    l = torch.where(real, l, 0.0)
    at = torch.arange(c["tokens"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["start"], at, right=True) - 1
    if c["score"] == "softmax":
        e = torch.exp(l - l.max(dim=1, keepdim=True).values)
        rest = 1.0
    else:
        e = 1 / (1 + torch.exp(-l))
        rest = 1 / (1 + torch.exp(l))
    p = torch.where(real, e / e.sum(dim=1, keepdim=True), 0.0)
    mine = (seq == torch.arange(q, device=DEV)[:, None]).to(F32)
    prob_sum = mine @ p
    tokens = torch.zeros(q, dtype=torch.int32, device=DEV).scatter_add_(0, seq, real.flatten().to(torch.int32))
    place = seq[:, None] * n + idx.clamp(min=0)
    counts = torch.zeros(q * n, dtype=torch.int32, device=DEV)
    counts.scatter_add_(0, place.flatten(), (idx >= 0).flatten().to(torch.int32))
    counts = counts.reshape(q, n)
    length = tokens.to(F32).clamp(min=1)[:, None]
    f = counts.to(F32) * (n / c["top_k"]) / length
    loss = ALPHA * (f * prob_sum / length).sum(dim=1)
    w = (s["d_loss"][:, None] * ALPHA * f / length)[seq]
    d = p * rest * (w - (p * w).sum(dim=1, keepdim=True))
    return {"loss": loss, "counts": counts, "seq_tokens": tokens, "prob_sum": prob_sum, "d_logits": d.to(s["logits"].dtype)}


def _adapters_own(s):
    import mixture_experts_layer_adjusted_amd as moe
    c = s["case"]
    if "shape" not in s:
        s["shape"] = moe.make_adapter_shape(c["rows"], c["d_in"], c["d_out"], c["adapters"], c["rank"],
                                            moe.MOE_DTYPE_F32 if c["out"] == "f32" else moe.MOE_DTYPE_BF16)
        s["workspace"] = _workspace(moe.moe_adapters_workspace_size(s["shape"]))
    moe.moe_adapters(s["shape"], s["x"], s["which"], s["a"], s["b"], s["scale"], s["ranks"], s["base"], s["out"],
                     s["workspace"])
    return s["out"]


def _adapters_plain(s):
    """Every row against every adapter; the row's own is kept."""
    c, n, r = s["case"], s["case"]["adapters"], s["case"]["rank"]
    low = (s["x"].to(F32) @ s["a"].to(F32).reshape(n * r, c["d_in"]).t()).reshape(-1, n, r)
    keep = (s["which"][:, None] == torch.arange(n, device=DEV))[:, :, None]
    if s["ranks"] is not None:
        keep = keep & (torch.arange(r, device=DEV) < s["ranks"][:, None])
    low = torch.where(keep, low * s["scale"][:, None], 0.0).reshape(-1, n * r)
    up = s["b"].to(F32).permute(0, 2, 1).reshape(n * r, c["d_out"])
    return (s["base"].to(F32) + low @ up).to(s["out"].dtype)


# ---------------------------------------------------------------- values in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(case, s)
    if case["op"] == "balance":
        return _balance_exact(case, s)
    return _adapters_exact(case, s)


def _norm_exact(case, s):
    """Block by block of the rows; the gradient from the Jacobian of h / |h|."""
    out, dw = {}, torch.zeros(case["cols"], dtype=torch.float64, device=DEV)
    w = s["weight"].double()
    for at in range(0, case["rows"], 2048):
        rows = slice(at, at + 2048)
        x = s["x"][rows]
        h = x.double()
        got = {}
        if case["residual"]:
            got["sum"] = h + s["residual"][rows].double()
            h = got["sum"].to(x.dtype).double()
        size = (h.square().sum(1, keepdim=True) / case["cols"] + EPS).sqrt()
        y = h / size * w
        if case["y"]:
            got["y"] = y
        if case["codes"]:
            top = y.unflatten(1, (-1, 128)).abs().amax(2)
            got["scales"] = torch.where(top > 0, top / 448, 1.0)
            got["codes"] = (y.unflatten(1, (-1, 128)) / got["scales"][:, :, None]).float().to(F8).double().flatten(1)
        if case["train"]:
            dy = s["d_y"][rows].double()
            v = dy * w
            d = v / size - h * (v * h).sum(1, keepdim=True) / (case["cols"] * size ** 3)
            got["d_x"] = d + s["d_sum"][rows].double() if case["residual"] else d
            dw += (dy * h / size).sum(0)
        for k, v in got.items():
            out.setdefault(k, []).append(v)
    out = {k: torch.cat(v) for k, v in out.items()}
    if case["train"]:
        out["d_weight"] = dw
    return out


def _balance_exact(case, s):
    """Sequence by sequence."""
    n, k = case["experts"], case["top_k"]
    l, idx = s["logits"].double(), s["idx"].long()
    start = s["start"].tolist()
    out = {"loss": [], "counts": [], "seq_tokens": [], "prob_sum": [], "d_logits": []}
    for j in range(case["seqs"]):
        lj, ij = l[start[j]:start[j + 1]], idx[start[j]:start[j + 1]]
        live = (ij >= 0).any(1) if ij.numel() else torch.zeros(len(ij), dtype=torch.bool, device=DEV)
        size = int(live.sum())
        counts = torch.bincount(ij[ij >= 0], minlength=n)
        d = torch.zeros_like(lj)
        total = torch.zeros(n, dtype=torch.float64, device=DEV)
        loss = 0.0
        if size:
            z = lj[live]
            slope = torch.ones_like(z)
            if case["score"] == "softmax":
                p = torch.softmax(z, 1)
            else:
                p = torch.special.expit(z)
                p, slope = p / p.sum(1, keepdim=True), torch.special.expit(-z)
            total = p.sum(0)
            f = counts.double() * n / (k * size)
            loss = ALPHA * float((f * total).sum()) / size
            pull = float(s["d_loss"][j]) * ALPHA * f / size
            d[live] = p * slope * (pull - (p @ pull)[:, None])
        out["loss"].append(torch.tensor(loss, dtype=torch.float64, device=DEV))
        out["counts"].append(counts.to(torch.int32))
        out["seq_tokens"].append(torch.tensor(size, dtype=torch.int32, device=DEV))
        out["prob_sum"].append(total)
        out["d_logits"].append(d)
    return {"loss": torch.stack(out["loss"]), "counts": torch.stack(out["counts"]),
            "seq_tokens": torch.stack(out["seq_tokens"]), "prob_sum": torch.stack(out["prob_sum"]),
            "d_logits": torch.cat(out["d_logits"])}


def _adapters_exact(case, s):
    """Adapter by adapter, its own rows alone."""
    out = s["base"].double()
    for j in range(case["adapters"]):
        rows = torch.nonzero(s["which"] == j).flatten()
        r = case["rank"] if s["ranks"] is None else int(s["ranks"][j])
        if rows.numel():
            low = s["x"][rows].double() @ s["a"][j, :r].double().t().contiguous()
            out[rows] += float(s["scale"][j]) * (low @ s["b"][j, :, :r].double().t().contiguous())
    return out
