"""moe_norm_forward and moe_norm_backward on the GPU against float64.

The sum is one fp32 addition and one rounding: compared bit for bit.  rstd is fp32: the squares' sum has at most 3 + 2 +
6 + 16 roundings behind a square's (8 values, 4 vectors, 64 lanes, 16 wavefronts) and is halved by the root; division and
root add three: under 20 of 2^-24, and 2^-19 is asked.  y has two products more and its type's rounding (bf16 2^-8).  A
code is within half a step (2^-4 of the value, 2^-10 of the scale below 2^-6 of it) and y's fp32 error.  dh is a difference, so its error counts
against its terms; d_weight has D additions one after another, the rows of a workgroup and the workgroups:
(2^-18 + D 2^-24) of its terms."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from oracle import block as B  # noqa: E402

TYPES = {"bf16": (torch.bfloat16, moe.MOE_DTYPE_BF16, 2.0 ** -8), "f32": (torch.float32, moe.MOE_DTYPE_F32, 2.0 ** -24)}
EPS = 1e-6


def np_(t):
    return t.float().cpu().numpy()


def inputs(rows, cols, stream, seed, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    t = TYPES[stream][0]
    some = lambda s: (s * torch.randn(rows, cols, device="cuda", generator=g)).to(t)  # noqa: E731
    x, r, d_y, d_s = some(size), some(size), some(1.0), some(1.0)
    w = 1 + 0.2 * torch.randn(cols, device="cuda", generator=g)
    return x, r, w, d_y, d_s


def empty_codes(rows, cols):
    return torch.full((rows, cols), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)


def forward(x, r, w, stream, codes=False, y=True, total=True, rstd=True, eps=EPS, on=None):
    rows, cols = x.shape
    shape = moe.make_norm_shape(rows, cols, TYPES[stream][1], eps)
    out = {"sum": torch.full_like(x, float("nan")) if total and r is not None else None,
           "y": torch.full_like(x, float("nan")) if y else None,
           "codes": empty_codes(rows, cols) if codes else None,
           "scales": torch.full((rows, cols // 128), float("nan"), device="cuda") if codes else None,
           "rstd": torch.full((rows,), float("nan"), device="cuda") if rstd else None}
    moe.moe_norm_forward(shape, x, r, w, out["sum"], out["y"], out["codes"], out["scales"], out["rstd"], on)
    return out


def backward(d_y, d_s, h, w, rstd, stream, weight=True, on=None):
    rows, cols = h.shape
    shape = moe.make_norm_shape(rows, cols, TYPES[stream][1], EPS)
    d_x = torch.full_like(h, float("nan"))
    d_w = torch.full((cols,), float("nan"), device="cuda") if weight else None
    ws = torch.full((moe.moe_norm_workspace_size(shape),), 255, dtype=torch.uint8, device="cuda") if weight else None
    moe.moe_norm_backward(shape, d_y, d_s, h, w, rstd, d_x, d_w, ws, on)
    return d_x, d_w


def same(a, b):
    return all((a[k] is None and b[k] is None) or torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)


def check_codes(out, y_ref):
    s, q = np_(out["scales"]).astype(np.float64), np_(out["codes"]).astype(np.float64)
    v = y_ref.reshape(*s.shape, 128)
    amax = np.abs(v).max(axis=2)
    want = np.where(amax > 0, amax / 448, 1.0)
    assert (np.abs(s - want) <= 2.0 ** -18 * want).all()
    got = q.reshape(v.shape) * s[:, :, None]
    assert (np.abs(got - v) <= (2.0 ** -4 + 2.0 ** -17) * np.abs(v) + 2.0 ** -10 * s[:, :, None]).all()


def depth(rows):
    """Additions one after another: the rows of one of 128 or more workgroups, its wavefronts, the workgroups."""
    return -(-rows // 128) + 3 + 4 + 16


CASES = [(1, 8, "bf16"), (1, 7168, "bf16"), (3, 128, "f32"), (5, 520, "bf16"), (77, 2048, "bf16"), (9, 2056, "f32"),
         (255, 1408, "f32"), (33, 4096, "bf16"), (2, 16392, "bf16"), (3, 32768, "f32"), (1021, 1024, "bf16"),
         (700, 7168, "bf16")]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("rows,cols,stream", CASES)
def test_against_float64(rows, cols, stream, residual):
    x, r, w, d_y, d_s = inputs(rows, cols, stream, rows + cols)
    if not residual:
        r = d_s = None
    codes = cols % 128 == 0
    out = forward(x, r, w, stream, codes=codes)
    h = B.norm_sum(np_(x), np_(r) if residual else None, stream)
    if residual:
        assert np.array_equal(np_(out["sum"]), h)
    y, rstd = B.norm(h, np_(w), EPS)
    half = TYPES[stream][2]
    assert (np.abs(np_(out["rstd"]) - rstd) <= 2.0 ** -19 * rstd).all()
    assert (np.abs(np_(out["y"]) - y) <= (half + 2.0 ** -18) * np.abs(y)).all()
    if codes:
        check_codes(out, y)
    held = out["sum"] if residual else x
    d_x, d_w = backward(d_y, d_s, held, w, out["rstd"], stream)
    ref, ref_w = B.norm_backward(h, np_(w), EPS, np_(d_y), np_(d_s) if residual else None)
    u, gr = h * rstd[:, None], np_(d_y) * np_(w).astype(np.float64)
    size = rstd[:, None] * (np.abs(gr) + np.abs(u) * np.abs(gr * u).mean(axis=1, keepdims=True))
    size += np.abs(np_(d_s)) if residual else 0
    assert (np.abs(np_(d_x) - ref) <= half * np.abs(ref) + 2.0 ** -17 * size).all()
    size = np.abs(np_(d_y) * u).sum(axis=0)
    assert (np.abs(np_(d_w) - ref_w) <= (2.0 ** -18 + depth(rows) * 2.0 ** -24) * size).all()


@pytest.mark.parametrize("rows,cols,stream", [
    (1, 8, "bf16"), (2, 8, "f32"), (3, 40, "bf16"), (384, 520, "f32"), (385, 520, "f32"), (383, 1032, "bf16"),
    (384, 2056, "bf16"), (292, 7168, "f32"), (293, 7168, "f32"), (64, 32768, "f32"), (65, 32768, "f32"), (129, 32760, "bf16"),
    (333, 24, "f32"), (100, 16384, "bf16")])
def test_weight_gradient_by_columns_and_by_rows(rows, cols, stream):
    """Few rows sum it up by columns in one kernel: both sides of where that ends.  Also rows whose d_y is zero."""
    x, r, w, d_y, d_s = inputs(rows, cols, stream, rows + cols)
    d_y[rows // 2] = 0
    out = forward(x, r, w, stream)
    d_x, d_w = backward(d_y, d_s, out["sum"], w, out["rstd"], stream)
    u = np_(out["sum"]).astype(np.float64) * np_(out["rstd"]).astype(np.float64)[:, None]
    terms = np_(d_y) * u
    assert (np.abs(np_(d_w) - terms.sum(axis=0)) <= (2.0 ** -18 + depth(rows) * 2.0 ** -24) * np.abs(terms).sum(axis=0)).all()
    alone, _ = backward(d_y, d_s, out["sum"], w, out["rstd"], stream, weight=False)
    again, w2 = backward(d_y, d_s, out["sum"], w, out["rstd"], stream)
    assert torch.equal(alone, d_x) and torch.equal(again, d_x) and torch.equal(w2, d_w)
    in_place = d_s.clone()
    shape = moe.make_norm_shape(rows, cols, TYPES[stream][1], EPS)
    w3, ws = torch.empty_like(w), torch.empty(moe.moe_norm_workspace_size(shape), dtype=torch.uint8, device="cuda")
    moe.moe_norm_backward(shape, d_y, in_place, out["sum"], w, out["rstd"], in_place, w3, ws)
    assert torch.equal(in_place, d_x) and torch.equal(w3, d_w)


def test_codes_are_the_quantisers():
    """fp32 y and codes of one call: the codes are those of the fp32 quotients; and with moe_quantize_act on values that
    bf16 holds (a weight of ones, rows whose rstd is a power of two)."""
    x, r, w, _, _ = inputs(64, 1024, "f32", 5)
    w[:128] = 0                                        # a run of zeros
    w[200] = 1e4                                       # one value that hides its run
    out = forward(x, r, w, "f32", codes=True)
    v = np_(out["y"]).reshape(64, 8, 128)              # (numpy divides; torch on the GPU multiplies by 1 / 448)
    amax = np.abs(v).max(axis=2)
    scale = np.where(amax > 0, amax / np.float32(448), np.float32(1))
    assert np.array_equal(np_(out["scales"]), scale)
    assert torch.equal(out["codes"].cpu().view(torch.uint8),
                       torch.from_numpy(v / scale[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(64, 1024))
    signs = torch.where(torch.rand(8, 2048, device="cuda") < 0.5, -4.0, 4.0).bfloat16()
    out = forward(signs, None, torch.linspace(0.5, 3, 2048, device="cuda").bfloat16().float(), "bf16", codes=True, eps=0.0)
    q, s = torch.empty_like(out["codes"]), torch.empty_like(out["scales"])
    moe.moe_quantize_act(8, 2048, out["y"], q, s)
    assert torch.equal(out["codes"].view(torch.uint8), q.view(torch.uint8)) and torch.equal(out["scales"], s)


@pytest.mark.parametrize("cols", [1024, 4096])
def test_outputs_that_are_left_out_change_nothing(cols):
    x, r, w, d_y, d_s = inputs(37, cols, "bf16", 6)
    full = forward(x, r, w, "bf16", codes=True)
    for kw in (dict(y=False), dict(codes=False), dict(total=False), dict(rstd=False)):
        part = forward(x, r, w, "bf16", **{**dict(codes=True), **kw})
        for k, v in part.items():
            assert v is None or torch.equal(v.view(torch.uint8), full[k].view(torch.uint8)), (kw, k)
    a, _ = backward(d_y, d_s, full["sum"], w, full["rstd"], "bf16")
    b, none = backward(d_y, d_s, full["sum"], w, full["rstd"], "bf16", weight=False)
    assert torch.equal(a, b) and none is None
    # an addition of its own and a call without a residual
    alone = forward(full["sum"], None, w, "bf16", codes=True)
    assert all(torch.equal(alone[k].view(torch.uint8), full[k].view(torch.uint8)) for k in ("y", "codes", "scales", "rstd"))


@pytest.mark.parametrize("cols", [520, 7168])
def test_a_rows_results_are_its_own(cols):
    x, r, w, d_y, d_s = inputs(203, cols, "bf16", 7)
    full = forward(x, r, w, "bf16")
    d, _ = backward(d_y, d_s, full["sum"], w, full["rstd"], "bf16")
    for at in (0, 1, 101, 202):
        one = forward(x[at:at + 1], r[at:at + 1], w, "bf16")
        assert all(torch.equal(one[k], full[k][at:at + 1]) for k in ("sum", "y", "rstd"))
        e, _ = backward(d_y[at:at + 1], d_s[at:at + 1], one["sum"], w, one["rstd"], "bf16")
        assert torch.equal(e, d[at:at + 1])


@pytest.mark.parametrize("cols,stream", [(2048, "bf16"), (1032, "f32"), (1408, "bf16")])
def test_many_rows_and_few_have_the_same_bits(cols, stream):
    """Rows of 1025 to 2048 values lie on one wavefront or on two."""
    x, r, w, _, _ = inputs(4097, cols, stream, 12)
    codes = cols % 128 == 0
    full = forward(x, r, w, stream, codes=codes)
    part = forward(x[1000:1300].contiguous(), r[1000:1300].contiguous(), w, stream, codes=codes)
    for k, v in part.items():
        assert v is None or torch.equal(v.view(torch.uint8), full[k][1000:1300].contiguous().view(torch.uint8)), k


def test_rows_that_are_zero_or_not_finite():
    x, _, w, d_y, _ = inputs(8, 1024, "bf16", 8)
    x[1] = 0
    x[2, 17] = float("nan")
    x[3, 500] = float("inf")
    x[4] = 1e-30                               # squares below fp32's range: eps alone
    x[5, 3] = 3e38                             # a square past it
    out = forward(x, None, w, "bf16", codes=True)
    y, rstd = out["y"].float(), out["rstd"]
    assert (y[1] == 0).all() and (out["scales"][1] == 1).all() and (np_(out["codes"])[1] == 0).all()
    assert torch.isnan(y[2]).all() and torch.isnan(rstd[2])
    assert rstd[3] == 0 and torch.isnan(y[3, 500]) and rstd[5] == 0
    assert torch.allclose(y[4], (1e-27 * w).bfloat16().float(), rtol=2.0 ** -6)
    ok = torch.tensor([0, 6, 7], device="cuda")
    clean = forward(x[ok].contiguous(), None, w, "bf16", codes=True)
    assert torch.equal(clean["y"], out["y"][ok]) and torch.equal(clean["scales"], out["scales"][ok])
    d, _ = backward(d_y, None, x, w, rstd, "bf16")
    assert torch.isfinite(d[ok].float()).all() and torch.isnan(d[2].float()).all()


@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [512, 2560])
def test_strides_and_sums_in_place(cols, stream):
    rows = 29
    x, r, w, d_y, d_s = inputs(rows, cols, stream, 9)
    ref = forward(x, r, w, stream, codes=True)
    d_ref, w_ref = backward(d_y, d_s, ref["sum"], w, ref["rstd"], stream)
    t, ty = TYPES[stream][0], TYPES[stream][1]
    x_ld, y_ld = cols + 24, cols + 64
    wide = lambda v, ld: torch.cat([v, torch.full((rows, ld - cols), 7.0, dtype=t, device="cuda")], 1)  # noqa: E731
    shape = moe.make_norm_shape(rows, cols, ty, EPS, x_ld, y_ld)
    for place in ("own", "x", "residual"):
        X, R, Y = wide(x, x_ld), wide(r, x_ld), torch.full((rows, y_ld), 7.0, dtype=t, device="cuda")
        H = {"own": torch.full((rows, x_ld), 7.0, dtype=t, device="cuda"), "x": X, "residual": R}[place]
        q, s, rs = torch.empty_like(ref["codes"]), torch.empty_like(ref["scales"]), torch.empty_like(ref["rstd"])
        moe.moe_norm_forward(shape, X, R, w, H, Y, q, s, rs)
        assert torch.equal(H[:, :cols], ref["sum"]) and torch.equal(Y[:, :cols], ref["y"]) and torch.equal(rs, ref["rstd"])
        assert torch.equal(q.view(torch.uint8), ref["codes"].view(torch.uint8)) and torch.equal(s, ref["scales"])
        assert (H[:, cols:] == 7).all() and (Y[:, cols:] == 7).all()
        DY, DS = wide(d_y, y_ld), wide(d_s, x_ld)
        D = DS if place == "x" else torch.full((rows, x_ld), 7.0, dtype=t, device="cuda")
        dw = torch.empty(cols, device="cuda")
        ws = torch.empty(moe.moe_norm_workspace_size(shape), dtype=torch.uint8, device="cuda")
        moe.moe_norm_backward(shape, DY, DS, H, w, rs, D, dw, ws)
        assert torch.equal(D[:, :cols], d_ref) and torch.equal(dw, w_ref) and (D[:, cols:] == 7).all()


def test_no_rows():
    w = torch.ones(256, device="cuda")
    shape = moe.make_norm_shape(0, 256, moe.MOE_DTYPE_BF16, EPS)
    moe.moe_norm_forward(shape, None, None, w)
    d_w = torch.full((256,), 3.0, device="cuda")
    moe.moe_norm_backward(shape, None, None, None, None, None, None, d_w)
    assert (d_w == 0).all()


def test_another_stream_and_a_graph():
    x, r, w, d_y, d_s = inputs(300, 2560, "bf16", 10)
    first = forward(x, r, w, "bf16", codes=True)
    d1, w1 = backward(d_y, d_s, first["sum"], w, first["rstd"], "bf16")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = forward(x, r, w, "bf16", codes=True, on=side)
        d2, w2 = backward(d_y, d_s, again["sum"], w, again["rstd"], "bf16", on=side)
    side.synchronize()
    assert same(first, again) and torch.equal(d1, d2) and torch.equal(w1, w2)
    shape = moe.make_norm_shape(300, 2560, moe.MOE_DTYPE_BF16, EPS)
    ws = torch.empty(moe.moe_norm_workspace_size(shape), dtype=torch.uint8, device="cuda")
    d3, w3 = torch.empty_like(d1), torch.empty_like(w1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_norm_forward(shape, x, r, w, again["sum"], again["y"], again["codes"], again["scales"], again["rstd"])
        moe.moe_norm_backward(shape, d_y, d_s, again["sum"], w, again["rstd"], d3, w3, ws)
    for k in range(4):
        x.copy_(torch.randn_like(x))
        want = forward(x, r, w, "bf16", codes=True)
        d1, w1 = backward(d_y, d_s, want["sum"], w, want["rstd"], "bf16")
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, again) and torch.equal(d1, d3) and torch.equal(w1, w3)


@pytest.mark.parametrize("rows,cols", [((1 << 20) + 3, 4096), ((1 << 23) + 5, 520)])
def test_offsets_past_32_bits(rows, cols):
    """2^32 elements and more: the last rows come out as they do alone."""
    block, r, w, d_y, _ = inputs(64, cols, "bf16", 11)
    x = block.repeat(rows // 64 + 1, 1)[:rows]
    codes = cols % 128 == 0
    out = forward(x, None, w, "bf16", codes=codes)
    tail = x[rows - 64:].contiguous()
    alone = forward(tail, None, w, "bf16", codes=codes)
    assert all(alone[k] is None or torch.equal(alone[k].view(torch.uint8), out[k][rows - 64:].contiguous().view(torch.uint8))
               for k in alone)
    del out["y"], out["codes"]
    d_big = d_y.repeat(rows // 64 + 1, 1)[:rows]
    d, d_w = backward(d_big, None, x, w, out["rstd"], "bf16")
    e, _ = backward(d_big[rows - 64:].contiguous(), None, tail, w, alone["rstd"], "bf16")
    assert torch.equal(d[rows - 64:], e)
    del d_big, d, x
    _, one = backward(d_y, None, block, w, forward(block, None, w, "bf16")["rstd"], "bf16")
    # the rows repeat: d_weight is near so many times that of the block
    size = (d_y.float() * block.float()).abs().sum(0) * (rows / 64)
    assert ((d_w - one * (rows / 64)).abs() <= 2.0 ** -8 * size).all()


@pytest.mark.parametrize("cols", [8, 2056])
def test_more_rows_than_a_launch_has_workgroups_for(cols):
    """2^32 threads and more at a row a wavefront; 2^21 workgroups and more at a row each."""
    rows = (1 << 26) + 7 if cols == 8 else (1 << 21) + 5
    block, _, w, _, _ = inputs(512, cols, "bf16", 13)
    x = block.repeat(rows // 512 + 1, 1)[:rows]
    out = forward(x, None, w, "bf16", rstd=False)["y"]
    want = forward(block, None, w, "bf16", rstd=False)["y"]
    whole = rows // 512 * 512
    assert torch.equal(out[:whole].view(-1, 512, cols), want.expand(rows // 512, 512, cols))
    assert torch.equal(out[whole:], want[:rows - whole])
