"""moe_adapters on the GPU against float64.

The products' fp32 sums have `in` and parts * r terms: at most (in + 3 r + 16) 2^-24 of the sum of magnitudes (additions
one after another).  Under a bf16 output the low-rank values keep two bf16 parts, each half a step (2^-8) off: 2^-16; under fp32
three: 2^-24.  The output's own rounding: 2^-8 or 2^-24 of it."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from oracle import block as B  # noqa: E402

DT = {torch.float32: moe.MOE_DTYPE_F32, torch.bfloat16: moe.MOE_DTYPE_BF16}


def np_(t):
    return t.float().cpu().numpy()


def problem(rows, d_in, d_out, n, r, seed, out=torch.bfloat16, order="mixed", ranks=False):
    g = torch.Generator("cuda").manual_seed(seed)
    some = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    p = {"x": some(rows, d_in).bfloat16(), "a": (some(n, r, d_in) / d_in ** 0.5).bfloat16(),
         "b": (some(n, d_out, r) / r ** 0.5).bfloat16(), "scale": 0.5 + torch.rand(n, device="cuda", generator=g),
         "base": some(rows, d_out).to(out),
         "ranks": torch.randint(0, r + 1, (n,), device="cuda", generator=g).to(torch.int32) if ranks else None}
    which = torch.randint(-1, n, (rows,), device="cuda", generator=g)
    if order == "prompts":
        which = torch.sort(which).values
    p["which"] = which.to(torch.int32)
    return p


def run(p, base="base", into=None, on=None, ws=None, **ld):
    rows, d_in = p["x"].shape
    n, r = p["a"].shape[:2]
    d_out = p["b"].shape[1]
    kind = p["base"].dtype
    shape = moe.make_adapter_shape(rows, d_in, d_out, n, r, DT[kind], **ld)
    out = torch.full((rows, d_out), float("nan"), dtype=kind, device="cuda") if into is None else into
    if ws is None:
        ws = torch.full((max(16, moe.moe_adapters_workspace_size(shape)),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_adapters(shape, p["x"], p["which"], p["a"], p["b"], p["scale"], p["ranks"], p[base] if base else None, out, ws, on)
    return out


def check(p, out, base=True):
    ref, size = B.adapters(np_(p["x"]), p["which"].cpu().numpy(), np_(p["a"]), np_(p["b"]), np_(p["scale"]),
                           None if p["ranks"] is None else p["ranks"].cpu().numpy(),
                           np_(p["base"]) if base else np.zeros(p["base"].shape))
    d_in, r = p["x"].shape[1], p["a"].shape[1]
    half, kept = (2.0 ** -8, 2.0 ** -16) if p["base"].dtype == torch.bfloat16 else (2.0 ** -24, 2.0 ** -24)
    tol = half * np.abs(ref) + ((d_in + 3 * r + 16) * 2.0 ** -24 + kept) * size + 2.0 ** -22 * np.abs(ref) + 1e-37
    assert (np.abs(np_(out) - ref) <= tol).all()
    none = ((p["which"] < 0) | (p["which"] >= p["a"].shape[0]))
    if base:
        assert torch.equal(out[none], p["base"][none])


@pytest.mark.parametrize("order", ["mixed", "prompts"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d_in,d_out,n,r,ranks", [
    (1, 8, 8, 1, 8, False), (1, 7168, 4096, 3, 16, False), (2, 136, 264, 2, 24, True), (15, 256, 72, 5, 8, True),
    (16, 1408, 2048, 20, 64, True), (17, 520, 1000, 3, 128, True), (64, 2048, 512, 32, 32, False), (33, 40, 56, 7, 48, False),
    (300, 392, 328, 4, 96, True), (1000, 264, 200, 9, 16, True)])
def test_against_float64(rows, d_in, d_out, n, r, ranks, out, order):
    p = problem(rows, d_in, d_out, n, r, rows + d_in + r, out, order, ranks)
    if rows > 1:
        p["which"][rows // 2] = n + 3                # no such adapter: none
        p["which"][0] = 0
    check(p, run(p))
    check(p, run(p, base=None), base=False)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d_in,d_out,n,r,ranks", [
    (16, 2048, 640, 6, 32, True), (16, 2056, 136, 2, 32, False), (17, 264, 520, 2, 16, True), (100, 1032, 328, 2, 16, False),
    (128, 520, 256, 40, 32, True), (128, 264, 72, 1, 64, False), (129, 264, 72, 1, 64, False), (140, 328, 136, 5, 32, True),
    (200, 456, 72, 3, 64, True), (257, 72, 8, 60, 8, False), (300, 8, 328, 3, 128, True)])
def test_rows_by_adapter_and_by_tile(rows, d_in, d_out, n, r, ranks, out):
    """Few rows and little of A (one kernel), workgroups by adapter (more than 16 rows of one), tiles."""
    for order in ("mixed", "prompts"):
        p = problem(rows, d_in, d_out, n, r, rows + d_out, out, order, ranks)
        check(p, run(p))


@pytest.mark.parametrize("rows,r,out", [(128, 16, torch.bfloat16), (100, 64, torch.float32), (97, 128, torch.bfloat16),
                                        (66, 32, torch.float32)])
def test_many_rows_of_one_adapter_among_many(rows, r, out):
    """Workgroups by adapter: one of them with more rows than a tile, and rows without an adapter likewise."""
    p = problem(rows, 1096, 264, 40, r, rows + r, out)
    pick = torch.rand(rows, device="cuda")
    p["which"] = torch.where(pick < 0.4, 7, torch.where(pick < 0.7, -1, p["which"])).to(torch.int32)
    check(p, run(p))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d_in,d_out,n,r,ranks", [
    (1024, 520, 136, 64, 16, False), (1023, 264, 328, 100, 32, True), (1025, 264, 72, 100, 32, False),
    (500, 1032, 520, 32, 64, True), (513, 264, 72, 32, 24, False), (700, 136, 264, 1200, 8, False),
    (1024, 72, 72, 1025, 24, True), (320, 264, 1096, 40, 128, True), (257, 2056, 264, 16, 16, False),
    (128, 40, 2056, 8, 48, True), (256, 264, 520, 8, 64, True), (257, 264, 520, 8, 64, False),
    (600, 328, 264, 20, 128, True)])
def test_decode_batches(rows, d_in, d_out, n, r, ranks, out):
    """Up to 1024 rows and 16 an adapter (32 above rank 32) go by adapters: one, two and four workgroups that share an adapter's rows, fewer
    rows than adapters, one adapter with most rows; rows without one copied, or left where they are."""
    p = problem(rows, d_in, d_out, n, r, rows + d_in + n, out, ranks=ranks)
    for k in range(3):
        if k == 1:
            p["which"] = torch.sort(p["which"]).values.flip(0).contiguous()
        if k == 2:
            pick = torch.rand(rows, device="cuda")
            p["which"] = torch.where(pick < 0.6, n - 1, torch.where(pick < 0.8, n + 5, p["which"])).to(torch.int32)
        first = run(p)
        check(p, first)
        in_place = p["base"].clone()
        run({**p, "own": in_place}, base="own", into=in_place)
        assert torch.equal(in_place, first)
    p["which"][:] = -9
    assert torch.equal(run(p), p["base"])
    check(p, run(p, base=None), base=False)


@pytest.mark.parametrize("rows", [511, 600])
def test_rows_far_apart(rows):
    """x beyond 2^32 elements: by adapters up to there, by tiles past it."""
    p = problem(rows, 264, 136, 64, 16, rows)
    first = run(p)
    far = torch.empty((rows - 1 << 23) + 264, dtype=torch.bfloat16, device="cuda").as_strided((rows, 264), (1 << 23, 1))
    far.copy_(p["x"])
    p["x"] = far
    out = run(p, x_ld=1 << 23)
    check({**p, "x": far.contiguous()}, out)
    if rows == 511:
        assert torch.equal(out, first)


def test_large_and_long():
    p = problem(5000, 512, 640, 6, 16, 1, order="prompts")
    out = run(p)
    rows = torch.randperm(5000, device="cuda")[:200]
    q = {**p, "x": p["x"][rows], "which": p["which"][rows], "base": p["base"][rows]}
    check(q, out[rows])


def test_a_rows_result_is_its_own():
    """Another row's, adapter's or unused rank's infinity and NaN do not reach it, nor its neighbours' adapters."""
    p = problem(40, 264, 520, 6, 24, 2, ranks=True)
    p["ranks"][:] = torch.tensor([24, 5, 8, 0, 13, 24], dtype=torch.int32)
    p["which"][:] = torch.arange(40, device="cuda") % 6
    clean = run(p)
    for e in range(6):
        k = int(p["ranks"][e])
        p["a"][e, k:] = float("nan")                 # behind the rank
        p["b"][e, :, k:] = float("inf")
    assert torch.equal(run(p), clean)
    p["a"][5] = float("nan")                         # an adapter, and two rows
    p["x"][2] = float("inf")
    p["x"][9, 7] = float("nan")
    out = run(p)
    other = (p["which"] != 5) & (torch.arange(40, device="cuda") != 2)
    bad = (p["which"] == 5)
    assert torch.isnan(out[bad].float()).all()
    assert not torch.isfinite(out[2].float()).any()
    other &= torch.arange(40, device="cuda") != 9    # (row 9 has adapter 3, of rank 0)
    assert torch.equal(out[other], clean[other])


def test_infinite_sums_stay_infinite():
    p = problem(3, 16, 16, 1, 8, 3, out=torch.float32)
    p["which"][:] = 0
    p["x"][:] = 1e30
    p["a"][:] = 1e30                                  # the sums pass fp32's range
    p["b"][:] = 1.0
    assert torch.isposinf(run(p)).all()


def test_gradual_sizes_of_the_low_rank_values():
    """Low-rank values far apart in size: each keeps its own bits."""
    p = problem(32, 64, 64, 1, 16, 4, out=torch.float32)
    p["which"][:] = 0
    p["a"] *= (10.0 ** torch.linspace(-12, 6, 16, device="cuda")).bfloat16()[None, :, None]
    check(p, run(p, base=None), base=False)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_strides_and_in_place(out):
    p = problem(45, 256, 328, 4, 32, 5, out)
    ref = run(p)
    in_place = p["base"].clone()
    run({**p, "own": in_place}, base="own", into=in_place)
    assert torch.equal(in_place, ref)
    wide = lambda v, more: torch.cat([v, torch.full((45, more), 7.0, dtype=v.dtype, device="cuda")], 1)  # noqa: E731
    X, O = wide(p["x"], 40), torch.full((45, 336), 7.0, dtype=out, device="cuda")
    P2 = {**p, "wide": wide(p["base"], 24)}
    shape = moe.make_adapter_shape(45, 256, 328, 4, 32, DT[out], 296, 352, 336)
    ws = torch.empty(moe.moe_adapters_workspace_size(shape), dtype=torch.uint8, device="cuda")
    moe.moe_adapters(shape, X, p["which"], p["a"], p["b"], p["scale"], None, P2["wide"], O, ws)
    assert torch.equal(O[:, :328], ref) and (O[:, 328:] == 7).all()


def test_rows_in_another_batch_keep_their_bits_when_split_alike():
    """Rows side by side with others: the same tile of rows, other adapters around it."""
    p = problem(16, 264, 256, 8, 16, 6)
    p["which"][:] = torch.arange(16, device="cuda") % 8
    a = run(p)
    p["which"][1:] = -1
    b = run(p)
    assert torch.equal(a[0], b[0]) and torch.equal(b[1:], p["base"][1:])


def test_no_rows_another_stream_and_a_graph():
    shape = moe.make_adapter_shape(0, 64, 64, 2, 16, moe.MOE_DTYPE_BF16)
    moe.moe_adapters(shape, *[None] * 9)
    p = problem(70, 1024, 768, 5, 16, 7)
    first = run(p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = run(p, on=side)
    side.synchronize()
    assert torch.equal(first, again)
    shape = moe.make_adapter_shape(70, 1024, 768, 5, 16, moe.MOE_DTYPE_BF16)
    ws = torch.empty(moe.moe_adapters_workspace_size(shape), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adapters(shape, p["x"], p["which"], p["a"], p["b"], p["scale"], None, p["base"], again, ws)
    for k in range(4):
        p["x"].copy_(torch.randn_like(p["x"]))
        p["which"].copy_(torch.randint(-1, 5, (70,), device="cuda"))
        want = run(p)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, again)


@pytest.mark.parametrize("wide", ["x", "out"])
def test_offsets_past_32_bits(wide):
    rows, d_in, d_out = ((1 << 19) + 21, 8200, 64) if wide == "x" else ((1 << 19) + 21, 64, 8200)
    p = problem(64, d_in, d_out, 3, 16, 8)
    reps = rows // 64 + 1
    big = {**p, **{k: p[k].repeat(reps, *[1] * (p[k].ndim - 1))[:rows] for k in ("x", "which")}}
    big["base"] = torch.empty(rows, d_out, dtype=torch.bfloat16, device="cuda")
    out = run(big, base=None)
    tail = {**p, "x": big["x"][rows - 37:].contiguous(), "which": big["which"][rows - 37:].contiguous(),
            "base": big["base"][rows - 37:].contiguous()}
    check(tail, out[rows - 37:], base=False)
    assert torch.equal(out[:64], out[64:128])
