"""What test_gpu_adapters.py asks of a few shapes, in each of moe_adapters' forms: one kernel (few rows and little of A; no
workspace), by adapters, and by tiles of neighbouring rows (above 1024 rows, or above 32 rows of the only adapter), the form
whose rows meet other rows' adapters."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from test_gpu_adapters import DT, check, problem, run  # noqa: E402
from test_gpu_adapters_edges import FEW, FORMS, TILES  # noqa: E402

ONE_ADAPTER = [(100, 264, 72, 1, 24), (45, 520, 136, 1, 64), (70, 136, 264, 1, 128)]     # (by tiles)
SHAPES = FORMS + ONE_ADAPTER
OUT = [torch.bfloat16, torch.float32]


def shape_of(p, kind=torch.bfloat16, **ld):
    rows, d_in = p["x"].shape
    n, r = p["a"].shape[:2]
    return moe.make_adapter_shape(rows, d_in, p["b"].shape[1], n, r, DT[kind], **ld)


@pytest.mark.parametrize("rows,d_in,d_out,n,r", SHAPES)
def test_one_kernel_takes_no_workspace(rows, d_in, d_out, n, r):
    need = moe.moe_adapters_workspace_size(moe.make_adapter_shape(rows, d_in, d_out, n, r, moe.MOE_DTYPE_BF16))
    assert (need == 0) == ((rows, d_in, d_out, n, r) in FEW)


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("rows,d_in,d_out,n,r", SHAPES)
def test_a_rows_result_is_its_own(rows, d_in, d_out, n, r, out):
    """An infinity or NaN in a row, in an adapter, or behind an adapter's rank does not reach a row that does not use it: the
    same bits as without."""
    p = problem(rows, d_in, d_out, n, r, rows + r, out)
    at = torch.arange(rows, device="cuda")
    p["which"][:] = (at % (n + 1)) - 1                 # (neighbours differ)
    ranks = torch.tensor([r, r // 2, 0, 1, r - 1, r], dtype=torch.int32, device="cuda")
    p["ranks"] = ranks[torch.arange(n, device="cuda") % 6].contiguous()
    clean = run(p)
    check(p, clean)
    for e in range(n):
        k = int(p["ranks"][e])
        p["a"][e, k:] = float("nan")                   # behind the rank
        p["b"][e, :, k:] = float("inf")
    assert torch.equal(run(p), clean)
    bad_rows = torch.tensor([1, rows // 2, rows - 1], device="cuda")
    p["x"][bad_rows[0]] = float("inf")
    p["x"][bad_rows[1], d_in - 1] = float("nan")
    p["x"][bad_rows[2], 0] = -float("inf")
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[bad_rows] = True
    if n > 1:
        p["a"][n - 1] = float("nan")
        p["b"][n - 1] = float("inf")
        bad |= p["which"] == n - 1
    got = run(p)
    assert torch.equal(got[~bad], clean[~bad])
    none = p["which"] < 0                               # a bad row without an adapter keeps its base all the same
    assert torch.equal(got[none], p["base"][none])
    used = bad & (p["which"] >= 0) & (p["ranks"][p["which"].clamp(min=0).long()] > 0)
    if n > 1:
        used &= p["which"] != n - 1
    assert not torch.isfinite(got[used].float()).all(dim=1).any()


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("rows,d_in,d_out,n,r", SHAPES)
def test_strides_and_in_place(rows, d_in, d_out, n, r, out):
    p = problem(rows, d_in, d_out, n, r, rows + d_in, out)
    ref = run(p)
    check(p, ref)
    in_place = p["base"].clone()
    run({**p, "own": in_place}, base="own", into=in_place)
    assert torch.equal(in_place, ref)
    wide = lambda v, more: torch.cat([v, torch.full((rows, more), 7.0, dtype=v.dtype, device="cuda")], 1)  # noqa: E731
    shape = shape_of(p, out, x_ld=d_in + 40, base_ld=d_out + 24, out_ld=d_out + 8)
    ws = torch.full((max(16, moe.moe_adapters_workspace_size(shape)),), 255, dtype=torch.uint8, device="cuda")
    o = torch.full((rows, d_out + 8), 7.0, dtype=out, device="cuda")
    moe.moe_adapters(shape, wide(p["x"], 40), p["which"], p["a"], p["b"], p["scale"], None, wide(p["base"], 24), o, ws)
    assert torch.equal(o[:, :d_out], ref) and (o[:, d_out:] == 7).all()


@pytest.mark.parametrize("rows,d_in,d_out,n,r", SHAPES)
def test_another_stream_and_a_graph(rows, d_in, d_out, n, r):
    p = problem(rows, d_in, d_out, n, r, rows + d_out)
    first = run(p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = run(p, on=side)
    side.synchronize()
    assert torch.equal(first, again)
    shape = shape_of(p)
    ws = torch.empty(max(16, moe.moe_adapters_workspace_size(shape)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adapters(shape, p["x"], p["which"], p["a"], p["b"], p["scale"], None, p["base"], again, ws)
    for k in range(3):
        p["x"].copy_(torch.randn_like(p["x"]))
        p["which"].copy_(torch.randint(-1, n, (rows,), device="cuda"))
        want = run(p)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, again)


@pytest.mark.parametrize("rows,d_in,d_out,n,r", FEW + TILES)
def test_a_row_keeps_its_bits_whatever_its_neighbours_have(rows, d_in, d_out, n, r):
    """The same place in the batch, the other rows without adapters.  (By adapters, the order of the slices' sums goes by the rows
    that a group has.)"""
    p = problem(rows, d_in, d_out, n, r, rows)
    p["which"][:] = torch.arange(rows, device="cuda") % n
    a = run(p)
    keep = torch.arange(rows, device="cuda") % 7 == 0
    p["which"] = torch.where(keep, p["which"], -1).to(torch.int32)
    b = run(p)
    assert torch.equal(a[keep], b[keep]) and torch.equal(b[~keep], p["base"][~keep])
