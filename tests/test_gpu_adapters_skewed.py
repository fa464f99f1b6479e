"""moe_adapters where a few of many resident adapters have most of the rows: a workgroup by adapters stands for 16 rows of one,
whichever has them.  Bounds: test_gpu_adapters.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from test_gpu_adapters import check, problem, run  # noqa: E402


def spread(rows, n, how, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    some = torch.randint(-1, n, (rows,), device="cuda", generator=g)
    at = torch.arange(rows, device="cuda")
    if how == "one":
        some[:] = n - 1
    if how == "most":
        some[torch.rand(rows, device="cuda", generator=g) < 0.85] = n // 2
    if how == "two":
        some = torch.where(at % 2 == 0, 0, n - 1)
    if how == "last":                                  # the others have a row each
        some = torch.where(at < n, at, n - 1)
    if how == "none but the last row":
        some[:] = -1
        some[-1] = n - 1
    return some.to(torch.int32)


@pytest.mark.parametrize("how", ["one", "most", "two", "last", "none but the last row"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d_in,d_out,n,r", [
    (17, 264, 136, 40, 16), (63, 2056, 72, 9, 32), (64, 136, 264, 64, 64), (65, 264, 72, 16, 8), (128, 520, 136, 11, 24),
    (255, 136, 72, 300, 128), (256, 264, 72, 16, 16), (257, 136, 136, 64, 48), (500, 264, 72, 1000, 16), (512, 72, 264, 17, 128),
    (1023, 264, 72, 64, 32), (1024, 136, 72, 1025, 64)])
def test_against_float64(rows, d_in, d_out, n, r, out, how):
    p = problem(rows, d_in, d_out, n, r, rows + n, out, ranks=True)
    p["which"] = spread(rows, n, how, rows)
    first = run(p)
    check(p, first)
    assert torch.equal(run(p), first)
    in_place = p["base"].clone()
    run({**p, "own": in_place}, base="own", into=in_place)
    assert torch.equal(in_place, first)


@pytest.mark.parametrize("rows", [40, 200, 700])
@pytest.mark.parametrize("r", [8, 32, 64, 128])
def test_adapters_that_are_counted_together(rows, r):
    """Above 1024 adapters, those a multiple of 1024 apart: a group of 16 rows has rows of several."""
    n = 3100
    p = problem(rows, 136, 72, 1, r, rows + r)
    g = torch.Generator("cuda").manual_seed(rows)
    p["a"] = (torch.randn(n, r, 136, device="cuda", generator=g) / 12).bfloat16()
    p["b"] = (torch.randn(n, 72, r, device="cuda", generator=g) / r ** 0.5).bfloat16()
    p["scale"] = 0.5 + torch.rand(n, device="cuda", generator=g)
    few = torch.tensor([5, 1029, 2053, 3077, 6, 1030, -1, 3099], device="cuda")
    p["which"] = few[torch.randint(0, 8, (rows,), device="cuda", generator=g)].to(torch.int32)
    out = run(p)
    check(p, out)
    assert torch.equal(run(p), out)


def test_another_stream_and_graphs_on_one_workspace():
    """Replays find the groups of what the rows' adapters are by then; two graphs in turn on one buffer."""
    shapes = [(300, 520, 264, 64, 16), (130, 264, 136, 20, 64), (900, 264, 72, 40, 128)]
    ps = [problem(*s, 5) for s in shapes]
    ws = torch.empty(max(moe.moe_adapters_workspace_size(moe.make_adapter_shape(*s, moe.MOE_DTYPE_BF16)) for s in shapes),
                     dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(p["base"]) for p in ps], []
    for p, o, s in zip(ps, outs, shapes):
        run(p)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            moe.moe_adapters(moe.make_adapter_shape(*s, moe.MOE_DTYPE_BF16), p["x"], p["which"], p["a"], p["b"], p["scale"], None,
                             p["base"], o, ws)
    for k in range(8):
        i = k % 3
        rows, n = shapes[i][0], shapes[i][3]
        ps[i]["which"].copy_(spread(rows, n, ("one", "most", "last", "two")[k % 4], k))
        want = run(ps[i])
        ws.fill_(255)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = run(ps[0], on=side)
    side.synchronize()
    assert torch.equal(again, run(ps[0]))


@pytest.mark.parametrize("rows,n,r", [(1000, 256, 16), (500, 64, 64)])
def test_a_prompt_on_one_of_many_adapters_takes_no_longer(rows, n, r):
    """All rows on one adapter against rows of all of them: less is read.  (Workgroups that stood for an adapter and all of its
    rows took 34 times as long.)  Three times as long is allowed."""
    p = problem(rows, 2048, 1024, n, r, 9)
    ws = torch.empty(moe.moe_adapters_workspace_size(moe.make_adapter_shape(rows, 2048, 1024, n, r, moe.MOE_DTYPE_BF16)),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(p["base"])

    def time_of(which):
        p["which"].copy_(which)
        run(p, into=out, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(10):
                run(p, into=out, ws=ws)
        best = []
        for _ in range(7):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        return min(best)

    even = time_of(torch.arange(rows, device="cuda").to(torch.int32) % n)
    one = time_of(torch.full((rows,), 7, dtype=torch.int32, device="cuda"))
    assert one < 3 * even
