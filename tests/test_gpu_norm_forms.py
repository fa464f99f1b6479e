"""The norm's backward pass where its weight gradient goes through the workspace (more than 384 rows, or 8 MB of them): strides,
graphs, streams, workspaces with old values.  Rows of a wavefront (up to 2048 values) and of a workgroup."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from test_gpu_block import TrainBlock, train_inputs  # noqa: E402
from test_gpu_norm import EPS, TYPES, backward, forward, inputs, same  # noqa: E402

SHAPES = [(385, 8, "bf16"), (401, 520, "bf16"), (1021, 1408, "f32"), (390, 2048, "f32"), (500, 2560, "bf16"), (641, 7168, "f32"),
          (300, 7168, "f32"), (130, 32768, "bf16")]


def shape_of(rows, cols, stream, *ld):
    shape = moe.make_norm_shape(rows, cols, TYPES[stream][1], EPS, *ld)
    assert moe.moe_norm_workspace_size(shape) > 0
    return shape


def space(shape, fill=255):
    return torch.full((moe.moe_norm_workspace_size(shape),), fill, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("rows,cols,stream", SHAPES)
def test_strides_and_old_values_in_the_workspace(rows, cols, stream):
    x, r, w, d_y, d_s = inputs(rows, cols, stream, rows + cols)
    ref = forward(x, r, w, stream)
    d_ref, w_ref = backward(d_y, d_s, ref["sum"], w, ref["rstd"], stream)
    t = TYPES[stream][0]
    shape = shape_of(rows, cols, stream, cols + 24, cols + 64)
    wide = lambda v, more: torch.cat([v, torch.full((rows, more), 7.0, dtype=t, device="cuda")], 1)  # noqa: E731
    for place in ("own", "d_sum"):
        for fill in (0, 255):
            d_sum = wide(d_s, 24)
            d_x = d_sum if place == "d_sum" else torch.full((rows, cols + 24), 7.0, dtype=t, device="cuda")
            d_w = torch.full((cols,), float("nan"), device="cuda")
            moe.moe_norm_backward(shape, wide(d_y, 64), d_sum, wide(ref["sum"], 24), w, ref["rstd"], d_x, d_w, space(shape, fill))
            assert torch.equal(d_x[:, :cols], d_ref) and torch.equal(d_w, w_ref) and (d_x[:, cols:] == 7).all()


@pytest.mark.parametrize("rows,cols,stream", SHAPES)
def test_another_stream_and_a_graph(rows, cols, stream):
    x, r, w, d_y, d_s = inputs(rows, cols, stream, 10)
    first = forward(x, r, w, stream)
    d1, w1 = backward(d_y, d_s, first["sum"], w, first["rstd"], stream)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = forward(x, r, w, stream, on=side)
        d2, w2 = backward(d_y, d_s, again["sum"], w, again["rstd"], stream, on=side)
    side.synchronize()
    assert same(first, again) and torch.equal(d1, d2) and torch.equal(w1, w2)
    shape = shape_of(rows, cols, stream)
    ws, d3, w3 = space(shape), torch.empty_like(d1), torch.empty_like(w1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_norm_forward(shape, x, r, w, again["sum"], again["y"], None, None, again["rstd"])
        moe.moe_norm_backward(shape, d_y, d_s, again["sum"], w, again["rstd"], d3, w3, ws)
    for _ in range(4):
        x.copy_(torch.randn_like(x))
        want = forward(x, r, w, stream)
        d1, w1 = backward(d_y, d_s, want["sum"], w, want["rstd"], stream)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, again) and torch.equal(d1, d3) and torch.equal(w1, w3)


def test_two_graphs_that_share_a_workspace():
    """Captured one after the other on one buffer and replayed in turn on one stream; the buffer is the larger one's."""
    calls, ws = [], None
    for rows, cols, stream in ((1021, 1408, "f32"), (500, 2560, "bf16")):
        x, r, w, d_y, d_s = inputs(rows, cols, stream, rows)
        f = forward(x, r, w, stream)
        shape = shape_of(rows, cols, stream)
        ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda") if ws is None else ws
        assert moe.moe_norm_workspace_size(shape) <= ws.numel()
        want = backward(d_y, d_s, f["sum"], w, f["rstd"], stream)
        got = torch.empty_like(want[0]), torch.empty_like(want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_norm_backward(shape, d_y, d_s, f["sum"], w, f["rstd"], *got, ws)
        calls.append((graph, want, got, (d_y, d_s, f, w)))         # (the graph reads them: they have to live)
    for _ in range(3):
        for graph, _, got, _ in calls:
            for t in got:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for _, want, got, _ in calls for a, b in zip(want, got))


def test_two_training_steps_on_two_streams():
    """Whole steps of more than 384 rows, each with its own workspaces: the results of each alone, bit for bit."""
    blks = [TrainBlock(700, 256, 16, 4, 128, [0, 64, 700], 3), TrainBlock(450, 512, 24, 3, 128, [0, 450], 4)]
    assert all(moe.moe_norm_workspace_size(b.norm) > 0 for b in blks)
    data = [train_inputs(b.T, b.d, len(b.starts) - 1, 5 + i) for i, b in enumerate(blks)]
    alone = []
    for b, (fwd, bwd) in zip(blks, data):
        b.forward(*fwd)
        b.backward(*bwd)
        alone.append(b.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blks]
    for _ in range(5):
        for b, (fwd, bwd), s in zip(blks, data, streams):
            with torch.cuda.stream(s):
                b.ws2.fill_(255)
                b.forward(*fwd)
                b.backward(*bwd)
    torch.cuda.synchronize()
    for b, want in zip(blks, alone):
        assert all(torch.equal(x, y) for x, y in zip(b.results(), want))
