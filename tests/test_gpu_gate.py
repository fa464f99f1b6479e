"""moe_gate and moe_gate_backward on the GPU against the float64 statement.

Tolerances.  A gate is a quotient of sums of at most 512 values of expf (2 units in the last place each), summed in at
most 14 steps, of arguments whose rounding moves exp by 2^-25 |l - max|: with logits of size 12 at most, below
40 * 2^-24 = 2.4e-6 relative; 5e-6 is asked.  A gradient is a difference of such products times d_gate: 1e-5 of the
row's largest |d_gate| (times scale); rounding to bf16 adds 2^-8 of the value.  A row that was
decided by less than 4e-6 of its largest key (fp32 ranks it either way) may have other picks."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from oracle import operators as P  # noqa: E402

INF = float("inf")


def make(T, N, K, softmax, G=1, TG=1, top2=False, renorm=True, bias=False, bf16=False, scale=1.0, ld=0):
    return moe.make_gate_config(T, N, K, moe.MOE_DTYPE_BF16 if bf16 else moe.MOE_DTYPE_F32,
                                moe.MOE_SCORE_SOFTMAX if softmax else moe.MOE_SCORE_SIGMOID, G, TG,
                                moe.MOE_GROUP_TOP2 if top2 else moe.MOE_GROUP_MAX, renorm, scale, ld)


def run(cfg, logits, bias, load=True, stream=None):
    T, K, N = cfg.tokens, cfg.top_k, cfg.n_routed
    idx = torch.full((T, K), -77, dtype=torch.int32, device="cuda")
    gate = torch.full((T, K), float("nan"), device="cuda")
    cnt = torch.full((N,), -77, dtype=torch.int32, device="cuda") if load else None
    ws = torch.full((max(1, moe.moe_gate_workspace_size(cfg)),), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_gate(cfg, logits, bias, idx, gate, cnt, ws, stream)
    return idx, gate, cnt


def check(cfg, logits, bias, softmax, G, TG, top2, renorm, scale):
    idx, gate, load = run(cfg, logits, bias)
    torch.cuda.synchronize()
    l = logits.float().cpu().numpy()
    b = None if bias is None else bias.cpu().numpy()
    want, g, cnt, gap = P.gate(l, b, cfg.top_k, softmax, G, TG, top2, renorm, scale)
    got = idx.cpu().numpy()
    keys = P.gate_scores(l, softmax) + (0 if b is None else np.where(np.isneginf(b), 0, b))
    clear = gap > 4e-6 * np.abs(keys).max(axis=1)
    assert np.array_equal(got[clear], want[clear])
    assert clear.mean() > 0.8 or cfg.tokens < 8
    gates = P.gate_values(P.gate_scores(l, softmax), got, renorm, scale)
    assert (np.abs(gate.cpu().numpy() - gates) <= 5e-6 * np.abs(gates)).all()
    assert (gate.cpu().numpy()[got < 0] == 0).all()
    assert np.array_equal(load.cpu().numpy(), np.bincount(got[got >= 0], minlength=cfg.n_routed))
    # the gradient of these picks
    dg = torch.randn(cfg.tokens, cfg.top_k, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    d = torch.full((cfg.tokens, cfg.n_routed), float("nan"), dtype=logits.dtype, device="cuda")
    moe.moe_gate_backward(cfg, logits, idx, dg, d)
    torch.cuda.synchronize()
    ref = P.gate_backward(l, got, dg.cpu().numpy(), softmax, renorm, scale)
    tol = 1e-5 * scale * np.abs(dg.cpu().numpy()).max(axis=1, keepdims=True)
    if logits.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(d.float().cpu().numpy() - ref) <= tol).all()


CASES = [  # T, N, K, softmax, G, TG, top2, renorm, bias, bf16, scale
    (1, 1, 1, False, 1, 1, False, True, False, False, 1.0),
    (1, 256, 8, False, 8, 4, True, True, True, False, 2.5),
    (3, 8, 8, True, 1, 1, False, True, False, False, 1.0),
    (17, 60, 4, True, 1, 1, False, False, False, True, 1.0),
    (16, 63, 5, False, 9, 2, False, True, True, False, 1.0),
    (100, 64, 6, True, 1, 1, False, True, True, False, 1.0),
    (257, 65, 32, False, 1, 1, False, False, True, True, 0.5),
    (130, 192, 7, True, 64, 3, True, True, True, False, 1.0),
    (515, 128, 2, False, 2, 1, True, True, False, True, 1.0),
    (200, 512, 32, True, 16, 5, False, False, True, False, 16.0),
    (90, 511, 31, False, 7, 3, True, True, True, False, 1.0),
    (64, 300, 3, True, 300 // 5, 1, True, True, False, False, 1.0),
    (1100, 16, 4, False, 16, 9, True, True, True, False, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(int(v)) for v in c))
def test_against_float64(case):
    T, N, K, softmax, G, TG, top2, renorm, bias, bf16, scale = case
    g = torch.Generator("cuda").manual_seed(T * 1000 + N)
    logits = (1.5 * torch.randn(T, N, device="cuda", generator=g)).clamp(-6, 6)
    logits = logits.bfloat16() if bf16 else logits
    b = (0.1 if not softmax else 0.3 / N) * torch.randn(N, device="cuda", generator=g) if bias else None
    check(make(T, N, K, softmax, G, TG, top2, renorm, bias, bf16, scale), logits, b, softmax, G, TG, top2, renorm, scale)


@pytest.mark.parametrize("K", [5, 16, 17, 30])
@pytest.mark.parametrize("N,G", [(16, 1), (30, 1), (64, 1), (117, 1), (256, 1), (500, 1), (63, 9), (120, 5), (252, 9), (511, 7)])
def test_every_layout_of_a_token_on_lanes(N, G, K):
    """Experts a lane and lanes a token, groups of whole lanes and others, both types and both scores."""
    if K > N // G * max(1, G // 2):
        K = N // G * max(1, G // 2)
    for softmax in (False, True):
        for renorm in (False, True):
            for bf16 in (False, True):
                g = torch.Generator("cuda").manual_seed(N + K)
                logits = (1.5 * torch.randn(40, N, device="cuda", generator=g)).clamp(-6, 6)
                logits = logits.bfloat16() if bf16 else logits
                b = (0.3 / N if softmax else 0.1) * torch.randn(N, device="cuda", generator=g)
                args = softmax, G, max(1, G // 2), True, renorm
                check(make(40, N, K, *args, True, bf16, 1.0), logits, b, *args, 1.0)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_experts_and_empty_rows(softmax, renorm):
    T, N, K = 40, 48, 6
    g = torch.Generator("cuda").manual_seed(3)
    logits = torch.randn(T, N, device="cuda", generator=g)
    logits[torch.rand(T, N, device="cuda", generator=g) < 0.7] = -INF
    logits[7] = -INF                                  # a padding row
    logits[8] = -INF
    logits[8, 47] = 0.25                              # one expert left
    logits[9, :] = torch.finfo(torch.float32).min     # the lowest value is a number, not a mask
    bias = torch.zeros(N, device="cuda")
    bias[5] = -INF                                    # an expert out of service
    check(make(T, N, K, softmax, 4, 2, True, renorm), logits, bias, softmax, 4, 2, True, renorm, 1.0)
    idx, gate, _ = run(make(T, N, K, softmax, 4, 2, True, renorm), logits, bias)
    assert (idx[7] == -1).all() and (gate[7] == 0).all() and idx[8].tolist() == [47] + [-1] * 5
    assert (idx != 5).all() and (idx[9] >= 0).all()


@pytest.mark.parametrize("softmax", [False, True])
def test_equal_scores_go_to_the_lower_index(softmax):
    T, N, K = 5, 200, 9
    logits = torch.zeros(T, N, device="cuda")
    logits[1, 100:] = 1.0
    logits[2, ::3] = 2.0
    logits[3] = -0.0
    logits[4, 190:] = 30.0    # a sigmoid of 30 rounds to 1, as one of 40 does: equal in fp32
    logits[4, 180:190] = 40.0 if not softmax else 30.0
    idx, _, _ = run(make(T, N, K, softmax), logits, None)
    assert idx[0].tolist() == list(range(9)) and idx[1].tolist() == list(range(100, 109))
    assert idx[2].tolist() == list(range(0, 27, 3)) and idx[3].tolist() == list(range(9))
    assert idx[4].tolist() == list(range(180, 189))


def test_nan_ranks_last_and_infinity_first():
    N, K = 70, 3
    logits = torch.linspace(-1, 1, N, device="cuda").repeat(3, 1)
    logits[0, 69] = float("nan")
    logits[1, 0] = INF
    logits[2] = -INF
    logits[2, 10], logits[2, 20] = float("nan"), 0.5
    idx, gate, _ = run(make(3, N, K, False, renorm=False), logits, None)
    assert idx[0].tolist() == [68, 67, 66] and idx[1].tolist() == [0, 69, 68] and gate[1, 0].item() == 1.0
    assert idx[2].tolist() == [20, 10, -1]
    assert torch.isnan(gate[2, 1]) and gate[2, 2].item() == 0 and not torch.isnan(gate[2, 0])
    # a softmax over a NaN has no number left: its gates say so
    _, gate, _ = run(make(3, N, K, True), logits, None)
    assert torch.isnan(gate[0]).all() and torch.isnan(gate[1]).all()


def test_rows_apart_and_no_load():
    T, N, K = 37, 50, 4
    wide = torch.randn(T, 77, device="cuda")
    logits = wide[:, 3:53]
    cfg = make(T, N, K, True, ld=77)
    idx, gate, _ = run(cfg, logits, None, load=False)
    idx2, gate2, _ = run(make(T, N, K, True), logits.contiguous(), None)
    assert torch.equal(idx, idx2) and torch.equal(gate, gate2)
    dg = torch.randn(T, K, device="cuda")
    out = torch.full((T, 64), 5.0, device="cuda")
    moe.moe_gate_backward(cfg, logits, idx, dg, out[:, 7:], 64)
    ref = torch.empty(T, N, device="cuda")
    moe.moe_gate_backward(make(T, N, K, True), logits.contiguous(), idx, dg, ref)
    assert torch.equal(out[:, 7:57], ref) and (out[:, :7] == 5).all() and (out[:, 57:] == 5).all()


def test_entries_out_of_range_get_no_gradient():
    T, N, K = 6, 20, 3
    logits, dg = torch.randn(T, N, device="cuda"), torch.randn(T, K, device="cuda")
    idx = torch.tensor([[0, 1, 2], [-1, 5, 20], [19, -1, -1], [-1, -1, -1], [3, 999, 4], [2, 1, 0]], dtype=torch.int32,
                       device="cuda")
    for softmax in (False, True):
        for renorm in (False, True):
            d = torch.full((T, N), float("nan"), device="cuda")
            moe.moe_gate_backward(make(T, N, K, softmax, renorm=renorm), logits, idx, dg, d)
            ref = P.gate_backward(logits.cpu().numpy(), idx.cpu().numpy(), dg.cpu().numpy(), softmax, renorm)
            assert (np.abs(d.cpu().numpy() - ref) <= 1e-5 * dg.abs().max().item()).all()


def test_same_bits_again_on_another_stream_and_no_tokens():
    T, N, K = 5000, 256, 8
    logits = torch.randn(T, N, device="cuda")
    cfg = make(T, N, K, False, 8, 4, True)
    first = run(cfg, logits, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run(cfg, logits, None, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    load = torch.full((N,), 7, dtype=torch.int32, device="cuda")
    moe.moe_gate(make(0, N, K, False), None, None, None, None, load, None)
    assert (load == 0).all()


def test_offsets_past_32_bits():
    """More than 2^32 bytes of logits: the last rows come out as they do alone."""
    T, N, K = (1 << 21) + 37, 512, 4
    logits = torch.randn(64, N, device="cuda").repeat(T // 64 + 1, 1)[:T]
    cfg = make(T, N, K, True)
    idx, gate, load = run(cfg, logits, None)
    small = make(64, N, K, True)
    i2, g2, _ = run(small, logits[T - 64:].contiguous(), None)
    assert torch.equal(idx[T - 64:], i2) and torch.equal(gate[T - 64:], g2) and int(load.sum()) == T * K
    dg = torch.randn(T, K, device="cuda")
    d = torch.empty(T, N, device="cuda")
    moe.moe_gate_backward(cfg, logits, idx, dg, d)
    d2 = torch.empty(64, N, device="cuda")
    moe.moe_gate_backward(small, logits[T - 64:].contiguous(), i2, dg[T - 64:].contiguous(), d2)
    assert torch.equal(d[T - 64:], d2)


def test_replayed_in_a_graph():
    T, N, K = 3000, 64, 6
    cfg = make(T, N, K, True)
    logits = torch.randn(T, N, device="cuda")
    dg = torch.randn(T, K, device="cuda")
    ws = torch.empty(moe.moe_gate_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
    gate, load = torch.empty(T, K, device="cuda"), torch.empty(N, dtype=torch.int32, device="cuda")
    d = torch.empty(T, N, device="cuda")

    def step():
        moe.moe_gate(cfg, logits, None, idx, gate, load, ws)
        moe.moe_gate_backward(cfg, logits, idx, dg, d)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        logits.copy_(torch.randn(T, N, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        step()
        want = [t.clone() for t in (idx, gate, load, d)]
        for t in (idx, gate, load, d):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, (idx, gate, load, d)))


@pytest.mark.parametrize("softmax,renorm,K", [(False, True, 8), (True, True, 19), (True, False, 8)])
@pytest.mark.parametrize("N,G", [(70, 1), (256, 8), (512, 4), (288, 3)])
def test_a_token_alone_and_in_any_batch(N, G, softmax, renorm, K):
    """The same bits, whatever the number of lanes and of wavefronts that a call of this length takes."""
    g = torch.Generator("cuda").manual_seed(N + K)
    logits, bias = torch.randn(9001, N, device="cuda", generator=g), 0.01 * torch.randn(N, device="cuda", generator=g)
    outs = []
    for T in (1, 4, 5, 300, 9001):
        idx, gate, _ = run(make(T, N, K, softmax, G, (G + 1) // 2, True, renorm), logits[:T], bias)
        outs.append((T, idx, gate))
    for T, idx, gate in outs[:-1]:
        assert torch.equal(idx, outs[-1][1][:T]) and torch.equal(gate, outs[-1][2][:T])
