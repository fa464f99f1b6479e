"""moe_balance_loss and moe_balance_backward on the GPU against float64.

Counts and tokens are whole numbers: equal.  A token's p is fp32: an exponential (2 units in the last place), a sum of
positive terms (under 16 roundings), two quotients: under 2^-19 of the value.  A sequence's sum of p has at most 64 + 64 + 16 additions of
positive terms one after another: 2^-24 each, so 2^-16 in all is asked; values below 2^-126 may be 0.  The gradient
p (c - D) counts against p (|c| + sum p |c|), its terms, with 2^-18, and its type's rounding (bf16 2^-8)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from oracle import block as B  # noqa: E402
from oracle import operators as P  # noqa: E402

SCORE = {True: moe.MOE_SCORE_SOFTMAX, False: moe.MOE_SCORE_SIGMOID}
DT = {torch.float32: moe.MOE_DTYPE_F32, torch.bfloat16: moe.MOE_DTYPE_BF16}
ALPHA = 0.01


def problem(T, N, K, seed, dtype=torch.float32, ld=0):
    g = torch.Generator("cuda").manual_seed(seed)
    wide = torch.randn(T, ld or N, device="cuda", generator=g).to(dtype)
    logits = wide[:, :N]
    idx = torch.rand(T, N, device="cuda", generator=g).topk(K, dim=1).indices.to(torch.int32)
    return logits, idx


def config(logits, idx, S, softmax, ld=0, alpha=ALPHA):
    return moe.make_balance_config(*logits.shape, idx.shape[1], DT[logits.dtype], SCORE[softmax], S, alpha, ld)


def forward(logits, idx, starts, softmax, ld=0, S=None, on=None):
    S = S if S is not None else (1 if starts is None else len(starts) - 1)
    N = logits.shape[1]
    cfg = config(logits, idx, S, softmax, ld)
    ws = torch.full((max(16, moe.moe_balance_workspace_size(cfg)),), 255, dtype=torch.uint8, device="cuda")
    out = [torch.full((S,), float("nan"), device="cuda"), torch.full((S, N), -7, dtype=torch.int32, device="cuda"),
           torch.full((S,), -7, dtype=torch.int32, device="cuda"), torch.full((S, N), float("nan"), device="cuda")]
    moe.moe_balance_loss(cfg, logits, idx, starts, *out, ws, on)
    return out


def backward(logits, idx, starts, softmax, out, d_loss, ld=0, into=None, d_ld=0, on=None):
    S, N = out[1].shape
    cfg = config(logits, idx, S, softmax, ld)
    d = torch.full(logits.shape, float("nan"), dtype=logits.dtype, device="cuda") if into is None else into
    moe.moe_balance_backward(cfg, logits, idx, starts, out[1], out[2], d_loss, d, d_ld, into is not None, on)
    return d


def check(logits, idx, starts, softmax, d_loss=None, ld=0):
    T, N = logits.shape
    s_host = [0, T] if starts is None else starts.tolist()
    out = forward(logits, idx, starts, softmax, ld)
    l, i = logits.float().cpu().numpy(), idx.cpu().numpy()
    loss, counts, tokens, total = B.balance(l, i, s_host, softmax, ALPHA)
    assert np.array_equal(out[1].cpu().numpy(), counts) and np.array_equal(out[2].cpu().numpy(), tokens)
    assert (np.abs(out[3].cpu().numpy() - total) <= 2.0 ** -16 * total + 2.0 ** -120).all()
    assert (np.abs(out[0].cpu().numpy() - loss) <= 2.0 ** -15 * loss).all()
    if d_loss is None:
        d_loss = torch.linspace(-1, 2, len(s_host) - 1, device="cuda")
    d = backward(logits, idx, starts, softmax, out, d_loss, ld).float().cpu().numpy()
    dl = d_loss.cpu().numpy().astype(np.float64)
    ref = B.balance_backward(l, i, s_host, softmax, ALPHA, dl)
    p, size = B.shares(l, softmax), np.zeros((T, N))
    for s in range(len(s_host) - 1):
        if tokens[s]:
            c = np.abs(dl[s]) * ALPHA * N * counts[s] / (i.shape[1] * float(tokens[s]) ** 2)
            rows = slice(s_host[s], s_host[s + 1])
            size[rows] = p[rows] * (c + (p[rows] @ c)[:, None])
    if not softmax:
        size *= P.sigmoid(-l.astype(np.float64))
    half = 2.0 ** -8 if logits.dtype == torch.bfloat16 else 2.0 ** -24
    assert (np.abs(d - ref) <= half * np.abs(ref) + 2.0 ** -18 * size + 2.0 ** -126).all()
    return out, d


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("T,N,K,dtype", [
    (1, 1, 1, torch.float32), (3, 8, 2, torch.bfloat16), (64, 60, 4, torch.float32), (65, 64, 6, torch.float32),
    (777, 129, 8, torch.bfloat16), (500, 256, 8, torch.float32), (130, 511, 32, torch.float32),
    (200, 512, 17, torch.bfloat16), (70, 2, 1, torch.bfloat16)])
def test_one_sequence(T, N, K, dtype, softmax):
    logits, idx = problem(T, N, K, T + N, dtype)
    check(logits, idx, None, softmax, torch.tensor([1.5], device="cuda"))
    whole = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    a, b = forward(logits, idx, None, softmax), forward(logits, idx, whole, softmax)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("lengths", [[1, 63, 64, 65, 0, 0, 200, 7, 1], [0, 5, 0], [1] * 100, [3] * 90 + [300, 0, 0, 0],
                                     [128, 128, 16, 16]])
def test_sequences(lengths, softmax):
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    logits, idx = problem(int(starts[-1]), 48, 3, len(lengths))
    idx[::7] = -1                                  # padding tokens
    idx[3::11, 1] = 48                             # picks that are none
    idx[4::13, 0] = -5
    out, d = check(logits, idx, starts, softmax)
    real = ((idx >= 0) & (idx < 48)).any(1).cpu().numpy()
    assert (d[~real] == 0).all()
    # a sequence's results are its own, wherever it begins in the batch
    for s in (0, len(lengths) // 2, len(lengths) - 1):
        a, b = int(starts[s]), int(starts[s + 1])
        if b > a:
            alone = forward(logits[a:b].contiguous(), idx[a:b].contiguous(), None, softmax)
            assert torch.equal(alone[1][0], out[1][s]) and torch.equal(alone[2][0], out[2][s])
            assert torch.allclose(alone[0][0], out[0][s], rtol=2.0 ** -15, atol=0)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("N,dtype,lengths", [
    (64, torch.float32, [256]), (64, torch.bfloat16, [257]), (61, torch.float32, [31]), (61, torch.bfloat16, [33]),
    (256, torch.float32, [64]), (256, torch.bfloat16, [65]), (500, torch.bfloat16, [20, 0, 44, 1, 15]),
    (64, torch.float32, [1, 63, 64, 65, 0, 0, 200, 7, 1] * 9), (60, torch.bfloat16, [0, 0, 1000, 1, 0, 47] * 3),
    (256, torch.float32, [1, 31, 32, 33, 0, 0, 200, 7, 1] * 4), (130, torch.bfloat16, [5, 300, 1, 1, 0, 9] * 3),
    (512, torch.float32, [1, 15, 16, 17, 0, 0, 100, 7, 1] * 4)])
def test_one_kernel_and_two(N, dtype, lengths, softmax):
    """Few tokens in one kernel and more in two: where the one ends, with sequences that begin anywhere in a block."""
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    logits, idx = problem(int(starts[-1]), N, 5, N + len(lengths), dtype)
    idx[::5] = -1
    idx[1::9, 2] = N + 7
    check(logits, idx, starts, softmax)


def test_tokens_outside_the_sequences():
    logits, idx = problem(300, 40, 4, 3)
    starts = torch.tensor([20, 90, 90, 211], dtype=torch.int32, device="cuda")
    out = forward(logits, idx, starts, True)
    d_loss = torch.tensor([1.0, 2.0, 3.0], device="cuda")
    d = backward(logits, idx, starts, True, out, d_loss)
    inner = logits[20:211].contiguous(), idx[20:211].contiguous(), starts - 20
    ref = forward(*inner, True)
    assert torch.equal(ref[1], out[1]) and torch.equal(ref[2], out[2])
    assert torch.allclose(ref[0], out[0], rtol=2.0 ** -15, atol=0)
    assert torch.equal(d[20:211], backward(*inner, True, ref, d_loss)) and (d[:20] == 0).all() and (d[211:] == 0).all()
    into = torch.full_like(logits, 5.0)
    backward(logits, idx, starts, True, out, d_loss, into=into)
    assert (into[:20] == 5).all() and (into[211:] == 5).all() and (into[20:90] != 5).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_added_to_the_gates_gradient(dtype):
    logits, idx = problem(150, 60, 4, 4, dtype)
    idx[5] = -1
    out = forward(logits, idx, None, True)
    one = torch.ones(1, device="cuda")
    d = backward(logits.float(), idx, None, True, out, one)
    was = torch.randn(150, 60, device="cuda").to(dtype)
    got = backward(logits, idx, None, True, out, one, into=was.clone())
    want = was.double() + d.double()
    assert torch.equal(got[5], was[5])
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert ((got.double() - want).abs() <= half * want.abs() + 2.0 ** -18 * d.abs()).all()


def test_strides():
    logits, idx = problem(90, 50, 5, 5, ld=61)
    dense = logits.contiguous()
    a, b = forward(logits, idx, None, False, ld=61), forward(dense, idx, None, False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    one = torch.ones(1, device="cuda")
    into = torch.full((90, 55), 3.0, device="cuda")
    moe.moe_balance_backward(config(logits, idx, 1, False, 61), logits, idx, None, a[1], a[2], one, into, 55)
    assert torch.equal(into[:, :50], backward(dense, idx, None, False, b, one)) and (into[:, 50:] == 3).all()


@pytest.mark.parametrize("softmax", [True, False])
def test_masked_extreme_and_not_finite_logits(softmax):
    logits, idx = problem(140, 64, 4, 6)
    logits[:, 7] = -float("inf")                     # an expert that is out
    logits[3] = -float("inf")                        # a token with none (its picks count all the same)
    logits[4] = -200.0                               # every sigmoid below fp32's range: equal shares
    logits[5] = torch.where(torch.arange(64, device="cuda") == 9, -3.4e38, -100.0)
    logits[6] = 200.0
    logits[8] = -3.4e38
    check(logits, idx, None, softmax)
    logits[11] = float("nan")
    idx[11] = -1                                     # a padding row's values do not matter
    out, d = check_padding(logits, idx, softmax, 11)
    idx[11] = idx[12]
    out = forward(logits, idx, None, softmax)
    assert torch.isnan(out[0]).all() and torch.isnan(out[3]).any()


@pytest.mark.parametrize("softmax", [True, False])
def test_extreme_logits_in_a_large_batch(softmax):
    """The same where the sums take two kernels, in a sequence of its own and among others."""
    logits, idx = problem(900, 64, 6, 21)
    logits[:, 7] = -float("inf")
    logits[300] = -float("inf")
    logits[301] = -200.0
    logits[302] = torch.where(torch.arange(64, device="cuda") == 9, -3.4e38, -100.0)
    logits[303:305] = 200.0
    logits[899] = -3.4e38
    for starts in (None, torch.tensor([0, 299, 302, 303, 900], dtype=torch.int32, device="cuda")):
        check(logits, idx, starts, softmax)
    logits[511] = float("nan")
    idx[511] = -1
    check_padding(logits, idx, softmax, 511)
    idx[511] = idx[512]
    out = forward(logits, idx, torch.tensor([0, 500, 600, 900], dtype=torch.int32, device="cuda"), softmax)
    assert torch.isnan(out[0]).tolist() == [False, True, False] and torch.isfinite(out[3][0]).all()


def test_two_graphs_share_a_workspace():
    g = torch.Generator("cuda").manual_seed(4)
    calls, ws = [], None
    for T, N, K in ((5000, 64, 4), (3000, 200, 8)):
        logits, idx = problem(T, N, K, T)
        cfg = config(logits, idx, 1, True)
        need = moe.moe_balance_workspace_size(cfg)
        ws = torch.empty(max(need, 1 << 21), dtype=torch.uint8, device="cuda") if ws is None else ws
        assert 0 < need <= ws.numel()
        out = [torch.empty(1, device="cuda"), torch.empty(1, N, dtype=torch.int32, device="cuda"),
               torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, N, device="cuda")]
        forward(logits, idx, None, True)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_balance_loss(cfg, logits, idx, None, *out, ws)
        calls.append((graph, logits, idx, out))
    for k in range(6):
        graph, logits, idx, out = calls[k % 2]
        logits.copy_(torch.randn(logits.shape, device="cuda", generator=g))
        want = forward(logits, idx, None, True)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out))


def test_few_tokens_need_no_workspace():
    logits, idx = problem(60, 64, 6, 22)
    cfg = config(logits, idx, 1, True)
    assert moe.moe_balance_workspace_size(cfg) == 0
    out = [torch.empty(1, device="cuda"), torch.empty(1, 64, dtype=torch.int32, device="cuda"),
           torch.empty(1, dtype=torch.int32, device="cuda")]
    moe.moe_balance_loss(cfg, logits, idx, None, *out, None, None)
    assert all(torch.equal(x, y) for x, y in zip(out, forward(logits, idx, None, True)))


def check_padding(logits, idx, softmax, row):
    out = forward(logits, idx, None, softmax)
    keep = torch.arange(logits.shape[0], device="cuda") != row
    others = logits[keep].contiguous(), idx[keep].contiguous(), None, softmax
    ref = forward(*others)
    assert torch.equal(out[1], ref[1]) and torch.equal(out[2], ref[2])
    assert torch.allclose(out[3], ref[3], rtol=2.0 ** -15, atol=2.0 ** -120)
    one = torch.ones(1, device="cuda")
    d = backward(logits, idx, None, softmax, out, one)
    assert (d[row] == 0).all() and torch.equal(d[keep], backward(*others, out, one))
    return out, d


def test_gradient_against_differences():
    logits, idx = problem(40, 16, 2, 7)
    out = forward(logits, idx, None, False)
    one = torch.ones(1, device="cuda")
    d = backward(logits, idx, None, False, out, one)
    v = torch.randn(40, 16, device="cuda")
    h = 2.0 ** -6
    up, down = (forward(logits + s * h * v, idx, None, False)[0].double() for s in (1, -1))
    slope, along = ((up - down) / (2 * h)).item(), (d.double() * v.double()).sum().item()
    # the loss is fp32 (2^-22 of 0.01 over 2 h), its third derivative moves the slope by h^2 of it or so
    assert abs(slope - along) <= 2.0 ** -22 * ALPHA / h + 4 * h * h * (d.double() * v.double()).abs().sum().item()


def test_counts_of_a_whole_job():
    """Two ranks' counts, tokens and sums added up: the loss and gradients of the whole batch."""
    logits, idx = problem(400, 64, 6, 8)
    whole = forward(logits, idx, None, True)
    one = torch.ones(1, device="cuda")
    parts = [(logits[r].contiguous(), idx[r].contiguous()) for r in (slice(0, 150), slice(150, 400))]
    outs = [forward(*p, None, True) for p in parts]
    total = [outs[0][i] + outs[1][i] for i in range(4)]
    assert torch.equal(total[1], whole[1]) and torch.equal(total[2], whole[2])
    L = total[2].double()
    loss = ALPHA * ((64 * total[1].double() / (6 * L)) * total[3].double() / L).sum()
    assert abs(loss.item() - whole[0].item()) <= 2.0 ** -15 * loss.item()
    d = torch.cat([backward(*p, None, True, total, one) for p in parts])
    assert torch.equal(d, backward(logits, idx, None, True, whole, one))


def test_no_tokens_and_no_sum():
    cfg = moe.make_balance_config(0, 40, 4, 0, 1, 3, 1.0)
    out = [torch.full((3,), 5.0, device="cuda"), torch.full((3, 40), 5, dtype=torch.int32, device="cuda"),
           torch.full((3,), 5, dtype=torch.int32, device="cuda"), torch.full((3, 40), 5.0, device="cuda")]
    moe.moe_balance_loss(cfg, None, None, torch.zeros(4, dtype=torch.int32, device="cuda"), *out, None)
    assert all((o == 0).all() for o in out)
    logits, idx = problem(100, 40, 4, 9)
    a = forward(logits, idx, None, True)
    b = [torch.empty_like(o) for o in a[:3]]
    cfg = config(logits, idx, 1, True)
    ws = torch.empty(moe.moe_balance_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss(cfg, logits, idx, None, *b, None, ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_more_sequences_than_tokens():
    """Most of them empty; and so many that the counts take several rounds to clear."""
    logits, idx = problem(90, 12, 2, 14)
    S = 5000
    starts = torch.sort(torch.randint(0, 91, (S + 1,), device="cuda")).values.to(torch.int32)
    starts[0], starts[-1] = 0, 90
    out, _ = check(logits, idx, starts, True)
    assert int(out[2].sum()) == 90
    S, N = 70000, 512
    cfg = moe.make_balance_config(0, N, 4, 0, 1, S, 1.0)
    res = [torch.full((S,), 5.0, device="cuda"), torch.full((S, N), 5, dtype=torch.int32, device="cuda"),
           torch.full((S,), 5, dtype=torch.int32, device="cuda"), torch.full((S, N), 5.0, device="cuda")]
    moe.moe_balance_loss(cfg, None, None, torch.zeros(S + 1, dtype=torch.int32, device="cuda"), *res, None)
    assert all((o == 0).all() for o in res)


def test_large_batch_another_stream_and_a_graph():
    """More tokens than places of 64: longer chunks; the same bits again."""
    T, N, K = 150000, 64, 6
    logits, idx = problem(T, N, K, 10)
    starts = torch.tensor([0, 70001, 70002, T], dtype=torch.int32, device="cuda")
    first = forward(logits, idx, starts, True)
    p = torch.softmax(logits.double(), 1)
    for s in range(3):
        a, b = int(starts[s]), int(starts[s + 1])
        counts = torch.bincount(idx[a:b].flatten().long(), minlength=N)
        assert torch.equal(first[1][s].long(), counts) and first[2][s] == b - a
        total = p[a:b].sum(0)
        assert ((first[3][s].double() - total).abs() <= 2.0 ** -14 * total).all()
        loss = ALPHA * (N * counts.double() / (K * (b - a)) * total / (b - a)).sum()
        assert abs(first[0][s].double() - loss) <= 2.0 ** -14 * loss
    d_loss = torch.tensor([1.0, 2.0, 3.0], device="cuda")
    d1 = backward(logits, idx, starts, True, first, d_loss)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = forward(logits, idx, starts, True, on=side)
        d2 = backward(logits, idx, starts, True, again, d_loss, on=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, again)) and torch.equal(d1, d2)
    cfg = config(logits, idx, 3, True)
    ws = torch.empty(moe.moe_balance_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_balance_loss(cfg, logits, idx, starts, *again, ws)
        moe.moe_balance_backward(cfg, logits, idx, starts, again[1], again[2], d_loss, d2)
    for k in range(4):
        logits.copy_(torch.randn_like(logits))
        want = forward(logits, idx, starts, True)
        d1 = backward(logits, idx, starts, True, want, d_loss)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, again)) and torch.equal(d1, d2)


def test_offsets_past_32_bits():
    T, N = (1 << 23) + 77, 512
    block, idx = problem(64, N, 2, 11, torch.bfloat16)
    reps = T // 64 + 1
    logits, idx_all = block.repeat(reps, 1)[:T], idx.repeat(reps, 1)[:T]
    starts = torch.tensor([0, T - 50, T], dtype=torch.int32, device="cuda")
    out = forward(logits, idx_all, starts, True)
    tail = logits[T - 50:].contiguous(), idx_all[T - 50:].contiguous()
    ref = forward(*tail, None, True)
    assert torch.equal(ref[1][0], out[1][1]) and torch.allclose(ref[3][0], out[3][1], rtol=2.0 ** -15, atol=0)
    one = torch.ones(2, device="cuda")
    d = backward(logits, idx_all, starts, True, out, one)
    last = [o[1:].contiguous() for o in out]
    assert torch.equal(d[T - 50:], backward(*tail, None, True, last, one[:1].contiguous()))
    assert torch.equal(d[:64], d[64:128])
