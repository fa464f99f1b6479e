"""One buffer, sized for the largest batch, under smaller ones: the results of a workspace of each call's own, and nothing
written behind the size that the query names for the call."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
import test_gpu_adapters as A  # noqa: E402
import test_gpu_balance as L  # noqa: E402


def guarded(size):
    return torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("n,r,d_in,d_out", [(8, 16, 2048, 520), (32, 64, 1032, 264), (5, 128, 520, 136), (300, 32, 264, 72)])
def test_adapters(n, r, d_in, d_out):
    size = lambda t: moe.moe_adapters_workspace_size(  # noqa: E731
        moe.make_adapter_shape(t, d_in, d_out, n, r, moe.MOE_DTYPE_BF16))
    most = size(2500)
    for rows in (1, 17, 64, 65, 200, 511, 1024, 1025, 1037, 2049, 2500):
        p = A.problem(rows, d_in, d_out, n, r, rows)
        want = A.run(p)
        ws = guarded(most)
        assert torch.equal(A.run(p, ws=ws[:most]), want)
        assert (ws[size(rows):] == 0xA5).all()


@pytest.mark.parametrize("N,softmax", [(64, True), (60, True), (61, False), (256, False), (512, True)])
def test_balance(N, softmax):
    size = lambda t, s: moe.moe_balance_workspace_size(  # noqa: E731
        moe.make_balance_config(t, N, 4, moe.MOE_DTYPE_F32, moe.MOE_SCORE_SOFTMAX, s))
    most = size(20000, 40)
    for T, S in ((1, 1), (64, 40), (300, 3), (1021, 7), (1021, 40), (4099, 1), (8194, 40), (16391, 2), (20000, 40)):
        logits, idx = L.problem(T, N, 4, T + S)
        inner = torch.randint(0, T + 1, (S - 1,), device="cuda")
        starts = torch.sort(torch.cat([inner, torch.tensor([0, T], device="cuda")])).values.to(torch.int32)
        want = L.forward(logits, idx, starts, softmax)
        got = [torch.empty_like(t) for t in want]
        ws = guarded(most)
        moe.moe_balance_loss(L.config(logits, idx, S, softmax), logits, idx, starts, *got, ws[:most])
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert (ws[size(T, S):] == 0xA5).all()


@pytest.mark.parametrize("T,N,S", [(1021, 60, 7), (2048, 64, 64), (500, 256, 20)])
def test_few_tokens_of_several_sequences_take_none(T, N, S):
    """The query answers for fewer sequences too; the call that one kernel does takes none."""
    logits, idx = L.problem(T, N, 4, T)
    starts = (torch.arange(S + 1, device="cuda") * T // S).to(torch.int32)
    cfg = L.config(logits, idx, S, True)
    assert moe.moe_balance_workspace_size(cfg) > 0
    want = L.forward(logits, idx, starts, True)
    got = [torch.empty_like(t) for t in want]
    moe.moe_balance_loss(cfg, logits, idx, starts, *got, None)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
