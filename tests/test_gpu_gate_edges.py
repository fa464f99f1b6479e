"""moe_gate at its edges, on the GPU against the float64 statement: experts out of service in rows that hold a NaN or an
infinity.

Picks are compared exactly, but for rows that were decided by less than 4e-6 of their largest key (fp32 ranks those either
way); gates to 5e-6, as quotients of sums of exponentials of arguments that fp32 holds exactly or that are small."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from oracle import operators as P  # noqa: E402

INF, NAN = float("inf"), float("nan")


def run(l, bias, K, softmax, G=1, TG=1, top2=False, renorm=True, scale=1.0):
    T, N = l.shape
    cfg = moe.make_gate_config(T, N, K, moe.MOE_DTYPE_BF16 if l.dtype == torch.bfloat16 else moe.MOE_DTYPE_F32,
                               moe.MOE_SCORE_SOFTMAX if softmax else moe.MOE_SCORE_SIGMOID, G, TG,
                               moe.MOE_GROUP_TOP2 if top2 else moe.MOE_GROUP_MAX, renorm, scale)
    idx = torch.full((T, K), -77, dtype=torch.int32, device="cuda")
    gate = torch.full((T, K), 5.0, device="cuda")
    load = torch.full((N,), -77, dtype=torch.int32, device="cuda")
    ws = torch.full((max(1, moe.moe_gate_workspace_size(cfg)),), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_gate(cfg, l, bias, idx, gate, load, ws)
    torch.cuda.synchronize()
    return cfg, idx, gate, load


# tokens, experts, groups: 16 lanes a token, 32, 64 (few tokens), groups of whole lanes and groups that are not
LAYOUTS = [(40, 48, 1), (40, 48, 4), (40, 63, 9), (40, 256, 8), (40, 500, 1), (40, 500, 5), (4, 200, 1), (4, 256, 8)]


@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("T,N,G", LAYOUTS)
def test_a_nan_or_an_infinity_opens_no_expert_out_of_service(T, N, G, softmax):
    K, gs = 6, N // G
    rng = np.random.default_rng(N + G)
    l = rng.standard_normal((T, N)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(N)).astype(np.float32)
    bias[[0, 1, 3, N - 1]] = -INF
    if G > 2:
        bias[gs:2 * gs] = -INF             # a whole group
    l[0, [0, N // 2]] = NAN                # of one that is out, and of one that is not
    l[1, 3] = NAN                          # only of one that is out
    l[2, N // 2 + 1] = INF
    l[3] = NAN
    l[3, 5:] = -INF                        # all masked or NaN: 2 and 4 are left
    for top2 in (False, True) if G > 1 else (False,):
        TG = max(1, G // 2)
        _, idx, _, load = run(torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda(), K, softmax, G, TG, top2)
        with np.errstate(invalid="ignore"):
            want, _, _, gap = P.gate(l, bias, K, softmax, G, TG, top2)
            keys = P.gate_scores(l, softmax) + np.where(np.isneginf(bias), 0, bias)
        clear = gap > 4e-6 * np.abs(np.where(np.isfinite(keys), keys, 0)).max(axis=1)
        got = idx.cpu().numpy()
        assert clear[:4].all() and np.array_equal(got[clear], want[clear])
        assert not np.isneginf(bias[got[got >= 0]]).any()
        assert np.array_equal(load.cpu().numpy(), np.bincount(got[got >= 0], minlength=N))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
def test_an_empty_place_beside_a_nan_has_gate_zero(softmax, renorm):
    for T, N in ((4, 200), (5, 30), (5, 400)):
        l = torch.full((T, N), -INF, device="cuda")
        l[:, 7], l[:, 9] = 0.5, NAN
        _, idx, gate, _ = run(l, None, 5, softmax, renorm=renorm)
        assert idx.tolist() == [[7, 9, -1, -1, -1]] * T
        assert (gate[:, 2:] == 0).all() and torch.isnan(gate[:, 1]).all()


# tokens, experts, groups, the step between neighbouring logits of a row (the last ones are 500 below the first), type
SPREAD = [(40, 48, 1, 8), (40, 64, 4, 8), (40, 63, 9, 8), (40, 256, 8, 2), (4, 128, 4, 4), (4, 256, 1, 2)]


@pytest.mark.parametrize("T,N,G,step,bf16", [(*c, b) for c in SPREAD for b in (False, True)] + [(40, 500, 5, 1, False)])
def test_softmax_picks_among_scores_too_small_for_fp32(T, N, G, step, bf16):
    """Without a bias (none, or zeros) the order is that of the logits, exp(-90) and exp(-91) told apart."""
    K = 9
    rng = np.random.default_rng(N)
    l = (step * (np.argsort(rng.random((T, N)), axis=1) - N // 2)).astype(np.float32)
    l[0] = 0
    l[0, [N // 2, N // 3]] = 95, 5         # the rest ties at 0
    x = torch.from_numpy(l).cuda()
    x = x.bfloat16() if bf16 else x
    assert np.array_equal(x.float().cpu().numpy(), l)
    zeros = np.zeros(N, np.float32)
    out = zeros.copy()
    out[[1, N // 2 + 1, N - 1]] = -INF
    for bias in (None, zeros, out):
        b = None if bias is None else torch.from_numpy(bias).cuda()
        for top2 in (False, True) if G > 1 else (False,):
            for renorm in (False, True):
                TG = (G + 1) // 2
                cfg, idx, gate, load = run(x, b, K, True, G, TG, top2, renorm)
                want, gates, cnt, _ = P.gate(l, bias, K, True, G, TG, top2, renorm)
                assert np.array_equal(idx.cpu().numpy(), want) and np.array_equal(load.cpu().numpy(), cnt)
                # (differences of these logits are exact; a score below 2^-126 may be 0)
                assert (np.abs(gate.cpu().numpy() - gates) <= 5e-6 * gates + 2.0 ** -126).all()


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("N,K", [(40, 6), (256, 8), (500, 20)])
def test_gates_and_gradients_of_large_logits(N, K, softmax, bf16):
    """Logits of up to 80: saturated sigmoids, and softmax rows that one expert has to itself.  A sigmoid keeps its own
    5e-6; a softmax's argument is rounded by up to 2^-24 of 160 besides (1e-5), and its gates may underflow."""
    T = 60
    g = torch.Generator("cuda").manual_seed(N + K)
    l = 160 * torch.rand(T, N, device="cuda", generator=g) - 80
    l[:8] = -60 - 20 * torch.rand(8, N, device="cuda", generator=g)     # rows of small sigmoids alone
    l[8:16] = 20 + 60 * torch.rand(8, N, device="cuda", generator=g)    # and of saturated ones
    l = l.bfloat16() if bf16 else l
    bias = 0.1 * torch.randn(N, device="cuda", generator=g)
    dg = torch.randn(T, K, device="cuda", generator=g)
    host = l.float().cpu().numpy()
    for b in (None, bias):
        for renorm in (False, True):
            cfg, idx, gate, _ = run(l, b, K, softmax, renorm=renorm, scale=2.0)
            got = idx.cpu().numpy()
            assert (got >= 0).all() and all(len(set(r)) == K for r in got.tolist())
            gates = P.gate_values(P.gate_scores(host, softmax), got, renorm, 2.0)
            tol = (1.5e-5 if softmax else 5e-6) * gates + 2.0 ** -124
            assert (np.abs(gate.cpu().numpy() - gates) <= tol).all()
            d = torch.full_like(l, NAN)
            moe.moe_gate_backward(cfg, l, idx, dg, d)
            ref = P.gate_backward(host, got, dg.cpu().numpy(), softmax, renorm, 2.0)
            tol = (3e-5 if softmax else 1e-5) * 2.0 * dg.abs().amax(dim=1, keepdim=True).cpu().numpy()
            tol = tol + (2.0 ** -8 * np.abs(ref) if bf16 else 0)
            assert (np.abs(d.float().cpu().numpy() - ref) <= tol).all()
