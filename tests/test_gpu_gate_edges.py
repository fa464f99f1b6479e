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
