"""The layer under a router of the caller's own: moe_gate, moe_forward_train8, moe_backward_gates, moe_gate_backward.

* With the sigmoid router's own logits the chain is moe_backward taken apart: the weight gradients are the same kernels on
  the same rows (same bits without saved inputs), and du and the centroids' gradient, completed by the caller from
  d_logits, agree with moe_backward's to the bf16 rounding of du (2^-8 of a row's largest value, twice rounded) and to
  fp32 sums.
* d_gate against float64 <dout, FFN_k(u)>: bf16 H and dH, 2^-8 each over sums of random terms: 2e-2 of the largest.
* What moe_forward_train8 keeps are the codes of the bf16 rows that moe_forward_train keeps, and its output is the same.
* Gradients from 8 bits stay within 3% (Frobenius) of those recomputed: the codes' error is 0.6% of a normal input."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from oracle import operators as P  # noqa: E402

SHAPES = [(300, 256, 16, 4, 1, 128), (77, 512, 8, 2, 2, 384), (1, 128, 4, 1, 0, 256)]   # T, d, N, K, N_s, I


class Layer:
    def __init__(self, T, d, N, K, Ns, I, fp8, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.T, self.d, self.N, self.K, self.Ns, self.I = T, d, N, K, Ns, I
        self.shape = moe.make_shape(T, d, N, K, Ns, I, moe.MOE_DTYPE_FP8_B128 if fp8 else moe.MOE_DTYPE_BF16)
        self.u, self.dout = rnd(T, d).bfloat16(), rnd(T, d).bfloat16()
        self.e = rnd(N, d) / d ** 0.5
        self.w = [(rnd(n, *s) / s[1] ** 0.5).bfloat16() for n in (N, Ns) for s in ((I, d), (I, d), (d, I))]
        logical = moe.make_weights(*(self.w if Ns else self.w[:3]))
        if fp8:
            self.packed = torch.empty(moe.moe_prepare_weights(self.shape, logical, size_only=True), dtype=torch.uint8,
                                      device="cuda")
            self.weights = moe.moe_prepare_weights(self.shape, logical, self.packed)
        else:
            self.weights = logical
        self.ws = torch.full((moe.moe_backward_workspace_size(self.shape),), 0xFF, dtype=torch.uint8, device="cuda")

    def route(self, softmax=False):
        self.cfg = moe.make_gate_config(self.T, self.N, self.K, moe.MOE_DTYPE_F32,
                                        moe.MOE_SCORE_SOFTMAX if softmax else moe.MOE_SCORE_SIGMOID)
        self.logits = self.u.float() @ self.e.t()
        self.idx = torch.empty(self.T, self.K, dtype=torch.int32, device="cuda")
        self.gate = torch.empty(self.T, self.K, device="cuda")
        moe.moe_gate(self.cfg, self.logits, None, self.idx, self.gate, None, None)

    def grads(self):
        g = [torch.full_like(w, float("nan")) for w in self.w]
        return g, moe.make_weight_grads(*(g if self.Ns else g[:3]))

    def forward8(self):
        out = torch.empty_like(self.u)
        saved = torch.full((moe.moe_saved8_size(self.shape),), 0xA5, dtype=torch.uint8, device="cuda")
        ws = torch.full((moe.moe_train8_workspace_size(self.shape),), 0xFF, dtype=torch.uint8, device="cuda")
        moe.moe_forward_train8(self.shape, self.u, self.weights, self.idx, self.gate, out, saved, ws)
        return out, saved

    def backward_gates(self, saved=None):
        du = torch.full_like(self.u, float("nan"))
        dg = torch.full((self.T, self.K), float("nan"), device="cuda")
        g, wg = self.grads()
        moe.moe_backward_gates(self.shape, self.u, self.weights, self.idx, self.gate, saved, self.dout, du, dg, wg, self.ws)
        return du, dg, g

    def d_logits(self, dg):
        d = torch.empty(self.T, self.N, device="cuda")
        moe.moe_gate_backward(self.cfg, self.logits, self.idx, dg, d)
        return d


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("dims", SHAPES, ids=lambda d: "x".join(map(str, d)))
def test_the_sigmoid_router_taken_apart(dims, fp8):
    x = Layer(*dims, fp8)
    x.route()
    du, dg, g = x.backward_gates()
    whole = torch.empty_like(x.u)
    de = torch.empty(x.N, x.d, device="cuda")
    g2, wg = x.grads()
    moe.moe_backward(x.shape, x.u, x.e, x.weights, x.idx, x.gate, x.dout, whole, de, wg, x.ws)
    for a, b in zip(g, g2):
        assert torch.equal(a, b)
    dl = x.d_logits(dg)
    mine, ref = du.double() + dl.double() @ x.e.double(), whole.double()
    row = ref.abs().amax(dim=1, keepdim=True)
    assert ((mine - ref).abs() <= 2.0 ** -7 * row).all()
    if x.K == 1:   # a renormalised single gate is constant
        assert (dl == 0).all()
        return
    dc = dl.double().t() @ x.u.double()
    # (moe_backward computes the logits anew, in another order of sums)
    assert ((dc - de.double()).abs() <= 1e-4 * dc.abs().max()).all()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("dims", SHAPES, ids=lambda d: "x".join(map(str, d)))
def test_gate_gradients_against_float64(dims, softmax):
    x = Layer(*dims, False, seed=3)
    x.route(softmax)
    x.idx[0, 0] = -1                                  # a pick that moe_gate could not make
    _, dg, _ = x.backward_gates()
    u, dout = x.u.double(), x.dout.double()
    wg, wu, wd = (w.double() for w in x.w[:3])
    ref = torch.zeros(x.T, x.K, dtype=torch.float64, device="cuda")
    for k in range(x.K):
        for t in range(x.T):
            e = int(x.idx[t, k])
            if e >= 0:
                a, b = wg[e] @ u[t], wu[e] @ u[t]
                ref[t, k] = dout[t] @ (wd[e] @ (torch.nn.functional.silu(a) * b))
    assert dg[0, 0].item() == 0
    assert ((dg.double() - ref).abs() <= 2e-2 * max(ref.abs().max().item(), 1e-30)).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("dims", SHAPES, ids=lambda d: "x".join(map(str, d)))
def test_saved_in_8_bits(dims, fp8):
    x = Layer(*dims, fp8, seed=1)
    x.route(softmax=True)
    out, saved8 = x.forward8()
    full = torch.zeros(moe.moe_saved_inputs_size(x.shape) // 2, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_workspace_size(x.shape), dtype=torch.uint8, device="cuda")
    out2 = torch.empty_like(out)
    moe.moe_forward_train(x.shape, x.u, x.weights, x.idx, x.gate, out2, full, ws)
    assert torch.equal(out, out2)
    ab = full.view(-1, 2 * x.I).float().cpu().numpy()
    rows = ab.shape[0]
    size = -(-rows * 2 * x.I // 256) * 256
    codes = saved8[:rows * 2 * x.I].view(torch.int8).view(rows, 2 * x.I).cpu().numpy()
    scales = saved8[size:].view(torch.float32).view(rows, 2 * x.I // 128).cpu().numpy()
    idx = x.idx.cpu().numpy()
    at, real = 0, []
    for e in range(x.N + x.Ns):
        n = int((idx == e).sum()) if e < x.N else x.T
        real += range(at, at + n)
        at += -(-n // 128) * 128
    want, want_s = P.codes8(ab[real])
    assert np.array_equal(codes[real], want) and np.array_equal(scales[real], want_s)
    # gradients from the codes against recomputed ones
    du8, dg8, g8 = x.backward_gates(saved8)
    du, dg, g = x.backward_gates()
    near = lambda a, b: ((a.double() - b.double()).norm() <= 0.03 * b.double().norm() + 1e-30)  # noqa: E731
    assert near(du8, du) and near(dg8, dg)
    for a, b in zip(g8, g):
        assert torch.isfinite(a.float()).all() and (a.numel() == 0 or near(a, b))


def test_no_tokens():
    x = Layer(0, 128, 4, 1, 1, 128, False)
    x.idx, x.gate = torch.empty(0, 1, dtype=torch.int32, device="cuda"), torch.empty(0, 1, device="cuda")
    g, wg = x.grads()
    moe.moe_backward_gates(x.shape, x.u, x.weights, None, None, None, x.ws, x.ws[64:], None, wg, x.ws)
    assert all((w == 0).all() for w in g)
    moe.moe_forward_train8(x.shape, None, x.weights, None, None, None, None, None)


def test_same_bits_in_a_graph():
    x = Layer(300, 256, 16, 4, 1, 128, False, seed=5)
    x.route(True)
    out = torch.empty_like(x.u)
    saved = torch.empty(moe.moe_saved8_size(x.shape), dtype=torch.uint8, device="cuda")
    ws = torch.empty(moe.moe_train8_workspace_size(x.shape), dtype=torch.uint8, device="cuda")
    du, dg = torch.empty_like(x.u), torch.empty(x.T, x.K, device="cuda")
    dl = torch.empty(x.T, x.N, device="cuda")
    g, wg = x.grads()

    def step():
        moe.moe_gate(x.cfg, x.logits, None, x.idx, x.gate, None, None)
        moe.moe_forward_train8(x.shape, x.u, x.weights, x.idx, x.gate, out, saved, ws)
        moe.moe_backward_gates(x.shape, x.u, x.weights, x.idx, x.gate, saved, x.dout, du, dg, wg, x.ws)
        moe.moe_gate_backward(x.cfg, x.logits, x.idx, dg, dl)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.logits.copy_(torch.randn(x.T, x.N, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        step()
        want = [t.clone() for t in (out, du, dg, dl, *g)]
        for t in (out, du, dg, dl):
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (out, du, dg, dl, *g)))
