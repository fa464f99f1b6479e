"""The norm, the balance loss and the adapters beside the layer, the gate and the FP8 product, as a step uses them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from oracle import block as B  # noqa: E402
from oracle import operators as P  # noqa: E402

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
EPS, ALPHA = 1e-6, 2e4     # (a balance gradient as large as the gates')


def empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def bytes_of(n):
    return torch.full((max(16, n),), 255, dtype=torch.uint8, device="cuda")


class TrainBlock:
    """x + residual, the norm, a softmax router with its balance loss, the experts with 8-bit saved inputs."""

    def __init__(self, T, d, N, K, I, starts, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.T, self.d, self.N, self.K = T, d, N, K
        self.weight, self.router = 1 + 0.2 * r(d), r(N, d) / d ** 0.5
        self.w = [(r(n, *s) / s[1] ** 0.5).to(BF16) for n in (N, 1) for s in ((I, d), (I, d), (d, I))]
        self.g = [torch.empty_like(w) for w in self.w]
        self.weights, self.grads = moe.make_weights(*self.w), moe.make_weight_grads(*self.g)
        self.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        S = len(starts) - 1
        self.norm = moe.make_norm_shape(T, d, moe.MOE_DTYPE_BF16, EPS)
        self.gate = moe.make_gate_config(T, N, K, moe.MOE_DTYPE_F32, moe.MOE_SCORE_SOFTMAX)
        self.balance = moe.make_balance_config(T, N, K, moe.MOE_DTYPE_F32, moe.MOE_SCORE_SOFTMAX, S, ALPHA)
        self.layer = moe.make_shape(T, d, N, K, 1, I, moe.MOE_DTYPE_BF16)
        self.h, self.y, self.rstd = empty(T, d, dtype=BF16), empty(T, d, dtype=BF16), empty(T)
        self.idx, self.gates, self.load = empty(T, K, dtype=torch.int32), empty(T, K), empty(N, dtype=torch.int32)
        self.loss, self.counts, self.tokens = empty(S), empty(S, N, dtype=torch.int32), empty(S, dtype=torch.int32)
        self.out, self.du, self.dx = (empty(T, d, dtype=BF16) for _ in range(3))
        self.d_gate, self.d_logits, self.dw = empty(T, K), empty(T, N), empty(d)
        self.saved = bytes_of(moe.moe_saved8_size(self.layer))
        self.ws = bytes_of(max(moe.moe_train8_workspace_size(self.layer), moe.moe_backward_workspace_size(self.layer)))
        self.ws2 = bytes_of(max(moe.moe_gate_workspace_size(self.gate), moe.moe_balance_workspace_size(self.balance),
                                moe.moe_norm_workspace_size(self.norm)))

    def forward(self, x, residual):
        moe.moe_norm_forward(self.norm, x, residual, self.weight, self.h, self.y, None, None, self.rstd)
        self.logits = self.y.float() @ self.router.t()
        moe.moe_gate(self.gate, self.logits, None, self.idx, self.gates, self.load, self.ws2)
        moe.moe_balance_loss(self.balance, self.logits, self.idx, self.starts, self.loss, self.counts, self.tokens, None,
                             self.ws2)
        moe.moe_forward_train8(self.layer, self.y, self.weights, self.idx, self.gates, self.out, self.saved, self.ws)

    def backward(self, d_out, d_h, d_loss):
        moe.moe_backward_gates(self.layer, self.y, self.weights, self.idx, self.gates, self.saved, d_out, self.du, self.d_gate,
                               self.grads, self.ws)
        moe.moe_gate_backward(self.gate, self.logits, self.idx, self.d_gate, self.d_logits)
        moe.moe_balance_backward(self.balance, self.logits, self.idx, self.starts, self.counts, self.tokens, d_loss,
                                 self.d_logits, accumulate=True)
        self.d_router = self.d_logits.t() @ self.y.float()
        dy = (self.du.float() + self.d_logits @ self.router).to(BF16)
        moe.moe_norm_backward(self.norm, dy, d_h, self.h, self.weight, self.rstd, self.dx, self.dw, self.ws2)

    def results(self):
        return [t.clone() for t in (self.out, self.loss, self.counts, self.d_logits, self.dx, self.dw, self.d_router, *self.g)]


def train_inputs(T, d, S, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    some = [r(T, d).to(BF16) for _ in range(4)]
    return some[:2], (*some[2:], 1 + torch.rand(S, device="cuda", generator=g))


def test_a_training_step_against_float64():
    """The logits' gradient against the float64 statements on the GPU's own d_gate: fp32 sums of two gradients, each within
    2^-18 of its terms.  Everything that passes the layer against autograd: the layer's own bar is 2% (bf16 storage, SwiGLU
    inputs in 8 bits), and y, dy and dx are rounded to bf16 around it (2^-8 each at most): 3.2% of a gradient."""
    T, d, N, K, I, starts = 200, 256, 8, 2, 128, [0, 90, 90, 200]
    blk = TrainBlock(T, d, N, K, I, starts, 1)
    (x, res), (d_out, d_h, d_loss) = train_inputs(T, d, 3, 2)
    blk.forward(x, res)
    blk.backward(d_out, d_h, d_loss)
    n = lambda t: t.float().cpu().numpy()  # noqa: E731
    logits, idx = n(blk.logits), blk.idx.cpu().numpy()
    part = P.gate_backward(logits, idx, n(blk.d_gate), True), B.balance_backward(logits, idx, starts, True, ALPHA, n(d_loss))
    assert np.linalg.norm(part[1]) > 0.05 * np.linalg.norm(part[0])      # (both count)
    row = sum(np.abs(p).sum(axis=1, keepdims=True) for p in part)
    row = row + np.abs(n(blk.d_gate)).sum(axis=1, keepdims=True)
    assert (np.abs(n(blk.d_logits) - part[0] - part[1]) <= 2.0 ** -16 * row).all()
    f = lambda t: t.double().requires_grad_()  # noqa: E731
    h, weight, router = f(blk.h), f(blk.weight), f(blk.router)
    w = [f(t) for t in blk.w]
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * weight
    p = torch.softmax(y @ router.t(), dim=1)
    s = p.gather(1, blk.idx.long())
    gate = s / s.sum(1, keepdim=True)
    ffns = [(torch.nn.functional.silu(y @ wg.t()) * (y @ wu.t())) @ wd.t() for k in (0, 3) for wg, wu, wd in zip(*w[k:k + 3])]
    out = y + ffns[-1]
    for k in range(K):
        out = out + gate[:, k:k + 1] * torch.stack(ffns[:N], 1)[torch.arange(T, device="cuda"), blk.idx[:, k].long()]
    total = (out * d_out.double()).sum() + (h * d_h.double()).sum()
    for j in range(3):
        rows = slice(starts[j], starts[j + 1])
        if starts[j + 1] > starts[j]:
            L = starts[j + 1] - starts[j]
            counts = torch.bincount(blk.idx[rows].flatten().long(), minlength=N).double()
            total = total + d_loss[j].double() * ALPHA * (N * counts / (K * L) * p[rows].mean(0)).sum()
    total.backward()
    near = lambda a, b: ((a.double() - b).norm() / b.norm()).item() < 0.032  # noqa: E731
    assert near(blk.out, out.detach()) and near(blk.dx, h.grad)
    assert near(blk.dw, weight.grad) and near(blk.d_router, router.grad)
    assert near(blk.dx.double() - d_h.double(), h.grad - d_h.double())
    assert all(near(a, b.grad) for a, b in zip(blk.g, w))


def test_two_steps_on_two_streams_and_again():
    """Two blocks at once, each on its own stream with its own workspaces: the results of each alone, bit for bit."""
    blks = [TrainBlock(300, 256, 16, 4, 128, [0, 64, 300], 3), TrainBlock(177, 512, 24, 3, 128, [0, 177], 4)]
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


class ServeBlock:
    """x + residual, the norm with an 8-bit output, the shared FP8 projection, the requests' adapters on top."""

    def __init__(self, T, d, out, adapters, rank, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.weight, w = 1 + 0.2 * r(d), (r(out, d) / d ** 0.5).to(BF16)
        self.wq, self.ws = empty(out, d, dtype=F8), empty(-(-out // 128), d // 128)
        moe.moe_quantize_weights(1, out, d, w, self.wq, self.ws)
        self.a, self.b = (r(adapters, rank, d) / d ** 0.5).to(BF16), (r(adapters, out, rank) / rank ** 0.5).to(BF16)
        self.scale = 0.5 + torch.rand(adapters, device="cuda", generator=g)
        self.norm = moe.make_norm_shape(T, d, moe.MOE_DTYPE_BF16, EPS)
        self.product = moe.make_matmul_shape(T, out, d, moe.MOE_FP8_FORWARD, moe.MOE_DTYPE_BF16)
        self.adapters = moe.make_adapter_shape(T, d, out, adapters, rank, moe.MOE_DTYPE_BF16)
        self.h, self.y, self.codes, self.scales = empty(T, d, dtype=BF16), empty(T, d, dtype=BF16), empty(T, d, dtype=F8), \
            empty(T, d // 128)
        self.base, self.out = empty(T, out, dtype=BF16), empty(T, out, dtype=BF16)
        self.w1 = bytes_of(moe.moe_matmul_fp8_workspace_size(self.product))
        self.w2 = bytes_of(moe.moe_adapters_workspace_size(self.adapters))

    def __call__(self, x, residual, which):
        moe.moe_norm_forward(self.norm, x, residual, self.weight, self.h, self.y, self.codes, self.scales)
        moe.moe_matmul_fp8(self.product, self.codes, self.scales, self.wq, self.ws, self.base, self.w1)
        moe.moe_adapters(self.adapters, self.y, which, self.a, self.b, self.scale, None, self.base, self.out, self.w2)


def serve_inputs(T, d, adapters, g):
    x, res = (torch.randn(T, d, device="cuda", generator=g).to(BF16) for _ in range(2))
    return x, res, torch.randint(-1, adapters, (T,), device="cuda", generator=g).to(torch.int32)


@pytest.mark.parametrize("T", [1, 24, 300])
def test_a_serving_step_against_float64_and_in_a_graph(T):
    """The product on the norm's codes (bf16: 2^-8 of the value, 2^-10 of its terms), the adapters on its y and on the
    product (their own bounds).  Then captured: replays on new inputs are the eager step, bit for bit."""
    d, out, n, r = 512, 384, 5, 16
    blk = ServeBlock(T, d, out, n, r, 7)
    g = torch.Generator("cuda").manual_seed(8)
    make = lambda: serve_inputs(T, d, n, g)  # noqa: E731
    x, res, which = make()
    blk(x, res, which)
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    base, size = P.matmul_fp8("forward", f(blk.codes), f(blk.scales), f(blk.wq), f(blk.ws))
    assert (np.abs(f(blk.base) - base) <= 2.0 ** -8 * np.abs(base) + 2.0 ** -10 * size).all()
    ref, low = B.adapters(f(blk.y), which.cpu().numpy(), f(blk.a), f(blk.b), f(blk.scale), None, f(blk.base))
    tol = 2.0 ** -8 * np.abs(ref) + ((d + 3 * r + 16) * 2.0 ** -24 + 2.0 ** -16) * low + 1e-30
    assert (np.abs(f(blk.out) - ref) <= tol).all()
    got = torch.empty_like(blk.out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk(x, res, which)
        got.copy_(blk.out)
    for _ in range(4):
        for t, v in zip((x, res, which), make()):
            t.copy_(v)
        blk(x, res, which)
        want = blk.out.clone()
        blk.w2.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_two_graphs_that_share_a_workspace():
    """Captured one after the other on one workspace and replayed in turn on one stream."""
    blk = ServeBlock(40, 512, 384, 5, 64, 9)
    g = torch.Generator("cuda").manual_seed(10)
    sets = [serve_inputs(40, 512, 5, g) for _ in range(2)]
    want, got, graphs = [], [torch.empty_like(blk.out) for _ in sets], []
    for s, o in zip(sets, got):
        blk(*s)
        want.append(blk.out.clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            blk(*s)
            o.copy_(blk.out)
    for _ in range(3):
        for k in (0, 1):
            graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
