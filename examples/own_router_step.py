"""Training a block whose router is a softmax of its own: a dense FP8 FFN, then a mixture-of-experts layer.

    python examples/own_router_step.py            (one MI355X; random data, a few seconds)

The dense FFN runs on moe_matmul_fp8 in its three forms and keeps its SwiGLU inputs in 8 bits; the experts run on
moe_forward_train8 / moe_backward_gates under moe_gate's picks, and moe_gate_backward carries their gradient into the
router.  Buffers are made once and used in every step, as the library leaves all memory to its caller.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixture_experts_layer_adjusted_amd as moe  # noqa: E402

DEV, F8, BF16 = "cuda", torch.float8_e4m3fn, torch.bfloat16


def empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device=DEV)


class Fp8Product:
    """One moe_matmul_fp8 shape with its output and workspace."""

    def __init__(self, m, n, k, form, out_dtype=BF16):
        self.shape = moe.make_matmul_shape(m, n, k, form, moe.MOE_DTYPE_BF16 if out_dtype == BF16 else moe.MOE_DTYPE_F32)
        self.out = empty(m, n, dtype=out_dtype)
        self.ws = empty(max(1, moe.moe_matmul_fp8_workspace_size(self.shape)), dtype=torch.uint8)

    def __call__(self, a, b):
        moe.moe_matmul_fp8(self.shape, *a, *b, self.out, self.ws)
        return self.out


class Runs:
    """E4M3 codes and scales of a [rows, cols] activation in runs of 128 along its rows, or transposed."""

    def __init__(self, rows, cols, transposed=False):
        self.rows, self.cols, self.transposed = rows, cols, transposed
        r, c = (cols, -(-rows // 128) * 128) if transposed else (rows, cols)
        self.codes, self.scales = empty(r, c, dtype=F8), empty(r, c // 128)

    def __call__(self, x):
        (moe.moe_quantize_act_t if self.transposed else moe.moe_quantize_act)(self.rows, self.cols, x, self.codes,
                                                                            self.scales)
        return self.codes, self.scales


class DenseFfn:
    """y = x + (silu(x Wg^T) * (x Wu^T)) Wd^T with Wg and Wu stacked in w1 [2I, d] and Wd = w2 [d, I]."""

    def __init__(self, tokens, d, inter, gen):
        T, I = tokens, inter
        self.T, self.d, self.I = T, d, I
        self.w1 = torch.randn(2 * I, d, device=DEV, generator=gen) / d ** 0.5
        self.w2 = torch.randn(d, I, device=DEV, generator=gen) / I ** 0.5
        self.q1 = (empty(2 * I, d, dtype=F8), empty(2 * I // 128, d // 128))
        self.q2 = (empty(d, I, dtype=F8), empty(d // 128, I // 128))
        self.up = Fp8Product(T, 2 * I, d, moe.MOE_FP8_FORWARD)
        self.down = Fp8Product(T, d, I, moe.MOE_FP8_FORWARD)
        self.d_h = Fp8Product(T, I, d, moe.MOE_FP8_INPUT_GRAD)
        self.d_x = Fp8Product(T, d, 2 * I, moe.MOE_FP8_INPUT_GRAD)
        pad = -(-T // 128) * 128
        self.d_w1 = Fp8Product(2 * I, d, pad, moe.MOE_FP8_WEIGHT_GRAD, torch.float32)
        self.d_w2 = Fp8Product(d, I, pad, moe.MOE_FP8_WEIGHT_GRAD, torch.float32)
        self.qx, self.qh, self.qdy, self.qdab = Runs(T, d), Runs(T, I), Runs(T, d), Runs(T, 2 * I)
        self.tx, self.th, self.tdy, self.tdab = (Runs(T, c, True) for c in (d, I, d, 2 * I))
        self.h, self.d_ab = empty(T, I, dtype=BF16), empty(T, 2 * I, dtype=BF16)
        self.saved = (empty(T, 2 * I, dtype=torch.int8), empty(T, 2 * I // 128))

    def forward(self, x):
        moe.moe_quantize_weights(1, 2 * self.I, self.d, self.w1.to(BF16), *self.q1)
        moe.moe_quantize_weights(1, self.d, self.I, self.w2.to(BF16), *self.q2)
        self.x = x
        ab = self.up(self.qx(x), self.q1)
        moe.moe_swiglu_forward8(self.T, self.I, ab, self.h, *self.saved)      # ab and h need not outlive this call
        return x + self.down(self.qh(self.h), self.q2)

    def backward(self, dy):
        d_h = self.d_h(self.qdy(dy), self.q2)
        moe.moe_swiglu_backward8(self.T, self.I, d_h, *self.saved, self.d_ab, self.h)
        self.d_w2(self.tdy(dy), self.th(self.h))
        self.d_w1(self.tdab(self.d_ab), self.tx(self.x))
        return dy + self.d_x(self.qdab(self.d_ab), self.q1)

    def update(self, lr):
        self.w1 -= lr * self.d_w1.out
        self.w2 -= lr * self.d_w2.out


class Experts:
    """The bf16 layer under a softmax router: gates renormalised over the picks, balanced by a bias."""

    def __init__(self, tokens, d, experts, top_k, shared, inter, gen):
        self.shape = moe.make_shape(tokens, d, experts, top_k, shared, inter, moe.MOE_DTYPE_BF16)
        self.cfg = moe.make_gate_config(tokens, experts, top_k, moe.MOE_DTYPE_F32, moe.MOE_SCORE_SOFTMAX)
        self.router = torch.randn(experts, d, device=DEV, generator=gen) / d ** 0.5
        self.bias = torch.zeros(experts, device=DEV)
        self.w = [(torch.randn(n, *s, device=DEV, generator=gen) / s[1] ** 0.5).to(BF16)
                  for n in (experts, shared) for s in ((inter, d), (inter, d), (d, inter))]
        self.g = [torch.empty_like(w) for w in self.w]
        self.weights, self.grads = moe.make_weights(*self.w), moe.make_weight_grads(*self.g)
        self.idx, self.gate = empty(tokens, top_k, dtype=torch.int32), empty(tokens, top_k)
        self.load, self.d_gate, self.d_logits = empty(experts, dtype=torch.int32), empty(tokens, top_k), empty(tokens, experts)
        self.out, self.du = empty(tokens, d, dtype=BF16), empty(tokens, d, dtype=BF16)
        u8 = dict(dtype=torch.uint8)
        self.saved = empty(moe.moe_saved8_size(self.shape), **u8)
        self.ws = empty(max(moe.moe_train8_workspace_size(self.shape), moe.moe_backward_workspace_size(self.shape)), **u8)
        self.gate_ws = empty(max(1, moe.moe_gate_workspace_size(self.cfg)), **u8)

    def forward(self, u):
        self.u = u
        self.logits = u.float() @ self.router.t()
        moe.moe_gate(self.cfg, self.logits, self.bias, self.idx, self.gate, self.load, self.gate_ws)
        moe.moe_forward_train8(self.shape, u, self.weights, self.idx, self.gate, self.out, self.saved, self.ws)
        return self.out

    def backward(self, dout):
        moe.moe_backward_gates(self.shape, self.u, self.weights, self.idx, self.gate, self.saved, dout, self.du, self.d_gate,
                               self.grads, self.ws)
        moe.moe_gate_backward(self.cfg, self.logits, self.idx, self.d_gate, self.d_logits)
        self.d_router = self.d_logits.t() @ self.u.float()
        return (self.du.float() + self.d_logits @ self.router).to(BF16)

    def update(self, lr):
        self.router -= lr * self.d_router
        for w, g in zip(self.w, self.g):
            w.sub_(lr * g)
        tokens, top_k = self.idx.shape
        moe.moe_update_bias(self.cfg.n_routed, tokens * top_k, self.load, self.bias, 0.001)


def train(steps=8, tokens=300, d=256, inter=384, experts=16, top_k=4, shared=1, lr=8.0, seed=0):
    """Losses of `steps` steps towards a fixed random target."""
    gen = torch.Generator(DEV).manual_seed(seed)
    ffn, layer = DenseFfn(tokens, d, inter, gen), Experts(tokens, d, experts, top_k, shared, inter, gen)
    x = torch.randn(tokens, d, device=DEV, generator=gen).to(BF16)
    target = torch.randn(tokens, d, device=DEV, generator=gen)
    losses = []
    for _ in range(steps):
        out = layer.forward(ffn.forward(x))
        off = out.float() - target
        losses.append(off.square().mean())
        ffn.backward(layer.backward((2.0 / off.numel() * off).to(BF16)))
        layer.update(lr)
        ffn.update(lr)
    return [float(v) for v in losses]


if __name__ == "__main__":
    for step, loss in enumerate(train()):
        print(f"step {step}: loss {loss:.4f}", flush=True)
