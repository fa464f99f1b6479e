"""The FP8 quantisers on the GPU: the transposing one beside the plain one on the transposed matrix; weights in 16s are
quantised as if filled up with zeros."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402


def quantized(x):
    """moe_quantize_act of x [rows, cols] bf16: codes, scales."""
    rows, cols = x.shape
    q = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, cols // 128), 7.0, device="cuda")
    moe.moe_quantize_act(rows, cols, x, q, s)
    return q, s


@pytest.mark.parametrize("rows,cols", [(128, 8), (100, 128), (1000, 264)])
def test_transposed_codes_beside_those_of_the_transpose(rows, cols):
    """moe_quantize_act_t multiplies by fp32(1/448) where moe_quantize_act divides by 448: scales one unit in the last
    place apart at most, the same codes where they are equal, neighbouring ones where not."""
    g = torch.Generator("cuda").manual_seed(rows)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    x = (x * torch.exp2(torch.randint(-20, 20, (1, cols), device="cuda", generator=g).float())).bfloat16()
    # largest values of every bf16 mantissa, and values at a half between two codes of each
    m = torch.arange(cols, device="cuda") % 128
    x[0] = (448 * (1 + m.float() / 128)).bfloat16()
    x[1:9] = x[0].float() * torch.arange(1, 16, 2, device="cuda")[:, None].float() / 64
    x[:, 2] = 0
    x[20, 3] = float("inf")
    x[21, 4] = float("nan")
    pad = -(-rows // 128) * 128
    q = torch.full((cols, pad), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((cols, pad // 128), 7.0, device="cuda")
    moe.moe_quantize_act_t(rows, cols, x, q, s)
    wide = torch.zeros(pad, cols, dtype=torch.bfloat16, device="cuda")
    wide[:rows] = x
    q2, s2 = quantized(wide.t().contiguous())
    assert (s.view(torch.int32) - s2.view(torch.int32)).abs().max().item() <= 1
    number = (q2 & 0x7F) != 0x7F                 # (a NaN's sign says nothing)
    assert torch.equal(number, (q & 0x7F) != 0x7F)
    apart = (q.int() - q2.int()).abs() * number
    assert apart.max().item() <= 1 and (apart * (s == s2).repeat_interleave(128, 1)).max().item() == 0


@pytest.mark.parametrize("n,rows,cols", [(1, 16, 128), (2, 144, 256), (3, 288, 400), (1, 128, 16), (1, 2320, 384)])
def test_weights_whose_last_blocks_are_smaller(n, rows, cols):
    """A block's codes and scale are those of the same block filled up with zeros."""
    g = torch.Generator("cuda").manual_seed(rows)
    w = torch.randn(n, rows, cols, device="cuda", generator=g).bfloat16()
    rb, cb = -(-rows // 128), -(-cols // 128)
    q = torch.full((n, rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((n, rb, cb), 7.0, device="cuda")
    moe.moe_quantize_weights(n, rows, cols, w, q, s)
    full = torch.zeros(n, rb * 128, cb * 128, dtype=torch.bfloat16, device="cuda")
    full[:, :rows, :cols] = w
    q2, s2 = torch.empty_like(full, dtype=torch.uint8), torch.empty_like(s)
    moe.moe_quantize_weights(n, rb * 128, cb * 128, full, q2, s2)
    assert torch.equal(s, s2) and torch.equal(q, q2[:, :rows, :cols])


def test_product_with_quantised_weights_of_odd_size():
    """Forward and input gradient of a layer whose 144 outputs do not fill their blocks, from the quantisers to the
    product: against float64 of what the codes stand for (fp32 outputs: (k + 64) 2^-24 of the products' magnitudes)."""
    T, n, d = 70, 144, 256
    g = torch.Generator("cuda").manual_seed(2)
    w = (torch.randn(n, d, device="cuda", generator=g) * torch.linspace(0.1, 9, n, device="cuda")[:, None]).bfloat16()
    q = torch.empty(n, d, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(2, 2, device="cuda")
    moe.moe_quantize_weights(1, n, d, w, q, s)
    wide = q.double() * s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    assert ((wide - w.double()).norm() <= 0.05 * w.double().norm()).item()     # (E4M3: 2.6% of a normal value)
    x, xs = quantized(torch.randn(T, d, device="cuda", generator=g).bfloat16())
    out = torch.empty(T, n, device="cuda")
    shape = moe.make_matmul_shape(T, n, d, moe.MOE_FP8_FORWARD, moe.MOE_DTYPE_F32)
    ws = torch.empty(max(1, moe.moe_matmul_fp8_workspace_size(shape)), dtype=torch.uint8, device="cuda")
    moe.moe_matmul_fp8(shape, x, xs, q, s, out, ws)
    a = x.view(torch.float8_e4m3fn).double() * xs.double().repeat_interleave(128, 1)
    y = wide.t().contiguous()
    assert ((out.double() - a @ y).abs() <= (d + 64) * 2.0 ** -24 * (a.abs() @ y.abs())).all()
    # the input gradient contracts over a stored matrix's rows, here 256 of them, and has its 144 columns
    w2 = w.t().contiguous()
    q2, s2 = torch.empty(d, n, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(2, 2, device="cuda")
    moe.moe_quantize_weights(1, d, n, w2, q2, s2)
    wide = q2.double() * s2.double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :n]
    shape = moe.make_matmul_shape(T, n, d, moe.MOE_FP8_INPUT_GRAD, moe.MOE_DTYPE_F32)
    ws = torch.empty(max(1, moe.moe_matmul_fp8_workspace_size(shape)), dtype=torch.uint8, device="cuda")
    moe.moe_matmul_fp8(shape, x, xs, q2, s2, out, ws)
    assert ((out.double() - a @ wide).abs() <= (d + 64) * 2.0 ** -24 * (a.abs() @ wide.abs())).all()
