"""The FP8 quantisers beside each other, on the GPU: the transposing one gives what the plain one gives for the
transposed matrix, to the bit."""
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
def test_transposed_codes_are_those_of_the_transpose(rows, cols):
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
    assert torch.equal(s, s2)
    number = (q2 & 0x7F) != 0x7F                 # (a NaN's sign says nothing)
    assert torch.equal(number, (q & 0x7F) != 0x7F) and torch.equal(q[number], q2[number])
