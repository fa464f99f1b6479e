"""moe_matmul_fp8 and moe_quantize_act_t on the GPU against float64.

Tolerances.  fp32 outputs are exact products summed in fp32: each of the k + 2 k / 128 roundings is at most 2^-24 of the
sum S of the products' magnitudes so far, so the error stays below (k + 64) 2^-24 S.  bf16 outputs come from the FP8
matrix instruction, where each of eight products added together keeps 13 bits below the largest: 8 * 2^-13 = 2^-10 of S
at the very most (and 2^-8 of the value for the rounding to bf16); over a whole matrix the errors are random, and the
relative error of the matrix stays near bf16's own 1.7e-3: 3e-3 is asked."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from oracle import operators as P  # noqa: E402

F8 = torch.float8_e4m3fn
FORMS = {"forward": moe.MOE_FP8_FORWARD, "input_grad": moe.MOE_FP8_INPUT_GRAD, "weight_grad": moe.MOE_FP8_WEIGHT_GRAD}


def codes(rows, cols, g, ld=None):
    """E4M3 codes of every size (subnormal ones too), rows ld apart."""
    v = torch.randn(rows, ld or cols, device="cuda", generator=g) * torch.exp2(
        torch.randint(-6, 7, (rows, 1), device="cuda", generator=g).float())
    return v.clamp(-448, 448).to(F8)[:, :cols]


def operands(form, m, n, k, g, lda=0, ldb=0):
    a = codes(m, k, g, lda)
    b = codes(k, n, g, ldb) if form == "input_grad" else codes(n, k, g, ldb)
    nb = -(-n // 128)
    shape = {"forward": (nb, k // 128), "input_grad": (k // 128, nb), "weight_grad": (n, k // 128)}[form]
    scale = lambda *s: torch.exp2(torch.rand(*s, device="cuda", generator=g) * 6 - 5)  # noqa: E731
    return a, scale(m, k // 128), b, scale(*shape)


def product(form, m, n, k, a, sa, b, sb, f32, lda=0, ldb=0, ldo=0, out=None, accumulate=False, stream=None):
    shape = moe.make_matmul_shape(m, n, k, FORMS[form], moe.MOE_DTYPE_F32 if f32 else moe.MOE_DTYPE_BF16, accumulate,
                                  lda, ldb, ldo)
    ws = torch.full((max(1, moe.moe_matmul_fp8_workspace_size(shape)),), 0xFF, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((m, n), float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    moe.moe_matmul_fp8(shape, a, sa, b, sb, out, ws, stream)
    return out


def check(out, form, a, sa, b, sb, f32, before=None):
    ref, size = P.matmul_fp8(form, a.float().cpu().numpy(), sa.cpu().numpy(), b.float().cpu().numpy(), sb.cpu().numpy())
    if before is not None:
        ref = ref + before
        size = size + np.abs(before)
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    if f32:
        assert (err <= (a.shape[1] + 64) * 2.0 ** -24 * size).all()
    else:
        assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * size).all()
        assert np.linalg.norm(err) <= 3e-3 * np.linalg.norm(ref)


SIZES = [(1, 16, 128), (1, 4096, 256), (16, 144, 1152), (17, 128, 2048), (31, 272, 384), (33, 64, 512), (64, 112, 1024),
         (65, 400, 640), (77, 1040, 2048), (128, 128, 128), (129, 256, 256), (300, 528, 896), (1000, 272, 384),
         (257, 2064, 1536), (2100, 2320, 256)]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_against_float64(size, form, f32):
    g = torch.Generator("cuda").manual_seed(sum(size))
    ops = operands(form, *size, g)
    check(product(form, *size, *ops, f32), form, *ops, f32)


# every tile, alone and with the contraction split, and rows left over from whole tiles
LARGER = [("forward", False, 1, 16, 2176), ("forward", True, 1, 16, 2432), ("forward", False, 25, 16, 2176),
          ("forward", True, 25, 16, 2304), ("forward", False, 2710, 752, 128), ("forward", True, 775, 2512, 128),
          ("forward", False, 2783, 2848, 1024), ("forward", True, 1695, 2576, 128), ("forward", True, 2213, 928, 2176),
          ("forward", False, 1537, 2624, 128), ("forward", False, 2987, 2800, 256), ("forward", True, 2696, 2800, 256),
          ("forward", True, 1690, 1184, 1408), ("forward", False, 7319, 2208, 768),
          ("input_grad", False, 703, 2992, 128), ("input_grad", True, 670, 2992, 128),
          ("input_grad", False, 2707, 2944, 1280), ("input_grad", True, 2325, 1824, 128),
          ("input_grad", True, 1162, 1760, 2304), ("input_grad", False, 1799, 2272, 128),
          ("input_grad", False, 2949, 3040, 1280), ("input_grad", True, 2847, 2912, 128), ("input_grad", False, 1, 16, 2816),
          ("input_grad", True, 11002, 144, 3456), ("input_grad", False, 2428, 6880, 640),
          ("weight_grad", False, 2345, 864, 128), ("weight_grad", True, 671, 3040, 128),
          ("weight_grad", False, 2738, 2832, 896), ("weight_grad", True, 1722, 2448, 128),
          ("weight_grad", True, 2718, 736, 2304), ("weight_grad", False, 2370, 1744, 128),
          ("weight_grad", True, 2933, 3008, 1408), ("weight_grad", True, 4852, 3424, 384),
          ("weight_grad", False, 1176, 6992, 1408), ("weight_grad", False, 1, 16, 2688),
          ("forward", False, 1, 16, 5120), ("forward", False, 67, 4992, 5120), ("forward", False, 69, 4080, 2432),
          ("forward", False, 772, 5920, 768), ("forward", True, 1, 16, 4864), ("forward", True, 132, 752, 3584),
          ("forward", True, 133, 5504, 2816), ("forward", True, 3443, 2528, 896), ("forward", True, 68, 4560, 3200),
          ("forward", True, 71, 4224, 3968), ("input_grad", False, 199, 4368, 4992),
          ("input_grad", False, 21, 2128, 3584), ("input_grad", False, 2375, 1680, 896),
          ("input_grad", True, 1283, 6256, 384), ("input_grad", True, 3074, 2816, 896),
          ("input_grad", True, 44, 3936, 2048), ("input_grad", True, 65, 4448, 3968),
          ("input_grad", True, 65, 5024, 3200), ("weight_grad", False, 12, 5040, 2688),
          ("weight_grad", False, 8366, 80, 4224), ("weight_grad", True, 147, 1200, 2048),
          ("weight_grad", True, 65, 4336, 3584), ("weight_grad", True, 66, 4144, 3968),
          ("forward", False, 198, 4112, 4992), ("forward", False, 845, 4688, 896), ("forward", False, 17, 400, 3200),
          ("forward", True, 66, 4112, 3712), ("input_grad", True, 65, 4592, 3584),
          ("forward", False, 475, 4192, 256), ("forward", False, 1000, 2816, 1024), ("input_grad", False, 8687, 208, 256),
          ("weight_grad", False, 540, 3696, 256),
          # two sets of wavefronts, the last slice a single K block
          ("input_grad", False, 25, 2272, 4736), ("forward", True, 65, 2736, 5248), ("weight_grad", False, 28, 2000, 5504),
          ("weight_grad", True, 384, 336, 4736), ("input_grad", True, 186, 704, 4736)]


@pytest.mark.parametrize("case", LARGER, ids=lambda c: "-".join(map(str, c)))
def test_larger_sizes(case):
    """As test_against_float64, the float64 product computed on the GPU."""
    form, f32, m, n, k = case
    a, sa, b, sb = operands(form, m, n, k, torch.Generator("cuda").manual_seed(m + n + k))
    out = product(form, m, n, k, a, sa, b, sb, f32).double()
    wide = lambda s, cols: s.double().repeat_interleave(128, 1)[:, :cols]  # noqa: E731
    x, y = a.double() * wide(sa, k), wide(sb, b.shape[1])
    if form != "weight_grad":
        y = y.repeat_interleave(128, 0)[:b.shape[0]]
    y = y * b.double()
    y = y if form == "input_grad" else y.t().contiguous()
    ref, size = x @ y, x.abs() @ y.abs()
    err = (out - ref).abs()
    if f32:
        assert (err <= (k + 64) * 2.0 ** -24 * size).all()
    else:
        assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * size).all()
        assert err.norm() <= 3e-3 * ref.norm()


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("m", [5, 200, 2100])
def test_rows_apart_and_accumulating(m, form, f32):
    n, k = 272, 384
    g = torch.Generator("cuda").manual_seed(m)
    lda, ldb, ldo = k + 48, (n if form == "input_grad" else k) + 32, n + 20
    a, sa, b, sb = operands(form, m, n, k, g, lda, ldb)
    wide = torch.randn(m, ldo, device="cuda", generator=g).to(torch.float32 if f32 else torch.bfloat16)
    before = wide.clone()
    product(form, m, n, k, a, sa, b, sb, f32, lda, ldb, ldo, out=wide, accumulate=True)
    check(wide[:, :n], form, a, sa, b, sb, f32, before[:, :n].double().cpu().numpy())
    assert torch.equal(wide[:, n:], before[:, n:])


@pytest.mark.parametrize("form", list(FORMS))
def test_empty_contraction_and_empty_output(form):
    g = torch.Generator("cuda").manual_seed(1)
    a, sa, b, sb = operands(form, 40, 32, 128, g)
    for f32 in (False, True):
        out = product(form, 40, 32, 0, a, sa, b, sb, f32)
        assert (out == 0).all()
        product(form, 0, 32, 128, a, sa, b, sb, f32, out=out)
        product(form, 40, 0, 128, a, sa, b, sb, f32, out=out)
        assert (out == 0).all()


@pytest.mark.parametrize("m", [3, 90, 600])
def test_nan_stays_in_its_row_and_column(m):
    """A NaN code reaches its row (of a) or column (of b), nothing else."""
    n, k = 256, 512
    g = torch.Generator("cuda").manual_seed(9)
    for f32 in (False, True):
        a, sa, b, sb = operands("forward", m, n, k, g)
        a.view(torch.uint8)[1, 300] = 0x7F
        b.view(torch.uint8)[77, 5] = 0x7F
        bad = torch.isnan(product("forward", m, n, k, a, sa, b, sb, f32))
        want = torch.zeros_like(bad)
        want[1], want[:, 77] = True, True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 256, 7168), (77, 7168, 2048), (600, 512, 1024), (4096, 2048, 512)],
                         ids=lambda s: "x".join(map(str, s)))
def test_same_bits_again_on_another_stream(size, f32):
    g = torch.Generator("cuda").manual_seed(2)
    ops = operands("forward", *size, g)
    first = product("forward", *size, *ops, f32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = product("forward", *size, *ops, f32, stream=side)
    side.synchronize()
    assert torch.equal(first, again)


@pytest.mark.parametrize("form", ["forward", "input_grad"])
def test_offsets_past_32_bits(form):
    """More than 2^32 bytes of a (and, in the input gradient's case, of b): the last rows as they come out alone."""
    m, n, k = 300, 128, 128
    ld = (1 << 24) - 16
    g = torch.Generator("cuda").manual_seed(4)
    a, sa, b, sb = operands(form, m, n, k, g)
    far = torch.zeros(m, ld, dtype=torch.uint8, device="cuda")
    far[:, :k] = a.view(torch.uint8)
    want = product(form, m, n, k, a, sa, b, sb, False)
    assert torch.equal(product(form, m, n, k, far, sa, b, sb, False, lda=ld), want)
    if form == "input_grad":
        a, sa, b, sb = operands(form, m, n, 384, g)
        far = torch.zeros(384, ld, dtype=torch.uint8, device="cuda")
        far[:, :n] = b.view(torch.uint8)
        want = product(form, m, n, 384, a, sa, b, sb, False)
        assert torch.equal(product(form, m, n, 384, a, sa, far, sb, False, ldb=ld), want)


@pytest.mark.parametrize("rows,cols", [(1, 8), (127, 64), (128, 72), (129, 200), (1000, 136), (300, 4104)])
def test_quantize_act_t(rows, cols):
    g = torch.Generator("cuda").manual_seed(rows + cols)
    x = (torch.randn(rows, cols, device="cuda", generator=g) * 3).bfloat16()
    x[:, 1] = 0                                  # a run of zeros
    x[0, 2] = 1e-39                              # a subnormal maximum
    x[1:, 2] = 0
    pad = -(-rows // 128) * 128
    q = torch.full((cols, pad), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((cols, pad // 128), float("nan"), device="cuda")
    moe.moe_quantize_act_t(rows, cols, x, q, s)
    v = np.zeros((cols, pad), np.float32)
    v[:, :rows] = x.float().cpu().numpy().T
    want = P.run_scales(v, 448)
    assert np.array_equal(s.cpu().numpy(), want)
    quot = (v.reshape(cols, -1, 128) / want[:, :, None]).reshape(cols, pad)
    codes = torch.from_numpy(np.clip(quot, -448, 448)).to(F8).view(torch.uint8)
    assert torch.equal(q.cpu(), codes)


def test_weight_gradient_of_a_linear_layer():
    """dW = dy^T x from the transposing quantiser, over a ragged batch: against the float64 product of what the
    codes stand for, and near the product of the bf16 values (E4M3 keeps 4 bits: 2.6% a value, random)."""
    T, n, d = 500, 144, 256
    g = torch.Generator("cuda").manual_seed(6)
    dy = torch.randn(T, n, device="cuda", generator=g).bfloat16()
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    q = []
    for v in (dy, x):
        c = torch.empty(v.shape[1], 512, dtype=F8, device="cuda")
        s = torch.empty(v.shape[1], 4, device="cuda")
        moe.moe_quantize_act_t(T, v.shape[1], v, c, s)
        q += [c, s]
    out = product("weight_grad", n, d, 512, *q, True)
    check(out, "weight_grad", *q, True)
    ref = dy.double().t() @ x.double()
    assert ((out.double() - ref).norm() / ref.norm()).item() < 0.06


def test_replayed_in_a_graph():
    m, n, k = 200, 512, 2048     # a split contraction: two kernels
    g = torch.Generator("cuda").manual_seed(8)
    a, sa, b, sb = operands("forward", m, n, k, g)
    shape = moe.make_matmul_shape(m, n, k, moe.MOE_FP8_FORWARD, moe.MOE_DTYPE_BF16)
    ws = torch.empty(moe.moe_matmul_fp8_workspace_size(shape), dtype=torch.uint8, device="cuda")
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    moe.moe_matmul_fp8(shape, a, sa, b, sb, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_matmul_fp8(shape, a, sa, b, sb, out, ws)
    for seed in range(4):
        sa.copy_(torch.rand(sa.shape, device="cuda", generator=g))
        moe.moe_matmul_fp8(shape, a, sa, b, sb, out, ws)
        want = out.clone()
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
