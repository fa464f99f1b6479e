"""moe_adapters on the GPU at the ends of the number range, in each of its forms.

FORMS: (rows, in, out, adapters, rank) that one kernel takes (few rows and little of A), that go by adapter, and that go by
tiles of neighbouring rows (above 1024 rows in any case)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_adapters import np_, problem, run  # noqa: E402
from oracle import block as B  # noqa: E402

FEW = [(5, 264, 136, 3, 16), (16, 1032, 72, 2, 32)]
BY_ADAPTER = [(40, 264, 200, 6, 24), (33, 520, 136, 8, 8), (60, 264, 328, 9, 64), (48, 264, 72, 7, 128)]
TILES = [(1030, 264, 136, 5, 16), (1025, 72, 264, 3, 32), (1041, 264, 72, 4, 64), (1100, 136, 136, 6, 128)]
FORMS = FEW + BY_ADAPTER + TILES
OUT = [torch.bfloat16, torch.float32]


def check_with_infinities(p, out):
    """The formula's infinities and NaN where it has them, its values elsewhere (bounds: test_gpu_adapters.py)."""
    host = lambda t: t.cpu().numpy()  # noqa: E731
    with np.errstate(invalid="ignore", over="ignore"):
        ref, _ = B.adapters(np_(p["x"]), host(p["which"]), np_(p["a"]), np_(p["b"]), host(p["scale"]),
                            None if p["ranks"] is None else host(p["ranks"]), np_(p["base"]))
        finite_b = np.where(np.isfinite(np_(p["b"])), np_(p["b"]), 0)
        _, size = B.adapters(np_(p["x"]), host(p["which"]), np_(p["a"]), finite_b, host(p["scale"]),
                             None if p["ranks"] is None else host(p["ranks"]), np_(p["base"]))
    got = np_(out).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    inf = np.isinf(ref)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(np.sign(got[inf]), np.sign(ref[inf]))
    d_in, r = p["x"].shape[1], p["a"].shape[1]
    half, kept = (2.0 ** -8, 2.0 ** -16) if p["base"].dtype == torch.bfloat16 else (2.0 ** -24, 2.0 ** -24)
    some = np.isfinite(ref)
    got, ref, size = got[some], ref[some], size[some]
    tol = half * np.abs(ref) + ((d_in + 3 * r + 16) * 2.0 ** -24 + kept) * size + 2.0 ** -22 * np.abs(ref) + 1e-37
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("rows,d_in,d_out,n,r", FORMS)
def test_low_rank_values_near_the_largest(rows, d_in, d_out, n, r, out):
    """Finite sums that bf16 rounds to infinity (above 3.396e38) stay finite."""
    p = problem(rows, d_in, d_out, n, r, rows + r, out)
    p["x"][:] = 0
    p["x"][:, 1] = 3.3895e38                           # (bf16's largest)
    p["x"][:, 2] = 1e36
    p["a"][:] = 0
    p["a"][:, : r // 2, 1:3] = 1
    p["a"][:, r // 2:, 1:3] = -1
    p["b"][:] = (torch.rand(p["b"].shape, device="cuda") + 0.5).bfloat16() * 2.0 ** -100
    p["scale"][:] = 1
    check_with_infinities(p, run(p))


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("rows,d_in,d_out,n,r", FORMS)
def test_an_infinite_weight_makes_an_infinity(rows, d_in, d_out, n, r, out):
    """B's infinities meet low-rank values that bf16 holds (their remainder is zero) and others (their remainder has either
    sign): the value's own sign decides, once."""
    p = problem(rows, d_in, d_out, n, r, rows + r, out)
    p["which"][:] = (torch.arange(rows, device="cuda") % (n + 1)) - 1
    p["a"][:, 0] = 0
    p["a"][:, 0, 0] = 1                                # the first low-rank value is x's first
    p["x"][:, 0] = torch.where(torch.arange(rows, device="cuda") % 3 == 0, -1.5, 2.0).bfloat16()
    p["b"][:, 3, 0] = float("inf")
    p["b"][:, 9, 0] = -float("inf")
    p["b"][:, 17, r // 2] = float("inf")               # (that value is a sum: nonzero)
    p["b"][:, 40, 0] = float("inf")
    p["b"][:, 40, r - 1] = float("nan")
    if n > 1:
        p["b"][1, 50] = torch.where(torch.arange(r, device="cuda") % 2 == 0, float("inf"), -float("inf")).bfloat16()
    check_with_infinities(p, run(p))


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("rows,d_in,d_out,n,r", FORMS)
def test_rows_without_an_adapter_keep_their_bits(rows, d_in, d_out, n, r, out):
    """Whatever they hold: signalling NaN, payloads, the zeros' signs, subnormals."""
    p = problem(rows, d_in, d_out, n, r, rows + r, out)
    p["which"][::2] = -1
    p["which"][1::8] = n
    bits = torch.int16 if out == torch.bfloat16 else torch.int32
    odd = [0x7F81, 0xFFA5, 0x7FC1, 0x8000, 0x0001, 0xFF80] if out == torch.bfloat16 else \
        [0x7F800001, 0xFFA00005, 0x7FC12345, 0x80000000, 0x00000001, 0xFF800000]
    wrap = 1 << (16 if out == torch.bfloat16 else 32)
    values = torch.tensor([v - wrap if v >= wrap // 2 else v for v in odd], dtype=bits, device="cuda")
    none = (p["which"] < 0) | (p["which"] >= n)
    held = p["base"].view(bits)
    held[none] = values[torch.randint(0, 6, (int(none.sum()), d_out), device="cuda")]
    assert torch.equal(run(p).view(bits)[none], held[none])
    in_place = p["base"].clone()
    run({**p, "own": in_place}, base="own", into=in_place)
    assert torch.equal(in_place.view(bits)[none], held[none])
