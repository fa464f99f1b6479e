"""The norm of values near the bottom of the range.  E4M3 codes of subnormal runs: a scale that amax / 448 rounds to is never
zero.  Below 448 half steps of fp32's subnormals (3.1e-43) a run counts as zeros: codes of zero under the scale 1."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_norm import forward  # noqa: E402


@pytest.mark.parametrize("stream", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [256, 1152, 2560, 16384])
def test_runs_of_subnormal_values(cols, stream):
    t = torch.float32 if stream == "f32" else torch.bfloat16
    x = torch.randn(5, cols, device="cuda")
    x[:, 0] = 1e4                                        # (rstd well below 1)
    tiny = torch.zeros(5, 128, device="cuda")
    tiny[0, 3] = 1e-43
    tiny[1, ::7] = -9.2e-41
    tiny[2] = 9.2e-41
    tiny[3, 100] = 1.2e-38
    x[:, 128:256] = tiny
    x = x.to(t)
    w = torch.ones(cols, device="cuda")
    out = forward(x, None, w, stream, codes=True)
    y = x.double() / (x.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    codes, scales = out["codes"].double().view(5, -1, 128)[:, 1], out["scales"].double()[:, 1]
    assert torch.isfinite(out["codes"].float()).all() and (out["scales"] > 0).all()
    v = y.view(5, -1, 128)[:, 1]
    # half a step of the code (2^-4 of the value, 2^-10 of the scale); 448 half steps of a subnormal scale, two steps of y
    step = torch.where(scales == 1, 0, scales)[:, None]
    tol = (2.0 ** -4 + 2.0 ** -17) * v.abs() + 2.0 ** -10 * step + 448 * 2.0 ** -150 + 2.0 ** -148
    assert ((codes * scales[:, None] - v).abs() <= tol).all()
    assert (codes[tiny == 0] == 0).all()


def test_squares_that_are_zero_without_an_eps():
    x = torch.full((4, 264), 1e-25, device="cuda")
    x[1] = 0
    x[2, 5] = 1.0
    x[3] = 1e-15
    out = forward(x, None, torch.ones(264, device="cuda"), "f32", eps=0.0)
    assert torch.isposinf(out["y"][0]).all() and torch.isposinf(out["rstd"][0]) and torch.isnan(out["y"][1]).all()
    assert torch.allclose(out["y"][2, 5], torch.tensor(264.0, device="cuda").sqrt(), rtol=2.0 ** -20)
    assert torch.allclose(out["y"][3], torch.ones(264, device="cuda"), rtol=2.0 ** -18)
