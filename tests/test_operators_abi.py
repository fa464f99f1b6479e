"""Host-side refusals of the gate, the FP8 product and the 8-bit SwiGLU: the documented status, nothing launched."""
import ctypes

import pytest

import mixture_experts_layer_adjusted_amd as moe
from mixture_experts_layer_adjusted_amd import binding

lib = binding.raw_lib()
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(8)]     # plausible, never dereferenced
BIG = ctypes.c_size_t(1 << 40)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def gate(**kw):
    d = dict(tokens=100, n_routed=64, top_k=4, logits_dtype=0, score=0, n_groups=1, topk_groups=1, group_score=0,
             renormalize=True, scale=1.0, logits_ld=0)
    d.update(kw)
    return moe.make_gate_config(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), INVALID), (dict(n_routed=0), INVALID), (dict(top_k=0), INVALID), (dict(top_k=65), INVALID),
    (dict(logits_dtype=2), INVALID), (dict(score=2), INVALID), (dict(group_score=-1), INVALID),
    (dict(n_groups=0), INVALID), (dict(n_groups=3), INVALID), (dict(n_groups=4, topk_groups=5), INVALID),
    (dict(n_groups=4, topk_groups=0), INVALID), (dict(n_groups=32, topk_groups=1), INVALID),
    (dict(n_routed=512, n_groups=128), INVALID), (dict(logits_ld=63), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(n_routed=513), UNSUPPORTED), (dict(top_k=33), UNSUPPORTED),
    (dict(tokens=1 << 30), UNSUPPORTED), (dict(), OK), (dict(logits_ld=64, n_groups=64, topk_groups=4), OK),
])
def test_gate_limits(kw, status):
    c, n = gate(**kw), ctypes.c_size_t(0)
    assert lib.moe_gate_workspace_size(ctypes.byref(c), ctypes.byref(n)) == status
    if status:
        assert lib.moe_gate(ctypes.byref(c), P[0], P[1], P[2], P[3], P[4], P[5], BIG, None) == status
        assert lib.moe_gate_backward(ctypes.byref(c), P[0], P[1], P[2], P[3], 0, None) == status


def test_gate_pointers_and_workspace():
    c, n = gate(), ctypes.c_size_t(0)
    assert lib.moe_gate_workspace_size(ctypes.byref(c), None) == INVALID
    assert lib.moe_gate_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.moe_gate_workspace_size(ctypes.byref(c), ctypes.byref(n)) == OK and n.value > 0
    call = lambda *a: lib.moe_gate(ctypes.byref(c), *a, None)  # noqa: E731
    for i in (0, 2, 3):
        a = [P[0], P[1], P[2], P[3], P[4], P[5], BIG]
        a[i] = None
        assert call(*a) == INVALID
    assert call(P[0], P[1], P[2], P[3], P[4], P[5], ctypes.c_size_t(n.value - 1)) == WORKSPACE
    assert call(P[0], P[1], P[2], P[3], P[4], None, BIG) == INVALID
    back = lambda *a: lib.moe_gate_backward(ctypes.byref(c), *a, None)  # noqa: E731
    assert back(P[0], P[1], P[2], P[0], 0) == INVALID            # in place
    assert back(P[0], P[1], P[2], P[3], 63) == INVALID
    for i in range(4):
        a = list(P[:4])
        a[i] = None
        assert back(*a, 0) == INVALID
    none = gate(tokens=0)
    assert lib.moe_gate(ctypes.byref(none), None, None, None, None, None, None, 0, None) == OK
    assert lib.moe_gate_backward(ctypes.byref(none), None, None, None, None, 0, None) == OK


@pytest.mark.parametrize("args,kw,status", [
    ((-1, 32, 128, 0, 1), {}, INVALID), ((4, 32, 128, 3, 1), {}, INVALID), ((4, 32, 128, 0, 2), {}, INVALID),
    ((4, 32, 128, 0, 1), dict(lda=112), INVALID), ((4, 32, 128, 1, 1), dict(ldb=16), INVALID),
    ((4, 32, 128, 0, 1), dict(ldo=28), INVALID), ((4, 24, 128, 0, 1), {}, UNSUPPORTED),
    ((4, 32, 64, 0, 1), {}, UNSUPPORTED), ((4, 32, 128, 0, 1), dict(lda=136), UNSUPPORTED),
    ((4, 32, 128, 0, 1), dict(ldb=1 << 24), UNSUPPORTED), ((4, 32, 128, 0, 1), dict(ldo=34), UNSUPPORTED),
    (((1 << 31) - 1, 1 << 24, 128, 0, 1), {}, UNSUPPORTED),
    ((4, 32, 128, 0, 1), {}, OK), ((4, 32, 128, 1, 0), dict(ldb=48), OK), ((0, 0, 0, 2, 0), {}, OK),
])
def test_matmul_limits(args, kw, status):
    s, n = moe.make_matmul_shape(*args, **kw), ctypes.c_size_t(0)
    assert lib.moe_matmul_fp8_workspace_size(ctypes.byref(s), ctypes.byref(n)) == status
    if status:
        assert lib.moe_matmul_fp8(ctypes.byref(s), P[0], P[1], P[2], P[3], P[4], P[5], BIG, None) == status


def test_matmul_pointers_and_workspace():
    s, n = moe.make_matmul_shape(200, 512, 8192, moe.MOE_FP8_FORWARD, moe.MOE_DTYPE_BF16), ctypes.c_size_t(0)
    assert lib.moe_matmul_fp8_workspace_size(ctypes.byref(s), ctypes.byref(n)) == OK and n.value > 0   # split
    call = lambda *a: lib.moe_matmul_fp8(ctypes.byref(s), *a, None)  # noqa: E731
    assert call(*P[:6], ctypes.c_size_t(n.value - 1)) == WORKSPACE
    assert call(*P[:5], None, BIG) == INVALID
    for i in range(5):
        a = list(P[:6])
        a[i] = None
        assert call(*a, BIG) == INVALID
    for i in (0, 2, 4):
        a = list(P[:6])
        a[i] = ctypes.c_void_p(a[i].value + 8)                                # not 16-byte aligned
        assert call(*a, BIG) == INVALID
    assert call(P[0], P[1], P[2], P[3], P[0], P[5], BIG) == INVALID           # out is a
    assert lib.moe_matmul_fp8_workspace_size(ctypes.byref(s), None) == INVALID
    empty = moe.make_matmul_shape(0, 512, 128, moe.MOE_FP8_FORWARD, moe.MOE_DTYPE_BF16)
    assert lib.moe_matmul_fp8(ctypes.byref(empty), None, None, None, None, None, None, 0, None) == OK


def test_quantize_act_t_and_swiglu8():
    q = lambda r, c, *a: lib.moe_quantize_act_t(r, c, *a, None)  # noqa: E731
    assert q(-1, 8, *P[:3]) == INVALID and q(4, 12, *P[:3]) == UNSUPPORTED and q(4, 8 << 20, *P[:3]) == UNSUPPORTED
    assert q(4, 8, None, P[1], P[2]) == INVALID and q(0, 8, None, None, None) == OK
    f = lambda r, i, *a: lib.moe_swiglu_forward8(r, i, *a, None)  # noqa: E731
    assert f(-1, 128, *P[:4]) == INVALID and f(4, 192, *P[:4]) == UNSUPPORTED and f(0, 128, *[None] * 4) == OK
    for i in (0, 2, 3):
        a = list(P[:4])
        a[i] = None
        assert f(4, 128, *a) == INVALID
    assert f(4, 128, P[0], P[0], P[2], P[3]) == INVALID and f(4, 128, P[0], P[1], P[0], P[3]) == INVALID
    b = lambda r, i, *a: lib.moe_swiglu_backward8(r, i, *a, None)  # noqa: E731
    assert b(4, -128, *P[:5]) == INVALID and b(4, 64, *P[:5]) == UNSUPPORTED and b(4, 0, *[None] * 5) == OK
    for i in range(4):
        a = list(P[:5])
        a[i] = None
        assert b(4, 128, *a) == INVALID
    assert b(4, 128, P[0], P[1], P[2], P[1], P[4]) == INVALID and b(4, 128, P[0], P[1], P[2], P[3], P[0]) == INVALID


def test_weights_in_16s_can_be_quantised():
    """Every n that moe_matmul_fp8 takes."""
    w = lambda n, r, c: lib.moe_quantize_weights(n, r, c, None, None, None, None)  # noqa: E731
    assert w(0, 144, 256) == OK and w(0, 128, 16) == OK
    assert w(1, 144, 256) == INVALID and w(1, 136, 128) == UNSUPPORTED and w(1, 128, 24) == UNSUPPORTED


def test_swiglu8_outputs_in_one_place():
    """The codes and h may not share a buffer (both are written, by different lanes)."""
    assert lib.moe_swiglu_forward8(4, 128, P[0], P[1], P[1], P[3], None) == INVALID
    assert lib.moe_swiglu_backward8(4, 128, P[0], P[1], P[2], P[3], P[3], None) == INVALID
    assert lib.moe_swiglu_backward8(4, 128, P[0], P[1], P[2], P[3], P[1], None) == INVALID


def test_layer_under_a_given_router():
    sb = moe.make_shape(300, 256, 16, 4, 1, 128, moe.MOE_DTYPE_BF16)
    s32 = moe.make_shape(300, 256, 16, 4, 1, 128, moe.MOE_DTYPE_F32)
    n, m = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert lib.moe_saved8_size(ctypes.byref(sb), ctypes.byref(n)) == OK
    rows = 128 * ((300 * 4 + 16 * 127) // 128 + 3)
    assert n.value == rows * 256 + rows * 2 * 4                     # codes (a multiple of 256 bytes), scales
    assert lib.moe_saved8_size(ctypes.byref(s32), ctypes.byref(n)) == UNSUPPORTED
    assert lib.moe_saved8_size(ctypes.byref(sb), None) == INVALID
    assert lib.moe_workspace_size(ctypes.byref(sb), ctypes.byref(m)) == OK
    t8 = ctypes.c_size_t(0)
    assert lib.moe_train8_workspace_size(ctypes.byref(sb), ctypes.byref(t8)) == OK and t8.value == m.value   # 2I <= d
    wide = moe.make_shape(300, 256, 16, 4, 1, 256, moe.MOE_DTYPE_BF16)
    assert lib.moe_workspace_size(ctypes.byref(wide), ctypes.byref(m)) == OK
    assert lib.moe_train8_workspace_size(ctypes.byref(wide), ctypes.byref(t8)) == OK
    assert t8.value == m.value + rows * 512 * 2
    w = moe.Weights(*(0x10000,) * 6)
    fwd = lambda s, sv, sb_, wsb: lib.moe_forward_train8(  # noqa: E731
        ctypes.byref(s), P[0], ctypes.byref(w), P[1], P[2], P[3], sv, sb_, P[5], wsb, None)
    assert fwd(sb, None, BIG, BIG) == INVALID and fwd(sb, P[4], 16, BIG) == WORKSPACE
    assert fwd(sb, P[0], BIG, BIG) == INVALID and fwd(sb, P[4], BIG, 16) == WORKSPACE
    assert fwd(sb, ctypes.c_void_p(P[4].value + 8), BIG, BIG) == INVALID and fwd(s32, P[4], BIG, BIG) == UNSUPPORTED
    wg = moe.WeightGrads(*(0x70000,) * 6)
    bwd = lambda s, sv, sb_, du, dg, wsb: lib.moe_backward_gates(  # noqa: E731
        ctypes.byref(s), P[0], ctypes.byref(w), P[1], P[2], sv, sb_, P[3], du, dg, ctypes.byref(wg), P[5], wsb, None)
    assert bwd(sb, None, 0, P[4], None, BIG) == INVALID and bwd(sb, None, 0, None, P[6], BIG) == INVALID
    assert bwd(sb, P[7], 16, P[4], P[6], BIG) == WORKSPACE and bwd(sb, P[7], BIG, P[7], P[6], BIG) == INVALID
    assert bwd(sb, None, 0, P[0], P[6], BIG) == INVALID and bwd(sb, None, 0, P[4], P[6], 16) == WORKSPACE
    assert bwd(s32, None, 0, P[4], P[6], BIG) == UNSUPPORTED


def test_misaligned_pointers():
    off = lambda i: ctypes.c_void_p(P[i].value + 8)  # noqa: E731
    assert lib.moe_quantize_act_t(4, 8, off(0), P[1], P[2], None) == INVALID
    assert lib.moe_swiglu_forward8(4, 128, P[0], off(1), P[2], P[3], None) == INVALID
    assert lib.moe_swiglu_backward8(4, 128, P[0], P[1], P[2], off(3), P[4], None) == INVALID
