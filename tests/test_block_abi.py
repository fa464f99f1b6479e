"""Host-side refusals of the norm, the balance loss and the adapters: the documented status, nothing launched."""
import ctypes

import pytest

import mixture_experts_layer_adjusted_amd as moe
from mixture_experts_layer_adjusted_amd import binding

lib = binding.raw_lib()
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(12)]     # plausible, never dereferenced
BIG = ctypes.c_size_t(1 << 40)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def off(p, n=8):
    return ctypes.c_void_p(p.value + n)


def with_none(args, i):
    a = list(args)
    a[i] = None
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(dtype=2), INVALID), (dict(eps=-1e-6), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x_ld=248), INVALID),
    (dict(y_ld=128), INVALID), (dict(x_ld=-8), INVALID), (dict(cols=12), UNSUPPORTED), (dict(cols=32776), UNSUPPORTED),
    (dict(x_ld=260), UNSUPPORTED), (dict(y_ld=257), UNSUPPORTED), (dict(), OK), (dict(x_ld=264, y_ld=512, eps=0.0), OK),
    (dict(cols=32768), OK), (dict(rows=0), OK),
])
def test_norm_limits(kw, status):
    d = dict(rows=10, cols=256, dtype=1, eps=1e-6, x_ld=0, y_ld=0)
    d.update(kw)
    s, n = moe.make_norm_shape(**d), ctypes.c_size_t(0)
    assert lib.moe_norm_workspace_size(ctypes.byref(s), ctypes.byref(n)) == status
    if status:
        assert lib.moe_norm_forward(ctypes.byref(s), *P[:8], None) == status
        assert lib.moe_norm_backward(ctypes.byref(s), *P[:8], BIG, None) == status


def test_norm_pointers():
    s, n = moe.make_norm_shape(10, 256, 1, 1e-6), ctypes.c_size_t(0)
    assert lib.moe_norm_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.moe_norm_workspace_size(ctypes.byref(s), None) == INVALID
    f = lambda *a: lib.moe_norm_forward(ctypes.byref(s), *a, None)  # noqa: E731
    x, r, w, h, y, c, sc, rs = P[:8]
    for i in (0, 2):
        assert f(*with_none(P[:8], i)) == INVALID
    assert f(x, r, w, h, None, None, None, rs) == INVALID          # neither y nor codes
    assert f(x, r, w, h, y, c, None, rs) == INVALID and f(x, r, w, h, y, None, sc, rs) == INVALID
    assert f(x, None, w, h, y, c, sc, rs) == INVALID               # a sum of nothing
    for a in ((off(x), r, w, h, y, c, sc, rs), (x, off(r), w, h, y, c, sc, rs), (x, r, off(w), h, y, c, sc, rs),
              (x, r, w, off(h), y, c, sc, rs), (x, r, w, h, off(y), c, sc, rs), (x, r, w, h, y, off(c), sc, rs)):
        assert f(*a) == INVALID
    for a in ((x, r, w, h, x, c, sc, rs), (x, r, w, h, y, r, sc, rs), (x, r, w, h, h, c, sc, rs), (x, r, w, h, y, y, sc, rs),
              (x, r, w, h, y, c, c, rs), (x, r, w, h, y, c, sc, sc), (x, r, w, w, y, c, sc, rs), (x, r, w, h, y, c, sc, w)):
        assert f(*a) == INVALID
    odd = moe.make_norm_shape(10, 264, 1, 1e-6)                    # runs of 128 need whole ones
    assert lib.moe_norm_forward(ctypes.byref(odd), *P[:8], None) == UNSUPPORTED
    none = moe.make_norm_shape(0, 256, 1, 1e-6)
    assert lib.moe_norm_forward(ctypes.byref(none), *[None] * 8, None) == OK
    assert lib.moe_norm_backward(ctypes.byref(none), *[None] * 8, 0, None) == OK


def test_norm_backward_pointers_and_workspace():
    s, n = moe.make_norm_shape(1000, 256, 1, 1e-6), ctypes.c_size_t(0)
    assert lib.moe_norm_workspace_size(ctypes.byref(s), ctypes.byref(n)) == OK and n.value > 0
    b = lambda *a: lib.moe_norm_backward(ctypes.byref(s), *a, None)  # noqa: E731
    dy, ds, h, w, rs, dx, dw, ws = P[:8]
    for i in (0, 2, 3, 4, 5, 7):
        assert b(*with_none(P[:8], i), BIG) == INVALID
    assert b(dy, ds, h, w, rs, dx, dw, ws, ctypes.c_size_t(n.value - 1)) == WORKSPACE
    for a in ((off(dy), ds, h, w, rs, dx, dw, ws), (dy, off(ds), h, w, rs, dx, dw, ws), (dy, ds, off(h), w, rs, dx, dw, ws),
              (dy, ds, h, off(w), rs, dx, dw, ws), (dy, ds, h, w, rs, off(dx), dw, ws), (dy, ds, h, w, rs, dx, dw, off(ws)),
              (dy, ds, h, w, rs, dy, dw, ws), (dy, ds, h, w, rs, h, dw, ws), (dy, ds, h, w, rs, dx, dx, ws),
              (dy, ds, h, w, rs, dx, w, ws), (dy, ds, h, w, rs, dx, ds, ws), (dy, ds, h, w, rs, dx, dw, dx),
              (dy, ds, h, w, rs, dx, dw, h), (dy, ds, h, w, rs, dx, dw, ds), (dy, ds, h, w, rs, dx, dw, dw)):
        assert b(*a, BIG) == INVALID


def balance(**kw):
    d = dict(tokens=100, n_routed=64, top_k=4, logits_dtype=0, score=1, n_seqs=3, alpha=1e-4, logits_ld=0)
    d.update(kw)
    return moe.make_balance_config(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), INVALID), (dict(n_routed=0), INVALID), (dict(top_k=0), INVALID), (dict(top_k=65), INVALID),
    (dict(logits_dtype=2), INVALID), (dict(score=2), INVALID), (dict(n_seqs=0), INVALID), (dict(logits_ld=63), INVALID),
    (dict(alpha=float("inf")), INVALID), (dict(alpha=float("nan")), INVALID), (dict(n_routed=513), UNSUPPORTED),
    (dict(top_k=33), UNSUPPORTED), (dict(tokens=1 << 30), UNSUPPORTED), (dict(), OK), (dict(logits_ld=65, alpha=-1.0), OK),
    (dict(tokens=0), OK), (dict(n_seqs=(1 << 24) + 1), UNSUPPORTED), (dict(n_seqs=1 << 24), OK),
])
def test_balance_limits(kw, status):
    c, n = balance(**kw), ctypes.c_size_t(0)
    assert lib.moe_balance_workspace_size(ctypes.byref(c), ctypes.byref(n)) == status
    if status:
        assert lib.moe_balance_loss(ctypes.byref(c), *P[:8], BIG, None) == status
        assert lib.moe_balance_backward(ctypes.byref(c), *P[:7], 0, 0, None) == status


def test_balance_pointers_and_workspace():
    c, n = balance(tokens=20000), ctypes.c_size_t(0)
    assert lib.moe_balance_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.moe_balance_workspace_size(ctypes.byref(c), None) == INVALID
    assert lib.moe_balance_workspace_size(ctypes.byref(c), ctypes.byref(n)) == OK and n.value > 0
    f = lambda *a: lib.moe_balance_loss(ctypes.byref(c), *a, None)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert f(*with_none(P[:8], i), BIG) == INVALID
    assert f(*P[:8], ctypes.c_size_t(n.value - 1)) == WORKSPACE
    assert f(*P[:7], off(P[7], 4), BIG) == INVALID
    for i in (3, 4, 5, 6, 7):                                      # an output in place of an input, or of another output
        for j in (0, 1, 2, 3 if i != 3 else 4):
            a = list(P[:8])
            a[i] = a[j]
            assert f(*a, BIG) == INVALID
    g = lambda *a: lib.moe_balance_backward(ctypes.byref(c), *a, None)  # noqa: E731
    for i in range(7):
        assert g(*with_none(P[:7], i), 0, 0) == INVALID
    assert all(g(*P[:6], P[j], 0, 0) == INVALID for j in range(6)) and g(*P[:7], 63, 0) == INVALID
    none = balance(tokens=0)
    assert lib.moe_balance_backward(ctypes.byref(none), P[0], P[1], P[2], *[None] * 4, 0, 0, None) == OK
    assert lib.moe_balance_loss(ctypes.byref(none), P[0], P[1], P[2], None, P[4], P[5], None, None, 0, None) == INVALID


def adapters(**kw):
    d = dict(rows=40, in_cols=256, out_cols=512, n_adapters=4, rank=16, out_dtype=1, x_ld=0, base_ld=0, out_ld=0)
    d.update(kw)
    return moe.make_adapter_shape(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(in_cols=0), INVALID), (dict(out_cols=-8), INVALID), (dict(n_adapters=0), INVALID),
    (dict(rank=0), INVALID), (dict(out_dtype=2), INVALID), (dict(x_ld=248), INVALID), (dict(base_ld=8), INVALID),
    (dict(out_ld=504), INVALID), (dict(in_cols=252), UNSUPPORTED), (dict(out_cols=500), UNSUPPORTED),
    (dict(rank=12), UNSUPPORTED), (dict(rank=136), UNSUPPORTED), (dict(in_cols=(1 << 20) + 8), UNSUPPORTED),
    (dict(out_cols=(1 << 20) + 8), UNSUPPORTED), (dict(x_ld=260), UNSUPPORTED), (dict(base_ld=516), UNSUPPORTED),
    (dict(out_ld=513), UNSUPPORTED), (dict(x_ld=1 << 24), UNSUPPORTED), (dict(rows=1 << 27), UNSUPPORTED),
    (dict(rows=(1 << 27) - 1), OK), (dict(x_ld=(1 << 24) - 8), OK), (dict(), OK),
    (dict(rank=128, out_dtype=0, x_ld=264), OK), (dict(rows=0), OK),
])
def test_adapter_limits(kw, status):
    s, n = adapters(**kw), ctypes.c_size_t(0)
    assert lib.moe_adapters_workspace_size(ctypes.byref(s), ctypes.byref(n)) == status
    if status:
        assert lib.moe_adapters(ctypes.byref(s), *P[:9], BIG, None) == status


def test_adapter_pointers_and_workspace():
    byte = lambda p: ctypes.c_void_p(p.value + 2)  # noqa: E731
    s, n = adapters(), ctypes.c_size_t(0)
    assert lib.moe_adapters_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.moe_adapters_workspace_size(ctypes.byref(s), None) == INVALID
    assert lib.moe_adapters_workspace_size(ctypes.byref(s), ctypes.byref(n)) == OK and n.value > 0
    f = lambda *a: lib.moe_adapters(ctypes.byref(s), *a, None)  # noqa: E731
    x, wh, a, b, sc, rk, base, out, ws = P[:9]
    for i in (0, 1, 2, 3, 4, 7, 8):
        assert f(*with_none(P[:9], i), BIG) == INVALID
    assert f(*P[:9], ctypes.c_size_t(n.value - 1)) == WORKSPACE
    for q in ((off(x), wh, a, b, sc, rk, base, out, ws), (x, wh, off(a), b, sc, rk, base, out, ws),
              (x, wh, a, off(b), sc, rk, base, out, ws), (x, wh, a, b, sc, rk, off(base), out, ws),
              (x, wh, a, b, sc, rk, base, off(out), ws), (x, wh, a, b, sc, rk, base, out, off(ws)),
              (x, wh, a, b, sc, rk, base, x, ws), (x, wh, a, b, sc, rk, base, a, ws), (x, wh, a, b, sc, rk, base, b, ws),
              (x, wh, a, b, sc, rk, base, ws, ws), (x, wh, a, b, sc, rk, base, wh, ws), (x, wh, a, b, sc, rk, base, sc, ws),
              (x, wh, a, b, sc, rk, base, rk, ws), (x, wh, a, b, sc, rk, base, out, wh),
              (x, wh, a, b, sc, rk, base, out, x), (x, wh, a, b, sc, rk, base, out, a), (x, wh, a, b, sc, rk, base, out, b),
              (x, wh, a, b, sc, rk, base, out, base), (x, byte(wh), a, b, sc, rk, base, out, ws),
              (x, wh, a, b, byte(sc), rk, base, out, ws), (x, wh, a, b, sc, byte(rk), base, out, ws)):
        assert f(*q, BIG) == INVALID
    wide = adapters(base_ld=520)
    assert lib.moe_adapters(ctypes.byref(wide), x, wh, a, b, sc, rk, out, out, ws, BIG, None) == INVALID
    none = adapters(rows=0)
    assert lib.moe_adapters(ctypes.byref(none), *[None] * 9, 0, None) == OK
