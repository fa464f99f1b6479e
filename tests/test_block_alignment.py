"""The norm's documented alignment: multiples of 16, of 4 for scales, rstd and d_weight."""
import ctypes

import pytest

import mixture_experts_layer_adjusted_amd as moe
from mixture_experts_layer_adjusted_amd import binding

lib = binding.raw_lib()
P = [0x10000 * (i + 1) for i in range(8)]     # plausible, never dereferenced
INVALID = 1


def args(i, by):
    return [ctypes.c_void_p(p + (by if j == i else 0)) for j, p in enumerate(P)]


@pytest.mark.parametrize("by", [1, 2, 3, 6])
@pytest.mark.parametrize("i", range(8))
def test_forward(i, by):
    shape = moe.make_norm_shape(10, 256, 1, 1e-6)
    assert lib.moe_norm_forward(ctypes.byref(shape), *args(i, by), None) == INVALID


@pytest.mark.parametrize("rows", [10, 1000])
@pytest.mark.parametrize("by", [1, 2, 3, 6])
@pytest.mark.parametrize("i", range(8))
def test_backward(i, by, rows):
    shape = moe.make_norm_shape(rows, 256, 1, 1e-6)
    assert lib.moe_norm_backward(ctypes.byref(shape), *args(i, by), ctypes.c_size_t(1 << 40), None) == INVALID


@pytest.mark.parametrize("by", [1, 2, 3])
def test_backward_of_no_rows(by):
    shape = moe.make_norm_shape(0, 256, 1, 1e-6)
    assert lib.moe_norm_backward(ctypes.byref(shape), *[None] * 6, ctypes.c_void_p(P[6] + by), None, ctypes.c_size_t(0),
                                 None) == INVALID
