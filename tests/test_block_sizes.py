"""Host-side size queries of the norm, the balance loss and the adapters at their limits."""
import ctypes

import pytest

import mixture_experts_layer_adjusted_amd as moe
from mixture_experts_layer_adjusted_amd import binding

lib = binding.raw_lib()


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 48, 64, 128])
@pytest.mark.parametrize("in_cols", [8, 256, 7168, 1 << 20])
@pytest.mark.parametrize("n", [1, 8, 5000])
def test_adapters_of_no_rows(n, in_cols, rank):
    """A batch that has run empty: no bytes, and the call returns, whatever the adapters' sizes are."""
    shape = moe.make_adapter_shape(0, in_cols, 4096, n, rank, moe.MOE_DTYPE_BF16)
    assert moe.moe_adapters_workspace_size(shape) == 0
    assert lib.moe_adapters(ctypes.byref(shape), *[None] * 9, 0, None) == 0


@pytest.mark.parametrize("cols", [8, 2048, 7168, 32768])
def test_norm_of_no_rows(cols):
    assert moe.moe_norm_workspace_size(moe.make_norm_shape(0, cols, moe.MOE_DTYPE_BF16, 1e-6)) == 0


@pytest.mark.parametrize("n,seqs", [(1, 1), (64, 7), (512, 1 << 24)])
def test_balance_of_no_tokens(n, seqs):
    cfg = moe.make_balance_config(0, n, 1, moe.MOE_DTYPE_F32, moe.MOE_SCORE_SOFTMAX, seqs)
    assert moe.moe_balance_workspace_size(cfg) == 0


BATCHES = [*range(0, 1200), *range(1200, 9000, 7), *range(9000, 200000, 997)]


@pytest.mark.parametrize("n,rank,in_cols", [(8, 16, 7168), (32, 64, 7168), (64, 32, 2048), (4, 128, 4096), (1, 8, 2048),
                                            (300, 24, 1000), (1, 128, 8)])
def test_a_smaller_batch_of_adapters_needs_no_more(n, rank, in_cols):
    """A server sizes its buffer for its largest batch."""
    sizes = [moe.moe_adapters_workspace_size(moe.make_adapter_shape(t, in_cols, 4096, n, rank, moe.MOE_DTYPE_BF16))
             for t in BATCHES]
    assert sizes == sorted(sizes) and sizes[0] == 0 and sizes[-1] > 0


@pytest.mark.parametrize("n", [2, 60, 61, 64, 128, 130, 256, 512])
def test_a_smaller_batch_of_the_balance_loss_needs_no_more(n):
    """Fewer tokens, fewer sequences or both."""
    size = lambda t, s: moe.moe_balance_workspace_size(  # noqa: E731
        moe.make_balance_config(t, n, 1, moe.MOE_DTYPE_F32, moe.MOE_SCORE_SOFTMAX, s))
    seqs = [1, 2, 3, 7, 15, 16, 31, 64, 4096, 4097, 70000]
    table = [[size(t, s) for s in seqs] for t in BATCHES[::3]]
    assert all(row == sorted(row) for row in table)
    assert all(list(c) == sorted(c) for c in zip(*table))
    assert size(0, 5) == 0 and size(1, 5) == 0 and size(100000, 1) > 0
    # every chunk and sequence that two kernels may need has its place (the sums and counts of n columns, and a count)
    for t in BATCHES[1::3]:
        for s in seqs:
            block = 16 * (1 if n % 4 else 4 if n <= 128 else 2 if n <= 256 else 1)
            places = min(-(-t // block), 256) + s
            assert size(t, s) in (0, places * (2 * -(-n // 4) * 4 + 4) * 4) and (size(t, s) > 0 or s <= 4096)


@pytest.mark.parametrize("cols,dtype", [(8, 0), (1408, 0), (7168, 0), (7168, 1), (520, 1), (2048, 1), (32768, 0)])
def test_a_smaller_batch_of_the_norm_needs_no_more(cols, dtype):
    sizes = [moe.moe_norm_workspace_size(moe.make_norm_shape(t, cols, dtype, 1e-6)) for t in BATCHES]
    assert sizes == sorted(sizes) and sizes[0] == 0 and sizes[-1] > 0
