"""The balance loss's sums over long sequences.

A wavefront's lane adds up its tokens one after another, every 64 of them into a second sum: at T tokens in 256 places of whole
blocks (64 tokens at up to 128 experts in fours, 16 at 512) at most 64 + T / (256 block 64) additions, then 16 wavefronts, 4
tokens and 256 places.  2^-24 each on positive terms, the share itself 2^-19: under 2^-16 here."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import mixture_experts_layer_adjusted_amd as moe  # noqa: E402
from test_gpu_balance import config, forward  # noqa: E402


@pytest.mark.parametrize("T,N,softmax", [((1 << 23) + 77, 512, True), ((1 << 26) + 5, 64, True), ((1 << 25) + 5, 64, False),
                                         ((1 << 24) + 9, 61, True)])
def test_the_same_token_over_and_over(T, N, softmax):
    """Each addition rounds the same way as the last: nothing averages out."""
    g = torch.Generator("cuda").manual_seed(N)
    row = torch.randn(1, N, device="cuda", generator=g).bfloat16()
    logits = row.expand(T, N).contiguous()
    idx = torch.full((T, 1), N - 1, dtype=torch.int32, device="cuda")
    loss, counts, tokens, total = forward(logits, idx, None, softmax)
    assert tokens.item() == T and counts[0, N - 1].item() == T and int(counts.sum()) == T
    l = row[0].double()
    p = torch.softmax(l, 0) if softmax else torch.sigmoid(l) / torch.sigmoid(l).sum()
    assert ((total[0].double() / T - p).abs() <= 2.0 ** -16 * p).all()
    want = config(logits, idx, 1, softmax).alpha * N * p[N - 1].item()
    assert abs(loss.item() - want) <= 2.0 ** -15 * want


def test_long_sequences_that_begin_anywhere():
    """The second sum goes with its sequence."""
    T, N = (1 << 23) + 3, 512
    g = torch.Generator("cuda").manual_seed(3)
    rows = torch.randn(3, N, device="cuda", generator=g).bfloat16()
    starts = torch.tensor([0, 2800001, 2800001 + 3600000, T], dtype=torch.int32, device="cuda")
    which = torch.searchsorted(starts, torch.arange(T, device="cuda", dtype=torch.int32), right=True) - 1
    logits = rows[which]
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    _, _, tokens, total = forward(logits, idx, starts, True)
    p = torch.softmax(rows.double(), 1)
    assert torch.equal(tokens, starts[1:] - starts[:-1])
    assert ((total.double() / tokens[:, None] - p).abs() <= 2.0 ** -16 * p).all()
