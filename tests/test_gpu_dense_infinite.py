"""Infinite weights: a result is infinite where the definition's is, whatever the number of rows."""

import pytest
import torch

from moe_decode_layer_gb300 import batch

pytestmark = pytest.mark.gpu


# one to four rows, and up to sixteen of a small block: h is the sum of two numbers
@pytest.mark.parametrize("rows,hidden,inter", [(1, 256, 512), (3, 512, 264), (4, 2560, 2064), (8, 256, 512), (12, 264, 136), (16, 512, 1032),
                                               (40, 256, 512), (300, 256, 512)])
def test_infinite_down_weights(rows, hidden, inter):
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    w13, w2, x = (n(2 * inter, hidden) * hidden ** -0.5).bfloat16(), n(hidden, inter), n(rows, hidden)
    at = torch.arange(0, hidden, 3, device="cuda")
    w2[at, at % inter] = float("inf")
    w2[at[::2], at[::2] % inter] = float("-inf")
    both = x.double() @ w13.double().t()
    a, b = both.chunk(2, 1)
    h = a * torch.sigmoid(a) * b
    assert bool((h.abs() > 1e-30).all())  # no h is near enough to 0 for its sign, or itself, to be lost
    want = h @ w2.double().t()
    out = batch.feed_forward(x, w13, w2).double()
    assert bool((torch.isinf(want) == torch.isinf(out)).all())
    assert torch.equal(out[torch.isinf(want)], want[torch.isinf(want)]) and not bool(torch.isnan(out).any())
