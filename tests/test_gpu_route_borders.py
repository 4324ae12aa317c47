"""The choice of moe_decode_route where fp32 cannot tell keys apart: the indexes are those
of a 64-bit computation, whoever else has equal inputs."""

import pytest
import torch

from moe_decode_layer_gb300 import batch
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *s):
    return torch.randn(s, generator=g, device="cuda")


def _check(logits, k, score, bias=None, groups=1, kept=1, best=1, renormalise=True):
    idx, w = batch.route(logits, k, score=score, bias=bias, num_groups=groups, top_groups=kept, group_best=best,
                         renormalise=renormalise)
    want, want_w = ref.route(logits, k, score, bias, groups, kept, best, renormalise)
    wrong = (idx.cpu() != want).any(1)
    assert not bool(wrong.any()), f"{int(wrong.sum())} of {len(wrong)} rows, the first: {idx[wrong.to(idx.device)][0].tolist()} " \
        f"for {want[wrong][0].tolist()}"
    return w.cpu().double(), want_w


def test_equal_groups_at_the_border_beside_a_better_one():
    """Three sums that fp32 holds as 2: two equal ones, and a larger one after them."""
    logits = torch.tensor([[20.0, 20, 20, 20, 21, 21], [21.0, 21, 20, 20, 20, 20], [20.0, 20, 21, 21, 20, 20],
                           [20.0, 20, 20, 20, 20, 20], [20.0, 21, 21, 20, 20, 20]], device="cuda")
    for kept in (1, 2):
        _check(logits, 2, "sigmoid", None, 3, kept, 2)
        _check(logits, 2, "sigmoid", torch.zeros(6, device="cuda"), 3, kept, 2)


@pytest.mark.parametrize("shift", [12.0, 18.0, 30.0, -95.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_groups_of_saturated_scores(shift, dtype):
    """Sums of two sigmoids that fp32 holds as nearly equal, with many equal logits (bf16)."""
    logits = (_normal(_gen(int(shift) + 200), 500, 128) + shift).to(dtype)
    for kept in (1, 4):
        _check(logits, 8, "sigmoid", None, 8, kept, 2)


def test_equal_experts_at_the_border_beside_a_better_one():
    """Three keys that fp32 holds as 1: two equal ones, and a larger one after them."""
    logits = torch.tensor([[20.0, 20, 21], [20.0, 21, 20], [21.0, 20, 20], [20.0, 20, 20]], device="cuda")
    for k in (1, 2, 3):
        _check(logits, k, "sigmoid", torch.zeros(3, device="cuda"))
        _check(logits, k, "sigmoid", torch.full((3,), 0.25, device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_equal_keys_with_a_bias(score):
    """Few distinct logits around a saturated score, few distinct biases: long runs of equal inputs."""
    g = _gen(3)
    for experts, k in ((24, 4), (96, 8), (300, 16)):
        logits = 19 + torch.randint(0, 4, (200, experts), generator=g, device="cuda").float()
        bias = 0.125 * torch.randint(0, 2, (experts,), generator=g, device="cuda").float()
        _check(logits, k, score, bias)
        _check(logits.bfloat16(), k, score, torch.zeros_like(bias))
        _check(logits, k, score, bias, 4, 2, 2)


def test_group_sums_that_underflow():
    """Scores at and below the smallest that fp32 holds: exp overflows (sigmoid) or vanishes (softmax)."""
    inf = float("inf")
    _check(torch.tensor([[-88.6, -89.0, -88.5, -120.0]], device="cuda"), 1, "sigmoid", None, 2, 1, 2)
    _check(torch.tensor([[0.0, 0.0, -103.9, -500.0, -104.2, -104.2], [0.0, -inf, -103.9, -inf, -104.2, -104.2]],
                        device="cuda"), 2, "softmax", None, 3, 2, 2)
    g = _gen(4)
    for mean in (-86.0, -88.5, -100.0, -104.0):
        logits = mean + 2 * _normal(g, 300, 64)
        _check(logits, 4, "sigmoid", None, 8, 3, 2)
        _check(logits.bfloat16(), 4, "sigmoid", None, 8, 3, 2)
        logits[:, :8] = _normal(g, 300, 8)  # one group far above the others
        _check(logits, 4, "softmax", None, 8, 3, 2)


def test_keys_that_underflow_with_a_bias():
    """Without a bias to speak of the keys are the scores themselves."""
    g = _gen(5)
    for mean in (-87.0, -88.7, -95.0):
        logits = mean + _normal(g, 200, 64)
        _check(logits, 6, "sigmoid", torch.zeros(64, device="cuda"))
        _check(logits, 6, "sigmoid", torch.zeros(64, device="cuda"), 8, 3, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_that_cancel(score):
    """Large biases of opposite sign: the keys' roundings are far above the sums' own."""
    g = _gen(6)
    for size, big in ((2, 1000.0), (4, 5e5)):
        bias = torch.zeros(8 * size, device="cuda")
        bias[0::size], bias[1::size] = big, 1 - big
        if size > 2:
            bias[2::size] = bias[3::size] = -2 * big
        logits = 0.3 + 1e-4 * _normal(g, 400, 8 * size)
        for best in (1, 2):
            _check(logits, 4, score, bias, 8, 3, best)


def test_infinite_biases_at_the_border():
    """+inf is a key like any other: equal ones go to the lower index, and nothing is NaN."""
    g = _gen(7)
    bias = 0.1 * _normal(g, 64)
    bias[3] = bias[40] = bias[41] = float("inf")
    for kept, best in ((1, 1), (2, 2), (3, 2)):
        idx, w = batch.route(_normal(g, 50, 64), 4, score="sigmoid", bias=bias, num_groups=8, top_groups=kept, group_best=best)
        assert bool((idx[:, 0] == 3).all()) and bool(torch.isfinite(w).all())
        if kept > 1:
            assert bool((idx[:, 1] == 40).all()) and bool((idx[:, 2] == 41).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [1000.0, 3e4])
def test_groups_with_and_without_cancelling_biases(score, big):
    """A border between two groups of small keys, which is clear, beside groups whose keys are rounded far more."""
    g = _gen(8)
    bias = torch.zeros(64, device="cuda")
    for n in range(0, 32, 2):
        bias[2 * n], bias[2 * n + 1] = big, -big
    for spread in (1e-4, 1e-5):
        logits = -1.5 + spread * _normal(g, 500, 64)
        for kept in (5, 16, 28):
            _check(logits, 8, score, bias, 32, kept, 2)


def _check_weights(logits, k, score, bias, renormalise, scale=1.0):
    idx, w = batch.route(logits, k, score=score, bias=bias, renormalise=renormalise, scale=scale)
    want_idx, want = ref.route(logits, k, score, bias, renormalise=renormalise, scale=scale)
    assert torch.equal(idx.cpu(), want_idx)
    off = (w.cpu().double() - want).abs()
    assert bool((off <= ref.route_tolerance(logits, score, renormalise) * want.abs() + 1e-37).all()), float((off / want.clamp(min=1e-37)).max())
    return want


@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_weights_of_experts_far_below_the_rows_largest(scale):
    """A bias chooses experts whose softmax scores fp32 does not hold; their weights are between themselves."""
    g = _gen(9)
    logits = _normal(g, 100, 40)
    logits[:, 20:] -= 95 + 10 * torch.rand(100, 1, generator=g, device="cuda")
    bias = torch.zeros(40, device="cuda")
    bias[20:] = torch.arange(20, device="cuda") + 2.0
    for k in (1, 4, 16):
        want = _check_weights(logits, k, "softmax", bias, True, scale)
        assert bool((want.sum(1) > 0.99 * scale).all())
        _check_weights(logits - 30, k, "softmax", bias, True, scale)
        _check_weights(logits, k, "softmax", bias, False, scale)


@pytest.mark.parametrize("renormalise", [False, True])
def test_weights_of_sigmoids_far_below_zero(renormalise):
    """Chosen logits from a little below 0 to -110: the small ones of a renormalised row are held too."""
    g = _gen(10)
    for top in (2.0, -1.0, -10.0, -29.0, -31.0, -80.0):
        logits = top - 80 * torch.rand(100, 24, generator=g, device="cuda")
        bias = torch.arange(24, device="cuda").float()
        for k in (1, 5, 16):
            _check_weights(logits, k, "sigmoid", None, renormalise)
            _check_weights(logits, k, "sigmoid", bias, renormalise)
