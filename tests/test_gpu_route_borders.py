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


@pytest.mark.parametrize("shift", [12.0, 18.0, 30.0])
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
