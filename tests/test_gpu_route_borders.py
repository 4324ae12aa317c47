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
