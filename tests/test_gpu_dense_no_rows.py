"""Batches without rows through the binding."""

import pytest
import torch

from moe_decode_layer_gb300 import batch

pytestmark = pytest.mark.gpu


def test_gradients_of_no_rows():
    w13, w2 = torch.ones(144, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, 72, dtype=torch.bfloat16, device="cuda")
    x, kept = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 144, dtype=torch.bfloat16, device="cuda")
    dx, d13, d2 = batch.feed_forward_backward(x, x, w13, w2, kept, weight_grad=False)
    assert dx.shape == (0, 64) and d13 is None and d2 is None
    dx, d13, d2 = batch.feed_forward_backward(x, x, w13, w2, kept, input_grad=False)
    assert dx is None and not bool(d13.any()) and not bool(d2.any())


@pytest.mark.parametrize("swiglu", [False, True])
def test_products_of_no_rows(swiglu):
    w = torch.ones(64, 48, dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    x = torch.empty(0, 48, dtype=torch.bfloat16, device="cuda")
    for rows in (x, x.float(), batch.quantise(x)):
        assert batch.project_int8(rows, w, swiglu=swiglu).shape == (0, 32 if swiglu else 64)
