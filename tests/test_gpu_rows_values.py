"""Values at the ends of the types' ranges in the many-row operators."""

import math

import pytest
import torch

from moe_decode_layer_gb300 import LayerShape, batch
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu

BF16_MAX = torch.finfo(torch.bfloat16).max


def _adapter_at_the_limit(rows, first, rank):
    """Rows 0 and 1 of x meet an adapter whose first product is `first` (its terms) times 1 and -1."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, 64, generator=g, device="cuda").bfloat16()
    x[:, :2] = 0
    x[0, :2], x[1, :2] = 1, -1
    weight = (0.1 * torch.randn(32, 64, generator=g, device="cuda")).bfloat16()
    a = (0.1 * torch.randn(1, rank, 64, generator=g, device="cuda")).bfloat16()
    a[0, 0] = 0
    a[0, 0, 0], a[0, 0, 1] = first
    b = (0.1 + torch.rand(1, 32, rank, generator=g, device="cuda")).bfloat16()
    return x, weight, batch.Adapters(a, b), torch.zeros(rows, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows", [8, 100, 700])
@pytest.mark.parametrize("rank", [8, 72])
def test_adapter_products_beyond_bf16(rows, rank):
    """A x above bf16's largest number, but not fp32's, is held; every row count gives the formula's value."""
    x, weight, ad, ids = _adapter_at_the_limit(rows, (BF16_MAX, 2.0 ** 119 * 1.5), rank)
    ad.b[:, :, 0] *= 2.0 ** -100
    for dtype in (torch.float32, torch.bfloat16):
        out = batch.project(x, weight, adapters=ad, adapter_ids=ids, out_dtype=dtype)
        want, bound = ref.project(x, weight.double(), ad, ids, bf16=dtype == torch.bfloat16)
        assert bool(torch.isfinite(out).all()) and bool(((out.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("rows", [8, 100, 700])
@pytest.mark.parametrize("rank", [8, 72])
def test_infinite_adapter_products(rows, rank):
    """A x past fp32's range is an infinity, as the sum it goes into, for every row count; the other rows stay as they are."""
    x, weight, ad, ids = _adapter_at_the_limit(rows, (BF16_MAX, BF16_MAX), rank)
    out = batch.project(x, weight, adapters=ad, adapter_ids=ids)
    assert bool((out[0] == math.inf).all()) and bool((out[1] == -math.inf).all())
    want, bound = ref.project(x[2:], weight.double(), ad, ids[2:])
    assert bool(((out[2:].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("rows", [3, 200])
def test_silu_far_below_zero(rows):
    """exp(-g) above 2^126: the quotient is small and not zero, which a large up value shows."""
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    weight = torch.zeros(64, 8, dtype=torch.bfloat16, device="cuda")
    gates = torch.linspace(-88.25, -80.0, 32)
    weight[:32, 0], weight[32:, 0] = gates.bfloat16(), 2.0 ** 120
    out = batch.project(x, weight, swiglu=True)
    want, bound = ref.project(x, weight.double(), swiglu=True)
    assert bool((want.abs() > 0).all()) and bool(((out.double() - want).abs() <= bound).all())
    # the same in the experts' intermediate row, through a down matrix of ones
    layer = {"w13": weight[None].contiguous(), "w2": torch.ones(1, 8, 32, dtype=torch.bfloat16, device="cuda")}
    shape = LayerShape(8, 32, 1, 1, 0)
    idx, w = torch.zeros(rows, 1, dtype=torch.int32, device="cuda"), torch.ones(rows, 1, device="cuda")
    got = batch.experts(shape, layer, x, idx, w)
    want, bound = ref.experts(shape, layer, x, idx, w)
    assert bool(((got.double() - want).abs() <= bound).all())
