"""The projection beyond a few hundred rows, with quantised weights in every form, and how exactly
the adapters' first product is held."""

import math

import pytest
import torch

from moe_decode_layer_gb300 import _lib, batch, synth
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *s):
    return torch.randn(s, generator=g, device="cuda")


def _adapters(g, n, r, k, o):
    return batch.Adapters((_normal(g, n, r, k) / math.sqrt(k)).bfloat16(), (0.1 * _normal(g, n, o, r)).bfloat16(),
                          0.5 + torch.rand(n, generator=g, device="cuda"))


def _tight(x, weight, ad, ids, one_bf16=False):
    """(out, bound) of an fp32 result whose A x has 16 bits, or 24; one_bf16: with A x rounded to 8 (on the CPU)."""
    x, k = x.double(), x.shape[1]
    y, bound = x @ weight.t(), k * ref.FP32 * (x.abs() @ weight.abs().t())
    for a in range(ad.a.shape[0]):
        rows = torch.nonzero(ids == a).flatten()
        s, a_, b_ = float(ad.scale[a]), ad.a[a].double(), ad.b[a].double()
        u = s * (x[rows] @ a_.t())
        # one step for each addition and for the scale; the second bf16 number is off by half a step of
        # what the first one left, 2^-8 of 2^-8
        du = (k + 2) * ref.FP32 * s * (x[rows].abs() @ a_.abs().t())
        du = du + ref.BF16 ** 2 * (u.abs() + du)
        y[rows] += (u.bfloat16().double() if one_bf16 else u) @ b_.t()
        # the additions of both numbers' products behind the weights' own
        bound[rows] += (du + (2 * b_.shape[1] + k) * ref.FP32 * (u.abs() + du)) @ b_.abs().t()
    return y, bound + 4 * ref.FP32 * (y.abs() + bound)


@pytest.mark.parametrize("rank", [8, 24, 72, 256])
@pytest.mark.parametrize("rows", [40, 300, 2000])
def test_adapter_products_have_sixteen_bits(rank, rows):
    """Few rows: fp32; many: the sum of two bf16 numbers. A result from one bf16 number would not pass."""
    g = _gen(rank)
    x = _normal(g, rows, 64).bfloat16()
    weight = (1e-3 * _normal(g, 128, 64)).bfloat16()
    ad = _adapters(g, 3, rank, 64, 128)
    ids = torch.randint(0, 3, (rows,), generator=g, device="cuda", dtype=torch.int32)
    out = batch.project(x, weight, adapters=ad, adapter_ids=ids, out_dtype=torch.float32)
    want, bound = _tight(x, weight.double(), ad, ids)
    off = (out.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    cpu = batch.Adapters(*(t.cpu() for t in ad))
    wrong, _ = _tight(x.cpu(), weight.double().cpu(), cpu, ids.cpu(), one_bf16=True)
    assert bool(((wrong - want.cpu()).abs() > bound.cpu()).any())


def _check(x, weight, w64, widened, **kw):
    ws = torch.empty(batch.project_workspace(x.shape[1], w64.shape[0] // (2 if kw.get("swiglu") else 1), x.shape[0],
                                             wdtype=kw.get("wdtype", "bf16"), swiglu=kw.get("swiglu", False),
                                             rank=kw["adapters"].a.shape[1] if kw.get("adapters") else 0,
                                             num_adapters=kw["adapters"].a.shape[0] if kw.get("adapters") else 0,
                                             out_dtype=kw.get("out_dtype", torch.bfloat16)), dtype=torch.uint8, device="cuda")
    out = batch.project(x, weight, workspace=ws, **kw)
    assert batch.status(ws) == _lib.MOE_OK
    want, bound = ref.project(x, w64, kw.get("adapters"), kw.get("adapter_ids"), kw.get("addend"), kw.get("swiglu", False),
                              widened, out.dtype == torch.bfloat16)
    off = (out.double() - want).abs()
    assert bool((off <= bound).all()), f"{float((off - bound).max()):.3e} over the bound {float(bound.max()):.3e}"


@pytest.mark.parametrize("rows", [1537, 5003, 15681, 20001])
@pytest.mark.parametrize("inner,outer,rank,count", [(136, 264, 24, 5), (320, 1032, 8, 300), (64, 2000, 72, 1)])
def test_project_of_thousands_of_rows(rows, inner, outer, rank, count):
    """Every tile width of the search for many rows, and the widest tiles of A x."""
    g = _gen(rows + rank)
    x = _normal(g, rows, inner).bfloat16()
    weight = (0.05 * _normal(g, outer, inner)).bfloat16()
    ad = _adapters(g, count, rank, inner, outer)
    ids = torch.randint(-1, count, (rows,), generator=g, device="cuda", dtype=torch.int32)
    ids[: rows // 3] = 0  # one adapter has far more rows than the others
    w64 = weight.double()
    _check(x, weight, w64, False, out_dtype=torch.float32)
    _check(x, weight, w64, False, adapters=ad, adapter_ids=ids, addend=_normal(g, rows, outer).bfloat16())
    if outer % 16 == 0:
        _check(x, weight, w64, False, adapters=ad, adapter_ids=ids, swiglu=True)


@pytest.mark.parametrize("wdtype", ["fp8", "nvfp4"])
@pytest.mark.parametrize("rows", [1, 50, 257, 3001])
def test_quantised_project_in_every_form(wdtype, rows):
    """An addend, an fp32 result and adapters, alone and together, as the layer's down projection has them."""
    g = _gen(rows)
    inner, outer = 768, 512
    w = 0.05 * _normal(g, outer, inner)
    weight = synth.quantize_fp8_block(w) if wdtype == "fp8" else tuple(synth.quantize_nvfp4(w))
    w64 = ref.fp8(*weight) if wdtype == "fp8" else ref.nvfp4(*weight)
    x = _normal(g, rows, inner).bfloat16()
    add = 4 * _normal(g, rows, outer).bfloat16()
    ad = _adapters(g, 4, 40, inner, outer)
    ids = torch.randint(-1, 4, (rows,), generator=g, device="cuda", dtype=torch.int32)
    for out_dtype in (torch.bfloat16, torch.float32):
        for addend in (None, add):
            kw = dict(wdtype=wdtype, out_dtype=out_dtype, addend=addend)
            _check(x, weight, w64, wdtype == "fp8", **kw)
            # (an NVFP4 weight is rounded with its tensor scale where adapters share the sum)
            _check(x, weight, w64, True, adapters=ad, adapter_ids=ids, **kw)
    out = add.clone()
    batch.project(x, weight, wdtype=wdtype, adapters=ad, adapter_ids=ids, addend=out, out=out)
    assert torch.equal(out, batch.project(x, weight, wdtype=wdtype, adapters=ad, adapter_ids=ids, addend=add))
