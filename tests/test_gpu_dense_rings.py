"""Integer products whose CTAs go round their ring of slots several times, and blocks as wide as that; weights
differ from step to step, so that a slot read too early would show."""

import pytest
import torch

from moe_decode_layer_gb300 import _lib, batch
from tests import dense_reference as ref

pytestmark = pytest.mark.gpu


def _int8(g, rows, cols):
    return torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8), \
        torch.randn(rows, generator=g, device="cuda") * 0.01


# 7 slots a CTA at 40 rows, 6 or (K split) 5 at 60, 5 at 96 and 112, 3 at 160 and 180
@pytest.mark.parametrize("rows,inner,outer,swiglu", [
    (40, 8192, 9800, False), (40, 16384, 1000, False), (40, 4096, 6000, True), (60, 16384, 1000, False), (60, 8192, 4800, True),
    (96, 4096, 9800, False), (96, 16384, 1032, True), (112, 8192, 1032, False), (112, 4096, 9000, True), (160, 8192, 4096, False),
    (180, 8192, 9728, False), (180, 4096, 4800, True), (192, 16384, 1000, False)])
def test_project_int8_round_the_ring(rows, inner, outer, swiglu):
    g = torch.Generator(device="cuda").manual_seed(rows + inner)
    q, s = _int8(g, rows, inner)
    w, c = _int8(g, outer * (2 if swiglu else 1), inner)
    ws = torch.full((batch.project_int8_workspace(inner, outer, rows, swiglu=swiglu, out_dtype=torch.float32),), 255, dtype=torch.uint8, device="cuda")
    y, bound = ref.int8(q, s, w, c, swiglu=swiglu, bf16=False)
    first = batch.project_int8((q, s), (w, c), swiglu=swiglu, out_dtype=torch.float32, workspace=ws)
    assert batch.status(ws) == _lib.MOE_OK and ref.within(first, y, bound)
    for _ in range(20):  # the same bits, whatever order copies land in
        assert torch.equal(batch.project_int8((q, s), (w, c), swiglu=swiglu, out_dtype=torch.float32, workspace=ws), first)
    assert batch.status(ws) == _lib.MOE_OK


# h so wide that a thread of the rows' quantisation goes a second round, and K of W2 round the ring
@pytest.mark.parametrize("rows,hidden,inter", [(5, 512, 9216), (40, 256, 9216), (60, 1024, 10000), (100, 256, 8208), (180, 256, 9216), (600, 256, 9216)])
def test_feed_forward_int8_wide(rows, hidden, inter):
    g = torch.Generator(device="cuda").manual_seed(rows + inter)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w13, w2 = batch.quantise(n(2 * inter, hidden) * hidden ** -0.5), batch.quantise(n(hidden, inter) * inter ** -0.5)
    x, residual = n(rows, hidden).bfloat16(), n(rows, hidden).bfloat16()
    ws = torch.full((batch.feed_forward_workspace(hidden, inter, rows, wdtype="int8"),), 255, dtype=torch.uint8, device="cuda")
    out = batch.feed_forward(x, w13, w2, wdtype="int8", residual=residual, workspace=ws)
    assert batch.status(ws) == _lib.MOE_OK
    assert ref.within(out, *ref.block_int8(x, *w13, *w2, residual))


@pytest.mark.parametrize("rows,wdtype", [(4, "bf16"), (100, "bf16"), (300, "bf16"), (12, "int8"), (100, "int8"), (300, "int8")])
def test_status_words_are_cleared(rows, wdtype):
    """All of them, also those that no block of the call has."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    w13, w2, x = n(528, 272), n(272, 264 if wdtype == "bf16" else 272), n(rows, 272)
    w13 = w13 if wdtype == "bf16" else n(544, 272)
    if wdtype == "int8":
        w13, w2 = batch.quantise(w13), batch.quantise(w2)
    inter = 264 if wdtype == "bf16" else 272
    ws = torch.full((batch.feed_forward_workspace(272, inter, rows, wdtype=wdtype),), 255, dtype=torch.uint8, device="cuda")
    batch.feed_forward(x, w13, w2, wdtype=wdtype, workspace=ws)
    assert not bool(ws[:_lib.ROWS_STATUS_BYTES].any()) and batch.status(ws) == _lib.MOE_OK
    ws[4 * 700:4 * 701] = 1  # a word that a block past the SMs' number would set
    assert batch.status(ws) == _lib.MOE_ERR_DEVICE_TIMEOUT
