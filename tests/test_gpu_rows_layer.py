"""The layer on any number of rows: its workspace and status, rows with a stride, adapters for each weight type."""

import dataclasses

import pytest
import torch

from moe_decode_layer_gb300 import LayerShape, _lib, batch, synth
from moe_decode_layer_gb300.layer import MoEDecodeLayer
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _adapters(g, n, r, k, o):
    return batch.Adapters((torch.randn(n, r, k, generator=g, device="cuda") / k ** 0.5).bfloat16(),
                          (0.1 * torch.randn(n, o, r, generator=g, device="cuda")).bfloat16(),
                          0.5 + torch.rand(n, generator=g, device="cuda"))


@pytest.mark.parametrize("rows", [3, 150])
@pytest.mark.parametrize("with_adapters", [False, True])
def test_workspace_and_status(rows, with_adapters):
    """A run in a workspace of the caller's gives the same bits, and a time-out of any of its operators is seen."""
    shape = LayerShape(256, 128, 16, 2, 1)
    mod = MoEDecodeLayer(shape, synth.make_layer(shape, seed=1, device="cuda"), max_rows=1)
    g = _gen(rows)
    x = torch.randn(rows, 256, generator=g, device="cuda").bfloat16()
    kw = {}
    if with_adapters:
        kw = dict(adapters=(_adapters(g, 4, 16, 256, 256), _adapters(g, 4, 8, 128, 256)),
                  adapter_ids=torch.randint(-1, 4, (rows,), generator=g, device="cuda", dtype=torch.int32))
    ad = kw.get("adapters")
    ws = torch.full((mod.rows_workspace(rows, ad),), 255, dtype=torch.uint8, device="cuda")
    want = mod.run_rows(x, **kw)
    assert torch.equal(mod.run_rows(x, workspace=ws, **kw), want)
    assert mod.rows_status(ws, rows, ad) == _lib.MOE_OK
    parts, _ = mod._rows_parts(rows, ad)
    assert len(parts) == (4 if with_adapters else 2)
    for at, _ in parts.values():  # a word that a wait past its limit would set
        ws[at:at + 4].view(torch.int32).fill_(1)
        assert mod.rows_status(ws, rows, ad) == _lib.MOE_ERR_DEVICE_TIMEOUT
        ws[at:at + 4].zero_()
    assert mod.rows_status(ws, rows, ad) == _lib.MOE_OK
    assert mod.rows_workspace(0, ad) == 0 and mod.run_rows(x[:0], workspace=ws, adapters=ad, adapter_ids=kw["adapter_ids"][:0] if ad else None).shape == (0, 256)
    for bad in (ws[:-256], ws.cpu(), ws.view(torch.int8)):
        with pytest.raises(ValueError):
            mod.run_rows(x, workspace=bad, **kw)
        with pytest.raises(ValueError):
            mod.rows_status(bad, rows, ad)
    mod.close()


@pytest.mark.parametrize("rows", [1, 40])
def test_rows_with_a_stride(rows):
    """x as a part of wider rows, with no residual of its own, also on another stream and captured."""
    shape = LayerShape(256, 128, 16, 2, 1)
    mod = MoEDecodeLayer(shape, synth.make_layer(shape, seed=2, device="cuda"), max_rows=1)
    wide = torch.randn(rows, 512, generator=_gen(rows), device="cuda").bfloat16()
    x = wide[:, 128:384]
    want = mod.run_rows(x.contiguous())
    assert torch.equal(mod.run_rows(x), want)
    assert torch.equal(mod.run_rows(x, x.contiguous()), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mod.run_rows(x, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mod.run_rows(x)
    wide.copy_(torch.randn(rows, 512, generator=_gen(9), device="cuda").bfloat16())
    graph.replay()
    assert torch.equal(got, mod.run_rows(x.contiguous()))
    mod.close()


@pytest.mark.parametrize("rows", [2, 100])
def test_one_rounding_with_adapters(rows):
    """256 + 1 (shared expert) + 1 (routed) is 258: a rounding to bf16 after the first sum would lose both."""
    shape = LayerShape(256, 128, 16, 1, 1)
    layer = {k: torch.zeros_like(v) if torch.is_tensor(v) else v for k, v in synth.make_layer(shape, seed=3, device="cuda").items()}
    for p in ("", "sh_"):  # h_0 = silu(64) / 64 = 1, y = h_0
        layer[p + "w13"][:, 0, 0], layer[p + "w13"][:, 128, 0] = 64, 1 / 64
        layer[p + "w2"][:, :, 0] = 1
    mod = MoEDecodeLayer(shape, layer, max_rows=1)
    x = torch.zeros(rows, 256, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    r = torch.full_like(x, 256)
    g = _gen(1)
    up, down = _adapters(g, 2, 8, 256, 256), _adapters(g, 2, 8, 128, 256)
    up.b.zero_(), down.b.zero_()
    ids = torch.randint(-1, 2, (rows,), generator=g, device="cuda", dtype=torch.int32)
    assert bool((mod.run_rows(x, r) == 258).all())
    assert bool((mod.run_rows(x, r, adapters=(up, down), adapter_ids=ids) == 258).all())
    mod.close()


@pytest.mark.parametrize("rows", [1, 50, 16384 + 3])
def test_fp32_residual(rows):
    shape = LayerShape(72, 24, 5, 2, 1)
    layer = synth.make_layer(shape, seed=4, device="cuda")
    g = _gen(rows)
    x = torch.randn(rows, 72, generator=g, device="cuda").bfloat16()
    idx = torch.randint(0, 5, (rows, 2), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(rows, 2, generator=g, device="cuda")
    r = torch.randn(rows, 72, generator=g, device="cuda")
    out = batch.experts(shape, layer, x, idx, w, residual=r)
    want, bound = ref.experts(shape, layer, x, idx, w, r)
    assert bool(((out.double() - want).abs() <= bound).all())
    with pytest.raises(ValueError):
        batch.experts(shape, layer, x, idx, w, residual=r.half())


@pytest.mark.parametrize("wdtype", ["bf16", "fp8", "nvfp4"])
def test_result_in_the_place_of_x(wdtype):
    """A step in place, as run() does it: one round of rows, and three."""
    shape = LayerShape(256, 256, 16, 2, 1, wdtype)
    mod = MoEDecodeLayer(shape, synth.make_layer(shape, seed=5, device="cuda"), max_rows=8)
    for rows in (1, 8, 700, 2 * 16384 + 77):
        x = torch.randn(rows, 256, generator=_gen(rows), device="cuda").bfloat16()
        want = mod.run_rows(x)
        assert mod.run_rows(x, out=x) is x and torch.equal(x, want)
    mod.close()


@pytest.mark.parametrize("wdtype", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("rows", [7, 150, 1200])
def test_adapters_of_every_weight_type(wdtype, rows):
    """The layer with requests' adapters on its shared expert, against its parts in 64 bits."""
    shape = LayerShape(512, 256, 24, 3, 1, wdtype)
    layer = synth.make_layer(shape, seed=6, device="cuda")
    mod = MoEDecodeLayer(shape, layer, max_rows=1)
    g = _gen(rows)
    x, r = (torch.randn(rows, 512, generator=g, device="cuda").bfloat16() for _ in range(2))
    up, down = _adapters(g, 5, 16, 512, 512), _adapters(g, 5, 8, 256, 512)
    ids = torch.randint(-1, 5, (rows,), generator=g, device="cuda", dtype=torch.int32)
    idx = torch.empty(rows, 3, dtype=torch.int32, device="cuda")
    w = torch.empty(rows, 3, device="cuda")
    out = mod.run_rows(x, r, topk_idx=idx, topk_w=w, adapters=(up, down), adapter_ids=ids)
    logits = batch.project(x, layer["router_w"], out_dtype=torch.float32)
    assert torch.equal(idx.cpu(), ref.route(logits, 3, "softmax")[0])
    w13, w2 = (ref.matrix(layer, n, wdtype, 0) for n in ("sh_w13", "sh_w2"))
    widened = wdtype != "bf16"
    h, dh = ref.project(x, w13, up, ids, swiglu=True, widened=widened)
    shared, ds = ref.project(h, w2, down, ids, addend=r, widened=widened, bf16=False)
    # h's own rounding and bound, through the down matrix and its adapters; then the bound again of what that adds
    extra = dh @ w2.abs().t()
    for a in range(5):
        of = ids == a
        extra[of] += float(down.scale[a]) * ((dh[of] @ down.a[a].double().abs().t()) @ down.b[a].double().abs().t())
    ds = ds + (1 + 2 * ref.BF16) * extra
    routed, dr = ref.experts(dataclasses.replace(shape, num_shared=0), layer, x, idx, w)
    total = shared + routed
    bound = ds + dr + ref.FP32 * (shared.abs() + routed.abs()) + ref.BF16 * (total.abs() + ds + dr)
    off = (out.double() - total).abs()
    assert bool((off <= bound).all()), f"{float((off - bound).max()):.3e} over the bound {float(bound.max()):.3e}"
    mod.close()


def test_status_leaves_a_capture_intact():
    """Asked for in the middle of a capture, the status is refused and the graph is whole."""
    shape = LayerShape(256, 128, 16, 2, 1)
    layer = synth.make_layer(shape, seed=7, device="cuda")
    x = torch.randn(9, 256, generator=_gen(7), device="cuda").bfloat16()
    idx = torch.randint(0, 16, (9, 2), generator=_gen(8), device="cuda", dtype=torch.int32)
    w = torch.rand(9, 2, generator=_gen(9), device="cuda")
    ws = torch.empty(batch.experts_workspace(shape, 9), dtype=torch.uint8, device="cuda")
    want = batch.experts(shape, layer, x, idx, w, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = batch.experts(shape, layer, x, idx, w, workspace=ws)
        code = batch.status(ws)
    assert code == _lib.MOE_ERR_INVALID_ARG
    graph.replay()
    assert torch.equal(out, want) and batch.status(ws) == _lib.MOE_OK
