"""The many-row operators on the GPU against their plain 64-bit restatements."""

import dataclasses
import math

import pytest
import torch

from moe_decode_layer_gb300 import LayerShape, _lib, batch, synth
from tests import helpers
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *s):
    return torch.randn(s, generator=g, device="cuda")


def _check_route(logits, k, score="softmax", bias=None, groups=1, kept=1, best=1, renormalise=True, scale=1.0):
    idx, w = batch.route(logits, k, score=score, bias=bias, num_groups=groups, top_groups=kept, group_best=best,
                         renormalise=renormalise, scale=scale)
    want_idx, want_w = ref.route(logits, k, score, bias, groups, kept, best, renormalise, scale)
    assert torch.equal(idx.cpu(), want_idx)
    off = (w.cpu().double() - want_w).abs()
    assert bool((off <= ref.route_tolerance(logits, score, renormalise) * want_w.abs() + 1e-37).all()), float(off.max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,k,groups,kept,best", [
    (1, 1, 1, 1, 1), (2, 2, 1, 1, 1), (7, 3, 1, 1, 1), (16, 16, 1, 1, 1), (61, 8, 1, 1, 1), (64, 8, 8, 3, 2),
    (65, 5, 5, 2, 2), (96, 16, 3, 2, 1), (128, 1, 32, 32, 1), (160, 6, 8, 3, 1), (255, 9, 5, 1, 2),
    (256, 8, 8, 4, 2), (512, 8, 16, 1, 2), (513, 16, 27, 5, 2), (1000, 16, 8, 8, 1), (1024, 16, 32, 1, 2),
])
def test_route(score, experts, k, groups, kept, best):
    g = _gen(experts + k)
    for rows, dtype in ((1, torch.float32), (70, torch.bfloat16), (133, torch.float32)):
        logits = (2 * _normal(g, rows, experts)).to(dtype)
        _check_route(logits, k, score, None, groups, kept, best, True, 1.0)
        _check_route(logits, k, score, 0.1 * _normal(g, experts), groups, kept, best, rows % 2 == 0, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("experts", [48, 256, 640])
def test_route_masks(score, bias, experts):
    """Masked experts in every way, rows with none or too few left, infinite logits."""
    g = _gen(experts)
    logits = _normal(g, 12, experts)
    logits[0] = -math.inf
    logits[1] = torch.finfo(torch.float32).min
    logits[2] = math.nan
    logits[3, 3:] = -math.inf
    logits[4, :experts - 5] = torch.finfo(torch.bfloat16).min
    logits[5, ::2] = math.nan
    logits[6, 17] = math.inf
    logits[7, 5:9] = math.inf
    logits[8] = math.inf
    logits[9, : experts // 2] = -math.inf
    logits[10, 1:] = -1e38
    b = 0.1 * _normal(g, experts) if bias else None
    for dtype in (torch.float32, torch.bfloat16):
        _check_route(logits.to(dtype), 8, score, b)
        _check_route(logits.to(dtype), 8, score, b, 8, 3, 2, False, 1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties(score):
    """Equal logits (all, many, in bf16), equal groups, keys one step of fp32 apart."""
    g = _gen(5)
    flat = torch.zeros(5, 512, device="cuda")
    _check_route(flat, 16, score)
    _check_route(flat, 8, score, None, 8, 3, 2)
    _check_route(flat, 8, score, torch.zeros(512, device="cuda"))
    few = torch.randint(0, 4, (64, 384), generator=g, device="cuda").float()
    _check_route(few, 9, score)
    _check_route(few.bfloat16(), 9, score, None, 8, 4, 2)
    _check_route(few, 9, score, 0.25 * torch.randint(0, 3, (384,), generator=g, device="cuda").float())
    # scores that fp32 keys confuse: logits one step apart around a common value
    near = torch.full((64, 256), 1.25, device="cuda").view(torch.int32)
    near = (near + torch.randint(0, 3, (64, 256), generator=g, device="cuda", dtype=torch.int32)).view(torch.float32)
    _check_route(near, 8, score)
    _check_route(near, 8, score, None, 8, 4, 2)
    _check_route(near, 8, score, 1e-8 * torch.randint(0, 3, (256,), generator=g, device="cuda").float())
    # -0 and +0 are one value
    zeros = torch.where(torch.rand(9, 64, generator=g, device="cuda") < 0.5, 0.0, -0.0)
    _check_route(zeros, 4, score)


def test_route_saturated_scores():
    """Sigmoids of large and very negative logits, which fp32 holds as 1 and 0."""
    g = _gen(6)
    b = 0.1 * _normal(g, 128)
    for shift in (18.0, 30.0, -60.0, -95.0, -300.0):
        logits = _normal(g, 20, 128) + shift
        _check_route(logits, 6, "sigmoid")
        if shift > 0:
            _check_route(logits, 6, "sigmoid", b)
    _check_route(100 * _normal(g, 20, 128), 6, "softmax", None, 4, 2, 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_strides_and_rows_behind(dtype):
    g = _gen(7)
    big = _normal(g, 40, 400).to(dtype)
    for logits in (big[:, :256], big[:, 1:257], big[:, 3:163], big[::2, :256], big[5:6, 8:72]):
        _check_route(logits, 4)
    idx = torch.full((40, 4), 77, dtype=torch.int32, device="cuda")
    w = torch.full((40, 4), 5.0, device="cuda")
    batch.route(big[:33, :256], 4, idx=idx[:33], w=w[:33])
    assert bool((idx[33:] == 77).all()) and bool((w[33:] == 5.0).all())
    assert batch.route(big[:0, :256], 4)[0].shape == (0, 4)


def test_route_captured():
    g = _gen(8)
    logits = _normal(g, 50, 256)
    bias = 0.1 * _normal(g, 256)
    kw = dict(score="sigmoid", bias=bias, num_groups=8, top_groups=4, group_best=2)
    batch.route(logits, 8, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx, w = batch.route(logits, 8, **kw)
    for seed in (1, 2):
        logits.copy_(_normal(_gen(seed), 50, 256))
        graph.replay()
        want = batch.route(logits, 8, **kw)
        assert torch.equal(idx, want[0]) and torch.equal(w, want[1])


# ------------------------------------------------------------------ experts


def _layer(shape, seed):
    return synth.make_layer(shape, seed=seed, device="cuda")


def _choice(g, rows, shape):
    top = torch.topk(_normal(g, rows, shape.num_experts), min(shape.top_k, shape.num_experts), dim=1)
    return top.indices.int(), torch.softmax(top.values, 1)


def _check_experts(shape, layer, x, idx, w, residual=None, **kw):
    out = batch.experts(shape, layer, x, idx, w, residual=residual, **kw)
    want, bound = ref.experts(shape, layer, x, idx, w, residual)
    off = (out.double() - want).abs()
    assert bool((off <= bound).all()), f"{float((off - bound).max()):.3e} over the bound {float(bound.max()):.3e}"
    return out


SHAPES = [
    LayerShape(256, 128, 16, 2, 1), LayerShape(8, 8, 3, 1, 0), LayerShape(136, 72, 5, 3, 2), LayerShape(2560, 768, 24, 8, 1),
    LayerShape(264, 520, 1, 1, 0), LayerShape(1032, 24, 40, 6, 0),
    LayerShape(256, 128, 16, 2, 1, "fp8"), LayerShape(640, 384, 7, 4, 0, "fp8"), LayerShape(2560, 768, 12, 8, 1, "fp8"),
    LayerShape(256, 256, 16, 2, 1, "nvfp4"), LayerShape(768, 512, 6, 3, 0, "nvfp4"), LayerShape(4096, 1024, 9, 8, 0, "nvfp4"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_experts(shape):
    layer = _layer(shape, 3)
    for rows in (1, 2, 17, 100, 333):
        g = _gen(rows)
        x = _normal(g, rows, shape.hidden).bfloat16()
        idx, w = _choice(g, rows, shape)
        _check_experts(shape, layer, x, idx, w)
        _check_experts(shape, layer, x, idx, w, residual=_normal(g, rows, shape.hidden).bfloat16())


@pytest.mark.parametrize("wdtype", ["bf16", "fp8", "nvfp4"])
def test_experts_choices(wdtype):
    """Every row to one expert, none at all, the same one twice, indexes out of range."""
    shape = LayerShape(512, 256, 10, 2, 1, wdtype)
    layer = _layer(shape, 4)
    g = _gen(4)
    rows = 600
    x = _normal(g, rows, 512).bfloat16()
    w = torch.rand(rows, 2, generator=g, device="cuda")
    one = torch.full((rows, 2), 7, dtype=torch.int32, device="cuda")
    _check_experts(shape, layer, x, one, w)
    none = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
    _check_experts(shape, layer, x, none, w)
    bare = dataclasses.replace(shape, num_shared=0)
    r = _normal(g, rows, 512).bfloat16()
    assert torch.equal(_check_experts(bare, layer, x, none, w, residual=r), r)
    mixed = torch.randint(-3, 13, (rows, 2), generator=g, device="cuda", dtype=torch.int32)
    mixed[5] = torch.tensor([2 ** 31 - 1, -2 ** 31], device="cuda")
    _check_experts(shape, layer, x, mixed, w)


def test_experts_row_is_its_own():
    """A row's result is bit for bit the same in any batch of the same launch shape, and bad rows stay among themselves."""
    shape = LayerShape(512, 256, 8, 2, 1)
    layer = _layer(shape, 5)
    g = _gen(5)
    x = _normal(g, 300, 512).bfloat16()
    idx, w = _choice(g, 300, shape)
    out = batch.experts(shape, layer, x, idx, w)
    perm = torch.randperm(300, generator=g, device="cuda")
    again = batch.experts(shape, layer, x[perm].contiguous(), idx[perm].contiguous(), w[perm].contiguous())
    assert torch.equal(out[perm], again)
    bad = x.clone()
    bad[10], bad[200] = math.nan, math.inf
    got = batch.experts(shape, layer, bad, idx, w)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[10] = keep[200] = False
    assert torch.equal(got[keep], out[keep]) and bool(torch.isnan(got[10]).all())


def test_experts_strides_places_and_workspace():
    """Rows with a stride, out in the residual's place, a used workspace, rows behind the batch."""
    shape = LayerShape(256, 128, 16, 2, 1)
    layer = _layer(shape, 6)
    g = _gen(6)
    wide = _normal(g, 64, 512).bfloat16()
    idx, w = _choice(g, 64, shape)
    ws = torch.full((batch.experts_workspace(shape, 64),), 255, dtype=torch.uint8, device="cuda")
    for x in (wide[:, :256], wide[:, 8:264], wide[::2, 256:], wide[3:4, 16:272]):
        n = x.shape[0]
        _check_experts(shape, layer, x, idx[:n], w[:n], workspace=ws)
        assert batch.status(ws) == _lib.MOE_OK
    r = _normal(g, 64, 256).bfloat16()
    want = batch.experts(shape, layer, wide[:40, :256], idx[:40], w[:40], residual=r[:40])
    out = r.clone()
    batch.experts(shape, layer, wide[:40, :256], idx[:40], w[:40], residual=out[:40], out=out[:40])
    assert torch.equal(out[:40], want) and torch.equal(out[40:], r[40:])
    with pytest.raises(ValueError):
        batch.experts(shape, layer, wide[:, :256], idx, w, workspace=ws[:1000])
    with pytest.raises(_lib.MoEDecodeError):  # rows off 16 bytes
        batch.experts(shape, layer, wide[:, 1:257], idx, w)
    assert batch.experts(shape, layer, wide[:0, :256], idx[:0], w[:0]).shape == (0, 256)


def test_experts_rounds():
    """More rows than one round of launches takes; the last round is short."""
    shape = LayerShape(64, 32, 4, 2, 1)
    layer = _layer(shape, 7)
    g = _gen(7)
    rows = 16384 * 2 + 5
    x = _normal(g, rows, 64).bfloat16()
    idx, w = _choice(g, rows, shape)
    ws = torch.empty(batch.experts_workspace(shape, rows), dtype=torch.uint8, device="cuda")
    _check_experts(shape, layer, x, idx, w, residual=x, workspace=ws)
    assert batch.status(ws) == _lib.MOE_OK


def test_experts_streams_and_graphs():
    """Two calls at once on two streams; two captured graphs, each with its own workspace, replayed in turn and at once."""
    shape = LayerShape(512, 256, 32, 4, 1)
    layer = _layer(shape, 8)
    sets = []
    for seed in (1, 2):
        g = _gen(seed)
        x = _normal(g, 200 * seed, 512).bfloat16()
        sets.append((x, *_choice(g, 200 * seed, shape)))
    want = [batch.experts(shape, layer, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [batch.experts(shape, layer, *s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(batch.experts(shape, layer, *s))
    for st, gr in zip(streams, graphs):
        with torch.cuda.stream(st):
            gr.replay()
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    sets[0][0].copy_(_normal(_gen(9), 200, 512).bfloat16())
    graphs[0].replay()
    assert torch.equal(outs[0], batch.experts(shape, layer, *sets[0]))


# ------------------------------------------------------------------ project


def _adapters(g, n, r, k, o, scale=True):
    return batch.Adapters((_normal(g, n, r, k) / math.sqrt(k)).bfloat16(), (0.1 * _normal(g, n, o, r)).bfloat16(),
                          0.5 + torch.rand(n, generator=g, device="cuda") if scale else None)


def _check_project(x, weight, wdtype="bf16", **kw):
    out = batch.project(x, weight, wdtype=wdtype, **kw)
    w64 = weight.double() if wdtype == "bf16" else ref.fp8(*weight) if wdtype == "fp8" else ref.nvfp4(*weight)
    # the NVFP4 tensor scale is rounded into the weights where adapters share the sum
    widened = wdtype == "fp8" or (wdtype == "nvfp4" and kw.get("adapters") is not None)
    want, bound = ref.project(x, w64, kw.get("adapters"), kw.get("adapter_ids"), kw.get("addend"),
                              kw.get("swiglu", False), widened, out.dtype == torch.bfloat16)
    off = (out.double() - want).abs()
    assert bool((off <= bound).all()), f"{float((off - bound).max()):.3e} over the bound {float(bound.max()):.3e}"
    return out


@pytest.mark.parametrize("inner,outer,rank,count", [(8, 8, 8, 1), (256, 128, 16, 3), (200, 520, 24, 5), (2560, 1536, 64, 16),
                                                    (1024, 4096, 128, 4), (72, 264, 72, 200), (512, 256, 256, 2),
                                                    (128, 64, 8, 1024)])
def test_project(inner, outer, rank, count):
    g = _gen(inner + rank)
    weight = (0.05 * _normal(g, outer, inner)).bfloat16()
    ad = _adapters(g, count, rank, inner, outer, scale=rank != 24)
    for rows in (1, 5, 16, 64, 300, 700):
        x = _normal(g, rows, inner).bfloat16()
        ids = torch.randint(-1, count, (rows,), generator=g, device="cuda", dtype=torch.int32)
        add = _normal(g, rows, outer).bfloat16()
        _check_project(x, weight)
        _check_project(x, weight, out_dtype=torch.float32)
        _check_project(x, weight, adapters=ad, adapter_ids=ids)
        _check_project(x, weight, adapters=ad, adapter_ids=ids, addend=add, out_dtype=torch.float32)
        _check_project(x, weight, addend=add)
        if outer % 16 == 0:
            _check_project(x, weight, adapters=ad, adapter_ids=ids, swiglu=True)
            _check_project(x, weight, swiglu=True)


@pytest.mark.parametrize("wdtype", ["fp8", "nvfp4"])
@pytest.mark.parametrize("swiglu", [False, True])
def test_project_quantised(wdtype, swiglu):
    g = _gen(11)
    inner, outer = 512, 512
    w = 0.05 * _normal(g, outer, inner)
    if wdtype == "fp8":
        weight = synth.quantize_fp8_block(w)
    else:
        parts = [synth.quantize_nvfp4(h) for h in (w.chunk(2) if swiglu else (3 * w,))]
        weight = (torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts]),
                  torch.stack([p[2] for p in parts]) if swiglu else parts[0][2])
    ad = _adapters(g, 3, 16, inner, outer)
    for rows in (1, 40, 257):
        x = _normal(g, rows, inner).bfloat16()
        ids = torch.randint(-1, 3, (rows,), generator=g, device="cuda", dtype=torch.int32)
        _check_project(x, weight, wdtype, swiglu=swiglu)
        _check_project(x, weight, wdtype, swiglu=swiglu, adapters=ad, adapter_ids=ids)


@pytest.mark.parametrize("outer", [2, 6, 20, 60, 126, 250])
def test_project_even_widths(outer):
    """As many columns as a router has experts."""
    g = _gen(outer)
    weight = (0.05 * _normal(g, outer, 264)).bfloat16()
    ad = _adapters(g, 3, 16, 264, outer)
    for rows in (1, 33, 400):
        x = _normal(g, rows, 264).bfloat16()
        ids = torch.randint(-1, 3, (rows,), generator=g, device="cuda", dtype=torch.int32)
        add = _normal(g, rows, outer).bfloat16()
        _check_project(x, weight, out_dtype=torch.float32)
        _check_project(x, weight, adapters=ad, adapter_ids=ids, addend=add)
        if outer % 4 == 0:
            _check_project(x, weight, adapters=ad, adapter_ids=ids, swiglu=True)


def test_project_ids():
    """All rows one adapter's, none at all, every row its own, ids out of range; adapters of no row may hold anything."""
    g = _gen(12)
    weight = (0.05 * _normal(g, 384, 256)).bfloat16()
    ad = _adapters(g, 40, 32, 256, 384)
    ad.a[11], ad.b[11] = math.nan, math.inf
    x = _normal(g, 40, 256).bfloat16()
    add = _normal(g, 40, 384).bfloat16()
    every = torch.randperm(40, generator=g, device="cuda").int()
    every[every == 11] = 12
    odd = every.clone()
    odd[:6] = torch.tensor([-1, -5, 40, 41, 2 ** 31 - 1, -2 ** 31], device="cuda")
    for ids in (torch.full_like(every, 39), torch.full_like(every, -1), every, odd):
        _check_project(x, weight, adapters=ad, adapter_ids=ids)
        out = add.clone()
        want = _check_project(x, weight, adapters=ad, adapter_ids=ids, addend=add)
        assert torch.equal(batch.project(x, weight, adapters=ad, adapter_ids=ids, addend=out, out=out), want)
    # rows of NaN and infinities, and adapters that make them, stay among themselves
    bad = x.clone()
    bad[3] = math.nan
    ids = every.clone()
    ids[8] = 11
    good = batch.project(x, weight, adapters=ad, adapter_ids=every)
    got = batch.project(bad, weight, adapters=ad, adapter_ids=ids)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[3] = keep[8] = False
    assert torch.equal(got[keep], good[keep]) and bool(torch.isnan(got[3]).all()) and bool(torch.isnan(got[8]).any())


def test_project_strides_streams_and_graphs():
    g = _gen(13)
    weight = (0.05 * _normal(g, 256, 512)).bfloat16()
    ad = _adapters(g, 8, 16, 512, 256)
    wide = _normal(g, 90, 1024).bfloat16()
    ids = torch.randint(-1, 8, (90,), generator=g, device="cuda", dtype=torch.int32)
    for x in (wide[:, :512], wide[:, 8:520], wide[::3, 512:]):
        _check_project(x, weight, adapters=ad, adapter_ids=ids[:x.shape[0]].contiguous())
    out = torch.full((90, 256), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((batch.project_workspace(512, 256, 90, rank=16, num_adapters=8),), 255, dtype=torch.uint8, device="cuda")
    batch.project(wide[:77, :512], weight, adapters=ad, adapter_ids=ids[:77], out=out[:77], workspace=ws)
    assert bool((out[77:] == 9.0).all()) and batch.status(ws) == _lib.MOE_OK
    batch.project(wide[:20, :512], weight, out=out[:20], workspace=ws)
    assert batch.status(ws) == _lib.MOE_OK
    x = wide[:, :512].contiguous()
    want = batch.project(x, weight, adapters=ad, adapter_ids=ids)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [batch.project(x, weight, adapters=ad, adapter_ids=ids, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) for a in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = batch.project(x, weight, adapters=ad, adapter_ids=ids)
    ids.copy_(torch.randint(-1, 8, (90,), generator=g, device="cuda", dtype=torch.int32))
    graph.replay()
    assert torch.equal(out, batch.project(x, weight, adapters=ad, adapter_ids=ids))


def test_project_of_few_rows_on_many_streams():
    """Calls whose CTAs wait for one another (a tile's K shared in a cluster), several at once on the same SMs."""
    g = _gen(14)
    weight = (0.05 * _normal(g, 1536, 4096)).bfloat16()
    ad = _adapters(g, 8, 16, 4096, 1536)
    xs = [_normal(g, n, 4096).bfloat16() for n in (1, 7, 16, 40)]
    ids = [torch.randint(-1, 8, (x.shape[0],), generator=g, device="cuda", dtype=torch.int32) for x in xs]
    want = [_check_project(x, weight, adapters=ad, adapter_ids=i, swiglu=n % 2 == 1) for n, (x, i) in enumerate(zip(xs, ids))]
    want32 = [_check_project(x, weight, out_dtype=torch.float32) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        got, got32 = [], []
        for n, st in enumerate(streams):
            got.append(batch.project(xs[n], weight, adapters=ad, adapter_ids=ids[n], swiglu=n % 2 == 1, stream=st))
            got32.append(batch.project(xs[n], weight, out_dtype=torch.float32, stream=st))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got + got32, want + want32))


@pytest.mark.parametrize("bias", [math.inf, -math.inf, math.nan])
def test_route_bias_not_finite(bias):
    """An expert whose bias is +inf is chosen first; one whose bias is -inf or NaN is not to be had."""
    g = _gen(15)
    logits = _normal(g, 30, 96)
    b = 0.1 * _normal(g, 96)
    b[40] = bias
    idx, w = batch.route(logits, 6, score="sigmoid", bias=b)
    if bias == math.inf:
        assert bool((idx[:, 0] == 40).all())
    else:
        masked = logits.clone()
        masked[:, 40] = -math.inf
        want = batch.route(masked, 6, score="sigmoid", bias=torch.where(torch.isfinite(b), b, torch.zeros_like(b)))
        assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
        kw = dict(score="sigmoid", num_groups=8, top_groups=2, group_best=2)
        got = batch.route(logits, 6, bias=b, **kw)
        want = batch.route(masked, 6, bias=torch.where(torch.isfinite(b), b, torch.zeros_like(b)), **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ the layer


def test_layer_with_an_even_number_of_experts():
    """A layer whose experts are no multiple of 8, on 50 rows against the C++ oracle."""
    shape = LayerShape(256, 128, 22, 3, 1)
    layer = _layer(shape, 16)
    layer["router_w"] = (4 * layer["router_w"].float()).bfloat16()
    x = helpers.hidden_with_margin(layer["router_w"], 50, 3, seed=3, margin=0.002)
    from moe_decode_layer_gb300.layer import MoEDecodeLayer
    mod = MoEDecodeLayer(shape, layer, max_rows=1)
    want, ridx, rw = helpers.oracle_layer(shape, layer, x, x)
    idx = torch.empty(50, 3, dtype=torch.int32, device="cuda")
    w = torch.empty(50, 3, device="cuda")
    helpers.assert_close(mod.run_rows(x.cuda(), topk_idx=idx, topk_w=w).cpu(), want)
    helpers.assert_routing(idx, w, ridx, rw)
    mod.close()


@pytest.mark.parametrize("wdtype,score", [("bf16", 0), ("bf16", 1), ("fp8", 0), ("nvfp4", 1)])
def test_layer_of_many_rows(wdtype, score):
    """The layer on a batch beyond the decode step's 16 rows, against the C++ oracle, and on 8 rows against the step itself."""
    shape = LayerShape(256, 256, 32, 4, 1, wdtype)
    layer = _layer(shape, 14)
    layer["router_w"] = (4 * layer["router_w"].float()).bfloat16()
    if score:
        layer["router_bias"] = synth.router_bias(32, 3, "cuda", 0.2)
    x = helpers.hidden_with_margin(layer["router_w"], 40, 4, seed=2, score=score, bias=layer.get("router_bias"), margin=0.002)
    from moe_decode_layer_gb300.layer import MoEDecodeLayer
    mod = MoEDecodeLayer(shape, layer, max_rows=8, score=score, routed_scale=1.5)
    xd = x.cuda()
    idx = torch.empty(40, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(40, 4, device="cuda")
    out = mod.run_rows(xd, topk_idx=idx, topk_w=w)
    want, ridx, rw = helpers.oracle_layer(shape, layer, x, x, 1.5, score, layer.get("router_bias"))
    helpers.assert_routing(idx, w / 1.5, ridx, rw, by_weight=score == 0)
    helpers.assert_close(out.cpu(), want)
    step = mod.run(xd[:8].contiguous())
    helpers.assert_close(step.cpu(), want[:8])
    mod.close()


def test_layer_with_adapters_and_groups():
    """A run of all operators: groups in the choice, and requests' adapters on the shared expert."""
    shape = LayerShape(512, 256, 32, 4, 1)
    layer = _layer(shape, 15)
    layer["router_bias"] = synth.router_bias(32, 3, "cuda", 0.2)
    from moe_decode_layer_gb300.layer import MoEDecodeLayer
    mod = MoEDecodeLayer(shape, layer, max_rows=1, score=1, routed_scale=2.5)
    g = _gen(15)
    x, r = _normal(g, 150, 512).bfloat16(), _normal(g, 150, 512).bfloat16()
    up, down = _adapters(g, 6, 16, 512, 512), _adapters(g, 6, 8, 256, 512)
    ids = torch.randint(-1, 6, (150,), generator=g, device="cuda", dtype=torch.int32)
    idx = torch.empty(150, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(150, 4, device="cuda")
    out = mod.run_rows(x, r, topk_idx=idx, topk_w=w, num_groups=8, top_groups=3, group_best=2, adapters=(up, down),
                       adapter_ids=ids)
    logits = batch.project(x, layer["router_w"], out_dtype=torch.float32)
    want_idx, want_w = ref.route(logits, 4, "sigmoid", layer["router_bias"], 8, 3, 2, True, 2.5)
    assert torch.equal(idx.cpu(), want_idx)
    h, dh = ref.project(x, layer["sh_w13"][0].double(), up, ids, swiglu=True)
    shared, ds = ref.project(h.bfloat16(), layer["sh_w2"][0].double(), down, ids, addend=r)
    # h is off by its bound on the way through the down matrix and its adapters
    through = layer["sh_w2"][0].double().abs().expand(150, -1, -1)
    ds = ds + torch.einsum("toi,ti->to", through, dh + ref.BF16 * h.abs())
    for a in range(6):
        rows = ids == a
        ds[rows] += float(down.scale[a]) * (((dh + ref.BF16 * h.abs())[rows] @ down.a[a].double().abs().t()) @
                                            down.b[a].double().abs().t())
    routed, dr = ref.experts(dataclasses.replace(shape, num_shared=0), layer, x, idx, w)
    off = (out.double() - (shared + routed)).abs()
    assert bool((off <= 1.01 * (ds + dr + ref.BF16 * (shared + routed).abs()) + 1e-6).all())
    with pytest.raises(ValueError):
        mod.run_rows(x, r, adapter_ids=ids)
    mod.close()
    norm = MoEDecodeLayer(shape, layer, max_rows=1, pre_rmsnorm=True)
    with pytest.raises(ValueError):
        norm.run_rows(x)
    norm.close()
