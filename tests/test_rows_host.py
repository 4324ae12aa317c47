"""Host side of the many-row operators (no GPU): what the configuration checks take
and refuse, workspace sizes, and calls that are refused before any device work."""

import ctypes

import pytest
import torch

from moe_decode_layer_gb300 import LayerShape, _lib, batch

OK, BAD, UNSUPPORTED = _lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED


def _route(**kw):
    base = dict(num_experts=256, top_k=8, score=0, num_groups=1, top_groups=1, group_best=1, renormalise=1,
                logits_dtype=1, scale=1.0)
    base.update(kw)
    return _lib.RouteConfig(**base)


def _experts(**kw):
    base = dict(hidden=256, inter=128, num_experts=16, top_k=2, num_shared=1, wdtype=0)
    base.update(kw)
    return _lib.ExpertsConfig(**base)


def _project(**kw):
    base = dict(inner=256, outer=128, swiglu=0, wdtype=0, rank=16, num_adapters=4, out_dtype=0)
    base.update(kw)
    return _lib.ProjectConfig(**base)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(num_experts=1, top_k=1), OK), (dict(num_experts=1024, top_k=16), OK),
    (dict(num_groups=8, top_groups=4, group_best=2), OK), (dict(num_groups=32, top_groups=1), OK),
    (dict(num_experts=0), BAD), (dict(top_k=0), BAD), (dict(num_groups=0), BAD), (dict(top_groups=2), BAD),
    (dict(scale=float("nan")), BAD), (dict(num_experts=1025), UNSUPPORTED), (dict(top_k=17), UNSUPPORTED),
    (dict(num_experts=4), UNSUPPORTED), (dict(num_groups=64, top_groups=64), UNSUPPORTED),
    (dict(num_groups=3, top_groups=3), UNSUPPORTED), (dict(num_groups=64), UNSUPPORTED),
    (dict(num_groups=32, top_groups=1, top_k=9), UNSUPPORTED), (dict(group_best=3), UNSUPPORTED),
    (dict(score=2), UNSUPPORTED), (dict(logits_dtype=2), UNSUPPORTED),
])
def test_route_check(kw, status):
    assert _lib.load().moe_decode_route_check(_route(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(hidden=8, inter=8), OK), (dict(num_shared=0), OK), (dict(wdtype=2), OK),
    (dict(wdtype=1, inter=256), OK), (dict(top_k=16, num_experts=4), OK), (dict(hidden=16384), OK),
    (dict(hidden=0), BAD), (dict(num_shared=-1), BAD), (dict(top_k=0), BAD),
    (dict(hidden=12), UNSUPPORTED), (dict(inter=20), UNSUPPORTED), (dict(wdtype=2, inter=64), UNSUPPORTED),
    (dict(wdtype=1), UNSUPPORTED), (dict(wdtype=3), UNSUPPORTED), (dict(num_experts=1025), UNSUPPORTED),
    (dict(top_k=17), UNSUPPORTED), (dict(num_shared=5), UNSUPPORTED), (dict(hidden=16392), UNSUPPORTED),
])
def test_experts_check(kw, status):
    assert _lib.load().moe_decode_experts_check(_experts(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(num_adapters=0, rank=0), OK), (dict(rank=256), OK), (dict(swiglu=1), OK), (dict(out_dtype=1), OK),
    (dict(wdtype=2), OK), (dict(wdtype=1, outer=256), OK), (dict(num_adapters=1024), OK),
    (dict(inner=0), BAD), (dict(num_adapters=-1), BAD), (dict(rank=0), BAD),
    (dict(rank=12), UNSUPPORTED), (dict(rank=264), UNSUPPORTED), (dict(num_adapters=1025), UNSUPPORTED),
    (dict(inner=252), UNSUPPORTED), (dict(outer=100), OK), (dict(outer=101), UNSUPPORTED), (dict(outer=16386), UNSUPPORTED), (dict(wdtype=2, outer=100), UNSUPPORTED), (dict(swiglu=1, out_dtype=1), UNSUPPORTED),
    (dict(out_dtype=2), UNSUPPORTED), (dict(wdtype=2, inner=64), UNSUPPORTED),
])
def test_project_check(kw, status):
    assert _lib.load().moe_decode_project_check(_project(**kw)) == status


def test_null_configs():
    lib = _lib.load()
    for f in (lib.moe_decode_route_check, lib.moe_decode_experts_check, lib.moe_decode_project_check):
        assert f(None) == BAD


def test_workspace_grows_with_rows():
    shape = LayerShape(256, 128, 16, 2, 1)
    sizes = [batch.experts_workspace(shape, t) for t in range(0, 3000, 7)]
    assert sizes[0] == 0 and sizes == sorted(sizes)
    # rounds of at most 16384 rows share one workspace
    assert batch.experts_workspace(shape, 16384) == batch.experts_workspace(shape, 1 << 20)
    for e in (1, 16, 1024):
        small = LayerShape(8, 8, e, 1, 0)
        sizes = [batch.experts_workspace(small, t) for t in range(1, 9000)]
        assert sizes == sorted(sizes)
    for n in (1, 4, 64, 1024):
        sizes = [batch.project_workspace(256, 128, t, rank=256, num_adapters=n) for t in range(0, 3000)]
        assert sizes == sorted(sizes)


@pytest.mark.parametrize("rows,status", [(-1, BAD), ((1 << 24) + 1, BAD), (0, OK)])
def test_rows_out_of_range(rows, status):
    lib, n, p = _lib.load(), ctypes.c_size_t(), ctypes.c_void_p(1 << 20)
    assert lib.moe_decode_route(_route(), p, 256, None, rows, p, p, None) == status
    assert lib.moe_decode_experts_workspace(_experts(), rows, n) == status
    assert lib.moe_decode_project_workspace(_project(), rows, n) == status
    w = _lib.Weights()
    assert lib.moe_decode_experts(_experts(), w, p, 256, p, p, None, p, rows, p, 0, None) == status
    assert lib.moe_decode_project(_project(), _lib.ProjectWeights(), p, 256, p, None, p, rows, p, 0, None) == status


def _p(v):
    return ctypes.c_void_p(v)


@pytest.mark.parametrize("kw", [dict(logits=None), dict(idx=None), dict(w=None), dict(stride=255),
                                dict(logits=_p(4098)), dict(idx=_p(4097)), dict(bias=_p(4098))])
def test_route_refuses(kw):
    a = dict(logits=_p(4096), stride=256, bias=None, idx=_p(4096), w=_p(4096))
    a.update(kw)
    assert _lib.load().moe_decode_route(_route(), a["logits"], a["stride"], a["bias"], 4, a["idx"], a["w"], None) == BAD


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=_p(4104)), dict(stride=248), dict(stride=260), dict(idx=None),
                                dict(w=None), dict(out=None), dict(out=_p(4100)), dict(residual=_p(4104)),
                                dict(ws=None), dict(ws=_p(4104)), dict(ws_bytes=1000), dict(w13=None), dict(w2=_p(4104)),
                                dict(sh_w13=None), dict(wdtype=2), dict(wdtype=2, w13_scale=_p(4104))])
def test_experts_refuses(kw):
    a = dict(x=_p(4096), stride=256, idx=_p(4096), w=_p(4096), residual=None, out=_p(4096), ws=_p(4096), ws_bytes=1 << 30,
             wdtype=0, w13=_p(4096), w2=_p(4096), sh_w13=_p(4096), sh_w2=_p(4096), w13_scale=None)
    a.update(kw)
    wt = _lib.Weights()
    for n in ("w13", "w2", "sh_w13", "sh_w2", "w13_scale"):
        setattr(wt, n, a[n])
    assert _lib.load().moe_decode_experts(_experts(wdtype=a["wdtype"]), wt, a["x"], a["stride"], a["idx"], a["w"],
                                          a["residual"], a["out"], 4, a["ws"], a["ws_bytes"], None) == BAD


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=_p(4104)), dict(stride=248), dict(stride=260), dict(ids=None),
                                dict(out=None), dict(addend=_p(4104)), dict(swiglu=1, addend=_p(4096)), dict(ws=None),
                                dict(ws_bytes=100), dict(weight=None), dict(a=None), dict(b=_p(4104)), dict(wdtype=2)])
def test_project_refuses(kw):
    a = dict(x=_p(4096), stride=256, ids=_p(4096), addend=None, out=_p(4096), ws=_p(4096), ws_bytes=1 << 30,
             weight=_p(4096), a=_p(4096), b=_p(4096), swiglu=0, wdtype=0)
    a.update(kw)
    wt = _lib.ProjectWeights()
    wt.w, wt.a, wt.b = a["weight"], a["a"], a["b"]
    assert _lib.load().moe_decode_project(_project(swiglu=a["swiglu"], wdtype=a["wdtype"]), wt, a["x"], a["stride"],
                                          a["ids"], a["addend"], a["out"], 4, a["ws"], a["ws_bytes"], None) == BAD


def test_binding_refuses():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a CUDA device
        batch.route(x, 8)
    with pytest.raises(ValueError):
        batch.route(x.double(), 8)
    with pytest.raises(ValueError):
        batch.route(x, 8, score="other")
    with pytest.raises(ValueError):  # columns with a stride
        batch.route(torch.zeros(256, 4, dtype=torch.bfloat16).t(), 8)
    with pytest.raises(_lib.MoEDecodeError):
        batch.route(x, 17)
    with pytest.raises(ValueError):  # a bias of another length
        batch.route(x, 8, bias=torch.zeros(255))
    shape = LayerShape(256, 128, 16, 2, 0)
    layer = {"w13": torch.zeros(16, 256, 256, dtype=torch.bfloat16), "w2": torch.zeros(16, 256, 128, dtype=torch.bfloat16)}
    idx, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for bad in (dict(x=x.float()), dict(idx=idx.long()), dict(w=w.double()), dict(idx=idx[:3]),
                dict(residual=x[:, :128]), dict(weights={**layer, "w2_layout": "i_h"}),
                dict(weights={**layer, "w2": layer["w2"].transpose(1, 2)}), dict(weights={})):
        a = dict(weights=layer, x=x, idx=idx, w=w)
        a.update(bad)
        with pytest.raises(ValueError):
            batch.experts(shape, a["weights"], a["x"], a["idx"], a["w"], residual=a.get("residual"))
    weight = torch.zeros(128, 256, dtype=torch.bfloat16)
    ad = batch.Adapters(torch.zeros(4, 16, 256, dtype=torch.bfloat16), torch.zeros(4, 128, 16, dtype=torch.bfloat16))
    ids = torch.zeros(4, dtype=torch.int32)
    for bad in (dict(adapters=ad), dict(adapter_ids=ids), dict(adapters=ad, adapter_ids=ids.long()),
                dict(adapters=ad._replace(b=ad.b[:, :64]), adapter_ids=ids), dict(weight=weight[:, :128]),
                dict(weight=weight.float()), dict(out_dtype=torch.float16), dict(wdtype="fp8"), dict(wdtype="int8"),
                dict(addend=x), dict(adapters=ad._replace(scale=torch.zeros(3)), adapter_ids=ids)):
        a = dict(weight=weight)
        a.update(bad)
        with pytest.raises(ValueError):
            batch.project(x, a.pop("weight"), **a)
