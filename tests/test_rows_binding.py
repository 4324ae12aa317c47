"""The binding of the many-row operators without a GPU: weights kept as a C struct, devices and streams."""

import contextlib
import dataclasses
import gc
import types
import weakref

import pytest
import torch

from moe_decode_layer_gb300 import LayerShape, _lib, batch
from moe_decode_layer_gb300.layer import MoEDecodeLayer

SHAPE = LayerShape(256, 128, 16, 2, 1)


def _layer():
    return {n: torch.zeros(s, dtype=torch.bfloat16) for n, s in (("w13", (16, 256, 256)), ("w2", (16, 256, 128)),
                                                                 ("sh_w13", (1, 256, 256)), ("sh_w2", (1, 256, 128)))}


def test_weights_struct_keeps_its_tensors():
    """The addresses that a call will read stay valid when the dict goes."""
    layer = _layer()
    refs = [weakref.ref(t) for t in layer.values()]
    w = batch.expert_weights(SHAPE, layer, torch.device("cpu"))
    addresses = [t.data_ptr() for t in layer.values()]
    del layer
    gc.collect()
    assert all(r() is not None for r in refs)
    assert [w.w13, w.w2, w.sh_w13, w.sh_w2] == addresses
    del w
    gc.collect()
    assert all(r() is None for r in refs)


def test_weights_struct_of_another_layer_is_refused():
    """Sizes that the kernels would read past, and another device."""
    w = batch.expert_weights(SHAPE, _layer(), -1)
    x, idx, f = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for kw in (dict(inter=256), dict(num_experts=17), dict(num_shared=2), dict(wdtype="fp8")):
        with pytest.raises(ValueError, match="these weights are of"):
            batch.experts(dataclasses.replace(SHAPE, **kw), w, x, idx, f)
    with pytest.raises(ValueError, match="these weights are of"):
        batch._made_for(w, SHAPE, 0)
    with pytest.raises(ValueError, match="what expert_weights made"):
        batch.experts(SHAPE, _lib.Weights(), x, idx, f)
    # other choices, or without the shared expert: the same weights
    for kw in (dict(), dict(top_k=3), dict(num_shared=0)):
        assert batch._made_for(w, dataclasses.replace(SHAPE, **kw), -1) is w


def test_weights_on_the_current_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    with pytest.raises(ValueError, match="on device 3: got"):
        batch.expert_weights(SHAPE, _layer(), torch.device("cuda"))


@pytest.mark.parametrize("cfg,shape,kw", [
    (dict(pre_rmsnorm=1), SHAPE, {}), (dict(w2_layout=1), SHAPE, {}), ({}, SHAPE, dict(adapter_ids=0)), ({}, SHAPE, dict(adapters=(0, 0))),
    ({}, dataclasses.replace(SHAPE, num_shared=2), dict(adapters=(0, 0), adapter_ids=0)),
    ({}, dataclasses.replace(SHAPE, num_shared=0), dict(adapters=(0, 0), adapter_ids=0))], ids=str)
def test_layer_refuses_before_any_operator_runs(monkeypatch, cfg, shape, kw):
    """What run_rows does not take is refused as a whole: no operator of it has been called."""
    for name in ("project", "route", "experts", "contiguous"):
        monkeypatch.setattr(batch, name, lambda *a, **k: pytest.fail("an operator was called"))
    mod = MoEDecodeLayer.__new__(MoEDecodeLayer)
    mod.shape, mod._weights, mod._cfg = shape, {}, _lib.Config(**cfg)
    with pytest.raises(ValueError):
        mod.run_rows(torch.zeros(4, 256, dtype=torch.bfloat16), **kw)


@pytest.fixture
def two_devices(monkeypatch):
    """torch's device and stream contexts as a log; device 0 is current."""
    log = []

    def context(name):
        @contextlib.contextmanager
        def enter(what):
            log.append((name, what))
            yield
            log.append((name, "left"))
        return enter

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    monkeypatch.setattr(torch.cuda, "device", context("device"))
    monkeypatch.setattr(torch.cuda, "stream", context("stream"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: _stream(dev, 200 + dev))
    return log


def _stream(dev, handle):
    return types.SimpleNamespace(device=torch.device("cuda", dev), cuda_stream=handle)


def test_devices_and_streams_of_a_call(two_devices):
    """Tensors on the current device, on another one, and a stream that is given: the handle the library gets,
    what is current while it is called, and that both are left again in order."""
    assert batch._enter(0, None) == (100, None) and two_devices == []
    handle, leave = batch._enter(1, None)
    assert handle == 201 and two_devices == [("device", 1)]
    leave.close()
    assert two_devices == [("device", 1), ("device", "left")]
    for dev in (0, 1):
        two_devices.clear()
        stream = _stream(dev, 7)
        handle, leave = batch._enter(dev, stream)
        assert handle == 7 and two_devices == [("device", dev), ("stream", stream)]
        leave.close()
        assert two_devices[2:] == [("stream", "left"), ("device", "left")]


def test_streams_of_another_device_are_refused(two_devices):
    """The stream's context would make its own device current, which is not the buffers'."""
    for dev in (0, 1):
        with pytest.raises(ValueError, match="a stream of device"):
            batch._enter(dev, _stream(1 - dev, 7))
    with pytest.raises(ValueError, match="CUDA device"):
        batch._enter(-1, None)
    assert two_devices == []
