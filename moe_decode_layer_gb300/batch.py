"""The MoE layer's operators for any number of rows, over torch tensors.

``route``, ``experts`` and ``project`` marshal tensors into the C entry points of
include/moe_decode_rows.h, which document what is computed. They check shapes,
types and devices, allocate results (and a workspace, unless one is given) with
torch's allocator on the stream they run on, and enqueue their work on the current
stream (or ``stream``) without waiting. No arithmetic happens here.

A workspace that is handed in must not be in use by another call at the same time,
and must stay alive while a CUDA graph that captured a call with it is replayed.
``status`` reads from it whether the call's device-side waits ended in time; a call
without one leaves nothing behind that could be asked.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import NamedTuple

import torch

from . import _lib
from .synth import LayerShape

_DTYPES = {torch.bfloat16: _lib.MOE_BF16, torch.float32: _lib.MOE_F32}


class Adapters(NamedTuple):
    """Low-rank adapters: a bf16 [L, r, K], b bf16 [L, O, r] ([L, 2 O, r] beside a
    gate/up projection), scale fp32 [L] or None (1). r % 8 == 0."""

    a: torch.Tensor
    b: torch.Tensor
    scale: torch.Tensor | None = None


def _need(cond: bool, what: str) -> None:
    if not cond:
        raise ValueError(what)


def _tensor(t: torch.Tensor, name: str, dtype, shape, dev: int) -> int:
    """The address of a contiguous tensor of this type, shape and device index (-1: the CPU)."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on device {dev}: got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, cols: int, dev: int) -> tuple[int, int, int]:
    """(address, rows, row stride) of a bf16 [T, cols] tensor whose rows are contiguous."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not torch.bfloat16 or t.get_device() != dev or len(shape) != 2 or shape[1] != cols or \
            (shape[0] and stride[1] != 1):
        raise ValueError(f"{name} must be a bf16 [rows, {cols}] tensor on device {dev} with contiguous rows: got "
                         f"{t.dtype} {tuple(shape)} on {t.device}")
    # one row, or none, has no stride of its own
    return t.data_ptr(), shape[0], stride[0] if shape[0] > 1 else cols


def _enter(dev: int, stream):
    """(stream handle, what to leave): makes device ``dev`` the current one while the
    library is called, and ``stream`` the one that results and workspaces are allocated
    for. The usual call, on the current device and stream, has nothing to leave."""
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"a stream of device {stream.device.index} for tensors on device {dev}")
    if stream is None and dev == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(dev), None
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(dev))
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    else:
        stack.enter_context(torch.cuda.stream(stream))
    return stream.cuda_stream, stack


def contiguous(t: torch.Tensor, stream=None) -> torch.Tensor:
    """A contiguous copy of ``t``, made and allocated on the stream that the operators run on."""
    _, leave = _enter(t.get_device(), stream)
    try:
        return t.contiguous()
    finally:
        if leave is not None:
            leave.close()


@functools.lru_cache(maxsize=256)
def _route_config(e: int, top_k: int, score: str, num_groups: int, top_groups: int, group_best: int,
                  renormalise: bool, dtype, scale: float) -> _lib.RouteConfig:
    _need(score in _lib.ROUTE_SCORES, f"unknown score {score!r}")
    cfg = _lib.RouteConfig(e, top_k, _lib.ROUTE_SCORES[score], num_groups, top_groups, group_best, renormalise,
                           _DTYPES[dtype], scale)
    _lib.check(_lib.load().moe_decode_route_check(cfg), "moe_decode_route_check")
    return cfg


def route(logits: torch.Tensor, top_k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
          num_groups: int = 1, top_groups: int = 1, group_best: int = 1, renormalise: bool = True, scale: float = 1.0,
          idx: torch.Tensor | None = None, w: torch.Tensor | None = None, stream=None):
    """The chosen experts of each row of ``logits`` (bf16 or fp32 [T, E], any row
    stride) and their weights: (int32 [T, k], fp32 [T, k]), as moe_decode_route
    documents. ``score``: "softmax" or "sigmoid"; ``bias`` fp32 [E]."""
    dtype = logits.dtype
    if logits.dim() != 2 or dtype not in _DTYPES:
        raise ValueError("logits must be a bf16 or fp32 [rows, experts] tensor")
    t, e = logits.shape
    row, col = logits.stride()
    if col != 1 and t and e != 1:
        raise ValueError("a row of logits must be contiguous")
    cfg = _route_config(e, top_k, score, num_groups, top_groups, group_best, bool(renormalise), dtype, scale)
    dev = logits.get_device()
    b = None if bias is None else _tensor(bias, "bias", torch.float32, (e,), dev)
    s, leave = _enter(dev, stream)
    try:
        if idx is None:
            idx = torch.empty((t, top_k), dtype=torch.int32, device=dev)
            pi = idx.data_ptr()
        else:
            pi = _tensor(idx, "idx", torch.int32, (t, top_k), dev)
        if w is None:
            w = torch.empty((t, top_k), dtype=torch.float32, device=dev)
            pw = w.data_ptr()
        else:
            pw = _tensor(w, "w", torch.float32, (t, top_k), dev)
        st = _lib.load().moe_decode_route(cfg, logits.data_ptr(), row if t > 1 else e, b, t, pi, pw, s)
    finally:
        if leave is not None:
            leave.close()
    if st:
        _lib.check(st, "moe_decode_route")
    return idx, w


def _quantised(wdtype: str, n: tuple, rows: int, cols: int, halves: int):
    """(dtype, shape) of a matrix's codes, block scales and tensor scale; leading dims n."""
    if wdtype == "bf16":
        return ((torch.bfloat16, (*n, rows, cols)),)
    if wdtype == "fp8":
        return (torch.uint8, (*n, rows, cols)), (torch.float32, (*n, rows // 128, cols // 128))
    return ((torch.uint8, (*n, rows, cols // 2)), (torch.uint8, (*n, rows, cols // 16)),
            (torch.float32, (*n, 2) if halves == 2 else n))


_SUFFIX = {"bf16": ("",), "fp8": ("_q", "_s"), "nvfp4": ("_q", "_s", "_gs")}
_FIELDS = {"": "", "_q": "", "_s": "_scale", "_gs": "_gscale"}


@functools.lru_cache(maxsize=64)
def _expert_tensors(shape: LayerShape) -> tuple:
    """(key in a layer's dict, field of the C struct, type, size) of each weight tensor."""
    h, i = shape.hidden, shape.inter
    return tuple((prefix + name + sfx, prefix + name + _FIELDS[sfx], dtype, size)
                 for prefix, n in (("", shape.num_experts), ("sh_", shape.num_shared)) if n
                 for name, rows, cols, halves in (("w13", 2 * i, h, 2), ("w2", h, i, 1))
                 for sfx, (dtype, size) in zip(_SUFFIX[shape.wdtype],
                                               _quantised(shape.wdtype, (n,), rows, cols, halves)))


def expert_weights(shape: LayerShape, weights: dict, device) -> _lib.Weights:
    """The C struct of a layer's routed and shared expert weights (dict layout of
    synth.make_layer) on ``device`` (an index or a torch device). It keeps the tensors
    alive, and experts() takes it for these weights' sizes and device only."""
    if weights.get("w2_layout", "h_i") != "h_i":
        raise ValueError("down matrices must be stored [E, H, I] (w2_layout h_i)")
    if isinstance(device, int):
        dev = device
    elif device.type == "cpu":
        dev = -1
    else:
        dev = torch.cuda.current_device() if device.index is None else device.index
    out = _lib.Weights()
    out.made_for, out.tensors = (shape, dev), []
    for key, field, dtype, size in _expert_tensors(shape):
        t = weights.get(key)
        if t is None:
            raise ValueError(f"weights lack {key}")
        setattr(out, field, _tensor(t, key, dtype, size, dev))
        out.tensors.append(t)
    return out


def _made_for(weights: _lib.Weights, shape: LayerShape, dev: int) -> _lib.Weights:
    """``weights``, when expert_weights made it for this shape's weights on this device."""
    if not hasattr(weights, "made_for"):
        raise ValueError("weights must be a layer's dict or what expert_weights made of it")
    have, at = weights.made_for
    if at != dev or shape.num_shared > have.num_shared or \
            any(getattr(have, f) != getattr(shape, f) for f in ("hidden", "inter", "num_experts", "wdtype")):
        raise ValueError(f"these weights are of {have} on device {at}, and not of {shape} on device {dev}")
    return weights


def _workspace(workspace: torch.Tensor | None, need: int, dev: int) -> torch.Tensor:
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace.dtype == torch.uint8 and workspace.is_contiguous() and workspace.get_device() == dev and
          workspace.numel() >= need,
          f"the workspace must be a contiguous uint8 tensor of at least {need} bytes on device {dev}")
    return workspace


@functools.lru_cache(maxsize=1024)
def experts_workspace(shape: LayerShape, rows: int) -> int:
    """Bytes of workspace that :func:`experts` needs for at most ``rows`` rows."""
    n = ctypes.c_size_t()
    _lib.check(_lib.load().moe_decode_experts_workspace(_experts_config(shape), rows, n),
               "moe_decode_experts_workspace")
    return n.value


@functools.lru_cache(maxsize=256)
def _experts_config(shape: LayerShape, residual_dtype=torch.bfloat16) -> _lib.ExpertsConfig:
    _need(shape.wdtype in _lib.WDTYPE, f"unknown weight type {shape.wdtype!r}")
    cfg = _lib.ExpertsConfig(shape.hidden, shape.inter, shape.num_experts, shape.top_k, shape.num_shared,
                             _lib.WDTYPE[shape.wdtype], _DTYPES[residual_dtype])
    _lib.check(_lib.load().moe_decode_experts_check(cfg), "moe_decode_experts_check")
    return cfg


def experts(shape: LayerShape, weights, x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor, *,
            residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 [T, H]: residual + the weighted sum of the chosen experts' MLPs of x (and
    the shared experts'), as moe_decode_experts documents. ``weights``: the dict
    layout of synth.make_layer, or what :func:`expert_weights` made of it; ``x`` bf16
    [T, H], any row stride of a multiple of 8; ``idx`` int32 and ``w`` fp32 [T, k];
    an index outside the experts (-1) takes no part. ``residual`` bf16 or fp32 [T, H];
    ``out`` may be a bf16 one."""
    rdtype = torch.bfloat16 if residual is None else residual.dtype
    _need(rdtype in _DTYPES, "the residual is bf16 or fp32")
    cfg = _experts_config(shape, rdtype)
    dev = x.get_device()
    px, t, sx = _rows(x, "x", shape.hidden, dev)
    cw = _made_for(weights, shape, dev) if isinstance(weights, _lib.Weights) else expert_weights(shape, weights, dev)
    pi = _tensor(idx, "idx", torch.int32, (t, shape.top_k), dev)
    pw = _tensor(w, "w", torch.float32, (t, shape.top_k), dev)
    pr = None if residual is None else _tensor(residual, "residual", rdtype, (t, shape.hidden), dev)
    s, leave = _enter(dev, stream)
    try:
        if out is None:
            out = torch.empty((t, shape.hidden), dtype=torch.bfloat16, device=dev)
            po = out.data_ptr()
        else:
            po = _tensor(out, "out", torch.bfloat16, (t, shape.hidden), dev)
        ws = _workspace(workspace, experts_workspace(shape, t), dev)
        st = _lib.load().moe_decode_experts(cfg, cw, px, sx, pi, pw, pr, po, t, ws.data_ptr(), ws.numel(), s)
    finally:
        if leave is not None:
            leave.close()
    if st:
        _lib.check(st, "moe_decode_experts")
    return out


@functools.lru_cache(maxsize=1024)
def _project_config(wdtype: str, inner: int, outer: int, swiglu: bool, rank: int, count: int, out_dtype):
    _need(wdtype in _lib.WDTYPE, f"unknown weight type {wdtype!r}")
    _need(out_dtype in _DTYPES, "the result is bf16 or fp32")
    cfg = _lib.ProjectConfig(inner, outer, swiglu, _lib.WDTYPE[wdtype], rank, count, _DTYPES[out_dtype])
    _lib.check(_lib.load().moe_decode_project_check(cfg), "moe_decode_project_check")
    return cfg


@functools.lru_cache(maxsize=1024)
def _project_bytes(wdtype, inner, outer, swiglu, rank, num_adapters, out_dtype, rows) -> int:
    n = ctypes.c_size_t()
    cfg = _project_config(wdtype, inner, outer, swiglu, rank, num_adapters, out_dtype)
    _lib.check(_lib.load().moe_decode_project_workspace(cfg, rows, n), "moe_decode_project_workspace")
    return n.value


def project_workspace(inner: int, outer: int, rows: int, *, wdtype: str = "bf16", swiglu: bool = False, rank: int = 0,
                      num_adapters: int = 0, out_dtype=torch.bfloat16) -> int:
    """Bytes of workspace that :func:`project` needs for at most ``rows`` rows."""
    return _project_bytes(wdtype, inner, outer, bool(swiglu), rank, num_adapters, out_dtype, rows)


def project(x: torch.Tensor, weight, *, wdtype: str = "bf16", adapters: Adapters | None = None,
            adapter_ids: torch.Tensor | None = None, addend: torch.Tensor | None = None, swiglu: bool = False,
            out: torch.Tensor | None = None, out_dtype=torch.bfloat16, workspace: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """[T, O]: W x + the low-rank product of each row's adapter (+ addend), or with
    ``swiglu`` silu(gate) * up of its two halves, as moe_decode_project documents.
    ``x`` bf16 [T, K], any row stride of a multiple of 8. ``weight``: bf16 [O, K]
    ([2 O, K] with swiglu), or for ``wdtype`` "fp8" / "nvfp4" the tuple (codes, block
    scales) / (codes, block scales, tensor scale [] or [2]). ``adapter_ids`` int32 [T]: the
    adapter of each row, outside 0..L-1 (-1) none."""
    dev = x.get_device()
    parts = weight if isinstance(weight, (tuple, list)) else (weight,)
    if x.dim() != 2:
        raise ValueError("x must be [rows, inner]")
    halves = 2 if swiglu else 1
    t, k = x.shape
    rows = parts[0].shape[0]
    if rows % halves:
        raise ValueError("a gate/up weight has an even number of rows")
    o = rows // halves
    if (adapters is None) != (adapter_ids is None):
        raise ValueError("adapters and adapter_ids come together")
    n = r = 0
    if adapters is not None:
        size = adapters.a.shape
        if len(size) != 3 or not size[0] or not size[1]:
            raise ValueError("adapters.a must be [L, r, K]")
        n, r, _ = size
    if out is not None:
        out_dtype = out.dtype
    cfg = _project_config(wdtype, k, o, bool(swiglu), r, n, out_dtype)
    px, _, sx = _rows(x, "x", k, dev)
    if wdtype == "bf16" and len(parts) == 1:
        pw = (_tensor(parts[0], "weight", torch.bfloat16, (rows, k), dev), None, None)
    else:
        want = _quantised(wdtype, (), rows, k, halves)
        _need(len(parts) == len(want), f"a {wdtype} weight comes in {len(want)} tensors")
        pw = [_tensor(t_, "weight", dtype, size, dev) for t_, (dtype, size) in zip(parts, want)] + [None]
    ids = a = b = scale = None
    if adapters is not None:
        a = _tensor(adapters.a, "adapters.a", torch.bfloat16, (n, r, k), dev)
        b = _tensor(adapters.b, "adapters.b", torch.bfloat16, (n, rows, r), dev)
        if adapters.scale is not None:
            scale = _tensor(adapters.scale, "adapters.scale", torch.float32, (n,), dev)
        ids = _tensor(adapter_ids, "adapter_ids", torch.int32, (t,), dev)
    cw = _lib.ProjectWeights(pw[0], pw[1], pw[2], a, b, scale)
    pa = None if addend is None else _tensor(addend, "addend", torch.bfloat16, (t, o), dev)
    s, leave = _enter(dev, stream)
    try:
        if out is None:
            out = torch.empty((t, o), dtype=out_dtype, device=dev)
            po = out.data_ptr()
        else:
            po = _tensor(out, "out", out_dtype, (t, o), dev)
        ws = _workspace(workspace, _project_bytes(wdtype, k, o, bool(swiglu), r, n, out_dtype, t), dev)
        st = _lib.load().moe_decode_project(cfg, cw, px, sx, ids, pa, po, t, ws.data_ptr(), ws.numel(), s)
    finally:
        if leave is not None:
            leave.close()
    if st:
        _lib.check(st, "moe_decode_project")
    return out


def status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise and return the status code of the last call of one row or more that
    used ``workspace`` (from its first byte on)."""
    _workspace(workspace, _lib.ROWS_STATUS_BYTES, workspace.get_device())
    s, leave = _enter(workspace.get_device(), stream)
    try:
        return _lib.load().moe_decode_rows_status(workspace.data_ptr(), s)
    finally:
        if leave is not None:
            leave.close()
