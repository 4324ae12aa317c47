"""The operators for any number of rows, over torch tensors: the MoE layer's, and a dense layer's.

``route``, ``experts`` and ``project`` marshal tensors into the C entry points of
include/moe_decode_rows.h, and ``quantise``, ``project_int8``, ``feed_forward`` and
``feed_forward_backward`` into those of include/moe_decode_dense.h, which document what is
computed. They check shapes,
types and devices, allocate results (and a workspace, unless one is given) with
torch's allocator on the stream they run on, and enqueue their work on the current
stream (or ``stream``) without waiting. No arithmetic happens here, and no autograd graph
is recorded: results require no gradient, whatever their inputs do.

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


# (torch.empty with a device's index takes 2 us more than with this, among launches)
_DEVICES = [torch.device("cuda", i) for i in range(64)]


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
            idx = torch.empty((t, top_k), dtype=torch.int32, device=_DEVICES[dev])
            pi = idx.data_ptr()
        else:
            pi = _tensor(idx, "idx", torch.int32, (t, top_k), dev)
        if w is None:
            w = torch.empty((t, top_k), dtype=torch.float32, device=_DEVICES[dev])
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
        return torch.empty(need, dtype=torch.uint8, device=_DEVICES[dev])
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
            out = torch.empty((t, shape.hidden), dtype=torch.bfloat16, device=_DEVICES[dev])
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
            out = torch.empty((t, o), dtype=out_dtype, device=_DEVICES[dev])
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


def _row_major(t: torch.Tensor, name: str, dtypes, cols: int | None, dev: int) -> tuple[int, int, int]:
    """(address, rows, row stride) of a [rows, cols] tensor of one of these types whose rows are contiguous."""
    shape, stride = t.shape, t.stride()
    if t.dtype not in dtypes or t.get_device() != dev or len(shape) != 2 or (cols is not None and shape[1] != cols) or \
            (shape[0] and shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"{name} must be a [rows, {'columns' if cols is None else cols}] tensor of {dtypes} on device "
                         f"{dev} with contiguous rows: got {t.dtype} {tuple(shape)} on {t.device}")
    return t.data_ptr(), shape[0], stride[0] if shape[0] > 1 else shape[1]


_ROWS_DTYPES = (torch.bfloat16, torch.float32)


def quantise(x: torch.Tensor, *, codes: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None):
    """(int8 [T, K], fp32 [T]): the rows of ``x`` (bf16 or fp32 [T, K], any row stride of a multiple of 16
    bytes) as 8-bit integers with a scale each, as moe_decode_quantise documents. K % 8 == 0."""
    dev = x.get_device()
    px, t, sx = _row_major(x, "x", _ROWS_DTYPES, None, dev)
    k = x.shape[1]
    s, leave = _enter(dev, stream)
    try:
        if codes is None:
            codes = torch.empty((t, k), dtype=torch.int8, device=_DEVICES[dev])
            pc = codes.data_ptr()
        else:
            pc = _tensor(codes, "codes", torch.int8, (t, k), dev)
        if scale is None:
            scale = torch.empty((t,), dtype=torch.float32, device=_DEVICES[dev])
            ps = scale.data_ptr()
        else:
            ps = _tensor(scale, "scale", torch.float32, (t,), dev)
        st = _lib.load().moe_decode_quantise(_DTYPES[x.dtype], k, px, sx, t, pc, ps, s)
    finally:
        if leave is not None:
            leave.close()
    if st:
        _lib.check(st, "moe_decode_quantise")
    return codes, scale


@functools.lru_cache(maxsize=1024)
def _int8_config(inner: int, outer: int, swiglu: bool, x_dtype, out_dtype) -> _lib.Int8Config:
    _need(out_dtype in _DTYPES, "the result is bf16 or fp32")
    cfg = _lib.Int8Config(inner, outer, swiglu, _lib.MOE_I8 if x_dtype is torch.int8 else _DTYPES[x_dtype],
                          _DTYPES[out_dtype])
    _lib.check(_lib.load().moe_decode_project_int8_check(cfg), "moe_decode_project_int8_check")
    return cfg


@functools.lru_cache(maxsize=1024)
def _int8_bytes(inner, outer, swiglu, x_dtype, out_dtype, rows) -> int:
    n = ctypes.c_size_t()
    cfg = _int8_config(inner, outer, swiglu, x_dtype, out_dtype)
    _lib.check(_lib.load().moe_decode_project_int8_workspace(cfg, rows, n), "moe_decode_project_int8_workspace")
    return n.value


def project_int8_workspace(inner: int, outer: int, rows: int, *, swiglu: bool = False, x_dtype=torch.int8,
                           out_dtype=torch.bfloat16) -> int:
    """Bytes of workspace that :func:`project_int8` needs for at most ``rows`` rows; ``x_dtype``
    torch.int8: x comes as codes."""
    return _int8_bytes(inner, outer, bool(swiglu), x_dtype, out_dtype, rows)


def _codes(weight, name: str, rows: int, cols: int, dev: int) -> tuple[int, int]:
    """The addresses of an int8 matrix and of its rows' scales."""
    _need(isinstance(weight, (tuple, list)) and len(weight) == 2, f"{name} comes as (codes, scale)")
    return (_tensor(weight[0], name, torch.int8, (rows, cols), dev),
            _tensor(weight[1], f"{name}'s scale", torch.float32, (rows,), dev))


def project_int8(x, weight, *, addend: torch.Tensor | None = None, swiglu: bool = False,
                 out: torch.Tensor | None = None, out_dtype=torch.bfloat16, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """[T, O]: the product of 8-bit integers s_t c_o sum_k q_tk W_ok (+ addend), or with ``swiglu``
    silu(gate) * up of its two halves, as moe_decode_project_int8 documents. ``x``: (codes, scale) of
    :func:`quantise`, or bf16 or fp32 [T, K], which the call quantises; ``weight``: (int8 [O, K], fp32
    [O]), [2 O] rows with swiglu. K % 16 == 0, O % 8 == 0."""
    given = isinstance(x, (tuple, list))
    if given:
        _need(len(x) == 2, "quantised rows come as (codes, scale)")
    rows_t, scale = x if given else (x, None)
    _need(isinstance(weight, (tuple, list)) and len(weight) == 2, "an int8 weight comes as (codes, scale)")
    halves = 2 if swiglu else 1
    if rows_t.dim() != 2 or weight[0].dim() != 2 or weight[0].shape[0] % halves:
        raise ValueError("x must be [rows, inner] and the weight [outer, inner], with an even number of rows for gate/up")
    dev = rows_t.get_device()
    t, k = rows_t.shape
    rows = weight[0].shape[0]
    o = rows // halves
    px, _, sx = _row_major(rows_t, "x", (torch.int8,) if given else _ROWS_DTYPES, k, dev)
    if out is not None:
        out_dtype = out.dtype
    cfg = _int8_config(k, o, bool(swiglu), rows_t.dtype, out_dtype)
    ps = _tensor(scale, "x's scale", torch.float32, (t,), dev) if given else None
    pw, pc = _codes(weight, "weight", rows, k, dev)
    pa = None if addend is None else _tensor(addend, "addend", torch.bfloat16, (t, o), dev)
    s, leave = _enter(dev, stream)
    try:
        if out is None:
            out = torch.empty((t, o), dtype=out_dtype, device=_DEVICES[dev])
            po = out.data_ptr()
        else:
            po = _tensor(out, "out", out_dtype, (t, o), dev)
        pws = nws = None
        need = _int8_bytes(k, o, bool(swiglu), rows_t.dtype, out_dtype, t)
        if need or workspace is not None:
            ws = _workspace(workspace, need, dev)
            pws, nws = ws.data_ptr(), ws.numel()
        st = _lib.load().moe_decode_project_int8(cfg, pw, pc, px, ps, sx, pa, po, t, pws, nws or 0, s)
    finally:
        if leave is not None:
            leave.close()
    if st:
        _lib.check(st, "moe_decode_project_int8")
    return out


_FF_WDTYPE = {"bf16": _lib.MOE_W_BF16, "int8": _lib.MOE_W_INT8}


@functools.lru_cache(maxsize=256)
def _ff_config(hidden: int, inter: int, wdtype: str) -> _lib.FfConfig:
    _need(wdtype in _FF_WDTYPE, f"a feed-forward block's weights are bf16 or int8, not {wdtype!r}")
    cfg = _lib.FfConfig(hidden, inter, _FF_WDTYPE[wdtype])
    _lib.check(_lib.load().moe_decode_ff_check(cfg), "moe_decode_ff_check")
    return cfg


@functools.lru_cache(maxsize=1024)
def feed_forward_workspace(hidden: int, inter: int, rows: int, *, wdtype: str = "bf16") -> int:
    """Bytes of workspace that :func:`feed_forward` needs for at most ``rows`` rows."""
    n = ctypes.c_size_t()
    _lib.check(_lib.load().moe_decode_ff_workspace(_ff_config(hidden, inter, wdtype), rows, n), "moe_decode_ff_workspace")
    return n.value


@functools.lru_cache(maxsize=1024)
def feed_forward_backward_workspace(hidden: int, inter: int, rows: int) -> int:
    """Bytes of workspace that :func:`feed_forward_backward` needs for at most ``rows`` rows."""
    n = ctypes.c_size_t()
    _lib.check(_lib.load().moe_decode_ff_backward_workspace(_ff_config(hidden, inter, "bf16"), rows, n),
               "moe_decode_ff_backward_workspace")
    return n.value


def _ff_sizes(w13, w2) -> tuple[int, int]:
    """(hidden, inter) of the block with these weights."""
    if w13.dim() != 2 or w2.dim() != 2 or w13.shape[0] != 2 * w2.shape[1] or w13.shape[1] != w2.shape[0]:
        raise ValueError(f"weights must be [2 inter, hidden] and [hidden, inter]: got {tuple(w13.shape)}, {tuple(w2.shape)}")
    return w2.shape[0], w2.shape[1]


def feed_forward(x: torch.Tensor, w13, w2, *, wdtype: str = "bf16", residual: torch.Tensor | None = None,
                 gate_up: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 [T, H]: the gated feed-forward block W2 (silu(Wg x) * (Wu x)) (+ residual), as moe_decode_ff
    documents. ``x`` bf16 [T, H], any row stride of a multiple of 8; ``w13`` = [Wg; Wu] bf16 [2 I, H] and ``w2``
    bf16 [H, I], or for ``wdtype`` "int8" (codes, scale) of each, a scale a row. ``gate_up``: a bf16
    [T, 2 I] tensor that receives the sums which :func:`feed_forward_backward` needs (bf16 weights).
    ``out`` may be the residual, and x. Autograd does not see the call: its gradients are
    :func:`feed_forward_backward`'s."""
    int8 = wdtype == "int8"
    if int8:
        _need(all(isinstance(w, (tuple, list)) and len(w) == 2 for w in (w13, w2)), "int8 weights come as (codes, scale)")
    hidden, inter = _ff_sizes(w13[0], w2[0]) if int8 else _ff_sizes(w13, w2)
    cfg = _ff_config(hidden, inter, wdtype)
    dev = x.get_device()
    px, t, sx = _rows(x, "x", hidden, dev)
    if int8:
        (p13, s13), (p2, s2) = _codes(w13, "w13", 2 * inter, hidden, dev), _codes(w2, "w2", hidden, inter, dev)
    else:
        p13 = _tensor(w13, "w13", torch.bfloat16, (2 * inter, hidden), dev)
        p2, s13, s2 = _tensor(w2, "w2", torch.bfloat16, (hidden, inter), dev), None, None
    cw = _lib.FfWeights(p13, p2, s13, s2)
    pr = None if residual is None else _tensor(residual, "residual", torch.bfloat16, (t, hidden), dev)
    pk = None if gate_up is None else _tensor(gate_up, "gate_up", torch.bfloat16, (t, 2 * inter), dev)
    s, leave = _enter(dev, stream)
    try:
        if out is None:
            out = torch.empty((t, hidden), dtype=torch.bfloat16, device=_DEVICES[dev])
            po = out.data_ptr()
        else:
            po = _tensor(out, "out", torch.bfloat16, (t, hidden), dev)
        ws = _workspace(workspace, feed_forward_workspace(hidden, inter, t, wdtype=wdtype), dev)
        st = _lib.load().moe_decode_ff(cfg, cw, px, sx, pr, pk, po, t, ws.data_ptr(), ws.numel(), s)
    finally:
        if leave is not None:
            leave.close()
    if st:
        _lib.check(st, "moe_decode_ff")
    return out


def feed_forward_backward(grad: torch.Tensor, x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                          gate_up: torch.Tensor, *, dx: torch.Tensor | None = None, dw13: torch.Tensor | None = None,
                          dw2: torch.Tensor | None = None, accumulate: bool = False, input_grad: bool = True,
                          weight_grad: bool = True, workspace: torch.Tensor | None = None, stream=None):
    """(dx, dw13, dw2): the gradients of :func:`feed_forward` (bf16 weights) from ``grad``, that of its result,
    and ``gate_up``, which it kept; as moe_decode_ff_backward documents. ``grad`` and ``x`` bf16 [T, H], any row
    stride of a multiple of 8. The residual's gradient is ``grad``. The gradients are bf16; ``dw13`` and
    ``dw2`` may be given as fp32, and with ``accumulate`` are then added to. Without ``input_grad``
    or ``weight_grad`` what is not wanted is None."""
    hidden, inter = _ff_sizes(w13, w2)
    cfg = _ff_config(hidden, inter, "bf16")
    dev = x.get_device()
    px, t, sx = _rows(x, "x", hidden, dev)
    pg, tg, sg = _rows(grad, "grad", hidden, dev)
    _need(t == tg, "grad and x have the same rows")
    _need(input_grad or weight_grad, "no gradient is wanted")
    cw = _lib.FfWeights(_tensor(w13, "w13", torch.bfloat16, (2 * inter, hidden), dev),
                        _tensor(w2, "w2", torch.bfloat16, (hidden, inter), dev), None, None)
    pk = _tensor(gate_up, "gate_up", torch.bfloat16, (t, 2 * inter), dev)
    _need((input_grad or dx is None) and (weight_grad or (dw13 is None and dw2 is None)),
          "a gradient that is not wanted has no place")
    given = [d for d in (dw13, dw2) if d is not None]
    dtype = given[0].dtype if given else torch.bfloat16
    _need(dtype in _DTYPES, "weight gradients are bf16 or fp32")
    _need(not accumulate or (len(given) == 2 and dtype is torch.float32), "accumulate adds to fp32 dw13 and dw2 that are given")
    px_, p13, p2 = None, None, None
    s, leave = _enter(dev, stream)
    try:
        if input_grad:
            dx = torch.empty((t, hidden), dtype=torch.bfloat16, device=_DEVICES[dev]) if dx is None else dx
            px_ = _tensor(dx, "dx", torch.bfloat16, (t, hidden), dev)
        if weight_grad:
            dw13 = torch.empty((2 * inter, hidden), dtype=dtype, device=_DEVICES[dev]) if dw13 is None else dw13
            dw2 = torch.empty((hidden, inter), dtype=dtype, device=_DEVICES[dev]) if dw2 is None else dw2
            p13 = _tensor(dw13, "dw13", dtype, (2 * inter, hidden), dev)
            p2 = _tensor(dw2, "dw2", dtype, (hidden, inter), dev)
        ws = _workspace(workspace, feed_forward_backward_workspace(hidden, inter, t), dev)
        st = _lib.load().moe_decode_ff_backward(cfg, cw, pg, sg, px, sx, pk, px_, p13, p2, _DTYPES[dtype], accumulate, t,
                                                ws.data_ptr(), ws.numel(), s)
    finally:
        if leave is not None:
            leave.close()
    if st:
        _lib.check(st, "moe_decode_ff_backward")
    return dx, dw13, dw2


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
