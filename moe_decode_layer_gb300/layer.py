"""Python handle over the C ABI: marshals torch tensors into pointers and calls
moe_decode_create / moe_decode_run. No arithmetic happens here.
"""

from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _lib, batch
from .synth import LayerShape


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


class MoEDecodeLayer:
    """One MoE layer's decode step on the current CUDA device.

    ``weights`` is the dict layout of :func:`synth.make_layer` (device tensors);
    ``score`` 1 selects the bias-corrected sigmoid rule, whose fp32 [E] bias is
    ``weights["router_bias"]``.
    The tensors are borrowed: this object keeps references so they outlive the
    C handle. ``sched``: "persistent" (one kernel; the expert-range or
    slot-interleaved kernel where that measured faster), "phased" (one kernel,
    phases in order), "interleaved" (one kernel, slot-interleaved whenever its
    layout fits), "flat" (the expert-range kernel whenever its layout fits),
    "pdl_chain" or "chain" (three kernels). Weights whose ``w2_layout`` is "i_h"
    (down matrices transposed) run the split-K kernel, under "persistent" only.
    """

    def __init__(self, shape: LayerShape, weights: dict, max_rows: int, sched: str = "persistent",
                 pre_rmsnorm: bool = False, rms_eps: float = 1e-6, routed_scale: float = 1.0,
                 score: int = 0):
        self.lib = _lib.load()
        self.shape = shape
        self.max_rows = max_rows
        self._weights = weights
        cfg = _lib.Config(hidden=shape.hidden, inter=shape.inter, num_experts=shape.num_experts,
                          top_k=shape.top_k, num_shared=shape.num_shared, max_rows=max_rows,
                          wdtype=_lib.WDTYPE[shape.wdtype],
                          score=score, routed_scale=routed_scale,
                          pre_rmsnorm=int(pre_rmsnorm), rms_eps=rms_eps,
                          sched=_lib.SCHED_NAMES["persistent" if sched in ("phased", "interleaved", "flat")
                                                  else sched],
                          w2_layout=_lib.W2_LAYOUT[weights.get("w2_layout", "h_i")])
        w = _lib.Weights()
        g = weights.get
        w.router_w = _ptr(g("router_w"))
        w.router_bias = _ptr(g("router_bias"))
        if shape.wdtype == "bf16":
            w.w13, w.w2 = _ptr(g("w13")), _ptr(g("w2"))
            if shape.num_shared:
                w.sh_w13, w.sh_w2 = _ptr(g("sh_w13")), _ptr(g("sh_w2"))
        elif shape.wdtype == "fp8":
            w.w13, w.w13_scale = _ptr(g("w13_q")), _ptr(g("w13_s"))
            w.w2, w.w2_scale = _ptr(g("w2_q")), _ptr(g("w2_s"))
            if shape.num_shared:
                w.sh_w13, w.sh_w13_scale = _ptr(g("sh_w13_q")), _ptr(g("sh_w13_s"))
                w.sh_w2, w.sh_w2_scale = _ptr(g("sh_w2_q")), _ptr(g("sh_w2_s"))
        else:
            w.w13, w.w13_scale, w.w13_gscale = _ptr(g("w13_q")), _ptr(g("w13_s")), _ptr(g("w13_gs"))
            w.w2, w.w2_scale, w.w2_gscale = _ptr(g("w2_q")), _ptr(g("w2_s")), _ptr(g("w2_gs"))
            if shape.num_shared:
                w.sh_w13, w.sh_w13_scale, w.sh_w13_gscale = (_ptr(g("sh_w13_q")), _ptr(g("sh_w13_s")),
                                                             _ptr(g("sh_w13_gs")))
                w.sh_w2, w.sh_w2_scale, w.sh_w2_gscale = (_ptr(g("sh_w2_q")), _ptr(g("sh_w2_s")),
                                                          _ptr(g("sh_w2_gs")))
        self._cfg = cfg
        h = ctypes.c_void_p()
        _lib.check(self.lib.moe_decode_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)),
                   "moe_decode_create")
        self.handle = h
        if sched in ("phased", "interleaved"):  # the single kernel in phase order / always interleaved
            self.set_option(_lib.MOE_OPT_FLAT, 0)
            self.set_option(_lib.MOE_OPT_INTERLEAVE, 0 if sched == "phased" else 2)
        elif sched == "flat":  # the expert-range kernel whenever it fits
            self.set_option(_lib.MOE_OPT_FLAT, 2)

    # ------------------------------------------------------------------ runs
    def run(self, x: torch.Tensor, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
            topk_idx: torch.Tensor | None = None, topk_w: torch.Tensor | None = None, stream=None):
        """Enqueue one step; returns ``out`` (allocated when not given)."""
        residual = x if residual is None else residual
        if out is None:
            out = torch.empty_like(x)
        for t in (x, residual, out):
            if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("x, residual and out must be contiguous bf16 CUDA tensors")
        m = x.shape[0]
        _lib.check(self.lib.moe_decode_run(self.handle, _ptr(x), _ptr(residual), _ptr(out), m,
                                           _ptr(topk_idx), _ptr(topk_w), _stream_ptr(stream)),
                   "moe_decode_run")
        return out

    def run_host(self, x: torch.Tensor, residual: torch.Tensor, out: torch.Tensor,
                 topk_idx: torch.Tensor | None = None, topk_w: torch.Tensor | None = None, stream=None):
        """One step from host (CPU) tensors, copies included; synchronises."""
        for t in (x, residual, out):
            if t.dtype != torch.bfloat16 or t.is_cuda or not t.is_contiguous():
                raise ValueError("run_host takes contiguous bf16 CPU tensors")
        _lib.check(self.lib.moe_decode_run_host(self.handle, _ptr(x), _ptr(residual), _ptr(out), x.shape[0],
                                                _ptr(topk_idx), _ptr(topk_w), _stream_ptr(stream)),
                   "moe_decode_run_host")
        return out

    def run_rows(self, x: torch.Tensor, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 topk_idx: torch.Tensor | None = None, topk_w: torch.Tensor | None = None, *,
                 num_groups: int = 1, top_groups: int = 1, group_best: int = 1,
                 adapters: tuple[batch.Adapters, batch.Adapters] | None = None,
                 adapter_ids: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
        """The same layer for any number of rows (a chunk of a prompt, many requests):
        router logits, batch.route and batch.experts one after another, with this
        layer's weights, scoring rule and routed scale. Nothing of the handle is
        used, so runs on different streams may overlap. ``x`` may have any row stride of
        a multiple of 8; ``residual`` (x, when not given) is contiguous. ``num_groups``,
        ``top_groups`` and ``group_best`` limit the choice to the best groups of
        experts. ``adapters``: the low-rank adapters of the one shared expert's
        gate/up and down projections, and ``adapter_ids`` int32 [T] each row's. All terms
        and the residual are summed in fp32 and rounded once. ``out`` may be x. Not for
        layers with pre_rmsnorm or transposed down matrices.

        ``workspace``: uint8, of rows_workspace bytes; after a run with one rows_status
        tells whether its device-side waits ended in time (without one, each operator
        takes a workspace from torch's allocator, and nobody can be asked)."""
        if self._cfg.pre_rmsnorm:
            raise ValueError("run_rows takes the layer's normalised input: pre_rmsnorm is not computed")
        if adapters is not None and self.shape.num_shared != 1:
            raise ValueError("adapters belong to the one shared expert of a layer")
        if (adapters is None) != (adapter_ids is None):
            raise ValueError("adapters and adapter_ids come together")
        if self._cfg.w2_layout != _lib.W2_LAYOUT["h_i"]:
            raise ValueError("run_rows takes down matrices stored [E, H, I] (w2_layout h_i)")
        if residual is None:
            residual = x if x.is_contiguous() else batch.contiguous(x, stream)
        ws = dict.fromkeys(("router", "up", "down", "experts"))
        if workspace is not None:
            parts, need = self._rows_parts(x.shape[0], adapters)
            batch._workspace(workspace, need, x.get_device())
            ws.update({name: workspace[at:at + n] for name, (at, n) in parts.items()})
        sig = self._cfg.score == _lib.MOE_SCORE_SIGMOID_BIAS
        logits = batch.project(x, self._weights["router_w"], out_dtype=torch.float32, workspace=ws["router"],
                               stream=stream)
        idx, w = batch.route(logits, self.shape.top_k, score="sigmoid" if sig else "softmax",
                             bias=self._weights["router_bias"] if sig else None, num_groups=num_groups,
                             top_groups=top_groups, group_best=group_best, scale=self._cfg.routed_scale,
                             idx=topk_idx, w=topk_w, stream=stream)
        shape = self.shape
        if adapters is not None:
            sfx = batch._SUFFIX[shape.wdtype]
            w13, w2 = (tuple(self._weights["sh_" + n + f][0] for f in sfx) for n in ("w13", "w2"))
            h = batch.project(x, w13, wdtype=shape.wdtype, swiglu=True, adapters=adapters[0], adapter_ids=adapter_ids,
                              workspace=ws["up"], stream=stream)
            residual = batch.project(h, w2, wdtype=shape.wdtype, adapters=adapters[1], adapter_ids=adapter_ids,
                                     addend=residual, out_dtype=torch.float32, workspace=ws["down"], stream=stream)
            shape = dataclasses.replace(shape, num_shared=0)
        return batch.experts(shape, self._weights, x, idx, w, residual=residual, out=out,
                             workspace=ws["experts"], stream=stream)

    def _rows_parts(self, rows: int, adapters):
        """({operator: (offset, bytes)}, bytes in all) of a workspace of run_rows."""
        s = self.shape
        need = {"router": batch.project_workspace(s.hidden, s.num_experts, rows, out_dtype=torch.float32)}
        if adapters is not None:
            for name, ad, inner, outer, swiglu in (("up", adapters[0], s.hidden, s.inter, True),
                                                   ("down", adapters[1], s.inter, s.hidden, False)):
                need[name] = batch.project_workspace(inner, outer, rows, wdtype=s.wdtype, swiglu=swiglu,
                                                     rank=ad.a.shape[1], num_adapters=ad.a.shape[0],
                                                     out_dtype=torch.bfloat16 if swiglu else torch.float32)
            s = dataclasses.replace(s, num_shared=0)
        need["experts"] = batch.experts_workspace(s, rows)
        parts, at = {}, 0
        for name, n in need.items():
            parts[name] = at, n
            at += (n + 255) // 256 * 256
        return parts, at

    def rows_workspace(self, rows: int, adapters: tuple[batch.Adapters, batch.Adapters] | None = None) -> int:
        """Bytes of a workspace for run_rows with this many rows and these adapters."""
        return self._rows_parts(rows, adapters)[1]

    def rows_status(self, workspace: torch.Tensor, rows: int,
                    adapters: tuple[batch.Adapters, batch.Adapters] | None = None, stream=None) -> int:
        """Synchronise and return the status code of the last run_rows of this many rows
        with these adapters and this workspace: MOE_ERR_DEVICE_TIMEOUT when a device-side
        wait of any of its operators ran into its limit (the outputs are undefined then)."""
        parts, need = self._rows_parts(rows, adapters)
        batch._workspace(workspace, need, workspace.get_device())
        codes = [batch.status(workspace[at:at + n], stream) for at, n in parts.values() if n]
        return next((c for c in codes if c != _lib.MOE_OK), _lib.MOE_OK)

    def host_copy_bytes(self, m: int) -> tuple[int, int]:
        """Bytes run_host copies per call with m rows and x as the residual: (in, out).
        Out is one block from the status words to the m-th output row: the rest of the
        CTRL_WORDS control words, topk_idx and topk_w for max_rows rows (each padded
        to 16 bytes), then the output rows."""
        pad16 = lambda v: (v + 15) // 16 * 16  # noqa: E731
        k = self.shape.top_k
        out = _lib.CTRL_WORDS * 4 - 8 + 2 * pad16(self.max_rows * k * 4) + m * self.shape.hidden * 2
        return m * self.shape.hidden * 2, out

    def status(self, stream=None) -> int:
        """Synchronise and return (and clear) the device status code of run's steps
        (run_rows keeps nothing in the handle: rows_status)."""
        return self.lib.moe_decode_get_status(self.handle, _stream_ptr(stream))

    def set_option(self, option: int, value: int) -> None:
        _lib.check(self.lib.moe_decode_set_option(self.handle, option, value), "moe_decode_set_option")

    def info(self, what: int) -> int:
        v = ctypes.c_int64()
        _lib.check(self.lib.moe_decode_get_info(self.handle, what, ctypes.byref(v)), "moe_decode_get_info")
        return v.value

    def close(self) -> None:
        if getattr(self, "handle", None):
            self.lib.moe_decode_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
