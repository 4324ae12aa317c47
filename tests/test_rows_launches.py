"""What the many-row entry points put on a stream, over a stand-in for the CUDA runtime (no GPU)."""

import ctypes
import os
import random
import re

import pytest
import torch

from moe_decode_layer_gb300 import _lib, batch, build
from tests import fake_cuda

OK, CUDA, BAD = _lib.MOE_OK, _lib.MOE_ERR_CUDA, _lib.MOE_ERR_INVALID_ARG
P = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return fake_cuda.make(str(tmp_path_factory.mktemp("fake")))


def _weights(cls):
    w = cls()
    for name, _ in cls._fields_:
        setattr(w, name, P)
    return w


# places far enough apart for the largest call here
X, OUT, RES, WS = (ctypes.c_void_p(i << 40) for i in (1, 2, 3, 4))


def _experts(lib, rows, fail_encode=-1, fail_launch=-1, pending=0, stride=256, x=X, out=OUT, residual=RES, idx=P, w=P,
             weights=(), **kw):
    cfg = _lib.ExpertsConfig(**{**dict(hidden=256, inter=128, num_experts=16, top_k=2, num_shared=1, wdtype=0), **kw})
    need = ctypes.c_size_t()
    assert lib.moe_decode_experts_workspace(cfg, rows, need) == OK
    lib.fake_reset(fail_encode, fail_launch, pending)
    wt = _weights(_lib.Weights)
    for name, v in dict(weights).items():
        setattr(wt, name, v)
    return lib.moe_decode_experts(cfg, wt, x, stride, idx, w, residual, out, rows, WS, need, None)


def _project(lib, rows, fail_encode=-1, fail_launch=-1, pending=0, stride=256, x=X, out=OUT, addend=None, ids=P,
             weights=(), **kw):
    cfg = _lib.ProjectConfig(**{**dict(inner=256, outer=256, swiglu=0, wdtype=0, rank=16, num_adapters=4, out_dtype=0), **kw})
    need = ctypes.c_size_t()
    assert lib.moe_decode_project_workspace(cfg, rows, need) == OK
    lib.fake_reset(fail_encode, fail_launch, pending)
    wt = _weights(_lib.ProjectWeights)
    for name, v in dict(weights).items():
        setattr(wt, name, v)
    return lib.moe_decode_project(cfg, wt, x, stride, ids, addend, out, rows, WS, need, None)


def _names(lib):
    return [next(n for n in ("plan", "spread", "gemm", "combine", "shrink", "route") if n + "_kernel" in lib.fake_name(i).decode())
            for i in range(lib.fake_launches())]


@pytest.mark.parametrize("rows", [1, 16384 + 5, 2 * 16384])
@pytest.mark.parametrize("wdtype", [0, 2])
def test_experts_without_descriptors_enqueue_nothing(lib, rows, wdtype):
    """Whichever descriptor cannot be made, of the first round's or a later one's, nothing was launched."""
    assert _experts(lib, rows, wdtype=wdtype) == OK
    encodes, launches = lib.fake_encodes(), lib.fake_launches()
    assert launches >= 4
    for n in range(encodes):
        assert _experts(lib, rows, fail_encode=n, wdtype=wdtype) == CUDA
        assert lib.fake_launches() == 0, n


@pytest.mark.parametrize("rows", [8, 100, 5003])
def test_project_without_descriptors_enqueues_nothing(lib, rows):
    assert _project(lib, rows) == OK
    for n in range(lib.fake_encodes()):
        assert _project(lib, rows, fail_encode=n) == CUDA
        assert lib.fake_launches() == 0, n


def test_failed_launches_are_reported(lib):
    """A launch that fails ends the call with its error; the ones after it are left out."""
    for call, rows in ((_experts, 16384 + 5), (_project, 8), (_project, 5003)):
        assert call(lib, rows) == OK
        names = _names(lib)
        for n in range(len(names)):
            assert call(lib, rows, fail_launch=n) == CUDA
            assert _names(lib) == names[:n] and lib.fake_pending() == 0


def test_lists_of_the_launch_before_are_read_plainly():
    """With early launches the read-only path would be used on memory that changes while the grid is resident."""
    gemm, small = (open(os.path.join(build.CSRC, f)).read() for f in ("rows_gemm.cuh", "rows_kernels.cu"))
    for name in ("ents", "nent", "adapter_off", "src_row", "out_row", "u32"):
        assert f"p.{name}" in gemm and not re.search(rf"__ldg\(\s*p\.{name}\b", gemm), name
    combine = small[small.index("combine_kernel(const float*"):small.index("cudaError_t launch_plan")]
    assert not re.search(r"__ldg\([^;]*\b(y|pos)\b", combine) and not re.search(r"__restrict__ (y|pos)\b", combine)
    spread = small[small.index("spread_kernel(const"):small.index("constexpr int kShrinkWarps")]
    assert not re.search(r"__restrict__ (src_row|count)\b", spread) and not re.search(r"__ldg\((src_row|count)", spread)


def test_rounds(lib):
    """A call of many rows goes through its rounds in order."""
    assert _experts(lib, 3 * 16384 + 1) == OK
    full, short = ["plan", "spread", "gemm", "gemm", "combine"], ["plan", "gemm", "gemm", "combine"]
    assert _names(lib) == 3 * full + short


def test_an_earlier_error_is_not_this_call_s(lib):
    """An error that some call before left behind does not make a call fail whose launches went well."""
    cfg = _lib.RouteConfig(64, 4, 0, 1, 1, 1, 1, 1, 1.0)
    for bias in (None, P):
        lib.fake_reset(-1, -1, 1)
        assert lib.moe_decode_route(cfg, P, 64, bias, 100, P, P, None) == OK and _names(lib) == ["route"]
        lib.fake_reset(-1, 0, 0)
        assert lib.moe_decode_route(cfg, P, 64, bias, 100, P, P, None) == CUDA and lib.fake_launches() == 0
    for call, rows in ((_experts, 100), (_project, 8), (_project, 5003)):
        assert call(lib, rows, pending=1) == OK


def test_status_reads_what_the_binding_checks(lib):
    """The bytes that the status call copies are those that the binding asks a workspace for."""
    assert lib.moe_decode_rows_status(P, None) == OK
    assert lib.fake_bytes_read() == _lib.ROWS_STATUS_BYTES
    for rows in (1, 100):
        need = ctypes.c_size_t()
        assert lib.moe_decode_project_workspace(_lib.ProjectConfig(8, 8, 0, 0, 0, 0, 0), rows, need) == OK
        assert need.value >= _lib.ROWS_STATUS_BYTES


def test_status_of_a_stream_under_capture_is_refused(lib):
    """Nothing of it gets into the graph."""
    lib.fake_capture(1)
    assert lib.moe_decode_rows_status(P, None) == BAD and lib.fake_bytes_read() == 0
    lib.fake_capture(0)
    assert lib.moe_decode_rows_status(P, None) == OK


def test_status_of_a_short_workspace_is_refused():
    for bad in (torch.empty(_lib.ROWS_STATUS_BYTES - 1, dtype=torch.uint8), torch.empty(4096), torch.empty(0, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace must be"):
            batch.status(bad)


def test_residual_types(lib):
    """fp32 and bf16 residuals; the result may be in a bf16 one's place only."""
    check = lib.moe_decode_experts_check
    base = dict(hidden=256, inter=128, num_experts=16, top_k=2, num_shared=1, wdtype=0)
    assert [check(_lib.ExpertsConfig(**base, residual_dtype=d)) for d in (0, 1, 2)] == [OK, OK, _lib.MOE_ERR_UNSUPPORTED]
    assert _experts(lib, 8, residual=OUT) == OK
    assert _experts(lib, 8, residual=RES, residual_dtype=1) == OK
    assert _experts(lib, 8, residual=OUT, residual_dtype=1) == BAD


def _at(v):
    return ctypes.c_void_p(v)


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=_at(4104)), dict(stride=248), dict(stride=260), dict(idx=None), dict(idx=_at(4098)),
                                dict(w=None), dict(w=_at(4098)), dict(out=None), dict(out=_at(4104)), dict(residual=_at(4104))] +
                         [dict(weights={n: v}) for n in ("w13", "w2", "sh_w13", "sh_w2", "w13_scale", "w2_scale", "sh_w13_scale",
                                                         "sh_w2_scale") for v in (None, _at(4104))] +
                         [dict(weights={n: v}) for n in ("w13_gscale", "w2_gscale", "sh_w13_gscale", "sh_w2_gscale")
                          for v in (None, _at(4098))], ids=str)
def test_experts_refuse_one_bad_address(lib, kw):
    """Each argument alone, beside others that are taken."""
    shape = dict(hidden=256, inter=256, wdtype=1)
    assert _experts(lib, 4, **shape) == OK
    assert _experts(lib, 4, **{**shape, **kw}) == BAD and lib.fake_launches() == 0


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=_at(4104)), dict(stride=248), dict(stride=260), dict(ids=None), dict(ids=_at(4098)),
                                dict(out=None), dict(out=_at(4104)), dict(addend=_at(4104)), dict(swiglu=1, addend=RES)] +
                         [dict(weights={n: v}) for n in ("w", "w_scale", "a", "b") for v in (None, _at(4104))] +
                         [dict(weights={"w_gscale": None}), dict(weights={"w_gscale": _at(4098)}), dict(weights={"scale": _at(4098)})],
                         ids=str)
@pytest.mark.parametrize("rows", [4, 200])
def test_project_refuses_one_bad_address(lib, rows, kw):
    assert _project(lib, rows, wdtype=1) == OK and _project(lib, rows, wdtype=1, addend=RES, weights={"scale": None}) == OK
    assert _project(lib, rows, wdtype=1, **kw) == BAD and lib.fake_launches() == 0


def test_experts_overlaps(lib):
    """out in x's or the residual's place, row for row, is taken; anything between is refused."""
    rows, row = 40, 512  # bytes of a row
    size = rows * row
    for x, residual, out, stride, status in (
            (X, X, X, 256, OK), (X, None, X, 256, OK), (X, RES, RES, 256, OK), (X, X, X, 264, BAD), (X, RES, X, 264, BAD),
            (X, RES, _at(X.value + row), 256, BAD), (X, RES, _at(X.value - row), 256, BAD), (X, RES, _at(X.value + 16), 256, BAD),
            (X, RES, _at(X.value + size), 256, OK), (X, RES, _at(X.value - size), 256, OK), (X, RES, _at(X.value + size - 16), 256, BAD),
            (X, RES, _at(RES.value + row), 256, BAD), (X, RES, _at(RES.value - size + 16), 256, BAD), (X, RES, _at(RES.value + size), 256, OK),
            # out in a gap between two rows of x
            (X, RES, _at(X.value + 512), 16384, OK), (X, RES, _at(X.value + 32768 - size), 16384, OK),
            (X, RES, _at(X.value + 32784 - size), 16384, BAD), (X, RES, _at(X.value + 32768 + 512), 16384, OK)):
        assert _experts(lib, rows, x=x, residual=residual, out=out, stride=stride) == status, (x, residual, out, stride)
    # one row has no stride; fp32 residuals are twice as wide
    assert _experts(lib, 1, x=X, residual=X, out=X, stride=512) == OK
    assert _experts(lib, rows, residual=_at(OUT.value - 2 * size), residual_dtype=1) == OK
    assert _experts(lib, rows, residual=_at(OUT.value - 2 * size + 16), residual_dtype=1) == BAD


@pytest.mark.parametrize("rows", [4, 200])
def test_project_overlaps(lib, rows):
    size = rows * 512
    for kw, status in ((dict(out=X), BAD), (dict(out=_at(X.value + size)), OK), (dict(out=_at(X.value + size - 16)), BAD),
                       (dict(out=_at(X.value - size)), OK), (dict(out=_at(X.value - size + 16)), BAD),
                       (dict(addend=OUT), OK), (dict(addend=OUT, out_dtype=1), BAD), (dict(addend=_at(OUT.value + 16)), BAD),
                       (dict(addend=_at(OUT.value + size)), OK), (dict(addend=_at(OUT.value + size), out_dtype=1), BAD),
                       (dict(addend=_at(OUT.value - size), out_dtype=1), OK), (dict(out=_at(X.value - size), out_dtype=1), BAD)):
        assert _project(lib, rows, **kw) == status, kw


def _size(rng, low, high, step=1):
    return max(step, min(high, round(low * (high / low) ** rng.random()) // step * step))


@pytest.mark.parametrize("seed", range(8))
def test_every_supported_size_has_a_launch(lib, seed):
    """Sizes over the whole supported range: a tile shape whose stages fit, descriptors by the rules, whole clusters."""
    rng = random.Random(seed)
    for _ in range(200):
        wdtype = rng.randrange(3)
        step = (8, 256, 128)[wdtype]
        hidden, inter = _size(rng, step, 16384, step), _size(rng, step, 16384, step)
        rows = _size(rng, 1, rng.choice((16, 300, 5000, 1 << 24)))
        kw = dict(hidden=hidden, inter=inter, num_experts=_size(rng, 1, 1024), top_k=rng.randint(1, 16), num_shared=rng.randint(0, 4),
                  wdtype=wdtype, residual_dtype=rng.randrange(2), stride=hidden)
        assert _experts(lib, min(rows, 40000), **kw) == OK and lib.fake_bad_maps() == 0, (rows, kw)
        swiglu = rng.randrange(2)
        kw = dict(inner=hidden, outer=inter if wdtype else _size(rng, 2, 16384, 2), swiglu=swiglu, wdtype=wdtype, rank=8 * _size(rng, 1, 32),
                  num_adapters=rng.choice((0, 1, 3, 24, 200, 1024)), out_dtype=0 if swiglu else rng.randrange(2), stride=hidden)
        assert _project(lib, rows, addend=None if swiglu else RES, **kw) == OK and lib.fake_bad_maps() == 0, (rows, kw)
