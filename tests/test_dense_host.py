"""Host side of the dense operators (no GPU): what the checks take and refuse, workspace sizes, what is launched
and what is refused before anything is, over a stand-in for the CUDA runtime."""

import ctypes

import pytest
import torch

from moe_decode_layer_gb300 import _lib, batch
from tests import dense_reference as ref
from tests import fake_cuda

OK, BAD, UNSUPPORTED, CUDA = _lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_CUDA
X, OUT, RES, WS, W, S, GRAD, KEPT, DX, D13, D2 = (ctypes.c_void_p(i << 40) for i in range(1, 12))


def _at(p, offset):
    return ctypes.c_void_p(p.value + offset)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    stub = fake_cuda.STUB
    try:  # fp32 boxes are of 32 values
        fake_cuda.STUB = stub.replace("t == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 ? 2 : 1",
                                      "t == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : t == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 ? 2 : 1")
        assert fake_cuda.STUB != stub
        return fake_cuda.make(str(tmp_path_factory.mktemp("fake")))
    finally:
        fake_cuda.STUB = stub


def _int8_cfg(**kw):
    return _lib.Int8Config(**{**dict(inner=256, outer=128, swiglu=0, x_dtype=_lib.MOE_I8, out_dtype=0), **kw})


def _ff_cfg(**kw):
    return _lib.FfConfig(**{**dict(hidden=256, inter=128, wdtype=0), **kw})


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(inner=16, outer=8), OK), (dict(inner=65536, outer=65536), OK), (dict(swiglu=1, out_dtype=1), OK), (dict(x_dtype=0), OK), (dict(x_dtype=1), OK),
    (dict(inner=0), BAD), (dict(outer=-8), BAD), (dict(inner=24), UNSUPPORTED), (dict(outer=12), UNSUPPORTED), (dict(inner=65552), UNSUPPORTED),
    (dict(outer=65544), UNSUPPORTED), (dict(x_dtype=3), UNSUPPORTED), (dict(out_dtype=2), UNSUPPORTED)])
def test_int8_check(kw, status):
    assert _lib.load().moe_decode_project_int8_check(_int8_cfg(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(hidden=8, inter=8), OK), (dict(hidden=65536, inter=65536), OK), (dict(wdtype=3), OK), (dict(hidden=0), BAD), (dict(inter=-8), BAD),
    (dict(hidden=12), UNSUPPORTED), (dict(inter=65544), UNSUPPORTED), (dict(wdtype=3, inter=24), UNSUPPORTED), (dict(wdtype=1), UNSUPPORTED), (dict(wdtype=2), UNSUPPORTED)])
def test_ff_check(kw, status):
    assert _lib.load().moe_decode_ff_check(_ff_cfg(**kw)) == status


def test_null_configs(lib):
    n = ctypes.c_size_t()
    assert lib.moe_decode_project_int8_check(None) == lib.moe_decode_ff_check(None) == BAD
    assert lib.moe_decode_project_int8_workspace(None, 1, n) == lib.moe_decode_ff_workspace(None, 1, n) == BAD
    assert lib.moe_decode_ff_workspace(_ff_cfg(), 1, None) == lib.moe_decode_ff_workspace(_ff_cfg(), -1, n) == BAD
    assert lib.moe_decode_ff_workspace(_ff_cfg(), (1 << 24) + 1, n) == BAD
    assert lib.moe_decode_ff_backward_workspace(_ff_cfg(wdtype=3), 1, n) == UNSUPPORTED


def test_workspaces_grow_with_rows():
    rows = [*range(0, 40), *range(40, 1200, 13), 5000, 100000]
    for f in (lambda t: batch.feed_forward_workspace(264, 136, t), lambda t: batch.feed_forward_workspace(4096, 8192, t),
              lambda t: batch.feed_forward_workspace(272, 144, t, wdtype="int8"), lambda t: batch.feed_forward_workspace(4096, 8192, t, wdtype="int8"),
              lambda t: batch.feed_forward_backward_workspace(264, 136, t), lambda t: batch.feed_forward_backward_workspace(8, 72, t), lambda t: batch.project_int8_workspace(272, 136, t),
              lambda t: batch.project_int8_workspace(8192, 8192, t), lambda t: batch.project_int8_workspace(272, 136, t, x_dtype=torch.float32)):
        sizes = [f(t) for t in rows]
        assert sizes[0] == 0 and sizes == sorted(sizes)


def _need(lib, f, cfg, rows):
    n = ctypes.c_size_t()
    assert getattr(lib, f)(cfg, rows, n) == OK
    return n.value


def _quantise(lib, rows=4, dtype=0, inner=256, stride=256, x=X, codes=OUT, scale=S):
    lib.fake_reset(-1, -1, 0)
    return lib.moe_decode_quantise(dtype, inner, x, stride, rows, codes, scale, None)


def _project(lib, rows=4, w=W, ws=S, x=X, xs=S, stride=256, addend=None, out=OUT, fail_encode=-1, fail_launch=-1, work=WS, short=0, **kw):
    cfg = _int8_cfg(**kw)
    need = _need(lib, "moe_decode_project_int8_workspace", cfg, rows)
    lib.fake_reset(fail_encode, fail_launch, 0)
    return lib.moe_decode_project_int8(cfg, w, ws, x, xs, stride, addend, out, rows, work, max(0, need - short), None)


def _ff(lib, rows=4, weights=(W, W, S, S), x=X, stride=256, residual=RES, kept=None, out=OUT, fail_encode=-1, fail_launch=-1, work=WS, short=0, **kw):
    cfg = _ff_cfg(**kw)
    need = _need(lib, "moe_decode_ff_workspace", cfg, rows)
    lib.fake_reset(fail_encode, fail_launch, 0)
    return lib.moe_decode_ff(cfg, _lib.FfWeights(*weights), x, stride, residual, kept, out, rows, work, need - short, None)


def _backward(lib, rows=4, weights=(W, W, None, None), grad=GRAD, gstride=256, x=X, stride=256, kept=KEPT, dx=DX, d13=D13, d2=D2, dtype=0,
              accumulate=0, fail_encode=-1, fail_launch=-1, work=WS, short=0, **kw):
    cfg = _ff_cfg(**kw)
    need = _need(lib, "moe_decode_ff_backward_workspace", cfg, rows)
    lib.fake_reset(fail_encode, fail_launch, 0)
    return lib.moe_decode_ff_backward(cfg, _lib.FfWeights(*weights), grad, gstride, x, stride, kept, dx, d13, d2, dtype, accumulate, rows,
                                      work, need - short, None)


def _names(lib):
    found = []
    for i in range(lib.fake_launches()):
        name = lib.fake_name(i).decode()
        found.append(next(n for n in ("quantise", "widen", "zero", "stream", "lanes", "pair_gemm") if n + "_kernel" in name))
    return found


def test_launches(lib):
    assert _quantise(lib) == OK and _names(lib) == ["quantise"]
    assert _project(lib) == OK and _names(lib) == ["stream"]
    assert _project(lib, x_dtype=0) == OK and _names(lib) == ["quantise", "stream"]
    assert _project(lib, rows=100) == OK and _names(lib) == ["widen", "lanes"]
    assert _project(lib, rows=300) == OK and _names(lib) == ["widen", "pair_gemm"]
    assert _project(lib, rows=1000, x_dtype=1) == OK and _names(lib) == ["quantise", "pair_gemm"]
    assert _ff(lib) == OK and _names(lib) == ["stream"] * 2
    assert _ff(lib, rows=100) == OK and _names(lib) == ["lanes"] * 2
    assert _ff(lib, rows=300) == OK and _names(lib) == ["pair_gemm"] * 2
    assert _ff(lib, rows=20, wdtype=3) == OK and _names(lib) == ["quantise", "lanes"] * 2
    assert _ff(lib, rows=1000, wdtype=3) == OK and _names(lib) == ["quantise", "pair_gemm"] * 2
    assert _backward(lib) == OK and _names(lib) == ["pair_gemm"] * 3
    assert _backward(lib, d13=None, d2=None) == OK and _names(lib) == ["pair_gemm"] * 2
    assert _backward(lib, rows=0) == OK and _names(lib) == ["zero"] * 2
    assert _backward(lib, rows=0, dtype=1, accumulate=1) == OK and _names(lib) == []
    for f in (_project, _ff, _quantise):
        assert f(lib, rows=0) == OK and _names(lib) == []


def test_first_launch_is_ordered_behind_the_stream(lib):
    """The call's first kernel starts when what is before it is done: weights may have just been written."""
    for call in (lambda: _project(lib), lambda: _project(lib, rows=100), lambda: _project(lib, rows=1000, x_dtype=0), lambda: _ff(lib), lambda: _ff(lib, rows=100),
                 lambda: _ff(lib, rows=100, wdtype=3), lambda: _backward(lib)):
        assert call() == OK
        assert [lib.fake_pdl(i) for i in range(lib.fake_launches())] == [0] + [1] * (lib.fake_launches() - 1)


@pytest.mark.parametrize("rows", [1, 9, 17, 33, 64, 65, 128, 129, 192, 300, 1000, 20000, 1 << 24])
def test_every_size_can_be_launched(lib, rows):
    """Descriptors by the documented rules, grids in whole clusters and shared memory within the limit, for odd sizes."""
    for hidden, inter in ((8, 8), (256, 128), (2560, 6912), (65536, 8), (8, 65536), (4096, 16384), (65536, 65536)):
        kw = dict(hidden=hidden, inter=inter, stride=hidden)
        assert _ff(lib, rows=rows, x=_at(X, 0), out=ctypes.c_void_p(20 << 44), residual=None, **kw) == OK and lib.fake_bad_maps() == 0
        far = [ctypes.c_void_p(i << 44) for i in range(21, 28)]
        assert _ff(lib, rows=rows, x=far[0], kept=far[1], out=far[2], residual=None, **kw) == OK and lib.fake_bad_maps() == 0
        for dtype, acc in ((0, 0), (1, 0), (1, 1)):
            assert _backward(lib, rows=rows, gstride=hidden, grad=far[0], x=far[1], kept=far[2], dx=far[3], d13=far[4], d2=far[5], dtype=dtype, accumulate=acc, **kw) == OK
            assert lib.fake_bad_maps() == 0
    far = [ctypes.c_void_p(i << 44) for i in range(21, 28)]
    for inner, outer in ((16, 8), (256, 128), (65536, 8), (16, 65536), (4096, 16384)):
        for swiglu in (0, 1):
            for f32 in (0, 1):
                assert _project(lib, rows=rows, inner=inner, outer=outer, stride=inner, x=far[0], out=far[1], swiglu=swiglu, out_dtype=f32) == OK
                assert lib.fake_bad_maps() == 0


@pytest.mark.parametrize("call", [lambda lib, n: _ff(lib, rows=100, kept=KEPT, fail_encode=n), lambda lib, n: _ff(lib, rows=300, kept=KEPT, fail_encode=n), lambda lib, n: _backward(lib, rows=100, fail_encode=n),
                                  lambda lib, n: _project(lib, rows=100, fail_encode=n), lambda lib, n: _project(lib, rows=1000, fail_encode=n, addend=RES),
                                  lambda lib, n: _ff(lib, rows=100, wdtype=3, fail_encode=n), lambda lib, n: _ff(lib, rows=1000, wdtype=3, fail_encode=n)])
def test_without_descriptors_nothing_is_enqueued(lib, call):
    assert call(lib, -1) == OK
    for n in range(lib.fake_encodes()):
        assert call(lib, n) == CUDA and lib.fake_launches() == 0


@pytest.mark.parametrize("call", [lambda lib, n: _ff(lib, rows=4, fail_launch=n), lambda lib, n: _ff(lib, rows=100, fail_launch=n), lambda lib, n: _ff(lib, rows=300, fail_launch=n), lambda lib, n: _backward(lib, rows=100, fail_launch=n),
                                  lambda lib, n: _project(lib, rows=1000, fail_launch=n), lambda lib, n: _project(lib, rows=100, fail_launch=n), lambda lib, n: _ff(lib, rows=4, wdtype=3, fail_launch=n)])
def test_failed_launches_are_reported_once(lib, call):
    assert call(lib, -1) == OK
    for n in range(lib.fake_launches()):
        assert call(lib, n) == CUDA and lib.fake_launches() == n and lib.fake_pending() == 0


def test_quantise_refuses(lib):
    for kw in (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(inner=0), dict(x=None), dict(codes=None), dict(scale=None), dict(x=_at(X, 8)), dict(codes=_at(OUT, 8)),
               dict(scale=_at(S, 2)), dict(stride=248), dict(stride=260), dict(codes=_at(X, 1024)), dict(scale=_at(X, 64)), dict(scale=_at(OUT, 512))):
        assert _quantise(lib, **kw) == BAD and lib.fake_launches() == 0, kw
    for kw in (dict(dtype=2), dict(inner=12), dict(inner=65544, stride=65544)):
        assert _quantise(lib, **kw) == UNSUPPORTED and lib.fake_launches() == 0


@pytest.mark.parametrize("rows", [4, 100, 1000])
def test_project_refuses(lib, rows):
    bad = [dict(w=None), dict(ws=None), dict(x=None), dict(xs=None), dict(out=None), dict(w=_at(W, 8)), dict(ws=_at(S, 8)), dict(x=_at(X, 8)), dict(xs=_at(S, 2)),
           dict(out=_at(OUT, 8)), dict(addend=_at(RES, 8)), dict(work=_at(WS, 8)), dict(stride=240), dict(stride=264), dict(addend=RES, swiglu=1), dict(out=X),
           dict(out=_at(X, 256)), dict(addend=_at(OUT, 256)), dict(addend=OUT, out_dtype=1), dict(xs=_at(OUT, 64))]
    if rows > 32:
        bad += [dict(work=None), dict(short=1)]
    for kw in bad:
        assert _project(lib, rows=rows, **kw) == BAD and lib.fake_launches() == 0, kw
    assert _project(lib, rows=rows, addend=OUT) == OK
    assert lib.moe_decode_project_int8(_int8_cfg(), W, S, X, S, 256, None, OUT, -1, WS, 1 << 30, None) == BAD
    assert _project(lib, rows=4, work=None) == OK  # few rows of codes need none
    assert _project(lib, rows=4, work=None, x_dtype=0) == BAD


@pytest.mark.parametrize("wdtype", [0, 3])
@pytest.mark.parametrize("rows", [4, 100, 1000])
def test_ff_refuses(lib, rows, wdtype):
    kw = dict(rows=rows, wdtype=wdtype)
    n = rows * 512
    bad = [dict(x=None), dict(out=None), dict(work=None), dict(weights=(None, W, S, S)), dict(weights=(W, None, S, S)), dict(x=_at(X, 8)), dict(out=_at(OUT, 2)),
           dict(residual=_at(RES, 8)), dict(work=_at(WS, 8)), dict(weights=(_at(W, 8), W, S, S)), dict(stride=248), dict(stride=260), dict(short=1), dict(out=_at(X, 512)),
           dict(x=OUT, stride=264), dict(residual=_at(OUT, n - 16)), dict(residual=_at(OUT, 16))]
    if wdtype == 3:
        bad += [dict(weights=(W, W, None, S)), dict(weights=(W, W, S, None)), dict(weights=(W, W, _at(S, 4), S))]
    else:
        bad += [dict(kept=_at(KEPT, 8)), dict(kept=OUT), dict(kept=X), dict(kept=RES), dict(kept=_at(OUT, n - 16))]
    for b in bad:
        assert _ff(lib, **{**kw, **b}) == BAD and lib.fake_launches() == 0, b
    assert _ff(lib, **kw, residual=OUT) == OK and _ff(lib, **kw, x=OUT) == OK and _ff(lib, **kw, x=OUT, residual=OUT) == OK
    assert _ff(lib, **kw, residual=None) == OK
    if wdtype == 3:
        assert _ff(lib, **kw, kept=KEPT) == UNSUPPORTED


@pytest.mark.parametrize("rows", [4, 1000])
def test_backward_refuses(lib, rows):
    n = rows * 512
    bad = [dict(grad=None), dict(x=None), dict(kept=None), dict(work=None), dict(dx=None, d13=None, d2=None), dict(weights=(None, W, None, None)), dict(weights=(W, None, None, None)),
           dict(grad=_at(GRAD, 8)), dict(x=_at(X, 8)), dict(kept=_at(KEPT, 8)), dict(dx=_at(DX, 8)), dict(d13=_at(D13, 8)), dict(d2=_at(D2, 8)), dict(work=_at(WS, 8)),
           dict(gstride=248), dict(stride=260), dict(short=1), dict(dx=X), dict(dx=GRAD), dict(dx=KEPT), dict(dx=_at(X, n - 16)), dict(d13=X), dict(d2=GRAD), dict(d13=D2),
           dict(d2=_at(D13, 64)), dict(dx=_at(D13, 64)), dict(d13=W), dict(d2=W)]
    for b in bad:
        assert _backward(lib, rows=rows, **b) == BAD and lib.fake_launches() == 0, b
    assert _backward(lib, rows=rows, accumulate=1) == UNSUPPORTED and _backward(lib, rows=rows, dtype=2) == UNSUPPORTED
    # what a gradient does not need
    assert _backward(lib, rows=rows, dx=None, weights=(None, W, None, None)) == OK
    assert _backward(lib, rows=rows, d13=None, x=None) == OK


def test_binding_refuses():
    """Sizes, types and combinations, on CPU tensors: refused before any device is looked for."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    x, w13, w2, kept = bf(4, 64), bf(32, 64), bf(64, 16), bf(4, 32)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    wq = (torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8))
    for call in (
            lambda: batch.quantise(x.half()), lambda: batch.quantise(x[0]), lambda: batch.quantise(x.t()),
            lambda: batch.project_int8(q, wq), lambda: batch.project_int8((q,), wq), lambda: batch.project_int8((q, s), wq[0]), lambda: batch.project_int8((q, s[:3]), wq),
            lambda: batch.project_int8((q, s), (wq[0][:, :48], wq[1])), lambda: batch.project_int8((q, s), (wq[0].float(), wq[1])), lambda: batch.project_int8((q, s), (wq[0], wq[1][:7])),
            lambda: batch.project_int8((q, s), (wq[0][:7], wq[1][:7]), swiglu=True), lambda: batch.project_int8((q, s), wq, out_dtype=torch.float16),
            lambda: batch.project_int8((q, s), wq, addend=bf(4, 7)),
            lambda: batch.feed_forward(x, w13, w2, wdtype="fp8"), lambda: batch.feed_forward(x, w13, w2, wdtype="int8"), lambda: batch.feed_forward(x, w13[:, :32], w2),
            lambda: batch.feed_forward(x, w13, w2[:, :8]), lambda: batch.feed_forward(x.float(), w13, w2), lambda: batch.feed_forward(x, w13, w2, residual=x.float()),
            lambda: batch.feed_forward(x, w13, w2, gate_up=kept[:3]), lambda: batch.feed_forward(x, w13.float(), w2),
            lambda: batch.feed_forward_backward(x[:3], x, w13, w2, kept), lambda: batch.feed_forward_backward(x, x, w13, w2, kept[:, :16]),
            lambda: batch.feed_forward_backward(x, x, w13, w2, kept, input_grad=False, weight_grad=False), lambda: batch.feed_forward_backward(x, x, w13, w2, kept, accumulate=True),
            lambda: batch.feed_forward_backward(x, x, w13, w2, kept, dw13=bf(32, 64), dw2=bf(64, 16), accumulate=True),
            lambda: batch.feed_forward_backward(x, x, w13, w2, kept, dw13=torch.zeros(32, 64), accumulate=True),
            lambda: batch.feed_forward_backward(x, x, w13, w2, kept, dx=x, input_grad=False), lambda: batch.feed_forward_backward(x, x, w13, w2, kept, dw2=w2, weight_grad=False),
            lambda: batch.feed_forward_backward(x, x, w13, w2, kept, dw13=torch.zeros(32, 64, dtype=torch.float16)),
            lambda: batch.quantise(x), lambda: batch.project_int8((q, s), wq), lambda: batch.feed_forward(x, w13, w2), lambda: batch.feed_forward_backward(x, x, w13, w2, kept)):
        with pytest.raises(ValueError):
            call()


def test_reference_gradients_are_differences():
    """The restatement's gradients against differences of the loss, in 64 bits."""
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w13, w2, grad = n(5, 12), n(16, 12), n(12, 8), n(5, 12)

    def loss(x, w13, w2):
        a, b = (x @ w13.t()).chunk(2, 1)
        return float((((a * torch.sigmoid(a) * b) @ w2.t()) * grad).sum())

    found = [v for v, _ in ref.gradients(grad, x, w13, w2, x @ w13.t())]
    for k, t in enumerate((x, w13, w2)):
        v = n(*t.shape)
        args = [x, w13, w2]
        args[k] = t + 1e-6 * v
        up = loss(*args)
        args[k] = t - 1e-6 * v
        assert abs((up - loss(*args)) / 2e-6 - float((found[k] * v).sum())) < 1e-5 * (1 + abs(up))


def test_reference_codes():
    q, s = ref.codes(torch.tensor([[1.0, 0.5, -0.5, 0.0], [0.0, 0, 0, 0], [float("inf"), 1, 2, 3], [127, 1.5, -2.5, 0.5]]))
    assert q.tolist() == [[127, 64, -64, 0], [0, 0, 0, 0], [0, 0, 0, 0], [127, 2, -2, 0]]  # 63.5, 1.5, 2.5 and 0.5: to the even ones
    assert s[0] == torch.tensor(1.0) / 127 and s[1] == 0 and torch.isnan(s[2])
