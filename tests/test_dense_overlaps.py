"""Results in the weights' place are refused before anything is enqueued (no GPU), over a stand-in for the CUDA runtime."""

import ctypes

import pytest

from moe_decode_layer_gb300 import _lib
from tests import fake_cuda

OK, BAD = _lib.MOE_OK, _lib.MOE_ERR_INVALID_ARG
X, OUT, KEPT, WS, W, W2, S, S2, XS = (i << 40 for i in range(1, 10))
HIDDEN, INTER = 256, 128


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return fake_cuda.make(str(tmp_path_factory.mktemp("fake")))


def _spots(start, size, own):
    """Places of `own` bytes that share a byte with [start, start + size), at both ends and inside, and their neighbours that do not."""
    return (start, start + size - 16, start - own + 16), (start + size, start - own)


@pytest.mark.parametrize("rows", [4, 40, 1000])
@pytest.mark.parametrize("swiglu", [0, 1])
@pytest.mark.parametrize("f32", [0, 1])
def test_project_int8(lib, rows, swiglu, f32):
    cfg = _lib.Int8Config(HIDDEN, INTER, swiglu, _lib.MOE_I8, f32)
    outer = INTER * (1 + swiglu)

    def call(out):
        lib.fake_reset(-1, -1, 0)
        st = lib.moe_decode_project_int8(cfg, W, S, X, XS, HIDDEN, None, out, rows, WS, 1 << 39, None)
        assert st == OK or lib.fake_launches() == 0
        return st
    for start, size in ((W, outer * HIDDEN), (S, outer * 4)):
        bad, good = _spots(start, size, rows * INTER * (4 if f32 else 2))
        assert [call(o) for o in bad] == [BAD] * 3 and [call(o) for o in good] == [OK] * 2


@pytest.mark.parametrize("rows", [4, 40, 1000])
@pytest.mark.parametrize("wdtype", [0, 3])
def test_feed_forward(lib, rows, wdtype):
    size = 1 if wdtype else 2

    def call(out=OUT, kept=None):
        lib.fake_reset(-1, -1, 0)
        st = lib.moe_decode_ff(_lib.FfConfig(HIDDEN, INTER, wdtype), _lib.FfWeights(W, W2, S, S2), X, HIDDEN, None, kept, out, rows, WS, 1 << 39, None)
        assert st == OK or lib.fake_launches() == 0
        return st
    inputs = [(W, 2 * INTER * HIDDEN * size), (W2, INTER * HIDDEN * size)] + ([(S, 2 * INTER * 4), (S2, HIDDEN * 4)] if wdtype else [])
    for start, n in inputs:
        bad, good = _spots(start, n, rows * HIDDEN * 2)
        assert [call(out=o) for o in bad] == [BAD] * 3 and [call(out=o) for o in good] == [OK] * 2
        if not wdtype:
            bad, good = _spots(start, n, rows * INTER * 4)
            assert [call(kept=k) for k in bad] == [BAD] * 3 and [call(kept=k) for k in good] == [OK] * 2
    if not wdtype:  # scales are not read
        assert call(out=S) == OK
