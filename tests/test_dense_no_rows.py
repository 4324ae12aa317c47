"""Calls without rows (no GPU), over a stand-in for the CUDA runtime: nothing is refused for what no row needs."""

import ctypes

import pytest

from moe_decode_layer_gb300 import _lib
from tests import fake_cuda

P = ctypes.c_void_p(1 << 40)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return fake_cuda.make(str(tmp_path_factory.mktemp("fake")))


def test_backward_of_the_input_alone(lib):
    """A tensor of no rows has a null address."""
    cfg, w = _lib.FfConfig(256, 128, 0), _lib.FfWeights(P, P, None, None)
    lib.fake_reset(-1, -1, 0)
    assert lib.moe_decode_ff_backward(cfg, w, None, 256, None, 256, None, None, None, None, 0, 0, 0, None, 0, None) == _lib.MOE_OK
    assert lib.fake_launches() == 0
    assert lib.moe_decode_ff_backward(cfg, w, P, 256, P, 256, P, None, None, None, 0, 0, 1, P, 1 << 30, None) == _lib.MOE_ERR_INVALID_ARG


def test_other_calls(lib):
    lib.fake_reset(-1, -1, 0)
    assert lib.moe_decode_quantise(0, 256, None, 256, 0, None, None, None) == _lib.MOE_OK
    assert lib.moe_decode_project_int8(_lib.Int8Config(256, 128, 0, _lib.MOE_I8, 0), None, None, None, None, 256, None, None, 0, None, 0, None) == _lib.MOE_OK
    assert lib.moe_decode_ff(_lib.FfConfig(256, 128, 0), None, None, 256, None, None, None, 0, None, 0, None) == _lib.MOE_OK
    assert lib.fake_launches() == 0
