"""Streams of the weights (no GPU): all blocks of a launch fit the GPU at once, over a stand-in for the CUDA runtime."""

import ctypes

import pytest

from moe_decode_layer_gb300 import _lib
from tests import fake_cuda


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    stub = fake_cuda.STUB
    try:
        fake_cuda.STUB = stub.replace("int fake_bad_maps()", "int fake_smem(int i) { return (int)g_launches[i].smem; }\nint fake_bad_maps()")
        assert fake_cuda.STUB != stub
        return fake_cuda.make(str(tmp_path_factory.mktemp("fake")))
    finally:
        fake_cuda.STUB = stub


def _streams(lib):
    """How many launches were streams; each has at most the blocks that 152 SMs of 228 KB hold, 1 KB a block for the system."""
    found = 0
    for i in range(lib.fake_launches()):
        if "stream_kernel" in lib.fake_name(i).decode():
            found += 1
            assert lib.fake_grid(i) <= 152 * (228 * 1024 // (lib.fake_smem(i) + 1024))
    return found


@pytest.mark.parametrize("rows", [1, 4, 5, 8, 9, 16])
def test_streams_are_resident(lib, rows):
    far = [ctypes.c_void_p(i << 44) for i in range(1, 9)]
    found = 0
    for hidden, inter in ((256, 8192), (8192, 256), (512, 4096), (4096, 16384), (1024, 2048), (64, 64)):
        for wdtype in (0, 3):
            lib.fake_reset(-1, -1, 0)
            assert lib.moe_decode_ff(_lib.FfConfig(hidden, inter, wdtype), _lib.FfWeights(far[0], far[1], far[2], far[2]), far[3], hidden,
                                     None, None, far[4], rows, far[5], 1 << 43, None) == _lib.MOE_OK
            found += _streams(lib)
        for swiglu in (0, 1):
            lib.fake_reset(-1, -1, 0)
            assert lib.moe_decode_project_int8(_lib.Int8Config(hidden, inter, swiglu, _lib.MOE_I8, 0), far[0], far[1], far[2], far[3], hidden,
                                               None, far[4], rows, far[5], 1 << 40, None) == _lib.MOE_OK
            found += _streams(lib)
    assert found >= 12
