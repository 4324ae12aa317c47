"""What moe_decode_rows_status looks at (no GPU), over a stand-in for the CUDA runtime."""

import ctypes

import pytest

from moe_decode_layer_gb300 import _lib
from tests import fake_cuda

P = ctypes.c_void_p(1 << 40)
WORDS = _lib.ROWS_STATUS_BYTES // 4


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    stub = fake_cuda.STUB
    try:  # the workspace that is read back holds zeros, or one word that is set
        fake_cuda.STUB = stub.replace("memset(d, 0, n);", "memset(d, 0, n); if (g_word >= 0) ((int*)d)[g_word] = 1;") \
            .replace("int g_capturing = 0;", "int g_capturing = 0, g_word = -1;") \
            .replace("int fake_bad_maps()", "void fake_word(int i) { g_word = i; }\nint fake_bad_maps()")
        assert fake_cuda.STUB.count("g_word") == 4
        return fake_cuda.make(str(tmp_path_factory.mktemp("fake")))
    finally:
        fake_cuda.STUB = stub


def test_every_word_is_looked_at(lib):
    """A product with the weights on the lanes has up to 1024 CTAs, each with a word: more than the GPU has SMs."""
    assert lib.moe_decode_rows_status(P, None) == _lib.MOE_OK
    for i in range(WORDS):
        lib.fake_word(i)
        assert lib.moe_decode_rows_status(P, None) == _lib.MOE_ERR_DEVICE_TIMEOUT, i
    lib.fake_word(-1)
    assert lib.moe_decode_rows_status(P, None) == _lib.MOE_OK


def test_every_launch_has_a_word_for_each_block(lib):
    """Grids of the kernels that wait, for the widest matrices."""
    far = [ctypes.c_void_p(i << 44) for i in range(1, 9)]
    grids = set()
    for rows in (9, 33, 100, 128, 192, 300, 5000):
        for hidden, inter in ((65536, 65536), (16, 65536), (65536, 16), (4096, 14336)):
            for wdtype in (0, 3):
                lib.fake_reset(-1, -1, 0)
                assert lib.moe_decode_ff(_lib.FfConfig(hidden, inter, wdtype), _lib.FfWeights(far[0], far[1], far[2], far[2]), far[3], hidden,
                                         None, None, far[4], rows, far[5], 1 << 43, None) == _lib.MOE_OK
                grids |= {lib.fake_grid(i) for i in range(lib.fake_launches())
                          if "lanes_kernel" in lib.fake_name(i).decode() or "pair_gemm_kernel" in lib.fake_name(i).decode()}
    assert max(grids) == WORDS  # (the widest gate/up product, 64 columns a CTA)
