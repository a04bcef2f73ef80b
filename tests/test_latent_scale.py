"""CPU tests of the latent-attention calls' scale: they hand scale * log2(e) to the kernels, so a scale
for which that is past fp32's range is refused like an infinite one, and one just below is not."""
import ctypes

import pytest

import pagedattention_paged_kv_gb300 as pkv
from pagedattention_paged_kv_gb300 import _build

SOME, NULL, F = ctypes.c_void_p(4096), ctypes.c_void_p(0), ctypes.c_float
INVALID = -1


@pytest.fixture(scope="module")
def calls():
    _build.build_library()
    lib = pkv.lib()
    # no sequences: nothing is launched, and a call that is not refused returns 0
    return {
        "absorbed": lambda s: lib.pkv_latent_attention_absorbed(
            SOME, SOME, SOME, SOME, SOME, SOME, 0, 0, 4, 16, 512, 64, 16, 32, F(s), 1, 0, SOME, ctypes.c_size_t(0), NULL),
        "expanded": lambda s: lib.pkv_latent_attention_expanded(
            SOME, SOME, SOME, SOME, SOME, SOME, SOME, SOME, 0, 0, 100, 4, 16, 512, 64, 128, 128, 16, 32, F(s), 1, 0,
            SOME, ctypes.c_size_t(0), NULL)}


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("scale,status", [(2.4e38, INVALID), (3.4e38, INVALID), (float("inf"), INVALID), (0.0, INVALID),
                                          (-1e-30, INVALID), (float("nan"), INVALID),
                                          (2.3e38, 0), (1e-45, 0), (1.0, 0)])
def test_scale(calls, form, scale, status):
    assert calls[form](scale) == status
