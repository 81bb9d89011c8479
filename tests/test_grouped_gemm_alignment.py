"""Leading dimensions of float32 outputs (CPU only: refused before any device work).  The header asks
multiples of 16 bytes of every matrix, float32 ones too."""
import ctypes as C

import pytest

from expert_cached_sparse_b200 import _lib as L

P = C.c_void_p(0x100000)      # aligned dummy address, never read


def call(name, ldo, out=P, off=P):
    if name == "fwd":
        return L.lib.moe_grouped_gemm(4, 64, 64, P, 64, P, off, 8, out, ldo, L.DT_F32, None)
    if name == "dx":
        return L.lib.moe_grouped_gemm_dx(4, 64, 64, P, 64, P, off, 8, out, ldo, L.DT_F32, None)
    return L.lib.moe_grouped_gemm_fp8(4, 64, 64, P, 64, P, P, P, off, 8, out, ldo, L.DT_F32, None)


@pytest.mark.parametrize("name", ["fwd", "dx", "fp8"])
def test_float32_outputs(name):
    for ldo in (65, 66, 67, 70, 60):
        assert call(name, ldo) == L.MOE_ERR_INVALID_ARG
    assert call(name, 64, out=C.c_void_p(0x100008)) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["fwd", "dx", "fp8", "dw"])
def test_offsets_are_whole_words(name):
    odd = C.c_void_p(0x100002)
    if name == "dw":
        assert L.lib.moe_grouped_gemm_dw(4, 64, 64, P, 64, P, 64, odd, 8, P, L.DT_F32, 0, None) == L.MOE_ERR_INVALID_ARG
    else:
        assert call(name, 64, off=odd) == L.MOE_ERR_INVALID_ARG
