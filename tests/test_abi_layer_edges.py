"""Host-side checks of the layer products beside test_abi_layer_host.py (no GPU needed, no kernel launched)."""
from __future__ import annotations

import ctypes as C

import pytest

X, T, S, Y, O = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000


@pytest.fixture(scope="module")
def gq():
    from int6_int8_weight_b200 import build
    build.build()
    from int6_int8_weight_b200 import gq as mod
    return mod


@pytest.mark.parametrize("M,N,E,code", [(0, 8, 2, 3), (4, 0, 2, 3), (4, 8, 0, 3)])
def test_offsets_of_an_empty_product_are_aligned(gq, M, N, E, code):
    """They are read where there is a status to set, so their alignment is checked before anything is launched."""
    e = C.byref(gq.GQEpilogue(y_dtype=1))
    args = (X, M, 64, 64, O + 2, E, T, S, 6, N, e, Y, max(N, 1))
    assert gq.LIB.gq_gemm_grouped(*args, O + 64, None) == code
    assert gq.LIB.gq_gemm_grouped(*args, None, None) == code
    assert gq.LIB.gq_gemm_grouped(*args[:4], O, *args[5:], None, None) == 0
