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


def test_kinds_of_adamw_states(gq):
    """8-bit states with square codes want their scales like those with linear ones; other values of state_bits are none."""
    def call(**kw):
        t = gq.GQAdamWTensor(**{**dict(p=X, g=T, m=S + 1, v=Y + 3, numel=8), **kw})
        h = gq.GQAdamWHyper(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1)
        return gq.LIB.gq_adamw_step(C.byref(t), 1, C.byref(h), None)

    square = gq.ADAMW_CODES["square"]
    assert square == 0x108 and gq.ADAMW_CODES["linear"] == 8
    assert call(state_bits=square) == 1 and call(state_bits=square, m_scale=O) == 1
    assert call(state_bits=square, m_scale=O, v_scale=O + 2) == 3
    assert call(state_bits=square, m_scale=O, v_scale=O, reserved=1) == 1
    assert call(state_bits=square, m_scale=O, v_scale=O, numel=0) == 0
    for bits in (0, 7, 264 + 8, 0x208, 0x120, -8):
        assert call(state_bits=bits, m_scale=O, v_scale=O) == 1
