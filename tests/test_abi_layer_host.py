"""Host-side checks of the layer products and the AdamW step (no GPU needed, no
kernel launched): layouts of the structs, sizes, and argument errors that come
back before any CUDA call (fake device addresses are never dereferenced)."""
from __future__ import annotations

import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
X, T, S, Y, O = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000


@pytest.fixture(scope="module")
def gq():
    from int6_int8_weight_b200 import build
    build.build()
    from int6_int8_weight_b200 import gq as mod
    return mod


def test_struct_layouts(gq):
    src = """#include "gq.h"
_Static_assert(sizeof(gq_epilogue) == 40, "");
_Static_assert(sizeof(gq_adamw_tensor) == 88, "");
_Static_assert(sizeof(gq_adamw_hyper) == 72, "");
_Static_assert(GQ_ACT_GELU_TANH == 6, "");
int main(void) { return 0; }
"""
    out = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                          "-x", "c", "-"], input=src, text=True, capture_output=True)
    assert out.returncode == 0, out.stderr
    assert (C.sizeof(gq.GQEpilogue), C.sizeof(gq.GQAdamWTensor), C.sizeof(gq.GQAdamWHyper)) == (40, 88, 72)
    assert gq.GQEpilogue.y_dtype.offset == 36 and gq.GQAdamWTensor.weight_decay.offset == 80
    assert gq.GQAdamWHyper.d_grad_scale.offset == 64


def test_tile_bytes(gq):
    b = gq.LIB.gq_tile_bytes
    assert b(1, 1, 6) == 6144 and b(1, 1, 8) == 8192
    assert b(128, 64, 6) == 6144 and b(129, 65, 6) == 4 * 6144
    assert b(0, 5, 6) == 0 and b(5, 0, 8) == 0
    assert b(5, 5, 7) == -1 and b(-1, 5, 6) == -1 and b(1 << 31, 5, 6) == -1


def test_tile_weight_errors(gq):
    f = gq.LIB.gq_tile_weight
    assert f(X, 1, 8, 8, 7, T, None) == 1
    assert f(X, -1, 8, 8, 6, T, None) == 1
    assert f(None, 1, 8, 8, 6, T, None) == 1
    assert f(X, 1, 8, 8, 6, T + 8, None) == 3
    assert f(X, 1, 1 << 31, 8, 6, T, None) == 2
    assert f(X, 1 << 16, 8, 8, 6, T, None) == 2
    for empty in ((0, 8, 8), (1, 0, 8), (1, 8, 0)):
        assert f(None, *empty, 6, None, None) == 0


def _epi(gq, **kw):
    return C.byref(gq.GQEpilogue(**{**dict(y_dtype=1), **kw}))


@pytest.mark.parametrize("grouped", [False, True])
def test_product_errors(gq, grouped):
    def call(epi=None, **kw):
        a = {**dict(x=X, M=4, K=64, ldx=64, off=O, E=2, t=T, s=S, q=6, N=8, y=Y, ldy=8, st=None), **kw}
        e = _epi(gq) if epi is None else _epi(gq, **epi)
        group = (a["off"], a["E"]) if grouped else ()
        fn = gq.LIB.gq_gemm_grouped if grouped else gq.LIB.gq_gemm_epilogue
        return fn(a["x"], a["M"], a["K"], a["ldx"], *group, a["t"], a["s"], a["q"], a["N"], e, a["y"], a["ldy"],
                  a["st"], None)

    for kw, code in ((dict(q=7), 1), (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(ldx=56), 1),
                     (dict(ldy=7), 1), (dict(x=None), 1), (dict(t=None), 1), (dict(s=None), 1), (dict(y=None), 1),
                     (dict(x=X + 8), 3), (dict(ldx=68), 3), (dict(t=T + 8), 3), (dict(s=S + 1), 3), (dict(y=Y + 1), 3),
                     (dict(st=Y + 2), 3), (dict(M=1 << 31), 2), (dict(N=1 << 31, ldy=1 << 31), 2),
                     (dict(ldx=1 << 60), 1)):
        assert call(**kw) == code, kw
    for epi, code in ((dict(act=7), 1), (dict(act=-1), 1), (dict(y_dtype=2), 1), (dict(bias=T, bias_dtype=3), 1),
                      (dict(residual=T, ldr=8, residual_dtype=5), 1), (dict(residual=T, ldr=7), 1),
                      (dict(bias=T + 2), 3), (dict(bias=T + 1, bias_dtype=1), 3), (dict(residual=T + 2, ldr=8), 3)):
        assert call(epi) == code, epi
    assert call(dict(y_dtype=0), y=Y + 2) == 3
    # a residual that is Y itself has Y's type and pitch
    assert call(dict(residual=Y, ldr=8, residual_dtype=0)) == 1 and call(dict(residual=Y, ldr=16, residual_dtype=1)) == 1
    for kw in (dict(M=0, x=None, y=None), dict(N=0, t=None, y=None)):
        assert call(**kw) == 0
    if grouped:
        assert call(off=None) == 1 and call(off=O + 2) == 3 and call(E=-1) == 1 and call(E=65536) == 2
        assert call(E=0, t=None, s=None) == 0


def test_adamw_errors(gq):
    def call(n=1, hyper=None, **kw):
        t = (gq.GQAdamWTensor * 2)()
        for d in t:
            for k, v in {**dict(p=X, g=T, m=S, v=Y, numel=8, state_bits=32), **kw}.items():
                setattr(d, k, v)
        h = gq.GQAdamWHyper(**{**dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1), **(hyper or {})})
        return gq.LIB.gq_adamw_step(t, n, C.byref(h), None)

    nan, inf = float("nan"), float("inf")
    for kw, code in ((dict(p=0), 1), (dict(g=0), 1), (dict(m=0), 1), (dict(v=0), 1), (dict(numel=-1), 1),
                     (dict(p_dtype=2), 1), (dict(g_dtype=-1), 1), (dict(state_bits=16), 1), (dict(reserved=1), 1),
                     (dict(weight_decay=nan), 1), (dict(state_bits=8), 1), (dict(state_bits=8, m_scale=O), 1),
                     (dict(m_scale=O, v_scale=O), 1), (dict(p=X + 2), 3), (dict(g=T + 1, g_dtype=1), 3),
                     (dict(m=S + 2), 3), (dict(p_copy=O + 1), 3), (dict(state_bits=8, m_scale=O, v_scale=O + 2), 3)):
        assert call(**kw) == code, kw
    for hyper, code in ((dict(step=0), 1), (dict(lr=inf), 1), (dict(beta1=1.0), 1), (dict(beta2=-0.1), 1),
                        (dict(beta1=nan), 1), (dict(eps=-1.0), 1), (dict(eps=inf), 1), (dict(d_step=O + 4), 3),
                        (dict(d_lr=O + 2), 3), (dict(d_grad_scale=O + 1), 3)):
        assert call(hyper=hyper) == code, hyper
    assert call(n=-1) == 1
    assert call(n=0) == 0 and call(numel=0, p=0, g=0) == 0
    assert gq.LIB.gq_adamw_step(None, 1, None, None) == 1
