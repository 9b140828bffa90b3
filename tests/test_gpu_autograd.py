"""The layer products and the AdamW step beside autograd: what they write in place is known to it."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int6_int8_weight_b200 import gq as mod
    return mod


def _state(bits, n):
    if bits == 32:
        return [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")], None
    return ([torch.zeros(n, dtype=torch.int8, device="cuda")], [torch.zeros(n, dtype=torch.uint8, device="cuda")],
            tuple([torch.zeros(-(-n // 256), device="cuda")] for _ in range(2)))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_graph_kept_over_a_step_is_refused(gq, bits):
    """The backward pass of a graph that saved a weight before the step raises, as with torch's optimizers."""
    w = torch.randn(600, device="cuda", requires_grad=True)
    x = torch.randn(600, device="cuda", requires_grad=True)
    loss = (w * x).sum()                                       # saves w for x's gradient
    m, v, scales = _state(bits, 600)
    copy = torch.zeros(600, dtype=torch.bfloat16, device="cuda")
    written = [w, m[0], v[0], copy] + ([] if scales is None else [scales[0][0], scales[1][0]])
    before, grad = [t._version for t in written], torch.ones(600, device="cuda")
    with torch.no_grad():
        gq.adamw_step([w], [grad], m, v, step=1, lr=1e-3, scales=scales, copies=[copy])
    assert all(t._version > b for t, b in zip(written, before)) and grad._version == 0
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    (w * x).sum().backward()                                   # a graph made after the step is sound
    assert torch.equal(x.grad, w.detach())


@pytest.mark.parametrize("grouped", [False, True])
def test_a_gradient_through_an_exported_layer_is_refused(gq, grouped):
    """The layer products have no backward pass: asking for one raises instead of leaving the path out."""
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn(40, 64, device="cuda", generator=g)
    (o,) = gq.export_pack([gq.Request(w, 6, 1.0)])
    tiles = gq.tile_weight(o.packed, 64, 6)
    off = torch.tensor([0, 6], dtype=torch.int32, device="cuda")

    def call(x, **kw):
        if grouped:
            if kw.get("bias") is not None:
                kw["bias"] = kw["bias"][None]
            return gq.gemm_grouped(x, off, tiles[None], o.scale_f16[None], 6, **kw)
        return gq.gemm_epilogue(x, tiles, o.scale_f16, 6, **kw)

    x = torch.randn(6, 64, device="cuda", generator=g).to(torch.bfloat16)
    want = call(x)
    assert not want.requires_grad
    for kw in (dict(x=x.clone().requires_grad_()), dict(x=x, bias=torch.zeros(40, device="cuda", requires_grad=True)),
               dict(x=x, residual=torch.zeros(6, 40, device="cuda", requires_grad=True)),
               dict(x=x.clone().requires_grad_(), y=torch.empty(6, 40, dtype=torch.bfloat16, device="cuda"))):
        y = call(**kw)
        assert torch.equal(y.detach(), want) and (kw.get("y") is None or y is kw["y"])
        with pytest.raises(RuntimeError, match="no backward pass"):
            (y.float().sum() + sum(t.float().sum() for t in kw.values() if t.is_leaf and t.requires_grad)).backward()
        with torch.no_grad():                                  # serving: no graph
            assert not call(**{**kw, "y": None}).requires_grad
    with pytest.raises(ValueError):
        call(x, y=torch.empty(6, 40, device="cuda", requires_grad=True))


def test_a_result_in_place_of_a_saved_tensor_is_refused(gq):
    """y that a graph has saved, written over."""
    w = torch.randn(40, 64, device="cuda")
    (o,) = gq.export_pack([gq.Request(w, 8, 1.0)])
    y = torch.randn(6, 40, device="cuda")
    a = torch.randn(6, 40, device="cuda", requires_grad=True)
    loss = (a * y).sum()
    gq.gemm_epilogue(torch.ones(6, 64, dtype=torch.bfloat16, device="cuda"), gq.tile_weight(o.packed, 64, 8), o.scale_f16, 8,
                     residual=y, y=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
