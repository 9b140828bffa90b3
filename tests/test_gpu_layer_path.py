"""The operators together, as a quantization-aware training run and its exported
model use them: fake-quant weights in the forward pass, the straight-through
gradient, one AdamW step (32-bit and 8-bit states), the export, the tile layout,
and the exported two-layer block and a mixture of experts run from the codes.

Gradients are checked against the formula and against differences; the exported
block against binary64 on the weights that gq.dequant gives.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_adamw import reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int6_int8_weight_b200 import gq as mod
    return mod


def _block(gq, x, up, down):
    """relu(x up_hat^T)^2 down_hat^T + x on fake-quant weights."""
    h = torch.relu(x @ gq.FakeQuantSTE.apply(up, 6).t()) ** 2
    return h @ gq.FakeQuantSTE.apply(down, 6).t() + x


@pytest.mark.parametrize("bits", [32, 8])
def test_train_export_run(gq, bits):
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    d, hid, tokens = 192, 528, 77
    up, down = (rand(hid, d) * d ** -0.5).requires_grad_(), (rand(d, hid) * hid ** -0.5 * 0.3).requires_grad_()
    x, target = rand(tokens, d), rand(tokens, d)

    params = [up, down]
    if bits == 32:
        m, v, scales = [torch.zeros_like(p) for p in params], [torch.zeros_like(p) for p in params], None
    else:
        m = [torch.zeros(p.shape, dtype=torch.int8, device="cuda") for p in params]
        v = [torch.zeros(p.shape, dtype=torch.uint8, device="cuda") for p in params]
        scales = tuple([torch.zeros(-(-p.numel() // 256), device="cuda") for p in params] for _ in range(2))
    copies = [torch.empty(p.shape, dtype=torch.bfloat16, device="cuda") for p in params]
    for step in (1, 2, 3):
        loss = ((_block(gq, x, up, down) - target) ** 2).mean()
        up.grad = down.grad = None
        loss.backward()
        if step == 1:
            # the straight-through gradient is that of the loss in the fake-quant weights: by the formula ...
            (fu,), (fd,) = (gq.fakequant([gq.Request(p.detach(), 6, 1.0)]) for p in params)
            u, w = fu.dq.double(), fd.dq.double()
            x64 = x.double()
            a = x64 @ u.t()
            r = torch.relu(a)
            dy = 2 * ((r ** 2) @ w.t() + x64 - target.double()) / target.numel()
            want_w = dy.t() @ r ** 2
            want_u = (dy @ w * 2 * r).t() @ x64
            for got, want in ((up.grad, want_u), (down.grad, want_w)):
                assert (got.double() - want).norm() <= 1e-5 * want.norm()
            # ... and by differences along one direction
            t = torch.randn(u.shape, device="cuda", generator=g, dtype=torch.float64)
            f = lambda e: (((torch.relu(x64 @ (u + e * t).t()) ** 2) @ w.t() + x64 - target.double()) ** 2).mean()  # noqa: E731
            assert abs(float((f(1e-6) - f(-1e-6)) / 2e-6 - (want_u * t).sum())) <= 1e-5 * float(want_u.norm() * t.norm())
        flat = lambda t: None if t is None else t.detach().reshape(-1).cpu().numpy().copy()  # noqa: E731
        ms, vs = scales or ([None] * 2,) * 2
        before = [tuple(map(flat, t)) for t in zip(params, [up.grad, down.grad], m, v, ms, vs)]
        with torch.no_grad():
            gq.adamw_step(params, [up.grad, down.grad], m, v, step=step, lr=1e-3, betas=(0.9, 0.95), weight_decay=0.1,
                          scales=scales, copies=copies, seed=17)
        for i, (p, c) in enumerate(zip(params, copies)):
            want, wm, wv, _, _ = reference(*before[i], step, 17, i, 0.1, 1e-3, 0.9, 0.95, 1e-8)
            assert np.array_equal(flat(p), want) and np.array_equal(flat(m[i]), wm) and np.array_equal(flat(v[i]), wv)
            assert torch.equal(c, p.detach().to(torch.bfloat16))

    # export, lay out, run from the codes
    exported = gq.export_pack([gq.Request(p.detach(), 6, 0.9999) for p in params])
    tiles = [gq.tile_weight(o.packed, p.shape[1], 6) for o, p in zip(exported, params)]
    xb = x.to(torch.bfloat16)
    h = gq.gemm_epilogue(xb, tiles[0], exported[0].scale_f16, 6, act="relu2")
    y = gq.gemm_epilogue(h, tiles[1], exported[1].scale_f16, 6, residual=xb, out_dtype=torch.float32)
    wu, wd = (gq.dequant(o.packed, o.scale_f16, 6, *p.shape).double() for o, p in zip(exported, params))
    want_h = torch.relu(xb.double() @ wu.t()) ** 2
    assert (h.double() - want_h).abs().max() <= 2.0 ** -8 * want_h.max()
    want_y = h.double() @ wd.t() + xb.double()
    assert ((y.double() - want_y).abs() <= 2.0 ** -20 * (h.double().abs() @ wd.abs().t() + want_y.abs())).all()

    # the same as a mixture: three experts (the block's own first layer, scaled), rows sorted by expert
    E = 3
    etiles = torch.stack([tiles[0]] * E)
    escale = torch.stack([exported[0].scale_f16 * f for f in (1.0, 0.5, 2.0)])
    off = torch.tensor([0, 30, 30, tokens], dtype=torch.int32, device="cuda")
    ye = gq.gemm_grouped(xb, off, etiles, escale, 6, act="relu2")
    assert torch.equal(ye[:30], gq.gemm_epilogue(xb[:30], tiles[0], escale[0], 6, act="relu2"))
    want = torch.relu(xb[30:].double() @ (2 * wu).t()) ** 2
    assert (ye[30:].double() - want).abs().max() <= 2.0 ** -8 * want.max()


def test_decode_step_captured(gq):
    """A decode step of a small stack captured once and replayed on new tokens gives the eager results."""
    rng = np.random.default_rng(6)
    layers = []
    for n, k in ((528, 192), (192, 528)) * 2:
        w = torch.from_numpy((rng.standard_normal((n, k)) * k ** -0.5).astype(np.float32)).cuda()
        (o,) = gq.export_pack([gq.Request(w, 6, 0.9999)])
        layers.append((gq.tile_weight(o.packed, k, 6), o.scale_f16))

    def step(x):
        for a, b in zip(layers[::2], layers[1::2]):
            h = gq.gemm_epilogue(x, *a, 6, act="leaky_relu2")
            x = gq.gemm_epilogue(h, *b, 6, residual=x)
        return x

    x = torch.zeros((1, 192), dtype=torch.bfloat16, device="cuda")
    step(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(x)
    for seed in range(4):
        x.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((1, 192)).astype(np.float32)))
        want = step(x.clone())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
